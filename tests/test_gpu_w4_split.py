"""Products whose tiles are shared by a cluster: its CTAs add up in one another's shared memory, whenever each of them got to run.
Other work on the GPU, so that they do not begin together on idle SMs; results are those of a quiet GPU, bit by bit."""
import pytest
import torch

from test_gpu_nvfp4_matmul import check, matrix

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def vh():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import verify_head_gb300 as vh
    vh.build()
    return vh


# clusters of 8, of 4, of 2, of 8 with one tile, with as many as there are SMs for
SHAPES = [(3, 500, 4096), (32, 3000, 4096), (17, 8192, 1024), (1, 100, 65536), (5, 2432, 4096)]


@pytest.mark.parametrize("T,V,H", SHAPES)
def test_values(vh, T, V, H):
    check(vh, T, V, H, F32)
    check(vh, T, V, H, BF)


@pytest.mark.parametrize("T,V,H", SHAPES)
def test_on_a_busy_gpu(vh, T, V, H):
    x, w = (vh.nvfp4_tile(*matrix(i, n, H)[:2]) for i, n in ((1, T), (2, V)))
    want = vh.nvfp4_matmul(x, 0.1, w, 0.1, T, V, H, dtype=F32)
    torch.cuda.synchronize()
    side, main = torch.cuda.Stream(), torch.cuda.Stream()
    a = torch.randn(4096, 4096, device="cuda", dtype=BF)
    b = torch.empty_like(a)
    ys = [torch.empty_like(want) for _ in range(50)]
    torch.cuda.synchronize()
    for i, y in enumerate(ys):
        with torch.cuda.stream(side):  # blocks of another kernel come and go on the SMs
            if i % 5 == 0:
                torch.mm(a, a, out=b)
            b.mul_(0.5)
        vh.nvfp4_matmul(x, 0.1, w, 0.1, T, V, H, out=y, stream=main)
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in ys)


@pytest.mark.parametrize("T,V,H", SHAPES)
def test_table_written_by_the_call_before(vh, T, V, H):
    x = vh.nvfp4_tile(*matrix(1, T, H)[:2])
    heads = [matrix(i, V, H)[:2] for i in (2, 3)]
    ready = [vh.nvfp4_tile(*h) for h in heads]
    want = [vh.nvfp4_matmul(x, 0.1, t, 0.1, T, V, H, dtype=F32) for t in ready]
    table, ys = torch.zeros_like(ready[0]), [torch.empty_like(y) for y in want]
    for _ in range(40):
        for y in ys:
            y.zero_()
        torch.cuda.synchronize()
        for (c, s), y in zip(heads, ys):
            vh.nvfp4_tile(c, s, tiles=table)
            vh.nvfp4_matmul(x, 0.1, table, 0.1, T, V, H, out=y)
        assert all(torch.equal(a, b) for a, b in zip(ys, want))
