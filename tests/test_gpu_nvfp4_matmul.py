"""Products of two 4-bit matrices against the 64-bit product of their exact values: row counts on every side of the kernels'
tiles, odd vocabularies, widths that end inside a record, scales of rows, strided outputs."""
import pytest
import torch

import w4_util as u

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
LEAST = {F32: 2.0 ** -150, BF: 2.0 ** -134, HF: 2.0 ** -25}
HALF = {F32: 2.0 ** -24, BF: 2.0 ** -8, HF: 2.0 ** -11}


@pytest.fixture(scope="module")
def vh():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import verify_head_gb300 as vh
    vh.build()
    return vh


def matrix(seed, n, H, lo=40, hi=80):
    """Random codes and block scales (2^-2 to 8 and a few subnormal and zero ones) -> (codes, scales, values)."""
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(0, 256, (n, H // 2), generator=g, dtype=torch.uint8)
    s = torch.randint(lo, hi, (n, H // 16), generator=g, dtype=torch.uint8)
    s.view(-1)[::37] = 3
    s.view(-1)[5::41] = 0
    return q.cuda(), s.cuda(), torch.from_numpy(u.values64(q, s)).cuda()


def check(vh, T, V, H, dtype=F32, gx=0.013, gw=0.7, out=None, seed=0):
    xq, xs, xv = matrix(seed, T, H)
    wq, ws, wv = matrix(seed + 1, V, H)
    xt = torch.from_numpy(u.tile(xq, xs, 0x7F)).cuda()  # lines past T: scales that are no numbers
    wt = vh.nvfp4_tile(wq, ws)
    got = vh.nvfp4_matmul(xt, gx, wt, gw, T, V, H, out=out, dtype=dtype if out is None else None)
    col = lambda g: g.double()[:, None] if torch.is_tensor(g) else float(torch.tensor(g))  # noqa: E731
    row = lambda g: g.double()[None] if torch.is_tensor(g) else float(torch.tensor(g))  # noqa: E731
    want = xv @ wv.t() * col(gx) * row(gw)
    # A number below the type's normal ones is off by half its smallest: 2^-25 in fp16, whose normal ones begin at 2^-14.
    # Sums: one rounding per MMA of 64 elements and at most 64 within one (truncated: a whole unit, 2^-23), of at most the sum
    # of the magnitudes; two products and the rounding to the type follow.
    size = xv.abs() @ wv.abs().t() * abs(col(gx)) * abs(row(gw))
    tol = (H / 64 + 64) * 2.0 ** -23 * size + (2 * 2.0 ** -24 + HALF[got.dtype]) * want.abs() + LEAST[got.dtype]
    assert got.shape == (T, V)
    off = (got.double() - want).abs() - tol
    assert float(off.max()) <= 0, float(off.max())


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 31, 32, 33, 48, 64, 65, 127, 128, 129, 200, 255, 256, 257, 300, 511, 513])
def test_row_counts(vh, T):
    check(vh, T, 391, 576, F32)


@pytest.mark.parametrize("H", [16, 32, 48, 64, 80, 240, 256, 272, 320, 512, 1008, 2048, 2560, 4096])
@pytest.mark.parametrize("T", [3, 130, 260])
def test_widths(vh, T, H):
    check(vh, T, 257, H, BF)


@pytest.mark.parametrize("V", [1, 2, 31, 127, 128, 129, 255, 256, 257, 4097, 40001])
@pytest.mark.parametrize("T", [1, 20, 100, 290])
def test_vocabularies(vh, V, T):
    check(vh, T, V, 320, HF if V < 300 else F32, gx=1e-4)


@pytest.mark.parametrize("T,V,H", [(1, 8192, 8192), (4, 65536, 2048), (37, 4096, 65536), (1024, 2048, 1024), (2000, 5000, 512),
                                   (256, 40001, 2048)])
def test_larger(vh, T, V, H):
    check(vh, T, V, H, BF)


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("T", [5, 150])
def test_scales_and_strides(vh, dtype, T):
    V, H = 203, 336
    g = torch.Generator().manual_seed(3)
    gx, gw = torch.rand(T, generator=g).cuda() * 0.01, torch.rand(V, generator=g).cuda() - 0.5
    for a, b in ((gx, gw), (0.01, gw), (gx, -2.0), (-0.01, 1.0)):
        check(vh, T, V, H, dtype, a, b)
    pad = torch.full((T + 1, V + 13), 9.0, dtype=dtype, device="cuda")
    for lo in (0, 1, 8):
        pad.fill_(9.0)
        check(vh, T, V, H, gx=gx, gw=gw, out=pad[:T, lo:lo + V])
        rest = pad.clone()
        rest[:T, lo:lo + V] = 9.0
        assert bool((rest == 9.0).all())  # nothing outside is written


def test_no_numbers(vh):
    """A scale that is no number makes its row, or its column, and nothing else."""
    for T in (6, 140, 300):
        xq, xs, _ = matrix(1, T, 320)
        wq, ws, _ = matrix(2, 300, 320)
        xs[3, 17], ws[277, 0] = 0x7F, 0x7F
        gx = torch.ones(T, device="cuda")
        gx[4] = float("nan")
        y = vh.nvfp4_matmul(vh.nvfp4_tile(xq, xs), gx, vh.nvfp4_tile(wq, ws), 1.0, T, 300, 320, dtype=F32)
        want = torch.zeros(T, 300, dtype=torch.bool, device="cuda")
        want[3], want[4], want[:, 277] = True, True, True
        assert torch.equal(torch.isnan(y), want)


def test_same_bits_again(vh):
    """Results do not depend on the order in which CTAs run."""
    for T, V, H in ((1, 1000, 8192), (7, 4097, 4096), (300, 2049, 1024)):
        x, w = (vh.nvfp4_tile(*matrix(i, n, H)[:2]) for i, n in ((1, T), (2, V)))
        a = vh.nvfp4_matmul(x, 0.1, w, 0.1, T, V, H, dtype=F32)
        for _ in range(5):
            assert torch.equal(a, vh.nvfp4_matmul(x, 0.1, w, 0.1, T, V, H, dtype=F32))


def test_quantized_on_the_way_and_replayed(vh):
    """Quantise, multiply, again on new rows, from a captured graph; another stream."""
    T, V, H = 9, 777, 1040
    wq, ws, wv = matrix(4, V, H)
    wt = vh.nvfp4_tile(wq, ws)
    x = torch.zeros(T, H, dtype=BF, device="cuda")
    tiles = torch.empty(vh.vh_nvfp4_tiles_bytes(T, H), dtype=torch.uint8, device="cuda")
    rs, y = torch.empty(T, device="cuda"), torch.empty(T, V, device="cuda")

    def step(stream=None):
        vh.nvfp4_quantize_tiles(x, tiles=tiles, row_scales=rs, stream=stream)
        vh.nvfp4_matmul(tiles, rs, wt, 0.5, T, V, H, out=y, stream=stream)

    def right():
        v = vh.nvfp4_dequantize(*vh.nvfp4_quantize(x)[:2], 1.0, dtype=F32).double() * rs.double()[:, None]
        want = v @ wv.t() * 0.5
        size = v.abs() @ wv.abs().t() * 0.5
        assert float(((y.double() - want).abs() - (H / 64 + 70) * 2.0 ** -23 * size).max()) <= 0

    for seed in range(2):
        x.copy_(torch.randn(T, H, generator=torch.Generator().manual_seed(seed)))
        step()
        right()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y.zero_()
    step(side)
    torch.cuda.current_stream().wait_stream(side)
    right()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(3, 6):
        x.copy_(torch.randn(T, H, generator=torch.Generator().manual_seed(seed)) * seed)
        graph.replay()
        right()


def test_refusals(vh):
    q, s, _ = matrix(0, 5, 64)
    t = vh.nvfp4_tile(q, s)
    y = torch.zeros(5, 5, dtype=BF, device="cuda")
    for bad in (lambda: vh.nvfp4_matmul(t, 1.0, t, 1.0, 129, 5, 64), lambda: vh.nvfp4_matmul(t, 1.0, t, 1.0, 5, 129, 64),
                lambda: vh.nvfp4_matmul(t, 1.0, t, 1.0, 5, 5, 512), lambda: vh.nvfp4_matmul(t.cpu(), 1.0, t, 1.0, 5, 5, 64),
                lambda: vh.nvfp4_matmul(t, 1.0, t.cpu(), 1.0, 5, 5, 64), lambda: vh.nvfp4_matmul(t, 1.0, t, 1.0, 5, 5, 64, out=y[:4]),
                lambda: vh.nvfp4_matmul(t, 1.0, t, 1.0, 5, 5, 64, out=y.t()),
                lambda: vh.nvfp4_matmul(t, y[0], t, 1.0, 5, 5, 64), lambda: vh.nvfp4_matmul(t, 1.0, t, torch.zeros(4, device="cuda"), 5, 5, 64),
                lambda: vh.nvfp4_matmul(t, 1.0, t, 1.0, 5, 5, 64, out=y.int()), lambda: vh.nvfp4_matmul(t, 1.0, t, 1.0, 5, 2 ** 40, 64)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: vh.nvfp4_matmul(t, float("nan"), t, 1.0, 5, 5, 64), lambda: vh.nvfp4_matmul(t, 1.0, t, 1.0, 5, 5, 72)):
        with pytest.raises((vh.VHError, ValueError)):
            bad()
