"""The product of 4-bit matrices right after the calls that write its operands, with no pause: it reads nothing before they have
ended, in each of its kernels, on a busy GPU, and from a captured graph."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def vh():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import verify_head_gb300 as vh
    vh.build()
    return vh


# up to 32 rows, up to 128, more, pairs
SHAPES = [(8, 30000, 1024), (100, 30000, 512), (260, 40000, 512), (1024, 8192, 2048)]
WRITERS = ["tile", "quantize", "quantize, then log probabilities"]


@pytest.mark.parametrize("writer", WRITERS)
@pytest.mark.parametrize("T,V,H", SHAPES)
def test_table_written_by_the_call_before(vh, T, V, H, writer):
    g = torch.Generator("cuda").manual_seed(T)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)  # noqa: E731
    x, W = randn(T, H), [randn(V, H) for _ in range(3)]
    xt, xs = torch.empty(vh.vh_nvfp4_tiles_bytes(T, H), dtype=torch.uint8, device="cuda"), torch.empty(T, device="cuda")
    wt, ws = torch.empty(vh.vh_nvfp4_tiles_bytes(V, H), dtype=torch.uint8, device="cuda"), torch.empty(V, device="cuda")
    codes = [vh.nvfp4_quantize(w) for w in W]
    big, tok, lws = randn(8, 50000), torch.zeros(8, dtype=torch.int32, device="cuda"), vh.logits_logprobs_workspace(8, 50000, 0)
    outs = dict(zip(("logprob", "entropy", "lse", "top_ids", "top_logprobs"), vh.logits_logprobs(big, tok, 0, ws=lws)))
    ys = [torch.empty(T, V, device="cuda") for _ in W]

    def run(pause):
        """The table of each head is written over the one before."""
        for w, (c, s, r), y in zip(W, codes, ys):
            if writer == "tile":
                vh.nvfp4_quantize_tiles(x, tiles=xt, row_scales=xs)
                pause()
                vh.nvfp4_tile(c, s, tiles=wt)
            else:
                vh.nvfp4_quantize_tiles(w, tiles=wt, row_scales=ws)
                pause()
                vh.nvfp4_quantize_tiles(x, tiles=xt, row_scales=xs)
                if writer != "quantize":  # a call that lets the next one start early
                    pause()
                    vh.logits_logprobs(big, tok, 0, ws=lws, **outs)
            pause()
            vh.nvfp4_matmul(xt, xs, wt, r if writer == "tile" else ws, T, V, H, out=y)
            pause()

    run(torch.cuda.synchronize)
    want = [y.clone() for y in ys]
    assert not torch.equal(want[0], want[1]) and not torch.equal(want[1], want[2])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(lambda: None)
    for i in range(40):
        for y in ys:
            y.fill_(7.0)
        wt.fill_(i)
        torch.cuda.synchronize()
        if i % 2:
            run(lambda: None)
        else:
            graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(ys, want))
