"""What one call writes can be the next call's weight table, hidden rows or list of row ids, with nothing in between: the
head kernels begin to read their table before the previous kernel has finished, so calls that write rows or ids must not
let them start early."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module")
def vh():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import verify_head_gb300 as vh
    vh.build()
    return vh


def randn(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(BF)


def readers(vh, R, H, V):
    """Calls that read a table [V,H]: each takes the table and returns its results."""
    g = torch.Generator("cuda").manual_seed(R + H)
    x = randn(g, R, H)
    cand = torch.arange(V, device="cuda", dtype=torch.int32)
    tokens = torch.arange(R, device="cuda", dtype=torch.int32)
    one = torch.zeros(R // 2, 1, dtype=torch.int32, device="cuda")
    ws, lws = vh.workspace(R), vh.head_logprobs_workspace(R, V, 4)
    calls = {"head_logprobs": lambda W: vh.head_logprobs(x, W, tokens, 4, ws=lws),
             "draft": lambda W: vh.mtp_draft_head_argmax(x, W, cand, ws=ws),
             "gather": lambda W: vh.mtp_draft_head_argmax_gather(x, W, cand, ws=ws)}
    for name, path in (("verify", vh.VH_PATH_AUTO), ("verify, tensor cores", vh.VH_PATH_TENSOR)):
        calls[name] = lambda W, path=path: vh.spec_verify_greedy(x, W, one, R // 2, 1, ws=ws, path=path)
    return calls


WRITERS = ["norm", "norm, then norm", "norm, then log probabilities", "norm grad", "norm grad, no dweight", "logits grad"]


@pytest.mark.parametrize("writer", WRITERS)
@pytest.mark.parametrize("R", [4, 200])
def test_table_written_by_the_call_before(vh, writer, R):
    H, V = 256, 3000
    g = torch.Generator("cuda").manual_seed(3)
    E, w, h, s = randn(g, V, H), randn(g, H), randn(g, V, H), randn(g, 64, H)
    W, y, big = torch.empty_like(E), torch.empty_like(s), randn(g, 8, 50000)
    dw, gws = torch.empty(H, device="cuda"), vh.add_rmsnorm_grad_workspace(V, H)
    lse = torch.full((V,), 6.0, device="cuda")
    tokens = torch.zeros(V, dtype=torch.int32, device="cuda")
    lws = vh.logits_logprobs_workspace(8, 50000, 0)
    o = vh.logits_logprobs(big, tokens[:8], 0, ws=lws)
    outs = dict(zip(("logprob", "entropy", "lse", "top_ids", "top_logprobs"), o))

    def write(table):
        if writer.startswith("norm grad"):
            given = "no dweight" not in writer
            vh.add_rmsnorm_grad(E, h, w if given else None, dx=table, dweight=dw if given else None, ws=gws if given else None)
        elif writer == "logits grad":
            vh.logits_logprobs_grad(E, tokens, lse, lse, lse, lse, dlogits=table)
        else:
            vh.add_rmsnorm(E, None, w, y=table)
            if writer == "norm, then norm":
                vh.add_rmsnorm(s, None, w, y=y)
            elif writer != "norm":
                vh.logits_logprobs(big, tokens[:8], 0, ws=lws, **outs)

    ready = torch.empty_like(W)
    write(ready)
    for name, call in readers(vh, R, H, V).items():
        torch.cuda.synchronize()
        want = [t.clone() for t in call(ready) if t is not None]
        for _ in range(20):
            W.zero_()
            torch.cuda.synchronize()
            write(W)
            got = call(W)
            for a, b in zip((t for t in got if t is not None), want):
                assert torch.equal(a, b), name


@pytest.mark.parametrize("source", ["logits, few rows", "logits, many rows", "head", "draft"])
def test_row_ids_written_by_the_call_before(vh, source):
    """The alternatives of one call as the list of rows of a gathering draft."""
    H, V, n = 512, 20000, 32
    g = torch.Generator("cuda").manual_seed(5)
    W, x = randn(g, V, H), randn(g, 2, H)
    R = 700 if source == "logits, many rows" else 16
    logits, hidden = randn(g, R, V), randn(g, R, H)
    cand = torch.arange(V, device="cuda", dtype=torch.int32)
    tokens = torch.zeros(R, dtype=torch.int32, device="cuda")
    ids = torch.zeros(R, n, dtype=torch.int32, device="cuda")
    f = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    o = dict(logprob=f(R), entropy=f(R), lse=f(R), top_ids=ids, top_logprobs=f(R, n))
    lws, hws, ws = vh.logits_logprobs_workspace(R, V, n), vh.head_logprobs_workspace(R, V, n), vh.workspace(16)

    def write():
        if source == "draft":
            vh.mtp_draft_head_argmax(hidden, W, cand, ws=ws, ids=ids.view(-1)[:R], maxlogit=o["lse"])
        elif source == "head":
            vh.head_logprobs(hidden, W, tokens, n, ws=hws, **o)
        else:
            vh.logits_logprobs(logits, tokens, n, ws=lws, **o)

    write()
    torch.cuda.synchronize()
    rows = ids.view(-1)[:R] if source == "draft" else ids.view(-1)
    want = [t.clone() for t in vh.mtp_draft_head_argmax_gather(x, W, rows, ws=ws)]
    for _ in range(20):
        ids.fill_(V - 1)
        torch.cuda.synchronize()
        write()
        got = vh.mtp_draft_head_argmax_gather(x, W, rows, ws=ws)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
