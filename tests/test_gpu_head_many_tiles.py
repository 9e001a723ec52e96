"""Log probabilities of heads with many tiles per CTA: both accumulators used again and again, later blocks of scores left
out once a bound of the alternatives is known, several row groups, ties at the bound, and fewer units than alternatives."""
import pytest
import torch

from rows_util import close, sums

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module")
def vh():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import verify_head_gb300 as vh
    vh.build()
    return vh


def head(seed, R, V, H):
    """Values on grids of 1/16 and 1/1024, so that every score is exact in 32 bits in any order."""
    g = torch.Generator("cuda").manual_seed(seed)
    x = (torch.randn(R, H, generator=g, device="cuda") * 16).round().clamp(-100, 100) / 16
    W = (torch.randn(V, H, generator=g, device="cuda") * 51).round().clamp(-120, 120) / 1024
    return x.to(BF), W.to(BF)


def check(got, x, W, tokens, n):
    """Every row against the 64-bit definition, some rows at a time; equal scores in the order of their ids."""
    V = W.shape[0]
    floor = sums(V) + 2.0 ** -20  # of ln s; score - maximum is exact
    Wt = W.double().t()
    for r in range(0, x.shape[0], 64):
        at = slice(r, r + 64)
        s = x[at].double() @ Wt
        lse = torch.logsumexp(s, 1)
        p = torch.softmax(s, 1)
        close(got[2][at], lse, 2.0 ** -22, floor)
        close(got[1][at], lse - (p * s).sum(1), 2.0 ** -22, 20 * sums(V))
        t = tokens[at].long()
        lp = torch.where(t >= 0, s.gather(1, t.clamp(min=0)[:, None])[:, 0] - lse, torch.zeros_like(lse))
        close(got[0][at], lp, 2.0 ** -22, floor)
        if n:
            best = torch.sort(s, dim=1, descending=True, stable=True)
            k = min(n, V)
            assert torch.equal(got[3][at, :k].long(), best.indices[:, :k])
            close(got[4][at, :k], best.values[:, :k] - lse[:, None], 2.0 ** -22, floor)


def run(vh, x, W, n, ws=None):
    R, V = x.shape[0], W.shape[0]
    tokens = (torch.arange(R, device="cuda") * 7919 % V).int()
    tokens[R // 2] = -100
    ws = vh.head_logprobs_workspace(R, V, n) if ws is None else ws
    got = vh.head_logprobs(x, W, tokens, n, ws=ws)
    check(got, x, W, tokens, n)
    assert vh.workspace_error(ws) == 0
    return ws


# 152 CTAs take 128 head rows each at a time, 76 pairs 256, or a quarter of the pairs in four row groups
@pytest.mark.parametrize("R,V", [(1, 99991), (4, 248320), (40, 60001), (100, 60000), (128, 80007), (129, 60000), (256, 99991),
                                 (300, 60000), (600, 59999), (1024, 60000), (1100, 40000)])
@pytest.mark.parametrize("n", [0, 20])
def test_many_tiles(vh, R, V, n):
    x, W = head(R + V, R, V, 64)
    ws = run(vh, x, W, n)
    run(vh, x.flip(0), W, n, ws)  # the counters and bounds of the first call are gone


@pytest.mark.parametrize("n", [1, 20, 32])
def test_full_head(vh, n):
    """The whole vocabulary at a usual width, on both kernels."""
    for R in (4, 256):
        x, W = head(R, R, 248320, 2048)
        run(vh, x, W, n)


KINDS = ["equal", "rising", "falling", "best last", "best first", "few values", "steps", "mostly low"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("R,n", [(3, 32), (100, 5), (256, 20), (600, 32), (1024, 1)])
def test_orders_and_ties(vh, R, n, kind):
    """Scores laid out so that the bound from the first tiles is met, or passed, by all, none or some of the later blocks.
    The score of head row v is the sum of two of its columns (256 a + b), the same in every hidden row up to a factor."""
    V, H = 60000, 64
    v = torch.arange(V, device="cuda")
    g = torch.Generator("cuda").manual_seed(R)
    value = {"equal": torch.zeros_like(v), "rising": v, "falling": V - v, "best last": (v >= V - 40) * 500 + v % 3,
             "best first": (v < 40) * 500 + v % 3, "few values": torch.randint(0, 4, (V,), generator=g, device="cuda"),
             "steps": v // 4096, "mostly low": (v % 997 == 0) * (v // 997)}[kind]
    W = torch.zeros(V, H, dtype=BF, device="cuda")
    W[:, 0] = (value // 256).to(BF)
    W[:, 1] = (value % 256).to(BF)
    x = torch.zeros(R, H, dtype=BF, device="cuda")
    scale = 2.0 ** -(torch.arange(R, device="cuda") % 4 + 6).float()
    x[:, 0], x[:, 1] = (256 * scale).to(BF), scale.to(BF)
    run(vh, x, W, n)


@pytest.mark.parametrize("V", [545, 700, 991, 1023])
@pytest.mark.parametrize("R", [2, 200])
def test_fewer_units_than_alternatives(vh, R, V):
    """18 to 32 blocks of 32 scores and 32 alternatives: equal scores overflow the lists, and the blocks are sorted."""
    H = 64
    x, W = head(V, R, V, H)
    run(vh, x, W, 32)
    for value in (torch.zeros(V), torch.arange(V) % 2, torch.arange(V) // 500, (torch.arange(V) % 37 == 0)):
        W = torch.zeros(V, H, dtype=BF, device="cuda")
        W[:, 0] = value.to(BF).cuda()
        x = torch.ones(R, H, dtype=BF, device="cuda")
        run(vh, x, W, 32)
