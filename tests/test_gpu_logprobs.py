"""Log probabilities with entropy and alternatives, from logits (and their
gradient) and from hidden rows and a head, against the 64-bit definitions:
odd vocabularies, ties, masked, empty, NaN and infinite rows, strided and
misaligned rows, rows split over CTAs, every kernel's row counts."""
import math

import pytest
import torch

from rows_util import TINY, U, close, logprobs64, logprobs_loss64, sums

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def vh():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import verify_head_gb300 as vh
    vh.build()
    return vh


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def logits(g, R, V, dtype, scale=2.0, pitch=None, offset=0):
    pitch = pitch or V
    flat = torch.full((R * pitch + offset + 16,), 1e4, dtype=dtype, device="cuda")  # a read past a row would show
    t = flat[offset:offset + R * pitch].view(R, pitch)[:, :V]
    t.copy_((torch.randn(R, V, generator=g) * scale).to(dtype))
    return t


def check(got, x, tokens, n):
    lp, ent, lse, ids, top = logprobs64(x, tokens, n)
    V = x.shape[1]
    # |x - c| and lse - c are at most a few hundred here; each is rounded once, ln s carries the sum's error
    floor = sums(V) + 2.0 ** -20
    close(got[0], lp, 2.0 ** -22, floor)
    close(got[1], ent, 2.0 ** -22, 20 * sums(V))
    close(got[2], lse, 2.0 ** -22, floor)
    if n:
        assert torch.equal(got[3].cpu(), ids)
        close(got[4], top, 2.0 ** -22, floor)


CASES = [(1, 1, 1), (2, 3, 5), (3, 31, 32), (5, 128, 3), (4, 1000, 20), (2, 4097, 7), (1, 40001, 32), (130, 777, 2),
         (1, 248320, 20), (3, 131072, 0), (700, 513, 5)]


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("R,V,n", CASES)
def test_logits_match_definition(vh, R, V, n, dtype):
    g = gen(R * 31 + V)
    x = logits(g, R, V, dtype)  # 16-bit rows hold many equal logits: the ids check the tie rule
    tokens = torch.randint(0, V, (R,), generator=g, dtype=torch.int32)
    tokens[R // 2] = -100
    tokens[R - 1] = V - 1 if R > 1 else tokens[R - 1]
    check(vh.logits_logprobs(x, tokens.cuda(), n), x, tokens, n)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V,pitch,offset", [(1000, 1000, 1), (1000, 1003, 0), (999, 1001, 5), (5, 7, 3), (70001, 70001, 1)])
def test_strides_and_alignment(vh, V, pitch, offset, dtype):
    g = gen(V + pitch)
    x = logits(g, 5, V, dtype, pitch=pitch, offset=offset)
    tokens = torch.tensor([0, V - 1, V, -1, V // 2], dtype=torch.int32)
    check(vh.logits_logprobs(x, tokens.cuda(), 4), x, tokens, 4)


def test_rows_past_32_bits(vh):
    """Rows more than 2^31 elements apart."""
    V, pitch = 4000, 1_500_000_000
    flat = torch.empty(2 * pitch + V, dtype=BF, device="cuda")
    x = flat.as_strided((3, V), (pitch, 1))
    x.copy_(torch.randn(3, V, generator=gen(1)).to(BF))
    tokens = torch.tensor([1, 2, 3], dtype=torch.int32)
    got = vh.logits_logprobs(x, tokens.cuda(), 5)
    check(got, x, tokens, 5)
    one = torch.ones(3, device="cuda")
    want = vh.logits_logprobs_grad(x.contiguous(), tokens.cuda(), got[2], got[1], one, one)
    vh.logits_logprobs_grad(x, tokens.cuda(), got[2], got[1], one, one, dlogits=x)
    assert torch.equal(x, want)


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("V", [5, 700, 9001, 100000])
def test_masks_and_special_rows(vh, V, dtype):
    g = gen(V)
    low = float(torch.finfo(dtype).min)
    x = logits(g, 9, V, dtype)
    x[0] = -math.inf                       # nothing allowed
    x[1] = -math.inf
    x[1, V - 1] = 0.25                     # one place allowed
    x[2] = low                             # masked with the type's lowest value throughout: uniform
    x[3, ::2] = low                        # half masked so
    x[4, ::2] = -math.inf
    x[5, V // 2] = math.inf
    x[6, 1] = math.nan                     # counts as -inf
    x[7] = 0.0
    x[7, 2:] = -0.0                        # equal
    x[8] = math.nan
    tokens = torch.tensor([0, V - 1, 1, 0, 1, 0, 1, 2, 3], dtype=torch.int32)
    got = vh.logits_logprobs(x, tokens.cuda(), 6)
    lp, ent, lse, ids, top = logprobs64(x, tokens, 6)
    # past the V-th: id -1 and -inf, in the row of NaN as elsewhere
    assert torch.equal(got[3].cpu(), ids)
    keep = [0, 1, 2, 3, 4, 6, 7, 8]
    floor = sums(V) + 2.0 ** -20
    close(got[0][keep], lp[keep], 2.0 ** -22, floor)
    close(got[1][keep], ent[keep], 2.0 ** -22, 20 * sums(V))
    close(got[2][keep], lse[keep], 2.0 ** -22, floor)
    close(got[4][keep], top[keep], 2.0 ** -22, floor)
    for k in range(3):
        assert math.isnan(float(got[k][5]))


def test_rising_and_falling_rows(vh):
    """Maxima that move with every element, and ties across segments."""
    V = 66000
    x = torch.stack([torch.arange(V).float() * 1e-3, -torch.arange(V).float() * 1e-3, torch.ones(V),
                     (torch.arange(V) // 64 % 2).float()]).cuda()
    tokens = torch.tensor([V - 1, 0, 77, 64], dtype=torch.int32)
    check(vh.logits_logprobs(x, tokens.cuda(), 32), x, tokens, 32)


def test_workspace_serves_other_sizes(vh):
    ws = vh.logits_logprobs_workspace(64, 20000, 20)
    for R, V, n, dtype in ((3, 20000, 20, F32), (64, 20000, 20, BF), (1, 9999, 3, HF), (17, 5000, 0, F32), (3, 20000, 20, F32)):
        g = gen(R)
        x = logits(g, R, V, dtype)
        tokens = torch.randint(0, V, (R,), generator=g, dtype=torch.int32)
        check(vh.logits_logprobs(x, tokens.cuda(), n, ws=ws), x, tokens, n)


def test_no_tokens_streams_and_graph(vh):
    g = gen(1)
    x = logits(g, 4, 50000, F32)
    tokens = torch.randint(0, 50000, (4,), generator=g, dtype=torch.int32).cuda()
    want = vh.logits_logprobs(x, tokens, 8)
    none = vh.logits_logprobs(x, None, 8)
    assert none[0] is None and torch.equal(none[3], want[3])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        got = vh.logits_logprobs(x, tokens, 8, stream=s)
    s.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    ws = vh.logits_logprobs_workspace(4, 50000, 8)
    outs = dict(logprob=want[0], entropy=want[1], lse=want[2], top_ids=want[3], top_logprobs=want[4])
    want = [t.clone() for t in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vh.logits_logprobs(x, tokens, 8, ws=ws, **outs)
        vh.logits_logprobs(x, tokens, 8, ws=ws, **outs)
    for t in outs.values():
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(outs.values(), want):
        assert torch.equal(a, b)


# ---------------------------------------------------------------------------
# Gradient


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("R,V", [(1, 1), (2, 3), (5, 1000), (3, 8193), (130, 777), (2, 70000)])
@pytest.mark.parametrize("parts", ["both", "logprob", "entropy"])
def test_grad_matches_formula(vh, R, V, dtype, parts):
    g = gen(R + V)
    x = logits(g, R, V, dtype)
    if V > 2:
        x[:, 1] = -math.inf
    tokens = torch.randint(0, V, (R,), generator=g, dtype=torch.int32)
    if V > 2:
        tokens[tokens == 1] = 0
    tokens[R // 2] = -100
    gl, ge = torch.randn(R, generator=g), torch.randn(R, generator=g)
    _, ent, lse = vh.logits_logprobs(x, tokens.cuda())[:3]
    d = vh.logits_logprobs_grad(x, tokens.cuda() if parts != "entropy" else None, lse,
                                ent if parts != "logprob" else None, gl.cuda() if parts != "entropy" else None,
                                ge.cuda() if parts != "logprob" else None)
    if parts == "logprob":
        ge = ge * 0
    if parts == "entropy":
        gl = gl * 0
    x64 = x.double().cpu().requires_grad_()
    want, = torch.autograd.grad(logprobs_loss64(x64, tokens, gl.double(), ge.double()), x64)
    want = torch.nan_to_num(want, nan=0.0)
    # p is e^(x - lse): the error of lse (sums, and its own rounding) and of the exponent is p's relative error
    p = torch.softmax(x64.detach(), 1)
    size = p * (gl.abs()[:, None] + ge.abs()[:, None] * 40)
    close(d, want, U[dtype] * (1 + 2 ** -10) + 2.0 ** -22, size.double() * (sums(V) + 2.0 ** -18) + TINY[dtype])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V,pitch,offset", [(1000, 1000, 1), (999, 1003, 0), (5, 7, 3), (9001, 9001, 5), (4096, 4104, 0)])
def test_grad_strides_and_in_place(vh, V, pitch, offset, dtype):
    """Rows that lie alike in their 16-byte slots (in place) and not (a new tensor), with the same results."""
    g = gen(V)
    x = logits(g, 6, V, dtype, pitch=pitch, offset=offset)
    tokens = torch.randint(0, V, (6,), generator=g, dtype=torch.int32).cuda()
    gl = torch.randn(6, generator=g).cuda()
    _, ent, lse = vh.logits_logprobs(x, tokens)[:3]
    d = vh.logits_logprobs_grad(x, tokens, lse, ent, gl, gl)
    whole = torch.empty(0, dtype=dtype, device="cuda").set_(x.untyped_storage())
    before = whole.clone()
    same = vh.logits_logprobs_grad(x, tokens, lse, ent, gl, gl, dlogits=x)
    assert same is x and torch.equal(x, d)
    mask = torch.ones_like(whole, dtype=torch.bool)
    mask.as_strided((6, V), (pitch, 1), x.storage_offset()).fill_(False)
    assert torch.equal(whole[mask], before[mask])


def test_grad_special_rows(vh):
    V = 3000
    x = logits(gen(2), 4, V, F32)
    x[0] = -math.inf
    x[1, 7] = math.inf
    x[2] = -math.inf
    x[2, 9] = 1.0
    tokens = torch.tensor([5, 5, 9, -1], dtype=torch.int32).cuda()
    one = torch.ones(4, device="cuda")
    _, ent, lse = vh.logits_logprobs(x, tokens)[:3]
    d = vh.logits_logprobs_grad(x, tokens, lse, ent, one, one)
    assert torch.equal(d[0], torch.zeros(V, device="cuda"))
    assert bool(torch.isnan(d[1]).all())
    assert torch.equal(d[2], torch.zeros(V, device="cuda"))  # one place holds all the probability
    assert bool(torch.isfinite(d[3]).all()) and abs(float(d[3].double().sum())) < 1e-5
    d = vh.logits_logprobs_grad(x, tokens, lse, None, one)
    assert torch.equal(d[3], torch.zeros(V, device="cuda"))  # no token, no entropy


def test_grad_matches_differences(vh):
    g = gen(4)
    R, V = 3, 50
    x = torch.randn(R, V, generator=g)
    tokens = torch.tensor([3, -100, 49], dtype=torch.int32)
    gl, ge = torch.randn(R, generator=g), torch.randn(R, generator=g)
    _, ent, lse = vh.logits_logprobs(x.cuda(), tokens.cuda())[:3]
    d = vh.logits_logprobs_grad(x.cuda(), tokens.cuda(), lse, ent, gl.cuda(), ge.cuda()).cpu()
    step = 1e-5
    for r, v in [(0, 3), (0, 0), (1, 20), (2, 49), (2, 48)]:
        e = torch.zeros(R, V, dtype=torch.float64)
        e[r, v] = step
        up = logprobs_loss64(x.double() + e, tokens, gl.double(), ge.double())
        down = logprobs_loss64(x.double() - e, tokens, gl.double(), ge.double())
        assert abs(float(d[r, v]) - float(up - down) / (2 * step)) < 1e-5


# ---------------------------------------------------------------------------
# From hidden rows and a head


def head(g, R, V, H, exact=True):
    """exact: values on grids of 1/16 and 1/1024, so that every score is exact in 32 bits in any order."""
    x, W = torch.randn(R, H, generator=g), torch.randn(V, H, generator=g) * 0.05
    if exact:
        x, W = (x * 16).round().clamp(-100, 100) / 16, (W * 1024).round().clamp(-120, 120) / 1024
    return x.to(BF).cuda(), W.to(BF).cuda()


# row counts on either side of each kernel's and row group's limit; widths that end inside a K stage
HEADS = [(1, 1, 16, 1), (1, 129, 64, 5), (4, 5000, 256, 20), (16, 127, 80, 32), (33, 1000, 144, 3), (64, 2049, 512, 0),
         (65, 300, 64, 2), (100, 20001, 128, 20), (128, 513, 272, 4), (129, 513, 272, 4), (256, 20001, 128, 20),
         (257, 255, 64, 1), (513, 1000, 48, 6), (1024, 3001, 64, 2), (1030, 777, 128, 3), (2, 200, 8192, 2)]


@pytest.mark.parametrize("R,V,H,n", HEADS)
def test_head_matches_definition(vh, R, V, H, n):
    g = gen(R + V + H)
    x, W = head(g, R, V, H)
    tokens = torch.randint(0, V, (R,), generator=g, dtype=torch.int32)
    tokens[R // 2] = V
    tokens[0] = V - 1
    ws = vh.head_logprobs_workspace(R, V, n)
    got = vh.head_logprobs(x, W, tokens.cuda(), n, ws=ws)
    check(got, x.double() @ W.double().t(), tokens, n)
    assert vh.workspace_error(ws) == 0


@pytest.mark.parametrize("R", [3, 70, 200])
def test_head_agrees_with_verify_and_logits(vh, R):
    """The first alternative is the verify kernel's argmax, and the statistics those of the scores themselves."""
    g = gen(R)
    V, H = 30000, 256
    x, W = head(g, R, V, H, exact=False)
    tokens = torch.randint(0, V, (R,), generator=g, dtype=torch.int32).cuda()
    lp, ent, lse, ids, top = vh.head_logprobs(x, W, tokens, 4)
    s = x.double() @ W.double().t()
    want = logprobs64(s, tokens.cpu(), 4)
    # an fp32 accumulation of H products, each addition off by at most a unit of the largest partial sum
    off = float((x.double().abs() @ W.double().abs().t()).max()) * (H / 8) * 2.0 ** -23
    close(lp, want[0], 0.0, 2 * off + sums(V))
    close(lse, want[2], 0.0, off + sums(V))
    close(ent, want[1], 0.0, 40 * off + 20 * sums(V))
    close(top, want[4], 0.0, 2 * off + sums(V))
    draft = torch.zeros(R, 1, dtype=torch.int32, device="cuda")
    _, nid, ml = vh.spec_verify_greedy(torch.cat([x, x]).view(2, R, H).transpose(0, 1).reshape(2 * R, H).contiguous(), W,
                                       draft, R, 1)
    clear = torch.topk(s, 2, dim=1).values
    clear = (clear[:, 0] - clear[:, 1] > 2 * off)
    assert torch.equal(nid[::2][clear], ids[:, 0][clear])


def test_head_nan_and_infinite_scores(vh):
    g = gen(12)
    x, W = head(g, 5, 400, 64)
    W[7] = math.nan                        # counts as -inf
    x[3] = math.nan                        # a row of NaN scores: empty
    tokens = torch.tensor([7, 1, 2, 3, 4], dtype=torch.int32)
    check(vh.head_logprobs(x, W, tokens.cuda(), 3), x.double() @ W.double().t(), tokens, 3)


def test_head_workspace_serves_other_sizes_in_a_row(vh):
    ws = vh.head_logprobs_workspace(300, 9000, 20)
    for R, V, H, n in ((300, 9000, 64, 20), (2, 9000, 256, 20), (40, 1000, 64, 0), (300, 9000, 64, 20)):
        g = gen(R)
        x, W = head(g, R, V, H)
        tokens = torch.randint(0, V, (R,), generator=g, dtype=torch.int32)
        check(vh.head_logprobs(x, W, tokens.cuda(), n, ws=ws), x.double() @ W.double().t(), tokens, n)
    assert vh.workspace_error(ws) == 0


@pytest.mark.parametrize("R", [4, 200])
def test_head_graph_replay(vh, R):
    g = gen(R)
    x, W = head(g, R, 5000, 128)
    tokens = torch.randint(0, 5000, (R,), generator=g, dtype=torch.int32).cuda()
    ws = vh.head_logprobs_workspace(R, 5000, 5)
    outs = vh.head_logprobs(x, W, tokens, 5, ws=ws)
    want = [t.clone() for t in outs]
    names = ("logprob", "entropy", "lse", "top_ids", "top_logprobs")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(2):
            vh.head_logprobs(x, W, tokens, 5, ws=ws, **dict(zip(names, outs)))
    for t in outs:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(outs, want):
        assert torch.equal(a, b)


def test_refusals(vh):
    x = torch.zeros(2, 100, device="cuda")
    t = torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        vh.logits_logprobs(x, t.long())
    with pytest.raises(ValueError):
        vh.logits_logprobs(x, t[:1])
    with pytest.raises(ValueError):
        vh.logits_logprobs(x.double(), t)
    with pytest.raises(ValueError):
        vh.logits_logprobs(x.cpu(), t)
    with pytest.raises(vh.VHError):
        vh.logits_logprobs(x, t, 33)
    with pytest.raises(vh.VHError):
        vh.logits_logprobs(x[:0], t[:0])
    with pytest.raises(vh.VHError):
        vh.logits_logprobs(x, t, 2, ws=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(vh.VHError):
        vh.logits_logprobs_grad(x, t, torch.zeros(2, device="cuda"), None, None, torch.zeros(2, device="cuda"))
    h, W = torch.zeros(2, 64, dtype=BF, device="cuda"), torch.zeros(9, 64, dtype=BF, device="cuda")
    with pytest.raises(ValueError):
        vh.head_logprobs(h.float(), W, t)
    with pytest.raises(ValueError):
        vh.head_logprobs(h, W[:, :32], t)
    with pytest.raises(vh.VHError):
        vh.head_logprobs(h[:, :24].contiguous(), W[:, :24].contiguous(), t)  # H % 16
    with pytest.raises(vh.VHError):
        vh.head_logprobs(h, W, t, ws=torch.zeros(16, dtype=torch.uint8, device="cuda"))


# ---------------------------------------------------------------------------
# The choice of alternatives: every way through it


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [33, 400, 513, 4633, 60771, 200001])
@pytest.mark.parametrize("n", [1, 20, 32])
@pytest.mark.parametrize("kind", ["plain", "few allowed", "equal", "two values", "late ties", "comb"])
def test_alternatives(vh, V, n, kind, dtype):
    """Units near and below n, rows with fewer allowed places than n, ties at the bound early and late in the row, and
    large values laid out in one group of units."""
    g = gen(V + n)
    R = 3
    x = (torch.randn(R, V, generator=g) * 2).to(dtype)
    if kind == "few allowed":
        keep = torch.randperm(V, generator=g)[:7]
        y = torch.full_like(x, -math.inf)
        y[:, keep] = x[:, keep]
        y[1] = -math.inf
        y[2, V // 2] = math.nan
        x = y
    elif kind == "equal":
        x = torch.full_like(x, 1.5)
        x[2] = 0.0
        x[2, ::3] = -0.0
    elif kind == "two values":
        x = (torch.rand(R, V, generator=g) < 0.5).to(dtype)
    elif kind == "late ties":
        x = x.clamp(max=0.5)
        x[:, : V // 2] = -1.0
        x[:, V // 2 + 3] = 9.0
    elif kind == "comb":  # descending values in every 64th slot of 32 bytes, so that one group holds them all
        per = 32 // x.element_size()
        at = torch.arange(V)
        x = torch.where(at // per % 64 == 0, 1000.0 - (at / V * 500), torch.zeros(V)).to(dtype).repeat(R, 1)
    tokens = torch.randint(0, V, (R,), generator=g, dtype=torch.int32)
    x = x.cuda()
    got = vh.logits_logprobs(x, tokens.cuda(), n)
    _, _, _, ids, top = logprobs64(x, tokens, n)
    assert torch.equal(got[3].cpu(), ids)
    close(got[4], top, 2.0 ** -22, sums(V) + 2.0 ** -18)


@pytest.mark.parametrize("R,V,n", [(2, 999, 32), (150, 999, 32), (3, 300, 20), (130, 9000, 32)])
def test_head_alternatives_with_ties(vh, R, V, n):
    """Equal scores throughout, then in half of the head, and none: in the order of the ids."""
    H = 64
    x = torch.ones(R, H, dtype=BF, device="cuda")
    for kind in range(3):
        W = torch.zeros(V, H, dtype=BF, device="cuda")
        if kind == 1:
            W[V // 2:, 0] = 1.0
        if kind == 2:
            W[:, 0] = torch.randint(-3, 4, (V,), generator=gen(V)).to(BF).cuda()
        tokens = torch.zeros(R, dtype=torch.int32)
        got = vh.head_logprobs(x, W, tokens.cuda(), n)
        _, _, _, ids, _ = logprobs64((x[:1].double() @ W.double().t()), tokens[:1], n)
        assert torch.equal(got[3].cpu(), ids.expand(R, n))


# how the scan is cut: rows into pieces, whole rows, a CTA per row past the SMs' places, even ranges (many rows of over 128
# segments, rows that fill half of the places, with alternatives)
@pytest.mark.parametrize("R,V,n", [(7, 30011, 0), (40, 60000, 0), (150, 20000, 0), (150, 20000, 3), (609, 2000, 0),
                                   (1301, 5003, 0), (1301, 5003, 2), (620, 70001, 0), (310, 131072, 0), (310, 131072, 4),
                                   (608, 33000, 0), (457, 40000, 1)])
def test_every_cut_of_the_rows(vh, R, V, n):
    g = torch.Generator(device="cuda")
    g.manual_seed(R + V)
    x = (torch.randn(R, V, generator=g, device="cuda") * 2).to(BF)
    tokens = torch.randint(0, V, (R,), generator=g, device="cuda", dtype=torch.int32)
    ws = vh.logits_logprobs_workspace(R, V, n)
    got = vh.logits_logprobs(x, tokens, n, ws=ws)
    lse = torch.cat([torch.logsumexp(p.double(), 1) for p in x.split(64)])
    close(got[2], lse, 2.0 ** -22, sums(V) + 2.0 ** -20)
    ent = torch.cat([l - (torch.softmax(p.double(), 1) * p.double()).sum(1) for p, l in zip(x.split(64), lse.split(64))])
    close(got[1], ent, 2.0 ** -22, 20 * sums(V))
    close(got[0], x.gather(1, tokens.long()[:, None])[:, 0].double() - lse, 2.0 ** -22, sums(V) + 2.0 ** -20)
    if n:
        some = sorted({0, 1, R // 3, R // 2, R // 2 + 1, R - 2, R - 1})
        check([t[some] for t in got], x[some], tokens[some].cpu(), n)
    again = vh.logits_logprobs(x, tokens, n, ws=ws)  # the counters are left as they were
    assert all(torch.equal(a, b) for a, b in zip(got, again) if a is not None)
