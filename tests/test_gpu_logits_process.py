"""Processing of logits and its gradient against the 64-bit definitions, row by row: every rule alone and together, odd
vocabularies, strided and misaligned rows, histories from none to long ones with padding, masks that leave nothing,
infinities and NaN in masked places, ids listed twice, drafts of many rows."""
import math

import pytest
import torch

from rows_util import TINY, U, close
from w4_util import process64

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def vh():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import verify_head_gb300 as vh
    vh.build()
    return vh


def rows(g, R, V, dtype, pitch=None, offset=0, scale=3.0):
    pitch = pitch or V
    flat = torch.full((R * pitch + offset + 16,), 1e4, dtype=dtype, device="cuda")
    t = flat[offset:offset + R * pitch].view(R, pitch)[:, :V]
    t.copy_((torch.randn(R, V, generator=g) * scale).to(dtype))
    return t


def words(on):
    """Truth values [R,V] as bits of int32 words, with a word more than needed."""
    R, V = on.shape
    n = -(-V // 32) + 1
    b = torch.ones(R, n * 32, dtype=torch.bool)
    b[:, :V] = on
    w = (b.view(R, n, 32).long() << torch.arange(32)).sum(2)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).int().cuda()


def rules(g, S, m, V, L, nb, masked):
    r = {}
    if L:
        h = torch.randint(-3, V + 3, (S, L), generator=g, dtype=torch.int32)  # ids that are none among them
        h[:, ::3] = h[:, :1].clone()  # one that comes back often
        r["history"] = h.cuda()
        r["history_len"] = torch.randint(0, L + 3, (S,), generator=g, dtype=torch.int32).cuda()
        r["prompt_len"] = torch.randint(0, L + 1, (S,), generator=g, dtype=torch.int32).cuda()
    if m > 1:
        d = torch.randint(0, V, (S, m - 1), generator=g, dtype=torch.int32)
        d[:, 1::2] = d[:, :1].clone()
        if L:
            d[:, 2::3] = r["history"][:, :1].cpu()
        r["draft_ids"] = d.cuda()
    r["repetition"] = (0.8 + torch.rand(S, generator=g)).cuda()
    r["frequency"] = (torch.rand(S, generator=g) - 0.3).cuda()
    r["presence"] = (torch.rand(S, generator=g) - 0.3).cuda()
    t = 0.3 + torch.rand(S, generator=g)
    t[2::3] = 0.0
    r["temperature"] = t.cuda()
    if nb:
        ids = torch.randint(-2, V + 2, (S, nb), generator=g, dtype=torch.int32)
        ids[:, nb // 2:] = ids[:, :nb - nb // 2].clone()  # twice: the last entry counts
        if L:
            ids[:, 0] = r["history"][:, 0].cpu()
        r["bias_ids"], r["bias"] = ids.cuda(), (torch.randn(S, nb, generator=g) * 4).cuda()
    if masked:
        on = torch.rand(S * m, V, generator=g) >= masked
        on[1::4] = False
        on[2::4] = True
        r["allowed"] = words(on)
    return r


def tolerance(out_dtype, x, r):
    """Per term one rounding of 2^-24: the bias, the penalty, three of frequency and presence, 1 / T and its product, and
    what those take off is relative to the largest of them; then the rounding to the type."""
    big = float(x.float()[torch.isfinite(x.float())].abs().max()) + 16
    L = 0 if r.get("history") is None else r["history"].shape[1]
    return U[out_dtype] + 2.0 ** -22, (big * 2 + 2 * (L + 16)) / 0.3 * 8 * 2.0 ** -24 + TINY[out_dtype]


def check(vh, x, S, r, out_dtype=None, out=None):
    out_dtype = out_dtype or (x.dtype if out is None else out.dtype)
    keep = x.clone()
    want = process64(x, S, r)
    got = vh.logits_process(x, out=torch.empty(x.shape, dtype=out_dtype, device="cuda") if out is None else out, **r)
    rel, floor = tolerance(out_dtype, x, r)
    # a number past the type's range (its lowest one times a repetition of 1.2) rounds to infinity
    want = torch.where(want.abs() > torch.finfo(out_dtype).max * (1 + U[out_dtype]), want * math.inf, want)
    close(got, want, rel, floor)
    if got.data_ptr() != x.data_ptr():
        assert torch.equal(torch.nan_to_num(x), torch.nan_to_num(keep))


def check_grad(vh, x, S, r, pitch=None):
    d = rows(torch.Generator().manual_seed(77), *x.shape, x.dtype, pitch, 0, 0.1)
    want = process64(x, S, r, d)
    got = vh.logits_process_grad(d, x, **r)
    # two roundings of 2^-24, the rounding to the type; the sign of z is that of the sum in fp32 (a logit and a bias that
    # cancel to within 2^-24 are not drawn)
    close(got, want, U[x.dtype] + 2.0 ** -22, TINY[x.dtype])
    same = d.clone()
    assert vh.logits_process_grad(same, x, dlogits=same, **r) is same
    assert torch.equal(same, got)


CASES = [(1, 1, 1, 0, 0, 0.0), (1, 1, 5, 3, 1, 0.5), (3, 2, 33, 40, 4, 0.3), (2, 4, 1000, 100, 10, 0.0), (5, 1, 4099, 500, 300, 0.6),
         (2, 16, 777, 50, 2, 0.2), (1, 41, 130, 7, 3, 0.1), (1, 4, 40001, 3000, 8, 0.9), (9, 3, 257, 1, 0, 0.0), (1, 1, 20000, 0, 5, 0.0),
         (2, 2, 30011, 20000, 3, 0.4)]


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("S,m,V,L,nb,masked", CASES)
def test_definition(vh, S, m, V, L, nb, masked, dtype):
    g = torch.Generator().manual_seed(S + V)
    for pitch, offset in ((V, 0), (V + 5, 3)):
        x = rows(g, S * m, V, dtype, pitch, offset)
        r = rules(g, S, m, V, L, nb, masked)
        check(vh, x, S, r)
        check_grad(vh, x, S, r, pitch)
        if dtype != F32:
            check(vh, x, S, r, F32)
            wide = torch.full((S * m, V + 3), 5.0, device="cuda")
            check(vh, x, S, r, out=wide[:, 1:V + 1])
            assert bool((wide[:, 0] == 5).all()) and bool((wide[:, V + 1:] == 5).all())


@pytest.mark.parametrize("name", ["history", "draft_ids", "bias", "allowed", "temperature", "none"])
def test_single_rules(vh, name):
    g = torch.Generator().manual_seed(1)
    S, m, V = 3, 4, 2003
    x = rows(g, S * m, V, BF)
    full = rules(g, S, m, V, 60, 5, 0.5)
    groups = {"history": ("history", "repetition"), "draft_ids": ("draft_ids", "frequency", "presence"), "bias": ("bias_ids", "bias"),
              "allowed": ("allowed",), "temperature": ("temperature",), "none": ()}
    r = {k: full[k] for k in groups[name]}
    S = S if name not in ("allowed", "none") else S * m
    check(vh, x, S, r)
    check_grad(vh, x, S, r)
    if name == "none":
        assert torch.equal(vh.logits_process(x), x)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_in_place(vh, dtype):
    g = torch.Generator().manual_seed(2)
    for V in (777, 16384 + 40):
        x = rows(g, 6, V, dtype)
        r = rules(g, 2, 3, V, 90, 4, 0.3)
        want = vh.logits_process(x.clone(), **r)
        assert vh.logits_process(x, out=x, **r) is x
        assert torch.equal(x, want)


def test_places_that_are_no_numbers(vh):
    """Behind the mask anything may stand; before it infinities stay, and NaN is NaN."""
    g = torch.Generator().manual_seed(3)
    for dtype in (F32, BF, HF):
        x = rows(g, 4, 900, dtype)
        x[0, ::3], x[1, ::3], x[2, ::3] = math.nan, math.inf, -math.inf
        x[3, 5], x[3, 6] = -math.inf, torch.finfo(dtype).min
        on = torch.ones(4, 900, dtype=torch.bool)
        on[:3, ::3] = False
        h = torch.arange(0, 900, 2, dtype=torch.int32, device="cuda").repeat(4, 1)
        one = torch.ones(4, device="cuda")
        r = dict(history=h, repetition=one * 1.2, frequency=one * 0.1, presence=one * 0.2, temperature=one, allowed=words(on))
        check(vh, x, 4, r)
        d = rows(g, 4, 900, dtype)
        d[0, ::3] = math.nan
        got = vh.logits_process_grad(d, x, **r)
        assert bool(torch.isfinite(got[:, ::3][:3]).all()) and float(got[:3, ::3].float().abs().max()) == 0
        bare = vh.logits_process(x, temperature=one * 2)
        assert bool(torch.isnan(bare[0, ::3]).all()) and bool((bare[1, ::3] == math.inf).all()) and bool((bare[2, ::3] == -math.inf).all())


def test_gradient_by_differences(vh):
    """fp32 differences over steps that cross no sign."""
    g = torch.Generator().manual_seed(4)
    S, m, V = 2, 3, 64
    x = rows(g, S * m, V, F32)
    r = rules(g, S, m, V, 30, 3, 0.2)
    near = x.clone()
    for s in range(S):
        for i, b in zip(r["bias_ids"][s].tolist(), r["bias"][s].tolist()):
            if 0 <= i < V:
                near[s * m:(s + 1) * m, i] = x[s * m:(s + 1) * m, i] + b
    step = 2.0 ** -6
    safe = near.abs() > 4 * step
    d = rows(g, S * m, V, F32)
    dx = vh.logits_process_grad(d, x, **r)
    up, down = (torch.nan_to_num(vh.logits_process(x + e, **r), neginf=0.0) for e in (step, -step))
    num = (up - down) / (2 * step) * d
    # values of up to about 100 / 0.3 rounded a few times at 2^-24, over a step of 2^-5
    assert float(((num - dx).abs() * safe).max()) < 1e3 * 4 * 2.0 ** -24 * 2 ** 5 * float(d.abs().max())


def test_then_log_probabilities(vh):
    """Logits of a 4-bit head, processed, and their log probabilities with alternatives; and the way back."""
    g = torch.Generator().manual_seed(5)
    S, m, V, H = 3, 4, 5003, 256
    hid = torch.randn(S * m, H, generator=g).to(BF).cuda()
    w = (torch.randn(V, H, generator=g) * 0.05).cuda()
    gw = float(w.abs().max()) / 2688
    codes, scales, _ = vh.nvfp4_quantize(w, gw)
    xt, xg = vh.nvfp4_quantize_tiles(hid)
    logits = vh.nvfp4_matmul(xt, xg, vh.nvfp4_tile(codes, scales), gw, S * m, V, H, dtype=F32)
    r = rules(g, S, m, V, 200, 4, 0.5)
    r["allowed"][1::4, 0] |= 1  # no row without a choice
    out = vh.logits_process(logits, **r)
    tok = torch.full((S * m,), 7, dtype=torch.int32, device="cuda")
    lp, ent, lse, ids, top = vh.logits_logprobs(out, tok, 5)
    want = process64(logits, S, r)
    ref = torch.log_softmax(want, 1)
    assert float((lse.cpu().double() - torch.logsumexp(want, 1)).abs().max()) < 1e-4
    best = want.max(1)
    near = want.gather(1, ids[:, :1].long().cpu())[:, 0] >= best.values - 1e-4
    assert bool(near.all())
    gl = torch.randn(S * m, generator=g).cuda()
    d = vh.logits_logprobs_grad(out, tok, lse, ent, gl)
    dl = vh.logits_process_grad(d, logits, **r)
    z = logits.double().cpu().requires_grad_()
    ones = torch.ones(S * m, V)
    slope = process64(logits, S, r, ones)  # d out / d logits
    p = torch.exp(ref)
    hot = torch.zeros_like(p)
    hot[:, 7] = 1.0
    full = gl.cpu().double()[:, None] * (hot - p) * slope
    assert float((dl.cpu().double() - full).abs().max()) < 1e-4
    dhid = dl @ vh.nvfp4_dequantize(codes, scales, gw, dtype=F32)
    assert bool(torch.isfinite(dhid).all()) and z.shape == logits.shape


def test_replayed_and_on_another_stream(vh):
    g = torch.Generator().manual_seed(6)
    x = rows(g, 8, 3001, BF)
    r = rules(g, 2, 4, 3001, 64, 3, 0.3)
    out = torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    vh.logits_process(x, out=out, **r)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        vh.logits_process(x, out=out, **r)
    for i in range(3):
        x.copy_(torch.randn(8, 3001, generator=g) * 3)
        r["history"].copy_(torch.randint(0, 3001, (2, 64), generator=g, dtype=torch.int32))
        r["history_len"].fill_(20 * i)
        graph.replay()
        close(out, process64(x, 2, r), *tolerance(BF, x, r))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out.zero_()
    vh.logits_process(x, out=out, stream=side, **r)
    torch.cuda.current_stream().wait_stream(side)
    close(out, process64(x, 2, r), *tolerance(BF, x, r))


def test_refusals(vh):
    x = torch.zeros(6, 100, dtype=BF, device="cuda")
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    f32 = lambda *s: torch.ones(*s, device="cuda")  # noqa: E731
    d = torch.zeros_like(x)
    for kw in (dict(history=i32(4, 5)), dict(history=i32(2, 5).long()), dict(history=i32(10)), dict(history=i32(2, 5), history_len=i32(3)),
               dict(repetition=f32(4)), dict(repetition=f32(2), frequency=f32(3)), dict(temperature=f32(2).double()),
               dict(draft_ids=i32(2, 3)), dict(bias_ids=i32(2, 3)), dict(bias_ids=i32(2, 3), bias=f32(2, 4)),
               dict(allowed=i32(6, 3)), dict(allowed=i32(5, 4)), dict(allowed=i32(6, 4).long()), dict(history=i32(2, 5).cpu())):
        with pytest.raises(ValueError):
            vh.logits_process(x, **kw)
        with pytest.raises(ValueError):
            vh.logits_process(x, out=torch.empty_like(x), **kw)
        with pytest.raises(ValueError):
            vh.logits_process_grad(d, x, **kw)
    for bad in (lambda: vh.logits_process(x.cpu()), lambda: vh.logits_process(x.int()), lambda: vh.logits_process(x.t()),
                lambda: vh.logits_process(x, out=x[:, :99]), lambda: vh.logits_process(x, out=x.half()),
                lambda: vh.logits_process_grad(d.float(), x), lambda: vh.logits_process_grad(d, x, dlogits=d[:5])):
        with pytest.raises(ValueError):
            bad()
