"""The two ways the norm and log-probability calls reach the library (compiled marshalling, and the Python checks that
take every other call) give the same results and refuse the same calls."""
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


@pytest.fixture(params=["compiled", "python"])
def way(request, vh, monkeypatch):
    if request.param == "python":
        monkeypatch.setattr(vh, "_compiled", False)
    elif not vh._compiled_calls():
        pytest.fail("the compiled marshalling has not been built")
    return request.param


def made(seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    d = dict(x=torch.randn(6, 528, generator=g, device="cuda").to(BF), r=torch.randn(6, 528, generator=g, device="cuda").to(BF),
             w=torch.randn(528, generator=g, device="cuda").to(BF), t=torch.arange(6, device="cuda", dtype=torch.int32))
    d["W"] = torch.randn(300, 528, generator=g, device="cuda").to(BF)
    return d


def all_calls(vh, d):
    """Every call with everything given."""
    e = torch.empty_like
    f = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    out = []
    x, r, w, t, W = d["x"], d["r"], d["w"], d["t"], d["W"]
    out += vh.add_rmsnorm(x, r, w, 1e-5, 1.0, y=e(x), h=e(x))
    out += vh.add_rmsnorm(x, None, None, y=e(x))
    out += vh.add_rmsnorm(x, r, w.float(), y=e(x), h=r.clone())
    out += vh.add_rmsnorm_q8(x, r, w, q=torch.empty(6, 528, dtype=torch.int8, device="cuda"), scales=f(6), h=e(x))
    out += vh.add_rmsnorm_q8(x, None, w, q=torch.empty(6, 528, dtype=torch.float8_e4m3fn, device="cuda"), scales=f(6))
    ws = vh.add_rmsnorm_grad_workspace(6, 528)
    out += vh.add_rmsnorm_grad(x, r, w, dh=x, dx=e(x), dweight=f(528), ws=ws)
    out += vh.add_rmsnorm_grad(x, r, None, dx=e(x))[:1]
    for n in (0, 4):
        o = dict(logprob=f(6), entropy=f(6), lse=f(6), top_ids=torch.empty(6, n, dtype=torch.int32, device="cuda"),
                 top_logprobs=f(6, n))
        got = vh.logits_logprobs(x, t, n, ws=vh.logits_logprobs_workspace(6, 528, n), **o)
        assert all(a is b for a, b in zip(got, o.values()))
        out += [q.clone() for q in got]
        out += [q.clone() for q in vh.head_logprobs(x, W, t, n, ws=vh.head_logprobs_workspace(6, 300, n), **o)]
        assert vh.logits_logprobs(x, None, n, ws=vh.logits_logprobs_workspace(6, 528, n), **o)[0] is None
        assert vh.head_logprobs(x, W, None, n, ws=vh.head_logprobs_workspace(6, 300, n), **o)[0] is None
    one = torch.ones(6, device="cuda")
    wide = torch.zeros(6, 600, dtype=BF, device="cuda")
    out += [vh.logits_logprobs_grad(x, t, one * 6, one, one, one, dlogits=e(x)),
            vh.logits_logprobs_grad(x, None, one * 6, one, None, one, dlogits=wide[:, :528]).contiguous(),
            vh.logits_logprobs_grad(x, t, one * 6, None, one, None, dlogits=e(x))]
    return out


def test_same_results(vh, way, request):
    d = made()
    got = all_calls(vh, d)
    vh_compiled, vh._compiled = vh._compiled, False
    try:
        want = all_calls(vh, d)
    finally:
        vh._compiled = vh_compiled
    assert len(got) == len(want)
    for a, b in zip(got, want):
        assert a.dtype == b.dtype and torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_current_stream_is_used(vh, way):
    d = made(1)
    y, h = torch.empty_like(d["x"]), torch.empty_like(d["x"])
    vh.add_rmsnorm(d["x"], d["r"], d["w"], y=y, h=h)
    want = y.clone()
    torch.cuda.synchronize()
    y.zero_()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(200_000)
        vh.add_rmsnorm(d["x"], d["r"], d["w"], y=y, h=h)
    s.synchronize()
    assert torch.equal(y, want)


def test_refusals(vh, way):
    d = made()
    x, r, w, t = d["x"], d["r"], d["w"], d["t"]
    y = torch.empty_like(x)
    for bad in (dict(y=y.float()), dict(y=y[:, :8]), dict(y=y.cpu()), dict(y=y, h=y[:3])):
        with pytest.raises(ValueError):
            vh.add_rmsnorm(x, r, w, **bad)
    with pytest.raises(ValueError):
        vh.add_rmsnorm(x, r, w[:7], y=y, h=y)
    with pytest.raises(ValueError):
        vh.add_rmsnorm(x.double(), None, None, y=y.double())
    with pytest.raises(vh.VHError) as e:
        vh.add_rmsnorm(x, r, w, -1.0, y=y, h=torch.empty_like(x))
    assert e.value.status == vh.VH_ERR_SHAPE
    with pytest.raises(vh.VHError) as e:
        vh.add_rmsnorm_grad(x, r, w, dx=y, dweight=torch.empty(528, device="cuda"),
                            ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == vh.VH_ERR_WORKSPACE
    with pytest.raises(ValueError):
        vh.add_rmsnorm_grad(x, r, None, dx=y, dweight=torch.empty(528, device="cuda"))
    one = torch.ones(6, device="cuda")
    o = dict(logprob=one, entropy=one.clone(), lse=one.clone(), top_ids=torch.empty(6, 2, dtype=torch.int32, device="cuda"),
             top_logprobs=torch.empty(6, 2, device="cuda"))
    ws = vh.logits_logprobs_workspace(6, 528, 2)
    with pytest.raises(ValueError):
        vh.logits_logprobs(x, t.long(), 2, ws=ws, **o)
    with pytest.raises(ValueError):
        vh.logits_logprobs(x, t, 2, ws=ws.float(), **o)
    with pytest.raises(ValueError):
        vh.logits_logprobs(x, t, 3, ws=ws, **o)
    with pytest.raises(vh.VHError) as e:
        vh.logits_logprobs(x, t, 2, ws=ws[:64].clone(), **o)
    assert e.value.status == vh.VH_ERR_WORKSPACE
    with pytest.raises(ValueError):
        vh.head_logprobs(x, d["W"][:, :512], t, 2, ws=ws, **o)
    with pytest.raises(ValueError):
        vh.logits_logprobs_grad(x, t, one, None, one[:3], None, dlogits=y)
    with pytest.raises(vh.VHError) as e:
        vh.logits_logprobs_grad(x, None, one, None, one, None, dlogits=y)
    assert e.value.status == vh.VH_ERR_NULL
