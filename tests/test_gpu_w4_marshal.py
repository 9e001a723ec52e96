"""The 4-bit and logit-processing calls through the compiled marshalling and through the Python checks: the same results, the same
refusals, the current stream; and calls of several threads at once."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
T, V, H = 6, 300, 528


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


def made(vh, seed=0, T=T, V=V, H=H):
    g = torch.Generator("cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    i = lambda hi, *s: torch.randint(0, hi, s, generator=g, device="cuda", dtype=torch.int32)  # noqa: E731
    d = dict(x=n(T, H).to(BF), w=n(V, H), logits=n(T, V).to(BF), d=n(T, V).to(BF))
    S = T // 3
    d["rules"] = dict(history=i(V, S, 40), history_len=i(40, S), prompt_len=i(20, S), draft_ids=i(V, S, 2), repetition=n(S).abs() + 0.5,
                      frequency=n(S), presence=n(S), bias_ids=i(V, S, 4), bias=n(S, 4), allowed=i(2 ** 31 - 1, T, (V + 31) // 32),
                      temperature=n(S).abs() + 0.5)
    d["wt"], d["ws"] = vh.nvfp4_quantize_tiles(d["w"])
    return d


def all_calls(vh, d):
    e = lambda *s: torch.zeros(*s, device="cuda", dtype=torch.uint8)  # noqa: E731
    f = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    out = []
    x = d["x"]
    for g, rs in ((None, f(T)), (0.01, None)):
        codes, scales, got = vh.nvfp4_quantize(x, g, codes=e(T, H // 2), scales=e(T, H // 16), row_scales=rs)
        assert got is rs
        tiles, got = vh.nvfp4_quantize_tiles(x, g, tiles=e(vh.vh_nvfp4_tiles_bytes(T, H)), row_scales=rs)
        s = g if rs is None else rs
        out += [codes, scales, tiles] + ([rs.clone()] if rs is not None else [])
        wide = torch.zeros(T, H + 8, device="cuda")
        out += [vh.nvfp4_dequantize(codes, scales, s, out=torch.empty_like(x)), vh.nvfp4_dequantize(codes, scales, s, out=wide[:, :H]).clone()]
        out += [vh.nvfp4_matmul(tiles, s, d["wt"], d["ws"], T, V, H, out=f(T, V)),
                vh.nvfp4_matmul(tiles, s, d["wt"], 0.5, T, V, H, out=torch.zeros(T, V, device="cuda", dtype=BF))]
    lg, r = d["logits"], d["rules"]
    for rules in (r, {}, {k: r[k] for k in ("temperature", "allowed")}, {k: r[k] for k in ("history", "repetition")}):
        out += [vh.logits_process(lg, out=torch.empty_like(lg), **rules), vh.logits_process(lg, out=f(T, V), **rules)]
        same = lg.clone()
        assert vh.logits_process(same, out=same, **rules) is same
        out += [same, vh.logits_process_grad(d["d"], lg, dlogits=torch.empty_like(lg), **rules)]
    return out


def test_same_results(vh, way):
    d = made(vh)
    got = all_calls(vh, d)
    was, vh._compiled = vh._compiled, False
    try:
        want = all_calls(vh, d)
    finally:
        vh._compiled = was
    assert len(got) == len(want)
    for a, b in zip(got, want):
        assert a.dtype == b.dtype and torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def test_current_stream_is_used(vh, way):
    d = made(vh, 1)
    calls = [lambda o: vh.logits_process(d["logits"], out=o[0], **d["rules"]),
             lambda o: vh.logits_process_grad(d["d"], d["logits"], dlogits=o[0], **d["rules"]),
             lambda o: vh.nvfp4_matmul(d["wt"], 1.0, d["wt"], 1.0, T, V, H, out=o[0]),
             lambda o: vh.nvfp4_quantize_tiles(d["x"], 0.5, tiles=o[1])]
    out = torch.zeros(T, V, dtype=BF, device="cuda"), torch.zeros(vh.vh_nvfp4_tiles_bytes(T, H), dtype=torch.uint8, device="cuda")
    for call in calls:
        call(out)
        want = [o.clone() for o in out]
        for o in out:
            o.zero_()
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            torch.cuda._sleep(200_000)
            call(out)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        for o in out:
            o.zero_()
        torch.cuda.synchronize()


def test_refusals(vh, way):
    d = made(vh)
    x, lg, r = d["x"], d["logits"], d["rules"]
    n = vh.vh_nvfp4_tiles_bytes(T, H)
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
    tiles, codes, scales, rs = u8(n), u8(T, H // 2), u8(T, H // 16), torch.zeros(T, device="cuda")
    y = torch.zeros(T, V, device="cuda")
    bad = [lambda: vh.nvfp4_quantize(x, None, codes=codes[:, :8], scales=scales, row_scales=rs),
           lambda: vh.nvfp4_quantize(x, None, codes=codes, scales=scales[:3], row_scales=rs),
           lambda: vh.nvfp4_quantize(x, None, codes=codes, scales=scales.float(), row_scales=rs),
           lambda: vh.nvfp4_quantize(x, None, codes=codes, scales=scales, row_scales=rs[:5]),
           lambda: vh.nvfp4_quantize(x, None, codes=codes.cpu(), scales=scales, row_scales=rs),
           lambda: vh.nvfp4_quantize(x.double(), 1.0, codes=codes, scales=scales),
           lambda: vh.nvfp4_quantize_tiles(x, 1.0, tiles=tiles[:-1]), lambda: vh.nvfp4_quantize_tiles(x, None, tiles=tiles, row_scales=rs.half()),
           lambda: vh.nvfp4_dequantize(codes, scales, rs[:5], out=x.clone()), lambda: vh.nvfp4_dequantize(codes, scales, 1.0, out=x[:, :-1]),
           lambda: vh.nvfp4_dequantize(codes, scales[:, :-1], 1.0, out=x.clone()),
           lambda: vh.nvfp4_matmul(tiles, rs[:5], d["wt"], 1.0, T, V, H, out=y), lambda: vh.nvfp4_matmul(tiles, 1.0, tiles, 1.0, T, V, H, out=y),
           lambda: vh.nvfp4_matmul(tiles, 1.0, d["wt"], 1.0, T, V, H, out=y[:, :-1]), lambda: vh.nvfp4_matmul(tiles, 1.0, d["wt"], 1.0, T, V, H, out=y.double()),
           lambda: vh.nvfp4_matmul(tiles.cpu(), 1.0, d["wt"], 1.0, T, V, H, out=y),
           lambda: vh.logits_process(lg, out=lg.half(), **r), lambda: vh.logits_process(lg, out=y[:3], **r),
           lambda: vh.logits_process(lg, out=y, **dict(r, draft_ids=None, frequency=r["frequency"][:1])),
           lambda: vh.logits_process(lg, out=y, **dict(r, bias=None)), lambda: vh.logits_process(lg, out=y, **dict(r, allowed=r["allowed"][:, 1:])),
           lambda: vh.logits_process(lg, out=y, **dict(r, history=r["history"].long())),
           lambda: vh.logits_process(lg, out=y, **dict(r, history=r["history"].t())),
           lambda: vh.logits_process_grad(d["d"].float(), lg, dlogits=lg.clone(), **r),
           lambda: vh.logits_process_grad(d["d"], lg, dlogits=y, **r), lambda: vh.logits_process_grad(d["d"][:3], lg, dlogits=lg.clone(), **r)]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(str(i))
    for call in (lambda: vh.nvfp4_quantize_tiles(x, 0.0, tiles=tiles), lambda: vh.nvfp4_dequantize(codes, scales, float("nan"), out=x.clone()),
                 lambda: vh.nvfp4_matmul(tiles, float("inf"), d["wt"], 1.0, T, V, H, out=y),
                 lambda: vh.logits_process_grad(d["d"], lg, dlogits=lg, **r)):
        with pytest.raises(vh.VHError) as e:
            call()
        assert e.value.status == vh.VH_ERR_SHAPE


def test_threads(vh):
    """Sizes on both sides of every choice of kernel, a stream each, over and over."""
    sizes = [(3, 257, 256), (48, 2000, 1040), (300, 5003, 512), (3, 40001, 2048), (33, 70003, 272), (6, 300, 16384)]
    jobs = []
    for k, (t, v, h) in enumerate(sizes):
        d = made(vh, k, t, v, h)
        xt, xs = vh.nvfp4_quantize_tiles(d["x"])
        jobs.append((d, xt, xs, t, v, h, torch.cuda.Stream()))
    torch.cuda.synchronize()
    wrong = []

    def step(job):
        d, _, _, t, v, h, _ = job
        xt, xs = vh.nvfp4_quantize_tiles(d["x"])
        y = vh.nvfp4_matmul(xt, xs, d["wt"], d["ws"], t, v, h, dtype=BF)
        p = vh.logits_process(y, **d["rules"])
        return y, p, vh.logits_process_grad(d["d"], y, **d["rules"])

    want = [step(j) for j in jobs]
    torch.cuda.synchronize()

    def run(job, right):
        try:
            with torch.cuda.stream(job[-1]):
                for _ in range(40):
                    got = step(job)
                    same = torch.stack([(a.view(torch.int16) == b.view(torch.int16)).all() for a, b in zip(got, right)])
                    if not bool(same.all()):
                        wrong.append((job[3:6], same.tolist()))
        except Exception as e:  # noqa: BLE001 - reported below
            wrong.append(repr(e))

    threads = [threading.Thread(target=run, args=a) for a in zip(jobs, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong
