"""Argument checks of the 4-bit row and logit-processing entry points (CPU: refused before any device access)."""
import ctypes

import pytest

P = 0x10000  # aligned, never dereferenced


@pytest.fixture(scope="module")
def vh():
    import verify_head_gb300 as vh
    vh.build()
    return vh


def quantize(vh, **kw):
    a = dict(x=P, dtype=1, T=3, H=64, xs=64, g=0.5, codes=P, scales=P, rows=None, stream=None)
    a.update(kw)
    return vh.lib().vh_nvfp4_quantize(*a.values())


def tile(vh, **kw):
    a = dict(codes=P, scales=P, V=3, H=64, tiles=P, n=18432, stream=None)
    a.update(kw)
    return vh.lib().vh_nvfp4_tile(*a.values())


def dequantize(vh, **kw):
    a = dict(codes=P, scales=P, T=3, H=64, g=0.5, rows=None, dtype=1, y=P, ys=64, stream=None)
    a.update(kw)
    return vh.lib().vh_nvfp4_dequantize(*a.values())


def matmul(vh, **kw):
    a = dict(x=P, gx=1.0, gxs=None, w=P, gw=1.0, gws=None, T=3, V=50, H=64, dtype=1, y=P, ys=50, stream=None)
    a.update(kw)
    return vh.lib().vh_nvfp4_matmul(*a.values())


def rules(vh, **kw):
    r = vh.LogitsRules()
    for n, v in dict(dict(history=P, history_stride=7, history_width=7, allowed=P, allowed_stride=4, bias_ids=P, bias=P,
                          n_bias=2), **kw).items():
        setattr(r, n, v)
    return r


def process(vh, **kw):
    a = dict(x=P, dtype=1, R=6, V=100, xs=100, per=3, rules=None, y=2 * P, yt=1, ys=100, stream=None)
    r = {k: kw.pop(k) for k in list(kw) if k not in a}
    a.update(kw)
    if "rules" not in kw:
        a["rules"] = ctypes.byref(rules(vh, **r))
    return vh.lib().vh_logits_process(*a.values())


def process_grad(vh, **kw):
    a = dict(d=P, x=2 * P, dtype=1, R=6, V=100, dys=100, xs=100, per=3, rules=None, y=3 * P, ys=100, stream=None)
    r = {k: kw.pop(k) for k in list(kw) if k not in a}
    a.update(kw)
    if "rules" not in kw:
        a["rules"] = ctypes.byref(rules(vh, **r))
    return vh.lib().vh_logits_process_grad(*a.values())


def test_null(vh):
    for call, names in ((quantize, ("x", "codes")), (tile, ("codes", "scales", "tiles")), (dequantize, ("codes", "y")),
                        (matmul, ("x", "w", "y")), (process, ("x", "y", "rules")), (process_grad, ("d", "x", "y", "rules"))):
        for n in names:
            assert call(vh, **{n: None}) == vh.VH_ERR_NULL, (call.__name__, n)
    for call in (process, process_grad):
        assert call(vh, bias=None) == vh.VH_ERR_NULL
        assert call(vh, bias_ids=None) == vh.VH_ERR_NULL


def test_shape(vh):
    nan, inf = float("nan"), float("inf")
    for kw in (dict(T=0), dict(H=0), dict(H=8), dict(H=72), dict(H=65552), dict(xs=63), dict(dtype=3), dict(g=0.0), dict(g=-1.0),
               dict(g=nan), dict(g=inf)):
        assert quantize(vh, **kw) == vh.VH_ERR_SHAPE, kw
    for kw in (dict(V=0), dict(H=24), dict(H=65552)):
        assert tile(vh, **kw) == vh.VH_ERR_SHAPE, kw
    for kw in (dict(T=0), dict(H=24), dict(ys=63), dict(dtype=-1), dict(g=nan), dict(g=inf)):
        assert dequantize(vh, **kw) == vh.VH_ERR_SHAPE, kw
    for kw in (dict(T=0), dict(V=0), dict(H=0), dict(H=24), dict(H=65552), dict(ys=49), dict(dtype=5), dict(gx=nan),
               dict(gw=inf), dict(V=2 ** 31 - 1, ys=2 ** 31)):
        assert matmul(vh, **kw) == vh.VH_ERR_SHAPE, kw
    for kw in (dict(R=0), dict(V=0), dict(xs=99), dict(ys=99), dict(dtype=3), dict(per=0), dict(per=4), dict(history_width=-1),
               dict(history_stride=6), dict(n_bias=-1), dict(n_bias=65536), dict(allowed_stride=3),
               dict(V=2 ** 31 - 1, xs=2 ** 31, ys=2 ** 31, allowed_stride=1 << 27)):
        assert process(vh, **kw) == vh.VH_ERR_SHAPE, kw
        assert process_grad(vh, **kw) == vh.VH_ERR_SHAPE, kw
    assert process(vh, yt=2) == vh.VH_ERR_SHAPE
    assert process(vh, y=P, ys=101) == vh.VH_ERR_SHAPE and process(vh, y=P, yt=0) == vh.VH_ERR_SHAPE
    assert process_grad(vh, y=2 * P) == vh.VH_ERR_SHAPE and process_grad(vh, y=P, ys=101) == vh.VH_ERR_SHAPE
    assert process_grad(vh, dys=99) == vh.VH_ERR_SHAPE


def test_sizes_past_the_counts(vh):
    """Rows whose numbers would pass 31 bits within a block of threads, and histories whose counts would reach the bits beside
    them."""
    n = 2 ** 31 - 1023
    assert quantize(vh, T=n) == vh.VH_ERR_SHAPE and dequantize(vh, T=n) == vh.VH_ERR_SHAPE
    assert tile(vh, V=n, n=2 ** 60) == vh.VH_ERR_SHAPE and matmul(vh, T=n) == vh.VH_ERR_SHAPE
    for call in (process, process_grad):
        assert call(vh, history_width=2 ** 28 + 1, history_stride=2 ** 29) == vh.VH_ERR_SHAPE


def test_alignment(vh):
    for kw in (dict(x=P + 1), dict(codes=P + 4), dict(codes=P + 8, scales=None), dict(rows=P + 2)):
        assert quantize(vh, **kw) == vh.VH_ERR_ALIGN, kw
    for kw in (dict(codes=P + 4), dict(tiles=P + 8)):
        assert tile(vh, **kw) == vh.VH_ERR_ALIGN, kw
    for kw in (dict(codes=P + 4), dict(codes=P + 8, scales=None), dict(rows=P + 2), dict(y=P + 1)):
        assert dequantize(vh, **kw) == vh.VH_ERR_ALIGN, kw
    for kw in (dict(x=P + 8), dict(w=P + 8), dict(gxs=P + 2), dict(gws=P + 1), dict(y=P + 1)):
        assert matmul(vh, **kw) == vh.VH_ERR_ALIGN, kw
    for kw in (dict(x=P + 1), dict(y=P + 1), dict(history=P + 2), dict(history_len=P + 2), dict(prompt_len=P + 1),
               dict(draft_ids=P + 2), dict(repetition=P + 1), dict(frequency=P + 2), dict(presence=P + 3),
               dict(temperature=P + 2), dict(bias_ids=P + 2), dict(bias=P + 1), dict(allowed=P + 2)):
        assert process(vh, **kw) == vh.VH_ERR_ALIGN, kw
        assert process_grad(vh, **kw) == vh.VH_ERR_ALIGN, kw
    assert process(vh, yt=0, y=P + 2) == vh.VH_ERR_ALIGN
    assert process_grad(vh, d=P + 1) == vh.VH_ERR_ALIGN


def test_tiles_bytes(vh):
    n = vh.vh_nvfp4_tiles_bytes
    assert n(1, 16) == 18432 and n(128, 256) == 18432 and n(129, 256) == 2 * 18432 and n(128, 272) == 2 * 18432
    assert n(248320, 2048) == 1940 * 8 * 18432
    assert n(0, 256) == 0 and n(1, 24) == 0 and n(1, 65552) == 0 and n(2 ** 31 - 1, 65536) > 2 ** 40
    assert tile(vh, n=18431) == vh.VH_ERR_WORKSPACE
    with pytest.raises(ValueError):
        n(1, 2 ** 32 + 16)


def test_no_device_is_no_abort(vh):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a device is there")
    for call in (quantize, tile, dequantize, matmul, process, process_grad):
        assert call(vh) == vh.VH_ERR_DEVICE, call.__name__
