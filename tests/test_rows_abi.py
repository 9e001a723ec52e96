"""Argument checks of the norm and log-probability entry points (CPU: refused
before any device access) and the sizes of their workspaces."""
import pytest

P = 0x10000  # aligned, never dereferenced


@pytest.fixture(scope="module")
def vh():
    import verify_head_gb300 as vh
    vh.build()
    return vh


def norm(vh, **kw):
    a = dict(x=P, r=P, w=P, dtype=1, w32=0, T=2, H=64, xs=64, rs=64, eps=1e-6, off=0.0, y=P, ys=64, out=0, h=P, hs=64,
             s=P, stream=None)
    a.update(kw)
    return vh.lib().vh_add_rmsnorm(*a.values())


def norm_grad(vh, **kw):
    a = dict(dy=P, h=P, w=P, dh=P, dtype=1, w32=0, T=2, H=64, dys=64, hs=64, dhs=64, eps=1e-6, off=0.0, dx=P, dxs=64,
             dw=P, ws=P, wsb=512, stream=None)
    a.update(kw)
    return vh.lib().vh_add_rmsnorm_grad(*a.values())


def lp(vh, **kw):
    a = dict(x=P, dtype=0, R=2, V=100, xs=100, t=P, n=3, lp=P, e=P, lse=P, ti=P, tl=P, ws=P, wsb=1 << 20, stream=None)
    a.update(kw)
    return vh.lib().vh_logits_logprobs(*a.values())


def lp_grad(vh, **kw):
    a = dict(x=P, dtype=0, R=2, V=100, xs=100, t=P, lse=P, e=P, gl=P, ge=P, d=P, ds=100, stream=None)
    a.update(kw)
    return vh.lib().vh_logits_logprobs_grad(*a.values())


def head(vh, **kw):
    a = dict(x=P, W=P, t=P, R=2, H=64, V=100, n=3, lp=P, e=P, lse=P, ti=P, tl=P, ws=P, wsb=1 << 24, stream=None)
    a.update(kw)
    return vh.lib().vh_head_logprobs(*a.values())


def test_null(vh):
    for call, names in ((norm, ("x", "y")), (norm_grad, ("dy", "h", "dx", "ws")), (lp, ("x", "t", "ti", "tl", "ws")),
                        (lp_grad, ("x", "lse", "d", "t", "e")), (head, ("x", "W", "t", "ti", "tl", "ws"))):
        for n in names:
            assert call(vh, **{n: None}) == vh.VH_ERR_NULL, (call.__name__, n)
    assert norm(vh, out=1, s=None) == vh.VH_ERR_NULL


def test_shape(vh):
    for kw in (dict(T=0), dict(H=0), dict(H=(1 << 24) + 1), dict(xs=63), dict(rs=63), dict(ys=63), dict(hs=63),
               dict(dtype=3), dict(dtype=-1), dict(out=3), dict(eps=-1.0), dict(eps=float("nan")),
               dict(eps=float("inf")), dict(off=float("nan"))):
        assert norm(vh, **kw) == vh.VH_ERR_SHAPE, kw
    for kw in (dict(T=0), dict(H=0), dict(dys=63), dict(hs=63), dict(dhs=63), dict(dxs=63), dict(dtype=9), dict(eps=-1.0)):
        assert norm_grad(vh, **kw) == vh.VH_ERR_SHAPE, kw
    for kw in (dict(R=0), dict(V=0), dict(xs=99), dict(n=-1), dict(n=33), dict(dtype=3), dict(V=2 ** 31 - 1, xs=2 ** 31)):
        assert lp(vh, **kw) == vh.VH_ERR_SHAPE, kw
    for kw in (dict(R=0), dict(V=0), dict(xs=99), dict(ds=99), dict(dtype=3)):
        assert lp_grad(vh, **kw) == vh.VH_ERR_SHAPE, kw
    for kw in (dict(R=0), dict(V=0), dict(H=24), dict(H=0), dict(H=65552), dict(n=33), dict(V=2 ** 31 - 1)):
        assert head(vh, **kw) == vh.VH_ERR_SHAPE, kw


def test_alignment(vh):
    for n in ("x", "r", "w", "y", "h"):
        assert norm(vh, **{n: P + 1}) == vh.VH_ERR_ALIGN, n
    assert norm(vh, w32=1, w=P + 2) == vh.VH_ERR_ALIGN
    assert norm(vh, out=1, s=P + 2) == vh.VH_ERR_ALIGN
    for n in ("dy", "h", "w", "dh", "dx"):
        assert norm_grad(vh, **{n: P + 1}) == vh.VH_ERR_ALIGN, n
    assert norm_grad(vh, ws=P + 8) == vh.VH_ERR_ALIGN
    for n in ("x", "t", "lp", "e", "lse", "ti", "tl"):
        assert lp(vh, **{n: P + 2}) == vh.VH_ERR_ALIGN, n
    assert lp(vh, ws=P + 8) == vh.VH_ERR_ALIGN
    for n in ("x", "t", "lse", "e", "gl", "ge", "d"):
        assert lp_grad(vh, **{n: P + 2}) == vh.VH_ERR_ALIGN, n
    for n, off in (("x", 8), ("W", 16), ("t", 2), ("lp", 2), ("e", 2), ("lse", 2), ("ti", 2), ("tl", 2), ("ws", 8)):
        assert head(vh, **{n: P + off}) == vh.VH_ERR_ALIGN, n


def test_workspaces(vh):
    L = vh.lib()
    assert L.vh_add_rmsnorm_grad_workspace_bytes(0, 5) == 0
    assert L.vh_add_rmsnorm_grad_workspace_bytes(2, 64) == 512
    assert norm_grad(vh, wsb=511) == vh.VH_ERR_WORKSPACE
    for size in (L.vh_logits_logprobs_workspace_bytes, L.vh_head_logprobs_workspace_bytes):
        assert size(0, 5, 1) == 0 and size(1, 0, 1) == 0 and size(1, 5, 33) == 0 and size(1, 5, -1) == 0
        assert 0 < size(1, 5, 0) <= size(1, 5, 1) and size(4, 1000, 3) % 16 == 0
    assert lp(vh, wsb=L.vh_logits_logprobs_workspace_bytes(2, 100, 3) - 1) == vh.VH_ERR_WORKSPACE
    assert head(vh, wsb=L.vh_head_logprobs_workspace_bytes(2, 100, 3) - 1) == vh.VH_ERR_WORKSPACE
    # alternatives of many rows: the blocks of one pass of 1,024 rows, past 32 bits
    assert L.vh_head_logprobs_workspace_bytes(5000, 2_000_000, 1) > 1024 * 2_000_000 * 4


def test_valid_calls_without_gpu_report_the_device(vh):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present; the device check passes")
    for call in (norm, norm_grad, lp, lp_grad, head):
        assert call(vh) == vh.VH_ERR_DEVICE
    assert norm(vh, r=None, w=None, h=None) == vh.VH_ERR_DEVICE
    assert norm_grad(vh, w=None, dh=None, dw=None, ws=None, wsb=0) == vh.VH_ERR_DEVICE
    assert lp(vh, t=None, lp=None, e=None, lse=None, n=0, ti=None, tl=None) == vh.VH_ERR_DEVICE
    assert lp_grad(vh, t=None, gl=None) == vh.VH_ERR_DEVICE and lp_grad(vh, e=None, ge=None) == vh.VH_ERR_DEVICE


def test_binding_refuses_cpu_tensors(vh):
    import torch
    x = torch.zeros(2, 64)
    t = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: vh.add_rmsnorm(x), lambda: vh.add_rmsnorm_q8(x), lambda: vh.add_rmsnorm_grad(x, x),
                 lambda: vh.logits_logprobs(x, t), lambda: vh.logits_logprobs_grad(x, t, x[:, 0]),
                 lambda: vh.head_logprobs(x.bfloat16(), x.bfloat16(), t)):
        with pytest.raises(ValueError):
            call()
