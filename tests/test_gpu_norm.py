"""Residual addition with RMS norm, its 8-bit form and its gradient against the
64-bit definitions: row widths inside and outside registers, odd widths,
strided and misaligned rows, in-place outputs, zero, infinite and NaN rows."""
import math

import pytest
import torch

from rows_util import TINY, U, close, norm64, norm_grad64, sums

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


def rows(g, T, H, dtype, scale=1.0, pitch=None, offset=0):
    """A [T,H] CUDA tensor, its rows `pitch` elements apart, starting `offset` elements into its storage."""
    pitch = pitch or H
    flat = torch.zeros(T * pitch + offset + 16, dtype=dtype, device="cuda")
    t = flat[offset:offset + T * pitch].view(T, pitch)[:, :H]
    t.copy_((torch.randn(T, H, generator=g) * scale).to(dtype))
    return t


# widths: one element, under a warp, odd, exact vectors, each register variant, past the registers
SHAPES = [(1, 1), (3, 7), (5, 64), (2, 255), (4, 2048), (1, 2560), (7, 2561), (3, 4104), (2, 8192), (130, 257),
          (2, 16384), (1, 16392), (2, 20001), (1, 65536)]


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("T,H", SHAPES)
def test_norm_matches_definition(vh, T, H, dtype):
    g = gen(T * 1000 + H)
    x, r = rows(g, T, H, dtype), rows(g, T, H, dtype, 2.0)
    w = (1 + 0.1 * torch.randn(H, generator=g)).to(dtype).cuda()
    y, h = vh.add_rmsnorm(x, r, w, 1e-6)
    want_y, want_h = norm64(x, r, w, 1e-6, 0.0)
    close(h, want_h, U[dtype] * (1 + 2 ** -10) + 2.0 ** -24, TINY[dtype])
    close(y, want_y, U[dtype] * (1 + 2 ** -10) + sums(H), TINY[dtype])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("w32", [False, True])
@pytest.mark.parametrize("residual", [False, True])
def test_weight_forms(vh, dtype, w32, residual):
    g = gen(5)
    T, H = 9, 1000
    x = rows(g, T, H, dtype)
    r = rows(g, T, H, dtype) if residual else None
    w = (0.1 * torch.randn(H, generator=g)).to(F32 if w32 else dtype).cuda()
    y, h = vh.add_rmsnorm(x, r, w, 1e-5, weight_offset=1.0)
    want_y, want_h = norm64(x, r, w, 1e-5, 1.0)
    close(y, want_y, U[dtype] * (1 + 2 ** -10) + sums(H), TINY[dtype])
    if residual:
        close(h, want_h, U[dtype] * (1 + 2 ** -10) + 2.0 ** -24, TINY[dtype])
    else:
        assert h is x
    y, _ = vh.add_rmsnorm(x, r, None, 1e-5)
    close(y, norm64(x, r, None, 1e-5, 0.0)[0], U[dtype] * (1 + 2 ** -10) + sums(H), TINY[dtype])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H,pitch,offset", [(256, 256, 1), (256, 264, 0), (256, 260, 0), (2048, 2056, 8), (33, 40, 3),
                                            (20000, 20016, 0), (20000, 20001, 0)])
def test_strides_and_alignment(vh, dtype, H, pitch, offset):
    g = gen(H + pitch)
    T = 6
    x = rows(g, T, H, dtype, pitch=pitch, offset=offset)
    r = rows(g, T, H, dtype, pitch=pitch)
    w = torch.randn(H, generator=g).to(dtype).cuda()
    y = rows(g, T, H, dtype, pitch=pitch, offset=offset)
    guard = y.storage_offset(), y.untyped_storage().nbytes()
    whole = torch.empty(0, dtype=dtype, device="cuda").set_(y.untyped_storage())
    before = whole.clone()
    got, h = vh.add_rmsnorm(x, r, w, 1e-6, y=y, h=r)  # h on the residual
    assert got is y and h is r and guard == (y.storage_offset(), y.untyped_storage().nbytes())
    g = gen(H + pitch)
    x0 = rows(g, T, H, dtype, pitch=pitch, offset=offset)
    r0 = rows(g, T, H, dtype, pitch=pitch)
    want_y, want_h = norm64(x0, r0, w, 1e-6, 0.0)
    close(y, want_y, U[dtype] * (1 + 2 ** -10) + sums(H), TINY[dtype])
    close(r, want_h, U[dtype] * (1 + 2 ** -10) + 2.0 ** -24, TINY[dtype])
    mask = torch.ones_like(whole, dtype=torch.bool)
    mask.as_strided((T, H), (pitch, 1), y.storage_offset()).fill_(False)
    assert torch.equal(whole[mask], before[mask])  # nothing beside the rows was written


def test_rows_past_32_bits(vh):
    """Rows more than 2^31 elements apart."""
    H, pitch = 2048, 1_500_000_000
    flat = torch.empty(2 * pitch + H, dtype=BF, device="cuda")
    x = flat.as_strided((3, H), (pitch, 1))
    x.copy_(torch.randn(3, H, generator=gen(1)).to(BF))
    w = torch.randn(H, generator=gen(2)).to(BF).cuda()
    near = x.contiguous()
    want = vh.add_rmsnorm(near, near, w)
    q = vh.add_rmsnorm_q8(x, near, w)
    dx, dw = vh.add_rmsnorm_grad(near, x, w, dh=x)
    want_dx, want_dw = vh.add_rmsnorm_grad(near, near, w, dh=near)
    assert torch.equal(dx, want_dx) and torch.equal(dw, want_dw)
    assert torch.equal(q[0], vh.add_rmsnorm_q8(near, near, w)[0])
    y, h = vh.add_rmsnorm(x, near, w, h=x)
    assert torch.equal(y, want[0]) and torch.equal(x, want[1])


@pytest.mark.parametrize("H", [2048, 20001])
def test_output_on_an_input(vh, H):
    g = gen(H)
    x, r = rows(g, 5, H, BF), rows(g, 5, H, BF)
    w = torch.randn(H, generator=g).to(BF).cuda()
    y0, h0 = vh.add_rmsnorm(x, r, w)
    x1 = x.clone()
    y1, h1 = vh.add_rmsnorm(x1, r, w, y=x1)
    assert torch.equal(y0, y1) and torch.equal(h0, h1)
    x2 = x.clone()
    y2, h2 = vh.add_rmsnorm(x2, r, w, h=x2)
    assert torch.equal(y0, y2) and torch.equal(h0, h2)


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("out", [torch.int8, torch.float8_e4m3fn])
@pytest.mark.parametrize("T,H", [(1, 1), (4, 7), (3, 2048), (5, 2561), (130, 96), (2, 16384), (2, 30000)])
def test_q8(vh, T, H, dtype, out):
    g = gen(T + H)
    x, r = rows(g, T, H, dtype), rows(g, T, H, dtype, 3.0)
    w = (1 + 0.1 * torch.randn(H, generator=g)).to(dtype).cuda()
    q, s, h = vh.add_rmsnorm_q8(x, r, w, 1e-6, dtype=out)
    want_y, want_h = norm64(x, r, w, 1e-6, 0.0)
    top = 127.0 if out == torch.int8 else 448.0
    close(h, want_h, U[dtype] * (1 + 2 ** -10) + 2.0 ** -24, TINY[dtype])
    close(s, want_y.abs().max(1).values / top, sums(H), 0.0)
    # the codes are those of the 32-bit formula, step by step (each step is one rounding, so any order agrees)
    u = (x.float() + r.float()) * w.float()
    v = u * (top / u.abs().amax(1, keepdim=True))
    want_q = torch.round(v).to(torch.int8) if out == torch.int8 else v.to(out)
    assert torch.equal(q.view(torch.int8), want_q.view(torch.int8))
    # and stand for the normed rows: half a code (int8), half a unit of three mantissa bits or of 2^-9 (e4m3)
    err = (q.double() * s.double()[:, None] - want_y).abs()
    step = 0.5 if out == torch.int8 else torch.clamp(v.double().abs() * 2.0 ** -4, min=2.0 ** -10)
    assert bool((err <= s.double()[:, None] * step * (1 + 1e-3) + want_y.abs() * sums(H)).all())


@pytest.mark.parametrize("out", [torch.int8, torch.float8_e4m3fn])
def test_q8_codes_of_many_rows(vh, out):
    """Enough codes for near ties: each step's rounding is part of the definition (a fused one is off in 3 of 10^7)."""
    T, H = 16384, 2048
    x = torch.randn(T, H, generator=torch.Generator("cuda").manual_seed(1), device="cuda").to(BF)
    w = (1 + 0.1 * torch.randn(H, generator=gen(2))).to(BF).cuda()
    q, _, _ = vh.add_rmsnorm_q8(x, None, w, 1e-6, dtype=out)
    u = x.float() * w.float()
    top = 127.0 if out == torch.int8 else 448.0
    v = u * (top / u.abs().amax(1, keepdim=True))
    want = torch.round(v).to(torch.int8) if out == torch.int8 else v.to(out)
    assert int((q.view(torch.int8) != want.view(torch.int8)).sum()) == 0


@pytest.mark.parametrize("H", [640, 24001])
def test_special_rows(vh, H):
    x = torch.zeros(6, H, dtype=F32, device="cuda")
    x[1, 3] = math.inf
    x[2, H - 1] = math.nan
    x[3] = 1e-38      # squares underflow, Q / max|u| would overflow
    x[4, 5] = -0.0
    x[5] = 1.0
    w = torch.ones(H, device="cuda")
    y, h = vh.add_rmsnorm(x, None, w, 1e-6)
    assert not torch.isfinite(y[1]).all() and torch.isnan(y[1, 3]) and float(y[1, 0]) == 0.0
    assert torch.isnan(y[2]).all()
    assert torch.equal(y[0], torch.zeros(H, device="cuda")) and torch.equal(y[4], y[0])
    close(y[5:], torch.ones(1, H, dtype=torch.float64) / math.sqrt(1 + 1e-6), sums(H) + 2.0 ** -24, 0.0)
    for out, top in ((torch.int8, 127), (torch.float8_e4m3fn, 448)):
        q, s, _ = vh.add_rmsnorm_q8(x, None, w, 1e-6, dtype=out)
        assert float(s[0]) == 0.0 and float(s[4]) == 0.0 and bool((q[0].float() == 0).all())
        assert math.isnan(float(s[1])) and math.isnan(float(s[2]))
        assert bool((q[3].float() == top).all()) and bool((q[5].float() == top).all())
        close(s[3:4], torch.tensor([1e-38 / math.sqrt(1e-6) / top], dtype=torch.float64), 1e-3, 0.0)


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("T,H", [(1, 1), (3, 7), (4, 2048), (700, 96), (9, 2561), (1300, 256), (5, 8192), (3, 8200),
                                 (2, 40001)])
@pytest.mark.parametrize("dh", [False, True])
def test_grad_matches_formula(vh, T, H, dtype, dh):
    g = gen(T * 7 + H)
    h, dy = rows(g, T, H, dtype, 2.0), rows(g, T, H, dtype)
    e = rows(g, T, H, dtype) if dh else None
    w = (1 + 0.1 * torch.randn(H, generator=g)).to(dtype).cuda()
    dx, dw = vh.add_rmsnorm_grad(dy, h, w, 1e-6, dh=e)
    want_dx, want_dw = norm_grad64(dy, h, w, e, 1e-6, 0.0)
    # dx = rstd g - rstd n mean(g n) + dh: the errors of its terms add up, and mean(g n) is a sum of both signs
    hd, gd = h.double(), dy.double() * w.double()
    rstd = 1 / torch.sqrt((hd * hd).mean(1, keepdim=True) + 1e-6)
    n = hd * rstd
    size = rstd * (gd.abs() + n.abs() * (gd * n).abs().mean(1, keepdim=True))
    close(dx, want_dx, U[dtype] * (1 + 2 ** -10) + 2.0 ** -24, size * sums(H) * 2 + TINY[dtype])
    # a column of dw: up to T / 608 terms one after the other in a CTA, then 608 / 16 shares, then 16
    close(dw, want_dw, 2.0 ** -24, (dy.double() * n).abs().sum(0) * (T / 608 + 80 + sums(H) * 2 ** 24) * 2.0 ** -24)


@pytest.mark.parametrize("H,pitch,offset", [(256, 264, 0), (256, 257, 1), (9000, 9008, 0)])
def test_grad_strides_in_place_and_forms(vh, H, pitch, offset):
    g = gen(pitch)
    T = 11
    h, dy = rows(g, T, H, F32, pitch=pitch, offset=offset), rows(g, T, H, F32, pitch=pitch, offset=offset)
    w = torch.randn(H, generator=g).cuda()
    dx, dw = vh.add_rmsnorm_grad(dy, h, w, 1e-5, weight_offset=1.0)
    want_dx, want_dw = norm_grad64(dy, h, w, None, 1e-5, 1.0)
    scale = float(want_dx.abs().max())
    close(dx, want_dx, 0.0, scale * sums(H) * 4)
    close(dw, want_dw, 0.0, float(want_dw.abs().max()) * sums(H) * 4)
    same, none = vh.add_rmsnorm_grad(dy, h, None, 1e-5)
    assert none is None
    close(same, norm_grad64(dy, h, None, None, 1e-5, 0.0)[0], 0.0, scale * sums(H) * 4)
    again, dw2 = vh.add_rmsnorm_grad(dy, h, w, 1e-5, weight_offset=1.0, dx=dy)  # on its input
    assert again is dy and torch.equal(dy, dx) and torch.equal(dw, dw2)


def test_grad_matches_differences(vh):
    g = gen(3)
    T, H = 3, 40
    h, dy, e = (torch.randn(T, H, generator=g) for _ in range(3))
    w = 1 + 0.3 * torch.randn(H, generator=g)
    dx, dw = vh.add_rmsnorm_grad(dy.cuda(), h.cuda(), w.cuda(), 1e-3, dh=e.cuda())

    def loss(hh, ww):
        return float((norm64(hh, None, ww, 1e-3, 0.0)[0] * dy.double()).sum() + (hh * e.double()).sum())

    step = 1e-5  # central differences in 64 bits: error about step^2 + 1e-16 / step
    for t, i in [(0, 0), (0, 39), (1, 7), (2, 20)]:
        d = torch.zeros(T, H, dtype=torch.float64)
        d[t, i] = step
        want = (loss(h.double() + d, w) - loss(h.double() - d, w)) / (2 * step)
        assert abs(float(dx[t, i]) - want) < 1e-5
    for i in (0, 13, 39):
        d = torch.zeros(H, dtype=torch.float64)
        d[i] = step
        want = (loss(h.double(), w.double() + d) - loss(h.double(), w.double() - d)) / (2 * step)
        assert abs(float(dw[i]) - want) < 1e-5


def test_same_call_same_bits_and_other_stream(vh):
    g = gen(8)
    T, H = 1500, 512
    h, dy = rows(g, T, H, BF), rows(g, T, H, BF)
    w = torch.randn(H, generator=g).to(BF).cuda()
    dx, dw = vh.add_rmsnorm_grad(dy, h, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        dx2, dw2 = vh.add_rmsnorm_grad(dy, h, w, stream=s)
        y2, _ = vh.add_rmsnorm(h, dy, w, stream=s)
    s.synchronize()
    y, _ = vh.add_rmsnorm(h, dy, w)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2) and torch.equal(y, y2)


def test_graph_capture(vh):
    g = gen(9)
    x, r = rows(g, 4, 2048, BF), rows(g, 4, 2048, BF)
    w = torch.randn(2048, generator=g).to(BF).cuda()
    y, h = torch.empty_like(x), torch.empty_like(x)
    vh.add_rmsnorm(x, r, w, y=y, h=h)
    want = y.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vh.add_rmsnorm(x, r, w, y=y, h=h)
    y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)


def test_refusals(vh):
    x = torch.zeros(2, 8, device="cuda")
    with pytest.raises(ValueError):
        vh.add_rmsnorm(x, torch.zeros(2, 9, device="cuda"))
    with pytest.raises(ValueError):
        vh.add_rmsnorm(x, torch.zeros(2, 8, device="cuda", dtype=BF))
    with pytest.raises(ValueError):
        vh.add_rmsnorm(x, None, torch.zeros(7, device="cuda"))
    with pytest.raises(ValueError):
        vh.add_rmsnorm(x.double())
    with pytest.raises(ValueError):
        vh.add_rmsnorm(torch.zeros(8, 2, device="cuda").t())
    with pytest.raises(ValueError):
        vh.add_rmsnorm(x, torch.zeros(2, 8))
    with pytest.raises(ValueError):
        vh.add_rmsnorm_q8(x, dtype=torch.uint8)
    with pytest.raises(vh.VHError):
        vh.add_rmsnorm(torch.zeros(0, 8, device="cuda"))
    with pytest.raises(vh.VHError):
        vh.add_rmsnorm(torch.zeros(1, 8, device="cuda").expand(3, 8))  # rows on one another
    with pytest.raises(vh.VHError):
        vh.add_rmsnorm(x, eps=-1.0)
    with pytest.raises(ValueError):
        vh.add_rmsnorm_grad(x, x, torch.zeros(8, device="cuda"), dx=torch.zeros(2, 8, device="cuda", dtype=BF))
    with pytest.raises(vh.VHError):
        vh.add_rmsnorm_grad(x, x, torch.zeros(8, device="cuda"), ws=torch.zeros(16, dtype=torch.uint8, device="cuda"))


def outside_unchanged(t, before):
    """Nothing beside the rows of t was written."""
    whole = torch.empty(0, dtype=t.dtype, device="cuda").set_(t.untyped_storage())
    mask = torch.ones_like(whole, dtype=torch.bool)
    mask.as_strided(t.shape, t.stride(), t.storage_offset()).fill_(False)
    return torch.equal(whole.view(torch.uint8 if t.element_size() == 1 else t.dtype)[mask], before[mask])


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("H,pitch,offset", [(1, 1, 3), (3, 5, 1), (9, 9, 7), (255, 255, 5), (520, 521, 2), (2561, 2561, 7),
                                            (4105, 4107, 1), (8185, 8185, 6), (16369, 16371, 3), (16383, 16383, 1)])
@pytest.mark.parametrize("w32", [False, True])
def test_rows_that_lie_alike(vh, dtype, H, pitch, offset, w32):
    """Rows of any alignment, the same for every tensor: 16-byte slots across the rows' ends, weights at an offset."""
    T = 9
    g = gen(H + pitch + offset)
    x, r = (rows(g, T, H, dtype, s, pitch=pitch, offset=offset) for s in (1.0, 2.0))
    w = torch.randn(H + 3, generator=g).to(F32 if w32 else dtype).cuda()[3:]
    want_y, want_h = norm64(x, r, w, 1e-6, 0.0)
    y, h = (rows(g, T, H, dtype, pitch=pitch, offset=offset) for _ in range(2))
    whole = [torch.empty(0, dtype=dtype, device="cuda").set_(t.untyped_storage()).clone() for t in (y, h)]
    vh.add_rmsnorm(x, r, w, 1e-6, y=y, h=h)
    close(h, want_h, U[dtype] * (1 + 2 ** -10) + 2.0 ** -24, TINY[dtype])
    close(y, want_y, U[dtype] * (1 + 2 ** -10) + sums(H), TINY[dtype])
    assert outside_unchanged(y, whole[0]) and outside_unchanged(h, whole[1])
    # the same values wherever the rows lie, up to the order of the squares' sum
    apart = vh.add_rmsnorm(x.contiguous(), r.contiguous(), w, 1e-6)
    assert torch.equal(h, apart[1])
    close(y, apart[0].double(), 2 * U[dtype] * (1 + 2 ** -10) + sums(H), TINY[dtype])
    # codes
    flat = torch.full((T * pitch + offset + 16,), 77, dtype=torch.int8, device="cuda")
    before = flat.clone()
    q = flat[offset:offset + T * pitch].view(T, pitch)[:, :H]
    _, s, _ = vh.add_rmsnorm_q8(x, r, w, 1e-6, q=q, h=h)
    u = (x.float() + r.float()) * w.float()
    assert torch.equal(q, torch.round(u * (127.0 / u.abs().amax(1, keepdim=True))).to(torch.int8))
    assert outside_unchanged(q, before)
    close(s, want_y.abs().max(1).values / 127.0, sums(H), 0.0)
    # outputs on the inputs: a slot that two rows share is written by both
    vh.add_rmsnorm(x, r, w, 1e-6, y=x, h=r)
    assert torch.equal(x, y) and torch.equal(r, h)


def test_grad_and_norm_of_ragged_batch(vh):
    """Many rows of an odd width, no residual, no weights."""
    g = gen(5)
    x = rows(g, 3001, 1027, HF)
    y = vh.add_rmsnorm(x, None, None, 1e-6)[0]
    close(y, norm64(x, None, None, 1e-6, 0.0)[0], U[HF] * (1 + 2 ** -10) + sums(1027), TINY[HF])


def grad_close(dx, dw, want_dx, want_dw, dy, h, w, dtype):
    """The bounds of test_grad_matches_formula."""
    T, H = h.shape
    hd, gd = h.double(), dy.double() * w.double()
    rstd = 1 / torch.sqrt((hd * hd).mean(1, keepdim=True) + 1e-6)
    n = hd * rstd
    size = rstd * (gd.abs() + n.abs() * (gd * n).abs().mean(1, keepdim=True))
    close(dx, want_dx, U[dtype] * (1 + 2 ** -10) + 2.0 ** -24, size * sums(H) * 2 + TINY[dtype])
    close(dw, want_dw, 2.0 ** -24, (dy.double() * n).abs().sum(0) * (T / 152 + 80 + sums(H) * 2 ** 24) * 2.0 ** -24)


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("T,H,pitch,offset", [(1, 1, 1, 3), (5, 3, 5, 1), (9, 9, 9, 7), (700, 255, 255, 5), (7, 520, 522, 2),
                                              (4999, 129, 129, 1), (1301, 2561, 2561, 7), (17, 4105, 4108, 1),
                                              (650, 8185, 8185, 6), (3, 16369, 16371, 3)])
@pytest.mark.parametrize("dh", [False, True])
def test_grad_of_rows_that_lie_alike(vh, dtype, T, H, pitch, offset, dh):
    """Rows of any alignment, the same for every tensor; rows shorter than their slot's rest; nothing else is written."""
    g = gen(T + H + offset)
    dy, h, e = (rows(g, T, H, dtype, pitch=pitch, offset=offset) for _ in range(3))
    for t in (dy, h, e):  # what lies beside the rows is no number
        whole = torch.empty(0, dtype=dtype, device="cuda").set_(t.untyped_storage())
        mask = torch.ones_like(whole, dtype=torch.bool)
        mask.as_strided((T, H), (pitch, 1), offset).fill_(False)
        whole[mask] = float("nan")
    w = torch.randn(H + 1, generator=g).to(dtype).cuda()[1:]
    dx = rows(g, T, H, dtype, pitch=pitch, offset=offset)
    before = torch.empty(0, dtype=dtype, device="cuda").set_(dx.untyped_storage()).clone()
    _, dw = vh.add_rmsnorm_grad(dy, h, w, 1e-6, dh=e if dh else None, dx=dx)
    want_dx, want_dw = norm_grad64(dy, h, w, e if dh else None, 1e-6, 0.0)
    grad_close(dx, dw, want_dx, want_dw, dy, h, w, dtype)
    assert outside_unchanged(dx, before)
    # dx on dy: a slot that two rows share is read by both and written by both
    vh.add_rmsnorm_grad(dy, h, w, 1e-6, dh=e if dh else None, dx=dy)
    assert torch.equal(dy, dx)
