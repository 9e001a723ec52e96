"""Rows to 4 bits and back on the GPU: the host encoder's bytes for every type, width, stride and scale, numbers on and next
to the borders between codes, numbers that are none; values exactly; the tiled layout place by place."""
import numpy as np
import pytest
import torch

import w4_util as u

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def vh():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import verify_head_gb300 as vh
    vh.build()
    return vh


@pytest.fixture(scope="module")
def synth():
    import synth
    synth.build()
    return synth


def rows(seed, T, H, dtype, pitch=None, offset=0, size=1.0):
    g = torch.Generator().manual_seed(seed)
    pitch = pitch or H
    flat = torch.full((T * pitch + offset + 32,), 6e4, dtype=dtype, device="cuda")  # a read past a row would show
    t = flat[offset:offset + T * pitch].view(T, pitch)[:, :H]
    x = torch.randn(T, H, generator=g) * torch.exp(torch.randn(T, 1, generator=g)) * size
    x[:, ::7] *= 0.01
    t.copy_(x.to(dtype))
    return t


def encoded(synth, x, g):
    """(codes, scales) of the host encoder, row by row with that row's scale."""
    x = x.float().cpu().numpy()
    if np.ndim(g) == 0:
        q, s, _ = synth.nvfp4_quantize(x, float(g))
        return q, s
    q = np.zeros((x.shape[0], x.shape[1] // 2), np.uint8)
    s = np.zeros((x.shape[0], x.shape[1] // 16), np.uint8)
    for r in range(x.shape[0]):
        if g[r] > 0:
            q[r:r + 1], s[r:r + 1], _ = synth.nvfp4_quantize(x[r:r + 1], float(g[r]))
    return q, s


def check(vh, synth, x, g):
    T, H = x.shape
    q, s, rs = vh.nvfp4_quantize(x, g)
    if g is None:
        want = x.float().cpu().abs().amax(1) / torch.full((T,), 2688.0)  # the quotient, rounded once
        assert torch.equal(rs.cpu(), want)
        g = want.numpy()
    else:
        assert rs is None
        g = np.float32(g)
    wq, ws = encoded(synth, x, g)
    assert np.array_equal(s.cpu().numpy(), ws)
    assert np.array_equal(q.cpu().numpy(), wq)
    # the tiled layout of the same bytes, made directly and from the row-major one; lines past T left alone, or zero
    t = torch.full((vh.vh_nvfp4_tiles_bytes(T, H),), 0xA5, dtype=torch.uint8, device="cuda")
    _, rs2 = vh.nvfp4_quantize_tiles(x, None if rs is not None else float(g), tiles=t)
    assert rs is None or torch.equal(rs, rs2)
    assert np.array_equal(t.cpu().numpy(), u.tile(q, s, 0xA5))
    assert np.array_equal(vh.nvfp4_tile(q, s).cpu().numpy(), u.tile(q, s))
    return q, s, rs


SHAPES = [(1, 16), (5, 48), (3, 256), (2, 272), (130, 64), (4, 2048), (7, 2576), (33, 4096), (2, 8208), (1, 65536)]


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("T,H", SHAPES)
def test_bytes_of_the_host_encoder(vh, synth, T, H, dtype):
    for seed, (pitch, offset) in enumerate([(H, 0), (H + 16, 0), (H + 3, 5), (H + 8, 8)]):
        x = rows(seed, T, H, dtype, pitch, offset)
        check(vh, synth, x, None)
        check(vh, synth, x, [0.003, 2.0 ** -9, 1e-3, 0.02][seed])


@pytest.mark.parametrize("g", [1.4e-45, 3e-42, 1e-38, 5e-20, 2.0 ** -64, 1e-6, 1.0, 37.5, 2.0 ** 64, 1e20, 1e33, 3e38])
def test_scales_of_every_size(vh, synth, g):
    """Including those whose product with a block scale, or its reciprocal, is past fp32's range."""
    gf = float(np.float32(g))
    x = rows(3, 4, 512, F32)
    for size in (gf, gf * 500, gf * 1e-3):
        check(vh, synth, (x.double() * size).clamp(-3.4e38, 3.4e38).float(), gf)
    check(vh, synth, (x.double() * gf * 300).clamp(-3.4e38, 3.4e38).float(), None)
    check(vh, synth, x, gf)


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("g", [2.0 ** -6, 0.0123, 0.7])
def test_on_and_next_to_the_borders(vh, synth, dtype, g):
    """Every border of the codes and of the block scales, its neighbours in the type, both signs."""
    gf = np.float32(g)
    out = []
    for code in (1, 7, 8, 9, 13, 60, 77, 126):
        s = u.E4M3[code]
        step = float(gf) * s
        b = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64) * step
        for d in (0, 1, -1):
            near = b.to(dtype)
            for _ in range(abs(d)):
                near = torch.nextafter(near.float(), torch.tensor(d * 1e30)).to(dtype) if dtype == F32 else \
                    (near.view(torch.int16) + d).view(dtype)
            blk = torch.zeros(16, dtype=dtype)
            blk[:7], blk[7:14] = near, -near
            blk[15] = torch.tensor(6 * step, dtype=torch.float64).to(dtype)
            out.append(blk)
    # largest magnitudes on the borders between two block scales
    for code in (0, 1, 5, 8, 20, 100, 125):
        mid = (u.E4M3[code] + u.E4M3[code + 1]) / 2 * 6 * float(gf)
        m = torch.tensor([mid], dtype=torch.float64).to(dtype)
        for d in (0, 1, -1):
            v = (m.view(torch.int16) + d).view(dtype) if dtype != F32 else (m.view(torch.int32) + d).view(dtype)
            blk = (torch.rand(16, generator=torch.Generator().manual_seed(code)) * float(v) * 0.9).to(dtype)
            blk[code % 16] = v
            out.append(blk)
    x = torch.cat(out)
    x = torch.cat([x, torch.zeros(-len(x) % 64, dtype=dtype)]).view(-1, 32).cuda()
    check(vh, synth, x, float(gf))


@pytest.mark.parametrize("dtype", [BF, HF, F32])
def test_rows_that_are_zero_or_no_numbers(vh, dtype):
    x = rows(9, 6, 64, dtype)
    x[0] = 0
    x[1, 3], x[2, 40], x[3, 63] = float("nan"), float("inf"), -float("inf")
    q, s, rs = vh.nvfp4_quantize(x)
    assert float(rs[0]) == 0 and torch.isnan(rs[1:4]).all() and torch.isfinite(rs[4:]).all()
    assert int(q[:4].sum()) == 0 and int(s[:4].sum()) == 0
    q, s, _ = vh.nvfp4_quantize(x, 0.01)
    bad = torch.zeros(6, 4, dtype=torch.bool)
    bad[1, 0], bad[2, 2], bad[3, 3] = True, True, True
    assert torch.equal((s == 0x7F).cpu(), bad)
    assert int(q.view(6, 4, 8)[bad].sum()) == 0
    y = vh.nvfp4_dequantize(q, s, 0.01, dtype=F32)
    assert torch.equal(torch.isnan(y).view(6, 4, 16).all(2).cpu(), bad) and torch.equal(torch.isnan(y).view(6, 4, 16).any(2).cpu(), bad)
    assert not torch.signbit(vh.nvfp4_dequantize(*vh.nvfp4_quantize(-torch.full((1, 16), 1e-3, device="cuda").index_fill(
        1, torch.tensor([0], device="cuda"), 6.0), 1.0)[:2], 1.0, dtype=F32))[0, 1:].any()  # a zero has no sign


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("T,H", [(1, 16), (3, 48), (130, 272), (5, 2048), (301, 2576)])
def test_values(vh, T, H, dtype):
    g = torch.Generator().manual_seed(T)
    codes = torch.randint(0, 256, (T, H // 2), generator=g, dtype=torch.uint8).cuda()
    scales = torch.randint(0, 127, (T, H // 16), generator=g, dtype=torch.uint8).cuda()
    rs = torch.rand(T, generator=g).cuda()
    v = torch.from_numpy(u.values64(codes, scales)).float()  # exact
    for scale in (0.37, rs):
        want = (v * (torch.tensor(scale, dtype=F32) if scale is not rs else rs.cpu()[:, None])).to(dtype)  # one rounding each
        wide = torch.full((T, H + 24), 7.0, dtype=dtype, device="cuda")
        for out in (torch.empty(T, H, dtype=dtype, device="cuda"), wide[:, 8:H + 8], wide[:, 3:H + 3]):
            wide.fill_(7.0)
            assert vh.nvfp4_dequantize(codes, scales, scale, out=out) is out
            assert torch.equal(out.cpu(), want)
            if out.data_ptr() != wide.data_ptr() and out.stride(0) != H:
                assert int((wide == 7.0).sum()) >= T * 24  # the rest of the rows
        tiles = torch.from_numpy(u.tile(codes, scales, 0xFF)).cuda()
        assert torch.equal(vh.nvfp4_dequantize_tiles(tiles, scale, T, H, dtype=dtype).cpu(), want)


def test_heads_take_the_rows(vh, synth):
    """A candidate table made on the GPU scores as one made on the host."""
    w = torch.randn(700, 512, generator=torch.Generator().manual_seed(5)) * 0.02
    g = float(w.abs().max()) / 2688
    q, s, _ = vh.nvfp4_quantize(w.cuda(), g)
    hq, hs, _ = synth.nvfp4_quantize(w.numpy(), float(np.float32(g)))
    assert np.array_equal(q.cpu().numpy(), hq) and np.array_equal(s.cpu().numpy(), hs)
    x = torch.randn(3, 512, generator=torch.Generator().manual_seed(6)).to(BF).cuda()
    ids = torch.arange(700, dtype=torch.int32, device="cuda")
    got, ml = vh.mtp_draft_head_argmax_nvfp4(x, q, s, g, ids)
    scores = x.double().cpu() @ torch.from_numpy(u.values64(q, s)).t() * float(np.float32(g))
    assert float((ml.double().cpu() - scores.max(1).values).abs().max()) < 1e-3
    assert torch.equal(scores.gather(1, got.long().cpu()[:, None])[:, 0] >= scores.max(1).values - 1e-3, torch.ones(3, dtype=torch.bool))


def test_refusals(vh):
    x = torch.zeros(4, 64, dtype=BF, device="cuda")
    q, s, _ = vh.nvfp4_quantize(x, 1.0)
    t = vh.nvfp4_tile(q, s)
    for bad in (lambda: vh.nvfp4_quantize(x.cpu(), 1.0), lambda: vh.nvfp4_quantize(x[0], 1.0), lambda: vh.nvfp4_quantize(x.int(), 1.0),
                lambda: vh.nvfp4_quantize(x.t(), 1.0), lambda: vh.nvfp4_quantize(x, 1.0, codes=q[:3]),
                lambda: vh.nvfp4_quantize(x, 1.0, scales=s.int()), lambda: vh.nvfp4_quantize(x, 1.0, row_scales=torch.zeros(4, device="cuda")),
                lambda: vh.nvfp4_quantize(x, row_scales=torch.zeros(3, device="cuda")), lambda: vh.nvfp4_quantize_tiles(x, 1.0, tiles=t[:-1]),
                lambda: vh.nvfp4_tile(q, s[:, :2]), lambda: vh.nvfp4_tile(q, s, tiles=t[1:]), lambda: vh.nvfp4_dequantize(q, s[:3], 1.0),
                lambda: vh.nvfp4_dequantize(q, s, torch.zeros(3, device="cuda")), lambda: vh.nvfp4_dequantize(q, s, 1.0, out=x[:3]),
                lambda: vh.nvfp4_dequantize(q, s, 1.0, out=x, dtype=F32), lambda: vh.nvfp4_dequantize_tiles(t[:100], 1.0, 4, 64),
                lambda: vh.nvfp4_dequantize(q, s, 1.0, out=x.int())):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: vh.nvfp4_quantize(x[:, :24], 1.0), lambda: vh.nvfp4_quantize(x, 0.0), lambda: vh.nvfp4_quantize(x, float("nan")),
                lambda: vh.nvfp4_dequantize(q, s, float("inf"))):
        with pytest.raises((vh.VHError, ValueError)):
            bad()
