"""The norm's gradient of rows that begin and end inside a 16-byte granule: the ends of the tensor, which are stored
element by element into the ring that the rest of the row is copied to, and rows that lie differently in each tensor."""
import pytest
import torch

from rows_util import TINY, U, close, norm_grad64, sums

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def vh():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import verify_head_gb300 as vh
    vh.build()
    return vh


def rows(g, T, H, dtype, scale=1.0, pitch=None, offset=0):
    """A [T,H] CUDA tensor with rows `pitch` apart and `offset` elements into its storage; NaN beside the rows."""
    pitch = pitch or H
    flat = torch.full((T * pitch + offset + 16,), float("nan"), dtype=dtype, device="cuda")
    t = flat[offset:offset + T * pitch].view(T, pitch)[:, :H]
    t.copy_((torch.randn(T, H, generator=g) * scale).to(dtype))
    return t


def check(dx, dw, dy, h, w, e, dtype):
    """dx = rstd g - rstd n mean(g n) + dh: the errors of its terms add up; dw: a sum over tokens in three steps."""
    want_dx, want_dw = norm_grad64(dy, h, w, e, 1e-6, 0.0)
    T, H = h.shape
    hd, gd = h.double(), dy.double() * w.double()
    rstd = 1 / torch.sqrt((hd * hd).mean(1, keepdim=True) + 1e-6)
    n = hd * rstd
    size = rstd * (gd.abs() + n.abs() * (gd * n).abs().mean(1, keepdim=True))
    close(dx, want_dx, U[dtype] * (1 + 2 ** -10) + 2.0 ** -24, size * sums(H) * 2 + TINY[dtype])
    close(dw, want_dw, 2.0 ** -24, (dy.double() * n).abs().sum(0) * (T / 152 + 80 + sums(H) * 2 ** 24) * 2.0 ** -24)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,H", [(1, 21), (2, 1029), (3, 2561)])
def test_ends_of_the_tensor_every_time(vh, T, H, dtype):
    """Nothing but first and last tokens, again and again with other values."""
    g = torch.Generator().manual_seed(H)
    w = torch.randn(H, generator=g).to(dtype).cuda()
    for i in range(40):
        dy, h, e = (rows(g, T, H, dtype, offset=1 + i % 7) for _ in range(3))
        dx, dw = vh.add_rmsnorm_grad(dy, h, w, 1e-6, dh=e)
        check(dx, dw, dy, h, w, e, dtype)


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("H", [1, 2, 3, 5, 7, 9])
@pytest.mark.parametrize("T", [1, 2, 4, 9, 40])
def test_rows_shorter_than_a_granule(vh, T, H, dtype):
    """Several tokens in the tensor's first and last granule."""
    g = torch.Generator().manual_seed(T * 10 + H)
    w = torch.randn(H, generator=g).to(dtype).cuda()
    for pitch, offset in ((H, 0), (H, 1), (H, 3), (H + 1, 2)):
        dy, h, e = (rows(g, T, H, dtype, pitch=pitch, offset=offset) for _ in range(3))
        dx, dw = vh.add_rmsnorm_grad(dy, h, w, 1e-6, dh=e)
        check(dx, dw, dy, h, w, e, dtype)


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("T,H", [(1, 1), (9, 5), (700, 33), (2, 255), (300, 257), (13, 2561), (5, 4096), (5, 4097), (1, 8191),
                                 (3, 8192), (2, 8200)])
@pytest.mark.parametrize("which", ["dy", "dh", "pitch"])
def test_rows_that_lie_differently(vh, T, H, dtype, which):
    """One tensor of another alignment, or of rows another distance apart, than the rest."""
    g = torch.Generator().manual_seed(T * 7 + H)
    dy = rows(g, T, H, dtype, offset=3 if which == "dy" else 1)
    h = rows(g, T, H, dtype, 2.0, offset=1)
    e = rows(g, T, H, dtype, offset=2 if which == "dh" else 1, pitch=H + 3 if which == "pitch" else None)
    w = (1 + 0.1 * torch.randn(H + 1, generator=g)).to(dtype).cuda()[1:]
    dx = rows(g, T, H, dtype, pitch=H + 5, offset=1)
    whole = torch.empty(0, dtype=dtype, device="cuda").set_(dx.untyped_storage())
    whole.fill_(7.0)
    _, dw = vh.add_rmsnorm_grad(dy, h, w, 1e-6, dh=e, dx=dx)
    check(dx, dw, dy, h, w, e, dtype)
    mask = torch.ones_like(whole, dtype=torch.bool)
    mask.as_strided((T, H), (H + 5, 1), 1).fill_(False)
    assert bool((whole[mask] == 7.0).all())  # nothing beside the rows was written
    if which != "pitch":
        assert torch.equal(vh.add_rmsnorm_grad(dy, h, w, 1e-6, dh=e, dx=dy)[0], dx)  # on its input
    alone, none = vh.add_rmsnorm_grad(rows(g, T, H, dtype, offset=5), h, None, 1e-6)
    assert none is None and bool(torch.isfinite(alone.float()).all())


@pytest.mark.parametrize("H", [8186, 8187, 8190, 8191])
def test_widest_single_precision_rows(vh, H):
    """On either side of the widest rows that go by slots."""
    g = torch.Generator().manual_seed(H)
    w = (1 + 0.1 * torch.randn(H, generator=g)).cuda()
    for T in (1, 7, 400):
        dy, h, e = (rows(g, T, H, F32, s) for s in (1.0, 2.0, 1.0))
        dx, dw = vh.add_rmsnorm_grad(dy, h, w, 1e-6, dh=e)
        check(dx, dw, dy, h, w, e, F32)
