"""Scales of 8-bit normed rows where a row or its weight is zero, infinite or NaN: 0 or NaN, never a number that passes
what the codes cannot stand for."""
import math

import pytest
import torch

from rows_util import close, norm64, sums

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
OUTS = [torch.int8, torch.float8_e4m3fn]


@pytest.fixture(scope="module")
def vh():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import verify_head_gb300 as vh
    vh.build()
    return vh


def nan(t):
    return bool(torch.isnan(t).all())


@pytest.mark.parametrize("out", OUTS)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H", [5, 640, 2561, 24001])  # each kernel's widths
def test_scales(vh, H, dtype, out):
    g = torch.Generator().manual_seed(H)
    x = torch.randn(7, H, generator=g).to(dtype).cuda()
    w = (1 + 0.1 * torch.randn(H, generator=g)).to(dtype).cuda()
    at = H // 2
    w[at] = 0.0
    x[0] = 0.0
    x[1] = 0.0
    x[1, at] = 3.0          # the weight takes all that there is
    x[2, at] = math.inf     # infinite where the weight is zero
    x[3, at] = math.nan
    x[4] = 1e30             # squares past the range of fp32
    x[5] = 0.0
    x[5, 0] = 1e-30         # squares vanish
    for eps in (0.0, 1e-6):
        q, s, _ = vh.add_rmsnorm_q8(x, None, w, eps, dtype=out)
        assert float(s[0]) == 0.0 and float(s[1]) == 0.0
        assert bool((q[0].float() == 0).all()) and bool((q[1].float() == 0).all())
        assert nan(s[2:5])
        assert float(s[5]) > 0.0 or eps == 0.0
        want = norm64(x[6:], None, w, eps, 0.0)[0].abs().max(1).values / (127 if out == torch.int8 else 448)
        close(s[6:], want, sums(H), 0.0)


@pytest.mark.parametrize("out", OUTS)
@pytest.mark.parametrize("H", [5, 640, 2561, 24001])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_weights_that_are_no_numbers(vh, H, bad, out):
    x = torch.randn(5, H, generator=torch.Generator().manual_seed(H)).to(BF).cuda()
    for at in (0, H // 2, H - 1):
        w = torch.ones(H, device="cuda")
        w[at] = bad
        assert nan(vh.add_rmsnorm_q8(x, None, w, dtype=out)[1])
        y = vh.add_rmsnorm(x, None, w)[0]
        assert not bool(torch.isfinite(y[:, at]).any())
        keep = torch.arange(H, device="cuda") != at
        assert bool(torch.isfinite(y[:, keep]).all())
