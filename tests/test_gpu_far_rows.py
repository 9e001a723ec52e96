"""Log probabilities of rows whose largest score lies far from zero: masks of -1e9, -1e10, -1e30 or the type's lowest
value throughout a row, and maxima that grow across the magnitude where the statistics change their formula."""
import math

import pytest
import torch

from rows_util import close, logprobs64, sums

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def vh():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import verify_head_gb300 as vh
    vh.build()
    return vh


def check(got, x, tokens, n):
    lp, ent, lse, ids, top = logprobs64(x, tokens, n)
    V = x.shape[1]
    floor = sums(V) + 2.0 ** -20  # of ln s; x - c is exact here or rounded once
    close(got[0], lp, 2.0 ** -22, floor)
    close(got[1], ent, 2.0 ** -22, 20 * sums(V))
    close(got[2], lse, 2.0 ** -22, floor)
    if n:
        assert torch.equal(got[3].cpu(), ids)
        close(got[4], top, 2.0 ** -22, floor)


FAR = [-1e6, -1e9, -3e9, -1e10, -1e12, -1e20, -1e30, -1e38, 1e6, 3e9, 1e12, 1e30, 2e38]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [7, 1000, 40001])
@pytest.mark.parametrize("n", [0, 3])
def test_rows_filled_with_one_far_value(vh, V, n, dtype):
    x = torch.tensor(FAR)[:, None].expand(len(FAR), V).to(dtype).contiguous().cuda()
    x[:, V // 3] = -math.inf
    tokens = torch.arange(len(FAR), dtype=torch.int32) % V
    check(vh.logits_logprobs(x, tokens.cuda(), n), x, tokens, n)


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("V", [700, 33333])
def test_far_masks_beside_scores(vh, V, dtype):
    """Part of a row masked with a far value: those places carry nothing, whatever the value is."""
    g = torch.Generator().manual_seed(V)
    masks = [-6e4] if dtype == HF else [-1e6, -1e10, -1e30, -3e38]
    x = (torch.randn(2 * len(masks), V, generator=g) * 2).to(dtype)
    for i, m in enumerate(masks):
        x[i, torch.rand(V, generator=g) < 0.6] = m
        x[len(masks) + i, : V - 5] = m  # nothing else until the row's end
    tokens = torch.randint(0, V, (x.shape[0],), generator=g, dtype=torch.int32)
    x = x.cuda()
    check(vh.logits_logprobs(x, tokens.cuda(), 4), x, tokens, 4)


@pytest.mark.parametrize("at", [2.0 ** 17, 2.0 ** 19, 2.0 ** 20, 2.0 ** 21, 2.0 ** 23])
@pytest.mark.parametrize("sign", [1, -1])
def test_maxima_that_grow_across_a_far_value(vh, at, sign):
    """Neighbouring values around `at`, each carrying weight, with the maximum last, first and in the middle."""
    V = 9000
    step = max(at * 2.0 ** -23, 2.0 ** -7)
    ramp = sign * at + (torch.arange(V, dtype=torch.float64) - V // 2) * step * (16 / step / V if step < 0.01 else 1)
    ramp = ramp.float()
    x = torch.stack([ramp, ramp.flip(0), ramp.roll(V // 2 + 3)]).cuda()
    tokens = torch.tensor([V - 1, 1, 5], dtype=torch.int32)
    check(vh.logits_logprobs(x, tokens.cuda(), 5), x, tokens, 5)


@pytest.mark.parametrize("R", [3, 200])
@pytest.mark.parametrize("scale", [2.0 ** 21, 2.0 ** 34, 2.0 ** 100])
@pytest.mark.parametrize("sign", [1, -1])
def test_head_scores_far_from_zero(vh, R, scale, sign):
    V, H = 3001, 64
    x = torch.zeros(R, H, dtype=BF, device="cuda")
    x[:, 0] = sign * scale
    W = torch.zeros(V, H, dtype=BF, device="cuda")
    W[:, 0] = 1.0
    W[::3, 0] = 1.5
    tokens = (torch.arange(R) % V).int()
    got = vh.head_logprobs(x, W, tokens.cuda(), 4)
    check(got, x.double() @ W.double().t(), tokens, 4)
