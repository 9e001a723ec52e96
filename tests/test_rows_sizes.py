"""Sizes past 32 bits are refused by the binding, not passed on by their low 32 bits."""
import pytest
import torch

PAST = 2 ** 32 + 3


@pytest.fixture(scope="module")
def vh():
    import verify_head_gb300 as vh
    vh.build()
    return vh


@pytest.mark.parametrize("args", [(PAST, 5, 1), (5, PAST, 1), (5, 5, PAST), (2 ** 31, 5, 1), (5, 5, -PAST)])
def test_workspaces(vh, args):
    for make in (vh.logits_logprobs_workspace, vh.head_logprobs_workspace):
        with pytest.raises(ValueError):
            make(*args, device="cpu")


@pytest.mark.parametrize("args", [(PAST, 8), (8, PAST), (2 ** 31, 8)])
def test_grad_workspace(vh, args):
    with pytest.raises(ValueError):
        vh.add_rmsnorm_grad_workspace(*args, device="cpu")


def test_sizes_within_32_bits_pass(vh):
    assert vh.logits_logprobs_workspace(3, 100, 2, device="cpu").numel() > 0
    assert vh.add_rmsnorm_grad_workspace(3, 100, device="cpu").numel() > 0


@pytest.mark.gpu
@pytest.mark.parametrize("given", [False, True])
def test_calls(vh, given):
    """One-column rows, one of whose sizes is past 32 bits."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    x = torch.empty(PAST, 1, dtype=torch.float16, device="cuda")
    x[:3] = 2.0
    y = torch.zeros_like(x) if given else None
    with pytest.raises(ValueError):
        vh.add_rmsnorm(x, None, None, y=y)
    with pytest.raises(ValueError):
        vh.add_rmsnorm_grad(x, x, None, dx=y)
    assert y is None or float(y[:3].abs().max()) == 0.0
    t = torch.zeros(1, dtype=torch.int32, device="cuda")
    wide = x.view(1, PAST)
    with pytest.raises(ValueError):
        vh.logits_logprobs(wide, t)
    with pytest.raises(ValueError):
        vh.logits_logprobs_grad(wide, t, t.float(), t.float(), t.float(), dlogits=y.view(1, PAST) if given else None)
    with pytest.raises(ValueError):
        vh.logits_logprobs(wide[:, :100], t, 2 ** 32)


@pytest.mark.gpu
def test_most_rows(vh):
    """2^31 - 1 rows: the launch's rounding up to whole blocks stays within 32 bits."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    x = torch.empty(2 ** 31 - 1, 1, dtype=torch.float16, device="cuda")
    x.fill_(2.0)
    x[-1] = -3.0
    y = torch.zeros_like(x)
    vh.add_rmsnorm(x, None, None, 1e-6, y=y)
    # 2 / sqrt(4 + eps) and -3 / sqrt(9 + eps) round to 1 and -1 in 16 bits
    assert float(y[-1]) == -1.0 and bool((y[:-1] == 1.0).all())
