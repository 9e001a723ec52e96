"""64-bit definitions of the row operators (norm, log probabilities) and the
tolerances that follow from the kernels' 32-bit sums."""
import math

import torch

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # half a unit in the last place
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}


def sums(n):
    """Relative error of an fp32 sum of n terms of one sign: a thread adds n / 256 of them one after the other, at
    most ten levels of a tree follow, and every term carries a few roundings of its own (64 in all is generous)."""
    return (n / 256 + 64) * 2.0 ** -24


def norm64(x, r, w, eps, off):
    h = x.double() + (0 if r is None else r.double())
    v = (torch.ones(x.shape[1], dtype=torch.float64, device=x.device) if w is None else w.double()) + off
    rstd = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    return h * rstd * v, h


def norm_grad64(dy, h, w, dh, eps, off):
    """By autograd of the 64-bit definition."""
    hh = h.double().requires_grad_()
    w = torch.ones(h.shape[1], dtype=torch.float64, device=h.device) if w is None else w.double()
    w.requires_grad_()
    y = hh / torch.sqrt((hh * hh).mean(1, keepdim=True) + eps) * (w + off)
    loss = (y * dy.double()).sum() + (0 if dh is None else (hh * dh.double()).sum())
    return torch.autograd.grad(loss, (hh, w))


def logprobs64(x, tokens, n):
    """(logprob, entropy, lse, ids, logprobs of the ids) of a [R,V] tensor, row by row, by the definitions:
    NaN counts as -inf, no token gives 0, a row of -inf gives -inf and entropy 0."""
    x = x.double().cpu()
    x = torch.where(torch.isnan(x), torch.full_like(x, -math.inf), x)
    R, V = x.shape
    lp, ent, lse = torch.zeros(R, dtype=torch.float64), torch.zeros(R, dtype=torch.float64), torch.empty(R, dtype=torch.float64)
    ids = torch.full((R, n), -1, dtype=torch.int32)
    top = torch.full((R, n), -math.inf, dtype=torch.float64)
    for r in range(R):
        m = x[r].max()
        if m == -math.inf:
            logp = torch.full((V,), -math.inf, dtype=torch.float64)
            lse[r] = -math.inf
        elif m == math.inf:
            logp = torch.full((V,), math.nan, dtype=torch.float64)
            lse[r] = ent[r] = math.nan
        else:
            s = torch.exp(x[r] - m).sum()
            lse[r] = m + torch.log(s)
            logp = (x[r] - m) - torch.log(s)
            p = torch.exp(logp)
            ent[r] = -torch.special.xlogy(p, p).sum()
        t = int(tokens[r])
        lp[r] = logp[t] if 0 <= t < V else 0.0
        order = torch.sort(x[r], descending=True, stable=True).indices[:n]
        ids[r, :len(order)] = order.int()
        top[r, :len(order)] = logp[order]
    return lp, ent, lse, ids, top


def logprobs_loss64(x, tokens, gl, ge):
    """sum gl * logprob + ge * entropy of float64 logits [R,V] (for gradients)."""
    logp = torch.log_softmax(x, 1)
    p = torch.exp(logp)
    given = (tokens >= 0) & (tokens < x.shape[1])
    lp = logp.gather(1, tokens.clamp(0, x.shape[1] - 1).long()[:, None])[:, 0]
    plogp = torch.where(p > 0, p * torch.where(p > 0, logp, torch.zeros_like(logp)), torch.zeros_like(p))
    return (torch.where(given, lp, torch.zeros_like(lp)) * gl).sum() - (plogp.sum(1) * ge).sum()


def close(got, want, rel, floor):
    """|got - want| <= rel |want| + floor everywhere, infinities and NaN in the same places."""
    got, want = got.double().cpu(), want.double().cpu()
    assert got.shape == want.shape
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.isinf(got), torch.isinf(want))
    assert torch.equal(got[torch.isinf(got)], want[torch.isinf(want)])
    fine = torch.isfinite(want)
    off = (got - want).abs()[fine] - (rel * want.abs() + (floor if not torch.is_tensor(floor) else floor.cpu()))[fine]
    assert off.numel() == 0 or float(off.max()) <= 0, float(off.max())
