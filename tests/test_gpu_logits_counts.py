"""Counts of tokens in the processing of logits, to the one: tolerances for each place from what is added up there, so that a draft
or a token of the history that is lost or counted twice is seen, in every kernel and with histories of any length.  On the CPU the same
tolerances against a definition with one such mistake."""
import math

import numpy as np
import pytest
import torch

import w4_util as u
from rows_util import TINY, U

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32

# sequences, rows of each, vocabulary, history: small calls with short and long histories (16-bit and 32-bit counts); large ones with
# each size of table, tables by tokens, and the long histories that are changed in registers
CASES = [(1, 4, 40001, 1500), (3, 2, 5003, 9000), (2, 3, 20011, 50000), (64, 4, 40001, 500), (64, 4, 40001, 3000), (70, 4, 40001, 9000),
         (70, 4, 40001, 40000), (170, 1, 70003, 6000)]


@pytest.fixture(scope="module")
def vh():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import verify_head_gb300 as vh
    vh.build()
    return vh


def case(S, m, V, L, dtype, seed=0):
    """Logits and rules on the CPU.  A count more or less moves a place by a frequency of 0.5 and more."""
    g = torch.Generator().manual_seed(seed + V + L)
    ints = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, dtype=torch.int32)  # noqa: E731
    x = (torch.randn(S * m, V, generator=g) * 3).to(dtype)
    r = dict(history=ints(-2, V + 2, S, L), history_len=ints(max(1, L // 2), L, S), prompt_len=ints(0, max(1, L // 2), S),
             repetition=0.8 + torch.rand(S, generator=g), frequency=0.5 + torch.rand(S, generator=g),
             presence=0.25 + torch.rand(S, generator=g) / 2, temperature=0.5 + torch.rand(S, generator=g))
    r["temperature"][1::3] = 0.0
    r["history"][:, ::7] = r["history"][:, :1].clamp(0, V - 1).clone()
    if m > 1:
        r["draft_ids"] = ints(0, V, S, m - 1)
        r["draft_ids"][:, 1::2] = r["history"][:, :1]
    return x, r


def part(x, r, s, m):
    """One sequence of a call."""
    return x[s * m:(s + 1) * m], {k: v[s:s + 1] for k, v in r.items()}


def tolerance(x, r, m, out_dtype):
    """Of one sequence, place by place.  Of |z| the roundings (2^-24 each) are those of the penalty and of two differences, of
    frequency * n its own and two, of presence one; then 1 / T and its product: six at most of what is added up, eight with what second
    orders may add.  Then the rounding to the type, of the value itself (added by `off`)."""
    V = x.shape[1]
    h = r["history"][0, :max(0, int(r["history_len"][0]))].cpu().numpy()
    p = max(0, int(r["prompt_len"][0]))
    rep, t = float(r["repetition"][0]), float(r["temperature"][0])
    rows = []
    for j in range(m):
        out = np.concatenate([h[p:], r["draft_ids"][0, :j].cpu().numpy()]) if m > 1 else h[p:]
        n = torch.from_numpy(np.bincount(out[(out >= 0) & (out < V)], minlength=V)).double()
        rows.append(x[j].cpu().double().abs() * max(rep, 1 / rep) + float(r["frequency"][0]) * n + float(r["presence"][0]) * (n > 0))
    return torch.stack(rows) / (t if t > 0 else 1.0) * 8 * 2.0 ** -24 + TINY[out_dtype]


def off(got, want, floor, dtype):
    """By how much the largest difference passes its tolerance."""
    return float(((got.cpu().double() - want).abs() - floor - U[dtype] * want.abs()).max())


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("S,m,V,L", CASES)
def test_one_mistake_is_seen(S, m, V, L, dtype):
    """The definition with one token dropped or added passes the tolerance that the kernels are held to."""
    x, r = part(*case(1, m, V, L, dtype), 0, m)
    want, floor = u.process64(x, 1, r), tolerance(x, r, m, dtype)
    assert off(want.to(dtype), want, floor, dtype) <= 0
    n, p = int(r["history_len"][0]), int(r["prompt_len"][0])
    # an output token whose logit is not so large that its rounding hides a count
    at = next(i for i in range(n - 1, p, -1) if 0 <= int(r["history"][0, i]) < V and float(x[:, int(r["history"][0, i])].abs().max()) < 4
              and int(r["history"][0, i]) != int(r["history"][0, 0]))
    lost, twice = r["history"].clone(), r["history"].clone()
    lost[0, at] = -1
    twice[0, n] = twice[0, at]  # the first place behind the history
    mistakes = [dict(r, history=lost), dict(r, history=twice, history_len=r["history_len"] + 1)]
    if m > 1:
        small = [k for k in range(m - 1) if float(x[:, int(r["draft_ids"][0, k])].abs().max()) < 6]
        for k in small[:1]:
            d = r["draft_ids"].clone()
            d[0, k] = -1
            mistakes.append(dict(r, draft_ids=d))
    for wrong in mistakes:
        assert off(u.process64(x, 1, wrong), want, floor, dtype) > 0.05


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("S,m,V,L", CASES)
def test_counts(vh, S, m, V, L, dtype):
    x, r = case(S, m, V, L, dtype)
    xd, rd = x.cuda(), {k: v.cuda() for k, v in r.items()}
    outs = {dtype: vh.logits_process(xd, **rd)}
    if dtype != F32:
        outs[F32] = vh.logits_process(xd, out=torch.empty(x.shape, device="cuda"), **rd)
    for s in sorted({0, 1, S // 2, S - 1} & set(range(S))):
        xs, rs = part(x, r, s, m)
        want = u.process64(xs, 1, rs)
        for t, out in outs.items():
            o = off(out[s * m:(s + 1) * m], want, tolerance(xs, rs, m, t), t)
            assert o <= 0, (s, t, o)
    same = xd.clone()
    vh.logits_process(same, out=same, **rd)
    assert torch.equal(same, outs[dtype])
    assert not math.isnan(float(same.float().sum()))
