"""The way from hidden rows through a 4-bit head, processing and log probabilities and back, by value: the gradient of the hidden
rows against the 64-bit definition on the head's exact values."""
import pytest
import torch

import w4_util as u
from test_gpu_logits_process import rules

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def vh():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import verify_head_gb300 as vh
    vh.build()
    return vh


@pytest.mark.parametrize("S,m,V,H,L,masked", [(3, 4, 5003, 256, 200, 0.5), (2, 1, 999, 512, 30, 0.0)])
def test_gradient_of_the_hidden_rows(vh, S, m, V, H, L, masked):
    g = torch.Generator().manual_seed(V)
    R = S * m
    hid = torch.randn(R, H, generator=g).to(BF).cuda()
    w = (torch.randn(V, H, generator=g) * 0.05).cuda()
    gw = float((w.abs().max() / 2688).item())
    codes, scales, _ = vh.nvfp4_quantize(w, gw)
    xt, xg = vh.nvfp4_quantize_tiles(hid)
    logits = vh.nvfp4_matmul(xt, xg, vh.nvfp4_tile(codes, scales), gw, R, V, H, dtype=F32)
    r = rules(g, S, m, V, L, 4, masked)
    if masked:
        r["allowed"][:, 0] |= 128  # token 7 may follow everywhere
    out = vh.logits_process(logits, **r)
    tok = torch.full((R,), 7, dtype=torch.int32, device="cuda")
    lp, ent, lse, _, _ = vh.logits_logprobs(out, tok, 0)
    gl = torch.randn(R, generator=g).cuda()
    d = vh.logits_logprobs_grad(out, tok, lse, ent, gl)
    dl = vh.logits_process_grad(d, logits, **r)
    dhid = dl @ vh.nvfp4_dequantize(codes, scales, gw, dtype=F32)

    z = u.process64(logits, S, r)
    slope = u.process64(logits, S, r, torch.ones(R, V))
    p = torch.exp(torch.log_softmax(z, 1))
    hot = torch.zeros_like(p)
    hot[:, 7] = 1.0
    gl64 = gl.double().cpu()[:, None]
    W = torch.from_numpy(u.values64(codes, scales)) * float(torch.tensor(gw))  # the scale as fp32
    full = gl64 * (hot - p) * slope
    want = full @ W
    # Scores of up to M, off by 8 roundings of 2^-24 of what is added up in them (three times M at most), so that p is off by twice
    # that; lse, its difference to the score and their product with log2(e) another 4 M, its sum V / 256 + 64 terms' roundings.  Then four of
    # the gradient's factors, of hot - p; and V of the matrix product, in any order, besides one of the table's values.
    M = float(z[torch.isfinite(z)].abs().max())
    share = gl64.abs() * slope.abs() * (p * (2 * 8 * 3 * M + 4 * M + V / 256 + 64) + 4 * (hot + p)) * 2.0 ** -24
    tol = share @ W.abs() + (V + 1) * 2.0 ** -24 * (full.abs() @ W.abs())
    gap = (dhid.double().cpu() - want).abs()
    assert float((gap - tol).max()) <= 0
    assert float(tol.max()) < 0.1 * float(want.abs().max())  # a wrong row of the table would be seen
