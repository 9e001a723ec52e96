"""Log probabilities of more rows than the scan has CTAs, on either side of the width up to which each row has a CTA of
its own, at several alignments."""
import pytest
import torch

from rows_util import close, sums

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def vh():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import verify_head_gb300 as vh
    vh.build()
    return vh


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("R", [608, 609, 700, 1217])
@pytest.mark.parametrize("V,pitch,offset", [(65536, 65536, 0), (65536, 65537, 3), (65537, 65537, 0), (65600, 65600, 0),
                                            (32768, 32768, 0), (32769, 32771, 1), (33100, 33100, 0)])
def test_a_cta_per_row_or_even_ranges(vh, R, V, pitch, offset, dtype):
    g = torch.Generator("cuda").manual_seed(R + V)
    flat = torch.full((R * pitch + offset + 16,), 1e4, dtype=dtype, device="cuda")  # a read past a row would show
    x = flat[offset:offset + R * pitch].view(R, pitch)[:, :V]
    x.copy_(torch.randn(R, V, generator=g, device="cuda") * 2)
    tokens = torch.randint(0, V, (R,), generator=g, device="cuda", dtype=torch.int32)
    ws = vh.logits_logprobs_workspace(R, V)
    got = vh.logits_logprobs(x, tokens, ws=ws)
    for r in range(0, R, 64):
        p = x[r:r + 64].double()
        lse = torch.logsumexp(p, 1)
        at = slice(r, r + 64)
        close(got[2][at], lse, 2.0 ** -22, sums(V) + 2.0 ** -20)
        close(got[1][at], lse - (torch.softmax(p, 1) * p).sum(1), 2.0 ** -22, 20 * sums(V))
        close(got[0][at], p.gather(1, tokens[at].long()[:, None])[:, 0] - lse, 2.0 ** -22, sums(V) + 2.0 ** -20)
    again = vh.logits_logprobs(x, tokens, ws=ws)
    assert all(torch.equal(a, b) for a, b in zip(got[:3], again[:3]))
