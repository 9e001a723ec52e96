"""The 4-bit and logit-processing calls at their ends: offsets past 32 bits, histories longer than the 16-bit counts hold, every
entry of a long list of biases, many rows of one sequence; and what one call writes as the next call's table, rows or ids."""
import pytest
import torch

import w4_util as u
from rows_util import TINY, U, close
from test_gpu_logits_process import check, check_grad, rows, tolerance

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def vh():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import verify_head_gb300 as vh
    vh.build()
    return vh


@pytest.fixture
def room():
    """About 25 GB, given back."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("not enough memory")
    yield
    torch.cuda.empty_cache()


def test_many_rows(vh, room):
    """2.2 million rows of 2048: elements pass 2^32, bytes of codes 2^31."""
    T, H = 2200064, 2048
    x = torch.zeros(T, H, dtype=BF, device="cuda")
    marks = (0, 2 ** 31 // H - 100, 2 ** 32 // H - 100, T - 256)
    marks = [m // 128 * 128 for m in marks]
    for m in marks:
        x[m:m + 256] = torch.randn(256, H, device="cuda").to(BF)
    codes, scales, rs = vh.nvfp4_quantize(x)
    tiles, rt = vh.nvfp4_quantize_tiles(x)
    again = vh.nvfp4_tile(codes, scales)
    assert torch.equal(rs, rt) and torch.equal(tiles, again)
    del again
    per = H // 256 * 18432
    for m in marks:
        c, s, r = vh.nvfp4_quantize(x[m:m + 256].clone())
        t, _ = vh.nvfp4_quantize_tiles(x[m:m + 256].clone())
        assert torch.equal(codes[m:m + 256], c) and torch.equal(scales[m:m + 256], s) and torch.equal(rs[m:m + 256], r)
        assert torch.equal(tiles[m // 128 * per:(m // 128 + 2) * per], t)
    y = vh.nvfp4_dequantize(codes, scales, rs, out=x)
    parts = [y[m:m + 256].clone() for m in marks]
    z = vh.nvfp4_dequantize_tiles(tiles, rs, T, H, out=y.fill_(3))
    for m, p in zip(marks, parts):
        assert torch.equal(p, vh.nvfp4_dequantize(codes[m:m + 256].clone(), scales[m:m + 256].clone(), rs[m:m + 256].clone()))
        assert torch.equal(p, z[m:m + 256])


def product_is(got, xv, wv, H):
    """As in test_gpu_nvfp4_matmul: (H / 64 + 64) truncations of 2^-23 of the magnitudes, two roundings, that to bf16."""
    want, size = xv @ wv.t(), xv.abs() @ wv.abs().t()
    tol = (H / 64 + 64) * 2.0 ** -23 * size + (2 * 2.0 ** -24 + 2.0 ** -8) * want.abs() + 2.0 ** -134
    assert float(((got.double() - want).abs() - tol).max()) <= 0


def random_matrix(n, H):
    q = torch.randint(0, 256, (n, H // 2), dtype=torch.uint8, device="cuda")
    return q, torch.randint(40, 80, (n, H // 16), dtype=torch.uint8, device="cuda")


def values(q, s):
    return torch.from_numpy(u.values64(q, s)).cuda()


def test_far_products(vh, room):
    """9000 x 248320 of y: 2.2 billion elements."""
    T, V, H = 9000, 248320, 256
    x, w = random_matrix(T, H), random_matrix(V, H)
    y = vh.nvfp4_matmul(vh.nvfp4_tile(*x), 1.0, vh.nvfp4_tile(*w), 1.0, T, V, H)
    wv = values(*w)
    for m in (0, 2 ** 31 // V - 20, T - 40):
        product_is(y[m:m + 40], values(x[0][m:m + 40], x[1][m:m + 40]), wv, H)


@pytest.mark.parametrize("T", [3, 50, 300])
def test_far_table(vh, room, T):
    """A table of 300000 x 16384: 2.8 GB."""
    V, H = 300000, 16384
    x, w = random_matrix(T, H), random_matrix(V, H)
    y = vh.nvfp4_matmul(vh.nvfp4_tile(*x), 1.0, vh.nvfp4_tile(*w), 1.0, T, V, H)
    xv = values(*x)
    for m in (0, 2 ** 31 // (H * 9 // 16) - 100, V - 200):
        product_is(y[:, m:m + 200], xv, values(w[0][m:m + 200], w[1][m:m + 200]), H)


@pytest.mark.parametrize("L", [40, 2000])
def test_far_logits(vh, room, L):
    """9000 rows of 248320 in 3000 sequences: what a call of the last ones alone gives."""
    S, m, V = 3000, 3, 248320
    g = torch.Generator("cuda").manual_seed(L)
    x = torch.randn(S * m, V, device="cuda", dtype=BF, generator=g)
    i = lambda hi, *s: torch.randint(0, hi, s, generator=g, device="cuda", dtype=torch.int32)  # noqa: E731
    f = lambda *s: torch.rand(*s, generator=g, device="cuda") + 0.5  # noqa: E731
    r = dict(history=i(V, S, L), prompt_len=i(L, S), draft_ids=i(V, S, m - 1), repetition=f(S), frequency=f(S), presence=f(S),
             temperature=f(S), bias_ids=i(V, S, 5), bias=f(S, 5), allowed=i(2 ** 31 - 1, S * m, V // 32))
    out = vh.logits_process(x, **r)
    grad = vh.logits_process_grad(x, x.clone(), **r)
    for a in (0, 2 ** 31 // V // m - 2, S - 5):
        some = {k: v[a * m:(a + 5) * m].clone() if k == "allowed" else v[a:a + 5].clone() for k, v in r.items()}
        part = x[a * m:(a + 5) * m].clone()
        assert torch.equal(out[a * m:(a + 5) * m], vh.logits_process(part, **some))
        assert torch.equal(grad[a * m:(a + 5) * m], vh.logits_process_grad(part, part.clone(), **some))
    assert vh.logits_process(x, out=x, **r) is x and torch.equal(x, out)


@pytest.mark.parametrize("L", [32765, 32766, 40000])
@pytest.mark.parametrize("prompt", [0, 1])
def test_one_token_over_and_over(vh, L, prompt):
    """32767 occurrences fill a 16-bit count beside the prompt's bit; three rows, two drafts."""
    g = torch.Generator().manual_seed(L)
    S, m, V = 1, 3, 3001
    x = rows(g, S * m, V, F32)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    r = dict(history=torch.full((S, L), 9, dtype=torch.int32, device="cuda"), prompt_len=i32(prompt), draft_ids=i32(9, 9)[None],
             repetition=torch.full((S,), 1.5, device="cuda"), frequency=torch.full((S,), 0.25, device="cuda"),
             presence=torch.full((S,), 0.5, device="cuda"))
    want = u.process64(x, S, r)
    got = vh.logits_process(x, **r)
    # of the one token: z within a rounding of 2^-24, frequency * n exact below 2^24 / 4, two differences of up to 2^14
    close(got, want, 4 * 2.0 ** -24, 4 * 2.0 ** -24 * 2.0 ** 14)
    assert torch.equal(vh.logits_process(x, out=x, **r), got)


def test_long_histories_in_place(vh):
    g = torch.Generator().manual_seed(3)
    S, m, V, L = 2, 3, 20011, 50000
    x = rows(g, S * m, V, BF)
    r = dict(history=torch.randint(0, V, (S, L), generator=g, dtype=torch.int32).cuda(),
             draft_ids=torch.randint(0, V, (S, m - 1), generator=g, dtype=torch.int32).cuda(),
             repetition=torch.full((S,), 1.3, device="cuda"), frequency=torch.full((S,), 0.125, device="cuda"))
    check(vh, x, S, r)
    check_grad(vh, x, S, r)
    want = u.process64(x, S, r)
    rel, floor = tolerance(BF, x, r)
    close(vh.logits_process(x, out=x, **r), want, rel, floor)


@pytest.mark.parametrize("V", [70001, 333])
def test_every_bias(vh, V):
    """65535 entries, the ids of most of them twice and more: the last counts."""
    g = torch.Generator().manual_seed(4)
    x = rows(g, 2, V, F32)
    r = dict(bias_ids=torch.randint(0, V, (2, 65535), generator=g, dtype=torch.int32).cuda(), bias=torch.randn(2, 65535, generator=g).cuda())
    check(vh, x, 2, r)
    check_grad(vh, x, 2, r)


def test_many_rows_of_a_sequence(vh):
    g = torch.Generator().manual_seed(5)
    m, V = 1500, 61
    x = rows(g, 2 * m, V, F32)
    r = dict(draft_ids=torch.randint(-1, V + 1, (2, m - 1), generator=g, dtype=torch.int32).cuda(),
             frequency=torch.full((2,), 0.5, device="cuda"), repetition=torch.full((2,), 1.25, device="cuda"))
    check(vh, x, 2, r)


def test_what_one_call_writes_the_next_reads(vh):
    """A table made right before its product, logits processed right after, ids drafted right before; no pause between them."""
    T, V, H = 8, 4099, 512
    g = torch.Generator("cuda").manual_seed(6)
    hid = torch.randn(T, H, generator=g, device="cuda").to(BF)
    tables = [torch.randn(V, H, generator=g, device="cuda").to(BF) for _ in range(6)]
    cand = torch.arange(V, dtype=torch.int32, device="cuda")
    wt = torch.zeros(vh.vh_nvfp4_tiles_bytes(V, H), dtype=torch.uint8, device="cuda")
    ws = torch.zeros(V, device="cuda")
    ids = [torch.zeros(4, 1, dtype=torch.int32, device="cuda") for _ in tables]
    max_logit = torch.zeros(4, device="cuda")
    f = torch.full((4,), 1.5, device="cuda")
    work = torch.zeros(vh.lib().vh_workspace_bytes(4), dtype=torch.uint8, device="cuda")
    outs = [torch.zeros(T, V, dtype=BF, device="cuda") for _ in tables]
    xt, xs = vh.nvfp4_quantize_tiles(hid)

    def run(pause):
        y = torch.zeros(T, V, dtype=BF, device="cuda")
        for W, i, o in zip(tables, ids, outs):
            pause()
            vh.nvfp4_quantize_tiles(W, tiles=wt, row_scales=ws)
            pause()
            vh.nvfp4_matmul(xt, xs, wt, ws, T, V, H, out=y)
            pause()
            st = vh.lib().mtp_draft_head_argmax(hid.data_ptr(), W.data_ptr(), cand.data_ptr(), 4, H, V, i.data_ptr(), max_logit.data_ptr(),
                                                work.data_ptr(), work.numel(), torch.cuda.current_stream().cuda_stream)
            assert st == vh.VH_OK
            pause()
            vh.logits_process(y, draft_ids=i, frequency=f, presence=f, out=o)
        torch.cuda.synchronize()
        return [o.clone() for o in outs]

    want = run(torch.cuda.synchronize)
    assert not torch.equal(want[0], want[1])
    for _ in range(10):
        for o, i in zip(outs, ids):
            o.zero_(), i.zero_()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(run(lambda: None), want))


@pytest.mark.parametrize("L", [0, 3, 4000])
@pytest.mark.parametrize("S", [1, 1200])
def test_temperatures_next_to_zero(vh, L, S):
    """A temperature whose reciprocal is no fp32 number: 0 stays 0, the others keep their sign and order."""
    V = 2055
    x = torch.zeros(S, V, device="cuda")
    x[:, 1::4], x[:, 2::4] = 1.0, -1.0
    t = torch.full((S,), 1e-42, device="cuda")
    r = dict(temperature=t)
    if L:
        r.update(history=torch.arange(L, dtype=torch.int32, device="cuda")[None].expand(S, L).contiguous() % V,
                 repetition=torch.full((S,), 1.5, device="cuda"))
    y = vh.logits_process(x, **r)
    assert bool((y[:, 0::4] == 0).all()) and bool((y[:, 3::4] == 0).all())
    assert bool((y[:, 1::4] > 1e37).all()) and bool((y[:, 2::4] < -1e37).all())
    d = vh.logits_process_grad(x, x.clone(), **r)
    assert not bool(torch.isnan(d).any()) and bool((d[:, 0::4] == 0).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("S,m,V,L", [(300, 1, 20011, 5000), (150, 2, 16384, 4200), (40, 2, 70003, 6000), (200, 1, 70003, 40000),
                                     (160, 3, 70003, 33000)])
def test_long_histories_of_many_sequences(vh, S, m, V, L, dtype):
    """Histories of a good part of the vocabulary, on both sides of a twentieth and of 4096 tokens; a few sequences are compared."""
    g = torch.Generator().manual_seed(S)
    x = rows(g, S * m, V, dtype, V + 3, 1)
    r = dict(history=torch.randint(0, V, (S, L), generator=g, dtype=torch.int32).cuda(),
             prompt_len=torch.randint(0, L, (S,), generator=g, dtype=torch.int32).cuda(),
             repetition=(0.8 + torch.rand(S, generator=g)).cuda(), frequency=torch.rand(S, generator=g).cuda(),
             presence=torch.rand(S, generator=g).cuda(), bias_ids=torch.randint(0, V, (S, 40), generator=g, dtype=torch.int32).cuda(),
             bias=torch.randn(S, 40, generator=g).cuda())
    if m > 1:
        r["draft_ids"] = torch.randint(0, V, (S, m - 1), generator=g, dtype=torch.int32).cuda()
    out = vh.logits_process(x, **r)
    d = rows(g, S * m, V, dtype, None, 0, 0.1)
    grad = vh.logits_process_grad(d, x, **r)
    for s in (0, S // 2, S - 1):
        some = {k: v[s:s + 1] for k, v in r.items()}
        at = slice(s * m, (s + 1) * m)
        rel, floor = tolerance(dtype, x[at], some)
        close(out[at], u.process64(x[at], 1, some), rel, floor)
        close(grad[at], u.process64(x[at], 1, some, d[at]), U[dtype] + 2.0 ** -22, TINY[dtype])
    same = x.clone()
    assert torch.equal(vh.logits_process(same, out=same, **r), out)
