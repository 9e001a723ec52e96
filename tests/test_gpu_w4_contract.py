"""What the header says about roundings: values of 4-bit rows in fp32 and then in the rows' type, the order of a product's scales,
the reciprocal of a temperature."""
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


@pytest.mark.parametrize("tiles", [False, True])
def test_values_are_rounded_to_fp32_first(vh, tiles):
    """1.25 g half an fp32 step and less above the middle of two bf16 numbers: after the first rounding a tie, and so the even one."""
    g = (257 * 2 ** 18 + 2) // 5 * 2.0 ** -24  # 5 times that is the middle, 257 / 256, and 2 of 2^-26
    assert float(torch.tensor(g, dtype=F32)) == g and 257 / 256 < 1.25 * g < 257 / 256 + 2.0 ** -24
    codes = torch.full((1, 8), 0x22, dtype=torch.uint8, device="cuda")  # 1 and 1
    scales = torch.full((1, 1), 0x3A, dtype=torch.uint8, device="cuda")  # 1.25
    if tiles:
        y = vh.nvfp4_dequantize_tiles(vh.nvfp4_tile(codes, scales), g, 1, 16, dtype=BF)
    else:
        y = vh.nvfp4_dequantize(codes, scales, g, dtype=BF)
    assert bool((y == 1).all())  # rounded once it would be 1 + 2^-7


@pytest.mark.parametrize("T", [2, 40, 1024])
def test_order_of_a_products_scales(vh, T):
    """The sum times W's scale, in fp32, then X's: infinite where the first product is."""
    V, H = (300, 256) if T < 1000 else (8192, 2048)
    one = torch.full((1, 8), 0x22, dtype=torch.uint8, device="cuda")  # 1 and 1
    x, w = (vh.nvfp4_tile(one.repeat(n, H // 16), torch.full((n, H // 16), 0x38, dtype=torch.uint8, device="cuda")) for n in (T, V))
    f = lambda a: torch.tensor(a, dtype=F32)  # noqa: E731
    for gx, gw in ((1e-30, 1e30), (3e-5, 7e-4), (1e-30, 3e38), (3e38, 1e-30), (1e-20, 1e-40)):
        want = f(float(H)) * f(gw) * f(gx)
        y = vh.nvfp4_matmul(x, gx, w, gw, T, V, H, dtype=F32)
        assert torch.equal(y.cpu(), want.expand(T, V)), (gx, gw)
        y = vh.nvfp4_matmul(x, torch.full((T,), gx, device="cuda"), w, torch.full((V,), gw, device="cuda"), T, V, H, dtype=F32)
        assert torch.equal(y.cpu(), want.expand(T, V)), (gx, gw)


@pytest.mark.parametrize("S,m,V,L", [(1, 2, 3001, 0), (1, 2, 3001, 50), (1, 2, 3001, 5000), (300, 4, 9001, 50), (300, 4, 9001, 0)])
def test_temperature_is_two_roundings(vh, S, m, V, L):
    """1 / T to the nearest and a product: 2^-24 each, relative, for every T whose reciprocal is a normal number."""
    g = torch.Generator().manual_seed(S + L)
    x = torch.randn(S * m, V, generator=g).cuda()
    t = torch.exp2(torch.rand(S, generator=g) * 60 - 30).cuda()
    r = dict(temperature=t)
    if L:
        r.update(history=torch.randint(0, V, (S, L), generator=g, dtype=torch.int32).cuda())  # seen, and no rule for it
    d = t.double().repeat_interleave(m)[:, None]
    want = x.double() / d
    bound = (2 * 2.0 ** -24 + 2.0 ** -48) * want.abs()
    for y in (vh.logits_process(x, **r), vh.logits_process_grad(x, x.clone(), **r)):
        assert float(((y.double() - want).abs() - bound).max()) <= 0
