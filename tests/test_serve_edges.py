"""GPU: the serving operators where f32's range or 32-bit offsets end. Codes and scale bytes are exact;
results of the same sums over weights that lie elsewhere are the same bits."""
import numpy as np
import pytest
import torch

from oracle import serve_oracle as ref

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_layer_03_gb300 as m
    return m


# Exponents of gates and of up values, and g: gates that are no normal f32 numbers before large up values;
# products below f32's normal numbers; large ones.
@pytest.mark.parametrize("gate,up,g", [(-140, 100, 2.0 ** -50), (-133, 110, 2.0 ** -31), (-126, 30, None),
                                       (-70, -60, None), (-64, -66, None), (5, 110, 2.0 ** 106)])
@pytest.mark.parametrize("fmt", [ref.MX, ref.NV])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_swiglu_at_the_ends_of_the_range(moe, dtype, fmt, gate, up, g):
    if fmt == ref.MX:
        g = None
    gen = torch.Generator().manual_seed(gate + 1000 * up)
    R, I = 40, 256
    v = torch.randn((R, I), generator=gen, dtype=torch.float64) * 2.0 ** gate
    u = (1 + torch.rand((R, I), generator=gen, dtype=torch.float64)) * 2.0 ** up
    gu = torch.cat([v, u], 1).to(dtype)
    q = moe.moe_swiglu_fp4(gu.cuda(), fmt, None if g is None else torch.full((1,), g, device="cuda"))
    codes, scales = ref.quantize(ref.swiglu(gu.double().numpy()), fmt, g)
    assert np.array_equal(q.scales.cpu().numpy(), scales)
    assert np.array_equal(q.codes.cpu().numpy(), codes)


@pytest.mark.parametrize("R,I", [(8460, 992), (586, 14336)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("fmt,g", [(ref.MX, None), (ref.NV, None), (ref.NV, 0.011)])
def test_swiglu_of_many_values(moe, fmt, g, dtype, R, I):
    """8.4 million values, of rows of very unequal size, some blocks not finite."""
    gen = torch.Generator().manual_seed(R)
    gu = torch.randn((R, 2 * I), generator=gen) * torch.exp(2 * torch.randn((R, 1), generator=gen))
    gu[5, 7], gu[9, I + 40], gu[R - 1, 2 * I - 1] = float("inf"), float("nan"), float("-inf")
    gu[3, :64] = -30.0
    if dtype == torch.bfloat16:
        gu[11:20] *= 2.0 ** -40
        gu[20, :I], gu[20, I:] = gu[20, :I] * 2.0 ** -128, gu[20, I:] * 2.0 ** 100
        gu[21, :96] = -95.0
    gu = gu.to(dtype)
    q = moe.moe_swiglu_fp4(gu.cuda(), fmt, None if g is None else torch.full((1,), g, device="cuda"))
    with np.errstate(invalid="ignore", over="ignore"):
        h = ref.swiglu(gu.double().numpy())
        codes, scales = ref.quantize(h, fmt, None if g is None else float(np.float32(g)))
    assert np.array_equal(q.scales.cpu().numpy(), scales)
    assert np.array_equal(q.codes.cpu().numpy(), codes)


def test_conversions_past_32_bit_offsets(moe):
    """4.3 billion channels: the last rows as they are alone."""
    R, K = 65552, 65536
    x = torch.zeros((R, K), dtype=torch.bfloat16, device="cuda")
    x[-16:] = torch.randn((16, K), device="cuda")
    q = moe.moe_quantize_fp4(x, moe.MOE_FP4_NV)
    alone = moe.moe_quantize_fp4(x[-16:].clone(), moe.MOE_FP4_NV)
    assert torch.equal(q.codes[-16:], alone.codes) and torch.equal(q.scales[-16:], alone.scales)
    assert not q.scales[:-16].any()
    back = moe.moe_dequantize_fp4(q, out=x)
    assert torch.equal(back[-16:], moe.moe_dequantize_fp4(alone)) and not back[:-16].any()


def codes4(moe, shape, gen, fmt):
    """Random codes with scales about 2^-6."""
    head, K = shape[:-1], shape[-1]
    c = torch.empty(head + (K // 2,), dtype=torch.uint8, device="cuda").random_(0, 256, generator=gen)
    s = torch.empty(head + (moe.Fp4.scale_columns(K, fmt),), dtype=torch.uint8, device="cuda")
    s.random_(120, 123, generator=gen) if fmt == moe.MOE_FP4_MX else s.random_(8, 16, generator=gen)
    return moe.Fp4(c, s, fmt)


def test_products_past_32_bit_offsets(moe):
    """Weights of 4.8 GB: the last expert's products as they are alone."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    E, N, K, R = 72, 65536, 2048, 40
    w = codes4(moe, (E, N, K), gen, moe.MOE_FP4_MX)
    x = codes4(moe, (R, K), gen, moe.MOE_FP4_MX)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[-1] = R
    y = moe.moe_experts_matmul_fp4(x, w, off)
    last = moe.Fp4(w.codes[-1:].clone(), w.scales[-1:].clone(), w.format)
    alone = moe.moe_experts_matmul_fp4(x, last, torch.tensor([0, R], dtype=torch.int32, device="cuda"))
    assert torch.isfinite(y).all() and torch.equal(y, alone)


def test_layer_past_32_bit_offsets(moe):
    """First products' weights of 8.6 GB: the chosen experts' layer as it is with those experts alone."""
    gen = torch.Generator(device="cuda").manual_seed(6)
    E, I, H, k = 256, 8192, 4096, 8
    w13, w2 = codes4(moe, (E, 2 * I, H), gen, moe.MOE_FP4_NV), codes4(moe, (E, H, I), gen, moe.MOE_FP4_NV)
    x = torch.randn((1, H), generator=gen, device="cuda").bfloat16()
    wg = torch.randn((E, H), generator=gen, device="cuda").bfloat16() * H ** -0.5
    wg[-1] = x[0] / 64                     # the last expert is chosen
    y, ids, scales = moe.moe_layer_few(x, wg, w13, w2, moe.MOE_ROUTE_RENORMALIZE_NAIVE, k)
    chosen = ids[0].long().sort()[0]
    assert E - 1 in chosen.tolist()
    part = [moe.Fp4(w.codes[chosen], w.scales[chosen], w.format) for w in (w13, w2)]
    y2, ids2, scales2 = moe.moe_layer_few(x, wg[chosen], *part, moe.MOE_ROUTE_RENORMALIZE_NAIVE, k)
    assert torch.equal(chosen[ids2[0].long()], ids[0].long())
    # (the gate's sums are the same for any number of rows)
    assert torch.equal(scales, scales2) and torch.isfinite(y).all() and torch.equal(y, y2)


@pytest.mark.parametrize("fmt,g", [(ref.MX, None), (ref.NV, None), (ref.NV, 0.011)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
def test_swiglu_of_zeros_beside_values_that_are_worked_out_again(moe, dtype, fmt, g):
    """Small gates of few bits: their SwiGLU is next to a tie. Zeros of both signs in gates and up values keep the
    sign of the product, in every segment."""
    gen = torch.Generator().manual_seed(3)
    R, I = 60, 800
    gate = torch.randint(-12, 13, (R, I), generator=gen) * 2.0 ** -24
    up = torch.randint(-9, 10, (R, I), generator=gen) * 0.25
    gate = torch.where(torch.rand((R, I), generator=gen) < 0.1, -0.0, gate.double())
    up = torch.where(torch.rand((R, I), generator=gen) < 0.1, -0.0, up.double())
    gu = torch.cat([gate, up], 1).to(dtype)
    q = moe.moe_swiglu_fp4(gu.cuda(), fmt, None if g is None else torch.full((1,), g, device="cuda"))
    codes, scales = ref.quantize(ref.swiglu(gu.double().numpy()), fmt, None if g is None else float(np.float32(g)))
    assert np.array_equal(q.scales.cpu().numpy(), scales) and np.array_equal(q.codes.cpu().numpy(), codes)
