"""GPU: the serving operators on microscaled 4-bit operands against their float64 restatement.

Codes and scale bytes are exact. Values read back and products are off by one rounding to their type
(U[dtype] and half its smallest subnormal), values of a tensor with a factor g by one of f32 before it,
sums of n terms in the tensor cores by n * 2^-23 of the terms' magnitudes."""
import numpy as np
import pytest
import torch

from oracle import serve_oracle as ref

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25, "f32": 2.0 ** -150}
FMT = {"mx": ref.MX, "nv": ref.NV}


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_layer_03_gb300 as m
    return m


def n64(t):
    return t.detach().cpu().double().numpy()


def close(got, want, bound, what):
    got = n64(got) if torch.is_tensor(got) else got
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaNs differ"
    ok = np.isfinite(want)
    err = np.abs(got - want)[ok] - np.broadcast_to(bound, want.shape)[ok]
    assert err.size == 0 or err.max() <= 0, f"{what}: {err.max():.3e} over the bound"


def rows(shape, dtype, seed):
    """Normal values, channels and rows of very unequal size."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g)
    x = x * torch.exp(torch.randn(shape[-1], generator=g)) * torch.exp(2 * torch.randn(shape[:-1] + (1,), generator=g))
    return x.to(DT[dtype]).cuda()


def same_codes(q, want, what):
    codes, scales = want
    assert np.array_equal(q.scales.cpu().numpy().reshape(scales.shape), scales), f"{what}: scales"
    assert np.array_equal(q.codes.cpu().numpy().reshape(codes.shape), codes), f"{what}: codes"


SHAPES = [(1, 32), (3, 64), (5, 96), (7, 256), (2, 288), (33, 512), (4, 544), (19, 1504), (600, 2048), (1, 65536)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("fmt,g", [("mx", None), ("nv", None), ("nv", 0.0037), ("nv", 30.0)])
@pytest.mark.parametrize("R,K", SHAPES)
def test_quantize_and_back(moe, R, K, fmt, g, dtype):
    x = rows((R, K), dtype, R + K)
    gt = None if g is None else torch.full((1,), g, device="cuda")
    q = moe.moe_quantize_fp4(x, FMT[fmt], gt)
    g64 = None if gt is None else float(gt.double())
    want = ref.quantize(n64(x), FMT[fmt], g64)
    same_codes(q, want, "quantize")
    for t in ("bf16", "f16", "f32"):
        v = ref.dequantize(*want, FMT[fmt], g64)
        bound = U[t] * np.abs(v) + TINY[t] + (0 if g is None else np.abs(v) * 2.0 ** -23)
        with np.errstate(invalid="ignore"):
            v = np.where(np.abs(v) * (1 + U[t]) > torch.finfo(DT[t]).max, np.inf * np.sign(v), v)
        close(moe.moe_dequantize_fp4(q, DT[t]), v, bound, t)


def test_planes_have_their_own_factor(moe):
    w = rows((5, 24, 96), "bf16", 4)
    g = (w.float().abs().amax((1, 2)) / (6 * 448)).contiguous()
    q = moe.moe_quantize_fp4(w, ref.NV, g)
    assert q.shape == (5, 24, 96)
    back = moe.moe_dequantize_fp4(q, torch.float32)
    for e in range(5):
        want = ref.quantize(n64(w[e]), ref.NV, float(g[e].double()))
        same_codes(type(q)(q.codes[e], q.scales[e], ref.NV), want, e)
        v = ref.dequantize(*want, ref.NV, float(g[e].double()))
        close(back[e], v, 2.0 ** -23 * np.abs(v), e)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_ties_borders_and_what_is_not_finite(moe, fmt):
    block = ref.BLOCK[FMT[fmt]]
    borders = np.array([0, 0.25, 0.5, 0.75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6])
    x = np.zeros((40, 512))
    rng = np.random.default_rng(0)
    for r in range(40):
        for b in range(512 // block):
            # a block whose largest value sets the scale 2^e (mx) or a number of e4m3, the rest on borders
            s = 2.0 ** rng.integers(-20, 20) if fmt == "mx" else ref.E4M3[rng.integers(1, 127)]
            v = rng.choice(borders, block) * rng.choice([-1, 1], block)
            v[rng.integers(block)] = 6
            x[r, b * block:(b + 1) * block] = v * s
    # amax on and just beside a border between two scales; zeros; subnormals; the largest number
    x[0, :block] = 0
    x[1, 0] = 6 * (1 + 2.0 ** -23)
    x[2, 0] = 6.0 * 1.0625
    x[3, 0] = 6.0 * 1.0625 * (1 + 2.0 ** -22)
    x[4, :block] = 2.0 ** -140
    x[5, :block] = 2.0 ** -149
    x[6, 0] = np.finfo(np.float32).max
    x[7, 3] = np.inf
    x[8, block] = -np.inf
    x[9, 2 * block + 1] = np.nan
    x[10, :block] = -0.0
    t = torch.from_numpy(x.astype(np.float32)).cuda()
    q = moe.moe_quantize_fp4(t, FMT[fmt])
    want = ref.quantize(n64(t), FMT[fmt])
    same_codes(q, want, fmt)
    v = ref.dequantize(*want, FMT[fmt])
    assert np.isnan(v).sum() == 3 * block
    # the largest f32 number is nearest to 4 * 2^126, which f32 does not have: read as an infinity
    with np.errstate(over="ignore"):
        v = v.astype(np.float32).astype(np.float64)
    got = n64(moe.moe_dequantize_fp4(q, torch.float32))
    assert np.array_equal(np.isinf(got), np.isinf(v)) and np.isinf(v).sum() == (fmt == "mx")
    close(moe.moe_dequantize_fp4(q, torch.float32), v, 0.0, fmt)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("fmt,g", [("mx", None), ("nv", None), ("nv", 0.011)])
@pytest.mark.parametrize("R,I", [(1, 32), (5, 96), (131, 992), (40, 2048), (3, 14336)])
def test_swiglu(moe, R, I, fmt, g, dtype):
    gu = rows((R, 2 * I), dtype, R * I)
    gu[0, 0] = 100.0
    gu[0, 1] = -100.0 if dtype != "f16" else -15.0
    gt = None if g is None else torch.full((1,), g, device="cuda")
    q = moe.moe_swiglu_fp4(gu, FMT[fmt], gt)
    h = ref.swiglu(n64(gu))
    same_codes(q, ref.quantize(h, FMT[fmt], None if gt is None else float(gt.double())), "swiglu")


def test_a_block_of_swiglu_with_an_infinity_or_a_nan(moe):
    gu = rows((3, 128), "bf16", 1)
    gu[0, 0], gu[1, 40], gu[2, 64 + 63] = float("inf"), float("nan"), float("-inf")
    for fmt in (ref.MX, ref.NV):
        v = n64(moe.moe_dequantize_fp4(moe.moe_swiglu_fp4(gu, fmt)))
        b = ref.BLOCK[fmt]
        want = np.zeros((3, 64), bool)
        want[0, :b] = want[1, 40 // b * b:40 // b * b + b] = want[2, 64 - b:] = True
        assert np.array_equal(np.isnan(v), want)


def test_into_given_memory(moe):
    x = rows((9, 288), "bf16", 3)
    q = moe.moe_quantize_fp4(x, ref.MX)
    q2 = type(q)(torch.full_like(q.codes, 77), torch.full_like(q.scales, 77), ref.MX)
    got = moe.moe_quantize_fp4(x, ref.MX, out=q2)
    assert got.codes.data_ptr() == q2.codes.data_ptr()
    assert torch.equal(q2.codes, q.codes) and torch.equal(q2.scales, q.scales)   # the filling too
    v = torch.empty((9, 288), dtype=torch.float16, device="cuda")
    assert moe.moe_dequantize_fp4(q, torch.float16, out=v) is v
    assert torch.equal(v, moe.moe_dequantize_fp4(q, torch.float16))


# ------------------------------------------------------------------ the experts' products

def four_bits(moe, shape, fmt, seed, g, std=1.0):
    """(Fp4, its values in float64) of normal values; the filling of the scales is not zeros."""
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=gen) * std * torch.exp(torch.randn(shape[:-1] + (1,), generator=gen))
    flat = x.double().numpy().reshape(-1, shape[-1])
    planes = shape[0] if len(shape) == 3 else 1
    gs = None if not g else 0.004 * (1 + torch.arange(planes, dtype=torch.float32))
    per = flat.shape[0] // planes
    parts = [ref.quantize(flat[p * per:(p + 1) * per], FMT[fmt], None if gs is None else float(gs[p].double())) for p in range(planes)]
    val = np.concatenate([ref.dequantize(*part, FMT[fmt], None if gs is None else float(gs[p].double())) for p, part in enumerate(parts)])
    codes, scales = (np.concatenate([p[i] for p in parts]) for i in (0, 1))
    blocks = shape[-1] // ref.BLOCK[FMT[fmt]]
    scales[:, blocks:] = 255
    q = moe.Fp4(torch.from_numpy(codes).view(*shape[:-1], -1).cuda(), torch.from_numpy(scales).view(*shape[:-1], -1).cuda(),
                FMT[fmt], None if gs is None else gs.cuda())
    return q, val.reshape(shape)


def ragged(R, E, kind, seed):
    rng = np.random.default_rng(seed)
    if kind == "even":
        return np.linspace(0, R, E + 1).astype(np.int32)
    if kind == "last":
        return np.array([0] * E + [R], np.int32)
    if kind == "empty":
        return np.zeros(E + 1, np.int32)
    cut = np.sort(rng.integers(0, R + 1, E + 1)).astype(np.int32)
    if kind != "part":
        cut[0] = 0
    return cut


PRODUCTS = [(1, 1, 32, 8, "even"), (2, 5, 2080, 72, "part"), (7, 40, 96, 16, "empty"), (9, 2, 4128, 136, "cut"),
            (16, 256, 64, 200, "cut"), (17, 4, 160, 520, "cut"), (31, 3, 256, 264, "last"), (33, 1, 288, 256, "even"),
            (128, 1, 512, 128, "even"), (129, 1, 544, 384, "even"), (223, 1, 256, 256, "even"),
            (224, 1, 800, 256, "even"), (225, 1, 256, 520, "even"), (300, 7, 1056, 136, "cut"),
            (449, 2, 1280, 264, "last"), (513, 256, 64, 64, "cut"), (700, 3, 224, 1032, "part"),
            (2100, 2, 96, 72, "cut"), (2000, 1, 192, 2056, "even"), (40, 3, 14336, 136, "cut")]


@pytest.mark.parametrize("fmt,g,out", [("mx", False, "bf16"), ("nv", True, "bf16"), ("nv", False, "f16"), ("mx", False, "f16")])
@pytest.mark.parametrize("R,E,K,N,kind", PRODUCTS)
def test_experts_products(moe, R, E, K, N, kind, fmt, g, out):
    off = ragged(R, E, kind, R + E)
    x, X = four_bits(moe, (R, K), fmt, 1, g)
    w, W = four_bits(moe, (E, N, K), fmt, 2, g, K ** -0.5)
    # rows of no expert reach nothing, whatever they are
    x.scales[off[E]:] = 255 if fmt == "mx" else 127
    x.scales[:off[0]] = 255 if fmt == "mx" else 127
    y = moe.moe_experts_matmul_fp4(x, w, torch.from_numpy(off).cuda(), DT[out])
    assert y.dtype == DT[out] and moe.moe_read_timeouts() == (moe.MOE_OK, 0)
    want = ref.experts_matmul(X, W, off)
    mag = ref.experts_matmul(np.abs(X), np.abs(W), off)
    # (the factors' product and the sum's multiplication by it: two roundings)
    close(y, want, U[out] * np.abs(want) + (K * 2.0 ** -23 + 2.0 ** -22) * mag * (1 + U[out]) + TINY[out], "y")
    assert torch.equal(y, moe.moe_experts_matmul_fp4(x, w, torch.from_numpy(off).cuda(), DT[out]))


def test_a_nan_stays_in_its_row_and_its_channel(moe):
    x, X = four_bits(moe, (70, 512), "nv", 1, False)
    w, W = four_bits(moe, (2, 264, 512), "nv", 2, False)
    off = torch.tensor([0, 30, 70], dtype=torch.int32, device="cuda")
    x.scales[33, 5] = 127
    w.scales[0, 100, 31] = 127
    y = n64(moe.moe_experts_matmul_fp4(x, w, off))
    want = np.zeros((70, 264), bool)
    want[33] = True
    want[:30, 100] = True
    assert np.array_equal(np.isnan(y), want)


def test_offsets_out_of_range_or_order(moe):
    """The kernel keeps offsets inside the rows and in order."""
    x, X = four_bits(moe, (50, 96), "mx", 1, False)
    w, W = four_bits(moe, (3, 40, 96), "mx", 2, False)
    y = moe.moe_experts_matmul_fp4(x, w, torch.tensor([-5, 20, 10, 900], dtype=torch.int32, device="cuda"))
    want = ref.experts_matmul(X, W, np.array([0, 20, 20, 50]))
    mag = ref.experts_matmul(np.abs(X), np.abs(W), np.array([0, 20, 20, 50]))
    close(y, want, U["bf16"] * np.abs(want) + 97 * 2.0 ** -23 * mag + TINY["bf16"], "y")


def test_the_experts_in_four_bits_together(moe):
    """Rows by expert, both products and SwiGLU between them in 4 bits, back to the tokens: as a layer
    whose weights are 4-bit runs them; against float64 on the codes, whose one difference is that SwiGLU
    starts from the first products' rounded values."""
    T, H, I, E, k = 90, 256, 160, 6, 2
    g = torch.Generator().manual_seed(0)
    x = torch.randn((T, H), generator=g).bfloat16().cuda()
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int().cuda()
    sc = torch.rand((T, k), generator=g).cuda()
    w13, W13 = four_bits(moe, (E, 2 * I, H), "nv", 2, True, H ** -0.5)
    w2, W2 = four_bits(moe, (E, H, I), "nv", 3, True, I ** -0.5)
    gx = torch.full((1,), 0.002, device="cuda")

    def run():
        xp, inv, off = moe.moe_dispatch(x, ids, E)
        a = moe.moe_experts_matmul_fp4(moe.moe_quantize_fp4(xp, moe.MOE_FP4_NV, gx), w13, off)
        h = moe.moe_swiglu_fp4(a, moe.MOE_FP4_NV, gx)
        return off, inv, a, h, moe.moe_combine(moe.moe_experts_matmul_fp4(h, w2, off), inv, sc)

    off, inv, a, h, y = run()
    o = off.cpu().numpy()
    gd = float(gx.double())
    xq = ref.dequantize(*ref.quantize(n64(moe.moe_dispatch(x, ids, E)[0]), ref.NV, gd), ref.NV, gd)
    want, mag = ref.experts_matmul(xq, W13, o), ref.experts_matmul(np.abs(xq), np.abs(W13), o)
    close(a, want, U["bf16"] * np.abs(want) + (H + 4) * 2.0 ** -23 * mag, "first products")
    hq = ref.quantize(ref.swiglu(n64(a)), ref.NV, gd)
    same_codes(h, hq, "h")
    hv = ref.dequantize(*hq, ref.NV, gd)
    want, mag = ref.experts_matmul(hv, W2, o), ref.experts_matmul(np.abs(hv), np.abs(W2), o)
    at, s = inv.cpu().numpy(), n64(sc)
    y64 = (want[at] * s[:, :, None]).sum(1)
    ymag = (mag[at] * s[:, :, None]).sum(1)
    # one rounding of each row and of the sum
    close(y, y64, U["bf16"] * (np.abs(y64) + 1.01 * (np.abs(want[at]) * s[:, :, None]).sum(1)) + (I + 8) * 2.0 ** -23 * ymag, "y")

    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        again = run()
    x.copy_(-x)
    graph.replay()
    assert not torch.equal(again[4], y)
    x.copy_(-x)
    graph.replay()
    assert all(torch.equal(p, q) for p, q in ((again[2], a), (again[3].codes, h.codes), (again[4], y)))
