"""GPU: the serving operators with scales and factors far from 1, where the results themselves are in range.
Multiplying by powers of two rounds nothing, so that such results are the same bits, moved."""
import numpy as np
import pytest
import torch

from oracle import serve_oracle as ref
from tests.test_layer_few import Layer

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_layer_03_gb300 as m
    return m


def moved(q, by):
    """mx weights times 2^by."""
    s = q.scales.int() + by
    blocks = q.shape[-1] // 32
    assert 0 < s[..., :blocks].min() and s[..., :blocks].max() < 255
    return type(q)(q.codes, s.clamp(0, 255).byte(), q.format)


def up_rows_moved(q, by):
    """The same of the up rows alone (the second half of each plane's)."""
    half = q.shape[-2] // 2
    out = moved(q, 0)
    out.scales[..., half:, :] = moved(q, by).scales[..., half:, :]
    return out


# h is moved by the first power, y by the product of both: first products whose scales are large (2^114 and such),
# then second products' that are (2^124).
@pytest.mark.parametrize("up,back", [(118, -118), (60, -60), (-60, 60), (-106, 128)])
@pytest.mark.parametrize("T,dtype", [(5, "bf16"), (11, "bf16"), (16, "f16")])
def test_mx_scales_at_the_ends_of_their_range(moe, T, dtype, up, back):
    if dtype == "f16":
        back = -up                         # (f16 does not hold y otherwise)
    layer = Layer(moe, T, 544, 352, 12, 3, 4, "mx", dtype, shared=96, seed=T)
    layer.x = (2 * layer.x.float() / layer.x.float().abs().amax(1, keepdim=True)).to(layer.x.dtype)
    y, ids, sc = layer()
    layer.check((y, ids, sc))
    layer.w13, layer.w2 = up_rows_moved(layer.w13, up), moved(layer.w2, back)
    layer.kw["w13_s"], layer.kw["w2_s"] = up_rows_moved(layer.kw["w13_s"], up), moved(layer.kw["w2_s"], back)
    again = layer()
    assert moe.moe_read_timeouts() == (moe.MOE_OK, 0)
    assert torch.isfinite(again[0]).all() and torch.equal(again[0].double(), y.double() * 2.0 ** (up + back))
    assert torch.equal(again[1], ids) and torch.equal(again[2], sc)


@pytest.mark.parametrize("T", [3, 12])
def test_small_tokens_and_large_mx_scales(moe, T):
    """x times 2^-120, weights of the first products times 2^120. The gate is zeros, so that it sees neither."""
    layer = Layer(moe, T, 256, 128, 4, 4, 3, "mx", "bf16")
    layer.wg.zero_()
    layer.x = torch.where(layer.x < 0, -1.0, 1.0).bfloat16() * (1 + layer.x.abs().clamp(max=0.75).mul(64).round() / 64).bfloat16()
    want = layer()
    layer.check(want)
    layer.x, layer.w13 = (layer.x.double() * 2.0 ** -120).bfloat16(), moved(layer.w13, 120)
    got = layer()
    assert torch.isfinite(want[0]).all() and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("T", [4, 13])
def test_a_small_token_changes_no_other(moe, T):
    layer = Layer(moe, T, 288, 160, 8, 2, 4, "mx", "bf16", shared=64)
    want = layer()
    x = layer.x.clone()
    x[1] = (x[1].double() * 2.0 ** -100).bfloat16()
    x[2] = 0
    got = layer(x=x)
    rest = [t for t in range(T) if t not in (1, 2)]
    assert all(torch.equal(a[rest], b[rest]) for a, b in zip(got, want))
    assert not got[0][2].any()
    layer.check(got, x=x)


def uneven_scales(moe, shape, fmt, seed):
    """(Fp4, its values in float64): random codes, neighbouring blocks' scales apart by up to 2^16 (mx) or 2^12."""
    rng = np.random.default_rng(seed)
    K = shape[-1]
    codes = rng.integers(0, 256, shape[:-1] + (K // 2,)).astype(np.uint8)
    scales = np.full(shape[:-1] + (moe.Fp4.scale_columns(K, fmt),), 255, np.uint8)
    blocks = K // ref.BLOCK[fmt]
    if fmt == ref.MX:
        scales[..., :blocks] = rng.integers(119, 136, shape[:-1] + (blocks,))
    else:
        scales[..., :blocks] = rng.integers(8, 104, shape[:-1] + (blocks,))
    q = moe.Fp4(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), fmt)
    flat = lambda a: a.reshape(-1, a.shape[-1])   # noqa: E731
    return q, ref.dequantize(flat(codes), flat(scales), fmt).reshape(shape)


# Wide and narrow tiles; rows on both sides of 64, 128, 208, 224 and a multiple of each; many blocks of contraction,
# one, and ones that end inside a block.
@pytest.mark.parametrize("rows,E,K,N", [(63, 1, 2048, 256), (65, 2, 1312, 520), (127, 1, 4096, 264), (129, 3, 1568, 256),
                                        (207, 1, 2080, 512), (208, 2, 256, 256), (209, 1, 3104, 264), (223, 1, 2048, 248),
                                        (225, 2, 2336, 256), (416, 1, 1024, 1032), (448, 3, 544, 512), (40, 60, 2048, 512)])
@pytest.mark.parametrize("fmt", [ref.MX, ref.NV])
def test_each_block_has_its_own_scales(moe, fmt, rows, E, K, N):
    x, X = uneven_scales(moe, (rows * E, K), fmt, rows)
    w, W = uneven_scales(moe, (E, N, K), fmt, rows + 1)
    off = np.arange(E + 1, dtype=np.int32) * rows
    o = torch.from_numpy(off).cuda()
    y = moe.moe_experts_matmul_fp4(x, w, o)
    want, mag = ref.experts_matmul(X, W, off), ref.experts_matmul(np.abs(X), np.abs(W), off)
    # one rounding to bf16, sums of K terms in the tensor cores
    assert (np.abs(y.double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + K * 2.0 ** -23 * mag * 1.01).all()
    for _ in range(20):
        assert torch.equal(y, moe.moe_experts_matmul_fp4(x, w, o))
    assert moe.moe_read_timeouts() == (moe.MOE_OK, 0)


def test_products_on_two_streams_at_once(moe):
    parts = []
    for fmt, rows, E in ((ref.NV, 300, 4), (ref.MX, 12, 64)):
        x, w = uneven_scales(moe, (rows * E, 2048), fmt, rows)[0], uneven_scales(moe, (E, 1536, 2048), fmt, E)[0]
        off = torch.arange(E + 1, dtype=torch.int32, device="cuda") * rows
        parts.append((x, w, off, moe.moe_experts_matmul_fp4(x, w, off)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in parts]
    got = [[], []]
    for _ in range(30):
        for i, (x, w, off, _) in enumerate(parts):
            with torch.cuda.stream(streams[i]):
                got[i].append(moe.moe_experts_matmul_fp4(x, w, off))
    torch.cuda.synchronize()
    assert moe.moe_read_timeouts() == (moe.MOE_OK, 0)
    assert all(torch.equal(g, parts[i][3]) for i in range(2) for g in got[i])


@pytest.mark.parametrize("gx,gw", [(1.3 * 2.0 ** 100, 1.1 * 2.0 ** 100), (2.0 ** 127, 2.0 ** 127), (1.3 * 2.0 ** -70, 1.7 * 2.0 ** -70),
                                   (2.0 ** -149, 1.5), (2.0 ** -149, None), (1.9 * 2.0 ** -126, 2.0 ** -20), (1.5 * 2.0 ** 120, 1.3 * 2.0 ** -120),
                                   (2.0 ** 127, 2.0 ** -149), (2.0 ** -100, 2.0 ** -100)])
@pytest.mark.parametrize("rows", [5, 300])
def test_factors_whose_product_f32_does_not_hold(moe, rows, gx, gw):
    """Rows and channels of zeros give zeros; the others what the factors make of them."""
    K, N = 4096, 264
    rng = np.random.default_rng(rows)
    parts = []
    for shape in ((rows, K), (2, N, K)):
        codes = np.full(shape[:-1] + (K // 2,), 0x77, np.uint8)           # 6 and 6
        codes ^= (rng.integers(0, 16, codes.shape) == 0).astype(np.uint8) * 0x84     # some -6 and 1
        codes[..., ::7, :] = 0
        parts.append((codes, rng.integers(100, 127, shape[:-1] + (K // 16,)).astype(np.uint8)))
    (cx, sx), (cw, sw) = parts
    t = lambda a: torch.from_numpy(a).cuda()   # noqa: E731
    g = lambda v, n: None if v is None else torch.full((n,), v, device="cuda")   # noqa: E731
    x, w = moe.Fp4(t(cx), t(sx), ref.NV, g(gx, 1)), moe.Fp4(t(cw), t(sw), ref.NV, g(gw, 2))
    off = np.array([0, rows // 2, rows - 1], np.int32)
    y = moe.moe_experts_matmul_fp4(x, w, t(off)).double().cpu().numpy()
    X, W = ref.dequantize(cx, sx, ref.NV), ref.dequantize(cw.reshape(2 * N, -1), sw.reshape(2 * N, -1), ref.NV).reshape(2, N, K)
    by = float(np.float32(gx)) * (1.0 if gw is None else float(np.float32(gw)))
    want, mag = by * ref.experts_matmul(X, W, off), by * ref.experts_matmul(np.abs(X), np.abs(W), off)
    assert np.array_equal(y == 0, np.abs(want) <= 2.0 ** -134) and not np.isnan(y).any()
    big = np.abs(want) > 2.0 ** 128
    assert np.isinf(y[big]).all() and (np.sign(y[big]) == np.sign(want[big])).all() and np.isfinite(y[~big]).all()
    # bf16's rounding and its subnormal step, sums of K terms, the factors' two roundings
    bound = 2.0 ** -8 * np.abs(want) + (K * 2.0 ** -23 + 2.0 ** -22) * mag * 1.01 + 2.0 ** -134
    assert (np.abs(y - want) <= bound)[~big].all()


@pytest.mark.parametrize("T", [2, 10])
def test_weights_of_zeros_and_large_tokens(moe, T):
    """First products that are zeros, whatever x and the experts' factor are."""
    layer = Layer(moe, T, 128, 64, 4, 2, 4, "nv", "bf16")
    layer.wg.zero_()
    layer.x.fill_(2.0 ** 125)
    layer.w13.codes.zero_()
    layer.w13.g.fill_(2.0 ** 60)
    y = layer()[0]
    assert not y.any()


def same_where(got, want, bad):
    """NaN at `bad`, elsewhere the same bits."""
    return torch.equal(torch.isnan(got), bad) and torch.equal(got[~bad], want[~bad])


# A block of the second products has some 27 rows of 4096: rows in both halves of a stage. 8 blocks of 32 channels
# of I, 128 of H: each byte of a word of four scales.
@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("T", [5, 12])
def test_a_scale_of_nan_reaches_its_expert_and_row_only(moe, T, fmt):
    layer = Layer(moe, T, 4096, 256, 4, 1, 3, fmt, "bf16", seed=1)
    want, ids, sc = layer()
    assert torch.isfinite(want).all()
    e = int(ids[0, 0])
    hit = (ids[:, 0] == e)[:, None]
    column = torch.arange(4096, device="cuda")[None]
    nan = 255 if fmt == "mx" else 127
    for at in range(8):
        for rows, of in ((layer.w13.scales[e, 3 + 31 * at], hit.expand(T, 4096)),            # a gate's
                         (layer.w13.scales[e, 256 + 17 * at], hit.expand(T, 4096)),          # an up's
                         (layer.w2.scales[e, 27 * at + 2], hit & (column == 27 * at + 2)),
                         (layer.w2.scales[e, 4095 - 27 * at], hit & (column == 4095 - 27 * at))):
            kept = int(rows[at])
            rows[at] = nan
            got = layer()
            assert same_where(got[0], want, of) and torch.equal(got[1], ids) and torch.equal(got[2], sc)
            rows[at] = kept
    assert torch.equal(layer()[0], want)


@pytest.mark.parametrize("T", [5, 12])
def test_the_largest_mx_scale_is_no_nan(moe, T):
    """2^127 on blocks of zeros."""
    layer = Layer(moe, T, 512, 256, 4, 2, 3, "mx", "bf16", seed=2)
    for q in (layer.w13, layer.w2):
        q.codes.view(*q.codes.shape[:-1], -1, 16)[..., 1::3, :] = 0
    want = layer()
    assert torch.isfinite(want[0]).all()
    for q in (layer.w13, layer.w2):
        q.scales[..., 1:q.shape[-1] // 32:3] = 254
    assert all(torch.equal(a, b) for a, b in zip(layer(), want))


def test_an_mx_nan_in_the_products_stays_in_its_row_and_its_channel(moe):
    x, w = uneven_scales(moe, (70, 512), ref.MX, 1)[0], uneven_scales(moe, (2, 264, 512), ref.MX, 2)[0]
    off = torch.tensor([0, 30, 70], dtype=torch.int32, device="cuda")
    want = moe.moe_experts_matmul_fp4(x, w, off)
    assert torch.isfinite(want).all()
    for at in range(16):
        kept = int(x.scales[33, at]), int(w.scales[0, 100 + at, at])
        x.scales[33, at] = w.scales[0, 100 + at, at] = 255
        bad = torch.zeros((70, 264), dtype=torch.bool, device="cuda")
        bad[33] = True
        bad[:30, 100 + at] = True
        assert same_where(moe.moe_experts_matmul_fp4(x, w, off), want, bad)
        x.scales[33, at], w.scales[0, 100 + at, at] = kept
    x.scales[33, 3] = 254                  # 2^127: whatever it makes, in that row alone
    got = moe.moe_experts_matmul_fp4(x, w, off)
    rest = torch.arange(70, device="cuda") != 33
    assert torch.equal(got[rest], want[rest])


@pytest.mark.parametrize("hot", [65, 128, 209, 700])
@pytest.mark.parametrize("fmt", [ref.MX, ref.NV])
def test_most_rows_in_one_of_many_experts(moe, fmt, hot):
    E, K, N = 64, 800, 328
    rows = np.zeros(E, int)
    rows[E // 2], rows[3], rows[E - 1] = hot, 5, 17
    off = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    x, X = uneven_scales(moe, (int(off[-1]), K), fmt, hot)
    w, W = uneven_scales(moe, (E, N, K), fmt, hot + 1)
    y = moe.moe_experts_matmul_fp4(x, w, torch.from_numpy(off).cuda())
    want, mag = ref.experts_matmul(X, W, off), ref.experts_matmul(np.abs(X), np.abs(W), off)
    assert (np.abs(y.double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + K * 2.0 ** -23 * mag * 1.01).all()
