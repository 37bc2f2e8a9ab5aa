"""GPU: the training operators (rows by expert and back, SwiGLU with an 8-bit checkpoint, the
experts' products, the router's gradient) against their float64 restatement.

Tolerances are elementwise and come from the arithmetic: one rounding of the result to its type
(unit roundoff U[dtype], plus half the smallest subnormal), and for what was summed in fp32 n
roundings of the terms' magnitudes, n * 2^-24 on the CUDA cores and n * 2^-23 in the tensor
cores' accumulators (which may truncate). Places, offsets, copies, codes and scale bytes are
exact."""
import numpy as np
import pytest
import torch

from oracle import train_oracle as ref

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25, "f32": 2.0 ** -150}


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_layer_03_gb300 as m
    return m


def n64(t):
    return t.detach().cpu().double().numpy()


def randn(shape, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(DT[dtype]).cuda()


def close(got, want, bound, what):
    got = n64(got) if torch.is_tensor(got) else got
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaNs differ"
    ok = np.isfinite(want)
    err = np.abs(got - want)[ok] - np.broadcast_to(bound, want.shape)[ok]
    assert err.size == 0 or err.max() <= 0, f"{what}: {err.max():.3e} over the bound"


# ------------------------------------------------------------------ rows by expert and back

def make_ids(T, E, k, kind, seed):
    rng = np.random.default_rng(seed)
    if kind == "one":                       # every slot of one expert
        ids = np.full((T, k), E - 1)
    elif kind == "none":                    # every slot dropped
        ids = np.full((T, k), -1)
    else:
        ids = rng.integers(0, E, (T, k))
        if kind == "dropped":
            ids[rng.random((T, k)) < 0.3] = -1
    return ids.astype(np.int32)


SORTS = [(1, 8, 4, 2, "plain"), (1, 1, 1, 1, "plain"), (2, 64, 3, 8, "dropped"),
         (64, 2048, 128, 8, "plain"), (63, 1001, 60, 6, "dropped"), (513, 72, 256, 8, "dropped"),
         (700, 20, 8, 7, "one"), (300, 36, 5, 3, "none"), (3000, 40, 17, 3, "dropped"),
         (5000, 8, 256, 8, "plain"), (13000, 12, 40, 1, "dropped"), (1500, 520, 2, 5, "one"), (1025, 100, 33, 4, "dropped")]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,H,E,k,kind", SORTS)
def test_dispatch_and_combine(moe, T, H, E, k, kind, dtype):
    ids = make_ids(T, E, k, kind, T + H)
    inv, offsets = ref.sort_slots(ids, E)
    x = randn((T, H), dtype, 1)
    xp, got_inv, got_off = moe.moe_dispatch(x, torch.from_numpy(ids).cuda(), E)
    assert np.array_equal(got_inv.cpu().numpy(), inv)
    assert np.array_equal(got_off.cpu().numpy(), offsets)
    want = ref.dispatch_rows(n64(x), inv)
    assert np.array_equal(n64(xp), want)
    again = moe.moe_dispatch_rows(x, got_inv)
    assert torch.equal(again, xp)

    rows = randn((T * k, H), dtype, 2)
    rows[offsets[E]:] = float("nan")        # rows of dropped slots are not read
    scales = torch.rand((T, k), generator=torch.Generator().manual_seed(3)).cuda()
    for s in (scales, None):
        y = moe.moe_combine(rows, got_inv, s)
        want, mag = ref.combine(n64(rows), inv, None if s is None else n64(s))
        close(y, want, U[dtype] * np.abs(want) + (k + 1) * 2.0 ** -24 * mag * (1 + U[dtype]) + TINY[dtype], "y")
    dx = moe.moe_dispatch_backward(rows, got_inv)
    assert torch.equal(dx, y)               # a sum without weights

    dy = randn((T, H), dtype, 4)
    for s in (scales, None):
        drows, ds = moe.moe_combine_backward(dy, rows, got_inv, s)
        wr, wds, mag = ref.combine_backward(n64(dy), n64(rows), inv, None if s is None else n64(s))
        close(drows, wr, (U[dtype] + 2.0 ** -24) * np.abs(wr) * (1 + U[dtype]) + TINY[dtype], "drows")
        close(ds, wds, (H + 8) * 2.0 ** -24 * mag, "dscales")


# Rows on 2, 4 and 8 bytes; a segment of a warp full, cut and alone; few and many warps' worth.
ODD_ROWS = [(4200, 301, 64, 3, "dropped"), (900, 514, 16, 5, "dropped"), (2100, 130, 8, 2, "plain"),
            (40, 2051, 8, 8, "dropped"), (600, 132, 7, 4, "dropped"), (2, 1, 3, 8, "plain"), (1100, 67, 5, 8, "one")]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,H,E,k,kind", ODD_ROWS)
def test_rows_of_any_width(moe, T, H, E, k, kind, dtype):
    test_dispatch_and_combine(moe, T, H, E, k, kind, dtype)


@pytest.mark.parametrize("H", [5, 131, 262])
def test_infinities_in_rows_of_any_width_stay_in_their_token(moe, H):
    """Neighbouring rows share words, not values."""
    T, E, k = 50, 6, 3
    ids = make_ids(T, E, k, "dropped", H)
    inv, _ = ref.sort_slots(ids, E)
    inv_gpu = torch.from_numpy(inv.astype(np.int32)).cuda()
    x, rows, dy = randn((T, H), "bf16", 1), randn((T * k, H), "bf16", 2), randn((T, H), "bf16", 3)
    clean = [moe.moe_dispatch_rows(x, inv_gpu), moe.moe_combine(rows, inv_gpu), *moe.moe_combine_backward(dy, rows, inv_gpu)]
    hit = 7
    mine = inv[hit][inv[hit] >= 0]
    x[hit], dy[hit], rows[mine] = float("inf"), float("nan"), float("inf")
    got = [moe.moe_dispatch_rows(x, inv_gpu), moe.moe_combine(rows, inv_gpu), *moe.moe_combine_backward(dy, rows, inv_gpu)]
    other_rows = torch.ones(T * k, dtype=torch.bool)
    other_rows[mine] = False
    other_tokens = torch.arange(T) != hit
    for a, b, keep in zip(clean, got, (other_rows, other_tokens, other_rows, other_tokens)):
        assert torch.equal(a.cpu()[keep], b.cpu()[keep])
    assert len(mine) and not torch.isfinite(got[0].cpu()[mine]).any() and not torch.isfinite(got[1].cpu()[hit]).any()


def test_combine_gradient_against_differences(moe):
    T, H, E, k = 5, 24, 4, 3
    ids = make_ids(T, E, k, "dropped", 9)
    inv, _ = ref.sort_slots(ids, E)
    rows, scales, dy = randn((T * k, H), "f32", 1), torch.rand(T, k).cuda(), randn((T, H), "f32", 2)
    drows, ds = moe.moe_combine_backward(dy, rows, torch.from_numpy(inv.astype(np.int32)).cuda(), scales)
    loss = lambda r, s: float((ref.combine(r, inv, s)[0] * n64(dy)).sum())   # noqa: E731
    r0, s0, h = n64(rows), n64(scales), 1e-4
    for got, base, put in ((ds, s0, lambda v: loss(r0, v)), (drows, r0, lambda v: loss(v, s0))):
        for i in np.ndindex(base.shape):
            up, dn = base.copy(), base.copy()
            up[i] += h
            dn[i] -= h
            # linear in each: the difference is exact but for rounding (values up to ~100 / h)
            assert abs((put(up) - put(dn)) / (2 * h) - n64(got)[i]) < 1e-5


def test_dispatch_flags_bad_ids_and_drops_them(moe):
    for T in (4, 7000):                     # one launch, three launches
        ids = make_ids(T, 8, 2, "plain", 1)
        ids[T // 2, 1] = 8
        ids[1, 0] = -2
        x = randn((T, 16), "bf16", 1)
        scratch = moe.alloc_dispatch_scratch(T, 8, 2)
        scratch.buf.fill_(0x5A)             # needs no clearing
        _, inv, off = moe.moe_dispatch(x, torch.from_numpy(ids).cuda(), 8, scratch=scratch)
        st, flags = moe.moe_read_device_status(scratch)
        assert st == moe.MOE_ERR_DEVICE_BAD_ID and flags == moe.MOE_DEVICE_FLAG_BAD_ID
        want, woff = ref.sort_slots(ids, 8)
        assert np.array_equal(inv.cpu().numpy(), want) and np.array_equal(off.cpu().numpy(), woff)
        ids[T // 2, 1] = ids[1, 0] = -1     # dropped on purpose: no flag
        moe.moe_dispatch(x, torch.from_numpy(ids).cuda(), 8, scratch=scratch)
        assert moe.moe_read_device_status(scratch) == (moe.MOE_OK, 0)


def test_places_out_of_range_are_left_out(moe):
    """A map that points past the rows neither reads nor writes there."""
    T, H, k = 6, 32, 2
    inv = torch.arange(T * k, dtype=torch.int32).view(T, k)
    inv[1, 0] = T * k                # past the end
    inv[2, 1] = -1 - T * k           # a dropped slot past the end
    inv[3, 0] = -2 ** 31
    rows, dy = randn((T * k, H), "f32", 1), randn((T, H), "f32", 2)
    eff = inv.numpy().copy()
    eff[1, 0] = eff[2, 1] = eff[3, 0] = -1
    y = moe.moe_combine(rows, inv.cuda())
    want, mag = ref.combine(n64(rows), eff)
    close(y, want, 4 * 2.0 ** -24 * mag, "y")
    guard = torch.full((3 * T * k, H), 7.0, device="cuda")
    moe.moe_combine_backward(dy, rows, inv.cuda(), drows=guard[T * k:2 * T * k])
    moe.moe_dispatch_rows(dy, inv.cuda(), x_perm=guard[T * k:2 * T * k])
    assert (guard[:T * k] == 7).all() and (guard[2 * T * k:] == 7).all()


def test_rows_past_two_to_the_31_elements(moe):
    """Places whose element offset passes 2^31 (8-bit copies of a short pattern)."""
    T, k, H, E = 66000, 8, 4104, 4          # 2.17e9 elements of x_perm
    g = torch.Generator().manual_seed(5)
    ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32).cuda()
    x = torch.randn((T, H), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16()
    xp, inv, off = moe.moe_dispatch(x, ids, E)
    assert int(off[E]) == T * k
    pick = torch.randint(0, T * k, (4096,), generator=g).cuda()
    assert torch.equal(xp[inv.view(-1)[pick].long()], x[pick // k])
    y = moe.moe_combine(xp, inv)             # eight times each token, exactly representable
    assert torch.equal(y, (x.float() * k).bfloat16())


# ----------------------------------------------------------------- SwiGLU and its checkpoint

def special_gu(R, I, dtype, seed):
    gu = randn((R, 2 * I), dtype, seed, 2.0)
    if R > 3:
        gu[1] = 0                                           # blocks of zeros
        gu[2, :] = 2.0 ** -14                               # one magnitude: code 448 or below
        if dtype != "f16":
            gu[3, : min(I, 5)] = 1e-39                      # subnormal blocks
    return gu


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("R,I", [(1, 1), (1, 8), (3, 31), (5, 33), (4, 40), (7, 256), (9, 264),
                                 (33, 1000), (6, 1001), (2, 4096), (130, 96)])
def test_swiglu_checkpoint(moe, R, I, dtype):
    gu = special_gu(R, I, dtype, R + I)
    h, (q, qs) = moe.moe_swiglu_ckpt(gu)
    g64 = n64(gu)
    wq, wqs = ref.quantise(g64)
    assert np.array_equal(qs.cpu().numpy(), wqs)
    assert np.array_equal(q.cpu().numpy(), wq)

    # sigma's error: __expf(-g) is within 2 + 1.173 |g| ulp, the sum, the quotient and the
    # products a few more
    def eps(g):
        return (12 + 1.2 * np.abs(g)) * 2.0 ** -23

    want = ref.swiglu(g64)
    close(h, want, U[dtype] * np.abs(want) + eps(g64[:, :I]) * np.abs(want) * (1 + U[dtype]) + TINY[dtype] + 1e-37, "h")

    k64 = ref.kept(wq, wqs)
    ok = np.abs(k64 - g64) <= np.maximum(np.abs(g64) / 16, np.concatenate(
        [np.repeat(ref.scale_of(s), 32, axis=1)[:, :I] for s in np.split(wqs, 2, 1)], 1) * 2.0 ** -10)
    assert ok.all()                          # what the header promises of the kept values
    dh = randn((R, I), dtype, 3)
    dgu, again = moe.moe_swiglu_ckpt_backward(dh, (q, qs), want_h=True)
    plain, none = moe.moe_swiglu_ckpt_backward(dh, (q, qs))
    assert none is None and torch.equal(plain, dgu)
    want = ref.swiglu(k64)
    e = eps(k64[:, :I])
    close(again, want, U[dtype] * np.abs(want) + e * np.abs(want) * (1 + U[dtype]) + TINY[dtype] + 1e-37, "h again")
    want = ref.swiglu_backward(n64(dh), k64)
    g, u = k64[:, :I], k64[:, I:]
    s = ref.sigmoid(g)
    mag = np.concatenate([np.abs(n64(dh) * u) * s * (1 + 2 * np.abs(g)), np.abs(n64(dh) * g) * s], 1)
    close(dgu, want, U[dtype] * np.abs(want) + 2 * np.concatenate([e, e], 1) * mag * (1 + U[dtype]) + TINY[dtype] + 1e-37, "dgu")


def test_checkpoint_object(moe):
    """One buffer for codes and scales, or the caller's own two tensors: the same bits; the sizes are
    checked."""
    R, I = 7, 33
    gu, dh = randn((R, 2 * I), "bf16", 1), randn((R, I), "bf16", 2)
    h, ck = moe.moe_swiglu_ckpt(gu)
    q = torch.zeros((R, 2 * I), dtype=torch.uint8, device="cuda")
    qs = torch.zeros((R, 4), dtype=torch.uint8, device="cuda")
    moe.moe_swiglu_ckpt(gu, ckpt=(q, qs))
    assert torch.equal(ck.q, q) and torch.equal(ck.q_scales, qs)
    again = moe.Checkpoint(ck.buf.clone(), R, I)
    moe.moe_swiglu_ckpt(gu, ckpt=again)
    for c in (ck, again, (q, qs)):
        assert torch.equal(moe.moe_swiglu_ckpt_backward(dh, c)[0], moe.moe_swiglu_ckpt_backward(dh, ck)[0])
    with pytest.raises(ValueError):
        moe.Checkpoint(ck.buf[:-1], R, I)
    with pytest.raises(ValueError):
        moe.moe_swiglu_ckpt_backward(dh[:6].contiguous(), ck)
    with pytest.raises(ValueError):
        moe.moe_swiglu_ckpt_backward(dh, (q, qs[:, :3].contiguous()))


def test_checkpoint_scale_boundaries(moe):
    """Largest magnitudes at, just under and just over 448 times a power of two, the type's own
    largest, and signs."""
    tops = [448.0, 449.0, 447.0, 1.75, np.nextafter(np.float32(1.75), np.float32(2)), 1.0, 2.0 ** -100,
            3.4e38, 2.0 ** -130, 2.0 ** -149, 1.75 * 2.0 ** -119, 2.0 ** -118]
    gu = torch.zeros((len(tops), 64))
    for i, v in enumerate(tops):
        gu[i, :32] = torch.linspace(-1, 1, 32) * float(np.float32(v))
        gu[i, 0] = -float(np.float32(v))
        gu[i, 32:] = float(np.float32(v)) * torch.linspace(0, 1, 32) ** 3
    _, (q, qs) = moe.moe_swiglu_ckpt(gu.cuda())
    wq, wqs = ref.quantise(gu.double().numpy())
    assert np.array_equal(qs.cpu().numpy(), wqs) and np.array_equal(q.cpu().numpy(), wq)


@pytest.mark.parametrize("I", [64, 33])
def test_checkpoint_of_infinities_and_nans(moe, I):
    """A block that is not finite reads as NaN; its neighbours are as before."""
    gu = randn((4, 2 * I), "bf16", 1)
    clean = moe.moe_swiglu_ckpt(gu)[1]
    gu[0, 3] = float("inf")
    gu[1, I + 2] = float("-inf")
    gu[2, 32] = float("nan")
    q, qs = moe.moe_swiglu_ckpt(gu)[1]
    nb = -(-I // 32)
    hit = np.zeros((4, 2 * nb), bool)
    hit[0, 0] = hit[1, nb] = hit[2, 1] = True
    assert np.array_equal(qs.cpu().numpy() == 255, hit)
    assert np.array_equal(qs.cpu().numpy()[~hit], clean[1].cpu().numpy()[~hit])
    dh = torch.ones((4, I), dtype=torch.bfloat16, device="cuda")
    dgu, h = moe.moe_swiglu_ckpt_backward(dh, (q, qs), want_h=True)
    bad = np.repeat(hit[:, :nb], 32, 1)[:, :I] | np.repeat(hit[:, nb:], 32, 1)[:, :I]
    assert np.array_equal(np.isnan(n64(h)), bad)
    assert np.isfinite(n64(dgu)[:, :I][~bad]).all() and np.isnan(n64(dgu)[:, :I][bad]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("R,I", [(3, 127), (2500, 70), (2, 129), (5, 255), (4, 257), (70, 2049), (1, 515), (40, 300)])
def test_swiglu_checkpoint_of_any_width(moe, R, I, dtype):
    test_swiglu_checkpoint(moe, R, I, dtype)


def test_swiglu_gradient_against_differences(moe):
    gu = randn((4, 80), "f32", 7)
    dh = randn((4, 40), "f32", 8)
    _, ckpt = moe.moe_swiglu_ckpt(gu)
    dgu, _ = moe.moe_swiglu_ckpt_backward(dh, ckpt)
    base, step = ref.kept(*(t.cpu().numpy() for t in ckpt)), 1e-5
    for i in np.ndindex(base.shape):
        up, dn = base.copy(), base.copy()
        up[i] += step
        dn[i] -= step
        num = ((ref.swiglu(up) - ref.swiglu(dn)) * n64(dh)).sum() / (2 * step)
        assert abs(num - n64(dgu)[i]) < 1e-4


# ------------------------------------------------------------------------ experts' products

def ragged(R, E, kind, seed):
    rng = np.random.default_rng(seed)
    if kind == "even":
        return np.linspace(0, R, E + 1).astype(np.int32)
    if kind == "last":                       # all rows with the last expert
        return np.array([0] * E + [R], np.int32)
    if kind == "first":
        return np.array([0] + [R] * E, np.int32)
    if kind == "empty":                      # no rows with any expert
        return np.zeros(E + 1, np.int32)
    cut = np.sort(rng.integers(0, R + 1, E + 1)).astype(np.int32)   # empties, a tail of no expert
    if kind != "part":                       # part: rows before the first expert's too
        cut[0] = 0
    return cut


EXPERTS = [(1, 1, 8, 8, "even"), (4, 3, 520, 3080, "cut"), (3, 1, 264, 136, "last"), (4, 200, 72, 9000, "part"), (2, 5, 2056, 72, "part"), (9, 2, 4104, 136, "cut"), (16, 256, 264, 200, "cut"),
           (13, 1, 72, 5000, "even"), (16, 3, 1032, 2056, "part"), (7, 40, 24, 16, "empty"),
           (17, 4, 136, 520, "cut"), (1, 3, 16, 24, "last"), (5, 4, 72, 8, "cut"), (127, 2, 64, 256, "cut"),
           (128, 1, 64, 128, "even"), (129, 1, 136, 264, "even"), (255, 1, 128, 256, "first"),
           (257, 1, 320, 520, "even"), (300, 7, 200, 136, "cut"), (513, 256, 64, 64, "cut"),
           (700, 3, 328, 1032, "cut"), (64, 5, 512, 512, "empty"), (2100, 2, 72, 72, "cut"),
           (1024, 4, 1024, 512, "even"), (2000, 1, 192, 2056, "even"), (40, 256, 256, 256, "cut"),
           (700, 3, 64, 96, "part"), (900, 255, 64, 40, "part"), (2600, 256, 32, 32, "part")]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("R,E,K,N,kind", EXPERTS)
def test_experts_products(moe, R, E, K, N, kind, dtype):
    off = ragged(R, E, kind, R + E)
    offsets = torch.from_numpy(off).cuda()
    x, dy = randn((R, K), dtype, 1), randn((R, N), dtype, 2)
    w = randn((E, N, K), dtype, 3, K ** -0.5)
    for t in (x, dy):                        # rows of no expert reach nothing
        t[off[E]:] = float("nan")
        t[:off[0]] = float("nan")
    X, Y, W = n64(x), n64(dy), n64(w)
    scratch = moe.alloc_experts_scratch(E)
    got = {"y": moe.moe_experts_matmul(x, w, offsets, scratch=scratch),
           "dx": moe.moe_experts_matmul_dx(dy, w, offsets, scratch=scratch),
           "dw": moe.moe_experts_matmul_dw(dy, x, offsets, scratch=scratch)}
    assert moe.moe_read_device_status(scratch) == (moe.MOE_OK, 0)
    rows = max(np.diff(off).max(), 1)
    for name, f, a, b, n in (("y", ref.experts_matmul, X, W, K), ("dx", ref.experts_matmul_dx, Y, W, N),
                             ("dw", ref.experts_matmul_dw, Y, X, rows)):
        want = f(a, b, off)
        mag = f(np.abs(a), np.abs(b), off)
        close(got[name], want, U[dtype] * np.abs(want) + n * 2.0 ** -23 * mag * (1 + U[dtype]) + TINY[dtype], name)
    want, mag = ref.experts_matmul_dw(Y, X, off), ref.experts_matmul_dw(np.abs(Y), np.abs(X), off)
    dw = moe.moe_experts_matmul_dw(dy, x, offsets, dw_dtype=torch.float32)
    close(dw, want, rows * 2.0 ** -23 * mag + 1e-40, "dw f32")
    start = randn((E, N, K), "f32", 4)
    sum_ = start.clone()
    moe.moe_experts_matmul_dw(dy, x, offsets, dw=sum_, accumulate=True)
    assert torch.equal(sum_, start + dw)     # one fp32 addition an element


SPLITS = [(100, 1, 6200, 136, "even"), (40, 2, 4104, 264, "cut"), (300, 1, 136, 6504, "part"),
          (9000, 1, 72, 264, "even"), (6500, 2, 136, 264, "cut"), (1500, 3, 256, 256, "part"),
          (513, 2, 520, 8200, "last"), (700, 2, 3080, 40, "empty"), (200, 3, 14344, 72, "cut")]


def test_which_contractions_are_split(moe):
    """Each product is in some of the cases of the next test (the sixth: in none, a short one)."""
    for p in range(3):
        assert sum(moe._lib.moe_experts_split_bytes(p, R, E, N, K) > 0 for R, E, K, N, _ in SPLITS) >= 2


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("R,E,K,N,kind", SPLITS)
def test_split_contractions(moe, R, E, K, N, kind, dtype):
    """Few tiles and a long contraction: parts of it side by side, where the workspace holds their
    sums. As close, and the same on every run."""
    off = ragged(R, E, kind, R + E)
    offsets = torch.from_numpy(off).cuda()
    x, dy, w = randn((R, K), dtype, 1), randn((R, N), dtype, 2), randn((E, N, K), dtype, 3, K ** -0.5)
    for t in (x, dy):
        t[off[E]:] = float("nan")
        t[:off[0]] = float("nan")
    X, Y, W = n64(x), n64(dy), n64(w)
    scratch = moe.alloc_experts_scratch(E, R, N, K)
    runs = []
    for sc in (scratch, None, scratch):
        if sc is not None:
            sc.buf[16:].fill_(0xFF)          # NaNs: nothing of it is read before it is written
        runs.append((moe.moe_experts_matmul(x, w, offsets, scratch=sc),
                     moe.moe_experts_matmul_dx(dy, w, offsets, scratch=sc),
                     moe.moe_experts_matmul_dw(dy, x, offsets, scratch=sc)))
    assert moe.moe_read_device_status(scratch) == (moe.MOE_OK, 0)
    for again in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], again))
    rows = max(np.diff(off).max(), 1)
    for name, got, f, a, b, n in (("y", runs[0][0], ref.experts_matmul, X, W, K),
                                  ("dx", runs[0][1], ref.experts_matmul_dx, Y, W, N),
                                  ("dw", runs[0][2], ref.experts_matmul_dw, Y, X, rows)):
        want, mag = f(a, b, off), f(np.abs(a), np.abs(b), off)
        close(got, want, U[dtype] * np.abs(want) + (n + 8) * 2.0 ** -23 * mag * (1 + U[dtype]) + TINY[dtype], name)
    dw = moe.moe_experts_matmul_dw(dy, x, offsets, dw_dtype=torch.float32)
    want, mag = ref.experts_matmul_dw(Y, X, off), ref.experts_matmul_dw(np.abs(Y), np.abs(X), off)
    close(dw, want, (rows + 8) * 2.0 ** -23 * mag + 1e-40, "dw f32")
    start = randn((E, N, K), "f32", 4)
    sum_ = start.clone()
    moe.moe_experts_matmul_dw(dy, x, offsets, dw=sum_, accumulate=True)
    assert torch.equal(sum_, start + dw)


@pytest.mark.parametrize("start", [8, 16])
@pytest.mark.parametrize("K", [8, 24, 72, 248, 264, 328, 776])
def test_dw_writes_its_own_elements_only(moe, K, start):
    """Rows of an odd number of 16 bytes, in a dw that starts on 16 or on 32 bytes; experts without
    rows beside others."""
    R, E, N = 150, 6, 136
    off = np.array([0, 0, 70, 71, 71, 140, 140], np.int32)
    offsets = torch.from_numpy(off).cuda()
    x, dy = randn((R, K), "bf16", 1), randn((R, N), "bf16", 2)
    buf = torch.full((E * N * K + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    dw = buf[start:start + E * N * K].view(E, N, K)
    moe.moe_experts_matmul_dw(dy, x, offsets, dw=dw)
    assert (buf[:start] == 7).all() and (buf[start + E * N * K:] == 7).all()
    want, mag = ref.experts_matmul_dw(n64(dy), n64(x), off), ref.experts_matmul_dw(np.abs(n64(dy)), np.abs(n64(x)), off)
    close(dw, want, U["bf16"] * np.abs(want) + 70 * 2.0 ** -23 * mag * (1 + U["bf16"]) + TINY["bf16"], "dw")


def test_a_neighbours_rows_do_not_reach_dw(moe):
    """Infinities and NaNs in the rows right behind (and before) an expert's leave its dw alone."""
    R, E, K, N = 200, 3, 64, 128
    off = np.array([0, 70, 133, 200], np.int32)
    x, dy = randn((R, K), "bf16", 1), randn((R, N), "bf16", 2)
    offsets = torch.from_numpy(off).cuda()
    clean = moe.moe_experts_matmul_dw(dy, x, offsets)
    x[:70] = float("nan")
    dy[133:] = float("inf")
    got = moe.moe_experts_matmul_dw(dy, x, offsets)
    assert torch.equal(got[1], clean[1]) and torch.isnan(got[0]).all()


def test_experts_products_repeat_bit_for_bit_and_on_another_stream(moe):
    R, E, K, N = 1111, 9, 264, 520
    offsets = torch.from_numpy(ragged(R, E, "cut", 4)).cuda()
    x, dy, w = randn((R, K), "bf16", 1), randn((R, N), "bf16", 2), randn((E, N, K), "bf16", 3)
    first = (moe.moe_experts_matmul(x, w, offsets), moe.moe_experts_matmul_dx(dy, w, offsets),
             moe.moe_experts_matmul_dw(dy, x, offsets))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(3):
            # made on this stream, right before
            x2, dy2, w2, o2 = x.clone(), dy.clone(), w.clone(), offsets.clone()
            again = (moe.moe_experts_matmul(x2, w2, o2), moe.moe_experts_matmul_dx(dy2, w2, o2),
                     moe.moe_experts_matmul_dw(dy2, x2, o2))
    side.synchronize()
    for a, b in zip(first, again):
        assert torch.equal(a, b)


def test_offsets_out_of_order_stay_in_range(moe):
    """Offsets that are not offsets give some result but touch nothing outside the tensors."""
    R, E, K, N = 300, 4, 64, 64
    x, dy, w = randn((R, K), "bf16", 1), randn((R, N), "bf16", 2), randn((E, N, K), "bf16", 3)
    offsets = torch.tensor([-5, 400, 20, -1, 10 ** 9], dtype=torch.int32).cuda()
    guard = torch.full((3 * R, N), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_experts_matmul(x, w, offsets, y=guard[R:2 * R])
    assert (guard[:R] == 7).all() and (guard[2 * R:] == 7).all()
    moe.moe_experts_matmul_dx(dy, w, offsets)
    moe.moe_experts_matmul_dw(dy, x, offsets)
    torch.cuda.synchronize()


def test_products_over_two_to_the_31_elements(moe):
    """Results and weights whose element offsets pass 2^31, at their ends."""
    R, E, K, N = 70000, 2, 64, 32768
    off = np.array([0, 100, R], np.int32)
    offsets = torch.from_numpy(off).cuda()
    x, w = randn((R, K), "bf16", 1), randn((E, N, K), "bf16", 2, K ** -0.5)
    y = moe.moe_experts_matmul(x, w, offsets)
    for r in (0, 99, 100, 65535, 65536, 65537, R - 1):
        e = int(r >= 100)
        want = n64(w[e]) @ n64(x[r])
        mag = np.abs(n64(w[e])) @ np.abs(n64(x[r]))
        close(y[r], want, U["bf16"] * np.abs(want) + K * 2.0 ** -23 * mag * 1.01, "y")
    del y
    E, N, K, R = 200, 4096, 2688, 400         # dw of 2.2e9 elements
    off = np.linspace(0, R, E + 1).astype(np.int32)
    dy, x = randn((R, N), "bf16", 3), randn((R, K), "bf16", 4)
    dw = moe.moe_experts_matmul_dw(dy, x, torch.from_numpy(off).cuda())
    for e in (0, 194, 195, 199):
        a, b = off[e], off[e + 1]
        want = n64(dy[a:b]).T @ n64(x[a:b])
        mag = np.abs(n64(dy[a:b])).T @ np.abs(n64(x[a:b]))
        close(dw[e], want, U["bf16"] * np.abs(want) + (b - a) * 2.0 ** -23 * mag * 1.01, "dw")


def test_dw_of_odd_rows_over_two_to_the_31_elements(moe):
    E, N, K, R = 200, 4096, 2696, 398         # the last expert has no rows
    off = np.minimum(np.arange(E + 1) * 2, R).astype(np.int32)
    dy, x = randn((R, N), "bf16", 3), randn((R, K), "bf16", 4)
    dw = moe.moe_experts_matmul_dw(dy, x, torch.from_numpy(off).cuda())
    for e in (0, 194, 195, 198, 199):
        a, b = off[e], off[e + 1]
        want = n64(dy[a:b]).T @ n64(x[a:b])
        mag = np.abs(n64(dy[a:b])).T @ np.abs(n64(x[a:b]))
        close(dw[e], want, U["bf16"] * np.abs(want) + (b - a) * 2.0 ** -23 * mag * 1.01, "dw")


# ------------------------------------------------------------------------------ the router

ROUTES = [(1, 1, 1), (3, 8, 8), (70, 60, 4), (257, 256, 8), (33, 33, 1), (5000, 16, 2)]


@pytest.mark.parametrize("method", [0, 1, 2, 3, 4, 5, 6, 16])
@pytest.mark.parametrize("T,E,k", ROUTES)
def test_route_backward(moe, T, E, k, method):
    rng = np.random.default_rng(T + E + method)
    logits = torch.from_numpy((rng.standard_normal((T, E)) * 3).astype(np.float32)).cuda()
    ids = np.argsort(-rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
    if T > 40:
        ids[5, 0] = -1                       # a dropped slot
        logits[6, int(ids[6, 0])] = float("-inf")
        logits[7] = float("nan")             # nothing finite
        logits[8, int(ids[8, 0])] = 80.0     # nearly one-hot
        logits[9] = -80.0
    ds = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda()
    rsf = 2.5 if method in (2, 16) else 1.0
    got = moe.moe_route_backward(logits, torch.from_numpy(ids).cuda(), ds, method, rsf)
    want, mag = ref.route_backward(logits.cpu().numpy(), ids, n64(ds), method, rsf)
    # expf within 2 ulp; k + log2(E) sums, two quotients and a few products
    close(got, want, 40 * 2.0 ** -24 * mag + 1e-37, "dlogits")


@pytest.mark.parametrize("method", [0, 1, 2, 3, 4, 5, 6, 16])
def test_route_backward_of_slots_that_take_no_part(moe, method):
    """What comes in for a dropped slot, or one whose logit is not finite, reaches nothing."""
    rng = np.random.default_rng(method)
    logits = torch.from_numpy(rng.standard_normal((3, 16)).astype(np.float32)).cuda()
    ids = torch.tensor([[1, 5, 9], [2, -1, 4], [0, 16, 3]], dtype=torch.int32).cuda()
    logits[0, 5] = float("nan")
    ds = torch.from_numpy(rng.standard_normal((3, 3)).astype(np.float32)).cuda()
    ds[:, 1] = 0
    want = moe.moe_route_backward(logits, ids, ds, method, 2.5)
    ds[:, 1] = float("nan")
    assert torch.equal(moe.moe_route_backward(logits, ids, ds, method, 2.5), want)
    assert torch.isfinite(want).all()


@pytest.mark.parametrize("method", [0, 1, 2, 3, 4, 5, 6, 16])
def test_route_gradient_against_differences(moe, method):
    rng = np.random.default_rng(method)
    T, E, k, rsf, step = 4, 12, 3, 2.5, 1e-5
    logits = rng.standard_normal((T, E)).astype(np.float32)
    ids = np.argsort(-logits, axis=1)[:, :k].astype(np.int32)
    ds = rng.standard_normal((T, k)).astype(np.float32)
    got = n64(moe.moe_route_backward(torch.from_numpy(logits).cuda(), torch.from_numpy(ids).cuda(),
                                     torch.from_numpy(ds).cuda(), method, rsf))
    for t in range(T):
        for e in range(E):
            up, dn = logits.astype(np.float64), logits.astype(np.float64)
            up[t, e] += step
            dn[t, e] -= step
            num = ((ref.route_weights(up, ids, method, rsf) - ref.route_weights(dn, ids, method, rsf)) * ds).sum() / (2 * step)
            assert abs(num - got[t, e]) < 1e-5


@pytest.mark.parametrize("method", [0, 1, 2, 3, 4, 5, 6])
def test_the_weights_whose_gradient_is_taken_are_the_routers(moe, method):
    """The formula differentiated here gives moe_route's own scales for the ids it chose."""
    rng = np.random.default_rng(3)
    logits = torch.from_numpy(rng.standard_normal((50, 64)).astype(np.float32)).cuda()
    kw = dict(n_group=4, topk_group=2, routed_scaling_factor=2.5) if method == 2 else {}
    ids, scales = moe.moe_route(logits, method, 4, **kw)
    want = ref.route_weights(logits.cpu().numpy(), ids.cpu().numpy(), method, 2.5)
    np.testing.assert_allclose(scales.cpu().numpy(), want, rtol=1e-6)


# ---------------------------------------------------------------------------------- graphs

def test_operators_in_a_captured_graph(moe):
    """Captured once and replayed on other values in the same tensors: what the calls give outside."""
    T, H, I, E, k = 70, 128, 96, 6, 3
    ids = torch.from_numpy(make_ids(T, E, k, "dropped", 1)).cuda()
    x, w13, w2 = randn((T, H), "bf16", 1), randn((E, 2 * I, H), "bf16", 2, 0.1), randn((E, H, I), "bf16", 3, 0.1)
    scales, dy, logits = torch.rand((T, k)).cuda(), randn((T, H), "bf16", 4), randn((T, E), "f32", 5)

    def step():
        xp, inv, off = moe.moe_dispatch(x, ids, E)
        h, ck = moe.moe_swiglu_ckpt(moe.moe_experts_matmul(xp, w13, off))
        rows = moe.moe_experts_matmul(h, w2, off)
        y = moe.moe_combine(rows, inv, scales)
        drows, ds = moe.moe_combine_backward(dy, rows, inv, scales)
        dgu, h2 = moe.moe_swiglu_ckpt_backward(moe.moe_experts_matmul_dx(drows, w2, off), ck, want_h=True)
        return (xp, inv, off, y, ds, moe.moe_experts_matmul_dw(drows, h2, off),
                moe.moe_experts_matmul_dw(dgu, xp, off),
                moe.moe_dispatch_backward(moe.moe_experts_matmul_dx(dgu, w13, off), inv),
                moe.moe_route_backward(logits, ids, ds, 4))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    x.copy_(randn((T, H), "bf16", 11))
    ids.copy_(torch.from_numpy(make_ids(T, E, k, "dropped", 12)))
    dy.copy_(randn((T, H), "bf16", 13))
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(out, step()):
        assert torch.equal(a, b)


# ------------------------------------------------------------------------- empty and refused

def test_no_rows(moe):
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    ids = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    xp, inv, off = moe.moe_dispatch(x, ids, 4)
    assert xp.shape == (0, 64) and (off == 0).all()
    assert moe.moe_combine(xp, inv).shape == (0, 64)
    w = randn((4, 32, 64), "bf16", 1)
    assert moe.moe_experts_matmul(xp, w, off).shape == (0, 32)
    dy = torch.empty((0, 32), dtype=torch.bfloat16, device="cuda")
    assert (moe.moe_experts_matmul_dw(dy, xp, off) == 0).all()
    start = torch.ones((4, 32, 64), device="cuda")
    moe.moe_experts_matmul_dw(dy, xp, off, dw=start, accumulate=True)
    assert (start == 1).all()
    h, ckpt = moe.moe_swiglu_ckpt(torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"))
    assert moe.moe_swiglu_ckpt_backward(h, ckpt)[0].shape == (0, 64)


def test_wrappers_refuse(moe):
    x = randn((4, 64), "bf16", 1)
    ids = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        moe.moe_dispatch(x, ids.long(), 4)
    with pytest.raises(ValueError):
        moe.moe_dispatch(x.double(), ids, 4)
    with pytest.raises(ValueError):
        moe.moe_dispatch(x[:, ::2], ids, 4)
    with pytest.raises(ValueError):
        moe.moe_dispatch(x[:3], ids, 4)
    with pytest.raises(moe.MoeError):
        moe.moe_dispatch(x, ids, 300)
    with pytest.raises(moe.MoeError):
        moe.moe_dispatch(randn((8, 64), "bf16", 1).view(-1)[4:4 + 256].view(4, 64), ids, 4)   # off by 8 bytes
    _, inv, off = moe.moe_dispatch(x, ids, 4)
    with pytest.raises(ValueError):
        moe.moe_combine(x, inv)
    with pytest.raises(ValueError):
        moe.moe_combine(randn((8, 64), "bf16", 1), inv, torch.ones((4, 3), device="cuda"))
    w = randn((4, 32, 64), "bf16", 1)
    with pytest.raises(ValueError):
        moe.moe_experts_matmul(x, w.half(), off)
    with pytest.raises(ValueError):
        moe.moe_experts_matmul(x, w, off[:4].contiguous())
    with pytest.raises(moe.MoeError):
        moe.moe_experts_matmul(x.float(), w.float(), off)
    with pytest.raises(moe.MoeError):
        moe.moe_experts_matmul(randn((4, 12), "bf16", 1), randn((4, 32, 12), "bf16", 1), off)
    with pytest.raises(ValueError):
        moe.moe_experts_matmul_dw(x, x, off, accumulate=True)
    with pytest.raises(moe.MoeError):
        moe.moe_experts_matmul_dw(x, x, off, dw=torch.zeros((4, 64, 64), dtype=torch.bfloat16, device="cuda"), accumulate=True)
    with pytest.raises(ValueError):
        moe.moe_swiglu_ckpt(randn((4, 63), "bf16", 1))
    with pytest.raises(moe.MoeError):
        moe.moe_route_backward(torch.zeros((4, 8), device="cuda"), ids, torch.zeros((4, 2), device="cuda"), 17)
