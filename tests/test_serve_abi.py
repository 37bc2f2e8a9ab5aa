"""CPU: what the serving operators refuse before anything is launched, and the float64 restatement that the
GPU tests compare with. Nothing here may be launched: every address is made up, so on a machine with a GPU
only calls whose refusal does not depend on one are made."""
import ctypes
import os
import shutil

import numpy as np
import pytest
import torch

from oracle import serve_oracle as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
GOOD = ctypes.c_void_p(1 << 20)         # never dereferenced: every call here is refused first
ODD = ctypes.c_void_p((1 << 20) + 8)
BYTE = ctypes.c_void_p((1 << 20) + 1)
INVALID, UNSUPPORTED, SMALL = 1, 2, 3


@pytest.fixture(scope="module")
def moe():
    if not os.path.exists(os.path.join(ROOT, "mixture_experts_layer_03_gb300", "libmoe_gb300.so")):
        if not (shutil.which("nvcc") or os.path.exists("/usr/local/cuda/bin/nvcc")):
            pytest.skip("library not built and nvcc unavailable")
        import __graft_entry__
        __graft_entry__.build()
    import mixture_experts_layer_03_gb300 as m
    return m


@pytest.mark.parametrize("kw,status", [
    (dict(planes=-1), UNSUPPORTED), (dict(rows=-1), UNSUPPORTED), (dict(planes=1 << 20, rows=1 << 20), UNSUPPORTED),
    (dict(planes=1 << 62, rows=4), UNSUPPORTED), (dict(K=0), UNSUPPORTED), (dict(K=48), UNSUPPORTED),
    (dict(K=65568), UNSUPPORTED), (dict(dt=3), UNSUPPORTED), (dict(fmt=2), UNSUPPORTED), (dict(fmt=-1), UNSUPPORTED),
    (dict(fmt=0, g=GOOD), INVALID), (dict(g=BYTE), INVALID), (dict(a=None), INVALID), (dict(a=ODD), INVALID),
    (dict(codes=None), INVALID), (dict(codes=ODD), INVALID), (dict(scales=ODD), INVALID), (dict(scales=None), INVALID)])
def test_conversions_refuse(moe, kw, status):
    kw = dict(a=GOOD, planes=2, rows=4, K=64, dt=0, fmt=1, g=None, codes=GOOD, scales=GOOD) | kw
    L = moe._lib
    a, p, r, K, dt, fmt, g, c, s = kw.values()
    assert L.moe_quantize_fp4(a, p, r, K, dt, fmt, g, c, s, None) == status
    assert moe._lib.moe_last_error()
    assert L.moe_dequantize_fp4(c, s, g, p, r, K, fmt, dt, a, None) == status
    if p == 2:
        assert L.moe_swiglu_fp4(a, r, K, dt, fmt, g, c, s, None) == status


def test_nothing_to_do(moe):
    L = moe._lib
    assert L.moe_quantize_fp4(None, 0, 4, 64, 0, 0, None, None, None, None) == 0
    assert L.moe_quantize_fp4(None, 4, 0, 64, 0, 0, None, None, None, None) == 0
    assert L.moe_swiglu_fp4(None, 0, 64, 0, 1, None, None, None, None) == 0
    assert L.moe_dequantize_fp4(None, None, None, 1, 0, 64, 1, 0, None, None) == 0
    assert L.moe_experts_matmul_fp4(None, None, None, None, None, None, None, 0, 2, 64, 64, 0, 0, None, None) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(R=-1), UNSUPPORTED), (dict(R=(1 << 23) + 1), UNSUPPORTED), (dict(E=0), UNSUPPORTED),
    (dict(E=257), UNSUPPORTED), (dict(N=12), UNSUPPORTED), (dict(N=0), UNSUPPORTED), (dict(N=65544), UNSUPPORTED),
    (dict(K=16), UNSUPPORTED), (dict(K=72), UNSUPPORTED), (dict(K=65568), UNSUPPORTED), (dict(dt=2), UNSUPPORTED),
    (dict(fmt=2), UNSUPPORTED), (dict(fmt=0, xg=GOOD), INVALID), (dict(fmt=0, wg=GOOD), INVALID),
    (dict(wg=BYTE), INVALID), (dict(x=None), INVALID), (dict(x=ODD), INVALID), (dict(xs=ODD), INVALID),
    (dict(w=None), INVALID), (dict(ws=ODD), INVALID), (dict(off=None), INVALID), (dict(off=BYTE), INVALID),
    (dict(y=None), INVALID), (dict(y=ODD), INVALID)])
def test_products_refuse(moe, kw, status):
    kw = dict(x=GOOD, xs=GOOD, xg=None, w=GOOD, ws=GOOD, wg=None, off=GOOD, R=4, E=2, N=64, K=64, fmt=1, dt=0, y=GOOD) | kw
    assert moe._lib.moe_experts_matmul_fp4(*kw.values(), None) == status
    assert moe._lib.moe_last_error()


def test_wrappers_refuse(moe):
    x = torch.zeros(4, 64).bfloat16()
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_quantize_fp4(x, moe.MOE_FP4_MX)
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_swiglu_fp4(x, moe.MOE_FP4_NV)
    with pytest.raises(ValueError, match="CUDA"):
        moe.Fp4(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 16, dtype=torch.uint8), moe.MOE_FP4_MX)
    with pytest.raises(ValueError, match="format"):
        moe.Fp4(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 16, dtype=torch.uint8), 2)
    with pytest.raises(ValueError, match="rows"):
        moe.Fp4(torch.zeros(32, dtype=torch.uint8), torch.zeros(16, dtype=torch.uint8), 0)


class OnGpu(torch.Tensor):
    """A CPU tensor that passes for a CUDA one."""
    is_cuda = True


def fake(shape, dtype):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)


def test_shapes_types_and_formats_are_checked(moe, monkeypatch):
    u8 = torch.uint8
    q = moe.Fp4(fake((3, 4, 48), u8), fake((3, 4, 16), u8), moe.MOE_FP4_NV, fake((3,), torch.float32))
    assert q.shape == (3, 4, 96)
    for kw in (dict(scales=fake((3, 4, 6), u8)),                     # not filled up to 16
               dict(scales=fake((3, 5, 16), u8)), dict(codes=fake((3, 4, 48), torch.int8)),
               dict(g=fake((1,), torch.float32)), dict(g=fake((3,), torch.float64)), dict(fmt=moe.MOE_FP4_MX)):
        a = dict(codes=q.codes, scales=q.scales, fmt=q.format, g=q.g) | kw
        with pytest.raises(ValueError):
            moe.Fp4(*a.values())
    launched = []
    for name in ("moe_quantize_fp4", "moe_swiglu_fp4", "moe_dequantize_fp4", "moe_experts_matmul_fp4"):
        monkeypatch.setattr(moe._lib, name, lambda *a, n=name: launched.append(n) or 0)
    monkeypatch.setattr(moe, "_stream", lambda s: 0)
    monkeypatch.setattr(moe, "_new", lambda shape, dtype, device, stream, result=True: fake(shape, dtype))
    x = fake((4, 96), torch.bfloat16)
    off = fake((4,), torch.int32)
    xq = moe.moe_quantize_fp4(x, moe.MOE_FP4_NV)
    assert xq.shape == (4, 96) and xq.scales.shape == (4, 16) and launched == ["moe_quantize_fp4"]
    assert moe.moe_experts_matmul_fp4(xq, q, off).shape == (4, 4)
    assert moe.moe_dequantize_fp4(q).shape == (3, 4, 96)
    assert moe.moe_swiglu_fp4(fake((5, 192), torch.float32), 0).shape == (5, 96)
    n = len(launched)
    mx = moe.moe_quantize_fp4(x, moe.MOE_FP4_MX)
    for call in (lambda: moe.moe_quantize_fp4(fake((4, 80), torch.bfloat16), 0),       # 80 channels
                 lambda: moe.moe_quantize_fp4(x, 5), lambda: moe.moe_quantize_fp4(x, 0, fake((1,), torch.float32)),
                 lambda: moe.moe_quantize_fp4(x, 1, fake((4,), torch.float32)),
                 lambda: moe.moe_quantize_fp4(x, 1, out=mx), lambda: moe.moe_quantize_fp4(fake((4, 96), torch.int32), 0),
                 lambda: moe.moe_swiglu_fp4(fake((4, 95), torch.bfloat16), 0),
                 lambda: moe.moe_swiglu_fp4(fake((4, 96), torch.bfloat16), 0),          # 48 channels
                 lambda: moe.moe_dequantize_fp4(q, torch.int32),
                 lambda: moe.moe_dequantize_fp4(q, out=fake((3, 4, 95), torch.bfloat16)),
                 lambda: moe.moe_experts_matmul_fp4(mx, q, off), lambda: moe.moe_experts_matmul_fp4(q, q, off),
                 lambda: moe.moe_experts_matmul_fp4(xq, xq, off), lambda: moe.moe_experts_matmul_fp4(xq, q, off[:3]),
                 lambda: moe.moe_experts_matmul_fp4(xq, q, off, y=fake((4, 5), torch.bfloat16))):
        with pytest.raises(ValueError):
            call()
    assert len(launched) == n + 1


# ------------------------------------------------------------------------- the restatement

def test_e2m1_by_hand():
    v = np.array([0.0, 0.25, 0.26, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.1, 99.0])
    assert ref._nearest(v, ref.E2M1).tolist() == [0, 0, 1, 2, 2, 4, 4, 6, 6, 7, 7]


def test_quantize_by_hand():
    x = np.zeros((2, 32))
    x[0, :4] = 6.0, -3.0, 0.25, -0.1
    x[1, 16:18] = 7.0, 1.0
    codes, scales = ref.quantize(x, ref.MX)
    assert codes[0, :3].tolist() == [7 | 13 << 4, 0 | 8 << 4, 0] and scales[:, 0].tolist() == [127, 128]
    assert codes[1, 8] == 6 | 1 << 4                     # 3.5 -> 4, 0.5, of 2
    assert not scales[:, 1:].any()
    codes, scales = ref.quantize(x, ref.NV, 0.5)
    assert scales[:, :2].tolist() == [[64, 0], [0, 65]]  # 6 / (6 g) = 2 and 7 / (6 g) = 2.33, held as 2.25
    assert ref.dequantize(codes, scales, ref.NV, 0.5)[0, :3].tolist() == [6.0, -3.0, 0.0]


def test_values_that_are_held_exactly_come_back():
    rng = np.random.default_rng(1)
    for fmt in (ref.MX, ref.NV):
        b = ref.BLOCK[fmt]
        v = rng.choice(ref.E2M1, (5, 8, b)) * rng.choice([-1, 1], (5, 8, b))
        v[:, :, 0] = 6
        s = 2.0 ** rng.integers(-5, 8, (5, 8, 1))
        x = (v * s).reshape(5, -1)
        assert np.array_equal(ref.dequantize(*ref.quantize(x, fmt), fmt), x)


def test_the_error_is_half_a_step():
    x = np.random.default_rng(2).standard_normal((20, 512))
    for fmt in (ref.MX, ref.NV):
        b = ref.BLOCK[fmt]
        err = np.abs(ref.dequantize(*ref.quantize(x, fmt), fmt) - x).reshape(20, -1, b)
        top = np.abs(x).reshape(20, -1, b).max(2, keepdims=True)
        # the largest step is 2 of 6, the mx scale up to twice, the nv scale 1/16 more than needed
        assert (err <= top * (1 / 3 if fmt == ref.MX else 1 / 6 * (1 + 1 / 16))).all()


# ------------------------------------------------------------------------- the layer for a few tokens

def few(moe, T=4, H=64, I=32, E=8, k=2, shared_I=0, method=1, gate=0, weights=-1, dt=0, bias=None, x=GOOD, wg=GOOD,
        w=GOOD, s=GOOD, g=None, w2=True, shared=True, ids=GOOD, scales=GOOD, y=GOOD, ws=ctypes.c_void_p(1 << 20), n=1 << 24,
        r_E=None, r_k=None, n_group=1):
    p = moe.MoeProblem(T, H, I, E, k, shared_I)
    r = moe.MoeRouteParams(r_E or E, r_k or k, method, n_group, 1, 1.0)
    m = moe.MoeWeights(w, s, g)
    ref_m = ctypes.byref(m)
    return moe._lib.moe_layer_few(ctypes.byref(p), ctypes.byref(r), x, wg, gate, bias, ref_m, ref_m if w2 else None,
                                  ref_m if shared else None, ref_m if shared else None, weights, dt, ids, scales, y, ws, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), UNSUPPORTED), (dict(T=17), UNSUPPORTED), (dict(H=48), UNSUPPORTED), (dict(H=0), UNSUPPORTED),
    (dict(H=32800), UNSUPPORTED), (dict(I=16), UNSUPPORTED), (dict(I=65568), UNSUPPORTED), (dict(shared_I=8), UNSUPPORTED),
    (dict(shared_I=-32), UNSUPPORTED), (dict(E=0), UNSUPPORTED), (dict(E=257), UNSUPPORTED), (dict(k=0), UNSUPPORTED),
    (dict(k=9, E=16), UNSUPPORTED), (dict(k=4, E=3), UNSUPPORTED), (dict(weights=2), UNSUPPORTED),
    (dict(weights=-2), UNSUPPORTED), (dict(dt=2), UNSUPPORTED), (dict(method=7), UNSUPPORTED), (dict(method=17), UNSUPPORTED),
    (dict(method=2, n_group=3), UNSUPPORTED), (dict(r_E=7), INVALID), (dict(r_k=1), INVALID), (dict(gate=1), INVALID),
    (dict(gate=2, shared_I=32), INVALID), (dict(method=16, bias=GOOD), INVALID), (dict(x=None), INVALID),
    (dict(x=ODD), INVALID), (dict(wg=ODD), INVALID), (dict(bias=ODD), INVALID), (dict(ids=None), INVALID),
    (dict(scales=ODD), INVALID), (dict(y=None), INVALID), (dict(w=None), INVALID), (dict(w=ODD), INVALID),
    (dict(w2=False), INVALID), (dict(shared=False, shared_I=32), INVALID), (dict(weights=0, s=None), INVALID),
    (dict(weights=1, s=ODD), INVALID), (dict(weights=0, g=GOOD), INVALID), (dict(g=GOOD), INVALID),
    (dict(weights=1, g=BYTE), INVALID), (dict(ws=None), INVALID), (dict(ws=ctypes.c_void_p((1 << 20) + 128)), INVALID),
    (dict(n=100), SMALL)])
def test_layer_few_refuses(moe, kw, status):
    assert few(moe, **kw) == status
    assert moe._lib.moe_last_error()


def test_layer_few_without_tokens_and_its_workspace(moe):
    assert few(moe, T=0, x=None, wg=None, w=None, y=None, ws=None) == 0
    assert moe._lib.moe_layer_few(None, None, *[None] * 2, 0, *[None] * 5, -1, 0, *[None] * 4, 0, None) == INVALID
    n = lambda *a: moe._lib.moe_layer_few_workspace_bytes(ctypes.byref(moe.MoeProblem(*a)))   # noqa: E731
    assert n(17, 64, 32, 8, 2, 0) == 0 == n(4, 48, 32, 8, 2, 0) == n(4, 64, 32, 257, 2, 0)
    # counters and sizes, logits [T, E], the shared gate's, h [T, k + 1, the wider of both] in f32
    assert n(16, 7168, 2048, 256, 8, 4096) == 256 + 4 * 16 * 256 + 256 + 4 * 16 * 9 * 4096
    assert n(0, 64, 32, 8, 2, 0) == 512


def test_layer_few_wrapper_refuses(moe, monkeypatch):
    launched = []
    monkeypatch.setattr(moe._lib, "moe_layer_few", lambda *a: launched.append(a) or 0)
    monkeypatch.setattr(moe, "_stream", lambda s: 0)
    monkeypatch.setattr(moe, "_new", lambda shape, dtype, device, stream, result=True: fake(shape, dtype))
    b16 = torch.bfloat16
    x, wg, w13, w2 = fake((3, 64), b16), fake((4, 64), b16), fake((4, 64, 64), b16), fake((4, 64, 32), b16)
    y, ids, sc = moe.moe_layer_few(x, wg, w13, w2, 1, 2)
    assert y.shape == (3, 64) and ids.shape == (3, 2) and sc.dtype == torch.float32 and len(launched) == 1
    q13 = moe.Fp4(fake((4, 64, 32), torch.uint8), fake((4, 64, 16), torch.uint8), moe.MOE_FP4_MX)
    q2 = moe.Fp4(fake((4, 64, 16), torch.uint8), fake((4, 64, 16), torch.uint8), moe.MOE_FP4_MX)
    q2nv = moe.Fp4(fake((4, 64, 16), torch.uint8), fake((4, 64, 16), torch.uint8), moe.MOE_FP4_NV)
    moe.moe_layer_few(x, wg, q13, q2, 1, 2)
    for a, kw in (((x.float(), wg, w13, w2), {}), ((x, fake((6, 64), b16), w13, w2), {}), ((x, fake((4, 32), b16), w13, w2), {}),
                  ((x, wg.half(), w13, w2), {}), ((x, wg, w13[0], w2), {}), ((x, wg, w13, fake((4, 64, 33), b16)), {}),
                  ((x, wg, w13, q2), {}), ((x, wg, q13, w2), {}), ((x, wg, q13, q2nv), {}), ((x, wg, w13.half(), w2.half()), {}),
                  ((x, wg, w13, w2), dict(w13_s=fake((64, 64), b16))), ((x, wg, w13, w2), dict(bias=fake((3,), torch.float32))),
                  ((x, wg, w13, w2), dict(y=fake((3, 63), b16))), ((x, wg, w13, w2), dict(ids=fake((3, 2), torch.int64))),
                  ((x, wg, w13, w2), dict(w13_s=fake((64, 64), b16), w2_s=fake((64, 64), b16)))):
        with pytest.raises(ValueError):
            moe.moe_layer_few(*a, 1, 2, **kw)
    assert len(launched) == 2
