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
