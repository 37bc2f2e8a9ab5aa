"""CPU: what the training operators refuse before anything is launched, their workspace sizes,
and the float64 restatement that the GPU tests compare with."""
import ctypes
import os
import shutil

import numpy as np
import pytest
import torch

from oracle import train_oracle as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
GOOD = ctypes.c_void_p(1 << 20)         # never dereferenced: every call here is refused first
ODD = ctypes.c_void_p((1 << 20) + 8)


@pytest.fixture(scope="module")
def moe():
    if not os.path.exists(os.path.join(ROOT, "mixture_experts_layer_03_gb300", "libmoe_gb300.so")):
        if not (shutil.which("nvcc") or os.path.exists("/usr/local/cuda/bin/nvcc")):
            pytest.skip("library not built and nvcc unavailable")
        import __graft_entry__
        __graft_entry__.build()
    import mixture_experts_layer_03_gb300 as m
    return m


INVALID, UNSUPPORTED, SMALL = 1, 2, 3


def dispatch(moe, x=GOOD, ids=GOOD, T=4, H=64, E=8, k=2, dt=0, xp=GOOD, inv=GOOD, off=GOOD, ws=GOOD,
             n=1 << 20):
    return moe._lib.moe_dispatch(x, ids, T, H, E, k, dt, xp, inv, off, ws, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), UNSUPPORTED), (dict(T=(1 << 24) + 1), UNSUPPORTED), (dict(H=0), UNSUPPORTED),
    (dict(H=65537), UNSUPPORTED), (dict(E=0), UNSUPPORTED), (dict(E=257), UNSUPPORTED),
    (dict(k=0), UNSUPPORTED), (dict(k=9), UNSUPPORTED), (dict(dt=3), UNSUPPORTED),
    (dict(x=None), INVALID), (dict(ids=ODD), INVALID), (dict(xp=ODD), INVALID),
    (dict(inv=None), INVALID), (dict(off=None), INVALID), (dict(ws=ODD), INVALID),
    (dict(T=6145, ws=None), INVALID), (dict(n=16), SMALL), (dict(T=7000, n=1000), SMALL)])
def test_dispatch_refuses(moe, kw, status):
    assert dispatch(moe, **kw) == status
    assert moe._lib.moe_last_error()


def test_row_operators_refuse(moe):
    L = moe._lib
    for bad in (dict(a=None), dict(a=ODD), dict(T=-1), dict(H=0), dict(k=9), dict(dt=7)):
        kw = dict(a=GOOD, T=4, H=64, k=2, dt=0) | bad
        want = INVALID if "a" in bad else UNSUPPORTED
        sizes = (kw["T"], kw["H"], kw["k"], kw["dt"])
        assert L.moe_dispatch_rows(kw["a"], GOOD, *sizes, GOOD, None) == want
        assert L.moe_dispatch_backward(kw["a"], GOOD, *sizes, GOOD, None) == want
        assert L.moe_combine(GOOD, kw["a"], None, *sizes, GOOD, None) == want
        assert L.moe_combine_backward(GOOD, GOOD, GOOD, None, *sizes, kw["a"], GOOD, None) == want
    assert L.moe_combine(GOOD, GOOD, ODD, 4, 64, 2, 0, GOOD, None) == INVALID
    # nothing to do: nothing is looked at
    assert L.moe_combine(None, None, None, 0, 64, 2, 0, None, None) == 0
    assert L.moe_combine_backward(None, None, None, None, 0, 64, 2, 0, None, None, None) == 0


def test_swiglu_checkpoint_refuses(moe):
    L = moe._lib
    for R, I, dt, a, want in ((-1, 64, 0, GOOD, UNSUPPORTED), (4, 0, 0, GOOD, UNSUPPORTED),
                              (4, 65537, 0, GOOD, UNSUPPORTED), (4, 64, 5, GOOD, UNSUPPORTED),
                              (4, 64, 0, None, INVALID), (4, 64, 2, ODD, INVALID)):
        assert L.moe_swiglu_ckpt(GOOD, R, I, dt, GOOD, a, GOOD, None) == want
        assert L.moe_swiglu_ckpt_backward(a, GOOD, GOOD, R, I, dt, GOOD, None, None) == want
    assert L.moe_swiglu_ckpt_backward(GOOD, GOOD, GOOD, 4, 64, 0, GOOD, ODD, None) == INVALID
    assert L.moe_swiglu_ckpt(None, 0, 64, 0, None, None, None, None) == 0


def test_experts_products_refuse(moe):
    L = moe._lib

    def all_three(R=4, E=2, N=64, K=64, dt=0, a=GOOD, w=GOOD, off=GOOD, ws=GOOD, n=1 << 20, out=GOOD,
                  odt=None, acc=0):
        odt = dt if odt is None else odt
        return (L.moe_experts_matmul(a, w, off, R, E, N, K, dt, out, ws, n, None),
                L.moe_experts_matmul_dx(a, w, off, R, E, N, K, dt, out, ws, n, None),
                L.moe_experts_matmul_dw(a, w, off, R, E, N, K, dt, odt, acc, out, ws, n, None))

    for kw in (dict(R=-1), dict(R=(1 << 23) + 1), dict(E=0), dict(E=257), dict(N=12), dict(K=4),
               dict(N=65544), dict(K=0), dict(dt=2)):
        assert all_three(**kw) == (UNSUPPORTED,) * 3, kw
    for kw in (dict(a=None), dict(w=ODD), dict(off=None), dict(out=ODD)):
        assert all_three(**kw) == (INVALID,) * 3, kw
    assert all_three(ws=ODD) == (INVALID,) * 3
    assert all_three(n=8) == (INVALID, INVALID, SMALL)
    assert all_three(ws=None, a=None) == (INVALID,) * 3
    assert all_three(odt=1)[2] == UNSUPPORTED           # bf16 rows, f16 dw
    assert all_three(acc=1)[2] == UNSUPPORTED           # only an f32 dw is added to
    assert L.moe_experts_matmul(None, None, None, 0, 2, 64, 64, 0, None, None, 0, None) == 0
    assert L.moe_experts_workspace_bytes(0) == 0 == L.moe_experts_workspace_bytes(257)
    assert L.moe_experts_workspace_bytes(256) == 128 + 2 * 256 * 128
    for bad in ((3, 100, 1, 64, 64), (0, -1, 1, 64, 64), (1, 100, 0, 64, 64), (2, 100, 1, 12, 64), (0, 0, 1, 64, 64)):
        assert L.moe_experts_split_bytes(*bad) == 0
    assert L.moe_dispatch_workspace_bytes(10, 0, 2) == 0 == L.moe_dispatch_workspace_bytes(10, 8, 9)
    assert 0 < L.moe_dispatch_workspace_bytes(1 << 24, 256, 8) < 2 << 20


def test_route_backward_refuses(moe):
    L = moe._lib

    def call(T=4, E=8, k=2, method=0, a=GOOD):
        p = moe.MoeRouteParams(E, k, method, 1, 1, 1.0)
        return L.moe_route_backward(a, GOOD, GOOD, T, ctypes.byref(p), GOOD, None)

    for kw in (dict(T=-1), dict(E=0), dict(E=257), dict(k=0), dict(k=9), dict(E=2, k=3),
               dict(method=17), dict(method=7), dict(method=-1)):
        assert call(**kw) == UNSUPPORTED, kw
    assert call(a=None) == INVALID and call(a=ODD) == INVALID
    assert L.moe_route_backward(GOOD, GOOD, GOOD, 4, None, GOOD, None) == INVALID
    assert call(T=0, a=None) == 0


def test_wrappers_want_cuda_tensors(moe):
    x, ids = torch.zeros(4, 64).bfloat16(), torch.zeros(4, 2, dtype=torch.int32)
    for f in (lambda: moe.moe_dispatch(x, ids, 4), lambda: moe.moe_combine(x, ids),
              lambda: moe.moe_swiglu_ckpt(x), lambda: moe.moe_experts_matmul(x, x[None], ids[0]),
              lambda: moe.moe_route_backward(x.float(), ids, x.float(), 0)):
        with pytest.raises(ValueError):
            f()


# ------------------------------------------------------------------------- the restatement

def test_e4m3_codes_are_torchs():
    rng = np.random.default_rng(0)
    v = np.clip(rng.standard_normal(5000) * np.exp(rng.uniform(-9, 6, 5000)), -448, 448).astype(np.float32)
    v[:4] = (448, -448, 0, 2.0 ** -10)
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.e4m3_code(v.astype(np.float64)), want)
    codes = np.arange(127, dtype=np.uint8)
    assert np.array_equal(torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy(), ref.E4M3)


def test_checkpoint_error_bound():
    rng = np.random.default_rng(1)
    gu = rng.standard_normal((20, 90)) * np.exp(rng.uniform(-5, 5, (20, 90)))
    q, qs = ref.quantise(gu)
    scale = np.concatenate([np.repeat(ref.scale_of(s), 32, 1)[:, :45] for s in np.split(qs, 2, 1)], 1)
    assert (np.abs(gu) <= 448 * scale).all() and (np.abs(gu).max() > 0)
    assert (np.abs(ref.kept(q, qs) - gu) <= np.maximum(np.abs(gu) / 16, scale * 2.0 ** -10)).all()


def test_sorting_restatement():
    ids = np.array([[2, 0], [-1, 2], [0, 5]], np.int32)
    inv, off = ref.sort_slots(ids, 3)
    assert inv.tolist() == [[2, 0], [-5, 3], [1, -6]] and off.tolist() == [0, 2, 2, 4]


@pytest.mark.parametrize("method", [0, 1, 2, 3, 4, 5, 6, 16])
def test_route_gradient_restatement_against_differences(method):
    rng = np.random.default_rng(method)
    logits = rng.standard_normal((3, 10))
    ids = np.argsort(-logits, axis=1)[:, :3]
    ids[2, 1] = -1
    ds = rng.standard_normal((3, 3))
    got, _ = ref.route_backward(logits, ids, ds, method, 2.5)
    for i in np.ndindex(logits.shape):
        up, dn = logits.copy(), logits.copy()
        up[i] += 1e-6
        dn[i] -= 1e-6
        num = ((ref.route_weights(up, ids, method, 2.5) - ref.route_weights(dn, ids, method, 2.5)) * ds).sum() / 2e-6
        assert abs(num - got[i]) < 1e-8


def test_swiglu_gradient_restatement_against_differences():
    rng = np.random.default_rng(2)
    gu, dh = rng.standard_normal((3, 12)), rng.standard_normal((3, 6))
    got = ref.swiglu_backward(dh, gu)
    for i in np.ndindex(gu.shape):
        up, dn = gu.copy(), gu.copy()
        up[i] += 1e-6
        dn[i] -= 1e-6
        assert abs(((ref.swiglu(up) - ref.swiglu(dn)) * dh).sum() / 2e-6 - got[i]) < 1e-8
