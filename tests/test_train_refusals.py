"""What dw refuses by its types, on the host, on any machine: nothing here is launched."""
import ctypes
import os
import shutil

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
GOOD = ctypes.c_void_p(1 << 20)         # never dereferenced
UNSUPPORTED = 2


@pytest.fixture(scope="module")
def moe():
    if not os.path.exists(os.path.join(ROOT, "mixture_experts_layer_03_gb300", "libmoe_gb300.so")):
        if not (shutil.which("nvcc") or os.path.exists("/usr/local/cuda/bin/nvcc")):
            pytest.skip("library not built and nvcc unavailable")
        import __graft_entry__
        __graft_entry__.build()
    import mixture_experts_layer_03_gb300 as m
    return m


@pytest.mark.parametrize("dtype,dw_dtype,accumulate", [
    (0, 1, 0), (1, 0, 0), (0, 3, 0), (2, 2, 0),     # neither the rows' type nor f32, or f32 rows
    (0, 0, 1), (1, 1, 1)])                          # only an f32 dw is added to
def test_dw_refuses_types(moe, dtype, dw_dtype, accumulate):
    assert moe._lib.moe_experts_matmul_dw(GOOD, GOOD, GOOD, 4, 2, 64, 64, dtype, dw_dtype, accumulate,
                                          GOOD, GOOD, 1 << 20, None) == UNSUPPORTED
    assert moe._lib.moe_last_error()
