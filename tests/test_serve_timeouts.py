"""A wait of the serving operators that runs out is read by moe_read_timeouts, each operator's word once, and
their results afterwards are what they were."""
import time

import pytest
import torch

from tests.test_timeouts import moe  # noqa: F401


def test_both_have_a_self_test(moe):  # noqa: F811
    assert {"moe_selftest_fp4_wait", "moe_selftest_few_wait"} <= set(moe.EXPORTED)


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")
@pytest.mark.parametrize("which", [("fp4",), ("few",), ("fp4", "few")])
def test_a_wait_that_runs_out_is_read_once(moe, which):  # noqa: F811
    gen = torch.Generator().manual_seed(2)
    draw = lambda *s: (torch.randn(s, generator=gen) * 0.1).bfloat16().cuda()   # noqa: E731
    x, wg, w13, w2 = draw(5, 64), draw(4, 64), draw(4, 128, 64), draw(4, 64, 64)
    off = torch.tensor([0, 1, 2, 4, 5], dtype=torch.int32, device="cuda")
    q, qw = moe.moe_quantize_fp4(x, moe.MOE_FP4_NV), moe.moe_quantize_fp4(w13, moe.MOE_FP4_NV)

    def run():
        return (moe.moe_experts_matmul_fp4(q, qw, off), *moe.moe_layer_few(x, wg, w13, w2, 1, 2))

    moe.moe_read_timeouts()
    before = run()
    assert moe.moe_read_timeouts() == (moe.MOE_OK, 0)
    streams = [torch.cuda.Stream() for _ in which]
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for name, s in zip(which, streams):
        getattr(moe, f"moe_selftest_{name}_wait")(stream=s)
    torch.cuda.synchronize()
    assert 1.5 < time.perf_counter() - t0 < 2.8      # the limit of every wait is 2 s; the abort flag ends a later one
    assert moe.moe_read_timeouts() == (moe.MOE_ERR_DEVICE_TIMEOUT, moe.MOE_DEVICE_FLAG_TIMEOUT)
    assert moe.moe_read_timeouts() == (moe.MOE_OK, 0)
    assert all(torch.equal(a, b) for a, b in zip(run(), before))
    assert moe.moe_read_timeouts() == (moe.MOE_OK, 0)
