"""A bounded wait that runs out is reported, whether or not the call has a workspace of the caller's:
moe_read_timeouts reads it, without a fault and with the context usable afterwards."""
import os
import shutil
import time

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def moe():
    if not os.path.exists(os.path.join(ROOT, "mixture_experts_layer_03_gb300", "libmoe_gb300.so")):
        if not (shutil.which("nvcc") or os.path.exists("/usr/local/cuda/bin/nvcc")):
            pytest.skip("library not built and nvcc unavailable")
        import __graft_entry__
        __graft_entry__.build()
    import mixture_experts_layer_03_gb300 as m
    return m


def test_the_layer_says_where_its_timeouts_are_read(moe):
    from mixture_experts_layer_03_gb300.training import moe_layer
    assert "moe_read_timeouts" in moe.EXPORTED and "moe_read_timeouts" in moe_layer.__doc__


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")
def test_a_wait_of_the_products_that_runs_out_is_read_without_a_workspace(moe):
    from mixture_experts_layer_03_gb300.training import moe_layer
    g = torch.Generator().manual_seed(1)
    draw = lambda *s: (torch.randn(s, generator=g) * 0.1).bfloat16().cuda().requires_grad_(True)   # noqa: E731
    args = draw(40, 64), draw(8, 64), draw(8, 128, 64), draw(8, 64, 64)
    moe.moe_read_timeouts()
    y = moe_layer(*args, 4, 2)
    grads = torch.autograd.grad(y.sum(), args)
    assert moe.moe_read_timeouts() == (moe.MOE_OK, 0)
    t0 = time.perf_counter()
    moe.moe_selftest_experts_wait()
    torch.cuda.synchronize()
    assert 1.5 < time.perf_counter() - t0 < 2.8      # the limit of every wait is 2 s
    assert moe.moe_read_timeouts() == (moe.MOE_ERR_DEVICE_TIMEOUT, moe.MOE_DEVICE_FLAG_TIMEOUT)
    assert moe.moe_read_timeouts() == (moe.MOE_OK, 0)       # the read cleared it
    again = moe_layer(*args, 4, 2)
    assert torch.equal(again, y)
    assert all(torch.equal(a, b) for a, b in zip(torch.autograd.grad(again.sum(), args), grads))
    assert moe.moe_read_timeouts() == (moe.MOE_OK, 0)


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")
def test_status_words_of_calls_without_rows(moe):
    """A dispatch writes its workspace's status word, and dw clears its own, with no rows too: what an
    older call or the memory's last user left is not read as theirs."""
    ids = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    scratch = moe.alloc_dispatch_scratch(0, 4, 2)
    scratch.buf.fill_(0x5A)
    moe.moe_dispatch(x, ids, 4, scratch=scratch)
    assert moe.moe_read_device_status(scratch) == (moe.MOE_OK, 0)
    offsets = torch.zeros(5, dtype=torch.int32, device="cuda")
    for start in (None, torch.ones((4, 32, 64), device="cuda")):
        scratch = moe.alloc_experts_scratch(4)
        scratch.buf.fill_(0x5A)
        moe.moe_experts_matmul_dw(torch.empty((0, 32), dtype=torch.bfloat16, device="cuda"), x, offsets,
                                  dw=start, accumulate=start is not None, scratch=scratch)
        assert moe.moe_read_device_status(scratch) == (moe.MOE_OK, 0)
    assert (start == 1).all()
