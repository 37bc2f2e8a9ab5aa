"""CPU: what the serving operators' Python wrappers hand on and give back. Nothing is launched."""
import pytest
import torch

from tests.test_serve_abi import fake, moe  # noqa: F401


@pytest.mark.parametrize("name,width", [("moe_quantize_fp4", 96), ("moe_swiglu_fp4", 192)])
def test_memory_that_is_written_again_gets_the_new_factor(moe, monkeypatch, name, width):  # noqa: F811
    status = []
    monkeypatch.setattr(moe._lib, name, lambda *a: status[-1])
    monkeypatch.setattr(moe, "_stream", lambda s: 0)
    monkeypatch.setattr(moe, "_new", lambda shape, dtype, device, stream, result=True: fake(shape, dtype))
    call, x = getattr(moe, name), fake((4, width), torch.bfloat16)
    one, two = fake((1,), torch.float32), fake((1,), torch.float32)
    status.append(moe.MOE_OK)
    q = call(x, moe.MOE_FP4_NV, one)
    codes = q.codes
    assert q.g is one
    assert call(x, moe.MOE_FP4_NV, two, out=q) is q and q.g is two and q.codes is codes
    assert call(x, moe.MOE_FP4_NV, out=q) is q and q.g is None
    call(x, moe.MOE_FP4_NV, two, out=q)
    status.append(1)                       # refused by the library: what it stands for is as before
    with pytest.raises(moe.MoeError):
        call(x, moe.MOE_FP4_NV, one, out=q)
    assert q.g is two
    mx = moe.Fp4(fake((4, 48), torch.uint8), fake((4, 16), torch.uint8), moe.MOE_FP4_MX)
    for bad in (dict(g=one, out=mx), dict(g=fake((2,), torch.float32), out=q), dict(g=one, out=moe.Fp4(
            fake((5, 48), torch.uint8), fake((5, 16), torch.uint8), moe.MOE_FP4_NV))):
        with pytest.raises(ValueError):
            call(x, moe.MOE_FP4_NV, **bad)
    assert q.g is two and mx.g is None
