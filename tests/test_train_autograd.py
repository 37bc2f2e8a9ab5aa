"""CPU: what autograd may ask of training.moe_layer, with the operators stood in for (their values do
not matter here)."""
import os
import shutil

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def layer(monkeypatch):
    if not os.path.exists(os.path.join(ROOT, "mixture_experts_layer_03_gb300", "libmoe_gb300.so")):
        if not (shutil.which("nvcc") or os.path.exists("/usr/local/cuda/bin/nvcc")):
            pytest.skip("library not built and nvcc unavailable")
        import __graft_entry__
        __graft_entry__.build()
    from mixture_experts_layer_03_gb300 import training

    def stand_in(name, f):
        monkeypatch.setattr(training, name, f)

    def gate(x, wg, method, k, E, *a, **kw):
        return (torch.zeros((len(x), k), dtype=torch.int32), torch.ones((len(x), k)),
                torch.ones((len(x), E)), None)

    stand_in("moe_gate_route", gate)
    stand_in("moe_dispatch", lambda x, ids, E: (x.repeat_interleave(ids.shape[1], 0), ids, torch.zeros(E + 1, dtype=torch.int32)))
    stand_in("moe_dispatch_rows", lambda x, inv: x.repeat_interleave(inv.shape[1], 0))
    stand_in("moe_experts_matmul", lambda x, w, off: x @ w[0].t())
    stand_in("moe_experts_matmul_dx", lambda dy, w, off: dy @ w[0])
    stand_in("moe_experts_matmul_dw", lambda dy, x, off: (dy.t() @ x)[None].expand(len(off) - 1, -1, -1).clone())

    def ckpt(gu):
        c = type("Kept", (), {})()
        c.buf = torch.zeros(training.Checkpoint.nbytes(len(gu), gu.shape[1] // 2), dtype=torch.uint8)
        return gu[:, :gu.shape[1] // 2] * 2, c

    stand_in("moe_swiglu_ckpt", ckpt)
    stand_in("moe_swiglu_ckpt_backward", lambda dh, c, want_h: (torch.cat([dh, dh], 1), dh))
    stand_in("moe_combine", lambda rows, inv, s: rows.view(*inv.shape, -1).sum(1))
    stand_in("moe_combine_backward", lambda dy, rows, inv, s: (dy.repeat_interleave(inv.shape[1], 0), torch.ones(inv.shape)))
    stand_in("moe_dispatch_backward", lambda d, inv: d.view(*inv.shape, -1).sum(1))
    stand_in("moe_route_backward", lambda logits, ids, ds, method, rsf: torch.ones_like(logits))
    return training.moe_layer


def arguments():
    g = torch.Generator().manual_seed(0)
    return [torch.randn(s, generator=g).requires_grad_(True) for s in ((4, 8), (8, 8), (8, 12, 8), (8, 8, 6))]


def test_gradients_reach_every_input(layer):
    args = arguments()
    layer(*args, 4, 2).sum().backward()
    assert all(t.grad is not None and t.grad.shape == t.shape for t in args)


def test_a_second_derivative_is_refused(layer):
    """The gradient's kernels have none: a term of it in a loss is an error, not a constant."""
    args = arguments()
    loss = layer(*args, 4, 2).sum()
    dx, = torch.autograd.grad(loss, args[0], create_graph=True)
    with pytest.raises(RuntimeError):
        (loss + dx.square().sum()).backward()


def test_a_graph_of_the_gradients_alone_is_not(layer):
    """create_graph, which another layer's penalty needs, changes nothing where these gradients stay out
    of the loss."""
    args = arguments()
    v = torch.randn(8, generator=torch.Generator().manual_seed(1)).requires_grad_(True)
    plain = torch.autograd.grad(layer(*args, 4, 2).sum(), args)
    loss = layer(*args, 4, 2).sum() + v.pow(3).sum()
    *first, dv = torch.autograd.grad(loss, [*args, v], create_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(plain, first))
    dv.sum().backward()
    assert torch.allclose(v.grad, 6 * v)
    some = arguments()
    some[1].requires_grad_(False)
    dx, dw2 = torch.autograd.grad(layer(*some, 4, 2).sum(), [some[0], some[3]], create_graph=True)
    assert torch.equal(dx, plain[0]) and torch.equal(dw2, plain[3])
    with pytest.raises(RuntimeError):
        dw2.sum().backward()
