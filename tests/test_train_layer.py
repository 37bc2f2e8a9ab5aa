"""GPU: the differentiable MoE layer (training.moe_layer) against a float64 layer built from
elementary operations, and the training example."""
import os
import sys

import pytest
import torch

from oracle import train_oracle as ref

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def reference(x, wg, w13, w2, ids, method, rsf, dy):
    """Gradients of the layer in float64 with the experts given: torch's autograd over products,
    exp and indexing."""
    x, wg, w13, w2 = (t.detach().double().cpu().requires_grad_(True) for t in (x, wg, w13, w2))
    ids = ids.cpu().long()
    logits = x @ wg.t()
    chosen = logits.gather(1, ids)
    if method == 0:
        s = (logits - logits.logsumexp(1, keepdim=True)).exp().gather(1, ids)
    elif method in (1, 4):
        s = torch.softmax(chosen, 1)
    elif method == 3:
        s = torch.sigmoid(chosen)
    else:
        s = torch.sigmoid(chosen)
        s = s / (s.sum(1, keepdim=True) + (1e-20 if method == 2 else 0)) * (rsf if method in (2, 16) else 1)
    I = w2.shape[2]
    y = torch.zeros_like(x)
    for e in range(w13.shape[0]):
        t, j = (ids == e).nonzero(as_tuple=True)
        gu = x[t] @ w13[e].t()
        h = gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]
        y = y.index_add(0, t, (h @ w2[e].t()) * s[t, j, None])
    y.backward(dy.double().cpu())
    return y.detach(), x.grad, wg.grad, w13.grad, w2.grad


@pytest.mark.parametrize("T,H,I,E,k,method,kw", [
    (96, 128, 64, 8, 2, 4, {}), (200, 192, 104, 16, 4, 0, {}), (65, 256, 128, 8, 1, 3, {}),
    (300, 128, 96, 32, 8, 2, dict(n_group=4, topk_group=2, routed_scaling_factor=2.5)),
    (1, 64, 64, 8, 2, 6, {})])
def test_layer_gradients(T, H, I, E, k, method, kw):
    import mixture_experts_layer_03_gb300 as moe
    from mixture_experts_layer_03_gb300.training import moe_layer
    g = torch.Generator().manual_seed(T + H)
    draw = lambda *s, std=1.0: (torch.randn(s, generator=g) * std).bfloat16().cuda()   # noqa: E731
    args = [draw(T, H), draw(E, H, std=H ** -0.5), draw(E, 2 * I, H, std=H ** -0.5),
            draw(E, H, I, std=I ** -0.5)]
    for t in args:
        t.requires_grad_(True)
    dy = draw(T, H)
    y = moe_layer(*args, method, k, **kw)
    y.backward(dy)
    with torch.no_grad():
        ids = moe.moe_gate_route(args[0], args[1], method, k, E,
                                 n_group=kw.get("n_group", 1), topk_group=kw.get("topk_group", 1),
                                 routed_scaling_factor=kw.get("routed_scaling_factor", 1.0))[0]
    want = reference(*args, ids, method, kw.get("routed_scaling_factor", 1.0), dy)
    # e4m3 keeps 3 fraction bits: a kept value is off by up to 2^-4 of itself, 2^-4 / sqrt(3) in the
    # mean square at worst, two of them enter a product: under 6% of a gradient in norm; the
    # output and the gradient of the gate, which no kept value reaches, only see bf16 (a few
    # roundings of 2^-8, the gate's through sums of k cancelling terms).
    for name, got, exp, tol in zip(("y", "dx", "dwg", "dw13", "dw2"),
                                   (y, *(t.grad for t in args)), want, (0.01, 0.06, 0.03, 0.06, 0.06)):
        got = got.detach().double().cpu()
        off = float((got - exp).norm() / exp.norm())
        assert off <= tol, f"{name}: {off:.4f} of its norm off"


def test_layer_without_some_gradients():
    from mixture_experts_layer_03_gb300.training import moe_layer
    g = torch.Generator().manual_seed(1)
    draw = lambda *s: (torch.randn(s, generator=g) * 0.1).bfloat16().cuda()   # noqa: E731
    x, wg, w13, w2 = draw(40, 64), draw(8, 64), draw(8, 128, 64), draw(8, 64, 64)
    full = [t.clone().requires_grad_(True) for t in (x, wg, w13, w2)]
    moe_layer(*full, 4, 2).sum().backward()
    for i in range(4):
        some = [t.clone() for t in (x, wg, w13, w2)]
        some[i].requires_grad_(True)
        moe_layer(*some, 4, 2).sum().backward()
        assert torch.equal(some[i].grad, full[i].grad)
    with pytest.raises(ValueError):
        moe_layer(x, wg[:6].contiguous(), w13[:6].contiguous(), w2[:6].contiguous(), 4, 2)


def test_example_learns():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import train_moe_layer
    finally:
        sys.path.pop(0)
    losses = train_moe_layer.main(["--tokens", "512", "--hidden", "256", "--inter", "128",
                                   "--experts", "16", "--top-k", "4", "--steps", "40"])
    assert losses[-1] < 0.5 * losses[0]
