"""The MoE layer with a gradient: gate, routing, SwiGLU experts and combine as one autograd
function over the training operators.

Forward and backward of ``y = sum_j s_j W2[e_j] swiglu(W13[e_j] x)`` with s, e from the router:

    logits, ids, s = moe_gate_route(x, wg)             dlogits = moe_route_backward(...)
    x_perm, inv, offsets = moe_dispatch(x, ids)        dx += moe_dispatch_backward(dx_perm)
    gu = moe_experts_matmul(x_perm, w13)               dx_perm, dw13 = ..._dx(dgu), ..._dw(dgu, x_perm)
    h, ckpt = moe_swiglu_ckpt(gu)                      dgu, h = moe_swiglu_ckpt_backward(dh, ckpt)
    rows = moe_experts_matmul(h, w2)                   dh, dw2 = ..._dx(drows), ..._dw(drows, h)
    y = moe_combine(rows, inv, s)                      drows, ds = moe_combine_backward(dy, rows)

Between the passes it keeps x, the logits, the map, rows and the 8-bit checkpoint of gu; x_perm
is gathered again and h comes out of the checkpoint's backward pass, so that neither (k times
x's size, and 6 I bytes a row of gu and h) is held.
"""
from __future__ import annotations

import torch

from . import (Checkpoint, moe_combine, moe_combine_backward, moe_dispatch, moe_dispatch_backward,
               moe_dispatch_rows, moe_experts_matmul, moe_experts_matmul_dw,
               moe_experts_matmul_dx, moe_gate_route, moe_route_backward, moe_swiglu_ckpt,
               moe_swiglu_ckpt_backward)


class _MoeLayer(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, wg, w13, w2, method, top_k, bias, n_group, topk_group, rsf):
        E = w13.shape[0]
        ids, scales, logits, _ = moe_gate_route(x, wg, method, top_k, E, bias, n_group, topk_group,
                                                rsf, want_logits=True)
        x_perm, inv, offsets = moe_dispatch(x, ids, E)
        gu = moe_experts_matmul(x_perm, w13, offsets)
        h, ckpt = moe_swiglu_ckpt(gu)
        rows = moe_experts_matmul(h, w2, offsets)
        y = moe_combine(rows, inv, scales)
        ctx.save_for_backward(x, wg, w13, w2, ids, scales, logits, inv, offsets, ckpt.buf, rows)
        ctx.method, ctx.rsf = method, rsf
        return y

    @staticmethod
    def backward(ctx, dy):
        with torch.no_grad():
            grads = _MoeLayer.gradients(ctx, dy)
        if torch.is_grad_enabled():   # create_graph
            grads = _refuse_second(grads, [dy, *ctx.saved_tensors[:4]])
        return (*grads, None, None, None, None, None, None)

    @staticmethod
    def gradients(ctx, dy):
        x, wg, w13, w2, ids, scales, logits, inv, offsets, ckpt, rows = ctx.saved_tensors
        need_x, need_wg, need_w13, need_w2 = ctx.needs_input_grad[:4]
        drows, dscales = moe_combine_backward(dy.contiguous(), rows, inv, scales)
        dh = moe_experts_matmul_dx(drows, w2, offsets)
        dgu, h = moe_swiglu_ckpt_backward(dh, Checkpoint(ckpt, *dh.shape), want_h=need_w2)
        dw2 = moe_experts_matmul_dw(drows, h, offsets) if need_w2 else None
        dw13 = moe_experts_matmul_dw(dgu, moe_dispatch_rows(x, inv), offsets) if need_w13 else None
        dx = dwg = None
        if need_x:
            dx = moe_dispatch_backward(moe_experts_matmul_dx(dgu, w13, offsets), inv)
        if need_x or need_wg:
            # The gate is the product of one expert that has every token; its gradient's rows are rounded
            # to the products' type, as all of theirs are.
            dlogits = moe_route_backward(logits, ids, dscales, ctx.method, ctx.rsf).to(x.dtype)
            all_rows = torch.arange(2, dtype=torch.int32, device=x.device) * x.shape[0]
            if need_x:
                dx += moe_experts_matmul_dx(dlogits, wg[None], all_rows)
            if need_wg:
                dwg = moe_experts_matmul_dw(dlogits, x, all_rows)[0]
        return dx, dwg, dw13, dw2


class _NoSecond(torch.autograd.Function):
    """First derivatives, as they are, in a graph whose backward pass is an error."""

    @staticmethod
    def forward(ctx, n, *tensors):
        return tuple(t.view_as(t) for t in tensors[:n])

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("moe_layer has no second derivative")


def _refuse_second(grads, inputs):
    """The gradient's kernels have no gradient: a loss that takes in the gradients `grads` (functions of
    `inputs`) must fail, and not count them as constants."""
    there = [g for g in grads if g is not None]
    out = iter(_NoSecond.apply(len(there), *there, *inputs))
    return [None if g is None else next(out) for g in grads]


def moe_layer(x, wg, w13, w2, method: int, top_k: int, bias=None, n_group: int = 1,
              topk_group: int = 1, routed_scaling_factor: float = 1.0):
    """y [T, H] of the MoE layer, differentiable in x [T, H], the gate wg [E, H], w13 [E, 2I, H]
    (gate rows, then up rows) and w2 [E, H, I], all bf16. Routing as moe_gate_route (the
    selection bias has no gradient); E a multiple of 8, H of 64, I of 8.

    What the backward pass rounds beside its products' results: gu is kept in 8 bits (always: gradients of
    x, w13 and w2 are within 6% in norm on normal data, y is not affected; the operators by themselves can
    keep it as it is), the gradient of the logits goes to x's type before the gate's two products,
    and dx is the sum of the experts' and the gate's, each in that type. A second derivative is an
    error.

    The kernels' waits are bounded. One that runs out leaves results incomplete and raises nothing, as
    that would take a synchronisation: read moe_read_timeouts() where the loop synchronises anyway."""
    if w13.shape[0] % 8 or wg.shape[0] != w13.shape[0]:
        raise ValueError(f"the gate's gradient takes a multiple of 8 experts, one row of wg each: "
                         f"got {w13.shape[0]} experts, wg {tuple(wg.shape)}")
    return _MoeLayer.apply(x, wg, w13, w2, method, top_k, bias, n_group, topk_group,
                           routed_scaling_factor)


__all__ = ["moe_layer"]
