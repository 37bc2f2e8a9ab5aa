"""Trains one MoE layer to reproduce another's output on random tokens: the training operators
together, as a training loop uses them.

    python examples/train_moe_layer.py [--tokens 4096] [--steps 30]

Prints the loss every few steps, then the time of a training step (forward, backward and the
update) and the bytes that the layer keeps between its passes.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import mixture_experts_layer_03_gb300 as moe  # noqa: E402
from mixture_experts_layer_03_gb300.training import moe_layer  # noqa: E402


def weights(E, H, I, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    draw = lambda *shape, std: torch.randn(shape, generator=g, device="cuda").mul_(std).bfloat16()  # noqa: E731
    return [draw(E, H, std=H ** -0.5), draw(E, 2 * I, H, std=H ** -0.5), draw(E, H, I, std=I ** -0.5)]


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--inter", type=int, default=768)
    ap.add_argument("--experts", type=int, default=128)
    ap.add_argument("--top-k", type=int, default=8)
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--lr", type=float, default=2e-3)
    a = ap.parse_args(argv)
    T, H, I, E, k = a.tokens, a.hidden, a.inter, a.experts, a.top_k
    route = dict(method=moe.MOE_ROUTE_RENORMALIZE_NAIVE, top_k=k)

    # The teacher differs in its second weights only, so that the target is in reach.
    teacher = weights(E, H, I, 0)
    student = [w.clone() for w in teacher]
    student[2].copy_(weights(E, H, I, 1)[2])
    master = [w.float() for w in student]
    first, second = [torch.zeros_like(w) for w in master], [torch.zeros_like(w) for w in master]
    for w in student:
        w.requires_grad_(True)
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((T, H), generator=g, device="cuda").bfloat16()
    with torch.no_grad():
        target = moe_layer(x, *teacher, **route)

    losses = []
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    held = 0
    for step in range(a.steps):
        if step == min(3, a.steps - 1):
            start.record()
            timed = step
        before = torch.cuda.memory_allocated()
        y = moe_layer(x, *student, **route)
        held = torch.cuda.memory_allocated() - before
        loss = (y.float() - target.float()).square().mean()
        loss.backward()
        with torch.no_grad():   # Adam, with f32 weights and moments beside the layer's bf16 ones
            for w, m, m1, m2 in zip(student, master, first, second):
                grad = w.grad.float()
                m1.lerp_(grad, 0.1)
                m2.lerp_(grad.square(), 0.01)
                scale = a.lr / (1 - 0.9 ** (step + 1))
                m.sub_(scale * m1 / ((m2 / (1 - 0.99 ** (step + 1))).sqrt() + 1e-8))
                w.copy_(m)
                w.grad = None
        losses.append(loss.detach())
    end.record()
    torch.cuda.synchronize()
    if moe.moe_read_timeouts()[0] != moe.MOE_OK:
        raise RuntimeError("a kernel's wait ran out: the results are incomplete")
    losses = [float(v) for v in losses]
    for i in range(0, a.steps, max(1, a.steps // 6)):
        print(f"step {i:4d}  loss {losses[i]:.5f}")
    print(f"step {a.steps - 1:4d}  loss {losses[-1]:.5f}")
    ms = start.elapsed_time(end) / (a.steps - timed)
    print(f"{ms:.2f} ms a step of {T} tokens; {held / 2**20:.0f} MiB kept between the passes "
          f"(gu and h in bf16 would take {T * k * I * 6 / 2**20:.0f} of them, the checkpoint takes "
          f"{T * k * I * 2 * 33 / 32 / 2**20:.0f})")
    return losses


if __name__ == "__main__":
    main()
