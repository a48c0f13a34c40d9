"""Trains a stack of 8-bit residual linear layers with the Dion step.

Layer l of the stack is  r <- r + W_l norm_l(r): the residual's addition, the
norm and the quantization of its rows are one call, the three products of a
layer (forward, dX, dW) read 8-bit operands, and each weight gradient is
written straight into the megabatch that dion_step_batched steps.  After the
step the new weights are quantized once, in both orders.

    python examples/q8_training.py [--layers 4 --width 1024 --tokens 2048 --steps 30]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import orthonormal_optimizer_step_gb300 as od  # noqa: E402
import workloads as wl  # noqa: E402


class Stack:
    """`layers` square residual layers with bf16 weights and Dion state."""

    def __init__(self, layers, width, device="cuda", seed=0):
        self.group = wl.Group(layers, width, width)
        self.X, self.M, self.Q = wl.make_state(self.group, self.group.rank(0.25), torch.bfloat16, device, seed)
        self.G = torch.empty_like(self.X)
        self.norm = torch.ones(layers, width, device=device)
        self.norm_grad = torch.empty_like(self.norm)
        self.quantize()

    def quantize(self):
        self.w8, self.w8t = od.dion_q8_quantize(self.X, form="both", square=True,
                                                out=getattr(self, "w8", None) and (self.w8, self.w8t))

    def layer(self, q, l):
        return od.Q8(q.data[l], q.scale[l])

    def forward(self, x):
        """Output of the stack and what the backward pass reads: h and rstd of each layer."""
        saved, delta, r = [], x, None
        for l in range(self.group.batch):
            x8, r, rstd = od.dion_rms_norm_q8(delta, self.norm[l], residual=r)
            delta = od.dion_q8_matmul(x8, self.layer(self.w8, l))
            saved.append((r, rstd))
        return r + delta, saved

    def backward(self, dout, saved):
        """Fills G (the weights' gradients) and norm_grad; returns the gradient of x."""
        d = dout
        for l in reversed(range(self.group.batch)):
            h, rstd = saved[l]
            dy8, dy8t = od.dion_q8_quantize(d, form="both")
            _, x8t = od.dion_q8_quantize(h, form="cols", rstd=rstd, weight=self.norm[l])
            od.dion_q8_matmul(dy8t, x8t, out=self.G[l])
            dx = od.dion_q8_matmul(dy8, self.layer(self.w8t, l))
            d, _ = od.dion_rms_norm_backward(dx, h, rstd, self.norm[l], dh=d, dweight=self.norm_grad[l])
        return d

    def step(self, lr):
        od.dion_step_batched(self.X, self.G, self.M, self.Q, mu=0.95, lr=lr, weight_decay=0.0)
        self.norm -= lr * self.norm_grad
        self.quantize()


def train(layers, width, tokens, steps, lr=0.02, seed=0, device="cuda", report=None):
    """Mean squared error before each step, learning a random linear map."""
    net = Stack(layers, width, device, seed)
    teacher = wl.randn((width, width), width ** -0.5, torch.float32, device, seed + 50)
    losses = []
    for t in range(steps):
        x = wl.randn((tokens, width), 1.0, torch.bfloat16, device, seed * 1000 + t)
        target = x.float() @ teacher.t() + x.float()
        out, saved = net.forward(x)
        err = out.float() - target
        net.backward((err / tokens).to(torch.bfloat16), saved)
        net.step(lr)
        losses.append(err.square().mean())
        if report and t % report == 0:
            print(f"step {t:4d}  loss {float(losses[-1]):.4f}")
    return [float(v) for v in losses]


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--lr", type=float, default=0.02)
    a = ap.parse_args()
    losses = train(a.layers, a.width, a.tokens, a.steps, a.lr, report=5)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {a.steps} steps; kernel status {od.dion_q8_status()}")


if __name__ == "__main__":
    main()
