"""A routed field learns a teacher's classes: several small networks share a
scene, a gate sends every sample point to two of them, and the field is trained
on the teacher's largest logits per point alone.

    python examples/distill_routed_field.py [--steps 200] [--points 65536]

The forward and backward pass run in this library's kernels: frequency
encoding, routing plan, the experts' products, the weighted sum, a dense head
(a layer with one expert) and the distillation loss with its gradient.  The
gate (a [features, experts] product) and Adam are plain torch.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import volume_rendering_amd as v  # noqa: E402

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
FREQS = 8
FEATURES = 6 * FREQS  # sines and cosines of three coordinates


class RoutedField:
    """encoding -> [gate] -> experts (FEATURES -> hidden -> width) -> sum -> classes."""

    def __init__(self, points, experts=16, choices=2, hidden=128, width=64, classes=1000, seed=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)

        def param(*shape, fan_in=None):
            scale = math.sqrt(2.0 / fan_in) if fan_in else 0.0
            return (torch.randn(shape, generator=gen, device="cuda") * scale).requires_grad_(True)

        self.n, self.k, self.experts, self.classes = points, choices, experts, classes
        self.gate = param(FEATURES, experts, fan_in=4 * FEATURES)
        self.w1, self.b1 = param(experts, hidden, FEATURES, fan_in=FEATURES), param(experts, hidden)
        self.w2, self.b2 = param(experts, width, hidden, fan_in=hidden), param(experts, width)
        self.head, self.head_b = param(1, classes, width, fan_in=width), param(1, classes)
        self.params = [self.gate, self.w1, self.b1, self.w2, self.b2, self.head, self.head_b]
        slots = points * choices

        def buf(*shape, dtype=BF16):
            return torch.empty(shape, dtype=dtype, device="cuda")

        self.enc = buf(points, FEATURES)
        self.offsets, self.order, self.place = buf(experts + 1, dtype=I32), buf(slots, dtype=I32), buf(points, choices,
                                                                                                       dtype=I32)
        self.h, self.y, self.feat, self.logits = (buf(slots, hidden), buf(slots, width), buf(points, width),
                                                  buf(points, classes))
        self.all_points = torch.tensor([0, points], dtype=I32, device="cuda")
        self.dlogits, self.dfeat, self.dy, self.dh = (torch.empty_like(t) for t in
                                                      (self.logits, self.feat, self.y, self.h))
        self.dweights = buf(points, choices, dtype=F32)
        self.loss, self.lse = buf(points, dtype=F32), buf(points, dtype=F32)
        sizes = [v.nerf_route_workspace_size(points, choices, experts),
                 v.nerf_expert_linear_grad_workspace_size(slots, experts, FEATURES, hidden),
                 v.nerf_expert_linear_grad_workspace_size(slots, experts, hidden, width),
                 v.nerf_expert_linear_grad_workspace_size(points, 1, width, classes),
                 v.nerf_distill_workspace_size(points, classes)]
        self.ws = buf(max(sizes) + 1, dtype=torch.uint8)

    def forward(self, x):
        """Class logits of points x [n, 3] (bfloat16)."""
        v.nerf_encode_freq(x, FREQS, False, True, v.NERF_BF16, self.enc)
        top, ids = (self.enc.float() @ self.gate.detach()).topk(self.k, dim=1)
        self.ids, self.weights = ids.to(I32), torch.softmax(top, 1)
        self.w1_, self.w2_, self.head_ = (w.detach().to(BF16) for w in (self.w1, self.w2, self.head))
        v.nerf_route_plan(self.ids, self.experts, self.offsets, self.order, self.place, workspace=self.ws)
        v.nerf_expert_linear(self.enc, self.w1_, self.b1.detach(), self.offsets, self.h, order=self.order, k=self.k,
                             relu=True)
        v.nerf_expert_linear(self.h, self.w2_, self.b2.detach(), self.offsets, self.y)
        v.nerf_route_combine(self.y, self.offsets, self.place, self.weights, self.feat)
        v.nerf_expert_linear(self.feat, self.head_, self.head_b.detach(), self.all_points, self.logits)
        return self.logits

    def backward(self, t_logits, t_ids, temperature):
        """Mean loss of the last forward pass against the teacher's largest
        logits; sets every parameter's gradient."""
        for p in self.params:
            if p.grad is None:
                p.grad = torch.empty_like(p)
        scale = torch.full((self.n,), 1.0 / self.n, device="cuda")
        v.nerf_distill_topk(self.logits, t_logits, t_ids, temperature, self.loss, lse=self.lse, grad=self.dlogits,
                            row_scale=scale, workspace=self.ws)
        v.nerf_expert_linear_grad(self.dlogits, self.feat, self.head_, self.all_points, self.dfeat, self.head.grad,
                                  self.head_b.grad, workspace=self.ws)
        v.nerf_route_combine_grad(self.dfeat, self.y, self.offsets, self.place, self.weights, self.dy, self.dweights)
        v.nerf_expert_linear_grad(self.dy, self.h, self.w2_, self.offsets, self.dh, self.w2.grad, self.b2.grad,
                                  relu_x=True, workspace=self.ws)
        v.nerf_expert_linear_grad(self.dh, self.enc, self.w1_, self.offsets, None, self.w1.grad, self.b1.grad,
                                  order=self.order, k=self.k, workspace=self.ws)
        dtop = self.weights * (self.dweights - (self.weights * self.dweights).sum(1, keepdim=True))
        dgate = torch.zeros((self.n, self.experts), device="cuda").scatter_(1, self.ids.long(), dtop)
        self.gate.grad.copy_(self.enc.float().t() @ dgate)
        return self.loss.mean()


def teacher_logits(x, classes, top, seed=1):
    """The `top` largest logits (and their classes) of a fixed smooth function of the points."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    a = torch.randn((3, 64), generator=gen, device="cuda") * 2.0
    b = torch.randn((64, classes), generator=gen, device="cuda") * 0.7
    t, ids = (torch.sin(x @ a) @ b).topk(top, dim=1)
    return t.contiguous(), ids.to(I32)


def train(steps=200, points=65536, classes=1000, top=16, temperature=1.0, lr=2e-3, every=20, say=print):
    field = RoutedField(points, classes=classes)
    opt = torch.optim.Adam(field.params, lr=lr)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(7)
    losses = []
    for step in range(steps):
        x = torch.rand((points, 3), generator=gen, device="cuda") * 2.0 - 1.0
        field.forward(x)
        loss = field.backward(*teacher_logits(x, classes, top), temperature)
        opt.step()
        if step % every == 0 or step == steps - 1:
            losses.append(loss.item())
            say(f"step {step:4d}  loss {losses[-1]:.4f}")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--points", type=int, default=65536)
    args = ap.parse_args()
    train(args.steps, args.points)
