"""A routed field with a memory along its rays: samples go through two of several
small networks, a gated recurrence carries what was seen from sample to sample,
and a head names a class after every one.  It is trained on whole rays against a
teacher's largest logits, and served sample by sample as they arrive.

    python examples/stream_routed_field.py [--steps 200] [--rays 512] [--samples 64]

Training runs the gate, the routing plan, the experts' products, the recurrence,
the distillation loss and all their gradients, and clips the gradients by their
norm; serving runs the gate, the whole routed layer and one step of the
recurrence.  Sigmoids, a few sums and Adam are plain torch.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import volume_rendering_amd as v  # noqa: E402

F32, I32 = torch.float32, torch.int32
FREQS = 6
FEATURES = 6 * FREQS  # sines and cosines of three coordinates


class StreamField:
    """encoding -> [gate] -> experts (FEATURES -> hidden -> width) -> sum -> recurrence -> classes.

    The recurrence is h = a h + (1 - a) f with f the sum's output and a =
    sigmoid(keep f + keep_b), a gate per channel.  Its state starts at `start`.
    """

    def __init__(self, experts=16, choices=2, hidden=64, width=32, classes=500, dtype=torch.bfloat16, seed=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)

        def param(*shape, fan_in=None, at=0.0):
            scale = math.sqrt(2.0 / fan_in) if fan_in else 0.0
            return (torch.randn(shape, generator=gen, device="cuda") * scale + at).requires_grad_(True)

        self.k, self.experts, self.hidden, self.width, self.classes, self.dtype = (choices, experts, hidden, width,
                                                                                   classes, dtype)
        self.gate, self.gate_b = param(1, experts, FEATURES, fan_in=4 * FEATURES), param(1, experts)
        self.w1, self.b1 = param(experts, hidden, FEATURES, fan_in=FEATURES), param(experts, hidden)
        self.w2, self.b2 = param(experts, width, hidden, fan_in=hidden), param(experts, width)
        self.keep, self.keep_b = param(1, width, width, fan_in=8 * width), param(1, width, at=2.0)
        self.head, self.head_b = param(1, classes, width, fan_in=width), param(1, classes)
        self.start = param(width)
        self.params = [self.gate, self.gate_b, self.w1, self.b1, self.w2, self.b2, self.keep, self.keep_b, self.head,
                       self.head_b, self.start]
        for p in self.params:
            p.grad = torch.zeros_like(p)
        self.grads = v.nerf_tensor_list([p.grad for p in self.params])
        self.norm = torch.empty(1, device="cuda")

    def _new(self, *shape, dtype=None):
        return torch.empty(shape, dtype=dtype or self.dtype, device="cuda")

    def _weights(self):
        """The matrices in the field's type."""
        return {name: getattr(self, name).detach().to(self.dtype) for name in ("gate", "w1", "w2", "keep", "head")}

    def _dense(self, x, weight, bias):
        """A linear layer: one expert that owns every row."""
        y = self._new(x.shape[0], weight.shape[1])
        rows = torch.tensor([0, x.shape[0]], dtype=I32, device="cuda")
        v.nerf_expert_linear(x, weight, bias.detach(), rows, y)
        return y

    def _dense_grad(self, dy, x, weight, dweight, dbias):
        dx = torch.empty_like(x)
        rows = torch.tensor([0, x.shape[0]], dtype=I32, device="cuda")
        v.nerf_expert_linear_grad(dy, x, weight, rows, dx, dweight, dbias)
        return dx

    def _route(self, points, w):
        """Encodings of points [n, 3], each one's experts and their weights."""
        enc = self._new(points.shape[0], FEATURES)
        v.nerf_encode_freq(points, FREQS, False, True, v.NERF_BF16 if self.dtype == torch.bfloat16 else v.NERF_F32, enc)
        logits = self._dense(enc, w["gate"], self.gate_b)
        ids, weights = self._new(points.shape[0], self.k, dtype=I32), self._new(points.shape[0], self.k, dtype=F32)
        v.nerf_route_gate(logits, ids, weights)
        return enc, ids, weights

    def forward(self, points, offsets):
        """Class logits after every sample: ``points`` [rows, 3], the rays'
        samples one after another, ray r's from offsets[r] on."""
        self.w, self.offsets_r = self._weights(), offsets
        n = points.shape[0]
        self.enc, self.ids, self.weights = self._route(points, self.w)
        self.offsets, self.order, self.place = (self._new(self.experts + 1, dtype=I32), self._new(n * self.k, dtype=I32),
                                                self._new(n, self.k, dtype=I32))
        v.nerf_route_plan(self.ids, self.experts, self.offsets, self.order, self.place)
        self.h, self.y, self.feat = (self._new(n * self.k, self.hidden), self._new(n * self.k, self.width),
                                     self._new(n, self.width))
        v.nerf_expert_linear(self.enc, self.w["w1"], self.b1.detach(), self.offsets, self.h, order=self.order, k=self.k,
                             relu=True)
        v.nerf_expert_linear(self.h, self.w["w2"], self.b2.detach(), self.offsets, self.y)
        v.nerf_route_combine(self.y, self.offsets, self.place, self.weights, self.feat)
        self.a = torch.sigmoid(self._dense(self.feat, self.w["keep"], self.keep_b).float())
        self.h0 = self.start.detach().expand(offsets.numel() - 1, self.width).contiguous()
        self.state = self._new(n, self.width)
        v.nerf_scan(self.a, self.feat, self.state, h0=self.h0, offsets=offsets, mix=True)
        self.logits = self._dense(self.state, self.w["head"], self.head_b)
        return self.logits

    def backward(self, t_logits, t_ids, temperature, max_norm):
        """Mean loss of the last forward pass against the teacher's largest
        logits; sets every parameter's gradient, together of at most
        ``max_norm`` (None: as they are)."""
        n = self.logits.shape[0]
        loss, dlogits = self._new(n, dtype=F32), torch.empty_like(self.logits)
        scale = torch.full((n,), 1.0 / n, device="cuda")
        v.nerf_distill_topk(self.logits, t_logits, t_ids, temperature, loss, grad=dlogits, row_scale=scale)
        dstate = self._dense_grad(dlogits, self.state, self.w["head"], self.head.grad, self.head_b.grad)
        da, dfeat, dh0 = torch.empty_like(self.a), torch.empty_like(self.feat), torch.empty_like(self.h0)
        v.nerf_scan_grad(dstate, self.a, self.feat, self.state, da, dfeat, h0=self.h0, dh0=dh0, offsets=self.offsets_r,
                         mix=True)
        self.start.grad.copy_(dh0.sum(0))
        dkeep = (da * self.a * (1.0 - self.a)).to(self.dtype)
        dfeat += self._dense_grad(dkeep, self.feat, self.w["keep"], self.keep.grad, self.keep_b.grad)
        dy, dweights = torch.empty_like(self.y), torch.empty_like(self.weights)
        v.nerf_route_combine_grad(dfeat, self.y, self.offsets, self.place, self.weights, dy, dweights)
        dh = torch.empty_like(self.h)
        v.nerf_expert_linear_grad(dy, self.h, self.w["w2"], self.offsets, dh, self.w2.grad, self.b2.grad, relu_x=True)
        v.nerf_expert_linear_grad(dh, self.enc, self.w["w1"], self.offsets, None, self.w1.grad, self.b1.grad,
                                  order=self.order, k=self.k)
        dgate = self._new(n, self.experts)
        v.nerf_route_gate_grad(dweights, None, self.ids, self.weights, dgate)
        self._dense_grad(dgate, self.enc, self.w["gate"], self.gate.grad, self.gate_b.grad)
        if max_norm is None:
            v.nerf_grad_norm(self.grads, self.norm)
        else:
            v.nerf_grad_clip(self.grads, max_norm, self.norm)
        return loss.mean()

    def streams(self, n):
        """Serving state of n rays that begin, and the weights to serve with."""
        state = self.start.detach().expand(n, self.width).contiguous()
        ws = torch.empty(v.nerf_routed_mlp_workspace_size(n, self.k, self.hidden, self.width), dtype=torch.uint8,
                         device="cuda")
        return dict(state=state, w=self._weights(), ws=ws)

    def step(self, streams, points):
        """Class logits after one more sample of each ray: ``points`` [n, 3]."""
        w, n = streams["w"], points.shape[0]
        enc, ids, weights = self._route(points, w)
        feat, out = self._new(n, self.width), self._new(n, self.width)
        v.nerf_routed_mlp(enc, ids, weights, w["w1"], self.b1.detach(), w["w2"], self.b2.detach(), feat,
                          workspace=streams["ws"])
        a = torch.sigmoid(self._dense(feat, w["keep"], self.keep_b).float())
        v.nerf_scan(a, feat, out, h0=streams["state"], h_last=streams["state"], n_seq=n, mix=True)
        return self._dense(out, w["head"], self.head_b)


def teacher_logits(points, offsets, classes, top, seed=1):
    """The `top` largest logits (and their classes) of a fixed smooth function
    of the mean of a ray's samples so far."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    a = torch.randn((3, 64), generator=gen, device="cuda") * 2.0
    b = torch.randn((64, classes), generator=gen, device="cuda") * 0.7
    rows = torch.arange(points.shape[0], device="cuda")
    first = offsets[torch.searchsorted(offsets, rows.to(I32), right=True) - 1].long()
    sums = torch.cat([points.new_zeros(1, 3), points.double().cumsum(0).float()])
    mean = (sums[rows + 1] - sums[first]) / (rows - first + 1)[:, None]
    t, ids = (torch.sin(mean @ a) @ b).topk(top, dim=1)
    return t.contiguous(), ids.to(I32)


def rays(n, samples, gen):
    """n rays of 0 to 2 `samples` samples each: points [rows, 3] and where each begins."""
    lengths = torch.randint(0, 2 * samples + 1, (n,), generator=gen, device="cuda")
    offsets = torch.cat([lengths.new_zeros(1), lengths.cumsum(0)]).to(I32)
    return torch.rand((int(offsets[-1]), 3), generator=gen, device="cuda") * 2.0 - 1.0, offsets


def train(steps=200, n=512, samples=64, classes=500, top=16, temperature=1.0, lr=2e-3, max_norm=1.0, every=20, say=print):
    field = StreamField(classes=classes)
    opt = torch.optim.Adam(field.params, lr=lr)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(7)
    losses = []
    for step in range(steps):
        points, offsets = rays(n, samples, gen)
        field.forward(points, offsets)
        loss = field.backward(*teacher_logits(points, offsets, classes, top), temperature, max_norm)
        opt.step()
        if step % every == 0 or step == steps - 1:
            losses.append(loss.item())
            say(f"step {step:4d}  loss {losses[-1]:.4f}  gradient norm {field.norm.item():.3f}")
    return field, losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--rays", type=int, default=512)
    ap.add_argument("--samples", type=int, default=64)
    args = ap.parse_args()
    field, _ = train(args.steps, args.rays, args.samples)
    streams, points = field.streams(8), torch.rand((20, 8, 3), device="cuda") * 2.0 - 1.0
    for p in points:
        logits = field.step(streams, p)
    print("classes after 20 samples of 8 streams:", logits.float().argmax(1).tolist())
