"""examples/stream_routed_field.py: the operators in one run.  Its gradients
against torch's autograd of the same network in float64, and serving sample by
sample against the pass over whole rays.

Bounds, for a float32 field.  Every value on the way is a sum of at most n terms
with n up to 800 (rows of the weight gradients), so off by n 2^-24 of the sum of
their magnitudes, over about ten operators in a row, forwards and back: 10 x 800 x
2^-24 = 2^-11 of the magnitudes; 2^-8 of the gradient's norm leaves a factor of
eight for terms that cancel.  Serving adds the same numbers up in another order:
2^-11 of the logits' largest magnitude.
"""
import os
import sys

import numpy as np
import pytest

from tests.gpu_util import say, torch_cuda

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def _field(torch, ex, dtype, classes=101):
    f = ex.StreamField(experts=5, choices=2, hidden=24, width=12, classes=classes, dtype=dtype, seed=3)
    gen = torch.Generator(device="cuda").manual_seed(2)
    lengths = torch.tensor([0, 7, 33, 1, 64, 0, 130, 20], device="cuda")
    offsets = torch.cat([lengths.new_zeros(1), lengths.cumsum(0)]).to(torch.int32)
    points = torch.rand((int(offsets[-1]), 3), generator=gen, device="cuda") * 2 - 1
    with torch.no_grad():
        f.start.copy_(torch.randn(12, generator=gen, device="cuda"))
    return f, points, offsets


def test_gradients_of_the_example_match_autograd():
    torch = torch_cuda()
    import stream_routed_field as ex
    f, points, offsets = _field(torch, ex, torch.float32)
    T = 2.0
    f.forward(points, offsets)
    t, ids = ex.teacher_logits(points, offsets, 101, 8)
    ids[5] = -1  # a sample outside the loss
    loss = f.backward(t, ids, T, None)

    names = ["gate", "gate_b", "w1", "b1", "w2", "b2", "keep", "keep_b", "head", "head_b", "start"]
    p = {n: getattr(f, n).detach().double().cpu().requires_grad_(True) for n in names}
    enc, eid, off = f.enc.double().cpu(), f.ids.long().cpu(), offsets.tolist()
    wt = torch.softmax((enc @ p["gate"][0].t() + p["gate_b"][0]).gather(1, eid), 1)
    feat = 0
    for j in range(2):
        e = eid[:, j]
        h = torch.relu(torch.bmm(p["w1"][e].contiguous(), enc[:, :, None])[:, :, 0] + p["b1"][e])
        feat = feat + wt[:, j:j + 1] * (torch.bmm(p["w2"][e].contiguous(), h[:, :, None])[:, :, 0] + p["b2"][e])
    a = torch.sigmoid(feat @ p["keep"][0].t() + p["keep_b"][0])
    states = []
    for r in range(len(off) - 1):
        state = p["start"]
        for i in range(off[r], off[r + 1]):
            state = a[i] * state + (1 - a[i]) * feat[i]
            states.append(state)
    logits = torch.stack(states) @ p["head"][0].t() + p["head_b"][0]
    logp = torch.log_softmax(t.double().cpu() / T, 1)
    logq = torch.log_softmax(logits / T, 1).gather(1, ids.long().cpu().clamp_min(0))
    rows = T * T * (logp.exp() * (logp - logq)).sum(1)
    want = torch.where((ids >= 0).all(1).cpu(), rows, 0.0).mean()
    want.backward()
    assert abs(loss.item() - want.item()) <= 2.0 ** -11 * want.item()
    for n in names:
        g, r = getattr(f, n).grad.double().cpu().numpy(), p[n].grad.numpy()
        err = np.linalg.norm(g - r) / np.linalg.norm(r)
        say(f"  {n}: gradient off by {err:.1e} of its norm")
        assert err <= 2.0 ** -8, n
    norm = np.sqrt(sum(np.square(p[n].grad.numpy()).sum() for n in names))
    assert abs(f.norm.item() - norm) <= 2.0 ** -8 * norm
    # clipped: the same direction, half the norm
    before = [q.grad.clone() for q in f.params]
    f.backward(t, ids, T, 0.5 * norm)
    factor = 0.5 * norm / f.norm.item()
    for old, q in zip(before, f.params):
        assert torch.allclose(q.grad, old * factor, rtol=1e-5, atol=1e-12)


def test_serving_sample_by_sample_equals_the_whole_rays():
    torch = torch_cuda()
    import stream_routed_field as ex
    f, _, _ = _field(torch, ex, torch.float32)
    n, steps = 9, 30
    points = torch.rand((n, steps, 3), device="cuda", generator=torch.Generator(device="cuda").manual_seed(4)) * 2 - 1
    offsets = (torch.arange(n + 1, device="cuda") * steps).to(torch.int32)
    whole = f.forward(points.reshape(-1, 3), offsets).view(n, steps, -1)
    streams = f.streams(n)
    for i in range(steps):
        logits = f.step(streams, points[:, i].contiguous())
        err = (logits - whole[:, i]).abs().max().item()
        assert err <= 2.0 ** -11 * whole.abs().max().item(), i


def test_training_and_serving_run():
    torch = torch_cuda()
    import stream_routed_field as ex
    field, losses = ex.train(steps=12, n=64, samples=16, classes=100, top=8, every=4, say=say)
    assert np.isfinite(losses).all()
    streams = field.streams(3)
    for _ in range(3):
        logits = field.step(streams, torch.rand((3, 3), device="cuda"))
    assert torch.isfinite(logits.float()).all()
