"""examples/distill_routed_field.py: its gradients against torch's autograd on
the same bfloat16 values in float64, and that training lowers the loss."""
import os
import sys

import numpy as np
import pytest

from tests.gpu_util import say, torch_cuda

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_gradients_of_the_example_match_autograd():
    """Every stored activation and gradient is rounded to bfloat16 (2^-8 each):
    at most six roundings lie between a parameter's gradient and the exact one
    (features, hidden, sum, logits and the gradients back through them), each
    relative to magnitudes of the size of the gradient's own terms.  2^-5 of
    the gradient's norm covers them."""
    torch = torch_cuda()
    import distill_routed_field as ex
    n, classes, T = 700, 203, 2.0
    f = ex.RoutedField(n, experts=5, choices=2, hidden=40, width=24, classes=classes, seed=3)
    x = torch.rand((n, 3), device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)) * 2 - 1
    t, ids = ex.teacher_logits(x, classes, 8)
    ids[5] = -1  # a point outside the loss
    f.forward(x)
    loss = f.backward(t, ids, T)

    d = lambda p: p.detach().to(torch.bfloat16).double().cpu().requires_grad_(True)
    full = lambda p: p.detach().double().cpu().requires_grad_(True)
    gate, b1, b2, hb = full(f.gate), full(f.b1), full(f.b2), full(f.head_b)
    w1, w2, head = d(f.w1), d(f.w2), d(f.head)
    enc, eid = f.enc.double().cpu(), f.ids.long().cpu()
    wt = torch.softmax((enc @ gate).gather(1, eid), 1)
    feat = 0
    for j in range(2):
        e = eid[:, j]
        h = torch.relu(torch.bmm(w1[e].contiguous(), enc[:, :, None])[:, :, 0] + b1[e])
        feat = feat + wt[:, j:j + 1] * (torch.bmm(w2[e].contiguous(), h[:, :, None])[:, :, 0] + b2[e])
    logits = feat @ head[0].t() + hb[0]
    logp = torch.log_softmax(t.double().cpu() / T, 1)
    logq = torch.log_softmax(logits / T, 1).gather(1, ids.long().cpu().clamp_min(0))
    rows = T * T * (logp.exp() * (logp - logq)).sum(1)
    rows = torch.where((ids >= 0).all(1).cpu(), rows, 0.0)
    want = rows.mean()
    want.backward()
    assert abs(loss.item() - want.item()) <= 2.0 ** -5 * want.item()
    for name, got, ref in (("gate", f.gate, gate), ("w1", f.w1, w1), ("b1", f.b1, b1), ("w2", f.w2, w2),
                           ("b2", f.b2, b2), ("head", f.head, head), ("head bias", f.head_b, hb)):
        g, r = got.grad.double().cpu().numpy(), ref.grad.numpy()
        err = np.linalg.norm(g - r) / np.linalg.norm(r)
        say(f"  {name}: gradient off by {err:.1e} of its norm")
        assert err <= 2.0 ** -5, name


def test_training_lowers_the_loss():
    import distill_routed_field as ex
    torch_cuda()
    losses = ex.train(steps=61, points=8192, classes=300, top=8, every=20, say=say)
    assert losses[-1] < 0.8 * losses[0] and np.isfinite(losses).all()
