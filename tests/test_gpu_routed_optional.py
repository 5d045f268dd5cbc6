"""Gradients of the experts' layers without the operand that they do not need:
the same bits as with it."""
import numpy as np
import pytest

import volume_rendering_amd as v
from tests.gpu_util import say, torch_cuda

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("d_in,d_out,per", [(7, 5, 40), (64, 64, 30), (136, 264, 300)])
def test_gradients_without_x_or_weight(d_in, d_out, per, bf16):
    torch = torch_cuda()
    say(f"optional operands {d_in} -> {d_out} bf16={bf16}")
    g = np.random.default_rng([31, d_in, d_out])
    E, k = 3, 2
    S = E * per
    dt = torch.bfloat16 if bf16 else torch.float32
    mk = lambda *s: torch.from_numpy(g.standard_normal(s).astype(np.float32)).cuda().to(dt)
    dz, x, w = mk(S, d_out), mk(S, d_in), mk(E, d_out, d_in)
    i32 = dict(dtype=torch.int32, device="cuda")
    off, order = torch.arange(E + 1, **i32) * per, torch.randperm(S, device="cuda").to(torch.int32)
    out = lambda: (torch.full_like(x, 4.0), torch.full(w.shape, 4.0, device="cuda"),
                   torch.full((E, d_out), 4.0, device="cuda"))
    for kw in ({}, dict(order=order, k=k)):
        (dx, dw, db), (dx1, dw1, db1) = out(), out()
        v.nerf_expert_linear_grad(dz, x, w, off, dx, dw, db, **kw)
        v.nerf_expert_linear_grad(dz, None, w, off, dx1, **kw)
        v.nerf_expert_linear_grad(dz, x, None, off, None, dw1, db1, **kw)
        torch.cuda.synchronize()
        assert torch.equal(dx, dx1) and torch.equal(dw, dw1) and torch.equal(db, db1)
        with pytest.raises(v.NerfError, match="x is NULL"):
            v.nerf_expert_linear_grad(dz, None, w, off, dx1, dw1, **kw)
        with pytest.raises(v.NerfError, match="x is NULL"):
            v.nerf_expert_linear_grad(dz, None, w, off, dx1, relu_x=True, **kw)
        with pytest.raises(v.NerfError, match="weights are NULL"):
            v.nerf_expert_linear_grad(dz, x, None, off, dx1, dw1, **kw)
