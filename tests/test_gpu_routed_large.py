"""Calls as large as the card allows: more work items than 2^32 / 4."""
import pytest

from tests.gpu_util import say, torch_cuda

pytestmark = pytest.mark.gpu


def test_expert_layer_of_many_slots_and_columns():
    """4,300,013 slots of 4096 columns (2^34 elements, 35 GB): every row is its
    expert's weight times the row's value, exact in bfloat16."""
    torch = torch_cuda()
    import volume_rendering_amd as v
    say("expert layer of 4,300,013 slots x 4096 columns")
    S, d, E = 4300013, 4096, 3
    bf = dict(dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([0, 5, S // 2, S - 7], dtype=torch.int32, device="cuda")  # the last 7 slots have no expert
    x = torch.zeros((S, 8), **bf)
    x[:, 2] = torch.arange(S, device="cuda").remainder(5).to(torch.bfloat16)
    w = torch.zeros((E, d, 8), **bf)
    w[:, :, 2] = torch.arange(E * d, device="cuda").remainder(13).to(torch.bfloat16).view(E, d)
    y = torch.full((S, d), 9.0, **bf)
    v.nerf_expert_linear(x, w, None, off, y)
    bounds = [0, 5, S // 2, S - 7, S]
    for e in range(E + 1):
        for a in range(bounds[e], bounds[e + 1], 1 << 19):
            b = min(a + (1 << 19), bounds[e + 1])
            want = x[a:b, 2:3] * w[e, :, 2] if e < E else torch.zeros((b - a, d), **bf)
            assert torch.equal(y[a:b], want), (e, a)
            del want
    # and its gradient: dx is the product of w with a dz that picks one column a row
    torch.cuda.synchronize()
    y.zero_()
    y[:, 4095] = 1.0
    dx = torch.full((S, 8), 9.0, **bf)
    v.nerf_expert_linear_grad(y, None, w, off, dx)
    want = torch.zeros_like(dx)
    for e in range(E):
        want[bounds[e]:bounds[e + 1]] = w[e, 4095]
    assert torch.equal(dx, want)
