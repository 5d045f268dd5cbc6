"""Weight gradients on either side of the rules that pick their tiles and split their
sums: experts of 2048 slots or fewer, as many tiles as CUs or fewer."""
import numpy as np
import pytest

import volume_rendering_amd as v
from tests.gpu_util import say, torch_cuda

pytestmark = pytest.mark.gpu

# (experts, slots an expert on average, d_in, d_out)
CASES = [(255, 40, 136, 136), (256, 40, 136, 136), (64, 48, 264, 264), (3, 2047, 136, 200), (3, 2048, 136, 200),
         (32, 100, 264, 264), (3, 4095, 136, 200), (3, 4096, 136, 200),
         (2, 5000, 264, 130), (1, 9001, 520, 136)]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("through_order", [False, True])
@pytest.mark.parametrize("E,per,d_in,d_out", CASES)
def test_weight_gradients(E, per, d_in, d_out, through_order, bf16):
    """Against products in float64 of the same rounded inputs, expert by expert:
    (terms + 2) 2^-23 of the terms' magnitudes."""
    torch = torch_cuda()
    say(f"weight gradients E={E} per={per} {d_in}->{d_out} order={through_order} bf16={bf16}")
    g = np.random.default_rng([51, E, per, d_in, d_out])
    S, dt = E * per, torch.bfloat16 if bf16 else torch.float32
    cuts = np.sort(g.integers(0, S + 1, E - 1)) if E > 1 else np.zeros(0, np.int64)
    off = torch.from_numpy(np.concatenate([[0], cuts, [S - min(3, S)]]).clip(0, S - min(3, S)).astype(np.int32)).cuda()
    x = torch.from_numpy(g.standard_normal((S, d_in)).astype(np.float32)).cuda().to(dt)
    z = torch.from_numpy(g.standard_normal((S, d_out)).astype(np.float32)).cuda().to(dt)
    order = torch.from_numpy(g.permutation(S).astype(np.int32)).cuda() if through_order else None
    dw, db = torch.full((E, d_out, d_in), 4.0, device="cuda"), torch.full((E, d_out), 4.0, device="cuda")
    v.nerf_expert_linear_grad(z, x, None, off, None, dw, db, order=order)
    torch.cuda.synchronize()
    xs = (x[order.long()] if through_order else x).double()
    zs, ho = z.double(), off.cpu().tolist()
    for e in range(E):
        a, b = zs[ho[e]:ho[e + 1]], xs[ho[e]:ho[e + 1]]
        tol = (ho[e + 1] - ho[e] + 2) * 2.0 ** -23
        assert torch.all((dw[e] - a.t() @ b).abs() <= tol * (a.abs().t() @ b.abs())), e
        assert torch.all((db[e] - a.sum(0)).abs() <= tol * a.abs().sum(0)), e
