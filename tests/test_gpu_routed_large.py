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


@pytest.mark.parametrize("n", [(1 << 24) + 3, (1 << 26) + 5])
def test_distillation_of_many_rows(n):
    """More rows than one launch holds workgroups for (2^24 of 256 threads, 2^26 of
    64): two classes of float32, one of them the teacher's, so that with d the
    other's lead the loss is ln(1 + e^d) and the gradient -+ s / (1 + e^-d).
    A row's terms are few: 16 u of their sizes cover their roundings."""
    torch = torch_cuda()
    import volume_rendering_amd as v
    say(f"distillation of {n} rows")
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    z = torch.randn((n, 2), generator=g, device="cuda")
    t = torch.zeros((n, 1), device="cuda")
    ids = torch.randint(0, 2, (n, 1), generator=g, device="cuda", dtype=torch.int32)
    scale = torch.rand(n, generator=g, device="cuda")
    loss, lse = torch.full((n,), 9.0, device="cuda"), torch.full((n,), 9.0, device="cuda")
    both, alone = torch.full_like(z, 9.0), torch.full_like(z, 9.0)
    v.nerf_distill_topk(z, t, ids, 1.0, loss, lse=lse, grad=both, row_scale=scale)
    v.nerf_distill_topk_grad(z, t, ids, 1.0, lse, alone, row_scale=scale)
    u = 2.0 ** -23
    for a in range(0, n, 1 << 22):
        s = slice(a, min(a + (1 << 22), n))
        x, at = z[s].double(), ids[s].long()
        mine = x.gather(1, at)[:, 0]
        d = x.gather(1, 1 - at)[:, 0] - mine
        want = torch.nn.functional.softplus(d)
        assert torch.all((loss[s] - want).abs() <= 16 * u * (1 + want + d.abs())), a
        want_lse = torch.logsumexp(x, 1)
        assert torch.all((lse[s] - want_lse).abs() <= 16 * u * (1 + want_lse.abs() + x.abs().amax(1))), a
        p = scale[s].double() * torch.sigmoid(d)
        want_g = torch.empty_like(x).scatter_(1, at, -p[:, None]).scatter_(1, 1 - at, p[:, None])
        size = scale[s].double()[:, None] * (1 + d.abs() + x.abs().amax(1) + want_lse.abs())[:, None]
        for got in (both, alone):
            assert torch.all((got[s] - want_g).abs() <= 16 * u * size), a
