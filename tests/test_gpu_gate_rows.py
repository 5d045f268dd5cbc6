"""Every row of large gates, and more rows than one pass of the grid takes,
against the definition in float64 on the device (ties by a stable sort).  Bounds
as in test_gpu_gate.py."""
import pytest

from tests.gpu_util import say, torch_cuda

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("n,E,k", [(20001, 16, 2), (262150, 260, 3)])  # (four rows a workgroup, 65536 workgroups at most)
def test_every_row(n, E, k, bf16, renorm):
    torch = torch_cuda()
    import volume_rendering_amd as v
    say(f"gate rows n={n} E={E} bf16={bf16} renorm={renorm}")
    gen = torch.Generator(device="cuda").manual_seed(n + E)
    z = 2.0 * torch.randn((n, E), generator=gen, device="cuda")
    z[torch.rand((n, E), generator=gen, device="cuda") < 0.3] = float("-inf")
    z[n // 3] = z[n - 1] = float("-inf")
    z[n - 2, 1:] = float("-inf")
    z = z.to(torch.bfloat16 if bf16 else torch.float32)
    dw = torch.randn((n, k), generator=gen, device="cuda")
    ids = torch.full((n, k), -9, dtype=torch.int32, device="cuda")
    w = torch.full((n, k), 7.0, device="cuda")
    v.nerf_route_gate(z, ids, w, renorm=renorm)

    zd = z.double()
    top, at = torch.sort(zd, dim=1, descending=True, stable=True)
    top, at = top[:, :k], at[:, :k]
    live = top > float("-inf")
    assert torch.equal(ids, torch.where(live, at, -1).to(torch.int32))
    m = torch.where(live[:, :1], top[:, :1], 0.0)
    e = torch.exp(zd - m)
    own = torch.where(live, torch.exp(top - m), 0.0)
    total = own.sum(1, keepdim=True) if renorm else e.sum(1, keepdim=True)
    want = own / torch.where(total > 0, total, 1.0)
    far = torch.where(live, m - top, 0.0).max()
    assert ((w.double() - want).abs() <= 2 * U * want * (E + far + 8) + 1e-37).all()

    dz = torch.full((n, E), 7.0, dtype=z.dtype, device="cuda")
    v.nerf_route_gate_grad(dw, None if renorm else z, ids, w, dz, renorm=renorm)
    wd = torch.where(live, w.double() * dw.double(), 0.0)
    S, absolute = wd.sum(1, keepdim=True), wd.abs().sum(1, keepdim=True)
    ref, mag = torch.zeros_like(zd), torch.zeros_like(zd)
    column = torch.where(live, at, 0)
    wl = torch.where(live, w.double(), 0.0)
    if renorm:
        ref.scatter_add_(1, column, torch.where(live, wl * (dw.double() - S), 0.0))
    else:
        p = e / torch.where(live[:, :1], e.sum(1, keepdim=True), 1.0)
        ref.sub_(p * S).scatter_add_(1, column, wd)
        mag.add_(p * absolute)
    mag.scatter_add_(1, column, wd.abs() + wl * absolute)
    tol = 2 * U * (E + k + 24 + far) * mag
    tol = tol + (2.0 ** -8 if bf16 else U) * (ref.abs() + tol) + 1e-37
    assert ((dz.double() - ref).abs() <= tol).all()
