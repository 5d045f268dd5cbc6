"""The copied bfloat16 kernels of the experts' products where the other tests do
not take them: around 64 experts (up to 63 their tiles are counted, beyond they
are searched for, and some are empty), rows further apart than they are wide but
still 16-byte aligned, samples with four and more choices, and workspaces of
exactly the size that is asked for.  Against the float64 oracle, with the bounds
of tests/test_gpu_routed.py: (terms + 2) 2^-23 of the terms' magnitudes, and 2^-8
of a bfloat16 result.
"""
import numpy as np
import pytest

import volume_rendering_amd as v
from oracle import routed as R
from tests.gpu_util import host, say, torch_cuda

pytestmark = pytest.mark.gpu

U32, UB = 2.0 ** -23, 2.0 ** -8


def _f64(t):
    torch = torch_cuda()
    torch.cuda.synchronize()
    return t.detach().float().cpu().numpy().astype(np.float64)


def _ids(g, n, k, E):
    """Every other expert has no pair, one has a third of them, some pairs no expert."""
    ids = 2 * g.integers(0, (E + 1) // 2, (n, k))
    ids[g.random((n, k)) < 0.33] = (E // 4) * 2
    ids[g.random((n, k)) < 0.07] = g.choice([-1, E])
    return ids.astype(np.int32)


def _apart(torch, t, pad, value):
    """t in rows `pad` elements further apart, a multiple of 8 of them before each."""
    if not pad:
        return t
    big = torch.full((t.shape[0], t.shape[1] + pad), value, dtype=t.dtype, device="cuda")
    big[:, 8:8 + t.shape[1]] = t
    return big[:, 8:8 + t.shape[1]]


def _untouched(t, pad, value):
    return not pad or bool((t._base[:, :8] == value).all() and (t._base[:, 8 + t.shape[1]:] == value).all())


# (n, k, E, d_in, d_out): with 32 slots an expert or more, more than 128 x 128 weights and more than 64 columns
LAYERS = [(2100, 1, 63, 136, 264), (2200, 1, 64, 136, 264), (1300, 2, 70, 264, 136), (900, 5, 129, 136, 136),
          (2400, 7, 500, 264, 72), (17000, 2, 65, 72, 264), (600, 4, 5, 264, 136), (700, 3, 2, 520, 72),
          (12160, 2, 64, 72, 264), (12160, 2, 64, 264, 72)]  # (tiles of 256 slots)


@pytest.mark.parametrize("pad", [0, 16, 8])
@pytest.mark.parametrize("through_order", [False, True])
@pytest.mark.parametrize("case", LAYERS)
def test_copied_tiles(case, through_order, pad):
    torch = torch_cuda()
    n, k, E, d_in, d_out = case
    say(f"copied tiles {case} order={through_order} pad={pad}")
    g = np.random.default_rng([41, *case])
    S, bf = n * k, torch.bfloat16
    mk = lambda *s, scale=1.0: torch.from_numpy((scale * g.standard_normal(s)).astype(np.float32)).cuda()
    off, order, place = (torch.empty(s, dtype=torch.int32, device="cuda") for s in ((E + 1,), (S,), (n, k)))
    v.nerf_route_plan(torch.from_numpy(_ids(g, n, k, E)).cuda(), E, off, order, place)
    ho, hord = host(off), host(order)
    live = int(ho[-1])
    assert (np.diff(ho) == 0).any() or E < 6
    rows = hord // k if through_order else None
    x = torch.relu(mk(n if through_order else S, d_in)).to(bf)
    w, b, dz = mk(E, d_out, d_in, scale=d_in ** -0.5).to(bf), mk(E, d_out), mk(S, d_out).to(bf)
    if not through_order:
        x[live:] = float("nan")
    dz[live:] = float("nan")
    hx, hw, hb, hz = np.nan_to_num(_f64(x)), _f64(w), _f64(b), np.nan_to_num(_f64(dz))
    kw = dict(order=order, k=k) if through_order else {}
    # what lies between the rows of an operand counts for nothing, and is left alone in a result
    xs, zs = _apart(torch, x, pad, float("nan")), _apart(torch, dz, pad, float("nan"))

    for relu in (False, True):
        y = _apart(torch, torch.full((S, d_out), 4.0, dtype=bf, device="cuda"), pad, 7.0)
        v.nerf_expert_linear(xs, w, b, off, y, relu=relu, **kw)
        want = R.expert_linear(hx, hw, hb, ho, S, rows, relu)
        mag = R.expert_linear(np.abs(hx), np.abs(hw), np.abs(hb), ho, S, rows)
        assert np.all(np.abs(_f64(y) - want) <= (d_in + 2) * U32 * mag + UB * np.abs(want))
        assert not _f64(y)[live:].any() and _untouched(y, pad, 7.0)

    counts = np.diff(ho)[:, None]
    size = v.nerf_expert_linear_grad_workspace_size(S, E, d_in, d_out)
    for relu_x in (False, True):
        dx = torch.full((S, d_in), 4.0, dtype=bf, device="cuda")
        dw, db = torch.full(w.shape, 4.0, device="cuda"), torch.full((E, d_out), 4.0, device="cuda")
        ws = torch.full((size + 4096,), 77, dtype=torch.uint8, device="cuda")
        v.nerf_expert_linear_grad(zs, xs, w, off, dx, dw, db, relu_x=relu_x, workspace=ws[:size] if size else None, **kw)
        want = R.expert_linear_grad(hz, hx, hw, ho, rows, relu_x)
        mag = R.expert_linear_grad(np.abs(hz), np.abs(hx), np.abs(hw), ho, rows)
        assert np.all(np.abs(_f64(dx) - want[0]) <= (d_out + 2) * U32 * mag[0] + UB * np.abs(want[0]))
        assert not _f64(dx)[live:].any()
        assert np.all(np.abs(_f64(dw) - want[1]) <= (counts[:, :, None] + 2) * U32 * mag[1])
        assert np.all(np.abs(_f64(db) - want[2]) <= (counts + 2) * U32 * mag[2])
        assert (ws[size:] == 77).all()


@pytest.mark.parametrize("n,k,E", [(3000, 2, 5), (9001, 3, 4096)])
def test_plan_stays_in_its_workspace(n, k, E):
    torch = torch_cuda()
    g = np.random.default_rng([42, n, k, E])
    size = v.nerf_route_workspace_size(n, k, E)
    assert size > 0
    ws = torch.full((size + 4096,), 77, dtype=torch.uint8, device="cuda")
    off, order, place = (torch.empty(s, dtype=torch.int32, device="cuda") for s in ((E + 1,), (n * k,), (n, k)))
    ids = _ids(g, n, k, E)
    v.nerf_route_plan(torch.from_numpy(ids).cuda(), E, off, order, place, workspace=ws[:size])
    ho, hord, hp = R.plan(ids, E)
    assert np.array_equal(host(off), ho) and np.array_equal(host(order), hord) and np.array_equal(host(place), hp)
    assert (ws[size:] == 77).all()


@pytest.mark.parametrize("n,V", [(1, 50001), (7, 9001), (255, 12345)])
def test_distillation_stays_in_its_workspace(n, V):
    torch = torch_cuda()
    g = np.random.default_rng([43, n, V])
    size = v.nerf_distill_workspace_size(n, V)
    assert size > 0
    z = torch.from_numpy(g.standard_normal((n, V)).astype(np.float32)).cuda()
    t = torch.from_numpy(g.standard_normal((n, 5)).astype(np.float32)).cuda()
    ids = torch.from_numpy(g.integers(0, V, (n, 5)).astype(np.int32)).cuda()
    ws = torch.full((size + 4096,), 77, dtype=torch.uint8, device="cuda")
    a, b = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    ga, gb = torch.empty_like(z), torch.empty_like(z)
    v.nerf_distill_topk(z, t, ids, 2.0, a, grad=ga, workspace=ws[:size])
    v.nerf_distill_topk(z, t, ids, 2.0, b, grad=gb)  # one of its own
    assert torch.equal(a, b) and torch.equal(ga, gb) and (ws[size:] == 77).all()
