"""Routed fields on the GPU against the float64 oracle (oracle/routed.py):
the plan, row movement, the experts' products and their gradients.

Bounds.  A float32 sum of n terms differs from the exact one by at most
n 2^-24 sum |terms| for any order, rounding each product adds 2^-24 of it:
(n + 1) 2^-23 sum |terms| covers both with a factor of two (the matrix cores
may round inside a step).  bfloat16 results round once more, by at most 2^-8 of
the result.  Inputs are rounded to the type first, so products are exact.
"""
import numpy as np
import pytest

from oracle import routed as R
from tests.gpu_util import host, say, torch_cuda

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -23
UB = 2.0 ** -8


def _dt(torch, bf16):
    return torch.bfloat16 if bf16 else torch.float32


def _f64(t):
    torch = torch_cuda()
    torch.cuda.synchronize()
    return t.detach().float().cpu().numpy().astype(np.float64)


def _ids(g, n, k, E, drop, skew=False):
    if skew:  # most pairs to one expert, some experts without any
        ids = np.where(g.random((n, k)) < 0.7, E // 2, g.integers(0, E, (n, k)))
    else:
        ids = g.integers(0, E, (n, k))
    ids[g.random((n, k)) < drop] = g.choice([-1, E, 2 ** 31 - 1, -2 ** 31])
    return ids.astype(np.int32)


def _plan(v, torch, ids, E):
    n, k = ids.shape
    mk = lambda *s: torch.full(s, -7, dtype=torch.int32, device="cuda")
    off, order, place = mk(E + 1), mk(n * k), mk(n, k)
    v.nerf_route_plan(torch.from_numpy(ids).cuda(), E, off, order, place)
    return off, order, place


def _randn(torch, g, *shape, bf16=False, scale=1.0):
    a = torch.from_numpy((scale * g.standard_normal(shape)).astype(np.float32)).cuda()
    return a.to(_dt(torch, bf16))


def _rows(torch, t, pad):
    """The same values in rows further apart, starting at an odd element."""
    if not pad:
        return t
    big = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device="cuda")
    big[:, 1:1 + t.shape[1]] = t
    return big[:, 1:1 + t.shape[1]]


PLANS = [(1, 1, 1, 0.0), (1, 2, 8, 0.0), (63, 1, 2, 0.5), (64, 3, 5, 0.1), (1000, 2, 64, 0.0), (4096, 1, 16, 1.0),
         (4097, 1, 4096, 0.2), (5000, 4, 511, 0.3), (20011, 3, 512, 0.0), (20011, 7, 7, 0.1), (300001, 1, 1, 0.0),
         (300001, 1, 1000, 0.4), (270000, 6, 4096, 0.1), (50, 64, 3, 0.0)]


@pytest.mark.parametrize("n,k,E,drop", PLANS)
def test_plan(n, k, E, drop):
    torch = torch_cuda()
    import volume_rendering_amd as v
    say(f"plan n={n} k={k} E={E} drop={drop}")
    ids = _ids(np.random.default_rng([n, k, E]), n, k, E, drop, skew=E > 100)
    got = [host(t) for t in _plan(v, torch, ids, E)]
    flat = ids.reshape(-1).astype(np.int64)
    key = np.where((flat >= 0) & (flat < E), flat, E)
    order = np.argsort(key, kind="stable")
    place = np.empty_like(order)
    place[order] = np.arange(order.size)
    off = np.searchsorted(key[order], np.arange(E + 1))
    assert np.array_equal(got[0], off) and np.array_equal(got[1], order)
    assert np.array_equal(got[2], place.reshape(n, k))


def test_plan_of_no_pairs_and_of_empty_experts():
    torch = torch_cuda()
    import volume_rendering_amd as v
    off, _, _ = _plan(v, torch, np.zeros((0, 2), np.int32), 5)
    assert not host(off).any()
    off, order, _ = _plan(v, torch, np.full((3, 2), 9, np.int32), 5)  # no such expert: all dropped
    assert not host(off).any() and np.array_equal(host(order), np.arange(6))


ROWS = [(1, 1, 1, 1, 0.0), (1, 2, 4, 64, 0.0), (33, 3, 5, 7, 0.3), (65, 2, 3, 63, 0.2), (40, 4, 6, 333, 0.5),
        (17, 1, 2, 512, 1.0), (9, 2, 3, 1030, 0.2), (260, 8, 16, 24, 0.1)]


@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("n,k,E,d,drop", ROWS)
def test_rows_there_and_back(n, k, E, d, drop, bf16, pad):
    torch = torch_cuda()
    import volume_rendering_amd as v
    say(f"rows n={n} k={k} E={E} d={d} drop={drop} bf16={bf16} pad={pad}")
    g = np.random.default_rng([n, k, E, d])
    S, dt = n * k, _dt(torch, bf16)
    off, order, place = _plan(v, torch, _ids(g, n, k, E, drop), E)
    ho, hp = host(off), host(place)
    live = int(ho[-1])
    x, y = _randn(torch, g, n, d, bf16=bf16), _randn(torch, g, S, d, bf16=bf16)
    dout = _randn(torch, g, n, d, bf16=bf16)
    w = torch.from_numpy(g.random((n, k)).astype(np.float32)).cuda()
    y[live:] = float("nan")  # rows and weights of pairs without an expert do not matter
    hw = host(w)
    w[torch.from_numpy(hp).cuda() >= live] = float("nan")

    rows = torch.full((S, d), 3.0, dtype=dt, device="cuda")
    v.nerf_route_gather(_rows(torch, x, pad), off, place, rows)
    assert np.array_equal(_f64(rows), R.gather(_f64(x), ho, hp))

    for weights, hweights in ((w, hw), (None, None)):
        out = _rows(torch, torch.zeros((n, d), dtype=dt, device="cuda"), pad)
        v.nerf_route_combine(y, off, place, weights, out)
        want = R.combine(_f64(y), ho, hp, hweights)
        mag = R.combine(np.abs(_f64(y)), ho, hp, hweights)
        tol = (k + 1) * U32 * mag + (UB * np.abs(want) if bf16 else 0)
        assert np.all(np.abs(_f64(out) - want) <= tol)
        if pad:  # nothing beside the rows is written
            assert torch.isnan(out._base[:, 0]).all() and torch.isnan(out._base[:, d + 1:]).all()

        dy, dw = torch.full((S, d), 5.0, dtype=dt, device="cuda"), torch.full((n, k), 5.0, device="cuda")
        v.nerf_route_combine_grad(_rows(torch, dout, pad), y, off, place, weights, dy, dw)
        wy, ww = R.combine_grad(_f64(dout), _f64(y), ho, hp, hweights)
        _, mw = R.combine_grad(np.abs(_f64(dout)), np.abs(_f64(y)), ho, hp)
        assert np.all(np.abs(_f64(dy) - wy) <= U32 * np.abs(wy) + (UB * np.abs(wy) if bf16 else 0))
        assert np.all(np.abs(_f64(dw) - ww) <= (d + 1) * U32 * mw)
        v.nerf_route_combine_grad(_rows(torch, dout, pad), y, off, place, weights, dy)  # no weight gradient asked for
        assert np.all(np.abs(_f64(dy) - wy) <= U32 * np.abs(wy) + (UB * np.abs(wy) if bf16 else 0))


# slots = n k; (n, k, E, d_in, d_out, drop)
LAYERS = [(1, 1, 1, 1, 1, 0.0), (1, 2, 16, 64, 96, 0.0), (1, 2, 16, 1024, 512, 0.0), (5, 3, 4, 63, 32, 0.3),
          (100, 1, 60, 63, 32, 0.4), (300, 2, 3, 64, 64, 0.0), (300, 2, 3, 256, 256, 0.2), (257, 1, 1, 319, 255, 0.0),
          (500, 2, 5, 130, 33, 0.1), (64, 1, 4, 8, 8, 1.0), (700, 3, 2, 40, 520, 0.1), (130, 1, 64, 16, 16, 0.0),
          (1500, 2, 4, 128, 192, 0.1), (2500, 2, 3, 72, 96, 0.05), (2100, 1, 100, 32, 24, 0.0), (900, 2, 2, 264, 384, 0.0),
          (25000, 2, 3, 264, 264, 0.05), (20000, 2, 5, 264, 272, 0.0), (3000, 3, 70, 104, 128, 0.1)]


@pytest.mark.parametrize("through_order", [False, True])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("case", LAYERS)
def test_expert_layer_and_its_gradient(case, bf16, through_order):
    torch = torch_cuda()
    import volume_rendering_amd as v
    n, k, E, d_in, d_out, drop = case
    say(f"expert layer {case} bf16={bf16} order={through_order}")
    g = np.random.default_rng(list(case[:5]))
    S, dt = n * k, _dt(torch, bf16)
    off, order, place = _plan(v, torch, _ids(g, n, k, E, drop, skew=n > 200), E)
    ho, hord = host(off), host(order)
    live = int(ho[-1])
    pad = 3 if n % 2 else 0
    rows = hord // k if through_order else None
    x = torch.relu(_randn(torch, g, n if through_order else S, d_in, bf16=bf16))
    if not through_order:
        x[live:] = float("nan")  # rows without an expert do not matter
    w, b = _randn(torch, g, E, d_out, d_in, bf16=bf16, scale=d_in ** -0.5), _randn(torch, g, E, d_out)
    dz = _randn(torch, g, S, d_out, bf16=bf16)
    dz[live:] = float("nan")
    hx, hw, hb, hz = np.nan_to_num(_f64(x)), _f64(w), _f64(b), np.nan_to_num(_f64(dz))
    kw = dict(order=order, k=k) if through_order else {}
    xs = _rows(torch, x, pad)

    for relu, bias in ((False, b), (True, b), (False, None)):
        y = _rows(torch, torch.full((S, d_out), 4.0, dtype=dt, device="cuda"), pad)
        v.nerf_expert_linear(xs, w, bias, off, y, relu=relu, **kw)
        want = R.expert_linear(hx, hw, hb if bias is not None else None, ho, S, rows, relu)
        mag = R.expert_linear(np.abs(hx), np.abs(hw), np.abs(hb) if bias is not None else None, ho, S, rows)
        err = np.abs(_f64(y) - want)
        assert np.all(err <= (d_in + 2) * U32 * mag + (UB * np.abs(want) if bf16 else 0)), err.max()
        assert not _f64(y)[live:].any()
        if pad:
            assert torch.isnan(y._base[:, 0]).all() and torch.isnan(y._base[:, d_out + 1:]).all()

    counts = np.zeros((E, 1))
    counts[:, 0] = np.diff(ho)
    for relu_x in (False, True):
        dx = torch.full((S, d_in), 4.0, dtype=dt, device="cuda")
        dw, db = torch.full(w.shape, 4.0, device="cuda"), torch.full((E, d_out), 4.0, device="cuda")
        v.nerf_expert_linear_grad(_rows(torch, dz, pad), xs, w, off, dx, dw, db, relu_x=relu_x, **kw)
        want = R.expert_linear_grad(hz, hx, hw, ho, rows, relu_x)
        mag = R.expert_linear_grad(np.abs(hz), np.abs(hx), np.abs(hw), ho, rows)
        err = np.abs(_f64(dx) - want[0])
        assert np.all(err <= (d_out + 2) * U32 * mag[0] + (UB * np.abs(want[0]) if bf16 else 0)), err.max()
        assert not _f64(dx)[live:].any()
        assert np.all(np.abs(_f64(dw) - want[1]) <= (counts[:, :, None] + 2) * U32 * mag[1])
        assert np.all(np.abs(_f64(db) - want[2]) <= (counts + 2) * U32 * mag[2])
    # each gradient alone, and again: the same bits
    dx2, dw2 = torch.empty_like(dx), torch.empty_like(dw)
    v.nerf_expert_linear_grad(_rows(torch, dz, pad), xs, w, off, dx=dx2, relu_x=True, **kw)
    v.nerf_expert_linear_grad(_rows(torch, dz, pad), xs, w, off, dweight=dw2, **kw)
    assert torch.equal(dx2, dx) and torch.equal(dw2, dw)


NARROW = [(1, 3), (3, 1), (2, 9), (7, 5), (5, 70), (8, 67), (9, 40), (66, 3), (71, 8), (129, 135), (133, 66), (65, 129)]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("d_in,d_out", NARROW)
def test_widths_around_a_piece(d_in, d_out, bf16):
    """Rows shorter than 16 bytes, and ones whose last piece is nearly empty or
    nearly full, in groups long enough for the widest tiles."""
    test_expert_layer_and_its_gradient((350, 2, 3, d_in, d_out, 0.1), bf16, True)


def test_gradient_of_no_slots_is_zero():
    torch = torch_cuda()
    import volume_rendering_amd as v
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    w = torch.ones((3, 5, 7), device="cuda")
    dw, db = torch.ones_like(w), torch.ones((3, 5), device="cuda")
    v.nerf_expert_linear_grad(torch.empty((0, 5), device="cuda"), torch.empty((0, 7), device="cuda"), w, off,
                              dweight=dw, dbias=db)
    assert not host(dw).any() and not host(db).any()


@pytest.mark.parametrize("bf16", [False, True])
def test_nan_and_inf_stay_in_their_rows(bf16):
    """A row that holds NaN or infinity spoils itself and its expert's weight
    gradient, and nothing of its tile neighbours or of other experts."""
    torch = torch_cuda()
    import volume_rendering_amd as v
    say(f"nan rows bf16={bf16}")
    g = np.random.default_rng([77])
    n, E, d = 90, 3, 72
    off, order, place = _plan(v, torch, (np.arange(n) % E).astype(np.int32)[:, None], E)
    x, w = _randn(torch, g, n, d, bf16=bf16), _randn(torch, g, E, d, d, bf16=bf16)
    dz = _randn(torch, g, n, d, bf16=bf16)
    y0, y1, dw0, dw1 = (torch.empty(s, dtype=t, device="cuda") for s, t in
                        (((n, d), x.dtype), ((n, d), x.dtype), ((E, d, d), torch.float32),
                         ((E, d, d), torch.float32)))
    v.nerf_expert_linear(x, w, None, off, y0, relu=True)
    v.nerf_expert_linear_grad(dz, x, w, off, dweight=dw0)
    x[35, 5], x[36, 0] = float("nan"), float("inf")  # expert 1
    v.nerf_expert_linear(x, w, None, off, y1, relu=True)
    v.nerf_expert_linear_grad(dz, x, w, off, dweight=dw1)
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    keep[35:37] = False
    assert torch.equal(y0[keep], y1[keep]) and torch.isnan(y1[35]).all()
    assert not torch.isfinite(y1[36]).all()
    assert torch.equal(dw0[[0, 2]], dw1[[0, 2]]) and torch.isnan(dw1[1][:, 5]).all()


def test_gradients_match_differences():
    """Directional derivatives of the oracle's float64 loss through the whole
    pass, against the GPU's float32 gradients.  The differences are good to
    1e-7; each GPU gradient element is within (terms + 2) 2^-23 of its terms'
    magnitude, at most three layers deep: 1e-4 of |g| |v| is far above both."""
    torch = torch_cuda()
    import volume_rendering_amd as v
    g = np.random.default_rng([5, 8])
    n, k, E, d, hid = 40, 2, 5, 24, 20
    S = n * k
    ids = _ids(g, n, k, E, 0.15)
    off, order, place = _plan(v, torch, ids, E)
    ho, hp, hord = host(off), host(place), host(order)
    f32 = lambda *s: g.standard_normal(s).astype(np.float32)
    x, w1, b1, w2, b2, wt, c = f32(n, d), f32(E, hid, d), f32(E, hid), f32(E, d, hid), f32(E, d), f32(n, k), f32(n, d)

    def loss(x, w1, b1, w2, b2, wt):
        h = R.expert_linear(x, w1, b1, ho, S, hord // k, relu=True)
        return float((c * R.combine(R.expert_linear(h, w2, b2, ho, S), ho, hp, wt)).sum())

    D = lambda a: torch.from_numpy(a).cuda()
    E_ = lambda *s: torch.empty(s, device="cuda")
    tx, tw1, tb1, tw2, tb2, twt, tc = map(D, (x, w1, b1, w2, b2, wt, c))
    h, y = E_(S, hid), E_(S, d)
    v.nerf_expert_linear(tx, tw1, tb1, off, h, order=order, k=k, relu=True)
    v.nerf_expert_linear(h, tw2, tb2, off, y)
    dy, dwt, dz1, drows, dx = E_(S, d), E_(n, k), E_(S, hid), E_(S, d), E_(n, d)
    gw1, gb1, gw2, gb2 = E_(E, hid, d), E_(E, hid), E_(E, d, hid), E_(E, d)
    v.nerf_route_combine_grad(tc, y, off, place, twt, dy, dwt)
    v.nerf_expert_linear_grad(dy, h, tw2, off, dz1, gw2, gb2, relu_x=True)
    v.nerf_expert_linear_grad(dz1, tx, tw1, off, drows, gw1, gb1, order=order, k=k)
    v.nerf_route_combine(drows, off, place, None, dx)
    args = [a.astype(np.float64) for a in (x, w1, b1, w2, b2, wt)]
    for i, gr in enumerate((dx, gw1, gb1, gw2, gb2, dwt)):
        gr = _f64(gr)
        dirn = g.standard_normal(gr.shape)
        step = 1e-6
        up, dn = (loss(*args[:i], args[i] + s * step * dirn, *args[i + 1:]) for s in (1, -1))
        want = (up - dn) / (2 * step)
        assert abs((gr * dirn).sum() - want) <= 1e-4 * np.linalg.norm(gr) * np.linalg.norm(dirn), i


def test_rows_beyond_32_bit_offsets():
    """Tensors of more than 2^31 elements (and more than 4 GiB): the last rows."""
    torch = torch_cuda()
    import volume_rendering_amd as v
    say("rows beyond 32-bit offsets")
    n, d, E = 70001, 32768, 2
    ids = torch.zeros((n, 1), dtype=torch.int32, device="cuda")
    ids[n // 2:] = 1
    off, order, place = (torch.empty(s, dtype=torch.int32, device="cuda") for s in ((E + 1,), (n,), (n, 1)))
    v.nerf_route_plan(ids, E, off, order, place)
    x = torch.zeros((n, d), dtype=torch.bfloat16, device="cuda")
    x[:, 0], x[-3:] = 1.0, torch.arange(d, device="cuda").remainder(199).to(torch.bfloat16)
    rows = torch.empty_like(x)
    v.nerf_route_gather(x, off, place, rows)
    assert torch.equal(rows[-5:], x[-5:]) and torch.equal(rows[:3], x[:3])
    out = torch.empty_like(x)
    v.nerf_route_combine(rows, off, place, torch.full((n, 1), 2.0, device="cuda"), out)
    assert torch.equal(out[-5:].float(), 2 * x[-5:].float())
    del out
    # wide rows in (through the order too), wide rows out
    w = torch.zeros((E, 32, d), dtype=torch.bfloat16, device="cuda")
    w[1, 3] = 1.0
    for kw in ({}, dict(order=order, k=1)):
        y = torch.empty((n, 32), dtype=torch.bfloat16, device="cuda")
        v.nerf_expert_linear(x, w, None, off, y, **kw)
        want = x[-4:].double().sum(1)
        assert torch.all((y[-4:, 3].double() - want).abs() <= want * (2 ** -8 + d * 2.0 ** -23))
        assert not y[-4:, 4:].any() and not y[0].any()
    z = torch.zeros((n, 32), dtype=torch.bfloat16, device="cuda")
    z[:, 3] = 1.0
    v.nerf_expert_linear_grad(z, x, w, off, dx=rows)
    assert (rows[-1] == 1).all() and not rows[0].any()
    wt = torch.ones((E, d, 32), dtype=torch.bfloat16, device="cuda")
    v.nerf_expert_linear(z, wt, None, off, rows)
    assert (rows[-1] == 1).all() and (rows[0] == 1).all()


def test_another_stream_and_graph_replay():
    """A pass on a stream of its own equals the default stream's, and captured
    in a HIP graph it gives the same bits on every replay with new inputs."""
    torch = torch_cuda()
    import volume_rendering_amd as v
    g = np.random.default_rng([6, 8])
    n, k, E, d = 6000, 2, 8, 64
    S = n * k
    batches = [(_ids(g, n, k, E, 0.1), _randn(torch, g, n, d, bf16=True)) for _ in range(3)]
    w = _randn(torch, g, E, d, d, bf16=True)
    wt = torch.full((n, k), 0.5, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")

    def buffers():
        bf = dict(dtype=torch.bfloat16, device="cuda")
        return dict(ids=torch.zeros((n, k), **i32), x=torch.zeros((n, d), **bf), off=torch.empty(E + 1, **i32),
                    order=torch.empty(S, **i32), place=torch.empty((n, k), **i32), y=torch.empty((S, d), **bf),
                    out=torch.empty((n, d), **bf), dw=torch.empty((E, d, d), device="cuda"),
                    ws=torch.empty(max(1, v.nerf_route_workspace_size(n, k, E)), dtype=torch.uint8, device="cuda"),
                    ws2=torch.empty(max(1, v.nerf_expert_linear_grad_workspace_size(S, E, d, d)), dtype=torch.uint8,
                                    device="cuda"))

    def one(b):
        v.nerf_route_plan(b["ids"], E, b["off"], b["order"], b["place"], workspace=b["ws"])
        v.nerf_expert_linear(b["x"], w, None, b["off"], b["y"], order=b["order"], k=k, relu=True)
        v.nerf_route_combine(b["y"], b["off"], b["place"], wt, b["out"])
        v.nerf_expert_linear_grad(b["y"], b["x"], w, b["off"], dweight=b["dw"], order=b["order"], k=k,
                                  workspace=b["ws2"])

    eager = []
    for ids, x in batches:
        b = buffers()
        b["ids"].copy_(torch.from_numpy(ids))
        b["x"].copy_(x)
        one(b)
        eager.append((b["out"].clone(), b["dw"].clone()))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    b = buffers()
    b["ids"].copy_(torch.from_numpy(batches[0][0]))
    b["x"].copy_(batches[0][1])
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        one(b)
    s.synchronize()
    assert torch.equal(b["out"], eager[0][0]) and torch.equal(b["dw"], eager[0][1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one(b)
    for rep in range(2):
        for i, (ids, x) in enumerate(batches):
            b["ids"].copy_(torch.from_numpy(ids))
            b["x"].copy_(x)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(b["out"], eager[i][0]) and torch.equal(b["dw"], eager[i][1]), (rep, i)
            (x.float() @ x.float().t()).sum().item()  # eager work in between
