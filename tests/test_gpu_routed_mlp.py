"""The whole routed layer for a few samples on the GPU against the float64
oracle (oracle/streaming.py), and against the calls that it stands for.

Bounds, with u = 2^-24 half a step of float32 and |.| over magnitudes: a float32
sum of n terms is off by at most (n + 2) u times the sum of magnitudes.
  hidden   e1 = (d_in + 2) u (|W1||x| + |b1|); ReLU keeps it; z1 sigmoid(z1) z2
           has slopes up to 1.1 |z2| and |z1|, and six more roundings
  output   e2 = |W2| e1 + (hidden + 10) u (|W2||h| + |b2|), summed with |w| over
           the choices, and k + 1 more roundings
bfloat16 results are off by another 2^-8 of themselves.
"""
import numpy as np
import pytest

from oracle import streaming as O
from tests.gpu_util import host, say, torch_cuda

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _f64(t):
    torch = torch_cuda()
    torch.cuda.synchronize()
    return t.detach().float().cpu().numpy().astype(np.float64)


def _bound(x, ids, weights, w1, b1, w2, b2, act):
    E, d_out, hid = w2.shape
    out = np.zeros((x.shape[0], d_out))
    for t in range(x.shape[0]):
        for j in range(ids.shape[1]):
            e = ids[t, j]
            if not 0 <= e < E:
                continue
            m1 = np.abs(w1[e]) @ np.abs(x[t]) + (0.0 if b1 is None else np.abs(b1[e]))
            z = w1[e] @ x[t] + (0.0 if b1 is None else b1[e])
            e1 = (x.shape[1] + 2) * U * m1
            if act == "gated":
                s = np.abs(z[:hid] / (1.0 + np.exp(-z[:hid])))
                h = s * np.abs(z[hid:])
                e1 = 1.1 * (np.abs(z[hid:]) + e1[hid:]) * e1[:hid] + s * e1[hid:] + 6 * U * h
            else:
                h = np.abs(np.maximum(z, 0.0) if act == "relu" else z)
            m2 = np.abs(w2[e]) @ h + (0.0 if b2 is None else np.abs(b2[e]))
            w = 1.0 if weights is None else abs(float(weights[t, j]))
            out[t] += w * (np.abs(w2[e]) @ e1 + (hid + 10 + ids.shape[1] + 1) * U * m2)
    return out


def _case(torch, g, n, k, E, d_in, hid, d_out, act, bf16, drop, pad):
    dt = torch.bfloat16 if bf16 else torch.float32
    put = lambda a, t=torch.float32: torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda().to(t)
    up = 2 * hid if act == "gated" else hid
    ids = g.integers(0, E, (n, k))
    ids[g.random((n, k)) < drop] = g.choice([-1, E, 2 ** 31 - 1, -2 ** 31])
    x = put(g.standard_normal((n, d_in)), dt)
    if pad:
        big = torch.full((n, d_in + pad), float("nan"), dtype=dt, device="cuda")
        big[:, 1:1 + d_in] = x
        x = big[:, 1:1 + d_in]
    w1 = put(g.standard_normal((E, up, d_in)) / np.sqrt(d_in), dt)
    w2 = put(g.standard_normal((E, d_out, hid)) / np.sqrt(hid), dt)
    b1, b2 = put(0.3 * g.standard_normal((E, up))), put(0.3 * g.standard_normal((E, d_out)))
    w = put(g.random((n, k)))
    tid = torch.from_numpy(ids.astype(np.int32)).cuda()
    w[(tid < 0) | (tid >= E)] = float("nan")  # weights of pairs without an expert do not matter
    return x, tid, w, w1, b1, w2, b2


# n, k, experts, d_in, hidden, d_out, act, drop
SIZES = [(1, 1, 1, 1, 1, 1, "relu", 0.0), (1, 2, 16, 96, 200, 64, "relu", 0.0), (3, 2, 4, 63, 32, 4, "none", 0.3),
         (5, 3, 7, 17, 33, 9, "gated", 0.2), (64, 1, 300, 63, 32, 4, "relu", 0.3), (16, 4, 64, 128, 72, 40, "gated", 0.0),
         (8, 64, 3, 40, 24, 5, "relu", 0.1), (512, 1, 1, 24, 40, 33, "relu", 0.0), (100, 5, 2, 130, 65, 12, "gated", 0.1),
         (7, 2, 5, 1025, 519, 513, "relu", 0.0), (2, 2, 3, 256, 2049, 1031, "gated", 0.0), (4, 1, 9, 8, 7, 3, "none", 1.0),
         (31, 3, 6, 3, 600, 2, "relu", 0.0), (2, 1, 2, 70, 1100, 1024, "none", 0.0),
         # rows of 24, 71 and 4100 weights, many columns, sorted pairs of few samples an expert
         (9, 2, 70, 24, 71, 30, "gated", 0.1), (40, 3, 90, 71, 23, 200, "relu", 0.1), (3, 1, 4, 40, 16, 4103, "none", 0.0),
         (2, 1, 3, 4100, 9, 6, "gated", 0.0), (150, 1, 100, 33, 20, 515, "gated", 0.2), (1, 5, 40, 16, 40, 1500, "relu", 0.0),
         # 65 pairs and more an expert
         (300, 1, 2, 40, 70, 64, "gated", 0.0), (256, 2, 3, 16, 130, 70, "relu", 0.2)]


@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("case", range(len(SIZES)))
def test_layer(case, bf16, pad):
    torch = torch_cuda()
    import volume_rendering_amd as v
    n, k, E, d_in, hid, d_out, act, drop = SIZES[case]
    say(f"layer n={n} k={k} E={E} {d_in}->{hid}->{d_out} {act} bf16={bf16} pad={pad}")
    g = np.random.default_rng([case, 2])
    x, ids, w, w1, b1, w2, b2 = _case(torch, g, n, k, E, d_in, hid, d_out, act, bf16, drop, pad)
    if case % 4 == 3:
        b1 = b2 = None
    if case % 5 == 2:
        w = None
    out = torch.full((n, d_out + pad), 7.0, dtype=x.dtype, device="cuda")
    view = out[:, 1:1 + d_out] if pad else out
    v.nerf_routed_mlp(x, ids, w, w1, b1, w2, b2, view, act=act)
    a = [None if t is None else _f64(t) for t in (x, w, w1, b1, w2, b2)]
    ref = O.routed_mlp(a[0], host(ids), a[1], *a[2:], act)
    tol = _bound(a[0], host(ids), a[1], *a[2:], act)
    tol = tol + (2.0 ** -8 if bf16 else U) * (np.abs(ref) + tol)
    got = _f64(view)
    worst = np.max(np.abs(got - ref) / (tol + 1e-30))
    say(f"  {worst:.2f} of the bound")
    assert worst <= 1.0
    if pad:
        assert (_f64(out)[:, 0] == 7.0).all() and (_f64(out)[:, 1 + d_out:] == 7.0).all()


def test_layer_stands_for_the_separate_calls():
    """Plan, two expert layers and the weighted sum give the same to bfloat16's rounding of the hidden layer."""
    torch = torch_cuda()
    import volume_rendering_amd as v
    say("layer against the separate calls")
    g = np.random.default_rng(9)
    n, k, E, d_in, hid, d_out = 40, 3, 12, 96, 128, 64
    for bf16 in (False, True):
        x, ids, w, w1, b1, w2, b2 = _case(torch, g, n, k, E, d_in, hid, d_out, "relu", bf16, 0.1, 0)
        out = torch.empty((n, d_out), dtype=x.dtype, device="cuda")
        v.nerf_routed_mlp(x, ids, w, w1, b1, w2, b2, out)
        i32 = dict(dtype=torch.int32, device="cuda")
        off, order, place = torch.empty(E + 1, **i32), torch.empty(n * k, **i32), torch.empty((n, k), **i32)
        h, y = (torch.empty((n * k, c), dtype=x.dtype, device="cuda") for c in (hid, d_out))
        sep = torch.empty_like(out)
        v.nerf_route_plan(ids, E, off, order, place)
        v.nerf_expert_linear(x, w1, b1, off, h, order=order, k=k, relu=True)
        v.nerf_expert_linear(h, w2, b2, off, y)
        v.nerf_route_combine(y, off, place, w, sep)
        a = [_f64(t) for t in (x, w, w1, b1, w2, b2)]
        tol = 2 * _bound(a[0], host(ids), *a[1:], "relu") + 1e-6
        if bf16:  # rounded: the hidden values and y (2^-8 each), both outputs
            hid_abs = O.routed_mlp(np.abs(a[0]), host(ids), np.nan_to_num(np.abs(a[1])), *[np.abs(t) for t in a[2:]],
                                   "relu")
            tol = tol + 2.0 ** -8 * (4 * hid_abs)
        assert (np.abs(_f64(out) - _f64(sep)) <= tol).all()


def test_one_bad_weight_reaches_only_its_samples():
    torch = torch_cuda()
    import volume_rendering_amd as v
    say("layer NaN")
    g = np.random.default_rng(3)
    x, ids, w, w1, b1, w2, b2 = _case(torch, g, 20, 2, 6, 50, 30, 20, "relu", False, 0.0, 0)
    w1[4] = float("nan")
    x[7] = float("inf")
    out = torch.empty((20, 20), device="cuda")
    v.nerf_routed_mlp(x, ids, w, w1, b1, w2, b2, out)
    bad = (host(ids) == 4).any(1)
    bad[7] = True
    fin = np.isfinite(_f64(out)).all(1)
    assert fin[~bad].all() and not fin[bad & (np.arange(20) != 7)].any()


def test_repeats_streams_graphs_and_workspaces():
    torch = torch_cuda()
    import volume_rendering_amd as v
    say("layer repeats")
    g = np.random.default_rng(4)
    args = _case(torch, g, 9, 3, 20, 200, 300, 100, "gated", True, 0.1, 0)
    x = args[0]
    size = v.nerf_routed_mlp_workspace_size(9, 3, 300, 100)
    guard = torch.full((size + 64,), 171, dtype=torch.uint8, device="cuda")

    def call(ws=None):
        out = torch.empty((9, 100), dtype=x.dtype, device="cuda")
        v.nerf_routed_mlp(*args, out, act="gated", workspace=ws)
        return out

    want = call()
    assert torch.equal(call(guard[:size]), want) and (guard[size:] == 171).all()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = call(guard[:size])
    s.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = call(guard[:size])
    for i in range(3):
        x.mul_(-1.5)
        args[1].copy_((args[1] + 7) % 20)  # other experts
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held, call())


def test_weights_of_more_than_2_to_31_elements():
    torch = torch_cuda()
    import volume_rendering_amd as v
    say("layer of 2^31 weights and more")
    E, d_in, hid, d_out = 4096, 1024, 520, 16
    w1 = torch.zeros((E, hid, d_in), dtype=torch.bfloat16, device="cuda")
    w2 = torch.zeros((E, d_out, hid), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    w1[-1] = torch.randn((hid, d_in), generator=g, device="cuda").to(torch.bfloat16)
    w2[-1] = torch.randn((d_out, hid), generator=g, device="cuda").to(torch.bfloat16)
    x = torch.randn((2, d_in), generator=g, device="cuda").to(torch.bfloat16)
    ids = torch.tensor([[4095], [0]], dtype=torch.int32, device="cuda")
    out = torch.empty((2, d_out), dtype=torch.bfloat16, device="cuda")
    v.nerf_routed_mlp(x, ids, None, w1, None, w2, None, out)
    h = np.maximum(_f64(w1[-1]) @ _f64(x)[0], 0.0)
    ref = _f64(w2[-1]) @ h
    mag = np.abs(_f64(w2[-1])) @ (np.abs(_f64(w1[-1])) @ np.abs(_f64(x)[0]))
    assert (np.abs(_f64(out)[0] - ref) <= 2.0 ** -8 * np.abs(ref) + 1600 * U * mag).all() and not _f64(out)[1].any()
