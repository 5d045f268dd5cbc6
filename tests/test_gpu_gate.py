"""The gate of a routed field and its gradient on the GPU against the float64
oracle (oracle/streaming.py).

Bounds, with u = 2^-24 half a step of float32.  A weight e^(z - m) / sum: the
difference is off by |z - m| u, which the exponential turns into a relative
error; exponential, division and store add at most 4 u, and the sum of E terms
E u: w (E + |z - m| + 8) u, doubled for the other terms' differences.  The
gradient's terms w dw and p S: each the same, times their magnitudes, and k + 2
additions.  bfloat16 results are off by another 2^-8 of themselves.
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


def _logits(g, n, E, bf16, masked):
    torch = torch_cuda()
    z = (2.0 * g.standard_normal((n, E))).astype(np.float32)
    z[g.random((n, E)) < masked] = -np.inf
    if masked and n > 1:
        z[n // 2] = -np.inf  # a row without an expert
    return torch.from_numpy(z).cuda().to(torch.bfloat16 if bf16 else torch.float32)


def _wide(t, pad):
    """The same values in rows further apart, starting at an odd element."""
    torch = torch_cuda()
    if not pad:
        return t
    big = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device="cuda")
    big[:, 1:1 + t.shape[1]] = t
    return big[:, 1:1 + t.shape[1]]


SIZES = [(1, 1, 1), (1, 16, 2), (3, 2, 2), (5, 5, 3), (300, 8, 8), (257, 16, 2), (130, 17, 4), (100, 33, 6), (70, 64, 8),
         (65, 65, 5), (64, 100, 7), (33, 256, 64), (21, 257, 9), (9, 513, 2), (17, 1000, 8), (5, 1025, 33), (6, 2049, 4),
         (7, 4096, 8), (3, 4095, 64), (20001, 16, 2)]


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("n,E,k", SIZES)
def test_gate_and_gradient(n, E, k, bf16, renorm):
    torch = torch_cuda()
    import volume_rendering_amd as v
    say(f"gate n={n} E={E} k={k} bf16={bf16} renorm={renorm}")
    g = np.random.default_rng([n, E, k])
    masked, pad = (0.3 if (n + E) % 2 else 0.0), 3 if E % 2 else 0
    t = _logits(g, n, E, bf16, masked)
    z = _f64(t)
    ids = torch.full((n, k), -9, dtype=torch.int32, device="cuda")
    w = torch.full((n, k), 7.0, device="cuda")
    v.nerf_route_gate(_wide(t, pad), ids, w, renorm=renorm)
    some = slice(0, n) if n <= 500 else slice(n - 300, n)  # (the oracle goes row by row)
    ri, rw = O.gate(z[some], k, renorm)
    assert np.array_equal(host(ids)[some], ri)
    with np.errstate(invalid="ignore"):
        top = np.where(ri >= 0, np.take_along_axis(z[some], np.maximum(ri, 0), 1), 0.0)
        far = np.where(ri >= 0, np.abs(top - top[:, :1]), 0.0)
    assert (np.abs(_f64(w)[some] - rw) <= 2 * U * rw * (E + far.max() + 8) + 1e-37).all()
    if n > 500:
        ref_i, ref_w = torch.sort(t.float(), dim=1, descending=True, stable=True)[1][:, :k].to(torch.int32), None
        assert torch.equal(torch.where(ids < 0, ref_i, ids), ref_i)

    # the gradient at the weights that came back; choices without an expert hold NaN
    dw = g.standard_normal((n, k)).astype(np.float32)
    hi, hw = host(ids), _f64(w)
    tdw, tw = torch.from_numpy(dw).cuda(), w.clone()
    tdw[ids < 0] = float("nan")
    tw[ids < 0] = float("nan")
    out = torch.full((n, E + pad), 7.0, dtype=t.dtype, device="cuda")
    view = out[:, 1:1 + E] if pad else out
    v.nerf_route_gate_grad(tdw, None if renorm else _wide(t, pad), ids, tw, view, renorm=renorm)
    ref = O.gate_grad(dw[some], z[some], hi[some], hw[some], E, renorm)
    live = hi[some] >= 0
    wd = np.where(live, np.abs(hw[some] * dw[some]), 0.0)
    S = wd.sum(1, keepdims=True)
    mag = np.zeros(ref.shape)
    rows = np.repeat(np.arange(ref.shape[0]), k).reshape(-1, k)
    np.add.at(mag, (rows[live], hi[some][live]), (wd + np.abs(hw[some]) * S)[live])
    if not renorm:
        with np.errstate(invalid="ignore"):
            m = z[some].max(1, keepdims=True)
            e = np.where(np.isneginf(z[some]), 0.0, np.exp(z[some] - np.where(np.isneginf(m), 0.0, m)))
        mag += e / np.maximum(e.sum(1, keepdims=True), 1e-300) * S
    tol = 2 * U * (E + k + 24 + far.max()) * mag
    tol = tol + (2.0 ** -8 if bf16 else U) * (np.abs(ref) + tol) + 1e-37
    got = _f64(view)[some]
    assert (np.abs(got - ref) <= tol).all(), np.max(np.abs(got - ref) / tol)
    if pad:
        assert (_f64(out)[:, 0] == 7.0).all() and (_f64(out)[:, 1 + E:] == 7.0).all()


@pytest.mark.parametrize("E", [7, 64, 600])
@pytest.mark.parametrize("bf16", [False, True])
def test_ties_go_to_the_lowest_expert(E, bf16):
    torch = torch_cuda()
    import volume_rendering_amd as v
    say(f"gate ties E={E} bf16={bf16}")
    g = np.random.default_rng(E)
    z = g.integers(-1, 2, (50, E)).astype(np.float32)
    z[z == 0] *= np.where(g.random((z == 0).sum()) < 0.5, -1.0, 1.0)  # 0 and -0 are equal
    t = torch.from_numpy(z).cuda().to(torch.bfloat16 if bf16 else torch.float32)
    k = min(E, 20)
    ids, w = torch.empty((50, k), dtype=torch.int32, device="cuda"), torch.empty((50, k), device="cuda")
    v.nerf_route_gate(t, ids, w)
    assert np.array_equal(host(ids), np.argsort(-z, axis=1, kind="stable")[:, :k])


@pytest.mark.parametrize("renorm", [True, False])
def test_values_at_the_ends_of_the_type(renorm):
    torch = torch_cuda()
    import volume_rendering_amd as v
    say(f"gate extremes renorm={renorm}")
    big = float(np.finfo(np.float32).max)
    rows = [[-big, -big, -big, -big], [big, big, -big, 0.0], [np.nan, 1.0, 2.0, -np.inf], [np.inf, 1.0, 2.0, 3.0],
            [-np.inf] * 4, [-np.inf, -big, -np.inf, -np.inf], [3e4, -3e4, 3e4, 1.0], [1e-40, 0.0, -1e-40, -1.0]]
    t = torch.tensor(rows, device="cuda")
    ids, w = torch.empty((8, 3), dtype=torch.int32, device="cuda"), torch.empty((8, 3), device="cuda")
    v.nerf_route_gate(t, ids, w, renorm=renorm)
    i, p = host(ids), host(w)
    assert i.tolist()[:4] == [[0, 1, 2], [0, 1, 3], [0, 2, 1], [0, 3, 2]]
    assert i[4].tolist() == [-1] * 3 and i[5].tolist() == [1, -1, -1] and i[6].tolist() == [0, 2, 3]
    assert np.allclose(p[0], 1 / 3 if renorm else 1 / 4) and np.allclose(p[1], [0.5, 0.5, 0.0])
    assert np.isnan(p[2]).all() and np.isnan(p[3]).all() and not p[4].any() and p[5].tolist() == [1.0, 0.0, 0.0]
    assert p[6].tolist() == [0.5, 0.5, 0.0]
    # gradient: rows without an expert are 0, whatever dweights hold
    dw = torch.full((8, 3), float("nan"), device="cuda")
    dw[0] = torch.tensor([1.0, 2.0, 3.0], device="cuda")
    dz = torch.full((8, 4), 7.0, device="cuda")
    v.nerf_route_gate_grad(dw, t, ids, w, dz, renorm=renorm)
    d = host(dz)
    assert not d[4].any()
    ref = O.gate_grad(host(dw)[:1], np.zeros((1, 4)), i[:1], p[:1], 4, renorm)
    assert np.allclose(d[:1], ref, atol=1e-6)


def test_repeated_and_foreign_ids_in_the_gradient():
    torch = torch_cuda()
    import volume_rendering_amd as v
    say("gate gradient ids")
    ids = torch.tensor([[2, 2, 1], [-7, 5, 0], [4, 2 ** 31 - 1, 3]], dtype=torch.int32, device="cuda")
    g = np.random.default_rng(1)
    w, dw = (torch.from_numpy(g.random((3, 3)).astype(np.float32)).cuda() for _ in range(2))
    z = torch.from_numpy(g.standard_normal((3, 5)).astype(np.float32)).cuda()
    for renorm in (True, False):
        dz = torch.empty_like(z)
        v.nerf_route_gate_grad(dw, z, ids, w, dz, renorm=renorm)
        assert np.allclose(host(dz), O.gate_grad(host(dw), host(z), host(ids), host(w), 5, renorm), atol=1e-6)


def test_streams_graphs_and_no_samples():
    torch = torch_cuda()
    import volume_rendering_amd as v
    say("gate streams")
    z = torch.randn((3000, 61), device="cuda")
    dw = torch.randn((3000, 4), device="cuda")

    def call():
        ids, w, dz = torch.empty((3000, 4), dtype=torch.int32, device="cuda"), torch.empty_like(dw), torch.empty_like(z)
        v.nerf_route_gate(z, ids, w, renorm=False)
        v.nerf_route_gate_grad(dw, z, ids, w, dz, renorm=False)
        return ids, w, dz

    want = call()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = call()
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = call()
    for _ in range(3):
        z.mul_(-1.1)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(held, call()))
    e = torch.empty((0, 5), device="cuda")
    v.nerf_route_gate(e, torch.empty((0, 2), dtype=torch.int32, device="cuda"), torch.empty((0, 2), device="cuda"))
