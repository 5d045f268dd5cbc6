"""The few-sample routed layer on each of its paths: pairs sorted by every
workgroup (up to 64) or by a kernel in front, layers by dot products (up to two
pairs per expert on average) or by matrix products; against the float64 oracle
(oracle/streaming.py)."""
import numpy as np
import pytest

from oracle import streaming as O
from tests.gpu_util import host, say, torch_cuda
from tests.test_gpu_routed_mlp import _bound, _case, _f64
from tests.test_gpu_routed_mlp_range import PATHS, _check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("act", ["relu", "gated"])
@pytest.mark.parametrize("share", [1.0, 0.5])
@pytest.mark.parametrize("n,k,E", [(512, 1, 300), (60, 1, 64), (256, 2, 400)])
def test_most_pairs_on_one_expert(n, k, E, share, act, bf16):
    """The average over the experts says little: all or half the pairs are one expert's."""
    torch = torch_cuda()
    import volume_rendering_amd as v
    say(f"layer collapsed n={n} k={k} E={E} share={share} {act} bf16={bf16}")
    g = np.random.default_rng([n, k])
    x, ids, w, w1, b1, w2, b2 = _case(torch, g, n, k, E, 40, 70, 33, act, bf16, 0.0, 0)
    one = torch.from_numpy(g.random((n, k)) < share).cuda()
    ids[one] = E - 2
    out = torch.empty((n, 33), dtype=x.dtype, device="cuda")
    v.nerf_routed_mlp(x, ids, w, w1, b1, w2, b2, out, act=act)
    a = _f64(x), host(ids), _f64(w), _f64(w1), _f64(b1), _f64(w2), _f64(b2)
    _check(_f64(out), O.routed_mlp(*a, act), bf16, _bound(*a, act))


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("path", PATHS)
def test_one_bad_weight_reaches_only_its_samples(path, bf16):
    torch = torch_cuda()
    import volume_rendering_amd as v
    n, k, E = PATHS[path]
    say(f"layer {path} NaN bf16={bf16}")
    x, ids, w, w1, b1, w2, b2 = _case(torch, np.random.default_rng(6), n, k, E, 50, 30, 20, "relu", bf16, 0.1, 0)
    w1[2] = float("nan")
    x[5] = float("nan")
    out = torch.empty((n, 20), dtype=x.dtype, device="cuda")
    v.nerf_routed_mlp(x, ids, w, w1, b1, w2, b2, out)
    i = host(ids)
    bad = (i == 2).any(1)
    bad[5] = ((i[5] >= 0) & (i[5] < E)).any()
    got = _f64(out)
    assert np.isfinite(got[~bad]).all() and np.isnan(got[bad]).all() and bad.any() and not bad.all()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("act", ["relu", "gated"])
@pytest.mark.parametrize("path", PATHS)
def test_repeats_streams_graphs_and_workspaces(path, act, bf16):
    """Odd widths, so that the workspace's last byte is one that the call writes."""
    torch = torch_cuda()
    import volume_rendering_amd as v
    n, k, E = PATHS[path]
    say(f"layer repeats {path} {act} bf16={bf16}")
    args = _case(torch, np.random.default_rng(4), n, k, E, 37, 71, 101, act, bf16, 0.0, 0)
    x, ids = args[:2]
    size = v.nerf_routed_mlp_workspace_size(n, k, 71, 101)
    guard = torch.full((size + 64,), 171, dtype=torch.uint8, device="cuda")

    def call(ws=None):
        out = torch.empty((n, 101), dtype=x.dtype, device="cuda")
        v.nerf_routed_mlp(*args, out, act=act, workspace=ws)
        return out

    want = call()
    assert torch.equal(call(guard[:size]), want) and (guard[size:] == 171).all()
    if "matrix" in path:
        assert (guard[size - 16:size] != 171).any()  # (the outputs per pair end there)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = call(guard[:size])
    s.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = call(guard[:size])
    for _ in range(3):
        x.mul_(-1.5)
        ids.copy_((ids + 1) % E)
        held.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held, call()) and (guard[size:] == 171).all()
