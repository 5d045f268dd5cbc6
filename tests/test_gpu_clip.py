"""The norm of a list of gradients and their clipping on the GPU against
float64 (oracle/streaming.py).

Bounds.  Squares and sums are float64 (2^-53 a term: nothing here), so the norm
is off by its one rounding to float32, 2^-24 of it; a clipped gradient by the
factor's rounding and the product's, 2 x 2^-24, and bfloat16 by 2^-8 more.
"""
import numpy as np
import pytest

from oracle import streaming as O
from tests.gpu_util import say, torch_cuda

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _f64(t):
    torch = torch_cuda()
    torch.cuda.synchronize()
    return t.detach().float().cpu().numpy().astype(np.float64)


def _make(torch, sizes, seed=0, scale=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for i, (n, bf16, odd) in enumerate(sizes):
        t = torch.randn(n + odd, generator=gen, device="cuda") * scale * 10.0 ** (i % 4 - 2)
        out.append(t.to(torch.bfloat16 if bf16 else torch.float32)[odd:])  # (odd: starts at an odd element)
    return out


LISTS = {
    "one": [(1, False, 0)],
    "odd": [(1, True, 1), (7, False, 1), (0, False, 0), (333, True, 1), (8192, False, 0), (8193, False, 1), (16384, True, 1),
            (70001, True, 0), (5, False, 0)],
    "many": [(37 * i % 5000, i % 3 == 0, i % 2) for i in range(150)],
    "large": [(20_000_003, False, 1), (50_000_001, True, 1), (3, False, 0)],
    "groups": [(200_000, i % 2 == 0, 0) for i in range(200)],  # more partial sums than one workgroup's share
}


@pytest.mark.parametrize("name", sorted(LISTS))
def test_norm_and_clip(name):
    torch = torch_cuda()
    import volume_rendering_amd as v
    say(f"clip {name}")
    grads = _make(torch, LISTS[name])
    norm = torch.full((1,), 7.0, device="cuda")
    lst = v.nerf_tensor_list(grads)
    v.nerf_grad_norm(lst, norm)
    ref = O.grad_norm([_f64(t) for t in grads])
    assert abs(float(norm) - ref) <= 1.001 * U * ref
    for max_norm in (0.5 * ref, 0.0, 2.0 * ref):
        outs = [torch.full_like(t, 7.0) for t in grads]
        norm.fill_(7.0)
        v.nerf_grad_clip(v.nerf_tensor_list(grads, outs), max_norm, norm)
        assert abs(float(norm) - ref) <= 1.001 * U * ref
        f = 1.0 if ref <= max_norm else max_norm / ref
        for t, o in zip(grads, outs):
            want = t.double() * f
            tol = 2.01 * U * want.abs() + (2.0 ** -8 if t.dtype == torch.bfloat16 else 0.0) * want.abs() + 1e-45
            assert bool(((o.double() - want).abs() <= tol).all())
    # in place: the same as beside
    outs = [torch.empty_like(t) for t in grads]
    v.nerf_grad_clip(v.nerf_tensor_list(grads, outs), 0.25 * ref, norm)
    before = [t.clone() for t in grads]
    v.nerf_grad_clip(lst, 4.0 * ref, norm)
    assert all(torch.equal(p, q) for p, q in zip(grads, before))  # a factor of 1
    v.nerf_grad_clip(lst, 0.25 * ref, norm)
    assert all(torch.equal(p, q) for p, q in zip(grads, outs))


def test_neighbours_of_a_tensor_are_left_alone():
    torch = torch_cuda()
    import volume_rendering_amd as v
    say("clip neighbours")
    for dt, n in ((torch.float32, 8191), (torch.bfloat16, 16385), (torch.bfloat16, 3), (torch.float32, 2)):
        buf = torch.full((n + 20,), 5.0, dtype=dt, device="cuda")
        norm = torch.empty(1, device="cuda")
        v.nerf_grad_clip(v.nerf_tensor_list([buf[9:9 + n]]), 1.0, norm)
        b = _f64(buf)
        assert (b[:9] == 5.0).all() and (b[9 + n:] == 5.0).all() and (b[9:9 + n] < 5.0).all()


def test_nothing_to_sum():
    torch = torch_cuda()
    import volume_rendering_amd as v
    say("clip nothing")
    e = torch.empty(0, device="cuda")
    for lst in (v.nerf_tensor_list([]), v.nerf_tensor_list([e, e.to(torch.bfloat16)])):
        for call in (v.nerf_grad_norm, lambda l, n: v.nerf_grad_clip(l, 1.0, n)):
            norm = torch.full((1,), 7.0, device="cuda")
            call(lst, norm)
            assert float(norm) == 0.0
    z = torch.zeros(1000, device="cuda")
    v.nerf_grad_clip(v.nerf_tensor_list([z]), 0.0, norm)
    assert float(norm) == 0.0 and not z.any()


def test_values_at_the_ends_of_the_type():
    torch = torch_cuda()
    import volume_rendering_amd as v
    say("clip extremes")
    norm = torch.empty(1, device="cuda")
    big = torch.full((100,), 3e37, device="cuda")       # squares beyond float32
    v.nerf_grad_clip(v.nerf_tensor_list([big]), 1.0, norm)
    assert abs(float(norm) - 3e38) <= 3e38 * 2 * U and np.allclose(_f64(big), 0.1, rtol=1e-6)
    huge = torch.full((1000,), 3e38, device="cuda")      # a norm beyond float32
    v.nerf_grad_clip(v.nerf_tensor_list([huge]), 1.0, norm)
    assert float(norm) == float("inf") and np.allclose(_f64(huge), 1000 ** -0.5, rtol=1e-6)
    tiny = torch.full((10000,), 1e-30, device="cuda")    # squares below float32
    v.nerf_grad_norm(v.nerf_tensor_list([tiny]), norm)
    assert abs(float(norm) - 1e-28) <= 1e-28 * 2 * U
    mixed = torch.cat([torch.full((1,), 1e4, device="cuda"), torch.full((1 << 20,), 1e-2, device="cuda")])
    v.nerf_grad_norm(v.nerf_tensor_list([mixed]), norm)
    ref = O.grad_norm([_f64(mixed)])
    assert abs(float(norm) - ref) <= 1.001 * U * ref
    bad = torch.ones(50, device="cuda")
    bad[3] = float("nan")
    other = torch.ones(50, device="cuda")
    v.nerf_grad_clip(v.nerf_tensor_list([bad, other]), 1.0, norm)
    assert np.isnan(float(norm)) and np.isnan(_f64(bad)).all() and np.isnan(_f64(other)).all()
    bad = torch.ones(50, device="cuda")
    bad[3] = float("inf")
    v.nerf_grad_clip(v.nerf_tensor_list([bad]), 1.0, norm)
    b = _f64(bad)
    assert float(norm) == float("inf") and np.isnan(b[3]) and not np.delete(b, 3).any()


def test_repeats_streams_graphs_and_workspaces():
    torch = torch_cuda()
    import volume_rendering_amd as v
    say("clip repeats")
    for name in ("odd", "many", "groups"):
        grads = _make(torch, LISTS[name], 3)
        outs = [torch.empty_like(t) for t in grads]
        lst, norm = v.nerf_tensor_list(grads, outs), torch.empty(1, device="cuda")
        size = v.nerf_grad_norm_workspace_size(lst)
        guard = torch.full((size + 64,), 171, dtype=torch.uint8, device="cuda")
        v.nerf_grad_clip(lst, 1.0, norm)
        want = [norm.clone()] + [t.clone() for t in outs]

        def same():
            torch.cuda.synchronize()
            return all(torch.equal(p, q) for p, q in zip([norm] + outs, want))

        for t in [norm] + outs:
            t.zero_()
        v.nerf_grad_clip(lst, 1.0, norm, workspace=guard[:size])
        assert same() and (guard[size:] == 171).all()
        with pytest.raises(v.NerfError, match="workspace"):
            v.nerf_grad_clip(lst, 1.0, norm, workspace=guard[:size - 8])
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            v.nerf_grad_clip(lst, 1.0, norm, workspace=guard[:size])
        s.synchronize()
        assert same()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            v.nerf_grad_clip(lst, 1.0, norm, workspace=guard[:size])
        for i in range(3):
            for t in grads:
                t.mul_(-2.0)
            graph.replay()
            torch.cuda.synchronize()
            got = [norm.clone()] + [t.clone() for t in outs]
            v.nerf_grad_clip(lst, 1.0, norm)
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip([norm] + outs, got))


def test_gradients_of_more_than_2_to_31_elements():
    torch = torch_cuda()
    import volume_rendering_amd as v
    say("clip of 2^31 elements and more")
    t = torch.zeros((1 << 31) + 100, dtype=torch.bfloat16, device="cuda")
    t[-7:] = 3.0
    t[0] = 4.0
    norm = torch.empty(1, device="cuda")
    v.nerf_grad_clip(v.nerf_tensor_list([t]), 1.0, norm)
    ref = (7 * 9 + 16) ** 0.5
    assert abs(float(norm) - ref) <= 1.001 * U * ref
    assert (np.abs(_f64(t[-7:]) - 3.0 / ref) <= 2.0 ** -8).all() and abs(float(t[0]) - 4.0 / ref) <= 2.0 ** -8
    assert not t[1:-7].any()
