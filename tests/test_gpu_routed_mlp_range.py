"""The few-sample routed layer with infinite weights and hidden values, and hidden
values of any size, on each of its paths, against the float64 oracle
(oracle/streaming.py): a rule on the pairs per expert picks dot or matrix
products, whose bfloat16 form holds a hidden value in three parts."""
import numpy as np
import pytest

from oracle import streaming as O
from tests.gpu_util import host, say, torch_cuda
from tests.test_gpu_routed_mlp import U, _bound, _case, _f64

pytestmark = pytest.mark.gpu

# samples, choices, experts
PATHS = {"self dots": (9, 3, 20), "planned dots": (40, 3, 70), "self matrix": (20, 3, 4), "planned matrix": (60, 3, 5)}


def _put(a, bf16):
    torch = torch_cuda()
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda().to(torch.bfloat16 if bf16 else torch.float32)


def _same_kind(got, ref):
    """NaN for NaN, each infinity for itself, a number for a number."""
    return (np.isnan(got) == np.isnan(ref)) & (np.isposinf(got) == np.isposinf(ref)) & (
        np.isneginf(got) == np.isneginf(ref))


def _check(got, ref, bf16, tol=0.0):
    """`tol`: of the finite numbers, on top of the output's rounding."""
    assert _same_kind(got, ref).all(), f"{(~_same_kind(got, ref)).sum()} of {ref.size} elements"
    fin = np.isfinite(ref)
    got, ref, tol = got[fin], ref[fin], np.broadcast_to(tol, ref.shape)[fin]
    assert (np.abs(got - ref) <= tol + (2.0 ** -8 if bf16 else U) * (np.abs(ref) + tol)).all()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("n,E", [(6, 3), (7, 3), (80, 40), (81, 40)])  # two pairs per expert, and one more
def test_infinite_weights(n, E, bf16):
    """Hidden values of few bits, and 0, times infinite weights: what the formula gives on either side of the rule."""
    torch = torch_cuda()
    import volume_rendering_amd as v
    say(f"layer infinite weights n={n} E={E} bf16={bf16}")
    g = np.random.default_rng([n, E])
    d_in, hid, d_out = 8, 40, 20
    x, w1 = g.integers(-3, 4, (n, d_in)), g.integers(-1, 2, (E, hid, d_in))
    w2 = g.integers(-4, 5, (E, d_out, hid)).astype(np.float64)
    w2[:, 3, 5], w2[:, 4, 2], w2[:, 5, 39] = np.inf, -np.inf, np.inf
    w2[:, 6, 7], w2[:, 6, 8] = np.inf, -np.inf
    ids = g.integers(0, E, (n, 1))
    with np.errstate(invalid="ignore"):
        ref = O.routed_mlp(x, ids, None, w1, None, w2, None, "none")
    assert np.isposinf(ref).any() and np.isneginf(ref).any() and np.isnan(ref).any()
    out = torch.empty((n, d_out), dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")
    v.nerf_routed_mlp(_put(x, bf16), torch.from_numpy(ids.astype(np.int32)).cuda(), None, _put(w1, bf16), None,
                      _put(w2, bf16), None, out, act="none")
    _check(_f64(out), ref, bf16)  # (sums of whole numbers below 2^24: exact)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("n,E", [(6, 3), (7, 3), (81, 40)])
def test_infinite_hidden_values(n, E, bf16):
    torch = torch_cuda()
    import volume_rendering_amd as v
    say(f"layer infinite hidden values n={n} E={E} bf16={bf16}")
    g = np.random.default_rng([n, E, 1])
    d_in, hid, d_out = 5, 33, 18
    x, w1 = g.integers(1, 4, (n, d_in)).astype(np.float64), g.integers(1, 3, (E, hid, d_in))
    x[::2, 1], x[1, 2] = np.inf, -np.inf
    w2 = g.integers(1, 5, (E, d_out, hid)).astype(np.float64)
    w2[:, 3] = np.inf
    w2[:, 4, 6], w2[:, 5, 7] = 0.0, -np.inf
    ids = g.integers(0, E, (n, 1))
    with np.errstate(invalid="ignore"):
        ref = O.routed_mlp(x, ids, None, w1, None, w2, None, "none")
    assert np.isposinf(ref).any() and np.isneginf(ref).any() and np.isnan(ref).any()
    out = torch.empty((n, d_out), dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")
    v.nerf_routed_mlp(_put(x, bf16), torch.from_numpy(ids.astype(np.int32)).cuda(), None, _put(w1, bf16), None,
                      _put(w2, bf16), None, out, act="none")
    _check(_f64(out), ref, bf16)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("scale", [2.0 ** -96, 2.0 ** -60, 2.0 ** 60])
@pytest.mark.parametrize("path", PATHS)
def test_hidden_values_of_any_size(path, scale, bf16):
    """Small and large hidden values keep their 24 bits (weights scaled back)."""
    torch = torch_cuda()
    import volume_rendering_amd as v
    n, k, E = PATHS[path]
    say(f"layer {path} hidden scale={scale} bf16={bf16}")
    x, ids, w, w1, _, w2, _ = _case(torch, np.random.default_rng(5), n, k, E, 40, 70, 33, "none", bf16, 0.1, 0)
    x, w2 = x * scale, w2 / scale  # (powers of two: exact)
    out = torch.empty((n, 33), dtype=x.dtype, device="cuda")
    v.nerf_routed_mlp(x, ids, w, w1, None, w2, None, out, act="none")
    a = _f64(x), host(ids), _f64(w), _f64(w1), None, _f64(w2), None
    _check(_f64(out), O.routed_mlp(*a, "none"), bf16, _bound(*a, "none"))


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("n,E", [(2, 2), (5, 2), (81, 40)])
@pytest.mark.parametrize("e", [0, 60, -60, -95, -97, -104, -109])
def test_hidden_values_keep_24_bits(e, n, E, bf16):
    """Differences of hidden values 2^e (1 + 2^-10 + 2^-20), 2^e (1 + 2^-10) and 2^e: powers of two, so exact."""
    torch = torch_cuda()
    import volume_rendering_amd as v
    say(f"layer 24 bits e={e} n={n} E={E} bf16={bf16}")
    a, b = 2.0 ** (e // 2), 2.0 ** (e - e // 2)
    x = np.tile([a, a * 2.0 ** -5, a * 2.0 ** -10], (n, 1))
    w1 = np.tile([[b, b * 2.0 ** -5, b * 2.0 ** -10], [b, b * 2.0 ** -5, 0.0], [b, 0.0, 0.0]], (E, 1, 1))
    w = 2.0 ** min(-e, 100)
    w2 = np.tile([[w, -w, 0.0], [0.0, w, -w], [w, 0.0, -w]], (E, 1, 1))
    out = torch.empty((n, 3), dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")
    ids = torch.arange(n, dtype=torch.int32, device="cuda").view(n, 1) % E
    v.nerf_routed_mlp(_put(x, bf16), ids, None, _put(w1, bf16), None, _put(w2, bf16), None, out, act="none")
    want = np.array([2.0 ** -20, 2.0 ** -10, 2.0 ** -10 + 2.0 ** -20]) * (w * 2.0 ** e)
    want[2] = want[1] if bf16 else want[2]  # (to eight bits)
    assert (_f64(out) == want).all()
