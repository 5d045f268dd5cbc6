"""The gated linear recurrence at the ends of its range: infinite inputs, states
and gradients behind gates whose products leave float32, and sequences of very
uneven lengths; against the float64 oracle (oracle/streaming.py), within the
bounds of test_gpu_scan.py."""
import numpy as np
import pytest

from oracle import streaming as O
from tests.gpu_util import say, torch_cuda
from tests.test_gpu_scan import HALF, _bounds, _f64, _offsets, _put
from tests.test_gpu_scan import _check as check_scan

pytestmark = pytest.mark.gpu


def _kinds(what, got, ref):
    """NaN for NaN, each infinity for itself, a number for a number, in the rows of sequences."""
    for name, kind in (("NaN", np.isnan), ("inf", np.isposinf), ("-inf", np.isneginf)):
        wrong = kind(got) != kind(ref)
        assert not wrong.any(), f"{what}: {name} {kind(got).sum()} for {kind(ref).sum()}, {wrong.sum()} elements differ"


# lengths, d, gates, reverse, mix, size of the gates
INFINITE = [
    ([4100], 5, 5, False, False, 0.4),              # chunks
    ([3000, 0, 2500], 70, 70, True, False, 1e-3),
    ([5000, 37], 130, 1, True, True, 1e-7),         # (a run's own product underflows)
    ([200, 130, 64], 16, 1, False, True, 1e-3),     # four and eight waves
    ([120, 200, 0, 65], 256, 256, True, False, 0.05),
    ([600, 511], 257, 257, False, False, 1e-7),
    ([18] * 50, 96, 96, False, True, 1e-6),         # single waves
    ([60] * 300, 24, 3, True, False, 1e-4),
    ([3, 4, 2, 4], 40, 8, False, False, 1e-30),     # walked alone
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", range(len(INFINITE)))
def test_infinities_stay_infinite_behind_small_gates(case, dtype):
    """a_t s with an infinite s is infinite for every a_t but 0, however far back s became so."""
    torch = torch_cuda()
    import volume_rendering_amd as v
    lens, d, gates, reverse, mix, size = INFINITE[case]
    say(f"scan infinities case={case} {dtype}")
    g = np.random.default_rng([case, 3])
    off = _offsets(g, lens)
    rows, n = int(off[-1]), len(lens)
    a = size * (0.5 + 0.5 * g.random((rows, gates))) * np.where(g.random((rows, gates)) < 0.2, -1.0, 1.0)
    a[g.random(a.shape) < 0.002] = 0.0              # (NaN from there on)
    x, h0 = g.standard_normal((rows, d)), g.standard_normal((n, d))
    hit = g.random((rows, d)) < 0.3 / max(lens)
    x[hit] = np.where(g.random(hit.sum()) < 0.5, np.inf, -np.inf)
    h0[:, ::3] = np.inf
    h0[:, 1::6] = -np.inf
    ta, tx, th0 = _put(a, "f32"), _put(x, dtype), _put(h0, "f32")
    a, x = _f64(ta), _f64(tx)
    toff = torch.from_numpy(off.astype(np.int32)).cuda()
    h, last = torch.empty_like(tx), torch.empty((n, d), device="cuda")
    v.nerf_scan(ta, tx, h, h0=th0, h_last=last, offsets=toff, reverse=reverse, mix=mix)
    with np.errstate(invalid="ignore"):
        ref, ref_last = O.scan(a, x, off, _f64(th0), reverse, mix)
    hh = _f64(h)
    assert np.isposinf(ref).any() and np.isneginf(ref).any() and np.isfinite(ref).any()
    _kinds("h", hh, ref)
    _kinds("h_last", _f64(last), ref_last)
    fin = np.isfinite(ref)
    A = np.repeat(a, d // gates, axis=1)
    with np.errstate(invalid="ignore", over="ignore"):
        b = (1.0 - A) * x if mix else x
        _, E, _ = _bounds(a, np.where(np.isfinite(b), b, 0.0), off, np.where(np.isfinite(h0), h0, 0.0), reverse)
    # (a finite state has finite terms only: after an infinite one a sequence has no finite state)
    hh, ref, E = hh[fin], ref[fin], E[fin]
    assert (np.abs(hh - ref) <= E + HALF[dtype] * (np.abs(ref) + E)).all()

    # the gradient: infinities in dh and dh_last, and finite states
    dh, dl = g.standard_normal((rows, d)), g.standard_normal((n, d))
    hit = g.random((rows, d)) < 0.3 / max(lens)
    dh[hit] = np.where(g.random(hit.sum()) < 0.5, np.inf, -np.inf)
    dl[:, ::3] = -np.inf
    hs, xs = g.standard_normal((rows, d)), g.standard_normal((rows, d))
    tdh, tdl, ths, txs = _put(dh, dtype), _put(dl, "f32"), _put(hs, dtype), _put(xs, dtype)
    da = torch.empty((rows, gates), device="cuda")
    dx, dh0 = torch.empty_like(txs), torch.empty((n, d), device="cuda")
    v.nerf_scan_grad(tdh, ta, txs if mix else None, ths, da, dx, dh_last=tdl, dh0=dh0, offsets=toff, reverse=reverse,
                     mix=mix)
    with np.errstate(invalid="ignore"):
        rda, rdx, rdh0 = O.scan_grad(_f64(tdh), _f64(tdl), a, _f64(txs), _f64(ths), None, off, reverse, mix)
    assert np.isposinf(rdx).any() and np.isneginf(rdx).any()
    _kinds("dx", _f64(dx), rdx)
    _kinds("dh0", _f64(dh0), rdh0)
    _kinds("da", _f64(da), rda)


def _uneven(n, long, at, short, seed):
    lens = np.random.default_rng(seed).integers(0, short + 1, n)
    lens[at] = long
    return [int(v) for v in lens]


# lengths, d, gates, reverse, mix, type, gates' type: one long sequence among many short ones
UNEVEN = [
    (_uneven(10000, 30000, 5000, 1, 1), 4, 4, False, True, "f32", "f32"),
    (_uneven(301, 32768, 0, 1, 2), 64, 64, True, False, "bf16", "f32"),
    (_uneven(301, 9000, 300, 1, 3), 24, 3, False, True, "f32", "f32"),
    (_uneven(40, 12000, 17, 3, 4), 130, 1, True, True, "bf16", "bf16"),
    (_uneven(20000, 3000, 19999, 2, 5), 6, 1, True, False, "f32", "f32"),
]


@pytest.mark.parametrize("case", range(len(UNEVEN)))
def test_very_uneven_lengths(case):
    check_scan(300 + case, UNEVEN[case][:5], *UNEVEN[case][5:], 0)
