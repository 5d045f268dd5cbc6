"""Distillation from a teacher's top logits on the GPU against the float64
oracle (oracle/routed.py).

Bounds, with z = logits / T, u = 2^-23: an exponential's argument is one
subtraction and one product of float32 (relative 2 u) and the hardware 2^x adds
2 u, so q's relative error is at most (2 |z - max| + 2) u plus that of the sum,
whose terms are added in chains of at most 1024 (1024 u = 2^-13 is the worst
case; chains of C classes a thread are at most classes / 64).  lse adds
(|lse| + chain) u.  A loss term is p times differences of such logarithms.
"""
import numpy as np
import pytest

from oracle import routed as R
from tests.gpu_util import host, say, torch_cuda

pytestmark = pytest.mark.gpu

U = 2.0 ** -23


def _f64(t):
    torch = torch_cuda()
    torch.cuda.synchronize()
    return t.detach().float().cpu().numpy().astype(np.float64)


def _check(n, V, K, T, bf16, logits, t_logits, t_ids, pad=0, scale=None):
    torch = torch_cuda()
    import volume_rendering_amd as v
    dt = torch.bfloat16 if bf16 else torch.float32
    z = torch.from_numpy(logits.astype(np.float32)).cuda().to(dt)
    hz = _f64(z)
    if pad:
        big = torch.full((n, V + pad), float("nan"), dtype=dt, device="cuda")
        big[:, 1:1 + V] = z
        z = big[:, 1:1 + V]
    tl, ti = torch.from_numpy(t_logits.astype(np.float32)).cuda(), torch.from_numpy(t_ids.astype(np.int32)).cuda()
    sc = None if scale is None else torch.from_numpy(scale.astype(np.float32)).cuda()
    hs = np.ones(n) if scale is None else _f64(sc)
    loss0, lse0, g0 = R.distill(hz, _f64(tl), t_ids, T, hs)

    def grad_buf():
        b = torch.full((n, V + 2 * pad), 9.0, dtype=dt, device="cuda")
        return b[:, pad:pad + V]

    loss, lse, loss1 = (torch.full((n,), 9.0, device="cuda") for _ in range(3))
    g1, g2 = grad_buf(), grad_buf()
    v.nerf_distill_topk(z, tl, ti, T, loss1)                               # loss alone
    v.nerf_distill_topk(z, tl, ti, T, loss, lse=lse, grad=g1, row_scale=sc)  # with the gradient
    v.nerf_distill_topk_grad(z, tl, ti, T, lse, g2, row_scale=sc)
    assert np.array_equal(host(loss), host(loss1), equal_nan=True)

    chain = V / 64 + 24
    fin = np.isfinite(lse0)
    with np.errstate(all="ignore"):
        zs = hz / T
        top = np.where(np.isfinite(zs), zs, -np.inf).max(1, keepdims=True)
        zmax = np.where(np.isfinite(zs) & (zs > top - 120), np.abs(zs), 0).max(1)  # (e^-120 of the largest: nothing)
        lse_tol = (2 * zmax + np.abs(lse0) + chain + 4) * U
        g_lse = _f64(lse)
        assert np.all(np.abs(g_lse - lse0)[fin] <= lse_tol[fin])
        assert np.array_equal(g_lse[~fin], lse0[~fin], equal_nan=True)
        tmax = np.where(np.isfinite(t_logits), np.abs(t_logits), 0).max(1) / T
        # sum of p (|ln p| + |ln q|) u-errors: every logarithm is below tmax, zmax + |lse| and ln K
        ltol = T * T * (lse_tol + (8 * (tmax + zmax + np.abs(lse0)) + 2 * K + 16) * U) * (1 + 2 * K * U) \
            + 8 * U * np.abs(loss0)
        gl = _f64(loss)
        ok = np.isfinite(loss0)
        assert np.all(np.abs(gl - loss0)[ok] <= np.broadcast_to(ltol, loss0.shape)[ok]), (gl, loss0)
        assert np.array_equal(gl[~ok], loss0[~ok], equal_nan=True)
        none = ~((t_ids >= 0) & (t_ids < V) & ~np.isneginf(t_logits)).any(1)
        for g in (g1, g2):
            gg = _f64(g)
            assert not gg[none].any()
            q = np.where(fin[:, None], np.exp(zs - np.where(fin, lse0, 0)[:, None]), 0)
            mass = np.abs(g0 / T / np.where(hs == 0, 1, hs)[:, None]) + 2 * q  # at least q + p
            rel = (4 * zmax[:, None] + 2 * tmax[:, None] + np.abs(np.where(fin, lse0, 0))[:, None] * 2 + 2 * chain
                   + 2 * K + 16) * U
            tol = T * np.abs(hs)[:, None] * mass * rel + (2.0 ** -8) * np.abs(g0) * bf16 + 1e-37
            good = np.isfinite(g0) & ~none[:, None]
            bad = np.abs(gg - g0)[good] > tol[good]
            assert not bad.any(), np.abs(gg - g0)[good].max()
            assert np.array_equal(np.isnan(gg[~none]), np.isnan(g0[~none]))
            if pad:
                assert (g._base[:, :pad] == 9).all() and (g._base[:, pad + V:] == 9).all()


CASES = [(1, 1, 1, 1.0), (3, 32, 4, 1.0), (5, 33, 16, 2.0), (2, 1000, 1, 0.5), (4, 2048, 64, 1.0), (3, 2049, 7, 4.0),
         (2, 5003, 100, 1.0), (1, 50001, 16, 1.0), (2, 40000, 256, 2.0), (1030, 4100, 8, 1.0), (2000, 64, 8, 2.0),
         (1025, 9001, 33, 1.0)]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("n,V,K,T", CASES)
def test_loss_and_gradient(n, V, K, T, bf16):
    say(f"distill n={n} V={V} K={K} T={T} bf16={bf16}")
    g = np.random.default_rng([n, V, K])
    logits = 3 * g.standard_normal((n, V))
    t_ids = np.stack([g.permutation(V)[:K] if V < 6000 else g.integers(0, V, K) for _ in range(n)])
    t_ids[g.random((n, K)) < 0.1] = -1
    t = 3 * g.standard_normal((n, K)) + 20
    scale = g.random(n) if n > 1 else None
    if n > 2:
        t_ids[1], scale[2] = -1, 0.0
    _check(n, V, K, T, bf16, logits, t, t_ids, pad=5 if V % 2 else 0, scale=scale)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("V", [70, 6000])
def test_masked_and_extreme_logits(V, bf16):
    """Lowest values, infinities and NaN on either side, repeated and
    impossible classes, large logits."""
    say(f"distill extremes V={V} bf16={bf16}")
    g = np.random.default_rng([9, V])
    n, K = 14, 6
    z = 2 * g.standard_normal((n, V))
    t = 2 * g.standard_normal((n, K))
    ids = np.stack([g.permutation(V)[:K] for _ in range(n)])
    z[0, ids[0, 0] - 1] = -np.inf                       # masked class without teacher mass
    z[1, ids[1, 2]] = -np.inf                           # with mass: infinite loss
    t[2, 3] = -np.inf                                   # teacher masked
    z[3, ids[3, 1]], t[3, 1] = -np.inf, -np.inf         # both masked
    z[4] = -np.inf                                      # no student
    t[5] = -np.inf                                      # no teacher mass
    z[6, 0] = np.nan
    t[7, 0] = np.nan
    z[8, V // 2] = np.inf
    lowest = -3.3895e38 if bf16 else -3.4028e38
    z[9, V // 3:] = lowest                              # masked by the type's lowest value
    ids[9] = np.arange(K)
    ids[10, 3], ids[10, 4] = ids[10, 0], ids[10, 0]     # one class three times
    ids[11, 0], ids[11, 1], ids[11, 2] = V, -5, 2 ** 31 - 1
    z[12] += 3000.0                                     # a shift
    z[13], ids[13, 1:] = 0.0, -1                        # uniform student, one entry
    _check(n, V, K, 1.0, bf16, z, t, ids, pad=1)


def test_rows_beyond_32_bit_offsets():
    torch = torch_cuda()
    import volume_rendering_amd as v
    say("distill beyond 32-bit offsets")
    n, V = 17000, 131072  # 2.2e9 elements
    z = torch.zeros((n, V), dtype=torch.bfloat16, device="cuda")
    z[-1, 7] = 3.0
    t, ids = torch.zeros((n, 2), device="cuda"), torch.full((n, 2), 5, dtype=torch.int32, device="cuda")
    ids[:, 1] = 7
    loss, lse, grad = torch.empty(n, device="cuda"), torch.empty(n, device="cuda"), torch.empty_like(z)
    v.nerf_distill_topk(z, t, ids, 1.0, loss, lse=lse, grad=grad)
    last = z[-1].double()
    want = torch.softmax(last, 0)
    want[5] -= 0.5
    want[7] -= 0.5
    assert torch.all((grad[-1].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -10 * torch.softmax(last, 0))
    assert abs(lse[0].item() - np.log(V)) < 1e-3 and abs(lse[-1].item() - torch.logsumexp(last, 0).item()) < 1e-3
    grad.zero_()
    v.nerf_distill_topk_grad(z, t, ids, 1.0, lse, grad)
    assert torch.all((grad[-1].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -10 * torch.softmax(last, 0))


def test_same_bits_and_another_stream():
    torch = torch_cuda()
    import volume_rendering_amd as v
    g = np.random.default_rng([10])
    for n, V in ((3, 30001), (1500, 5000)):
        z = torch.from_numpy(g.standard_normal((n, V)).astype(np.float32)).cuda()
        t = torch.from_numpy(g.standard_normal((n, 9)).astype(np.float32)).cuda()
        ids = torch.from_numpy(g.integers(0, V, (n, 9)).astype(np.int32)).cuda()
        outs = []
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        for stream in (torch.cuda.current_stream(), s, torch.cuda.current_stream()):
            with torch.cuda.stream(stream):
                loss, grad = torch.empty(n, device="cuda"), torch.empty_like(z)
                v.nerf_distill_topk(z, t, ids, 1.5, loss, grad=grad)
                outs.append((loss, grad))
            torch.cuda.synchronize()
        for o in outs[1:]:
            assert torch.equal(o[0], outs[0][0]) and torch.equal(o[1], outs[0][1])


@pytest.mark.parametrize("V", [500, 9001, 70000])
def test_loss_does_not_depend_on_a_shift(V):
    """Logits around 1e4 and teacher logits around -2e4: the bound knows only
    the differences within a row.  With R and Rt the largest of those, and
    u = 2^-23: a student's logarithm is off by at most (2 R + chain + 2 R + 2) u
    from the exponentials and their sum and 2 R u from its own difference, a
    teacher's by (4 Rt + K + 8) u, and the K terms of p times a difference of two
    logarithms (each at most R + Rt + ln V + ln K) add (K + 8) u of that."""
    torch = torch_cuda()
    import volume_rendering_amd as v
    say(f"distill shifted logits V={V}")
    g = np.random.default_rng([11, V])
    n, K, T = 6, 12, 2.0
    z = (1e4 + 3 * g.standard_normal((n, V))).astype(np.float32)
    t = (-2e4 + 3 * g.standard_normal((n, K))).astype(np.float32)
    ids = np.stack([g.permutation(V)[:K] for _ in range(n)]).astype(np.int32)
    want, _, _ = R.distill(z.astype(np.float64), t.astype(np.float64), ids, T)
    loss = torch.empty(n, device="cuda")
    v.nerf_distill_topk(torch.from_numpy(z).cuda(), torch.from_numpy(t).cuda(), torch.from_numpy(ids).cuda(), T, loss)
    rng_z, rng_t = (z.max(1) - z.min(1)).astype(np.float64) / T, (t.max(1) - t.min(1)).astype(np.float64) / T
    chain = V / 64 + 24
    tol = T * T * U * (6 * rng_z + chain + 4 * rng_t + K + 16
                       + (K + 8) * (rng_z + rng_t + np.log(V) + np.log(K)))
    assert np.all(np.abs(_f64(loss) - want) <= tol), (np.abs(_f64(loss) - want), tol)
