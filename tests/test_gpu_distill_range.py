"""Distillation where the size of the logits, and not their differences, could
spoil the result: rows shifted far from zero, rows masked with the type's lowest
value, temperatures far from one.  Against the float64 oracle, with bounds that
know only the differences within a row.

With u = 2^-23, R the largest difference of scaled logits z within a row (among
those whose share is above e^-120), Rt the teacher's, K the entries kept: an
exponent is one difference and two products, each rounded by at most half a u of
it: 1.5 R u; 2^x adds 2 u; the sum of exponentials is a chain of at most V / 64 +
24 additions.  From a saved log-sum-exp below 64 its own rounding and that of its
product with T add at most half of 64 u each.  So q is off by at most (2 (1.5 R +
2) + V / 64 + 24 + 64 + 8) u of itself, the teacher's p by (4 Rt + 2 K + 8) u,
bfloat16 results by another 2^-8 of themselves.
"""
import numpy as np
import pytest

from oracle import routed as R
from tests.gpu_util import say, torch_cuda

pytestmark = pytest.mark.gpu

U = 2.0 ** -23
LOWEST = {False: -3.4028234e38, True: -3.3895314e38}


def _f64(t):
    torch = torch_cuda()
    torch.cuda.synchronize()
    return t.detach().float().cpu().numpy().astype(np.float64)


def _run(z, t, ids, T, bf16, scale=None):
    """The rounded logits, loss, lse, the gradient of either call."""
    torch = torch_cuda()
    import volume_rendering_amd as v
    n = z.shape[0]
    x = torch.from_numpy(z.astype(np.float32)).cuda().to(torch.bfloat16 if bf16 else torch.float32)
    tl, ti = torch.from_numpy(t.astype(np.float32)).cuda(), torch.from_numpy(ids.astype(np.int32)).cuda()
    sc = None if scale is None else torch.from_numpy(scale.astype(np.float32)).cuda()
    loss, lse = torch.full((n,), 9.0, device="cuda"), torch.full((n,), 9.0, device="cuda")
    both, alone = torch.full_like(x, 9.0), torch.full_like(x, 9.0)
    v.nerf_distill_topk(x, tl, ti, T, loss, lse=lse, grad=both, row_scale=sc)
    v.nerf_distill_topk_grad(x, tl, ti, T, lse, alone, row_scale=sc)
    return _f64(x), _f64(tl), _f64(loss), _f64(lse), _f64(both), _f64(alone)


def _check_gradient(hx, ht, ids, T, bf16, scale, grads):
    n, V = hx.shape
    K = ids.shape[1]
    _, _, want = R.distill(hx, ht, ids, T, scale)
    z = hx / T
    d = z - z.max(1, keepdims=True)
    q = np.exp(d)
    q /= q.sum(1, keepdims=True)
    spread = np.where(d > -120, -d, 0).max(1, keepdims=True)
    rt = (ht.max(1) - ht.min(1))[:, None] / T
    s = T * (np.ones(n) if scale is None else scale)[:, None]
    p = np.abs(q - want / s)  # the teacher's mass at each class
    tol = s * U * (q * (2 * (1.5 * spread + 2) + V / 64 + 24 + 64 + 8) + (p + q) * (4 * rt + 2 * K + 8)) + 1e-37
    if bf16:
        tol += 2.0 ** -8 * np.abs(want)
    for name, got in zip(("with the loss", "from lse"), grads):
        err = np.abs(got - want)
        assert np.all(err <= tol), (name, (err / tol).max())


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("V", [70, 6000, 40001])
@pytest.mark.parametrize("shift", [0.0, 60.0, -70.0, 1e4, -1e6])
def test_gradients_of_shifted_rows(shift, V, bf16):
    say(f"distill gradients shift={shift} V={V} bf16={bf16}")
    g = np.random.default_rng([21, V, int(abs(shift))])
    n, K, T = 5, 9, 2.0
    z = shift + 3 * g.standard_normal((n, V))
    z[1] = shift  # all alike
    z[2, 1:] = LOWEST[bf16]  # all but one masked
    t = 3 * g.standard_normal((n, K)) - shift
    ids = np.stack([g.permutation(V)[:K] for _ in range(n)])
    scale = 0.5 + g.random(n).astype(np.float32).astype(np.float64)
    hx, ht, _, _, *grads = _run(z, t, ids, T, bf16, scale)
    _check_gradient(hx, ht, ids, T, bf16, scale, grads)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T", [0.5, 1.0, 4.0])
@pytest.mark.parametrize("V", [33, 5000, 50001])
def test_gradients_of_rows_of_the_lowest_value(V, T, bf16):
    """Every class masked with the type's lowest value: q is 1 / V."""
    say(f"distill gradients lowest V={V} T={T} bf16={bf16}")
    g = np.random.default_rng([22, V])
    n, K = 3, 5
    z = np.full((n, V), LOWEST[bf16])
    t, ids = g.standard_normal((n, K)), np.stack([g.permutation(V)[:K] for _ in range(n)])
    hx, ht, _, _, *grads = _run(z, t, ids, T, bf16)
    _check_gradient(hx, ht, ids, T, bf16, None, grads)


def _loss_tolerance(hx, ht, ids, T):
    """loss = T sum p (T (ln p + ln sum) - (s - max)): an entry's p is off by (4 min(Rt,
    120) + 2 K + 8) u of itself (below e^-120 it is nothing), the logarithm of the sum
    by the sum's relative error, the rest by 8 u of the terms."""
    n, V = hx.shape
    K = ids.shape[1]
    m = hx.max(1, keepdims=True)
    d = (hx - m) / T
    spread = np.where(d > -120, -d, 0).max(1, keepdims=True)
    t = (ht - ht.max(1, keepdims=True)) / T
    p = np.exp(t)
    p /= p.sum(1, keepdims=True)
    logp = np.where(p > 0, np.log(np.where(p > 0, p, 1)), 0)
    logs = np.log(np.exp(d).sum(1, keepdims=True))
    size = np.take_along_axis(m - hx, ids, 1) + T * (np.abs(logp) + logs)
    rel = 4 * np.minimum(-t.min(1, keepdims=True), 120) + 2 * K + 16
    return T * U * (p * (size * rel + T * (2 * (1.5 * spread + 2) + V / 64 + 24))).sum(1) + 1e-44


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T", [0.25, 0.5, 1.0, 2.0])
@pytest.mark.parametrize("V", [70, 6000, 40001])
def test_teacher_mass_on_a_class_of_the_lowest_value(V, T, bf16):
    """The loss of such a class is p T 3.4e38, which is finite."""
    say(f"distill mass on the lowest V={V} T={T} bf16={bf16}")
    g = np.random.default_rng([23, V])
    n, K = 4, 8
    z, t = 2 * g.standard_normal((n, V)), g.standard_normal((n, K))
    ids = np.stack([g.permutation(V)[:K] for _ in range(n)])
    z[np.arange(n), ids[:, 3]] = LOWEST[bf16]
    t[:, 3] -= 3.0 * T  # (its p is a few hundredths)
    hx, ht, loss, _, *_ = _run(z, t, ids, T, bf16)
    want, _, _ = R.distill(hx, ht, ids, T)
    assert np.all(np.abs(loss - want) <= _loss_tolerance(hx, ht, ids, T)), (loss, want)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T", [1e-45, 1e-40, 1e-30, 1e-10, 1e4, 1e37, 3e38])
@pytest.mark.parametrize("V", [70, 9000])
def test_temperatures_far_from_one(V, T, bf16):
    """Down to the smallest positive one both distributions are single classes; at
    the largest they are even, and the loss may pass the type's range."""
    say(f"distill T={T} V={V} bf16={bf16}")
    T = float(np.float32(T))
    g = np.random.default_rng([24, V])
    n, K = 4, 7
    z, t = 2 * g.standard_normal((n, V)), g.standard_normal((n, K)).astype(np.float32).astype(np.float64)
    ids = np.stack([g.permutation(V)[:K] for _ in range(n)])
    z[0, :9] = 30.0  # equal largest classes
    hx, ht, loss, _, both, alone = _run(z, t, ids, T, bf16)
    want, _, grad = R.distill(hx, ht, ids, T)
    inside = want < 3e38
    assert np.all(np.abs(loss - want)[inside] <= _loss_tolerance(hx, ht, ids, T)[inside]), (loss, want)
    assert np.all(loss[~inside] >= 3e38)
    d = (hx - hx.max(1, keepdims=True)) / T
    q = np.exp(d)
    q /= q.sum(1, keepdims=True)
    p = np.abs(q - grad / T)
    # (exponents above -120 count; a temperature below 2^-126 is itself rounded to few bits in 1 / T)
    spread = np.where(d > -120, -d, 0).max(1, keepdims=True)
    rt = np.minimum((ht.max(1) - ht.min(1))[:, None] / T, 120)
    tol = T * U * (q * (2 * (1.5 * spread + 2) + V / 64 + 24 + 64 + 8) + (p + q) * (4 * rt + 2 * K + 8)) + 1e-37
    if bf16:
        tol += 2.0 ** -8 * np.abs(grad)
    for got in (both, alone):
        assert np.all(np.abs(got - grad) <= tol)
