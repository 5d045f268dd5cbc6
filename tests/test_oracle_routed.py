"""The float64 oracle of routed fields and distillation: gradients against
central differences, and the definitions' invariants (no GPU)."""
import numpy as np
import pytest

from oracle import routed as R


def _case(seed, n, k, E, d, drop):
    g = np.random.default_rng([seed, 51])
    ids = g.integers(0, E, (n, k))
    ids[g.random((n, k)) < drop] = -1
    return g, ids, R.plan(ids, E)


@pytest.mark.parametrize("n,k,E,drop", [(1, 1, 1, 0.0), (7, 3, 5, 0.3), (20, 2, 40, 0.0), (4, 2, 3, 1.0)])
def test_plan_is_a_stable_sort(n, k, E, drop):
    _, ids, (off, order, place) = _case(1, n, k, E, 4, drop)
    flat = ids.reshape(-1)
    assert sorted(order) == list(range(n * k)) and np.array_equal(order[place.reshape(-1)], np.arange(n * k))
    for e in range(E):
        own = order[off[e]:off[e + 1]]
        assert np.all(flat[own] == e) and np.all(np.diff(own) > 0)
    assert off[0] == 0 and off[-1] == (flat >= 0).sum()


def _directional(f, x, v, h=1e-6):
    return (f(x + h * v) - f(x - h * v)) / (2 * h)


def test_routed_pass_gradients_match_differences():
    """gather -> linear -> ReLU -> linear -> weighted sum, one scalar loss."""
    g, ids, (off, order, place) = _case(2, 9, 2, 4, 6, 0.2)
    n, k, E, d, hid, S = 9, 2, 4, 6, 5, 18
    x, w1, b1 = g.standard_normal((n, d)), g.standard_normal((E, hid, d)), g.standard_normal((E, hid))
    w2, b2, w = g.standard_normal((E, d, hid)), g.standard_normal((E, d)), g.random((n, k))
    c = g.standard_normal((n, d))

    def loss(x, w1, b1, w2, b2, w):
        h = R.expert_linear(R.gather(x, off, place), w1, b1, off, S, relu=True)
        return float((c * R.combine(R.expert_linear(h, w2, b2, off, S), off, place, w)).sum())

    rows = R.gather(x, off, place)
    h = R.expert_linear(rows, w1, b1, off, S, relu=True)
    y = R.expert_linear(h, w2, b2, off, S)
    dy, dw = R.combine_grad(c, y, off, place, w)
    dz1, dw2, db2 = R.expert_linear_grad(dy, h, w2, off, relu_x=True)
    drows, dw1, db1 = R.expert_linear_grad(dz1, rows, w1, off)
    dx = R.combine(drows, off, place)
    args, grads = [x, w1, b1, w2, b2, w], [dx, dw1, db1, dw2, db2, dw]
    for i in range(6):
        v = g.standard_normal(args[i].shape)
        got = float((grads[i] * v).sum())
        want = _directional(lambda a: loss(*args[:i], a, *args[i + 1:]), args[i], v)
        assert abs(got - want) <= 1e-6 * (1 + abs(want)), (i, got, want)


@pytest.mark.parametrize("T", [0.5, 1.0, 3.0])
def test_distillation_gradient_matches_differences(T):
    g = np.random.default_rng([3, 51])
    n, V, K = 5, 23, 4
    z, t = 3 * g.standard_normal((n, V)), 2 * g.standard_normal((n, K))
    ids = np.stack([g.permutation(V)[:K] for _ in range(n)])
    ids[1, 2] = -1      # padding
    ids[2] = -1         # no teacher
    ids[3, 1] = ids[3, 0]  # one class twice
    t[0, 3] = -np.inf
    scale = g.random(n)
    loss, lse, grad = R.distill(z, t, ids, T, scale)
    assert loss[2] == 0 and not grad[2].any()
    # (with one class twice, the entropy term is the entries' own)
    assert np.all(np.delete(loss, 3) >= -1e-12)
    assert np.allclose(grad.sum(1), 0, atol=1e-12)  # a shift of the logits changes nothing
    v = g.standard_normal(z.shape)
    want = _directional(lambda a: float((scale * R.distill(a, t, ids, T)[0]).sum()), z, v)
    assert abs(float((grad * v).sum()) - want) <= 1e-6 * (1 + abs(want))


def test_distillation_is_zero_at_the_teacher():
    g = np.random.default_rng([4, 51])
    t = g.standard_normal((3, 8))
    ids = np.tile(np.arange(8), (3, 1))
    loss, _, grad = R.distill(t + 2.5, t, ids, 2.0)
    assert np.allclose(loss, 0, atol=1e-13) and np.allclose(grad, 0, atol=1e-13)
