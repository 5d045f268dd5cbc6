"""Pins of the streaming-field oracle (no GPU): gradients against central
differences, and the recurrence against the compositing oracle."""
import numpy as np
import pytest

from oracle import composite
from oracle import streaming as O


def _differences(f, x, step=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        old = x[i]
        x[i] = old + step
        up = f()
        x[i] = old - step
        down = f()
        x[i] = old
        g[i] = (up - down) / (2 * step)
    return g


@pytest.mark.parametrize("renorm", [True, False])
def test_gate_gradient(renorm):
    g = np.random.default_rng(0)
    z, dw = g.standard_normal((4, 7)), g.standard_normal((4, 3))
    z[1, 2] = z[2, 0] = -np.inf
    ids, w = O.gate(z, 3, renorm)
    fin = np.where(np.isfinite(z), z, -1e9)
    num = _differences(lambda: float((O.gate(fin, 3, renorm)[1] * dw).sum()), fin)
    assert np.allclose(O.gate_grad(dw, z, ids, w, 7, renorm), num, atol=1e-8)


@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("mix", [False, True])
@pytest.mark.parametrize("gates", [1, 2, 6])
def test_scan_gradient(gates, mix, reverse):
    g = np.random.default_rng(1)
    off, d = [0, 3, 3, 8], 6
    a, x, h0 = g.random((8, gates)), g.standard_normal((8, d)), g.standard_normal((3, d))
    dh, dl = g.standard_normal((8, d)), g.standard_normal((3, d))

    def total():
        h, last = O.scan(a, x, off, h0, reverse, mix)
        return float((h * dh).sum() + (last * dl).sum())

    h, _ = O.scan(a, x, off, h0, reverse, mix)
    da, dx, dh0 = O.scan_grad(dh, dl, a, x, h, h0, off, reverse, mix)
    for got, arg in ((da, a), (dx, x), (dh0, h0)):
        assert np.allclose(got, _differences(total, arg), atol=1e-7)


def test_reverse_mix_is_alpha_compositing():
    g = np.random.default_rng(2)
    R, N = 3, 12
    raw = g.standard_normal((R, N, 4))
    z = np.sort(g.random((R, N)) * 4 + 2, axis=1)
    d = g.standard_normal((R, 3))
    rgb, _, _, w = composite.volume_render(raw, z, d)
    # weights are T_i alpha_i, T the product of 1 - alpha of the samples in front
    T, alpha = np.ones(R), np.zeros((R, N))
    for i in range(N):
        alpha[:, i] = np.where(T > 0, w[:, i] / np.where(T > 0, T, 1.0), 0.0)
        T = T * (1.0 - alpha[:, i])
    colour = 1.0 / (1.0 + np.exp(-raw[..., :3]))
    off = np.arange(R + 1) * N
    _, last = O.scan((1.0 - alpha).reshape(-1, 1), colour.reshape(-1, 3), off, reverse=True, mix=True)
    assert np.allclose(last, rgb, atol=1e-6)


def test_layer_of_one_expert_is_the_network():
    g = np.random.default_rng(3)
    w1, w2, x = g.standard_normal((1, 5, 4)), g.standard_normal((1, 3, 5)), g.standard_normal((2, 4))
    out = O.routed_mlp(x, np.zeros((2, 1), int), None, w1, None, w2, None, "relu")
    assert np.allclose(out, np.maximum(x @ w1[0].T, 0) @ w2[0].T)
    assert not O.routed_mlp(x, np.full((2, 1), -1), None, w1, None, w2, None, "relu").any()


def test_clip():
    norm, out = O.grad_clip([np.array([3.0]), np.array([[4.0]])], 1.0)
    assert norm == 5.0 and np.allclose(out[0], 0.6) and np.allclose(out[1], 0.8)
    assert O.grad_clip([np.array([3.0])], 7.0)[1][0][0] == 3.0
