"""The distillation oracle on rows whose maximum is too large for ln V to be
added to it, even in 64 bits."""
import numpy as np
import pytest

from oracle import routed as R


@pytest.mark.parametrize("shift", [0.0, 1e6, -1e17, -3.4028234e38])
def test_shifted_rows_have_the_same_loss_and_gradient(shift):
    g = np.random.default_rng(5)
    V, T = 40, 2.0
    z = np.zeros((3, V))
    z[1, 7:] = -64.0  # (exact beside 1e6; lost beside the others, which are equal rows then)
    t, ids = g.standard_normal((3, 6)), np.stack([g.permutation(V)[:6] for _ in range(3)])
    seen = (z + shift) - (z + shift).max(1, keepdims=True)
    want = R.distill(seen, t, ids, T)
    got = R.distill(z + shift, t, ids, T)
    assert np.allclose(got[0], want[0], rtol=1e-12, atol=0)
    assert np.allclose(got[2], want[2], rtol=1e-12, atol=1e-14)
    assert np.allclose(got[2].sum(1), 0.0, atol=1e-13)  # T (sum q - sum p)
