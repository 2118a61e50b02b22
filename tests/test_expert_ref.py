"""The 64-bit statement of SwiGLU's gradient in expert_ref.py, which the kernel
is held to, against differences."""
import numpy as np
import pytest

import expert_ref as ex

INF = float("inf")


@pytest.mark.parametrize("clamp", [INF, 1.0])
def test_gradient_against_differences(clamp):
    """The statement in 64 bits that the kernel is held to, against central differences of y."""
    rng = np.random.default_rng(6)
    n, hidden, d = 3, 16, 1e-5
    h, w = rng.standard_normal((n, 2 * hidden)) * 2, rng.random(n)
    h = np.where(np.abs(np.abs(h) - clamp) < 0.01, 0.5, h)  # away from the clamp's kink
    dy = rng.standard_normal((n, hidden))
    dh, dw, _, _ = ex.swiglu_backward(dy, h, w, clamp)

    def loss(h, w):
        return (ex.swiglu(h, w, clamp)[0] * dy).sum(1)

    for c in range(2 * hidden):
        step = np.zeros((n, 2 * hidden))
        step[:, c] = d
        assert np.allclose((loss(h + step, w) - loss(h - step, w)) / (2 * d), dh[:, c], atol=1e-8, rtol=1e-6)
    assert np.allclose((loss(h, w + d) - loss(h, w - d)) / (2 * d), dw, atol=1e-8, rtol=1e-6)
