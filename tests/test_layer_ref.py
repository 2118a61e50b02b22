"""The plain references of the layer operators against differences and direct
evaluation (no GPU): what the GPU tests compare with."""
import numpy as np

import layer_ref as ref


def test_norm_gradient_is_the_difference_quotient():
    rng = np.random.default_rng(1)
    h, w, dy = rng.normal(size=(5, 48)), 1 + 0.3 * rng.normal(size=48), rng.normal(size=(5, 48))
    rstd, _ = ref.norm(h, w, 1e-6)
    dx, dw = ref.norm_backward(dy, h, w, rstd, None)
    for _ in range(6):
        u, v, t = rng.normal(size=h.shape), rng.normal(size=w.shape), 1e-5

        def loss(s):
            # norm() takes fp32 weights to 64 bits as they are, so the difference is taken in 64 bits
            hh, ww = h + s * u, w + s * v
            r = 1 / np.sqrt(np.square(hh).mean(1) + float(np.float32(1e-6)))
            return (dy * hh * r[:, None] * ww).sum()

        slope = (loss(t) - loss(-t)) / (2 * t)
        # central difference: error t^2 times a third derivative of order 10^2, and 1e-16 / t of rounding
        assert abs(slope - ((dx * u).sum() + (dw * v).sum())) < 1e-6


def test_route_gradients_are_difference_quotients():
    rng = np.random.default_rng(2)
    for softmax in (False, True):
        for normalise in (False, True):
            x = rng.normal(size=(4, 12))
            idx = np.argsort(-x, axis=1)[:, :3].astype(np.int32)
            idx[1, 2] = -1
            dw = rng.normal(size=(4, 3))
            g, _ = ref.route_backward(dw, idx, x, softmax, normalise, 2.5)
            u, t = rng.normal(size=x.shape), 1e-5

            def loss(s):
                p = ref.scores(x + s * u, softmax)
                total = 0.0
                for r in range(4):
                    e = [i for i in idx[r] if i >= 0]
                    ws = p[r, e] / (p[r, e].sum() if normalise else 1.0) * 2.5
                    total += sum(ws[i] * dw[r, i] for i in range(len(e)))
                return total

            assert abs((loss(t) - loss(-t)) / (2 * t) - (g * u).sum()) < 1e-7


def test_bit_helpers():
    assert ref.round_bf16(np.float32([1.00390625, 1.01171875, -3.0])).tolist() == [1.0, 1.015625, -3.0]
    v = ref.e4m3_values()
    assert v[0x7E] == 448 and v[0x01] == 2.0 ** -9 and np.isnan(v[0x7F]) and v[0xB8] == -1.0
    assert ref.fp4_values(np.array([[0x21, 0xF7]], np.uint8), np.array([[128]], np.uint8), True).tolist() == \
        [[1.0, 2.0, 12.0, -12.0]]


def test_route_reference_on_hand_rows():
    inf = np.inf
    x = np.float32([[0, 1, 2, 3], [-inf, 5, -inf, -inf], [-inf] * 4, [1, 1, 1, 1]])
    idx, w = ref.route(x, None, 2, 1, 1, False, True, 1.0)
    assert idx.tolist() == [[3, 2], [1, -1], [-1, -1], [0, 1]]
    assert w[1].tolist() == [1.0, 0.0] and w[3].tolist() == [0.5, 0.5]
    # two groups keeping one: the group with a single live expert counts that one alone
    idx, _ = ref.route(x, None, 2, 2, 1, False, False, 1.0)
    assert idx.tolist() == [[3, 2], [1, -1], [-1, -1], [0, 1]]
