"""The 64-bit forms that the GPU tests compare with: their gradients against
differences of their values (central differences in 64 bits: with a step of
1e-6 the quotient is good to about 1e-9 of the terms' sizes)."""
import numpy as np
import pytest

import mixer_reference as R


def _slope(f, x, v, step=1e-6):
    return (f(x + step * v) - f(x - step * v)) / (2 * step)


@pytest.mark.parametrize("complement", [False, True])
def test_scan_gradients_are_the_slopes(complement):
    rng = np.random.default_rng(1)
    cu, D = [0, 5, 5, 6, 13], 3
    x, g = rng.standard_normal((13, D)), -np.abs(rng.standard_normal((13, D)))
    h0, dh, df = (rng.standard_normal(s) for s in ((4, D), (13, D), (4, D)))

    def loss(x, g, h0):
        h, final, _, _ = R.scan(x, g, h0, cu, complement)
        return (h * dh).sum() + (final * df).sum()

    (dx, dg, dh0), _ = R.scan_bwd(dh, df, x, g, h0, cu, complement)
    for k, grad in enumerate((dx, dg, dh0)):
        args = [x, g, h0]
        v = rng.standard_normal(args[k].shape)
        f = lambda a: loss(*args[:k], a, *args[k + 1:])  # noqa: E731
        assert abs(_slope(f, args[k], v) - (grad * v).sum()) < 1e-6


@pytest.mark.parametrize("kind", [None, "silu", "sigmoid"])
def test_gated_norm_gradients_are_the_slopes(kind):
    rng = np.random.default_rng(2)
    x, z, dy = (rng.standard_normal((4, 7)) for _ in range(3))
    w = rng.standard_normal(7)
    grads, _ = R.gated_norm_bwd(dy, x, z, w, kind, 1e-5, "f32", 1)
    for k, grad in enumerate(grads):
        args = [x, z, w]
        v = rng.standard_normal(args[k].shape)
        f = lambda a: (R.gated_norm(*args[:k], a, *args[k + 1:], kind, 1e-5, "f32")[0] * dy).sum()  # noqa: E731
        assert abs(_slope(f, args[k], v) - (grad * v).sum()) < 1e-6


def test_add_norm_gradients_are_the_slopes():
    rng = np.random.default_rng(3)
    r, y, dn, dt = (rng.standard_normal((4, 7)) for _ in range(4))
    w, scale = rng.standard_normal(7), rng.standard_normal(7)

    def loss(r, y, w, scale):
        (t, n), _ = R.add_norm(r, y, w, scale, 1e-5)
        return (t * dt).sum() + (n * dn).sum()

    (d, dy, dw, ds), _ = R.add_norm_bwd(dn, dt, r + scale * y, y, w, scale, 1, 1e-5)
    for k, grad in enumerate((d, dy, dw, ds)):
        args = [r, y, w, scale]
        v = rng.standard_normal(args[k].shape)
        f = lambda a: loss(*args[:k], a, *args[k + 1:])  # noqa: E731
        assert abs(_slope(f, args[k], v) - (grad * v).sum()) < 1e-6
