"""The gate's gradient where the gate is nearly open or shut: the slope of a
sigmoid is s (1 - s), and 1 - s is small next to s's own rounding."""
import numpy as np
import pytest

import mixer_reference as R

pytestmark = pytest.mark.gpu

Z = [0.0, -0.0, 0.3, -0.3, 1.0, -1.2784645, 5.0, -5.0, 9.0, -9.0, 12.0, 15.0, -15.0, 16.6, 17.0, -17.0, 20.0, 30.0, -30.0,
     45.0, 60.0, -60.0, 80.0, -80.0]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("gate", ["sigmoid", "silu"])
@pytest.mark.parametrize("d", [48, 41, 1024])
def test_slope_of_large_gates(d, gate, io):
    """dz = dy u w s'(z), each factor within its own relative error: u and the
    products 64 u together (as everywhere here); s = 1 / (1 + e) and 1 - s = e / (1 + e),
    e = exp(-z), 16 u in fp32 and 2^-20 (1 + |z|) by the intrinsics.  Silu's slope,
    s (1 + z (1 - s)), is a sum: the sizes of its terms count."""
    import torch
    import gated_delta_rule_87_b200 as gdr
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    rng = np.random.default_rng([d, len(Z)])
    dev = lambda a, t=torch.float32: torch.from_numpy(np.asarray(a, np.float32)).cuda().to(t)  # noqa: E731
    host = lambda t: t.double().cpu().numpy()  # noqa: E731
    M = 5
    x, dy = (dev(rng.standard_normal((M, 2, d)), dt) for _ in range(2))
    z, w = dev(rng.choice(Z, (M, 2, d)), dt), dev(1 + 0.3 * rng.standard_normal(d))
    dx, dz, dw, _ = gdr.gated_norm_bwd(dy, x, z, w, gate=gate, eps=1e-5)
    X, Y, V, W = host(x), host(dy), host(z), host(w)
    u = X / np.sqrt((X * X).mean(-1, keepdims=True) + float(np.float32(1e-5)))
    e = np.exp(-np.abs(V))
    small, large = e / (1 + e), 1 / (1 + e)
    s, rest = np.where(V > 0, large, small), np.where(V > 0, small, large)
    slope = s * rest if gate == "sigmoid" else s * (1 + V * rest)
    size = s * rest if gate == "sigmoid" else s * (1 + np.abs(V) * rest)
    k = 64 * R.U + (32 * R.U if io == "f32" else 2.0 ** -19 * (1 + np.abs(V)))
    want = Y * u * W * slope
    R.check(host(dz), want, np.abs(Y * u * W) * size * k, io, "dz")
    value = s if gate == "sigmoid" else V * s
    want = (Y * u * value).sum((0, 1))
    R.check(host(dw), want, (np.abs(Y * u * value) * (k + 64 * R.U)).sum((0, 1)), "f32", "dw")
