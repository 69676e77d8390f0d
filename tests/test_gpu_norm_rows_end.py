"""Groups of threads that are past the last row while others of their block are
not: they add nothing to the column sums, not even 0 times an infinity."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128, 200, 250])
@pytest.mark.parametrize("io,res", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_an_infinite_gradient_stays_an_infinite_sum(D, io, res):
    """The gradient of the residual is infinite in one column, y is one there: so
    are its sum, the gradient of the scale, and nothing else.  M - 1 is a multiple
    of every block's groups: at the last step one group of one block has a row."""
    import torch
    import gated_delta_rule_87_b200 as gdr
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}
    M, c = 32 * 5000 + 1, 37
    gen = torch.Generator(device="cuda").manual_seed(D)
    rand = lambda k: torch.randn((M, D), generator=gen, device="cuda").to(dt[k])  # noqa: E731
    out, y, dn, dr = rand(res), rand(io), rand(io), rand(res)
    y[:, c], dr[:, c] = 1.0, float("inf")
    w, s = (torch.rand(D, generator=gen, device="cuda") + 0.5 for _ in range(2))
    dres, dy, dw, ds, _ = gdr.add_norm_bwd(dn, dr, out, y, w, s)
    assert bool((ds[c] == float("inf")).all()) and bool((dres[:, c] == float("inf")).all())
    keep = torch.arange(D, device="cuda") != c
    t, n = out.double(), dn.double()
    inv = (t.square().mean(-1, keepdim=True) + float(np.float32(1e-6))).rsqrt()
    du = n * w.double()
    d = dr.double() + inv * (du - t * inv * (du * t * inv).mean(-1, keepdim=True))
    # fp32 sums of M terms, each within 100 u of its size; at most M / 148 additions one after another
    u, chain = 2.0 ** -24, M / 148 + 100
    want, size = (d * y.double()).sum(0), ((d.abs() + 3 * inv * du.abs()) * y.double().abs()).sum(0)
    assert bool(((ds - want).abs() <= (chain + 100) * u * size)[keep].all())
    want, size = (n * t * inv).sum(0), (n * t * inv).abs().sum(0)
    assert bool(((dw - want).abs() <= (chain + 100) * u * size).all())


@pytest.mark.parametrize("d", [64, 128, 100])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_an_infinite_gate_stays_an_infinite_sum(d, io):
    """silu(inf) is inf: so is its column of the weight's gradient, and no other."""
    import torch
    import gated_delta_rule_87_b200 as gdr
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[io]
    M, c = 32 * 5000 + 1, 37
    gen = torch.Generator(device="cuda").manual_seed(d)
    x, z, dy = (torch.randn((M, 1, d), generator=gen, device="cuda").abs().add(0.1).to(dt) for _ in range(3))
    z[..., c] = float("inf")
    dw = gdr.gated_norm_bwd(dy, x, z, torch.ones(d, device="cuda"))[2]
    assert dw[c] == float("inf")
    keep = torch.arange(d, device="cuda") != c
    inv = (x.double().square().mean(-1, keepdim=True) + float(np.float32(1e-6))).rsqrt()
    want = (dy.double() * x.double() * inv * torch.nn.functional.silu(z.double())).sum((0, 1))
    # positive terms: each within 2^-19 (1 + |z|) of itself (|z| < 7), the sums of M / 148 and 100 additions
    assert bool(((dw - want).abs() <= (2.0 ** -16 + (M / 148 + 100) * 2.0 ** -24) * want)[keep].all())
