"""Gated RMS norm and residual add with RMS norm on the GPU, forward and
backward, against their 64-bit forms, element by element."""
import numpy as np
import pytest

import mixer_reference as R

pytestmark = pytest.mark.gpu

EPS = 1e-5


def _dt(io):
    import torch
    return torch.bfloat16 if io == "bf16" else torch.float32


def _dev(a, io="f32"):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda().to(_dt(io))


def _host(t):
    return t.float().cpu().numpy()


def _chain(rows, d):
    """Additions that a column sum takes one after another at most: a thread's
    rows, its block's groups, its part of the blocks and the join."""
    return rows / 148 + 32 + 40 + 8


def _gated(M, H, d, io, gate, weight=True, seed=0, scale=1.0):
    import torch
    import gated_delta_rule_87_b200 as gdr
    rng = np.random.default_rng([seed, M, H, d])
    n = lambda *s: rng.standard_normal(s)  # noqa: E731
    x, z, dy = _dev(scale * n(M, H, d), io), _dev(2 * n(M, H, d), io), _dev(n(M, H, d), io)
    w = _dev(1 + 0.3 * n(d)) if weight else None
    zz = z if gate else None
    y = gdr.gated_norm_fwd(x, zz, w, gate=gate, eps=EPS)
    flat = lambda t: _host(t).reshape(M * H, d)  # noqa: E731
    ww = _host(w) if weight else np.ones(d)
    eps = float(np.float32(EPS))
    want, err = R.gated_norm(flat(x), flat(z), ww, gate, eps, io)
    R.check(_host(y), want.reshape(M, H, d), err.reshape(M, H, d), io, "y")
    dx, dz, dw, _ = gdr.gated_norm_bwd(dy, x, zz, w, gate=gate, eps=EPS)
    want, err = R.gated_norm_bwd(flat(dy), flat(x), flat(z), ww, gate, eps, io, _chain(M * H, d))
    R.check(flat(dx), want[0], err[0], io, "dx")
    if gate:
        R.check(flat(dz), want[1], err[1], io, "dz")
    else:
        assert dz is None
    if weight:
        R.check(_host(dw), want[2], err[2], "f32", "dw")
    else:
        assert dw is None


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("gate", ["silu", "sigmoid", None])
@pytest.mark.parametrize("d", [1, 3, 8, 32, 64, 96, 100, 128, 129, 256, 264, 333, 1000])
def test_gated_norm_head_sizes(d, gate, io):
    _gated(9, 3, d, io, gate, seed=d)


@pytest.mark.parametrize("M,H,d", [(1, 1, 128), (1, 32, 128), (700, 32, 128), (1500, 5, 64), (3, 1, 4096), (2, 1, 16384),
                                   (2, 1, 16383), (5, 1, 8200), (3, 1, 5001)])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_gated_norm_row_counts(M, H, d, io):
    _gated(M, H, d, io, "silu", seed=M)


def test_gated_norm_without_weight():
    _gated(40, 4, 128, "bf16", "sigmoid", weight=False)


@pytest.mark.parametrize("scale", [1e-20, 1e-3, 1e3, 1e15])
def test_gated_norm_of_small_and_large_rows(scale):
    """Squares that underflow (eps rules) and rows of any size in range."""
    _gated(6, 2, 64, "f32", "silu", scale=scale)


def test_gated_norm_of_zeros_and_large_gates():
    import torch
    import gated_delta_rule_87_b200 as gdr
    x = torch.zeros((2, 2, 64), dtype=torch.bfloat16, device="cuda")
    z = torch.full_like(x, 5.0)
    assert bool((gdr.gated_norm_fwd(x, z) == 0).all())
    x[1] = 1.0
    for io in (torch.bfloat16, torch.float32):
        for gate in ("silu", "sigmoid"):
            low = gdr.gated_norm_fwd(x.to(io), torch.full((2, 2, 64), -200.0, dtype=io, device="cuda"), gate=gate)
            assert bool((low.abs() < 1e-30).all())
            dx, dz, _, _ = gdr.gated_norm_bwd(x.to(io), x.to(io), torch.full((2, 2, 64), -200.0, dtype=io, device="cuda"), gate=gate)
            assert bool(torch.isfinite(dx).all()) and bool(torch.isfinite(dz).all())
            high = gdr.gated_norm_fwd(x.to(io), torch.full((2, 2, 64), 200.0, dtype=io, device="cuda"), gate=gate)
            assert bool(((high[1] - (200.0 if gate == "silu" else 1.0)).abs() < 1.0).all())


def test_a_row_with_nan_leaves_the_others():
    import torch
    import gated_delta_rule_87_b200 as gdr
    x = torch.randn((50, 4, 128), device="cuda").bfloat16()
    z = torch.randn_like(x)
    want = gdr.gated_norm_fwd(x, z)
    x[17, 2, 5] = float("nan")
    got = gdr.gated_norm_fwd(x, z)
    keep = torch.ones((50, 4), dtype=torch.bool, device="cuda")
    keep[17, 2] = False
    assert torch.equal(got[keep], want[keep]) and bool(torch.isnan(got[17, 2]).all())


@pytest.mark.parametrize("off", [0, 1, 8])
def test_gated_norm_of_slices(off):
    """x, z and dy inside wider token rows, aligned and not.  Rows that do not
    begin on 16 bytes are summed in another order: two fp32 values a few u apart
    may round to neighbouring bf16 values, one step (2^-7 of the value) apart."""
    import torch
    import gated_delta_rule_87_b200 as gdr
    B, T, H, d = 2, 13, 4, 64
    wide = torch.randn((3, B, T, H * d + 24), device="cuda").bfloat16()
    x, z, dy = (wide[k, ..., off:off + H * d].unflatten(-1, (H, d)) for k in range(3))
    w = torch.randn(d, device="cuda")
    args = [t.contiguous() for t in (x, z)]
    got, want = (t.float() for t in (gdr.gated_norm_fwd(x, z, w), gdr.gated_norm_fwd(*args, w)))
    assert bool(((got - want).abs() <= 2.0 ** -7 * want.abs()).all())
    got = gdr.gated_norm_bwd(dy, x, z, w)[:3]
    want = gdr.gated_norm_bwd(dy.contiguous(), *args, w)[:3]
    for p, q in zip(got[:2], want[:2]):
        assert (p.float() - q.float()).abs().max() <= 2.0 ** -7 * q.float().abs().max()
    assert torch.allclose(got[2], want[2], rtol=1e-4, atol=1e-4)


def _add(M, D, io, res, scaled=True, weight=True, dt=True, seed=0):
    import torch
    import gated_delta_rule_87_b200 as gdr
    rng = np.random.default_rng([seed, M, D])
    n = lambda *s: rng.standard_normal(s)  # noqa: E731
    r, y, dn, dr = _dev(n(M, D), res), _dev(n(M, D), io), _dev(n(M, D), io), _dev(n(M, D), res)
    w, s = (_dev(1 + 0.3 * n(D)) if weight else None), (_dev(0.5 + 0.2 * n(D)) if scaled else None)
    hw, hs = _host(w) if weight else np.ones(D), _host(s) if scaled else np.ones(D)
    eps = float(np.float32(EPS))
    out, norm = gdr.add_norm_fwd(r, y, w, s, eps=EPS)
    want, err = R.add_norm(_host(r), _host(y), hw, hs, eps)
    R.check(_host(out), want[0], err[0], res, "residual_out")
    R.check(_host(norm), want[1], err[1], io, "n")
    d, dy, dw, ds, _ = gdr.add_norm_bwd(dn, dr if dt else None, out, y, w, s, eps=EPS)
    want, err = R.add_norm_bwd(_host(dn), _host(dr) if dt else np.zeros((M, D)), _host(out), _host(y), hw, hs,
                               _chain(M, D), eps)
    R.check(_host(d), want[0], err[0], res, "dresidual")
    R.check(_host(dy), want[1], err[1], io, "dy")
    if weight:
        R.check(_host(dw), want[2], err[2], "f32", "dweight")
    if scaled:
        R.check(_host(ds), want[3], err[3], "f32", "dscale")
    assert (dw is None) == (not weight) and (ds is None) == (not scaled)
    assert (dy is d) == (not scaled and io == res)


@pytest.mark.parametrize("io,res", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("D", [1, 7, 64, 100, 256, 257, 1024, 2047, 4096, 4104])
def test_add_norm_widths(D, io, res):
    _add(11, D, io, res, seed=D)


@pytest.mark.parametrize("io,res", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("M,D", [(1, 128), (2500, 72), (1200, 640), (3, 16384), (2, 16381), (2, 8199)])
def test_add_norm_row_counts(M, D, io, res):
    _add(M, D, io, res, seed=M)


@pytest.mark.parametrize("scaled,weight,dt", [(False, True, True), (True, False, True), (False, False, False), (True, True, False)])
@pytest.mark.parametrize("io,res", [("bf16", "bf16"), ("bf16", "f32")])
def test_add_norm_optional_parts(scaled, weight, dt, io, res):
    _add(20, 320, io, res, scaled, weight, dt)


def test_add_norm_in_place():
    import torch
    import gated_delta_rule_87_b200 as gdr
    r, y = torch.randn((300, 512), device="cuda"), torch.randn((300, 512), device="cuda").bfloat16()
    want, n0 = gdr.add_norm_fwd(r, y)
    out, n = gdr.add_norm_fwd(r, y, residual_out=r)
    assert out is r and torch.equal(r, want) and torch.equal(n, n0)
    dn, dr = torch.randn_like(y), torch.randn_like(r)
    want = gdr.add_norm_bwd(dn, dr, r)
    got = gdr.add_norm_bwd(dn, dr, r, dresidual=dr)
    assert torch.equal(got[0], want[0]) and got[0] is dr and torch.equal(got[1], want[1])


def test_no_rows():
    import torch
    import gated_delta_rule_87_b200 as gdr
    x, w = torch.zeros((0, 2, 64), device="cuda"), torch.ones(64, device="cuda")
    assert gdr.gated_norm_fwd(x, x, w).shape == (0, 2, 64)
    _, _, dw, _ = gdr.gated_norm_bwd(x, x, x, w, dweight=torch.full((64,), 3.0, device="cuda"))
    assert bool((dw == 0).all())
    r = torch.zeros((0, 64), device="cuda")
    assert gdr.add_norm_fwd(r, r, w, w)[1].shape == (0, 64)
    _, _, dw, ds, _ = gdr.add_norm_bwd(r, r, r, r, w, w)
    assert bool((dw == 0).all()) and bool((ds == 0).all())


def test_same_inputs_same_bits():
    import torch
    import gated_delta_rule_87_b200 as gdr
    x, z, dy = (torch.randn((3000, 8, 128), device="cuda").bfloat16() for _ in range(3))
    w = torch.randn(128, device="cuda")
    r, y, dn = (t.view(3000, 1024) for t in (x, z, dy))
    w2 = torch.randn(1024, device="cuda")
    first = [*gdr.gated_norm_bwd(dy, x, z, w)[:3], *gdr.add_norm_bwd(dn, r, r, y, w2, w2)[:4]]
    for _ in range(3):
        again = [*gdr.gated_norm_bwd(dy, x, z, w)[:3], *gdr.add_norm_bwd(dn, r, r, y, w2, w2)[:4]]
        assert all(torch.equal(p, q) for p, q in zip(first, again))


def test_captured_gradients_replay():
    import torch
    import gated_delta_rule_87_b200 as gdr
    x, z, dy = (torch.randn((200, 4, 128), device="cuda").bfloat16() for _ in range(3))
    w = torch.randn(128, device="cuda")
    call = lambda: [gdr.gated_norm_fwd(x, z, w), *gdr.gated_norm_bwd(dy, x, z, w)[:3]]  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    x.copy_(torch.randn_like(x))
    dy.copy_(torch.randn_like(dy))
    want = call()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(out, want))


def test_a_mixer_block_with_its_gradients():
    """Boundary norm, gated recurrence, gated norm, boundary norm, and back,
    against automatic differentiation of the same block in 64 bits.  All in
    fp32: each of the four operators is within 1e-5 of its terms here, and the
    gradients of a block this small grow them by less than ten."""
    import torch
    import gated_delta_rule_87_b200 as gdr
    torch.manual_seed(0)
    B, T, H, d = 2, 70, 2, 16
    D = H * d
    leaf = dict(r=(B, T, D), y=(B, T, D), g=(B, T, D), z=(B, T, H, d), w1=(D,), s1=(D,), w2=(d,), w3=(D,), s3=(D,), h0=(B, D))
    t = {k: torch.randn(s, device="cuda") for k, s in leaf.items()}
    t["g"] = -torch.nn.functional.softplus(t["g"])
    up = [torch.randn((B, T, D), device="cuda") for _ in range(2)]

    r1, n1 = gdr.add_norm_fwd(t["r"], t["y"], t["w1"], t["s1"])
    h, _, saved, _ = gdr.glr_scan_fwd(n1, t["g"], t["h0"], output_chunk_states=True)
    o = gdr.gated_norm_fwd(h.view(B, T, H, d), t["z"], t["w2"])
    r2, n2 = gdr.add_norm_fwd(r1, o.view(B, T, D), t["w3"], t["s3"])
    grad = {}
    dr1, do, grad["w3"], grad["s3"], _ = gdr.add_norm_bwd(up[1], up[0], r2, o.view(B, T, D), t["w3"], t["s3"])
    dh, grad["z"], grad["w2"], _ = gdr.gated_norm_bwd(do.view(B, T, H, d), h.view(B, T, H, d), t["z"], t["w2"])
    dn1, grad["g"], grad["h0"], _ = gdr.glr_scan_bwd(dh.view(B, T, D), n1, t["g"], t["h0"], chunk_states=saved)
    grad["r"], grad["y"], grad["w1"], grad["s1"], _ = gdr.add_norm_bwd(dn1, dr1, r1, t["y"], t["w1"], t["s1"])

    q = {k: v.double().cpu().requires_grad_() for k, v in t.items()}
    rms = lambda v: v / (v.square().mean(-1, keepdim=True) + 1e-6).sqrt()  # noqa: E731
    a1 = q["r"] + q["s1"] * q["y"]
    m1, s, hs = rms(a1) * q["w1"], q["h0"], []
    for k in range(T):
        s = q["g"][:, k].exp() * s + m1[:, k]
        hs.append(s)
    oo = rms(torch.stack(hs, 1).view(B, T, H, d)) * q["w2"] * torch.nn.functional.silu(q["z"])
    a2 = a1 + q["s3"] * oo.reshape(B, T, D)
    m2 = rms(a2) * q["w3"]
    (a2 * up[0].double().cpu()).sum().add((m2 * up[1].double().cpu()).sum()).backward()
    for got, want in ((r2, a2), (n2, m2)):
        want = want.detach()
        assert (got.double().cpu() - want).norm() <= 1e-5 * want.norm()
    assert set(grad) == set(q)
    for k, v in grad.items():
        assert (v.double().cpu().view(q[k].shape) - q[k].grad).norm() <= 1e-4 * q[k].grad.norm(), k


def test_the_gated_norm_takes_a_mixers_output():
    """KDA prefill, then its output gate and norm, on the layout as it comes."""
    import torch
    import gated_delta_rule_87_b200 as gdr
    torch.manual_seed(1)
    B, T, H, d = 1, 150, 2, 128
    q, k, v, z = (torch.randn((B, T, H, d), device="cuda").bfloat16() for _ in range(4))
    k = torch.nn.functional.normalize(k.float(), dim=-1).bfloat16()
    g, beta = -0.1 * torch.rand((B, T, H, d), device="cuda"), torch.rand((B, T, H), device="cuda")
    w = torch.randn(d, device="cuda")
    o, _, _ = gdr.kda_chunk_fwd(q, k, v, g, beta)
    y = gdr.gated_norm_fwd(o, z, w, gate="sigmoid", eps=EPS)
    want, err = R.gated_norm(_host(o), _host(z), _host(w), "sigmoid", float(np.float32(EPS)), "bf16")
    R.check(_host(y), want, err, "bf16", "y")


def test_binding_refusals():
    import torch
    import gated_delta_rule_87_b200 as gdr
    x = torch.zeros((5, 2, 64), device="cuda")
    w, r = torch.ones(64, device="cuda"), torch.zeros((5, 64), device="cuda")
    big = torch.zeros((1, 16400), device="cuda")
    bad = [
        lambda: gdr.gated_norm_fwd(x),                       # a gate without z
        lambda: gdr.gated_norm_fwd(x, x, gate=None),         # z without a gate
        lambda: gdr.gated_norm_fwd(x, x, gate="relu"),
        lambda: gdr.gated_norm_fwd(x, x.bfloat16()),
        lambda: gdr.gated_norm_fwd(x, x[:4]),
        lambda: gdr.gated_norm_fwd(x, x, w[:32]),
        lambda: gdr.gated_norm_fwd(x, x, w.bfloat16()),
        lambda: gdr.gated_norm_fwd(x, x.cpu()),
        lambda: gdr.gated_norm_fwd(x, x, eps=0.0),
        lambda: gdr.gated_norm_fwd(x, x, eps=float("nan")),
        lambda: gdr.gated_norm_fwd(x.transpose(0, 1), x.transpose(0, 1)),
        lambda: gdr.gated_norm_fwd(big[:, None], big[:, None]),
        lambda: gdr.gated_norm_bwd(x.bfloat16(), x, x),
        lambda: gdr.add_norm_fwd(r.bfloat16(), r),           # a bf16 residual with fp32 activations
        lambda: gdr.add_norm_fwd(r, r[:4]),
        lambda: gdr.add_norm_fwd(r, r, w[:3]),
        lambda: gdr.add_norm_fwd(r, r.clone(), n=r),
        lambda: gdr.add_norm_fwd(r.t(), r.t()),
        lambda: gdr.add_norm_fwd(big, big),
        lambda: gdr.add_norm_fwd(r, r, eps=-1.0),
        lambda: gdr.add_norm_bwd(r, r, r, None, w, w),       # a scale without y
        lambda: gdr.add_norm_bwd(r, r, r.bfloat16()),
    ]
    for call in bad:
        with pytest.raises((ValueError, TypeError, gdr.KdaError)):
            call()


@pytest.mark.parametrize("fn,kw", [
    (test_gated_norm_head_sizes, dict(d=128, gate="silu", io="bf16")),
    (test_gated_norm_head_sizes, dict(d=333, gate="sigmoid", io="f32")),
    (test_gated_norm_row_counts, dict(M=700, H=32, d=128, io="bf16")),
    (test_gated_norm_row_counts, dict(M=2, H=1, d=16383, io="bf16")),
    (test_add_norm_widths, dict(D=257, io="bf16", res="f32")),
    (test_add_norm_widths, dict(D=4096, io="bf16", res="bf16")),
    (test_add_norm_row_counts, dict(M=2500, D=72, io="f32", res="f32")),
    (test_gated_norm_of_slices, dict(off=1)),
], ids=lambda v: v.__name__ if callable(v) else "-".join(map(str, v.values())))
def test_checked_build_finds_no_access_out_of_bounds(fn, kw):
    import gated_delta_rule_87_b200 as gdr
    with gdr.use_library(gdr.checked_library_path):
        gdr.bounds_violations()
        fn(**kw)
        assert gdr.bounds_violations() == 0
