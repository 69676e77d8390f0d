"""Memories of 10^4 to 10^6 tokens over 2^18 tokens, inputs of one sign: nothing
cancels, so every value is held to a small part of itself, and a carry that is
lost or damaged anywhere shows in every channel behind it.

The bound, in u = 2^-24: what is carried meets one rounded decay (within 2 ulp,
4 u) and one product-sum (u) in each group of at least 1024 tokens, T / 1024
groups; inside a group at most 32 tokens, 4 + 4 warps and 16 tiles are joined in
this way, 5 u each (56 x 5), and the sums of log-decays, of size |g| T at most in
all, are off by 10 u of themselves (|g| T < 27: 270 u).  dg is the product of two
such values."""
import numpy as np
import pytest

import mixer_reference as R

T = 1 << 18
TOL = (5 * T / 1024 + 280 + 270) * R.U


def _inputs(D, io, seed):
    rng = np.random.default_rng(seed)
    g = np.broadcast_to(-10.0 ** rng.uniform(-6, -4, D), (T, D)).astype(np.float32)
    x, dh = (rng.uniform(0.5, 1.5, (T, D)).astype(np.float32) for _ in range(2))
    if io == "bf16":  # values that bf16 holds: 8 bits
        x, dh = (np.round(a * 128) / 128 for a in (x, dh))
    return x, g, rng.uniform(1, 2, D).astype(np.float32), dh, rng.uniform(1, 2, D).astype(np.float32)


def _exact(x, g, h0, dh, df, damage=None):
    """By the definition in 64 bits; ``damage``: (token, factor) of a carry."""
    x, g, h0, dh, df = (np.asarray(a, np.float64) for a in (x, g, h0, dh, df))
    a = np.exp(g)
    h, dx, dg = np.empty_like(x), np.empty_like(x), np.empty_like(x)
    s = h0
    for t in range(T):
        if damage and t == damage[0]:
            s = s * damage[1]
        s = a[t] * s + x[t]
        h[t] = s
    c = df
    for t in range(T - 1, -1, -1):
        d = dh[t] + c
        dx[t] = d
        c = a[t] * d
        dg[t] = c * (h[t - 1] if t else h0)
    return dict(h=h, final=s, dx=dx, dg=dg, dh0=c)


def _off(got, want, io):
    """Names of the outputs that have a value outside its bound."""
    bad = []
    for k, w in want.items():
        tol = (2 if k == "dg" else 1) * TOL + (R.HALF_STEP[io] if k in ("h", "dx") else 0)
        if not (np.abs(np.asarray(got[k], np.float64) - w) <= tol * np.abs(w)).all():
            bad.append(k)
    return bad


def test_the_bound_rejects_lost_and_damaged_carries():
    args = _inputs(6, "bf16", 0)
    want = _exact(*args)
    for io in ("f32", "bf16"):
        assert _off(want, want, io) == []
        assert _off({k: np.zeros_like(v) for k, v in want.items()}, want, io) == list(want)
        # 1 % of the carry at one tile's border, or a tenth of a percent: all that follows, states above all
        damaged = _exact(*args, damage=(T - 64 * 500, 0.99))
        assert {"h", "final", "dg"} <= set(_off(damaged, want, io))
        assert "final" in _off(_exact(*args, damage=(T - 64 * 500, 0.999)), want, io)


@pytest.mark.gpu
@pytest.mark.parametrize("io,D", [("f32", 40), ("f32", 33), ("bf16", 64), ("bf16", 35)])
def test_constant_decays_over_long_sequences(io, D):
    import torch
    import gated_delta_rule_87_b200 as gdr
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    args = _inputs(D, io, D)
    x, g, h0, dh, df = (torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in args)
    x, dh = x.to(dt)[None], dh.to(dt)[None]
    h, final, saved, _ = gdr.glr_scan_fwd(x, g[None], h0[None], output_chunk_states=True)
    host = lambda t: t.float().cpu().numpy()[0]  # noqa: E731
    want = _exact(*args)
    for chunks in (saved, None):
        dx, dg, dh0, _ = gdr.glr_scan_bwd(dh, x, g[None], h0[None], dfinal_state=df[None], chunk_states=chunks)
        got = dict(h=host(h), final=host(final), dx=host(dx), dg=host(dg), dh0=host(dh0))
        assert _off(got, want, io) == []
