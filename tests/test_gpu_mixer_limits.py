"""The recurrence and the norms at the ends of their ranges: offsets past 31 bits,
other streams, replayed graphs, shared workspaces, entries that share a slot."""
import numpy as np
import pytest

import mixer_reference as R

pytestmark = pytest.mark.gpu

EPS = 1e-5


def _host(t):
    return t.float().cpu().numpy()


def _wide(shape, seed, dtype, scale=1.0):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.empty(shape, dtype=dtype, device="cuda")
    return t.normal_(generator=gen).mul_(scale)


def test_scan_offsets_past_31_bits():
    """2^31 and more elements a tensor; channels of the first, a middle and the
    last tile against the 64-bit form."""
    import torch
    import gated_delta_rule_87_b200 as gdr
    T, D = 65600, 32768
    assert T * D > 2 ** 31
    x, dh = (_wide((1, T, D), s, torch.bfloat16) for s in (1, 2))
    g = _wide((1, T, D), 3, torch.float32, 0.3).abs_().neg_()
    h0, df = (_wide((2, D), s, torch.float32) for s in (4, 5))
    offsets = [0, 65000, T]
    cu = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    h, final, saved, ws = gdr.glr_scan_fwd(x, g, h0, cu, output_chunk_states=True)
    assert gdr.check_device_status(ws) == (gdr.KDA_OK, gdr.KDA_DEVICE_OK)
    dx, dg, dh0, ws = gdr.glr_scan_bwd(dh, x, g, h0, cu, dfinal_state=df, chunk_states=saved)
    assert gdr.check_device_status(ws) == (gdr.KDA_OK, gdr.KDA_DEVICE_OK)
    at = torch.tensor([0, 16385, D - 1], device="cuda")
    pick = lambda t: _host(t[..., at]).reshape(-1, 3)  # noqa: E731
    rh, rf, eh, ef = R.scan(pick(x), pick(g), pick(h0), offsets, False)
    R.check(pick(h), rh, eh, "bf16", "h")
    R.check(pick(final), rf, ef, "f32", "final")
    want, err = R.scan_bwd(pick(dh), pick(df), pick(x), pick(g), pick(h0), offsets, False)
    for got, w, e, io in zip((dx, dg, dh0), want, err, ("bf16", "f32", "f32")):
        R.check(pick(got), w, e, io)


@pytest.mark.parametrize("off", [0, 5])
def test_row_strides_past_31_bits(off):
    """Few channels of rows so far apart that their offsets pass 31 bits."""
    import torch
    import gated_delta_rule_87_b200 as gdr
    T, D, ld = 600, 40, 4_000_000
    assert (T - 1) * ld > 2 ** 31

    def strided(seed, dtype):
        small = _wide((1, T, D), seed, dtype)
        if dtype == torch.float32:
            small = small.abs_().neg_()
        wide = torch.empty((1, T, ld), dtype=dtype, device="cuda")[..., off:off + D]
        return wide.copy_(small), small

    (x, xs), (g, gs), (dh, dhs) = strided(1, torch.bfloat16), strided(2, torch.float32), strided(3, torch.bfloat16)
    h, _, saved, _ = gdr.glr_scan_fwd(x, g, output_chunk_states=True)
    flat = lambda t: _host(t).reshape(T, D)  # noqa: E731
    z = np.zeros((1, D))
    rh, _, eh, _ = R.scan(flat(xs), flat(gs), z, [0, T], False)
    R.check(flat(h), rh, eh, "bf16", "h")
    dx, dg, _, _ = gdr.glr_scan_bwd(dh, x, g, chunk_states=saved)
    want, err = R.scan_bwd(flat(dhs), z, flat(xs), flat(gs), z, [0, T], False)
    R.check(flat(dx), want[0], err[0], "bf16", "dx")
    R.check(flat(dg), want[1], err[1], "f32", "dg")
    state = torch.zeros((T, D), device="cuda")
    h = gdr.glr_step(x[0], g[0], state)
    R.check(flat(h), flat(xs), np.zeros(1), "bf16", "step")  # from no state: h is x
    assert torch.equal(state, xs[0].float())
    y = gdr.gated_norm_fwd(x[0].view(T, 1, D), dh[0].view(T, 1, D), None, eps=EPS)
    n, e = R.gated_norm(flat(xs), flat(dhs), np.ones(D), "silu", float(np.float32(EPS)), "bf16")
    R.check(flat(y), n, e, "bf16", "norm")


@pytest.mark.parametrize("d", [128, 127])
def test_gated_norm_offsets_past_31_bits(d):
    import torch
    import gated_delta_rule_87_b200 as gdr
    M, H = 2 ** 31 // (128 * d) + 9, 128
    assert M * H * d > 2 ** 31
    x, z = (_wide((M, H, d), s, torch.bfloat16) for s in (1, 2))
    w = _wide((d,), 4, torch.float32)
    at = torch.tensor([0, M // 2, M - 1], device="cuda")
    dy = torch.zeros_like(x)  # elsewhere: the sums are those of three tokens
    dy[at] = _wide((3, H, d), 3, torch.bfloat16)
    y = gdr.gated_norm_fwd(x, z, w, gate="silu", eps=EPS)
    dx, dz, dw, _ = gdr.gated_norm_bwd(dy, x, z, w, gate="silu", eps=EPS)
    pick = lambda t: _host(t[at]).reshape(-1, d)  # noqa: E731
    eps = float(np.float32(EPS))
    want, err = R.gated_norm(pick(x), pick(z), _host(w), "silu", eps, "bf16")
    R.check(pick(y), want, err, "bf16", "y")
    want, err = R.gated_norm_bwd(pick(dy), pick(x), pick(z), _host(w), "silu", eps, "bf16", 3 * H)
    R.check(pick(dx), want[0], err[0], "bf16", "dx")
    R.check(pick(dz), want[1], err[1], "bf16", "dz")
    R.check(_host(dw), want[2], err[2], "f32", "dw")


@pytest.mark.parametrize("D", [16384, 16383])
def test_add_norm_offsets_past_31_bits(D):
    import torch
    import gated_delta_rule_87_b200 as gdr
    M = 2 ** 31 // D + 5
    r, y = (_wide((M, D), s, torch.bfloat16) for s in (1, 2))
    w = _wide((D,), 3, torch.float32)
    t, n = gdr.add_norm_fwd(r, y, w, eps=EPS)
    at = torch.tensor([0, M // 2, M - 1], device="cuda")
    pick = lambda a: _host(a[at])  # noqa: E731
    eps = float(np.float32(EPS))
    (rt, rn), (et, en) = R.add_norm(pick(r), pick(y), _host(w), np.ones(D), eps)
    R.check(pick(t), rt, et, "bf16", "t")
    R.check(pick(n), rn, en, "bf16", "n")
    dn = torch.zeros_like(y)  # elsewhere: the sums are those of three rows
    dn[at] = _wide((3, D), 4, torch.bfloat16)
    dres, dy, dw, _, _ = gdr.add_norm_bwd(dn, None, t, y, w, eps=EPS)
    want, err = R.add_norm_bwd(pick(dn), np.zeros((3, D)), pick(t), pick(y), _host(w), np.ones(D), 3, eps)
    R.check(pick(dres), want[0], err[0], "bf16", "dresidual")
    R.check(_host(dw), want[2], err[2], "f32", "dw")
    assert dy is dres


def _step_and_norms(t):
    """Decode with its output norm, and the block boundary behind it."""
    import gated_delta_rule_87_b200 as gdr
    h = gdr.glr_step(t["x"], t["g"], t["state"], state_slots=t["slots"])
    y = gdr.gated_norm_fwd(h.view(-1, 4, h.shape[1] // 4), t["z"], t["w"], gate="silu", eps=EPS)
    return gdr.add_norm_fwd(t["r"], y.view(h.shape), t["v"], t["s"], eps=EPS)


def _decode_inputs(N, D, seed):
    import torch
    bf, f = torch.bfloat16, torch.float32
    t = dict(x=_wide((N, D), seed, bf), g=_wide((N, D), seed + 1, f).abs_().neg_(), z=_wide((N, 4, D // 4), seed + 2, bf),
             w=_wide((D // 4,), seed + 3, f), v=_wide((D,), seed + 4, f), s=_wide((D,), seed + 5, f),
             r=_wide((N, D), seed + 6, bf), state=_wide((N + 2, D), seed + 7, f))
    t["slots"] = torch.arange(N + 1, 1, -1, dtype=torch.int32, device="cuda")
    return t


def test_captured_decode_with_its_norms_replays():
    import torch
    t = _decode_inputs(5, 256, 1)
    _step_and_norms(t)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _step_and_norms(t)
    for seed in (20, 40):
        new = _decode_inputs(5, 256, seed)
        for k in t:
            t[k].copy_(new[k])
        graph.replay()
        graph.replay()  # the state moves on
        want = [_step_and_norms(new) for _ in range(2)][1]
        torch.cuda.synchronize()
        assert torch.equal(t["state"], new["state"])
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_side_stream_while_the_default_one_is_busy():
    """Calls on a given stream order with that stream alone."""
    import torch
    import gated_delta_rule_87_b200 as gdr
    side = torch.cuda.Stream()
    x, g = _wide((2, 700, 192), 1, torch.bfloat16), _wide((2, 700, 192), 2, torch.float32).abs_().neg_()
    want = gdr.glr_scan_fwd(x, g)[:2]
    a = torch.randn((4096, 4096), device="cuda")
    h, final = torch.empty_like(x), torch.empty((2, 192), device="cuda")
    ws = torch.empty_like(gdr.glr_scan_fwd(x, g)[3])
    torch.cuda.synchronize()
    for _ in range(4):
        a = a @ a * 1e-3  # the default stream is busy
    gdr.glr_scan_fwd(x, g, h=h, final_state=final, workspace=ws, stream=side)
    y = torch.empty_like(x)
    gdr.gated_norm_fwd(h.view(1400, 3, 64), None, None, gate=None, eps=EPS, y=y.view(1400, 3, 64), stream=side)
    side.synchronize()
    assert torch.equal(h, want[0]) and torch.equal(final, want[1])
    assert torch.equal(y.view(1400, 3, 64), gdr.gated_norm_fwd(want[0].view(1400, 3, 64), None, None, gate=None, eps=EPS))


def test_one_workspace_for_calls_of_all_sizes_in_turn():
    """A workspace keeps nothing of the call before: longer, shorter, other widths, types and directions."""
    import torch
    import gated_delta_rule_87_b200 as gdr
    ws = torch.full((64 << 20,), 0xab, dtype=torch.uint8, device="cuda")
    for k, (B, T, D, io) in enumerate([(1, 9000, 70, torch.bfloat16), (3, 100, 512, torch.float32), (70, 1, 33, torch.bfloat16),
                                       (1, 9000, 70, torch.bfloat16), (2, 64, 64, torch.float32)]):
        x, g = _wide((B, T, D), k, io), _wide((B, T, D), k + 9, torch.float32).abs_().neg_()
        h, final, saved, _ = gdr.glr_scan_fwd(x, g, output_chunk_states=True, workspace=ws)
        dx, dg, dh0, _ = gdr.glr_scan_bwd(x, x, g, workspace=ws)
        other = gdr.glr_scan_fwd(x, g)
        again = gdr.glr_scan_bwd(x, x, g, chunk_states=saved)
        for a, b in zip((h, final, dx, dg, dh0), (*other[:2], *again[:3])):
            assert torch.equal(a, b)


def test_two_graphs_that_share_a_workspace_take_turns():
    import torch
    import gated_delta_rule_87_b200 as gdr
    ws = torch.empty(8 << 20, dtype=torch.uint8, device="cuda")
    sets = [(_wide((1, T, D), T, torch.bfloat16), _wide((1, T, D), T + 1, torch.float32).abs_().neg_())
            for T, D in ((3000, 64), (700, 200))]
    want = [gdr.glr_scan_fwd(x, g)[:2] for x, g in sets]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x, g in sets:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(gdr.glr_scan_fwd(x, g, workspace=ws)[:2])
    for _ in range(5):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert torch.equal(w[0], o[0]) and torch.equal(w[1], o[1])


@pytest.mark.parametrize("io,T", [("bf16", 64), ("bf16", 96), ("f32", 48), ("f32", 64)])
def test_sequences_of_whole_warps_in_a_pool(io, T):
    """Starts and ends on the first and last tokens of warps, a state read and
    written by different tiles; the gradients beside it."""
    import torch
    import gated_delta_rule_87_b200 as gdr
    N, D = 70, 192
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    x, dh = _wide((N, T, D), 1, dt), _wide((N, T, D), 2, dt)
    g, h0, df = _wide((N, T, D), 3, torch.float32).abs_().neg_(), _wide((N, D), 4, torch.float32), _wide((N, D), 5, torch.float32)
    offsets, flat = [T * n for n in range(N + 1)], lambda t: _host(t).reshape(-1, D)  # noqa: E731
    rh, rf, eh, ef = R.scan(flat(x), flat(g), _host(h0), offsets, False)
    slots = torch.randperm(N, device="cuda").to(torch.int32)
    for _ in range(5):
        pool = torch.empty_like(h0)
        pool[slots.long()] = h0
        h = gdr.glr_scan_fwd(x, g, state_pool=pool, state_slots=slots)[0]
        R.check(flat(h), rh, eh, io, "h")
        R.check(_host(pool[slots.long()]), rf, ef, "f32", "pool")
    dx, dg, dh0, _ = gdr.glr_scan_bwd(dh, x, g, h0, dfinal_state=df)
    want, err = R.scan_bwd(flat(dh), _host(df), flat(x), flat(g), _host(h0), offsets, False)
    for got, w, e, kind in zip((dx, dg, dh0), want, err, (io, "f32", "f32")):
        R.check(flat(got), w, e, kind)


def test_entries_that_share_a_slot_keep_to_their_own_results():
    """Two sequences of one call in one slot: each is right from the state that
    the slot held before, or from the other's; other slots keep theirs."""
    import torch
    import gated_delta_rule_87_b200 as gdr
    T, D = 70, 64
    x, g = _wide((3, T, D), 1, torch.float32), _wide((3, T, D), 2, torch.float32).abs_().neg_()
    pool = _wide((4, D), 3, torch.float32)
    before = pool.clone()
    slots = torch.tensor([2, 0, 2], dtype=torch.int32, device="cuda")
    h = gdr.glr_scan_fwd(x, g, state_pool=pool, state_slots=slots)[0]
    one = gdr.glr_scan_fwd(x[1:2], g[1:2], before[:1])
    torch.cuda.synchronize()
    assert torch.equal(pool[[1, 3]], before[[1, 3]])
    assert torch.allclose(h[1], one[0][0], rtol=1e-5, atol=1e-5) and torch.allclose(pool[0], one[1][0], rtol=1e-5, atol=1e-5)
    assert torch.isfinite(h).all()


@pytest.mark.parametrize("D", [2048, 2047])
def test_norms_in_place(D):
    """Every alias that the calls allow, rows that begin inside a 16-byte piece too."""
    import torch
    import gated_delta_rule_87_b200 as gdr
    M = 3000
    r, y, dn, dt = (_wide((M, D), s, torch.bfloat16) for s in (1, 2, 3, 4))
    w = _wide((D,), 5, torch.float32)
    t, n = gdr.add_norm_fwd(r, y, w, eps=EPS)
    r2, y2 = r.clone(), y.clone()
    gdr.add_norm_fwd(r2, y2, w, eps=EPS, residual_out=r2, n=y2)
    assert torch.equal(r2, t) and torch.equal(y2, n)
    d, _, dw, _, _ = gdr.add_norm_bwd(dn, dt, t, None, w, eps=EPS)
    for alias in ("dt", "t"):
        dt2, t2 = dt.clone(), t.clone()
        got = gdr.add_norm_bwd(dn, dt2, t2, None, w, eps=EPS, dresidual=dt2 if alias == "dt" else t2)
        assert torch.equal(got[0], d) and torch.equal(got[2], dw)
