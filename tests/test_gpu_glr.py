"""Gated linear recurrence on the GPU (scan, gradients, one-token step) against
its 64-bit form, element by element."""
import numpy as np
import pytest

import mixer_reference as R

pytestmark = pytest.mark.gpu


def _dt(io):
    import torch
    return torch.bfloat16 if io == "bf16" else torch.float32


def _dev(a, io="f32"):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda().to(_dt(io))


def _host(t):
    return t.float().cpu().numpy()


def _inputs(M, D, N, io, seed=0, pace=(-3, 0)):
    """x, g, h0, dh, dfinal as the device sees them (bf16 values where io says so)."""
    rng = np.random.default_rng([seed, M, D, N])
    n = lambda *s: rng.standard_normal(s)  # noqa: E731
    g = -10.0 ** rng.uniform(*pace, D) * np.log1p(np.exp(n(M, D)))
    t = dict(x=_dev(n(M, D), io), g=_dev(g), h0=_dev(n(N, D)), dh=_dev(n(M, D), io), df=_dev(n(N, D)))
    return t, {k: _host(v) for k, v in t.items()}


def _padded(shape, dtype):
    """A tensor inside a NaN-filled buffer: what is written beside it shows."""
    import torch
    n, pad = int(np.prod(shape)), 256
    buf = torch.full((n + 2 * pad,), float("nan"), dtype=dtype, device="cuda")
    return buf[pad:pad + n].view(shape), lambda: bool(torch.isnan(buf[:pad]).all() and torch.isnan(buf[pad + n:]).all())


def _run(B, T, D, io, complement=False, cu=None, seed=0, train=True, chunks=True, pace=(-3, 0)):
    """Scan and gradients of one set of inputs, every output checked."""
    import torch
    import gated_delta_rule_87_b200 as gdr
    M = B * T
    offsets = list(cu) if cu is not None else [T * b for b in range(B + 1)]
    N = len(offsets) - 1
    d, a = _inputs(M, D, N, io, seed, pace)
    gate = "complement" if complement else "given"
    cud = None if cu is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    b3 = lambda t: t.view(B, T, D)  # noqa: E731
    h, h_ok = _padded((B, T, D), _dt(io))
    final, final_ok = _padded((N, D), torch.float32)
    _, _, saved, ws = gdr.glr_scan_fwd(b3(d["x"]), b3(d["g"]), d["h0"], cud, input_gate=gate, h=h,
                                       final_state=final, output_chunk_states=chunks)
    torch.cuda.synchronize()
    assert gdr.check_device_status(ws) == (gdr.KDA_OK, gdr.KDA_DEVICE_OK)
    assert h_ok() and final_ok()
    rh, rf, eh, ef = R.scan(a["x"], a["g"], a["h0"], offsets, complement)
    R.check(_host(h), rh, eh, io, "h")
    R.check(_host(final), rf, ef, "f32", "final")
    if not train:
        return
    dx, dx_ok = _padded((B, T, D), _dt(io))
    dg, dg_ok = _padded((B, T, D), torch.float32)
    dh0, dh0_ok = _padded((N, D), torch.float32)
    _, _, _, ws = gdr.glr_scan_bwd(b3(d["dh"]), b3(d["x"]), b3(d["g"]), d["h0"], cud, input_gate=gate,
                                   dfinal_state=d["df"], chunk_states=saved, dx=dx, dg=dg, dinitial_state=dh0)
    torch.cuda.synchronize()
    assert gdr.check_device_status(ws) == (gdr.KDA_OK, gdr.KDA_DEVICE_OK)
    assert dx_ok() and dg_ok() and dh0_ok()
    want, err = R.scan_bwd(a["dh"], a["df"], a["x"], a["g"], a["h0"], offsets, complement)
    for got, w, e, kind, what in zip((dx, dg, dh0), want, err, (io, "f32", "f32"), ("dx", "dg", "dh0")):
        R.check(_host(got), w, e, kind, what)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("complement", [False, True])
@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 63, 64, 65, 127, 200])
def test_lengths(T, complement, io):
    _run(1, T, 70, io, complement, seed=T)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("D", [1, 2, 3, 31, 32, 33, 64, 65, 130, 192, 257])
def test_widths(D, io):
    _run(2, 75, D, io, seed=D)


@pytest.mark.parametrize("B,T", [(3, 1), (70, 1), (5, 3), (9, 64), (3, 100), (2, 700)])
def test_dense_batches(B, T):
    _run(B, T, 66, "bf16", seed=B)
    _run(B, T, 33, "f32", True, seed=B)


@pytest.mark.parametrize("cu", [
    [0, 0], [0, 1], [0, 0, 1, 1], [0, 64, 128], [0, 63, 64, 65, 65, 65, 130], [0, 5, 5, 300, 301, 301],
    [0, 0, 0, 700], list(range(0, 131)), [0, 1000],
])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_packed_sequences(cu, io):
    for D, complement in ((66, False), (35, True)):
        _run(1, cu[-1], D, io, complement, cu=cu, seed=len(cu))


@pytest.mark.parametrize("D", [40, 63])
def test_long_sequences_cross_many_chunks(D):
    """Long memories (decays of 1e-5 a token) over hundreds of chunks."""
    _run(1, 20000, D, "f32", seed=7, pace=(-5, -2))
    _run(1, 9000, D, "bf16", True, cu=[0, 4000, 4001, 9000], seed=8, pace=(-5, -2))


def test_wide_rows():
    _run(1, 600, 2050, "bf16", seed=9)
    _run(4, 130, 1024, "f32", True, seed=9)


def test_more_sequences_than_a_block_has_threads():
    rng = np.random.default_rng(3)
    cu = [0] + sorted(rng.integers(0, 2000, 1500).tolist()) + [2000]
    _run(1, 2000, 34, "bf16", cu=cu, seed=11)


@pytest.mark.parametrize("chunks", [True, False])
def test_gradients_without_saved_chunk_states(chunks):
    _run(1, 500, 48, "bf16", cu=[0, 120, 120, 500], chunks=chunks, seed=2)


def test_saved_chunk_states_are_the_states_that_enter():
    import torch
    import gated_delta_rule_87_b200 as gdr
    d, _ = _inputs(300, 40, 1, "f32")
    h, _, saved, _ = gdr.glr_scan_fwd(d["x"][None], d["g"][None], d["h0"], output_chunk_states=True)
    assert saved.shape == (5, 40)
    # h is the fp32 state itself here
    for k in range(1, 5):
        got, want = saved[k], h[0, 64 * k - 1]
        assert torch.allclose(got, want, rtol=1e-5, atol=1e-5)


@pytest.mark.parametrize("g", [0.0, -1e-8, -90.0, -1e30, float("-inf")])
def test_extreme_decays(g):
    """No decay at all; decays that underflow; -inf, which forgets what came before."""
    import torch
    import gated_delta_rule_87_b200 as gdr
    M, D = 150, 36
    d, a = _inputs(M, D, 1, "f32", seed=4)
    gd = d["g"].clone()
    gd[40:] = g
    ga = a["g"].copy()
    ga[40:] = g
    for complement in (False, True):
        gate = "complement" if complement else "given"
        h, final, saved, _ = gdr.glr_scan_fwd(d["x"][None], gd[None], d["h0"], input_gate=gate, output_chunk_states=True)
        dx, dg, dh0, _ = gdr.glr_scan_bwd(d["dh"][None], d["x"][None], gd[None], d["h0"], input_gate=gate,
                                          dfinal_state=d["df"], chunk_states=saved)
        rh, rf, eh, ef = R.scan(a["x"], ga, a["h0"], [0, M], complement)
        R.check(_host(h), rh, eh, "f32", "h")
        R.check(_host(final), rf, ef, "f32", "final")
        want, err = R.scan_bwd(a["dh"], a["df"], a["x"], ga, a["h0"], [0, M], complement)
        for got, w, e in zip((dx, dg, dh0), want, err):
            R.check(_host(got), w, e, "f32")


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_one_sequence_does_not_reach_another(bad):
    """Non-finite inputs, states and gradients of the middle sequence stay in it."""
    import torch
    import gated_delta_rule_87_b200 as gdr
    cu, D = [0, 90, 210, 400], 34
    d, a = _inputs(400, D, 3, "f32", seed=5)
    clean = {k: v.clone() for k, v in d.items()}
    d["x"][150], d["dh"][160], d["h0"][1], d["df"][1] = bad, bad, bad, bad
    cud = torch.tensor(cu, dtype=torch.int32, device="cuda")

    def call(t):
        h, final, saved, _ = gdr.glr_scan_fwd(t["x"][None], t["g"][None], t["h0"], cud, output_chunk_states=True)
        dx, dg, dh0, _ = gdr.glr_scan_bwd(t["dh"][None], t["x"][None], t["g"][None], t["h0"], cud,
                                          dfinal_state=t["df"], chunk_states=saved)
        return [h[0], dx[0], dg[0]], [final, dh0]

    (rows, states), (rows0, states0) = call(d), call(clean)
    for got, want in zip(rows, rows0):
        assert torch.equal(got[:90], want[:90]) and torch.equal(got[210:], want[210:])
        assert not torch.isfinite(got[90:210]).all()
    for got, want in zip(states, states0):
        assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])


def test_missing_states_are_zeros():
    import torch
    import gated_delta_rule_87_b200 as gdr
    d, a = _inputs(100, 20, 2, "f32")
    x, g, dh = (d[k].view(2, 50, 20) for k in ("x", "g", "dh"))
    h, final, saved, _ = gdr.glr_scan_fwd(x, g, output_final_state=False, output_chunk_states=True)
    assert final is None
    z = np.zeros((2, 20))
    rh, _, eh, _ = R.scan(a["x"], a["g"], z, [0, 50, 100], False)
    R.check(_host(h), rh, eh, "f32", "h")
    dx, dg, dh0, _ = gdr.glr_scan_bwd(dh, x, g, chunk_states=saved, output_dinitial_state=False)
    assert dh0 is None
    want, err = R.scan_bwd(a["dh"], z, a["x"], a["g"], z, [0, 50, 100], False)
    R.check(_host(dx), want[0], err[0], "f32", "dx")
    R.check(_host(dg), want[1], err[1], "f32", "dg")


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_slices_of_wider_rows(io):
    """x, g and dh as slices of wider projections, at an odd offset too."""
    import torch
    import gated_delta_rule_87_b200 as gdr
    B, T, D = 2, 70, 38
    d, a = _inputs(B * T, D, B, io, seed=6)
    for off in (0, 1, 2):
        def wide(t, extra):
            w = torch.full((B, T, D + extra), float("nan"), dtype=t.dtype, device="cuda")
            w[..., off:off + D] = t.view(B, T, D)
            return w[..., off:off + D]
        x, g, dh = wide(d["x"], 10), wide(d["g"], 4), wide(d["dh"], 7)
        assert not x.is_contiguous()
        h, final, saved, _ = gdr.glr_scan_fwd(x, g, d["h0"], output_chunk_states=True)
        rh, rf, eh, ef = R.scan(a["x"], a["g"], a["h0"], [0, T, 2 * T], False)
        R.check(_host(h), rh, eh, io, "h")
        R.check(_host(final), rf, ef, "f32", "final")
        dx, dg, dh0, _ = gdr.glr_scan_bwd(dh, x, g, d["h0"], dfinal_state=d["df"], chunk_states=saved)
        want, err = R.scan_bwd(a["dh"], a["df"], a["x"], a["g"], a["h0"], [0, T, 2 * T], False)
        for got, w, e, kind in zip((dx, dg, dh0), want, err, (io, "f32", "f32")):
            R.check(_host(got), w, e, kind)


@pytest.mark.parametrize("T", [1, 4, 64, 200])
def test_state_pool_in_place(T):
    import torch
    import gated_delta_rule_87_b200 as gdr
    N, D, slots = 5, 44, [6, 2, -1, 0, 9]  # -1 and 9: no slot in a pool of 8
    d, a = _inputs(N * T, D, N, "bf16", seed=T)
    pool0 = _dev(np.random.default_rng(1).standard_normal((8, D)))
    pool = pool0.clone()
    h0 = np.stack([_host(pool0)[s] if 0 <= s < 8 else np.zeros(D, np.float32) for s in slots])
    h, fin, _, _ = gdr.glr_scan_fwd(d["x"].view(N, T, D), d["g"].view(N, T, D), state_pool=pool,
                                    state_slots=torch.tensor(slots, dtype=torch.int32, device="cuda"))
    assert fin is pool
    rh, rf, eh, ef = R.scan(a["x"], a["g"], h0, [T * n for n in range(N + 1)], False)
    R.check(_host(h), rh, eh, "bf16", "h")
    for n, s in enumerate(slots):
        if 0 <= s < 8:
            R.check(_host(pool)[s], rf[n], ef[n], "f32", f"slot {s}")
    rest = [s for s in range(8) if s not in slots]
    assert torch.equal(pool[rest], pool0[rest])


def test_many_sequences_over_many_tiles_in_place():
    """A sequence's last tile writes the slot that its first tile reads."""
    import torch
    import gated_delta_rule_87_b200 as gdr
    N, T, D = 60, 70, 256
    d, a = _inputs(N * T, D, N, "f32", seed=21)
    rh, rf, eh, ef = R.scan(a["x"], a["g"], a["h0"], [T * n for n in range(N + 1)], False)
    slots = torch.randperm(N, device="cuda").to(torch.int32)
    for _ in range(20):
        pool = torch.empty((N, D), device="cuda")
        pool[slots.long()] = d["h0"]
        h, _, _, _ = gdr.glr_scan_fwd(d["x"].view(N, T, D), d["g"].view(N, T, D), state_pool=pool, state_slots=slots)
        R.check(_host(h), rh, eh, "f32", "h")
        R.check(_host(pool[slots.long()]), rf, ef, "f32", "pool")


def test_empty_sequences_in_a_pool_leave_their_slots():
    import torch
    import gated_delta_rule_87_b200 as gdr
    d, _ = _inputs(70, 16, 1, "f32")
    pool = torch.randn((4, 16), device="cuda")
    before = pool.clone()
    cu = torch.tensor([0, 0, 70, 70], dtype=torch.int32, device="cuda")
    gdr.glr_scan_fwd(d["x"][None], d["g"][None], cu_seqlens=cu, state_pool=pool,
                     state_slots=torch.tensor([3, 1, 0], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(pool[[0, 2, 3]], before[[0, 2, 3]]) and not torch.equal(pool[1], before[1])


@pytest.mark.parametrize("cu", [None, [0, 0, 0]])
def test_no_tokens(cu):
    import torch
    import gated_delta_rule_87_b200 as gdr
    B = 2 if cu is None else 1
    x, g = torch.zeros((B, 0, 24), dtype=torch.bfloat16, device="cuda"), torch.zeros((B, 0, 24), device="cuda")
    cud = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    h0, df = torch.randn((2, 24), device="cuda"), torch.randn((2, 24), device="cuda")
    h, final, saved, _ = gdr.glr_scan_fwd(x, g, h0, cud, output_chunk_states=True)
    dx, dg, dh0, _ = gdr.glr_scan_bwd(x, x, g, h0, cud, dfinal_state=df, chunk_states=saved)
    torch.cuda.synchronize()
    assert h.shape == dx.shape == dg.shape == (B, 0, 24)
    assert torch.equal(final, h0) and torch.equal(dh0, df)


@pytest.mark.parametrize("cu", [[1, 100], [0, 60, 40, 100], [0, 99], [0, 101], [0, -5, 100]])
def test_bad_offsets_leave_the_outputs_unwritten(cu):
    import torch
    import gated_delta_rule_87_b200 as gdr
    d, _ = _inputs(100, 20, len(cu) - 1, "f32")
    cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
    full = lambda *s: torch.full(s, 7.0, device="cuda")  # noqa: E731
    h, final, dx, dg, dh0 = full(1, 100, 20), full(len(cu) - 1, 20), full(1, 100, 20), full(1, 100, 20), full(len(cu) - 1, 20)
    _, _, _, ws = gdr.glr_scan_fwd(d["x"][None], d["g"][None], d["h0"], cud, h=h, final_state=final)
    assert gdr.check_device_status(ws) == (gdr.KDA_ERR_DEVICE_CHECK, gdr.KDA_DEVICE_BAD_CU_SEQLENS)
    _, _, _, ws = gdr.glr_scan_bwd(d["dh"][None], d["x"][None], d["g"][None], d["h0"], cud, dx=dx, dg=dg, dinitial_state=dh0)
    assert gdr.check_device_status(ws) == (gdr.KDA_ERR_DEVICE_CHECK, gdr.KDA_DEVICE_BAD_CU_SEQLENS)
    for t in (h, final, dx, dg, dh0):
        assert bool((t == 7.0).all())
    # the same workspace serves the next call
    _, _, _, ws = gdr.glr_scan_fwd(d["x"][None], d["g"][None], d["h0"][:1], h=h, workspace=ws)
    assert gdr.check_device_status(ws) == (gdr.KDA_OK, gdr.KDA_DEVICE_OK)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("complement", [False, True])
@pytest.mark.parametrize("N,D", [(1, 1), (3, 33), (7, 64), (300, 130), (2, 1026)])
def test_step(N, D, complement, io):
    import torch
    import gated_delta_rule_87_b200 as gdr
    gate = "complement" if complement else "given"
    d, a = _inputs(N, D, N, io, seed=N)
    state = d["h0"].clone()
    h = gdr.glr_step(d["x"], d["g"], state, input_gate=gate)
    rh, rf, eh, ef = R.scan(a["x"], a["g"], a["h0"], list(range(N + 1)), complement)
    R.check(_host(h), rh, eh, io, "h")
    R.check(_host(state), rf, ef, "f32", "state")


def test_step_in_a_pool_with_padding_entries():
    import torch
    import gated_delta_rule_87_b200 as gdr
    N, D, slots = 6, 50, [4, -1, 0, 7, 2, -9]
    d, a = _inputs(N, D, N, "bf16")
    pool0 = torch.randn((6, D), device="cuda")
    pool, wide = pool0.clone(), torch.full((N, 2 * D), float("nan"), device="cuda")
    wide[:, D:] = d["g"]
    h = gdr.glr_step(d["x"], wide[:, D:], pool, state_slots=torch.tensor(slots, dtype=torch.int32, device="cuda"))
    live = [n for n, s in enumerate(slots) if 0 <= s < 6]
    at = [slots[n] for n in live]
    rh, rf, eh, ef = R.scan(a["x"][live], a["g"][live], _host(pool0)[at], list(range(len(live) + 1)), False)
    R.check(_host(h)[live], rh, eh, "bf16", "h")
    R.check(_host(pool)[at], rf, ef, "f32", "pool")
    assert bool((h[[1, 3, 5]] == 0).all())
    rest = [s for s in range(6) if s not in at]
    assert torch.equal(pool[rest], pool0[rest])


def test_steps_continue_a_scan():
    """Prefill into a pool, then token by token from it: one sequence of states."""
    import torch
    import gated_delta_rule_87_b200 as gdr
    N, T, D = 3, 90, 32
    d, a = _inputs(N * T, D, N, "f32", seed=3)
    x, g = d["x"].view(N, T, D), d["g"].view(N, T, D)
    pool = torch.zeros((4, D), device="cuda")
    slots = torch.tensor([3, 0, 2], dtype=torch.int32, device="cuda")
    pool[slots.long()] = d["h0"]
    h, _, _, _ = gdr.glr_scan_fwd(x[:, :70].contiguous(), g[:, :70].contiguous(), state_pool=pool, state_slots=slots)
    out = [h]
    for t in range(70, T):
        out.append(gdr.glr_step(x[:, t], g[:, t], pool, state_slots=slots)[:, None])
    rh, rf, eh, ef = R.scan(a["x"], a["g"], a["h0"], [0, T, 2 * T, 3 * T], False)
    R.check(_host(torch.cat(out, 1)).reshape(N * T, D), rh, eh, "f32", "h")
    R.check(_host(pool[slots.long()]), rf, ef, "f32", "state")


def test_same_inputs_same_bits():
    import torch
    import gated_delta_rule_87_b200 as gdr
    d, _ = _inputs(30000, 70, 3, "bf16", seed=12)
    cu = torch.tensor([0, 100, 29000, 30000], dtype=torch.int32, device="cuda")

    def call():
        h, f, s, _ = gdr.glr_scan_fwd(d["x"][None], d["g"][None], d["h0"], cu, output_chunk_states=True)
        return [h, f, s, *gdr.glr_scan_bwd(d["dh"][None], d["x"][None], d["g"][None], d["h0"], cu,
                                           dfinal_state=d["df"], chunk_states=s)[:3]]

    first = call()
    for _ in range(5):
        assert all(torch.equal(p, q) for p, q in zip(first, call()))


def test_two_streams_at_once():
    import torch
    import gated_delta_rule_87_b200 as gdr
    sets = [_inputs(8000, 96, 1, "bf16", seed=s)[0] for s in (1, 2)]
    one = lambda d: gdr.glr_scan_fwd(d["x"][None], d["g"][None], d["h0"])[:2]  # noqa: E731
    want = [one(d) for d in sets]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in sets], [[], []]
    for _ in range(10):
        for k, (d, s) in enumerate(zip(sets, streams)):
            with torch.cuda.stream(s):
                got[k].append(one(d))
    torch.cuda.synchronize()
    for w, many in zip(want, got):
        for g in many:
            assert torch.equal(w[0], g[0]) and torch.equal(w[1], g[1])


def test_captured_training_step_replays_on_new_inputs():
    import torch
    import gated_delta_rule_87_b200 as gdr
    d, _ = _inputs(3000, 64, 2, "bf16", seed=1)
    cu = torch.tensor([0, 1111, 3000], dtype=torch.int32, device="cuda")

    def call(t):
        h, f, s, _ = gdr.glr_scan_fwd(t["x"][None], t["g"][None], t["h0"], cu, output_chunk_states=True)
        return [h, f, *gdr.glr_scan_bwd(t["dh"][None], t["x"][None], t["g"][None], t["h0"], cu,
                                        dfinal_state=t["df"], chunk_states=s)[:3]]

    call(d)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(d)
    for seed in (2, 3):
        new, _ = _inputs(3000, 64, 2, "bf16", seed=seed)
        want = call(new)
        for k in d:
            d[k].copy_(new[k])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want))


def test_binding_refusals():
    import torch
    import gated_delta_rule_87_b200 as gdr
    x, g = torch.zeros((2, 5, 8), device="cuda"), torch.zeros((2, 5, 8), device="cuda")
    st = torch.zeros((2, 8), device="cuda")
    bad = [
        lambda: gdr.glr_scan_fwd(x.double(), g),
        lambda: gdr.glr_scan_fwd(x, g.bfloat16()),
        lambda: gdr.glr_scan_fwd(x, g[:, :4]),
        lambda: gdr.glr_scan_fwd(x[0], g[0]),
        lambda: gdr.glr_scan_fwd(x, g.cpu()),
        lambda: gdr.glr_scan_fwd(x.transpose(0, 1), g.transpose(0, 1)),       # uneven leading axes
        lambda: gdr.glr_scan_fwd(x.transpose(1, 2), g.transpose(1, 2)),       # channels not contiguous
        lambda: gdr.glr_scan_fwd(x[:, :1].expand(2, 5, 8), g),                # rows that overlap
        lambda: gdr.glr_scan_fwd(x, g, st[:1]),
        lambda: gdr.glr_scan_fwd(x, g, input_gate="sqrt"),
        lambda: gdr.glr_scan_fwd(x, g, st, state_pool=st, state_slots=torch.zeros(2, dtype=torch.int32, device="cuda")),
        lambda: gdr.glr_scan_fwd(x, g, cu_seqlens=torch.tensor([0, 5], dtype=torch.int32, device="cuda")),  # B = 2
        lambda: gdr.glr_scan_fwd(x, g, cu_seqlens=torch.tensor([0, 10], device="cuda")),                   # int64
        lambda: gdr.glr_scan_fwd(x, g, h=x),
        lambda: gdr.glr_scan_fwd(x, g, h=torch.empty((2, 5, 8), dtype=torch.bfloat16, device="cuda")),
        lambda: gdr.glr_scan_bwd(x.bfloat16(), x, g),
        lambda: gdr.glr_scan_bwd(x, x, g, chunk_states=torch.zeros((2, 8), device="cuda")),
        lambda: gdr.glr_scan_bwd(torch.zeros_like(x), x, g, dx=x),
        lambda: gdr.glr_step(x, g, st),
        lambda: gdr.glr_step(x[:, 0], g[:, 0], st[:1]),
        lambda: gdr.glr_step(x[:, 0], g[:, 0], st.cpu()),
        lambda: gdr.glr_step(x[:, 0], g[:, 0], st, state_slots=torch.zeros(3, dtype=torch.int32, device="cuda")),
    ]
    for call in bad:
        with pytest.raises((ValueError, TypeError, gdr.KdaError)):
            call()


@pytest.mark.parametrize("fn,kw", [
    (test_lengths, dict(T=65, complement=True, io="bf16")),
    (test_widths, dict(D=65, io="f32")), (test_widths, dict(D=130, io="bf16")),
    (test_dense_batches, dict(B=3, T=100)),
    (test_packed_sequences, dict(cu=[0, 5, 5, 300, 301, 301], io="bf16")),
    (test_more_sequences_than_a_block_has_threads, {}),
    (test_long_sequences_cross_many_chunks, dict(D=40)),
    (test_state_pool_in_place, dict(T=200)), (test_slices_of_wider_rows, dict(io="bf16")),
    (test_gradients_without_saved_chunk_states, dict(chunks=False)),
    (test_step, dict(N=7, D=64, complement=False, io="bf16")),
    (test_step_in_a_pool_with_padding_entries, {}), (test_no_tokens, dict(cu=[0, 0, 0])),
], ids=lambda v: v.__name__ if callable(v) else "-".join(map(str, v.values())))
def test_checked_build_finds_no_access_out_of_bounds(fn, kw):
    import gated_delta_rule_87_b200 as gdr
    with gdr.use_library(gdr.checked_library_path):
        gdr.bounds_violations()
        fn(**kw)
        assert gdr.bounds_violations() == 0
