"""Refusals of the gated linear recurrence and of the norms at the C boundary:
checked on the host, before the device is touched (no GPU needed)."""
import pytest

import gated_delta_rule_87_b200 as gdr

FAKE = 0x10000  # never dereferenced: every call below fails validation first
ARG, UNSUPPORTED, WORKSPACE = gdr.KDA_ERR_INVALID_ARG, gdr.KDA_ERR_UNSUPPORTED, gdr.KDA_ERR_WORKSPACE


def _fwd(**over):
    kw = dict(x=FAKE, ld_x=8, g=FAKE + 4096, ld_g=8, h=FAKE + 8192, h0=None, hT=None, slots=None, num_slots=0,
              chunks=None, cu=None, n=0, B=1, T=64, D=8, input=0, io=1, ws=FAKE, ws_bytes=1 << 20)
    kw.update(over)
    return gdr.lib().glr_scan_fwd(*kw.values(), None)


@pytest.mark.parametrize("over,status", [
    (dict(x=None), ARG), (dict(g=None), ARG), (dict(h=None), ARG),
    (dict(x=FAKE + 1), ARG), (dict(g=FAKE + 2), ARG), (dict(h=FAKE + 1), ARG), (dict(h0=FAKE + 2), ARG),
    (dict(io=0, x=FAKE + 2), ARG), (dict(hT=FAKE + 1), ARG), (dict(chunks=FAKE + 1), ARG),
    (dict(ld_x=7), ARG), (dict(ld_g=-8), ARG),
    (dict(h=FAKE), ARG), (dict(h=FAKE + 4096), ARG),  # h aliases x, g
    (dict(B=0), ARG), (dict(T=-1), ARG), (dict(D=0), ARG), (dict(B=70000, T=70000), ARG),
    (dict(input=2), ARG), (dict(input=-1), ARG), (dict(io=5), ARG),
    (dict(slots=FAKE, num_slots=-1), ARG), (dict(slots=FAKE + 1, num_slots=2), ARG),
    (dict(cu=FAKE, n=2, B=2), ARG), (dict(cu=FAKE, n=-1), ARG), (dict(cu=FAKE + 2, n=2), ARG),
    (dict(ws=None), WORKSPACE), (dict(ws=FAKE + 16), WORKSPACE), (dict(ws_bytes=255), WORKSPACE),
])
def test_scan_refusals(over, status):
    assert _fwd(**over) == status
    assert gdr.lib().kda_last_error()


def _bwd(**over):
    kw = dict(dh=FAKE, ld_dh=8, df=None, x=FAKE + 4096, ld_x=8, g=FAKE + 8192, ld_g=8, h0=None, chunks=None,
              dx=FAKE + 12288, dg=FAKE + 16384, dh0=None, cu=None, n=0, B=1, T=64, D=8, input=0, io=1, ws=FAKE,
              ws_bytes=1 << 20)
    kw.update(over)
    return gdr.lib().glr_scan_bwd(*kw.values(), None)


@pytest.mark.parametrize("over,status", [
    (dict(dh=None), ARG), (dict(x=None), ARG), (dict(g=None), ARG), (dict(dx=None), ARG), (dict(dg=None), ARG),
    (dict(ld_dh=4), ARG), (dict(dh=FAKE + 1), ARG), (dict(df=FAKE + 2), ARG), (dict(dh0=FAKE + 2), ARG),
    (dict(dx=FAKE), ARG), (dict(dg=FAKE + 8192), ARG), (dict(dx=FAKE + 4096), ARG),  # aliases
    (dict(h0=FAKE, dh0=FAKE), ARG), (dict(df=FAKE, dh0=FAKE), ARG),
    (dict(input=3), ARG), (dict(io=2), ARG), (dict(D=-1), ARG), (dict(cu=FAKE, n=1, B=3), ARG),
    (dict(ws=None), WORKSPACE), (dict(ws=FAKE + 128), WORKSPACE), (dict(ws_bytes=0), WORKSPACE),
])
def test_scan_gradient_refusals(over, status):
    assert _bwd(**over) == status
    assert gdr.lib().kda_last_error()


def test_scan_workspace_sizes():
    L = gdr.lib()
    assert L.glr_chunk_states_size(1, 64, 8) == 32 and L.glr_chunk_states_size(1, 65, 8) == 64
    assert L.glr_chunk_states_size(2, 0, 8) == 0
    for size in (L.glr_scan_fwd_workspace_size, lambda *a: L.glr_scan_bwd_workspace_size(*a, 1)):
        assert size(0, 64, 8) == 0 and size(1, 64, 0) == 0
        assert 256 <= size(1, 64, 8) <= size(1, 4096, 8) <= size(1, 4096, 80)
        assert size(1, 2 ** 31 - 1, 8192) > 2 ** 36  # no 32-bit arithmetic
    assert L.glr_scan_bwd_workspace_size(1, 4096, 80, 0) > L.glr_scan_bwd_workspace_size(1, 4096, 80, 1)


def test_scans_refuse_more_tiles_than_a_grid_holds():
    big = dict(B=1, T=2 ** 31 - 1, D=2 ** 20, ld_x=2 ** 20, ld_g=2 ** 20, ws_bytes=2 ** 62)
    assert _fwd(**big) == UNSUPPORTED and _bwd(**big, ld_dh=2 ** 20) == UNSUPPORTED


def _step(x=FAKE, ld_x=8, g=FAKE + 4096, ld_g=8, h=FAKE + 8192, state=FAKE + 12288, slots=None, num_slots=0, N=4,
          D=8, input=0, io=1):
    return gdr.lib().glr_step(x, ld_x, g, ld_g, h, state, slots, num_slots, N, D, input, io, None)


@pytest.mark.parametrize("over,status", [
    (dict(x=None), ARG), (dict(g=None), ARG), (dict(h=None), ARG), (dict(state=None), ARG),
    (dict(ld_x=0), ARG), (dict(ld_g=7), ARG), (dict(h=FAKE), ARG), (dict(h=FAKE + 12288), ARG),
    (dict(state=FAKE + 2), ARG), (dict(slots=FAKE, num_slots=-1), ARG), (dict(slots=FAKE + 3, num_slots=1), ARG),
    (dict(N=-1), ARG), (dict(D=0), ARG), (dict(input=9), ARG), (dict(io=9), ARG), (dict(io=0, x=FAKE + 2), ARG),
    (dict(N=0, x=None), gdr.KDA_OK),
])
def test_step_refusals(over, status):
    assert _step(**over) == status


def _gated(**over):
    kw = dict(x=FAKE, ld_x=128, z=FAKE, ld_z=128, w=None, y=FAKE + 4096, tokens=4, H=2, d=64, eps=1e-6, gate=1, io=1)
    kw.update(over)
    return gdr.lib().kda_gated_norm_fwd(*kw.values(), None)


@pytest.mark.parametrize("over,status", [
    (dict(x=None), ARG), (dict(z=None), ARG), (dict(y=None), ARG), (dict(ld_x=127), ARG), (dict(ld_z=64), ARG),
    (dict(w=FAKE + 1), ARG), (dict(x=FAKE + 1), ARG), (dict(y=FAKE + 1), ARG), (dict(tokens=-1), ARG),
    (dict(H=0), ARG), (dict(d=0), ARG), (dict(d=16385, H=1, ld_x=20000, ld_z=20000), UNSUPPORTED),
    (dict(tokens=2 ** 31, H=1), ARG), (dict(tokens=2 ** 30, H=4), ARG),
    (dict(eps=0.0), ARG), (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG), (dict(eps=float("inf")), ARG),
    (dict(gate=3), ARG), (dict(gate=-1), ARG), (dict(io=3), ARG), (dict(tokens=0, x=None), gdr.KDA_OK),
])
def test_gated_norm_refusals(over, status):
    assert _gated(**over) == status


@pytest.mark.parametrize("over,status", [
    (dict(dy=None), ARG), (dict(dx=None), ARG), (dict(dz=None), ARG), (dict(ld_dy=1), ARG), (dict(dw=FAKE + 2), ARG),
    (dict(ws=None), WORKSPACE), (dict(ws=FAKE + 8), WORKSPACE), (dict(ws_bytes=1024), WORKSPACE),
])
def test_gated_norm_gradient_refusals(over, status):
    kw = dict(dy=FAKE, ld_dy=128, x=FAKE, ld_x=128, z=FAKE, ld_z=128, w=FAKE, dx=FAKE, dz=FAKE, dw=FAKE, tokens=4,
              H=2, d=64, eps=1e-6, gate=1, io=1, ws=FAKE, ws_bytes=1 << 30)
    kw.update(over)
    assert gdr.lib().kda_gated_norm_bwd(*kw.values(), None) == status


@pytest.mark.parametrize("over,status", [
    (dict(r=None), ARG), (dict(y=None), ARG), (dict(out=None), ARG), (dict(n=None), ARG),
    (dict(n=FAKE), ARG), (dict(n=FAKE + 8192), ARG), (dict(out=FAKE + 4096), ARG),  # aliases
    (dict(r=FAKE + 1), ARG), (dict(w=FAKE + 2), ARG), (dict(rows=-1), ARG), (dict(rows=2 ** 31), ARG),
    (dict(D=0), ARG), (dict(D=16385), UNSUPPORTED), (dict(eps=0.0), ARG), (dict(res=1, io=0), UNSUPPORTED),
    (dict(res=4), ARG), (dict(rows=0, r=None), gdr.KDA_OK),
])
def test_add_norm_refusals(over, status):
    kw = dict(r=FAKE, y=FAKE + 4096, s=None, w=None, out=FAKE + 8192, n=FAKE + 12288, rows=4, D=64, eps=1e-6, res=0, io=1)
    kw.update(over)
    assert gdr.lib().kda_add_norm_fwd(*kw.values(), None) == status


@pytest.mark.parametrize("over,status", [
    (dict(dn=None), ARG), (dict(out=None), ARG), (dict(d=None), ARG), (dict(y=None), ARG), (dict(s=None), ARG),
    (dict(dy=FAKE + 4096), ARG), (dict(ws=None), WORKSPACE), (dict(ws=FAKE + 32), WORKSPACE),
    (dict(ws_bytes=4096), WORKSPACE), (dict(res=1, io=0), UNSUPPORTED), (dict(ds=FAKE + 1), ARG),
])
def test_add_norm_gradient_refusals(over, status):
    kw = dict(dn=FAKE, dt=None, out=FAKE, y=FAKE, s=FAKE, w=None, d=FAKE + 4096, dy=FAKE + 8192, ds=FAKE, dw=FAKE,
              rows=4, D=64, eps=1e-6, res=0, io=1, ws=FAKE, ws_bytes=1 << 30)
    kw.update(over)
    assert gdr.lib().kda_add_norm_bwd(*kw.values(), None) == status


def test_norm_workspace_sizes():
    L = gdr.lib()
    assert L.kda_gated_norm_bwd_workspace_size(0) == 0 and L.kda_add_norm_bwd_workspace_size(-3) == 0
    assert 0 < L.kda_gated_norm_bwd_workspace_size(64) < L.kda_add_norm_bwd_workspace_size(64)
