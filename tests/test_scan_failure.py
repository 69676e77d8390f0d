"""A wait in a scan's chain that nothing ends: it expires after its bound, the
status word says so after the whole call, and the context stays usable."""
import pytest

import gated_delta_rule_87_b200 as gdr

FAKE = 0x10000  # never dereferenced


@pytest.mark.parametrize("over,status", [
    (dict(T=1024), gdr.KDA_ERR_INVALID_ARG), (dict(out=None), gdr.KDA_ERR_INVALID_ARG),
    (dict(dg=None), gdr.KDA_ERR_INVALID_ARG), (dict(x=None), gdr.KDA_ERR_INVALID_ARG),
    (dict(D=0), gdr.KDA_ERR_INVALID_ARG), (dict(ws=None), gdr.KDA_ERR_WORKSPACE),
    (dict(ws_bytes=1024), gdr.KDA_ERR_WORKSPACE),
])
def test_selftest_refusals(over, status):
    kw = dict(backward=1, x=FAKE, g=FAKE, out=FAKE, dg=FAKE, T=2000, D=8, ws=FAKE, ws_bytes=1 << 20)
    kw.update(over)
    assert gdr.lib().glr_selftest_wait_timeout(*kw.values(), None) == status


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 100, 33])
@pytest.mark.parametrize("backward", [0, 1])
def test_an_expired_wait_in_the_chain_is_reported(backward, D):
    """Backward, the wait is one of the first of the call's two passes."""
    import torch
    L, T = gdr.lib(), 5000
    x, g = torch.randn((1, T, D), device="cuda"), -torch.rand((1, T, D), device="cuda")
    out, dg = torch.full_like(x, 7.0), torch.full_like(x, 7.0)
    ws = torch.zeros(L.glr_scan_bwd_workspace_size(1, T, D, 0), dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    for _ in range(2):
        assert L.glr_selftest_wait_timeout(backward, x.data_ptr(), g.data_ptr(), out.data_ptr(), dg.data_ptr(), T, D,
                                           ws.data_ptr(), ws.numel(), stream) == gdr.KDA_OK
        assert gdr.check_device_status(ws) == (gdr.KDA_ERR_DEVICE_CHECK, gdr.KDA_DEVICE_TIMEOUT)
        assert bool((out == 7).all()) and bool((dg == 7).all())
    # the same workspace serves the next call, whose status is its own
    if backward:
        got, want = gdr.glr_scan_bwd(x, x, g, workspace=ws), gdr.glr_scan_bwd(x, x, g)
    else:
        got, want = gdr.glr_scan_fwd(x, g, workspace=ws), gdr.glr_scan_fwd(x, g)
    assert got[-1] is ws and gdr.check_device_status(ws) == (gdr.KDA_OK, gdr.KDA_DEVICE_OK)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.gpu
def test_bad_offsets_are_reported_by_a_gradient_of_two_passes():
    import torch
    x, g = torch.randn((1, 300, 64), device="cuda"), -torch.rand((1, 300, 64), device="cuda")
    for cu in ([0, 200, 100, 300], [1, 300], [0, 299]):
        dx = torch.full_like(x, 7.0)
        cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
        ws = gdr.glr_scan_bwd(x, x, g, None, cud, dx=dx)[3]
        assert gdr.check_device_status(ws) == (gdr.KDA_ERR_DEVICE_CHECK, gdr.KDA_DEVICE_BAD_CU_SEQLENS)
        assert bool((dx == 7).all())


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [0x7fffffff, 0x7ffffffe, 0x7fc00000, -1, -2, -0x400000, -0x800000, 0x7f800000])
def test_decays_that_are_not_numbers_stall_nothing(bits):
    """NaN of every sign and payload, and infinities, in one channel of one
    sequence: the chain goes on, other channels and sequences keep their values."""
    import torch
    T, D, c = 6000, 70, 5
    for dt in (torch.float32, torch.bfloat16):
        x, g = torch.randn((1, T, D), device="cuda").to(dt), -torch.rand((1, T, D), device="cuda")
        cu = torch.tensor([0, 300, 4500, T], dtype=torch.int32, device="cuda")
        clean = (*gdr.glr_scan_fwd(x, g, None, cu)[:1], *gdr.glr_scan_bwd(x, x, g, None, cu)[:2])
        g.view(torch.int32)[0, 400:4400, c] = bits
        h, _, _, ws = gdr.glr_scan_fwd(x, g, None, cu)
        assert gdr.check_device_status(ws) == (gdr.KDA_OK, gdr.KDA_DEVICE_OK)
        dx, dg, _, ws = gdr.glr_scan_bwd(x, x, g, None, cu)
        assert gdr.check_device_status(ws) == (gdr.KDA_OK, gdr.KDA_DEVICE_OK)
        keep = torch.ones((T, D), dtype=torch.bool, device="cuda")
        keep[300:4500, c] = False
        for got, want in zip((h, dx, dg), clean):
            assert torch.equal(got[0][keep], want[0][keep])
        if bits != -0x800000:  # (-inf forgets)
            assert not bool(torch.isfinite(h[0, 4000, c].float()))
        else:
            assert torch.equal(h[0, 400:4400, c], x[0, 400:4400, c])
