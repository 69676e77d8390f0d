"""Outputs of the gated norm in the buffers of its inputs: allowed where rows lie
alike, refused where they do not."""
import pytest

import gated_delta_rule_87_b200 as gdr

FAKE = 0x10000  # never dereferenced
ARG = gdr.KDA_ERR_INVALID_ARG


@pytest.mark.parametrize("over", [dict(y=FAKE, ld_x=200), dict(y=FAKE + 4096, ld_z=136)])
def test_forward_refuses_a_shared_buffer_of_wider_rows(over):
    kw = dict(x=FAKE, ld_x=128, z=FAKE + 4096, ld_z=128, w=None, y=FAKE + 8192, tokens=4, H=2, d=64, eps=1e-6, gate=1, io=1)
    kw.update(over)
    assert gdr.lib().kda_gated_norm_fwd(*kw.values(), None) == ARG
    assert b"buffer" in gdr.lib().kda_last_error()


@pytest.mark.parametrize("over", [dict(dx=FAKE, ld_dy=200), dict(dz=FAKE + 4096, ld_x=200), dict(dx=FAKE + 8192, ld_z=200),
                                  dict(dx=FAKE + 12288, dz=FAKE + 12288)])
def test_gradient_refuses_buffers_that_it_would_overwrite(over):
    kw = dict(dy=FAKE, ld_dy=128, x=FAKE + 4096, ld_x=128, z=FAKE + 8192, ld_z=128, w=None, dx=FAKE + 12288, dz=FAKE + 16384,
              dw=None, tokens=4, H=2, d=64, eps=1e-6, gate=1, io=1, ws=None, ws_bytes=0)
    kw.update(over)
    assert gdr.lib().kda_gated_norm_bwd(*kw.values(), None) == ARG
    assert b"buffer" in gdr.lib().kda_last_error()


def test_gradient_of_one_token_refuses_one_buffer_for_two_outputs():
    assert gdr.lib().kda_gated_norm_bwd(FAKE, 128, FAKE + 4096, 128, FAKE + 8192, 128, None, FAKE + 12288, FAKE + 12288, None,
                                        1, 2, 64, 1e-6, 1, 1, None, 0, None) == ARG


@pytest.mark.gpu
def test_one_token_in_place_at_any_pitch():
    """The distance between tokens is of no account where there is one."""
    import torch
    x, z = (torch.randn((1, 2, 64), device="cuda") for _ in range(2))
    want = gdr.gated_norm_fwd(x, z)
    st = gdr.lib().kda_gated_norm_fwd(x.data_ptr(), 200, z.data_ptr(), 300, None, x.data_ptr(), 1, 2, 64, 1e-6, 1, 0,
                                      torch.cuda.current_stream().cuda_stream)
    assert st == gdr.KDA_OK and torch.allclose(x, want, rtol=1e-5, atol=1e-6)


def test_scan_gradient_refuses_one_buffer_for_two_outputs():
    kw = dict(dh=FAKE, ld_dh=8, df=None, x=FAKE + 4096, ld_x=8, g=FAKE + 8192, ld_g=8, h0=None, chunks=None, dx=FAKE + 12288,
              dg=FAKE + 12288, dh0=None, cu=None, n=0, B=1, T=64, D=8, input=0, io=0, ws=FAKE, ws_bytes=1 << 20)
    assert gdr.lib().glr_scan_bwd(*kw.values(), None) == ARG


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("M,H,d", [(3000, 4, 128), (3000, 4, 100), (900, 2, 333), (700, 1, 4096), (300, 1, 8199)])
def test_gated_norm_in_place(M, H, d, io):
    import torch
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    x, z, dy = (torch.randn((M, H, d), device="cuda").to(dt) for _ in range(3))
    w = torch.randn(d, device="cuda")
    want = gdr.gated_norm_fwd(x, z, w)
    for k in range(2):
        t = [x.clone(), z.clone()]
        assert torch.equal(gdr.gated_norm_fwd(*t, w, y=t[k]), want)
    want = gdr.gated_norm_bwd(dy, x, z, w)[:3]
    for i, j in ((0, 1), (1, 2), (2, 0)):
        t = [dy.clone(), x.clone(), z.clone()]
        got = gdr.gated_norm_bwd(*t, w, dx=t[i], dz=t[j])[:3]
        assert all(torch.equal(p, q) for p, q in zip(got, want))
