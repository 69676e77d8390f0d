"""Kernels that start while the one before them ends read what that one writes:
calls in quick turns on one workspace, each with other marks or partial sums."""
import pytest

pytestmark = pytest.mark.gpu


def test_packed_scans_of_changing_offsets_on_one_workspace():
    import torch
    import gated_delta_rule_87_b200 as gdr
    T, D = 4000, 256
    x, g = torch.randn((1, T, D), device="cuda").bfloat16(), -torch.rand((1, T, D), device="cuda")
    cus = [torch.tensor(c, dtype=torch.int32, device="cuda")
           for c in ([0, T], [0, 1, T], [0, 700, 701, 2222, T], list(range(0, T, 100)) + [T], [0, T - 1, T], [0, 2048, T])]
    want = [(*gdr.glr_scan_fwd(x, g, None, cu)[:2], *gdr.glr_scan_bwd(x, x, g, None, cu)[:3]) for cu in cus]
    ws = torch.empty(32 << 20, dtype=torch.uint8, device="cuda")
    got = []
    for k in range(60):
        cu = cus[k % len(cus)]
        got.append((*gdr.glr_scan_fwd(x, g, None, cu, workspace=ws)[:2], *gdr.glr_scan_bwd(x, x, g, None, cu, workspace=ws)[:3]))
    for k, outs in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(outs, want[k % len(cus)])), k


def test_column_sums_of_changing_gradients_on_one_workspace():
    import torch
    import gated_delta_rule_87_b200 as gdr
    M, D = 3000, 512
    r, y = (torch.randn((M, D), device="cuda").bfloat16() for _ in range(2))
    w = torch.randn(D, device="cuda")
    dns = [torch.randn((M, D), device="cuda").bfloat16() for _ in range(4)]
    want = [gdr.add_norm_bwd(dn, None, r, y, w, w)[2:4] for dn in dns]
    ws = torch.empty(gdr.lib().kda_add_norm_bwd_workspace_size(D), dtype=torch.uint8, device="cuda")
    got = [gdr.add_norm_bwd(dns[k % 4], None, r, y, w, w, workspace=ws)[2:4] for k in range(60)]
    for k, outs in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(outs, want[k % 4])), k
