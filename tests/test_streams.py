"""A call that is given a stream other than the current one: what it allocates
belongs to that stream, and tensors of other streams are recorded on it."""
import contextlib
import types

import pytest

import gated_delta_rule_87_b200 as gdr


class _Stream:
    def __init__(self, handle, device=0):
        self.cuda_stream, self.device = handle, types.SimpleNamespace(index=device)


class _External(_Stream):
    pass


class _Tensor:
    is_cuda = True

    def __init__(self):
        self.recorded = []

    def record_stream(self, stream):
        self.recorded.append(stream.cuda_stream)


def _fake_torch():
    """The few names that the helpers take of torch; `at` is (device, stream handle) now."""
    fake = types.SimpleNamespace(at=(0, 0), Tensor=_Tensor)

    @contextlib.contextmanager
    def device(index):
        before, fake.at = fake.at, (index, fake.at[1])
        yield
        fake.at = before

    @contextlib.contextmanager
    def stream(s):
        before, fake.at = fake.at, (s.device.index, s.cuda_stream)
        yield
        fake.at = before

    fake.cuda = types.SimpleNamespace(
        Stream=_Stream, device=device, stream=stream, current_device=lambda: fake.at[0],
        current_stream=lambda dev: _Stream(fake.at[1], dev),
        ExternalStream=_External)
    fake._C = types.SimpleNamespace()
    return fake


def test_a_call_runs_under_the_stream_that_it_is_given():
    torch, x, y = _fake_torch(), _Tensor(), _Tensor()
    assert gdr._here(torch, 0, None) and gdr._here(torch, 0, _Stream(0))
    assert not gdr._here(torch, 0, _Stream(7)) and not gdr._here(torch, 1, None)
    seen = []
    out = gdr._there(torch, 0, _Stream(7), lambda *a, **kw: seen.append(torch.at) or "out", x, None, kw=y, n=3)
    assert out == "out" and seen == [(0, 7)] and torch.at == (0, 0)
    assert x.recorded == [7] and y.recorded == [7]
    # a stream of another library, known by its handle alone or wrapped: it may be gone when x is freed
    for other in (types.SimpleNamespace(cuda_stream=9), _External(9)):
        gdr._there(torch, 0, other, lambda a: seen.append(torch.at), x)
        assert seen[-1] == (0, 9) and x.recorded == [7]
    # another device, its current stream: nothing to record
    gdr._there(torch, 1, None, lambda a: seen.append(torch.at), x)
    assert seen[-1] == (1, 0) and x.recorded == [7]
    with pytest.raises(ValueError, match="CUDA device 0"):
        gdr._there(torch, 0, _Stream(7, device=1), lambda: None)


def _calls(torch):
    """name -> (inputs, call of them and a stream, which allocates all that it returns)"""
    def t(*shape, dt=torch.bfloat16):
        return torch.randn(shape, device="cuda").to(dt)

    bf, f = torch.bfloat16, torch.float32
    decay = lambda *s: -torch.rand(s, device="cuda")  # noqa: E731
    x, g, w = t(2, 300, 192), decay(2, 300, 192), t(64, dt=f)
    y, r = t(50, 3, 64), t(50, 64)
    q = torch.nn.functional.normalize(t(1, 100, 2, 64, dt=f), dim=-1).bfloat16()
    b, st = torch.rand((1, 100, 2), device="cuda"), t(4, 2, 64, 64, dt=f)
    kg, one = decay(1, 100, 2, 64), t(4, 2, 64)
    slots = torch.arange(4, dtype=torch.int32, device="cuda")
    return {
        "glr_scan_fwd": ((x, g), lambda s, x, g: gdr.glr_scan_fwd(x, g, output_chunk_states=True, stream=s)),
        "glr_scan_bwd": ((x, g), lambda s, x, g: gdr.glr_scan_bwd(x, x, g, stream=s)),
        "glr_step": ((x[0], g[0], g[1]), lambda s, x, g, h: (gdr.glr_step(x, g, h.clone(), stream=s),)),
        "gated_norm_fwd": ((y, w), lambda s, y, w: (gdr.gated_norm_fwd(y, y, w, stream=s),)),
        "gated_norm_bwd": ((y, w), lambda s, y, w: gdr.gated_norm_bwd(y, y, y, w, stream=s)),
        "add_norm_fwd": ((r, w), lambda s, r, w: gdr.add_norm_fwd(r, r, w, stream=s)),
        "add_norm_bwd": ((r, w), lambda s, r, w: gdr.add_norm_bwd(r, r, r, r, w, w, stream=s)),
        "kda_chunk_fwd": ((q, kg, b), lambda s, q, g, b: gdr.kda_chunk_fwd(q, q, q, g, b, stream=s)),
        "gdn_chunk_fwd": ((q, kg, b), lambda s, q, g, b: gdr.gdn_chunk_fwd(q, q, q, g[..., 0].contiguous(), b, stream=s)),
        "kda_decode_step": ((one, st), lambda s, q, st: (gdr.kda_decode_step(
            q, q, q, -q.float().abs(), q[..., 0].float().contiguous(), st.clone(), stream=s),)),
        "kda_recurrent_fwd": ((q, kg, b, st), lambda s, q, g, b, st: (gdr.kda_recurrent_fwd(
            q, q, q, g, b, st[:1].clone(), stream=s),)),
        "state_gather": ((st, slots), lambda s, st, slots: (gdr.state_gather(st, slots, stream=s),)),
    }


NAMES = ["glr_scan_fwd", "glr_scan_bwd", "glr_step", "gated_norm_fwd", "gated_norm_bwd", "add_norm_fwd",
         "add_norm_bwd", "kda_chunk_fwd", "gdn_chunk_fwd", "kda_decode_step", "kda_recurrent_fwd", "state_gather"]


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_what_a_call_allocates_belongs_to_its_stream(name):
    """By the allocator's own records; with the same results as on the current stream."""
    import torch
    torch.manual_seed(3)
    inputs, call = _calls(torch)[name]
    side = torch.cuda.Stream()
    want = [t.clone() for t in call(None, *inputs) if t is not None]
    torch.cuda.synchronize()
    out = [t for t in call(side, *inputs) if t is not None]
    side.synchronize()
    owner = {}
    for seg in torch.cuda.memory_snapshot():
        for t in out:
            if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
                owner[t.data_ptr()] = seg["stream"]
    assert [owner[t.data_ptr()] for t in out] == [side.cuda_stream] * len(out)
    for a, b in zip(want, out):
        if a.dtype != torch.uint8:  # (a workspace)
            assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["glr_scan_fwd", "gated_norm_bwd", "kda_chunk_fwd"])
def test_an_input_dropped_after_the_call_is_kept_until_its_stream_is_past_it(name):
    import torch
    inputs, call = _calls(torch)[name]
    x = inputs[0].repeat(*(40 if k == 1 else 1 for k in range(inputs[0].dim()))).contiguous()
    rest = [t.repeat(1, 40, *([1] * (t.dim() - 2))).contiguous() if t.dim() > 2 else t for t in inputs[1:]]
    side = torch.cuda.Stream()
    call(side, x, *rest)  # (kernels are loaded by now)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(400_000_000)  # some 200 ms: the call waits its turn
    call(side, x, *rest)
    at, shape, dtype = x.data_ptr(), x.shape, x.dtype
    del x
    y = torch.empty(shape, dtype=dtype, device="cuda")
    assert not side.query() and y.data_ptr() != at
    side.synchronize()


@pytest.mark.gpu
def test_dropped_workspaces_of_a_busy_stream():
    """Calls on a side stream whose outputs and workspaces are dropped or kept by
    turns, the current stream busy with memory of its own."""
    import torch
    torch.manual_seed(5)
    x, g = torch.randn((2, 3000, 192), device="cuda").bfloat16(), -torch.rand((2, 3000, 192), device="cuda")
    saved = gdr.glr_scan_fwd(x, g, output_chunk_states=True)[2]
    want = gdr.glr_scan_bwd(x, x, g, chunk_states=saved)[:3]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    kept = []
    for _ in range(20):
        a = torch.full((1 << 20,), 3, dtype=torch.uint8, device="cuda")  # may be a block just dropped
        gdr.glr_scan_fwd(x, g, stream=side)
        dx, dg, dh0, _ = gdr.glr_scan_bwd(x, x, g, chunk_states=saved, stream=side)
        del a
        kept.append((dx, dg, dh0))
    side.synchronize()
    assert all(torch.equal(p, q) for got in kept for p, q in zip(got, want))
