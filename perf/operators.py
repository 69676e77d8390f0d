"""The gated linear recurrence and the norms around a mixer block: the cases that are measured.

``run`` computes an operator in plain torch operations, or, where ``own`` is true, through the library's calls.

Operators (all over the last axis' channels, per token):

* ``scan``   h_t = exp(g_t) h_{t-1} + b_t over sequences, b = x, or (1 - exp(g)) x ("complement"); with states
* ``train``  the same with its backward pass
* ``step``   one token for each sequence, the states updated in place in a pool of slots
* ``gnorm``  RMS norm over a head, times a weight, times SiLU or sigmoid of a gate; ``gnorm_bwd`` its gradients
* ``anorm``  residual + scale * y, and the RMS norm of the sum; ``anorm_bwd`` its gradients
"""
import math
import random

import torch

own = False

BF16, F32 = "bf16", "f32"
EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a small decode batch: latency
        dict(name="step_16x2048", op="step", N=16, D=2048, dtype=BF16, complement=False),
        # a full decode batch of 256 sequences, 32 heads x 128 channels, states in a pool
        dict(name="step_256x4096", op="step", N=256, D=4096, dtype=BF16, complement=True),
        # prefill of one prompt of 4096 tokens, 32 heads x 128 channels, a continued state
        dict(name="scan_4096x4096", op="scan", B=1, T=4096, D=4096, nseq=0, dtype=BF16, complement=False),
        # eight packed prompts of mixed lengths, 49,802 tokens together
        dict(name="scan_packed_49802x4096", op="scan", B=1, T=49802, D=4096, nseq=8, dtype=BF16, complement=False),
        # one long document
        dict(name="scan_65536x2048", op="scan", B=1, T=65536, D=2048, nseq=0, dtype=BF16, complement=True),
        # many short ragged sequences, an odd number of channels, all in 32 bits
        dict(name="scan_ragged_9001x1001", op="scan", B=1, T=9001, D=1001, nseq=37, dtype=F32, complement=False),
        # a training step on a dense batch
        dict(name="train_4x4096x2048", op="train", B=4, T=4096, D=2048, nseq=0, dtype=BF16, complement=False),
        # a training step on packed sequences, odd sizes, 32 bits
        dict(name="train_ragged_5003x777", op="train", B=1, T=5003, D=777, nseq=21, dtype=F32, complement=True),
        # the output gate and norm of a mixer of 32 heads x 128 in a decode step of 64 sequences
        dict(name="gnorm_64x32x128", op="gnorm", M=64, H=32, d=128, dtype=BF16, gate="silu"),
        # its gradients in training
        dict(name="gnorm_bwd_16384x32x128", op="gnorm_bwd", M=16384, H=32, d=128, dtype=BF16, gate="sigmoid"),
        # the boundary between two blocks: the residual stream in 32 bits
        dict(name="anorm_8192x4096", op="anorm", M=8192, D=4096, res=F32, dtype=BF16, scaled=True),
        # its gradients, an odd width
        dict(name="anorm_bwd_5001x4095", op="anorm_bwd", M=5001, D=4095, res=BF16, dtype=BF16, scaled=True),
    ]


MOST = 1.2e9  # bytes of a drawn case at most


def draw(rng):
    def size(lo, hi):
        n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        return min(max(n, lo), hi)

    def width(lo, hi):
        n = size(lo, hi)
        return n if rng.random() < 0.4 else max(lo, n // 64 * 64)

    while True:
        op = rng.choice(["step", "scan", "scan", "train", "train", "gnorm", "gnorm_bwd", "anorm", "anorm_bwd"])
        dtype = rng.choice([BF16, BF16, F32])
        if op == "step":
            c = dict(op=op, N=size(1, 512), D=width(64, 8192), dtype=dtype, complement=rng.random() < 0.5)
        elif op in ("scan", "train"):
            packed = rng.random() < 0.5
            B = 1 if packed else rng.choice([1, 1, 2, 3, 8, 32])
            T = size(1, 65536)
            c = dict(op=op, B=B, T=T, D=width(64, 8192), nseq=size(1, 64) if packed else 0, dtype=dtype,
                     complement=rng.random() < 0.5)
            if B * T > 65536:
                continue
        elif op in ("gnorm", "gnorm_bwd"):
            c = dict(op=op, M=size(1, 16384), H=rng.choice([1, 4, 16, 32]), d=rng.choice([32, 64, 96, 128, 128, 256, 333]),
                     dtype=dtype, gate=rng.choice(["silu", "sigmoid"]))
        else:
            c = dict(op=op, M=size(1, 32768), D=width(64, 8192), res=F32 if dtype == F32 else rng.choice([BF16, F32]),
                     dtype=dtype, scaled=rng.random() < 0.5)
        if work(c)["bytes"] <= MOST:
            return c


def _esize(name):
    return 2 if name == BF16 else 4


def work(case):
    e = _esize(case["dtype"])
    op = case["op"]
    if op == "step":
        n = case["N"] * case["D"]
        return {"bytes": n * (2 * e + 12) + 4 * case["N"], "flops": 4 * n}
    if op in ("scan", "train"):
        n, s = case["B"] * case["T"] * case["D"], (case["nseq"] or case["B"]) * case["D"]
        if op == "scan":
            return {"bytes": n * (2 * e + 4) + 8 * s, "flops": 4 * n}
        return {"bytes": n * (4 * e + 8) + 16 * s, "flops": 12 * n}
    if op in ("gnorm", "gnorm_bwd"):
        n = case["M"] * case["H"] * case["d"]
        return {"bytes": n * (3 if op == "gnorm" else 5) * e + 4 * case["d"], "flops": (8 if op == "gnorm" else 20) * n}
    n, r = case["M"] * case["D"], _esize(case["res"])
    w = 4 * case["D"] * (2 if case["scaled"] else 1)
    if op == "anorm":
        return {"bytes": n * (2 * r + 2 * e) + w, "flops": 6 * n}
    # reads dn, d residual_out, residual_out, writes d residual; with a scale also reads y and writes d y, without
    # one d y is d residual, and is written only where its type is another
    dy = 2 * e if case["scaled"] else e if e != r else 0
    return {"bytes": n * (3 * r + e + dy) + 2 * w, "flops": 14 * n}


# ------------------------------------------------------------------ inputs
def _cu(case):
    """Offsets of the packed sequences: cuts drawn by the case alone, so some sequences may be empty."""
    r = random.Random(case["T"] * 65537 + case["nseq"])
    return [0] + sorted(r.randint(0, case["T"]) for _ in range(case["nseq"] - 1)) + [case["T"]]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    io = torch.bfloat16 if case["dtype"] == BF16 else torch.float32
    normal = lambda *s, dt=torch.float32: torch.randn(s, generator=gen, device="cuda").to(dt)  # noqa: E731
    st = dict(case=case)
    op = case["op"]
    if op in ("step", "scan", "train"):
        D = case["D"]
        lead = (case["N"],) if op == "step" else (case["B"], case["T"])
        st["x"] = normal(*lead, D, dt=io)
        # log-decays: memories of about one to a thousand tokens, by channel
        pace = 10.0 ** (-3.0 * torch.rand(D, generator=gen, device="cuda"))
        st["g"] = -pace * torch.nn.functional.softplus(normal(*lead, D))
    if op == "step":
        slots = torch.randperm(2 * case["N"], generator=gen, device="cuda")[:case["N"]]
        st["slots"], st["pool"] = slots.to(torch.int32), normal(2 * case["N"], D)
        st["input"] = "complement" if case["complement"] else "given"
    elif op in ("scan", "train"):
        T = case["T"]
        cu = _cu(case) if case["nseq"] else [T * b for b in range(case["B"] + 1)]
        N = len(cu) - 1
        st["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda") if case["nseq"] else None
        st["offsets"], st["longest"] = cu, max(b - a for a, b in zip(cu, cu[1:]))
        st["cu64"] = torch.tensor(cu, dtype=torch.int64, device="cuda")
        st["h0"] = normal(N, D)
        st["input"] = "complement" if case["complement"] else "given"
        if op == "train":
            st["dh"], st["dfinal"] = normal(case["B"], T, D, dt=io), normal(N, D)
    elif op in ("gnorm", "gnorm_bwd"):
        shape = (case["M"], case["H"], case["d"])
        st["x"], st["z"] = normal(*shape, dt=io), normal(*shape, dt=io)
        st["w"] = 1 + 0.1 * normal(case["d"])
        if op == "gnorm_bwd":
            st["dy"] = normal(*shape, dt=io)
    else:
        M, D = case["M"], case["D"]
        res = torch.bfloat16 if case["res"] == BF16 else torch.float32
        st["r"], st["y"] = normal(M, D, dt=res), normal(M, D, dt=io)
        st["w"] = 1 + 0.1 * normal(D)
        st["scale"] = 0.5 + 0.1 * normal(D) if case["scaled"] else None
        if op == "anorm_bwd":
            st["dn"], st["dr"] = normal(M, D, dt=io), normal(M, D, dt=res)
    return st


# ------------------------------------------------------------------ plain forms
def _doubling(b, g, place, longest):
    """h_t = exp(g_t) h_{t-1} + b_t from zeros along axis 0, by doubling the span that each row has summed;
    `place`: the row's place in its sequence (the span stops at the sequence's start)."""
    h, span, k = b.clone(), g.clone(), 1
    while k < longest:
        inside = (place[k:] >= k)[:, None]
        h[k:] += torch.where(inside, torch.exp(span[k:]) * h[:-k], 0.0)
        span[k:] += torch.where(inside, span[:-k], 0.0)
        k *= 2
    return h


def _rows(st):
    """Per token: its sequence, its place from the start and from the end; which sequences have tokens."""
    cu = st["cu64"]
    length = cu[1:] - cu[:-1]
    seq = torch.repeat_interleave(torch.arange(len(length), device=cu.device), length, output_size=st["offsets"][-1])
    at = torch.arange(seq.numel(), device=cu.device)
    return seq, at - cu[seq], cu[seq + 1] - 1 - at, length > 0


def _plain_scan(st, back):
    x, g = st["x"].float().flatten(0, 1), st["g"].flatten(0, 1)
    complement = st["input"] == "complement"
    seq, place, left, full = _rows(st)
    first, last = st["cu64"][:-1][full], st["cu64"][1:][full] - 1
    a = torch.exp(g)
    b = -torch.expm1(g) * x if complement else x.clone()
    b[first] += a[first] * st["h0"][full]
    h = _doubling(b, g, place, st["longest"])
    final = st["h0"].clone()
    final[full] = h[last]
    out = [h.to(st["x"].dtype).view_as(st["x"]), final]
    if not back:
        return out
    d = st["dh"].float().flatten(0, 1)
    d[last] += st["dfinal"][full]
    later = torch.zeros_like(g)
    later[:-1] = g[1:]  # a token's gradient meets the decay of the next one
    d = _doubling(d.flip(0), later.flip(0), left.flip(0), st["longest"]).flip(0)
    before = torch.empty_like(h)
    before[1:] = h[:-1]
    before[first] = st["h0"][full]
    dx = -torch.expm1(g) * d if complement else d
    dg = d * a * (before - x if complement else before)
    dh0 = st["dfinal"].clone()
    dh0[full] = a[first] * d[first]
    return out + [dx.to(st["x"].dtype).view_as(st["x"]), dg.view_as(st["g"]), dh0]


def _plain_step(st):
    x, g, at = st["x"].float(), st["g"], st["slots"].long()
    b = -torch.expm1(g) * x if st["input"] == "complement" else x
    h = torch.exp(g) * st["pool"][at] + b
    st["pool"][at] = h
    return [h.to(st["x"].dtype), st["pool"]]


def _gate(z, kind):
    """The gate's value and its derivative."""
    s = 1 / (1 + torch.exp(-z))
    return (s, s * (1 - s)) if kind == "sigmoid" else (z * s, s * (1 + z * (1 - s)))


def _plain_gnorm(st, back):
    x, z, w = st["x"].float(), st["z"].float(), st["w"]
    inv = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    unit, (s, ds) = x * inv, _gate(z, st["case"]["gate"])
    if not back:
        return [(unit * w * s).to(st["x"].dtype)]
    dy = st["dy"].float()
    du = dy * w * s
    dx = inv * (du - unit * (du * unit).mean(-1, keepdim=True))
    return [dx.to(st["x"].dtype), (dy * unit * w * ds).to(st["x"].dtype), (dy * unit * s).sum((0, 1))]


def _plain_anorm(st):
    y, scale = st["y"].float(), st["scale"]
    r = st["r"].float() + (y if scale is None else scale * y)
    n = r / torch.sqrt((r * r).mean(-1, keepdim=True) + EPS) * st["w"]
    return [r.to(st["r"].dtype), n.to(st["y"].dtype)]


def _plain_anorm_bwd(st):
    r, dn, scale = st["r"].float(), st["dn"].float(), st["scale"]
    inv = 1 / torch.sqrt((r * r).mean(-1, keepdim=True) + EPS)
    unit, du = r * inv, dn * st["w"]
    d = st["dr"].float() + inv * (du - unit * (du * unit).mean(-1, keepdim=True))
    out = [d.to(st["r"].dtype), (d if scale is None else scale * d).to(st["y"].dtype), (dn * unit).sum(0)]
    return out if scale is None else out + [(d * st["y"].float()).sum(0)]


def run(state):
    st, op = state, state["case"]["op"]
    if own:
        return _own(st, op)
    if op == "step":
        return _plain_step(st)
    if op in ("scan", "train"):
        return _plain_scan(st, op == "train")
    if op in ("gnorm", "gnorm_bwd"):
        return _plain_gnorm(st, op == "gnorm_bwd")
    return _plain_anorm(st) if op == "anorm" else _plain_anorm_bwd(st)


def _own(st, op):
    import gated_delta_rule_87_b200 as gdr

    if op == "step":
        h = gdr.glr_step(st["x"], st["g"], st["pool"], state_slots=st["slots"], input_gate=st["input"])
        return [h, st["pool"]]
    if op in ("scan", "train"):
        h, final, chunks, _ = gdr.glr_scan_fwd(st["x"], st["g"], st["h0"], st["cu"], input_gate=st["input"],
                                               output_chunk_states=op == "train")
        if op == "scan":
            return [h, final]
        dx, dg, dh0, _ = gdr.glr_scan_bwd(st["dh"], st["x"], st["g"], st["h0"], st["cu"], input_gate=st["input"],
                                          dfinal_state=st["dfinal"], chunk_states=chunks)
        if st["dh"].dtype == torch.float32:
            # the plain form adds the final states' gradient into a 32-bit dh itself: so does this program,
            # or the two would go on from different inputs when a pass is run again
            cu = st["cu64"]
            full = (cu[1:] > cu[:-1])[:, None]
            st["dh"].flatten(0, 1).index_add_(0, (cu[1:] - 1).clamp_(min=0), torch.where(full, st["dfinal"], 0.0))
        return [h, final, dx, dg, dh0]
    if op == "gnorm":
        return [gdr.gated_norm_fwd(st["x"], st["z"], st["w"], gate=st["case"]["gate"], eps=EPS)]
    if op == "gnorm_bwd":
        dx, dz, dw, _ = gdr.gated_norm_bwd(st["dy"], st["x"], st["z"], st["w"], gate=st["case"]["gate"], eps=EPS)
        return [dx, dz, dw]
    if op == "anorm":
        return list(gdr.add_norm_fwd(st["r"], st["y"], st["w"], st["scale"], eps=EPS))
    dr, dy, dw, dscale, _ = gdr.add_norm_bwd(st["dn"], st["dr"], st["r"], st["y"], st["w"], st["scale"], eps=EPS)
    return [dr, dy, dw] if dscale is None else [dr, dy, dw, dscale]


# ------------------------------------------------------------------ from the definitions, in 64 bits
def exact(case, seed):
    st, op = prepare(case, seed), case["op"]
    f = lambda k: st[k].double()  # noqa: E731
    if op == "step":
        at = st["slots"].long()
        a = f("g").exp()
        h = a * f("pool")[at] + ((1 - a) * f("x") if case["complement"] else f("x"))
        pool = f("pool")
        pool[at] = h
        return [h, pool]
    if op in ("scan", "train"):
        return _exact_scan(st, case)
    if op in ("gnorm", "gnorm_bwd"):
        x, z, w = f("x"), f("z"), f("w")
        rms = (x.square().mean(-1, keepdim=True) + EPS).sqrt()
        sig = torch.sigmoid(z)
        act = sig if case["gate"] == "sigmoid" else z * sig
        if op == "gnorm":
            return [x / rms * w * act]
        slope = sig - sig.square()
        if case["gate"] == "silu":
            slope = sig + z * slope
        dy = f("dy")
        t = dy * w * act  # the gradient of x / rms
        dx = t / rms - x * (t * x).sum(-1, keepdim=True) / (case["d"] * rms**3)
        return [dx, dy * (x / rms) * w * slope, (dy * (x / rms) * act).flatten(0, 1).sum(0)]
    scale = f("scale") if case["scaled"] else torch.ones(case["D"], dtype=torch.float64, device="cuda")
    if op == "anorm":
        r = f("r") + scale * f("y")
        return [r, r * (r.square().mean(-1, keepdim=True) + EPS).rsqrt() * f("w")]
    r, t = f("r"), f("dn") * f("w")
    rms = (r.square().mean(-1, keepdim=True) + EPS).sqrt()
    d = f("dr") + t / rms - r * (t * r).sum(-1, keepdim=True) / (case["D"] * rms**3)
    out = [d, scale * d, (f("dn") * r / rms).sum(0)]
    return out + [(d * f("y")).sum(0)] if case["scaled"] else out


def _exact_scan(st, case):
    """Token by token."""
    cu = st["offsets"]
    x, g, h0 = st["x"].double().flatten(0, 1), st["g"].double().flatten(0, 1), st["h0"].double()
    a = g.exp()
    u = torch.expm1(g).neg_() if case["complement"] else torch.ones_like(a)
    b = u * x
    h, final = torch.empty_like(x), h0.clone()
    for n in range(len(cu) - 1):
        s = h0[n]
        for t in range(cu[n], cu[n + 1]):
            s = torch.addcmul(b[t], a[t], s, out=h[t])
        final[n] = s
    out = [h.view(st["x"].shape), final]
    if case["op"] == "scan":
        return out
    d, dh0 = st["dh"].double().flatten(0, 1), st["dfinal"].double()
    dg = torch.empty_like(a)
    for n in range(len(cu) - 1):
        carry = dh0[n]
        for t in range(cu[n + 1] - 1, cu[n] - 1, -1):
            d[t] += carry
            carry = torch.mul(a[t], d[t], out=dg[t])  # times h_{t-1} below
        dh0[n] = carry
    before = torch.empty_like(h)
    before[1:] = h[:-1]
    for n in range(len(cu) - 1):
        if cu[n + 1] > cu[n]:
            before[cu[n]] = h0[n]
    dh0 = dh0.clone()
    dg *= before - x if case["complement"] else before
    return out + [(u * d).view(st["x"].shape), dg.view(st["g"].shape), dh0]
