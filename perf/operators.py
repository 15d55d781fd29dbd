"""The selective state space mixer's operators, as they are measured.

Three operators make up the mixer: a short causal depthwise convolution with
SiLU, the selective scan, and a group norm with a gate, all channels last.
Each has a form for whole prompts (with the states that go in and come out),
one for training (forward and gradients) and, for the two that carry a state,
one for single tokens that updates the state in place.

``run`` computes a case with elementary torch operations in float32, or, where
``own`` is true, with the library's kernels.  Activations are bf16 or float32,
parameters and states are float32 (the convolution's state has the
activations' type).

Formulas (row r of a sequence, channel d, state n, g = the group of d):

    conv    v_r = bias + sum_k w[d, k] x_{r-W+1+k},  y = v sigmoid(v); the rows
            before a sequence are its x0
    scan    dt = softplus(raw + dt_bias),  h_r = exp(dt A) h_{r-1} + dt x B_r[g],
            y = sum_n C_r[g, n] h_r[n] + D x
    norm    o = (p - mean) rstd w + b over each group of channels of a row
            (rms: mean = 0, b = 0),  y = o silu(z)   (p = x),
            or gate first: p = x silu(z), y = o;  without z: y = silu(o)
"""
import math

import torch

own = False

EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # one user decoding: a single token through one layer's scan
        dict(name="scan_token_1x2048", op="scan", mode="token", B=1, T=1, D=2048, N=16, G=1, dtype="bf16", packed=False, h0=True),
        # a serving step of a full batch out of a larger pool of states, some rows idle
        dict(name="scan_token_256x4096", op="scan", mode="token", B=256, T=1, D=4096, N=16, G=1, dtype="bf16", packed=False, h0=True),
        # one long prompt: few channels' worth of rows, so time has to be split
        dict(name="scan_prompt_1x16384x2048", op="scan", mode="prompt", B=1, T=16384, D=2048, N=16, G=1, dtype="bf16", packed=False, h0=False),
        # prompts of uneven lengths packed back to back, continued from earlier states; odd sizes
        dict(name="scan_packed_5003x1000", op="scan", mode="prompt", B=7, T=5003, D=1000, N=12, G=1, dtype="fp32", packed=True, h0=True),
        # a layer's training step
        dict(name="scan_train_4x4096x2048", op="scan", mode="train", B=4, T=4096, D=2048, N=16, G=1, dtype="bf16", packed=False, h0=False),
        # a small float32 training step with two groups of shared B and C and odd sizes
        dict(name="scan_train_3x509x520", op="scan", mode="train", B=3, T=509, D=520, N=24, G=2, dtype="fp32", packed=False, h0=True),
        # the same serving step's convolution
        dict(name="conv_token_256x4096", op="conv", mode="token", B=256, T=1, D=4096, W=4, dtype="bf16", packed=False, h0=True),
        # packed prompts through the convolution
        dict(name="conv_packed_32768x4096", op="conv", mode="prompt", B=17, T=32768, D=4096, W=4, dtype="bf16", packed=True, h0=True),
        dict(name="conv_train_8x4096x2048", op="conv", mode="train", B=8, T=4096, D=2048, W=4, dtype="bf16", packed=False, h0=False),
        # the norm behind the scan: the whole row one group, gated first, no mean
        dict(name="norm_prompt_32768x4096", op="norm", mode="prompt", B=1, T=32768, D=4096, G=1, dtype="bf16", rms=True, gate="first", bias=False),
        # the norm of heads of 128 channels, gated after it
        dict(name="norm_train_8x4096x2048", op="norm", mode="train", B=8, T=4096, D=2048, G=16, dtype="bf16", rms=False, gate="after", bias=True),
        # odd float32 rows without a gate
        dict(name="norm_train_7x111x1000", op="norm", mode="train", B=7, T=111, D=1000, G=5, dtype="fp32", rms=False, gate="none", bias=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("scan", "scan", "conv", "norm"))
    dtype = rng.choice(("bf16", "bf16", "fp32"))
    if op == "scan":
        mode = rng.choice(("token", "prompt", "train"))
        N = rng.choice((4, 8, 12, 16, 16, 16, 24, 32, 64))
        G = rng.choice((1, 1, 1, 2, 4))
        D = G * _log_int(rng, 256 // G, 4096 // G)
        if mode == "token":
            return dict(op=op, mode=mode, B=_log_int(rng, 1, 256), T=1, D=D, N=N, G=G, dtype=dtype, packed=False, h0=True)
        packed = rng.random() < 0.4
        B = rng.randint(1, 8)
        room = (1 << 28) // (D * N * (1 if packed else B))
        T = _log_int(rng, 16, max(32, min(16384, room)))
        return dict(op=op, mode=mode, B=B, T=T, D=D, N=N, G=G, dtype=dtype, packed=packed, h0=rng.random() < 0.5)
    if op == "conv":
        mode = rng.choice(("token", "prompt", "train"))
        D, W = _log_int(rng, 256, 4096), rng.choice((2, 3, 4, 4))
        if mode == "token":
            return dict(op=op, mode=mode, B=_log_int(rng, 1, 256), T=1, D=D, W=W, dtype=dtype, packed=False, h0=True)
        packed = rng.random() < 0.5
        B = rng.randint(1, 8)
        T = _log_int(rng, 16, 8192 * (B if packed else 1))
        return dict(op=op, mode=mode, B=B, T=T, D=D, W=W, dtype=dtype, packed=packed, h0=packed or rng.random() < 0.5)
    G = rng.choice((1, 1, 2, 5, 8, 16, 32))
    gate = rng.choice(("first", "after", "none"))
    rms = rng.random() < 0.5
    return dict(op=op, mode=rng.choice(("prompt", "train")), B=rng.randint(1, 8), T=_log_int(rng, 16, 4096), D=G * _log_int(rng, max(8, 256 // G), 4096 // G),
                G=G, dtype=dtype, rms=rms, gate=gate, bias=not rms)


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(dev).manual_seed(seed * 7919 + 13)
    ty = TYPES[case["dtype"]]
    B, T, D = case["B"], case["T"], case["D"]

    def randn(*shape, scale=1.0, of=torch.float32):
        return (torch.randn(shape, generator=g, device=dev) * scale).to(of)

    def rand(*shape):
        return torch.rand(shape, generator=g, device=dev)

    s = dict(case, device=dev)
    packed, token, train = case.get("packed", False), case["mode"] == "token", case["mode"] == "train"
    lead = (B,) if token else ((1, T) if packed else (B, T))
    if packed:  # B sequences of uneven lengths, T rows in all
        weights = rand(B) + 0.05
        cuts = (weights.cumsum(0) / weights.sum() * T).long()
        cuts[-1] = T
        s["cu"] = torch.cat([torch.zeros(1, dtype=torch.int64, device=dev), cuts])
    if token:  # a pool of states, larger than the batch; every 17th row is idle
        pool = B + B // 2
        slots = torch.randperm(pool, generator=g, device=dev)[:B]
        if B > 1:
            slots[::17] = -1
        s["slots"] = slots

    if case["op"] == "scan":
        N, G = case["N"], case["G"]
        s["x"] = randn(*lead, D, of=ty)
        s["dt"] = randn(*lead, D, scale=0.5, of=ty)
        # B and C are slices of one projection's output
        bc = randn(*lead, 2 * G * N, of=ty)
        s["Bm"] = bc[..., :G * N].unflatten(-1, (G, N))
        s["Cm"] = bc[..., G * N:].unflatten(-1, (G, N))
        s["A"] = -torch.arange(1, N + 1, device=dev, dtype=torch.float32) * torch.exp(randn(D, N, scale=0.1))
        s["D_skip"] = 1 + randn(D, scale=0.1)
        step = torch.exp(rand(D) * (math.log(0.1) - math.log(1e-3)) + math.log(1e-3))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))  # softplus(dt_bias) = step
        if token:
            s["state"] = randn(B + B // 2, D, N, scale=0.5)
        else:
            s["h0"] = randn(B, D, N, scale=0.5) if case["h0"] else None
        if train:
            s["dy"] = randn(*lead, D, of=ty)
            s["dh_last"] = randn(B, D, N) if case["h0"] else None
    elif case["op"] == "conv":
        W = case["W"]
        # x is one half of the input projection's output
        s["x"] = randn(*lead, 2 * D, of=ty)[..., :D]
        s["w"], s["bias"] = randn(D, W, scale=0.5), randn(D, scale=0.1)
        if token:
            s["state"] = randn(B + B // 2, W - 1, D, of=ty)
        else:
            s["x0"] = randn(B, W - 1, D, of=ty) if case["h0"] else None
        if train:
            s["dy"] = randn(*lead, D, of=ty)
            s["dx_last"] = randn(B, W - 1, D, of=ty) if case["h0"] else None
    else:
        s["x"] = randn(B, T, D, of=ty)
        # z is one half of the input projection's output
        s["z"] = randn(B, T, 2 * D, of=ty)[..., D:] if case["gate"] != "none" else None
        s["w"] = 1 + randn(D, scale=0.1)
        s["b"] = randn(D, scale=0.1) if case["bias"] else None
        if train:
            s["dy"] = randn(B, T, D, of=ty)
    return s


# ------------------------------------------------------------------ a pass

def run(s):
    return (_own if own else _plain)[s["op"], s["mode"]](s)


def _own_scan_token(s):
    import linear_recurrence_scans_gb300 as mg
    y = mg.selective_scan_step(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["state"], D=s["D_skip"], dt_bias=s["dt_bias"], slots=s["slots"])
    return {"y": y, "state": s["state"]}


def _own_scan_prompt(s):
    import linear_recurrence_scans_gb300 as mg
    y, h_last, _ = mg.selective_scan_fwd(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], D=s["D_skip"], dt_bias=s["dt_bias"], h0=s["h0"], cu_seqlens=s.get("cu"))
    return {"y": y, "h_last": h_last}


def _own_scan_train(s):
    import linear_recurrence_scans_gb300 as mg
    args = (s["x"], s["dt"], s["A"], s["Bm"], s["Cm"])
    more = dict(D=s["D_skip"], dt_bias=s["dt_bias"], h0=s["h0"], cu_seqlens=s.get("cu"))
    y, h_last, saved = mg.selective_scan_fwd(*args, **more, save=True)
    dx, ddt, dA, dB, dC, dD, ddt_bias, dh0 = mg.selective_scan_bwd(s["dy"], saved, *args, **more, dh_last=s["dh_last"])
    return {"y": y, "h_last": h_last, "dx": dx, "ddt": ddt, "dA": dA, "dB": dB, "dC": dC, "dD": dD, "ddt_bias": ddt_bias, "dh0": dh0}


def _own_conv_token(s):
    import linear_recurrence_scans_gb300 as mg
    y = mg.causal_conv_step(s["x"], s["w"], s["state"], bias=s["bias"], slots=s["slots"])
    return {"y": y, "state": s["state"]}


def _own_conv_prompt(s):
    import linear_recurrence_scans_gb300 as mg
    y, x_last = mg.causal_conv_fwd(s["x"], s["w"], bias=s["bias"], x0=s["x0"], cu_seqlens=s.get("cu"))
    return {"y": y, "x_last": x_last}


def _own_conv_train(s):
    import linear_recurrence_scans_gb300 as mg
    y, x_last = mg.causal_conv_fwd(s["x"], s["w"], bias=s["bias"], x0=s["x0"], cu_seqlens=s.get("cu"))
    dx, dw, dbias, dx0 = mg.causal_conv_bwd(s["dy"], s["x"], s["w"], bias=s["bias"], x0=s["x0"], dx_last=s["dx_last"], cu_seqlens=s.get("cu"))
    return {"y": y, "x_last": x_last, "dx": dx, "dw": dw, "dbias": dbias, "dx0": dx0}


def _norm_options(s):
    return dict(bias=s["b"], z=s["z"], groups=s["G"], eps=EPS, rms=s["rms"], gate_first=s["gate"] == "first")


def _own_norm_prompt(s):
    import linear_recurrence_scans_gb300 as mg
    y, _ = mg.group_norm_fwd(s["x"], s["w"], **_norm_options(s))
    return {"y": y}


def _own_norm_train(s):
    import linear_recurrence_scans_gb300 as mg
    y, stats = mg.group_norm_fwd(s["x"], s["w"], **_norm_options(s))
    dx, dw, db, dz = mg.group_norm_bwd(s["dy"], stats, s["x"], s["w"], **_norm_options(s))
    return {"y": y, "dx": dx, "dw": dw, "db": db, "dz": dz}


# ------------------------------------------------------------- plain forms
# Float32 throughout, each output rounded once at the end.

def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))


def _rows(s):
    """Of each row of a packed batch: its sequence, that sequence's first row and its last."""
    r = torch.arange(s["T"], device=s["device"])
    seq = torch.searchsorted(s["cu"], r, right=True) - 1
    return seq, s["cu"][seq], s["cu"][seq + 1] - 1


def _scan_rows(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1 from h = 0, all rows at once: log2 T doublings of the span that each row has summed."""
    span, T = 1, b.shape[1]
    while span < T:
        b = torch.cat([b[:, :span], torch.addcmul(b[:, span:], a[:, span:], b[:, :-span])], 1)
        a = torch.cat([a[:, :span], a[:, span:] * a[:, :-span]], 1)
        span *= 2
    return b


def _groups(v, D):
    """(..., G, N) to (..., D, N): each group's row for each of its channels."""
    return v.float().unsqueeze(-2).expand(*v.shape[:-1], D // v.shape[-2], v.shape[-1]).flatten(-3, -2)


def _scan_parts(s):
    x, raw = s["x"].float(), s["dt"].float() + s["dt_bias"]
    dt = _softplus(raw)
    Bd, Cd = _groups(s["Bm"], s["D"]), _groups(s["Cm"], s["D"])
    return x, raw, dt, Bd, Cd


def _scan_states(s, x, dt, Bd):
    """(a, a with 0 at each sequence's first row, b with the start state in it, h) and where sequences begin and end."""
    a = torch.exp(dt[..., None] * s["A"])
    b = (dt * x)[..., None] * Bd
    if s.get("cu") is not None:
        seq, first, last = _rows(s)
        r = torch.arange(s["T"], device=s["device"])
        begins, ends = (r == first), (r == last)
        if s["h0"] is not None:
            b = b + a * s["h0"][seq] * begins[:, None, None]
        cut = a * (~begins)[:, None, None]
        has = s["cu"][1:] > s["cu"][:-1]
    else:
        cut, has = a, None
        begins = ends = seq = None
        if s["h0"] is not None:
            b = torch.cat([b[:, :1] + a[:, :1] * s["h0"][:, None], b[:, 1:]], 1)
    h = _scan_rows(cut, b)
    if s.get("cu") is not None:
        empty = torch.zeros_like(h[0, 0]) if s["h0"] is None else s["h0"]
        h_last = torch.where(has[:, None, None], h[0, (s["cu"][1:] - 1).clamp(min=0)], empty)
    else:
        h_last = h[:, -1].clone()
    return a, h, h_last, begins, ends, seq


def _plain_scan_prompt(s):
    x, _, dt, Bd, Cd = _scan_parts(s)
    _, h, h_last, *_ = _scan_states(s, x, dt, Bd)
    y = (h * Cd).sum(-1) + s["D_skip"] * x
    return {"y": y.to(s["x"].dtype), "h_last": h_last}


def _plain_scan_train(s):
    ty = s["x"].dtype
    x, raw, dt, Bd, Cd = _scan_parts(s)
    a, h, h_last, begins, ends, seq = _scan_states(s, x, dt, Bd)
    y = (h * Cd).sum(-1) + s["D_skip"] * x
    dy = s["dy"].float()
    dC = (h * dy[..., None]).unflatten(2, (s["G"], -1)).sum(3)
    # the adjoint of h_t: C_t dy_t, what comes back from h_{t+1}, and dh_last at a sequence's end
    e = Cd * dy[..., None]
    if s["dh_last"] is not None:
        e = e + s["dh_last"][seq] * ends[:, None, None] if seq is not None else torch.cat([e[:, :-1], e[:, -1:] + s["dh_last"][:, None]], 1)
    back = a if begins is None else a * (~begins)[:, None, None]
    back = torch.cat([back[:, 1:], torch.zeros_like(back[:, :1])], 1)
    g = _scan_rows(back.flip(1), e.flip(1)).flip(1)
    del e, back
    u = dt * x
    s1 = (g * Bd).sum(-1)
    dB = (g * u[..., None]).unflatten(2, (s["G"], -1)).sum(3)
    # a_t h_{t-1}, the decayed state before the row's own input came in
    w = g * (h - u[..., None] * Bd)
    dA = (w * dt[..., None]).sum((0, 1))
    ddt = (x * s1 + (w * s["A"]).sum(-1)) * torch.sigmoid(raw)
    if s["h0"] is None:
        dh0 = None
    elif seq is None:
        dh0 = a[:, 0] * g[:, 0]
    else:
        has = (s["cu"][1:] > s["cu"][:-1])[:, None, None]
        at = s["cu"][:-1].clamp(max=s["T"] - 1)
        dh0 = torch.where(has, a[0, at] * g[0, at], s["dh_last"])
    return {"y": y.to(ty), "h_last": h_last, "dx": (dt * s1 + s["D_skip"] * dy).to(ty), "ddt": ddt.to(ty), "dA": dA, "dB": dB.to(ty), "dC": dC.to(ty),
            "dD": (dy * x).sum((0, 1)), "ddt_bias": ddt.sum((0, 1)), "dh0": dh0}


def _live(s):
    """Which rows of the batch are not idle, and a slot to read for each (an idle row's is not used)."""
    return s["slots"] >= 0, s["slots"].clamp(min=0)


def _plain_scan_token(s):
    live, slot = _live(s)
    x, _, dt, Bd, Cd = _scan_parts(s)
    h = torch.exp(dt[..., None] * s["A"]) * s["state"][slot] + (dt * x)[..., None] * Bd
    y = (h * Cd).sum(-1) + s["D_skip"] * x
    s["state"][s["slots"][live]] = h[live]
    return {"y": (y * live[:, None]).to(s["x"].dtype), "state": s["state"]}


def _taps(s):
    """(rows, W, D): the W inputs that each row's convolution sees."""
    x, D, W = s["x"].float(), s["D"], s["W"]
    if s.get("cu") is not None:
        seq, first, _ = _rows(s)
        at = torch.arange(s["T"], device=s["device"])[:, None] + torch.arange(1 - W, 1, device=s["device"])
        before = at < first[:, None]
        # row first - 1 - j of the sequence is x0's row W - 2 - j
        old = s["x0"].float()[seq[:, None], (at - first[:, None] + W - 1).clamp(0, W - 2)] if s["x0"] is not None else torch.zeros(1, device=s["device"])
        return torch.where(before[..., None], old, x[0, at.clamp(min=0)])[None]
    x0 = s["x0"].float() if s["x0"] is not None else torch.zeros(s["B"], W - 1, D, device=s["device"])
    return torch.cat([x0, x], 1).unfold(1, W, 1).transpose(-1, -2)


def _last_rows(s):
    """The W - 1 last inputs of each sequence, with x0's where it has fewer rows."""
    W, x = s["W"], s["x"]
    x0 = s["x0"] if s["x0"] is not None else torch.zeros(s["B"], W - 1, s["D"], dtype=x.dtype, device=s["device"])
    if s.get("cu") is None:
        return torch.cat([x0, x], 1)[:, -(W - 1):].contiguous()
    at = s["cu"][1:, None] + torch.arange(1 - W, 0, device=s["device"])
    first = s["cu"][:-1, None]
    old = torch.gather(x0, 1, (at - first + W - 1).clamp(0, W - 2)[..., None].expand(-1, -1, s["D"]))
    return torch.where((at < first)[..., None], old, x[0, at.clamp(0, s["T"] - 1)])


def _plain_conv_prompt(s):
    v = (_taps(s) * s["w"].t()).sum(-2) + s["bias"]
    return {"y": (v * torch.sigmoid(v)).to(s["x"].dtype), "x_last": _last_rows(s)}


def _plain_conv_train(s):
    ty, W, D = s["x"].dtype, s["W"], s["D"]
    taps = _taps(s)
    v = (taps * s["w"].t()).sum(-2) + s["bias"]
    sg = torch.sigmoid(v)
    dv = s["dy"].float() * sg * (1 + v * (1 - sg))
    dw = (dv.unsqueeze(-2) * taps).sum((0, 1)).t().contiguous()
    parts = dv.unsqueeze(-2) * s["w"].t()  # what tap k of row r sends to row r - W + 1 + k
    if s.get("cu") is None:
        at = torch.arange(s["T"], device=s["device"])[:, None] + torch.arange(W, device=s["device"])
        wide = torch.zeros(s["B"], s["T"] + W - 1, D, device=s["device"])
        wide.index_add_(1, at.flatten(), parts.flatten(1, 2))
        if s["dx_last"] is not None:
            wide[:, -(W - 1):] += s["dx_last"].float()
        dx, dx0 = wide[:, W - 1:], wide[:, :W - 1]
    else:
        seq, first, _ = _rows(s)
        # each sequence with its W - 1 earlier rows in front: row r of the batch is row r + (seq + 1)(W - 1) there
        at = (torch.arange(s["T"], device=s["device"]) + seq * (W - 1))[:, None] + torch.arange(W, device=s["device"])
        wide = torch.zeros(s["T"] + s["B"] * (W - 1), D, device=s["device"])
        wide.index_add_(0, at.flatten(), parts[0].flatten(0, 1))
        j = torch.arange(W - 1, device=s["device"])
        n = torch.arange(s["B"], device=s["device"])[:, None]
        if s["dx_last"] is not None:
            wide.index_add_(0, (s["cu"][1:, None] + n * (W - 1) + j).flatten(), s["dx_last"].float().flatten(0, 1))
        dx, dx0 = wide[torch.arange(s["T"], device=s["device"]) + (seq + 1) * (W - 1)][None], wide[s["cu"][:-1, None] + n * (W - 1) + j]
    return {"y": (v * sg).to(ty), "x_last": _last_rows(s), "dx": dx.to(ty), "dw": dw, "dbias": dv.sum((0, 1)), "dx0": dx0.to(ty) if s["x0"] is not None else None}


def _plain_conv_token(s):
    live, slot = _live(s)
    taps = torch.cat([s["state"][slot], s["x"][:, None]], 1)
    v = (taps.float() * s["w"].t()).sum(1) + s["bias"]
    s["state"][s["slots"][live]] = taps[live, 1:]
    return {"y": (v * torch.sigmoid(v) * live[:, None]).to(s["x"].dtype), "state": s["state"]}


def _norm_parts(s):
    x = s["x"].float()
    z = s["z"].float() if s["z"] is not None else None
    p = x * z * torch.sigmoid(z) if s["gate"] == "first" else x
    q = p.unflatten(-1, (s["G"], -1))
    if not s["rms"]:
        q = q - q.mean(-1, keepdim=True)
    rstd = torch.rsqrt((q * q).mean(-1, keepdim=True) + EPS)
    n = (q * rstd).flatten(-2)
    o = n * s["w"] + s["b"] if s["b"] is not None else n * s["w"]
    return x, z, rstd, n, o


def _plain_norm_prompt(s):
    x, z, rstd, n, o = _norm_parts(s)
    y = o if s["gate"] == "first" else o * torch.sigmoid(o) if z is None else o * z * torch.sigmoid(z)
    return {"y": y.to(s["x"].dtype)}


def _plain_norm_train(s):
    ty = s["x"].dtype
    x, z, rstd, n, o = _norm_parts(s)
    dy = s["dy"].float()
    dz = None
    if s["gate"] == "first":
        y, do = o, dy
    elif z is None:
        sg = torch.sigmoid(o)
        y, do = o * sg, dy * sg * (1 + o * (1 - sg))
    else:
        sg = torch.sigmoid(z)
        y, do = o * z * sg, dy * z * sg
        dz = dy * o * sg * (1 + z * (1 - sg))
    dn = (do * s["w"]).unflatten(-1, (s["G"], -1))
    m = n.unflatten(-1, (s["G"], -1))
    dp = dn - m * (dn * m).mean(-1, keepdim=True)
    if not s["rms"]:
        dp = dp - dn.mean(-1, keepdim=True)
    dx = (rstd * dp).flatten(-2)
    if s["gate"] == "first":
        sg = torch.sigmoid(z)
        dz = dx * x * sg * (1 + z * (1 - sg))
        dx = dx * z * sg
    return {"y": y.to(ty), "dx": dx.to(ty), "dw": (do * n).sum((0, 1)), "db": do.sum((0, 1)) if s["b"] is not None else None, "dz": dz.to(ty) if dz is not None else None}


_plain = {("scan", "token"): _plain_scan_token, ("scan", "prompt"): _plain_scan_prompt, ("scan", "train"): _plain_scan_train,
          ("conv", "token"): _plain_conv_token, ("conv", "prompt"): _plain_conv_prompt, ("conv", "train"): _plain_conv_train,
          ("norm", "prompt"): _plain_norm_prompt, ("norm", "train"): _plain_norm_train}
_own = {("scan", "token"): _own_scan_token, ("scan", "prompt"): _own_scan_prompt, ("scan", "train"): _own_scan_train,
        ("conv", "token"): _own_conv_token, ("conv", "prompt"): _own_conv_prompt, ("conv", "train"): _own_conv_train,
        ("norm", "prompt"): _own_norm_prompt, ("norm", "train"): _own_norm_train}


# -------------------------------------------------------------------- work

def work(case):
    """Bytes: inputs once, outputs once (a forward and its gradients read what both need once).  Flops: multiplies, adds and exponentials counted as one each."""
    e = 2 if case["dtype"] == "bf16" else 4
    token, train = case["mode"] == "token", case["mode"] == "train"
    R = case["T"] if case.get("packed") else case["B"] * case["T"]
    D, act = case["D"], R * case["D"] * e
    if case["op"] == "scan":
        GN, state = case["G"] * case["N"], case["B"] * D * case["N"] * 4
        par, el = D * case["N"] * 4 + 8 * D, R * D * case["N"]
        by = 3 * act + 2 * R * GN * e + par + state * (2 if token or case["h0"] else 1)
        fl = 7 * el  # dt A, exp, a h, + u B (2), C h (2)
        if train:  # reads dy, writes dx, ddt, dB, dC, dA; the adjoint's own products
            by += 3 * act + 2 * R * GN * e + par + (state * 2 if case["h0"] else 0)
            fl += 16 * el
        return {"bytes": by, "flops": fl}
    if case["op"] == "conv":
        W = case["W"]
        state = case["B"] * (W - 1) * D * e
        by, fl = 2 * act + D * (W + 1) * 4 + state * (2 if case["h0"] else 1), R * D * (2 * W + 4)
        if train:
            by, fl = by + 2 * act + D * (W + 1) * 4 + (2 * state if case["h0"] else 0), fl + R * D * (4 * W + 8)
        return {"bytes": by, "flops": fl}
    z, par = case["gate"] != "none", D * (8 if case["bias"] else 4)
    by, fl = act * (3 if z else 2) + par, R * D * (9 + 4 * z)
    if train:
        by, fl = by + act * (3 if z else 2) + par, fl + R * D * (14 + 6 * z)
    return {"bytes": by, "flops": fl}


# ------------------------------------------------------------------- exact

def _f64(s):
    return {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}


def _spans(s):
    """(batch index, first row, end row, sequence) of every sequence."""
    if s.get("cu") is None:
        return [(b, 0, s["T"], b) for b in range(s["B"])]
    cu = s["cu"].tolist()
    return [(0, cu[i], cu[i + 1], i) for i in range(s["B"])]


def _exact_scan(s):
    """The recurrence row by row.  A dense batch is one loop over its rows, a packed one a loop for each sequence."""
    D, N, G, T = s["D"], s["N"], s["G"], s["T"]
    f = dict(device=s["device"], dtype=torch.float64)
    cells = [(slice(0, s["B"]), 0, T, slice(0, s["B"]))] if s.get("cu") is None else [(slice(b, b + 1), lo, hi, slice(i, i + 1)) for b, lo, hi, i in _spans(s)]
    raw = s["dt"] + s["dt_bias"]
    dt = torch.logaddexp(raw, torch.zeros((), **f))
    group = torch.arange(D, device=s["device"]) // (D // G)
    A, x = s["A"], s["x"]
    train = s["mode"] == "train"
    y = torch.empty_like(x)
    h_last = torch.zeros(s["B"], D, N, **f) if s["h0"] is None else s["h0"].clone()
    out = {"y": y, "h_last": h_last}
    if train:
        dy = s["dy"]
        dh0 = torch.zeros(s["B"], D, N, **f) if s["dh_last"] is None else s["dh_last"].clone()
        out |= {"dx": torch.empty_like(x), "ddt": torch.empty_like(x), "dA": torch.zeros(D, N, **f), "dB": torch.empty_like(s["Bm"]), "dC": torch.empty_like(s["Cm"]),
                "dD": (dy * x).sum((0, 1)), "ddt_bias": None, "dh0": dh0 if s["h0"] is not None else None}
    for b, lo, hi, i in cells:
        h = h_last[i].clone()
        kept = torch.empty(hi - lo, *h.shape, **f) if train else None
        for t in range(lo, hi):
            if train:
                kept[t - lo] = h
            h = h * torch.exp(dt[b, t, :, None] * A) + (dt[b, t] * x[b, t])[..., None] * s["Bm"][b, t][:, group]
            y[b, t] = torch.einsum("bdn,bdn->bd", h, s["Cm"][b, t][:, group]) + s["D_skip"] * x[b, t]
        h_last[i] = h
        if train:
            g = dh0[i].clone()
            for t in reversed(range(lo, hi)):
                a, Br, Cr = torch.exp(dt[b, t, :, None] * A), s["Bm"][b, t][:, group], s["Cm"][b, t][:, group]
                was = kept[t - lo]
                now = was * a + (dt[b, t] * x[b, t])[..., None] * Br
                out["dC"][b, t] = (now * dy[b, t][..., None]).unflatten(1, (G, -1)).sum(2)
                g = g + Cr * dy[b, t][..., None]
                out["dB"][b, t] = (g * (dt[b, t] * x[b, t])[..., None]).unflatten(1, (G, -1)).sum(2)
                gB = (g * Br).sum(-1)
                out["dx"][b, t] = gB * dt[b, t] + s["D_skip"] * dy[b, t]
                ga = g * a * was  # the gradient of dt A
                out["dA"] += (ga * dt[b, t, :, None]).sum(0)
                out["ddt"][b, t] = (gB * x[b, t] + (ga * A).sum(-1)) / (1 + torch.exp(-raw[b, t]))
                g = g * a
            dh0[i] = g
    if train:
        out["ddt_bias"] = out["ddt"].sum((0, 1))
    return out


def _exact_scan_token(s):
    group = torch.arange(s["D"], device=s["device"]) // (s["D"] // s["G"])
    dt = torch.logaddexp(s["dt"] + s["dt_bias"], torch.zeros((), device=s["device"], dtype=torch.float64))
    y, state = torch.zeros_like(s["x"]), s["state"].clone()
    on = (s["slots"] >= 0).nonzero().flatten()
    h = state[s["slots"][on]] * torch.exp(dt[on][..., None] * s["A"])
    h = h + (dt * s["x"])[on][..., None] * s["Bm"][on][:, group]
    y[on] = torch.einsum("bdn,bdn->bd", h, s["Cm"][on][:, group]) + (s["D_skip"] * s["x"])[on]
    state[s["slots"][on]] = h
    return {"y": y, "state": state}


def _exact_conv(s):
    """torch's convolution in 64 bits, a sequence at a time, and autograd for its gradients."""
    W, D = s["W"], s["D"]
    train = s["mode"] == "train"
    ys, lasts = torch.empty_like(s["x"]), torch.zeros(s["B"], W - 1, D, device=s["device"], dtype=torch.float64)
    w, bias = s["w"].clone().requires_grad_(train), s["bias"].clone().requires_grad_(train)
    dx, dx0 = torch.empty_like(s["x"]), torch.zeros_like(lasts)
    for b, lo, hi, i in _spans(s):
        old = s["x0"][i] if s["x0"] is not None else torch.zeros(W - 1, D, device=s["device"], dtype=torch.float64)
        both = torch.cat([old, s["x"][b, lo:hi]]).requires_grad_(train)
        lasts[i] = both.detach()[both.shape[0] - (W - 1):]
        if hi > lo:
            v = torch.stack([both[k:k + hi - lo] * w[:, k] for k in range(W)]).sum(0) + bias
            y = v / (1 + torch.exp(-v))
            ys[b, lo:hi] = y.detach()
        if train:
            total = (y * s["dy"][b, lo:hi]).sum() if hi > lo else 0.0
            if s["dx_last"] is not None:
                total = total + (both[both.shape[0] - (W - 1):] * s["dx_last"][i]).sum()
            if isinstance(total, torch.Tensor):
                total.backward()
                dx0[i], dx[b, lo:hi] = both.grad[:W - 1], both.grad[W - 1:]
    if not train:
        return {"y": ys, "x_last": lasts}
    return {"y": ys, "x_last": lasts, "dx": dx, "dw": w.grad, "dbias": bias.grad, "dx0": dx0 if s["x0"] is not None else None}


def _exact_conv_token(s):
    y, state = torch.zeros_like(s["x"]), s["state"].clone()
    on = (s["slots"] >= 0).nonzero().flatten()
    seen = torch.cat([state[s["slots"][on]], s["x"][on][:, None]], 1)
    v = torch.einsum("bkd,dk->bd", seen, s["w"]) + s["bias"]
    y[on] = v / (1 + torch.exp(-v))
    state[s["slots"][on]] = seen[:, 1:]
    return {"y": y, "state": state}


def _exact_norm(s):
    """The formula in 64 bits, and autograd for its gradients."""
    train = s["mode"] == "train"
    x, w = s["x"].clone().requires_grad_(train), s["w"].clone().requires_grad_(train)
    z = s["z"].clone().requires_grad_(train) if s["z"] is not None else None
    b = s["b"].clone().requires_grad_(train) if s["b"] is not None else None

    def silu(v):
        return v / (1 + torch.exp(-v))

    p = x * silu(z) if s["gate"] == "first" else x
    q = p.reshape(*p.shape[:-1], s["G"], -1)
    mean = 0 if s["rms"] else q.mean(-1, keepdim=True)
    q = (q - mean) / ((q - mean).pow(2).mean(-1, keepdim=True) + EPS).sqrt()
    o = q.reshape(p.shape) * w
    o = o if b is None else o + b
    y = o if s["gate"] == "first" else silu(o) if z is None else o * silu(z)
    if not train:
        return {"y": y}
    y.backward(s["dy"])
    return {"y": y.detach(), "dx": x.grad, "dw": w.grad, "db": None if b is None else b.grad, "dz": None if z is None else z.grad}


def exact(case, seed):
    s = _f64(prepare(case, seed))
    if case["op"] == "norm":
        return _exact_norm(s)
    if case["mode"] == "token":
        return _exact_scan_token(s) if case["op"] == "scan" else _exact_conv_token(s)
    if case["op"] == "conv":
        return _exact_conv(s)
    return _exact_scan(s)
