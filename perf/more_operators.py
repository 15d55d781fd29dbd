"""The gated block's operators, as they are measured.

A gated linear recurrence whose state is a matrix per head, and the norm that
such a block begins with: a root-mean-square norm with the residual's addition
in front of it, whose output may be 8 bits wide with scales.  The recurrence has
a form for whole prompts, one for training (forward and gradients) and one for
single tokens that updates a pool of states in place; the norm has a form whose
output keeps the activations' type, one with the output in 8 bits, and one for
training.

``run`` computes a case with elementary torch operations in float32 (in float64
where long sums of the gates are taken), or, where ``own`` is true, with the
library's kernels.  Activations are bf16 or float32; gates, states, weights of
the norm and scales are float32.

Formulas (row t of a sequence, head h of H, its group h // (H / G) of q and k):

    scan    S_t = exp(g_t) S_{t-1} + k_t v_t^T   (N x P),   o_t = scale S_t^T q_t
    norm    r = x + residual, rounded to the activations' type,
            y = r w / sqrt(mean(r^2) + eps)
    8 bits  of each block of a row: scale = max(largest |y|, 1e-30) / 448,
            q = y / scale rounded to e4m3
"""
import math

import torch

own = False

EPS = 1e-5
LEAST, E4M3_MAX = 1e-30, 448.0
CHUNK = 64
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # one user decoding: a single token through one layer's heads
        dict(name="scan_token_1x16x128x128", op="scan", mode="token", B=1, T=1, H=16, G=16, N=128, P=128, dtype="bf16", packed=False, state=True),
        # a serving step of a full batch out of a larger pool of states, some rows idle; all heads share q and k
        dict(name="scan_token_256x32x128x64", op="scan", mode="token", B=256, T=1, H=32, G=1, N=128, P=64, dtype="bf16", packed=False, state=True),
        # one long prompt: few heads, so the kernels have to work along time as well
        dict(name="scan_prompt_1x16384x16x128x128", op="scan", mode="prompt", B=1, T=16384, H=16, G=16, N=128, P=128, dtype="bf16", packed=False, state=False),
        # prompts of uneven lengths packed back to back, continued from earlier states; odd sizes, two groups
        dict(name="scan_packed_5003x6x80x48", op="scan", mode="prompt", B=7, T=5003, H=6, G=2, N=80, P=48, dtype="fp32", packed=True, state=True),
        # a layer's training step, every head with its own q and k
        dict(name="scan_train_4x4096x16x128x128", op="scan", mode="train", B=4, T=4096, H=16, G=16, N=128, P=128, dtype="bf16", packed=False, state=False),
        # a layer's training step with q and k shared by all heads
        dict(name="scan_train_2x4096x32x128x64", op="scan", mode="train", B=2, T=4096, H=32, G=1, N=128, P=64, dtype="bf16", packed=False, state=False),
        # a small float32 training step with odd sizes, from start states
        dict(name="scan_train_3x509x6x24x40", op="scan", mode="train", B=3, T=509, H=6, G=2, N=24, P=40, dtype="fp32", packed=False, state=True),
        # one user decoding: the residual and the norm of one row, 8 bits for the projection behind it
        dict(name="norm_quant_1x4096", op="norm", mode="quant", B=1, T=1, D=4096, block=0, dtype="bf16", residual=True),
        # long prompts, a scale for each 128 channels
        dict(name="norm_quant_32768x4096_b128", op="norm", mode="quant", B=1, T=32768, D=4096, block=128, dtype="bf16", residual=True),
        # long prompts whose projection takes the activations' type
        dict(name="norm_prompt_32768x2048", op="norm", mode="prompt", B=1, T=32768, D=2048, dtype="bf16", residual=True),
        # a layer's training step
        dict(name="norm_train_8x4096x2048", op="norm", mode="train", B=8, T=4096, D=2048, dtype="bf16", residual=True),
        # a small float32 training step, rows of an odd width
        dict(name="norm_train_7x111x1001", op="norm", mode="train", B=7, T=111, D=1001, dtype="fp32", residual=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    dtype = rng.choice(("bf16", "bf16", "fp32"))
    if rng.random() < 0.6:
        mode = rng.choice(("token", "prompt", "train"))
        H = rng.choice((1, 2, 4, 6, 8, 12, 16, 24, 32))
        G = rng.choice([d for d in range(1, H + 1) if H % d == 0])
        N, P = (rng.choice((16, 24, 32, 48, 64, 64, 80, 96, 128, 128, rng.randint(9, 127))) for _ in range(2))
        if mode == "token":
            return dict(op="scan", mode=mode, B=_log_int(rng, 1, 256), T=1, H=H, G=G, N=N, P=P, dtype=dtype, packed=False, state=True)
        packed = rng.random() < 0.4
        B = rng.randint(1, 8)
        # rows x heads at most those of the largest listed case, a quarter in float32
        room = (1 << 18) // H // (1 if dtype == "bf16" else 4)
        T = _log_int(rng, 16, max(32, min(16384, room if packed else room // B)))
        return dict(op="scan", mode=mode, B=B, T=T, H=H, G=G, N=N, P=P, dtype=dtype, packed=packed, state=rng.random() < 0.5)
    mode = rng.choice(("prompt", "quant", "train"))
    case = dict(op="norm", mode=mode, B=rng.randint(1, 8), T=_log_int(rng, 1, 4096), D=_log_int(rng, 64, 4096), dtype=dtype, residual=rng.random() < 0.8)
    if mode == "quant":
        case["block"] = rng.choice((0, 0, 32, 64, 128, 256))
        case["D"] = case["D"] if case["block"] == 0 else case["block"] * max(1, case["D"] // case["block"])
    return case


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(dev).manual_seed(seed * 7919 + 29)
    ty = TYPES[case["dtype"]]
    B, T = case["B"], case["T"]

    def randn(*shape, scale=1.0, of=torch.float32):
        return (torch.randn(shape, generator=gen, device=dev) * scale).to(of)

    s = dict(case, device=dev)
    train = case["mode"] == "train"
    if case["op"] == "norm":
        D = case["D"]
        s["x"] = randn(B, T, D, of=ty)
        # the residual stream has grown over the layers, unevenly over its channels
        s["res"] = (randn(B, T, D, scale=3.0) * torch.exp(randn(D, scale=0.5))).to(ty) if case["residual"] else None
        s["w"] = 1 + randn(D, scale=0.1)
        if train:
            s["dy"] = randn(B, T, D, of=ty)
            s["dres"] = randn(B, T, D, of=ty) if case["residual"] else None
        return s

    H, G, N, P = case["H"], case["G"], case["N"], case["P"]
    token, packed = case["mode"] == "token", case["packed"]
    lead = (B,) if token else ((1, T) if packed else (B, T))
    # q, k and v are slices of one projection's output
    qkv = randn(*lead, 2 * G * N + H * P, of=ty)
    s["q"] = qkv[..., :G * N].unflatten(-1, (G, N))
    s["k"] = qkv[..., G * N:2 * G * N].unflatten(-1, (G, N))
    s["v"] = qkv[..., 2 * G * N:].unflatten(-1, (H, P))
    # heads forget over spans from one row to about a thousand; now and then a row forgets at once
    rate = torch.exp(torch.rand(H, generator=gen, device=dev) * math.log(1e-3))
    gate = -rate * torch.nn.functional.softplus(randn(*lead, H) + 0.5)
    s["g"] = torch.where(torch.rand(*lead, H, generator=gen, device=dev) < 0.002, gate - 30.0, gate)
    s["scale"] = N ** -0.5
    if token:  # a pool of states, larger than the batch; every 17th row is idle
        pool = B + B // 2
        s["slots"] = torch.randperm(pool, generator=gen, device=dev)[:B]
        if B > 1:
            s["slots"][::17] = -1
        s["S"] = randn(pool, H, N, P, scale=2.0)
        return s
    if packed:  # B sequences of uneven lengths, T rows in all
        weights = torch.rand(B, generator=gen, device=dev) + 0.05
        cuts = (weights.cumsum(0) / weights.sum() * T).long()
        cuts[-1] = T
        s["cu"] = torch.cat([torch.zeros(1, dtype=torch.int64, device=dev), cuts])
        s["longest"] = int((s["cu"][1:] - s["cu"][:-1]).max())
    s["S0"] = randn(B, H, N, P, scale=2.0) if case["state"] else None
    if train:
        s["do"] = randn(*lead, H, P, of=ty)
        s["dS_last"] = randn(B, H, N, P) if case["state"] else None
    return s


# ------------------------------------------------------------------ a pass

def run(s):
    return (_own if own else _plain)[s["op"], s["mode"]](s)


def _own_scan_token(s):
    import linear_recurrence_scans_gb300 as mg
    o = mg.gated_scan_step(s["q"], s["k"], s["v"], s["g"], s["S"], slots=s["slots"], scale=s["scale"])
    return {"o": o, "S": s["S"]}


def _own_scan_prompt(s):
    import linear_recurrence_scans_gb300 as mg
    o, S_last, _ = mg.gated_scan_fwd(s["q"], s["k"], s["v"], s["g"], s["S0"], scale=s["scale"], cu_seqlens=s.get("cu"))
    return {"o": o, "S_last": S_last}


def _own_scan_train(s):
    import linear_recurrence_scans_gb300 as mg
    args, more = (s["q"], s["k"], s["v"], s["g"], s["S0"]), dict(scale=s["scale"], cu_seqlens=s.get("cu"))
    o, S_last, saved = mg.gated_scan_fwd(*args, **more, save=True)
    dq, dk, dv, dg, dS0 = mg.gated_scan_bwd(s["do"], saved, *args, s["dS_last"], **more)
    return {"o": o, "S_last": S_last, "dq": dq, "dk": dk, "dv": dv, "dg": dg, "dS0": dS0}


def _own_norm_prompt(s):
    import linear_recurrence_scans_gb300 as mg
    y, r, _ = mg.rms_norm_fwd(s["x"], s["w"], s["res"], eps=EPS)
    return {"y": y, "r": r}


def _own_norm_quant(s):
    import linear_recurrence_scans_gb300 as mg
    q, scale, r = mg.rms_norm_quant(s["x"], s["w"], s["res"], eps=EPS, block=s["block"] or None)
    return {"q": q, "scale": scale, "r": r}


def _own_norm_train(s):
    import linear_recurrence_scans_gb300 as mg
    y, r, rstd = mg.rms_norm_fwd(s["x"], s["w"], s["res"], eps=EPS)
    dx, dw = mg.rms_norm_bwd(s["dy"], rstd, r, s["w"], s["dres"])
    return {"y": y, "r": r, "dx": dx, "dw": dw}


# ------------------------------------------------------------- plain forms
# Float32 throughout (sums of gates in float64), each output rounded once at the end.

def _heads(v, H):
    """(B, T, G, N) to (B, H, T, N) in float32: each group's rows for each of its heads."""
    return v.float().repeat_interleave(H // v.shape[2], 2).transpose(1, 2)


def _dense(s, x):
    """Packed rows (1, T, ...) as a batch (sequences, longest, ...) with zeros behind each sequence."""
    at = s["cu"][:-1, None] + torch.arange(s["longest"], device=s["device"])
    inside = at < s["cu"][1:, None]
    return torch.where(inside.view(*inside.shape, *[1] * (x.dim() - 2)), x[0, at.clamp(max=s["T"] - 1)], torch.zeros((), dtype=x.dtype, device=x.device))


def _packed(s, x):
    """The rows of such a batch back in a row."""
    row = torch.arange(s["T"], device=s["device"])
    seq = torch.searchsorted(s["cu"], row, right=True) - 1
    return x[seq, row - s["cu"][seq]][None]


def _chunks(x):
    """(B, H, T, ...) to (B, H, chunks, CHUNK, ...), zeros behind."""
    B, H, T = x.shape[:3]
    C = -(-T // CHUNK)
    wide = torch.zeros(B, H, C * CHUNK, *x.shape[3:], dtype=x.dtype, device=x.device)
    wide[:, :, :T] = x
    return wide.unflatten(2, (C, CHUNK))


def _rows_again(x, T):
    """Back to (B, T, H, ...)."""
    return x.flatten(2, 3)[:, :, :T].transpose(1, 2)


def _decays(g):
    """Of gates (B, H, C, L): exp of the sums within a chunk up to each row, from each row on to the chunk's end and between its rows; of
    the sums over whole chunks from behind chunk c' to the start of chunk c (0 for c' >= c), and from the sequence's start to it."""
    G = g.double().cumsum(-1)
    ones = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=g.device).tril()
    between = torch.where(ones, (G[..., :, None] - G[..., None, :]).float().exp(), 0.0)
    ends = G[..., -1].cumsum(-1)
    starts = ends - G[..., -1]
    C = g.shape[2]
    earlier = torch.ones(C, C, dtype=torch.bool, device=g.device).tril(-1)
    across = torch.where(earlier, (starts[..., :, None] - ends[..., None, :]).float().exp(), 0.0)
    return G.float().exp(), (G[..., -1:] - G).float().exp(), between, across, starts.float().exp(), ends[..., -1].float().exp(), (ends[..., -1:] - ends).float().exp()


def _over(across, x):
    """Sums over chunks, weighted by `across`, of their matrices (B, H, C, N, P)."""
    return (across @ x.flatten(3)).unflatten(3, x.shape[3:])


def _scan_inputs(s, *names):
    pack = (lambda x: _dense(s, x)) if s.get("cu") is not None else (lambda x: x)
    return [_chunks(_heads(pack(s[n]), s["H"])) for n in names], _chunks(pack(s["g"]).transpose(1, 2))


def _states(k, v, tail, across, first, whole, S0):
    """States at the chunks' starts (B, H, C, N, P) and the last one."""
    added = (k * tail[..., None]).transpose(-1, -2) @ v
    S = _over(across, added)
    if S0 is not None:
        S = S + first[..., None, None] * S0[:, :, None]
    return S, added


def _scan_forward(s):
    (q, k, v), g = _scan_inputs(s, "q", "k", "v")
    up, tail, between, across, first, whole, behind = _decays(g)
    S, added = _states(k, v, tail, across, first, whole, s["S0"])
    S_last = (behind[:, :, None] @ added.flatten(3)).squeeze(2).unflatten(2, added.shape[3:])
    if s["S0"] is not None:
        S_last = S_last + whole[..., None, None] * s["S0"]
    scores = q @ k.transpose(-1, -2)
    o = s["scale"] * ((scores * between) @ v + up[..., None] * (q @ S))
    return (q, k, v), (up, tail, between, across, first, whole, behind), S, scores, S_last, o


def _back(s, x, of):
    """(B, H, C, L, ...) to the caller's rows, in type `of`."""
    rows = s["longest"] if s.get("cu") is not None else s["T"]
    x = _rows_again(x, rows)
    return (_packed(s, x) if s.get("cu") is not None else x).to(of).contiguous()


def _plain_scan_prompt(s):
    *_, S_last, o = _scan_forward(s)
    return {"o": _back(s, o, s["v"].dtype), "S_last": S_last}


def _plain_scan_train(s):
    ty, H, G = s["v"].dtype, s["H"], s["G"]
    (q, k, v), (up, tail, between, across, first, whole, behind), S, scores, S_last, o = _scan_forward(s)
    (do,), _ = _scan_inputs(s, "do")
    do = do * s["scale"]
    # the states' adjoints D behind each chunk, and before the first
    added = (q * up[..., None]).transpose(-1, -2) @ do
    D = _over(across.transpose(-1, -2), added)
    dS0 = (first[:, :, None] @ added.flatten(3)).squeeze(2).unflatten(2, added.shape[3:])
    if s["dS_last"] is not None:
        D = D + behind[..., None, None] * s["dS_last"][:, :, None]
        dS0 = dS0 + whole[..., None, None] * s["dS_last"]
    grads = (do @ v.transpose(-1, -2)) * between
    weights = scores * between
    from_S, from_D = up[..., None] * (do @ S.transpose(-1, -2)), tail[..., None] * (v @ D.transpose(-1, -2))
    dq = grads @ k + from_S
    dk = grads.transpose(-1, -2) @ q + from_D
    dv = weights.transpose(-1, -2) @ do + tail[..., None] * (k @ D)
    # gate t: what reaches rows t.. from rows before t, through the scores, the state before the chunk and the one behind it
    pairs = (scores * grads).tril(-1)
    after = (pairs.sum(-1) - pairs.sum(-2) + (q * from_S).sum(-1)).flip(-1).cumsum(-1).flip(-1)
    before = (k * from_D).sum(-1)
    through = up[..., -1] * (S * D).sum((-1, -2))
    dg = after + before.cumsum(-1) - before + through[..., None]

    def shared(x):  # sums over the heads that share a row
        x = _back(s, x, torch.float32)
        return x.unflatten(2, (G, H // G)).sum(3).to(ty)

    return {"o": _back(s, o, ty), "S_last": S_last, "dq": shared(dq), "dk": shared(dk), "dv": _back(s, dv, ty), "dg": _back(s, dg, torch.float32),
            "dS0": dS0 if s["S0"] is not None else None}


def _plain_scan_token(s):
    live, slot = s["slots"] >= 0, s["slots"].clamp(min=0)
    q, k = (x.float().repeat_interleave(s["H"] // s["G"], 1) for x in (s["q"], s["k"]))
    v = s["v"].float()
    S = s["g"].exp()[..., None, None] * s["S"][slot] + k[..., None] * v[..., None, :]
    o = s["scale"] * (q[..., None] * S).sum(-2)
    s["S"][s["slots"][live]] = S[live]
    return {"o": torch.where(live[:, None, None], o, 0.0).to(s["v"].dtype), "S": s["S"]}


def _norm_parts(s):
    """(the residual stream as it is stored, the same in float32, 1 / root mean square)."""
    r = s["x"] if s["res"] is None else (s["x"].float() + s["res"].float()).to(s["x"].dtype)
    f = r.float()
    return r, f, torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS)


def _plain_norm_prompt(s):
    r, f, rstd = _norm_parts(s)
    return {"y": (f * rstd * s["w"]).to(s["x"].dtype), "r": r}


def _plain_norm_quant(s):
    r, f, rstd = _norm_parts(s)
    y = (f * rstd * s["w"]).unflatten(-1, (-1, s["block"] or s["D"]))
    scale = y.abs().amax(-1).clamp(min=LEAST) / E4M3_MAX
    q = (y / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return {"q": q.flatten(-2), "scale": scale, "r": r}


def _plain_norm_train(s):
    ty = s["x"].dtype
    r, f, rstd = _norm_parts(s)
    n, dy = f * rstd, s["dy"].float()
    dn = dy * s["w"]
    dx = rstd * (dn - n * (dn * n).mean(-1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return {"y": (n * s["w"]).to(ty), "r": r, "dx": dx.to(ty), "dw": (dy * n).sum((0, 1))}


_plain = {("scan", "token"): _plain_scan_token, ("scan", "prompt"): _plain_scan_prompt, ("scan", "train"): _plain_scan_train,
          ("norm", "prompt"): _plain_norm_prompt, ("norm", "quant"): _plain_norm_quant, ("norm", "train"): _plain_norm_train}
_own = {("scan", "token"): _own_scan_token, ("scan", "prompt"): _own_scan_prompt, ("scan", "train"): _own_scan_train,
        ("norm", "prompt"): _own_norm_prompt, ("norm", "quant"): _own_norm_quant, ("norm", "train"): _own_norm_train}


# -------------------------------------------------------------------- work

def work(case):
    """Bytes: inputs once, outputs once (a forward and its gradients read what both need once).  Flops: the recurrence's own products row by row."""
    e = 2 if case["dtype"] == "bf16" else 4
    train = case["mode"] == "train"
    if case["op"] == "norm":
        M, D = case["B"] * case["T"], case["D"]
        act = M * D * e
        ins, outs = (2, 1) if case["residual"] else (1, 0)
        if case["mode"] == "quant":
            return {"bytes": act * (ins + outs) + M * D + 4 * M * (D // (case["block"] or D)) + 4 * D, "flops": 8 * M * D}
        by, fl = act * (ins + outs + 1) + 4 * D, 6 * M * D
        if train:  # reads dy and the residual's gradient, writes dx and dw
            by, fl = by + act * (2 + (1 if case["residual"] else 0)) + 4 * D, fl + 10 * M * D
        return {"bytes": by, "flops": fl}
    R = case["T"] if case["packed"] else case["B"] * case["T"]
    H, G, N, P = case["H"], case["G"], case["N"], case["P"]
    qk, v, g, S = 2 * R * G * N * e, R * H * P * e, 4 * R * H, 4 * case["B"] * H * N * P
    by, fl = qk + 2 * v + g + S * (2 if case["mode"] == "token" or case["state"] else 1), 5 * R * H * N * P
    if train:  # reads do, writes dq, dk, dv and dg
        by, fl = by + qk + 2 * v + g + (2 * S if case["state"] else 0), fl + 11 * R * H * N * P
    return {"bytes": by, "flops": fl}


# ------------------------------------------------------------------- exact

def _walk(q, k, v, g, scale, S, kept=None):
    """The recurrence row by row over (B, T, H, ...) in float64: o and the last state."""
    o = torch.empty_like(v)
    for t in range(v.shape[1]):
        if kept is not None:
            kept[t] = S
        S = torch.exp(g[:, t])[..., None, None] * S + torch.einsum("bhn,bhp->bhnp", k[:, t], v[:, t])
        o[:, t] = scale * torch.einsum("bhn,bhnp->bhp", q[:, t], S)
    return o, S


def _walk_back(q, k, v, g, do, scale, kept, D):
    """Gradients row by row, back from the adjoint D of the last state."""
    dq, dk, dv, dg = (torch.empty_like(x) for x in (q, k, v, g))
    for t in reversed(range(v.shape[1])):
        up = scale * do[:, t]
        a = torch.exp(g[:, t])[..., None, None]
        old = a * kept[t]
        S = old + torch.einsum("bhn,bhp->bhnp", k[:, t], v[:, t])
        dq[:, t] = torch.einsum("bhnp,bhp->bhn", S, up)
        D = D + torch.einsum("bhn,bhp->bhnp", q[:, t], up)
        dk[:, t] = torch.einsum("bhnp,bhp->bhn", D, v[:, t])
        dv[:, t] = torch.einsum("bhnp,bhn->bhp", D, k[:, t])
        dg[:, t] = (D * old).sum((-1, -2))
        D = a * D
    return dq, dk, dv, dg, D


def _exact_scan(s):
    H, G, train = s["H"], s["G"], s["mode"] == "train"
    q, k = (s[n].double()[:, :, torch.arange(H, device=s["device"]) // (H // G)] for n in ("q", "k"))
    v, g = s["v"].double(), s["g"].double()
    zero = torch.zeros(s["B"], H, s["N"], s["P"], dtype=torch.float64, device=s["device"])
    S = zero if s["S0"] is None else s["S0"].double()
    cu = s["cu"].tolist() if s.get("cu") is not None else None
    # (batch entries, rows, states) of what is walked together
    parts = [(slice(None), slice(None), slice(None))] if cu is None else [(slice(0, 1), slice(cu[i], cu[i + 1]), slice(i, i + 1)) for i in range(s["B"])]
    out = {"o": torch.empty_like(v), "S_last": zero.clone()}
    if train:
        do, D = s["do"].double(), zero if s["dS_last"] is None else s["dS_last"].double()
        more = {"dq": torch.empty_like(q), "dk": torch.empty_like(k), "dv": torch.empty_like(v), "dg": torch.empty_like(g), "dS0": zero.clone()}
    for b, r, i in parts:
        x = [y[b, r] for y in (q, k, v, g)]
        kept = torch.empty(x[2].shape[1], *S[i].shape, dtype=torch.float64, device=s["device"]) if train else None
        out["o"][b, r], out["S_last"][i] = _walk(*x, s["scale"], S[i], kept)
        if train:
            more["dq"][b, r], more["dk"][b, r], more["dv"][b, r], more["dg"][b, r], more["dS0"][i] = _walk_back(*x, do[b, r], s["scale"], kept, D[i])
    if train:
        for n in ("dq", "dk"):
            more[n] = more[n].unflatten(2, (G, H // G)).sum(3)
        if s["S0"] is None:
            more["dS0"] = None
        out |= more
    return out


def _exact_token(s):
    o, S = torch.zeros_like(s["v"], dtype=torch.float64), s["S"].double()
    on = (s["slots"] >= 0).nonzero().flatten()
    head = torch.arange(s["H"], device=s["device"]) // (s["H"] // s["G"])
    q, k, v = s["q"].double()[on][:, head], s["k"].double()[on][:, head], s["v"].double()[on]
    new = S[s["slots"][on]] * torch.exp(s["g"].double()[on])[..., None, None] + torch.einsum("bhn,bhp->bhnp", k, v)
    o[on] = s["scale"] * torch.einsum("bhn,bhnp->bhp", q, new)
    S[s["slots"][on]] = new
    return {"o": o, "S": S}


def _exact_norm(s):
    """The formulas in 64 bits, autograd for the gradients.  The stream is rounded as its definition says; q is what e4m3 rounds."""
    ty, train = s["x"].dtype, s["mode"] == "train"
    r = s["x"] if s["res"] is None else (s["x"].double() + s["res"].double()).to(ty)
    r, w = r.double().requires_grad_(train), s["w"].double().requires_grad_(train)
    y = r * w / (r.square().mean(-1, keepdim=True) + EPS).sqrt()
    if s["mode"] == "quant":
        blocks = y.reshape(*y.shape[:-1], -1, s["block"] or s["D"])
        scale = torch.clamp(blocks.abs().amax(-1), min=LEAST) / E4M3_MAX
        return {"q": (blocks / scale[..., None]).reshape(y.shape), "scale": scale, "r": r}
    if not train:
        return {"y": y, "r": r}
    y.backward(s["dy"].double())
    dx = r.grad if s["dres"] is None else r.grad + s["dres"].double()
    return {"y": y.detach(), "r": r.detach(), "dx": dx, "dw": w.grad}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s)
    return _exact_token(s) if case["mode"] == "token" else _exact_scan(s)
