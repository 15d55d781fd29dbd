"""Mixer layers built from the library's operators: a selective state space mixer,
and a gated block whose recurrence has a matrix state per head.

    python -m linear_recurrence_scans_gb300.mixer

runs a small one of each through its three uses: packed prompts, single tokens
out of a pool of states, and a training step.

The selective mixer maps u (B, T, E) to (B, T, E):

    x, z = u W_in                            (E -> 2 D, two halves)
    x    = causal_conv(x)                    short, depthwise, SiLU
    dt, B, C = x W_x, dt = dt W_dt           (D -> R + 2 G N, R -> D)
    y    = selective_scan(x, dt, A, B, C)    A = -exp(A_log)
    out  = group_norm(y, gate z) W_out       (D -> E)

The gated block maps u and the residual stream it adds to, both (B, T, E), to its
output and the new stream:

    r       = u + residual, y = rms_norm(r)
    qkv, z, dt = y W_in                      (E -> 2 G N + H P, H P, H)
    q, k, v = causal_conv(qkv)               short, depthwise, SiLU
    o       = gated_scan(q, k, v, g)         g = -exp(A_log) softplus(dt + dt_bias)
    out     = group_norm(o, gate z) W_out    (H P -> E), a group a head

The projections are torch's matrix products.  What the kernels take from them
(x, z, B and C; qkv and z) they read where the projections left it, as slices of
wider rows.
"""
from __future__ import annotations

import math

import torch

import linear_recurrence_scans_gb300 as mg


class States:
    """A pool of recurrent states: entry i belongs to one sequence.  Behind the
    pool lies an entry of zeros that stands for every slot outside it."""

    def __init__(self, mixer, count: int):
        conv, scan = mixer.state_shapes()
        self._conv = torch.zeros(count + 1, *conv, dtype=mixer.dtype, device=mixer.device)
        self._scan = torch.zeros(count + 1, *scan, dtype=torch.float32, device=mixer.device)
        self.conv, self.scan = self._conv[:count], self._scan[:count]

    def _at(self, slots):
        count = self.conv.shape[0]
        return torch.where((slots >= 0) & (slots < count), slots, count)

    def take(self, slots):
        """Copies of the slots' (conv, scan) states, zeros for a slot outside the pool."""
        at = self._at(slots)
        return self._conv[at], self._scan[at]

    def put(self, slots, conv, scan):
        """Writes the slots' states; those of a slot outside the pool go nowhere."""
        at = self._at(slots)
        self._conv[at], self._scan[at] = conv, scan
        self._conv[-1].zero_(), self._scan[-1].zero_()


class SelectiveMixer:
    """Parameters as plain tensors in ``self.p``: projections in the
    activations' type, everything else float32."""

    def __init__(self, width, channels, states=16, groups=1, taps=4, rank=None, norm_groups=1,
                 rms=True, gate_first=True, dtype=torch.bfloat16, device="cuda", seed=0):
        self.width, self.channels, self.states, self.groups = width, channels, states, groups
        self.taps, self.rank = taps, rank or -(-width // 16)
        self.norm = dict(groups=norm_groups, rms=rms, gate_first=gate_first)
        self.dtype, self.device = dtype, torch.device(device)
        g = torch.Generator(device).manual_seed(seed)

        def randn(*shape, scale, of=dtype):
            return (torch.randn(shape, generator=g, device=device) * scale).to(of)

        D, N, R = channels, states, self.rank
        step = torch.exp(torch.rand(D, generator=g, device=device) * math.log(100.0) + math.log(1e-3))
        f32 = torch.float32
        self.p = {
            "in": randn(width, 2 * D, scale=width ** -0.5),
            "conv_w": randn(D, taps, scale=taps ** -0.5, of=f32), "conv_b": torch.zeros(D, device=device),
            "x": randn(D, R + 2 * groups * N, scale=D ** -0.5), "dt": randn(R, D, scale=R ** -0.5),
            "A_log": torch.log(torch.arange(1, N + 1, device=device, dtype=f32)).repeat(D, 1),
            "D": torch.ones(D, device=device),
            "dt_bias": step + torch.log(-torch.expm1(-step)),   # softplus(dt_bias) = step
            "norm_w": torch.ones(D, device=device),
            "out": randn(D, width, scale=D ** -0.5),
        }

    def state_shapes(self):
        """Shapes of a sequence's states: the convolution's, the scan's."""
        return (self.taps - 1, self.channels), (self.channels, self.states)

    def _project(self, xc):
        """(dt_low, dt, B, C) of the convolution's output."""
        dbc = xc @ self.p["x"]
        R, GN = self.rank, self.groups * self.states
        shape = (self.groups, self.states)
        low = dbc[..., :R]
        return low, low @ self.p["dt"], dbc[..., R:R + GN].unflatten(-1, shape), dbc[..., R + GN:].unflatten(-1, shape)

    def prompt(self, u, states=None, slots=None, cu_seqlens=None, save=False):
        """out (B,T,E) for whole sequences, dense or (B = 1) packed by
        cu_seqlens.  With states the sequences go on from the entries slots[i]
        of the pool (i without slots) and leave their last states there; a
        sequence whose slot is not in the pool begins from zero and leaves none.
        save=True returns (out, what backward needs)."""
        p, D = self.p, self.channels
        xz = u @ p["in"]
        x, z = xz[..., :D], xz[..., D:]
        x0 = h0 = None
        if states is not None:
            if slots is None:
                slots = torch.arange(u.shape[0] if cu_seqlens is None else cu_seqlens.numel() - 1, device=u.device)
            x0, h0 = states.take(slots)
        xc, x_last = mg.causal_conv_fwd(x, p["conv_w"], p["conv_b"], x0, cu_seqlens=cu_seqlens)
        low, dt, B, C = self._project(xc)
        A = -torch.exp(p["A_log"])
        y, h_last, saved = mg.selective_scan_fwd(xc, dt, A, B, C, p["D"], p["dt_bias"], h0,
                                                 cu_seqlens=cu_seqlens, save=save)
        o, stats = mg.group_norm_fwd(y, p["norm_w"], z=z, **self.norm)
        if states is not None:
            states.put(slots, x_last, h_last)
        out = o @ p["out"]
        return (out, (u, x, z, xc, low, dt, B, C, A, y, o, stats, saved, x0, h0, cu_seqlens)) if save else out

    def token(self, u, states, slots=None):
        """out (B,E) for one token u (B,E) of each row's sequence; row i's state
        is entry slots[i] of the pool (i without slots), updated in place.
        Rows whose slot is not in the pool are idle."""
        p, D = self.p, self.channels
        xz = u @ p["in"]
        xc = mg.causal_conv_step(xz[..., :D], p["conv_w"], states.conv, p["conv_b"], slots=slots)
        _, dt, B, C = self._project(xc)
        y = mg.selective_scan_step(xc, dt, -torch.exp(p["A_log"]), B, C, states.scan, p["D"], p["dt_bias"],
                                   slots=slots)
        o, _ = mg.group_norm_fwd(y, p["norm_w"], z=xz[..., D:], **self.norm)
        return o @ p["out"]

    def backward(self, dout, kept):
        """(du, gradients by parameter name) of sum(dout * out)."""
        u, x, z, xc, low, dt, B, C, A, y, o, stats, saved, x0, h0, cu = kept
        p, g = self.p, {}

        def weight(a, b):   # a^T b over all rows
            return a.reshape(-1, a.shape[-1]).t() @ b.reshape(-1, b.shape[-1])

        g["out"] = weight(o, dout)
        dy, g["norm_w"], _, dz = mg.group_norm_bwd(dout @ p["out"].t(), stats, y, p["norm_w"], z=z, **self.norm)
        dxc, ddt, dA, dB, dC, g["D"], g["dt_bias"], _ = mg.selective_scan_bwd(
            dy, saved, xc, dt, A, B, C, p["D"], p["dt_bias"], h0, cu_seqlens=cu)
        g["A_log"] = dA * A
        g["dt"] = weight(low, ddt)
        ddbc = torch.cat([ddt @ p["dt"].t(), dB.flatten(-2), dC.flatten(-2)], -1)
        g["x"] = weight(xc, ddbc)
        dxc = dxc + ddbc @ p["x"].t()
        dx, g["conv_w"], g["conv_b"], _ = mg.causal_conv_bwd(dxc, x, p["conv_w"], p["conv_b"], x0, cu_seqlens=cu)
        dxz = torch.cat([dx, dz], -1)
        g["in"] = weight(u, dxz)
        return dxz @ p["in"].t(), g


class GatedMixer:
    """Parameters as plain tensors in ``self.p``: projections in the
    activations' type, everything else float32."""

    def __init__(self, width, heads, keys=64, values=64, groups=1, taps=4, dtype=torch.bfloat16, device="cuda", seed=0):
        self.width, self.heads, self.groups, self.keys, self.values, self.taps = width, heads, groups, keys, values, taps
        self.scale, self.dtype, self.device = keys ** -0.5, dtype, torch.device(device)
        self.mixed = 2 * groups * keys + heads * values      # q, k and v
        g = torch.Generator(device).manual_seed(seed)

        def randn(*shape, scale, of=dtype):
            return (torch.randn(shape, generator=g, device=device) * scale).to(of)

        D, C, f32 = heads * values, self.mixed, torch.float32
        step = torch.exp(torch.rand(heads, generator=g, device=device) * math.log(100.0) + math.log(1e-3))
        self.p = {
            "norm_w": torch.ones(width, device=device),
            "in": randn(width, C + D + heads, scale=width ** -0.5),
            "conv_w": randn(C, taps, scale=taps ** -0.5, of=f32), "conv_b": torch.zeros(C, device=device),
            "A_log": torch.log(1 + 15 * torch.rand(heads, generator=g, device=device)),
            "dt_bias": step + torch.log(-torch.expm1(-step)),   # softplus(dt_bias) = step
            "out_w": torch.ones(D, device=device),
            "out": randn(D, width, scale=D ** -0.5),
        }

    def state_shapes(self):
        """Shapes of a sequence's states: the convolution's, the scan's."""
        return (self.taps - 1, self.mixed), (self.heads, self.keys, self.values)

    def _split(self, xc):
        """q, k (..., G, N) and v (..., H, P) of the convolution's output."""
        GN = self.groups * self.keys
        return (xc[..., :GN].unflatten(-1, (self.groups, self.keys)), xc[..., GN:2 * GN].unflatten(-1, (self.groups, self.keys)),
                xc[..., 2 * GN:].unflatten(-1, (self.heads, self.values)))

    def _gates(self, f):
        """(dt + dt_bias, g) of the projection's last H values."""
        raw = f[..., -self.heads:].float() + self.p["dt_bias"]
        return raw, -torch.exp(self.p["A_log"]) * torch.nn.functional.softplus(raw)

    def _norm(self):
        return dict(groups=self.heads, rms=True, gate_first=True)

    def prompt(self, u, residual=None, states=None, slots=None, cu_seqlens=None, save=False):
        """(out, r), both (B,T,E), for whole sequences, dense or (B = 1) packed by
        cu_seqlens; the states as in SelectiveMixer.prompt.  save=True adds what
        backward needs."""
        p, C, D = self.p, self.mixed, self.heads * self.values
        y, r, rstd = mg.rms_norm_fwd(u, p["norm_w"], residual)
        f = y @ p["in"]
        x, z = f[..., :C], f[..., C:C + D]
        x0 = S0 = None
        if states is not None:
            if slots is None:
                slots = torch.arange(u.shape[0] if cu_seqlens is None else cu_seqlens.numel() - 1, device=u.device)
            x0, S0 = states.take(slots)
        xc, x_last = mg.causal_conv_fwd(x, p["conv_w"], p["conv_b"], x0, cu_seqlens=cu_seqlens)
        q, k, v = self._split(xc)
        raw, g = self._gates(f)
        o, S_last, saved = mg.gated_scan_fwd(q, k, v, g, S0, scale=self.scale, cu_seqlens=cu_seqlens, save=save)
        o = o.flatten(-2)
        n, stats = mg.group_norm_fwd(o, p["out_w"], z=z, **self._norm())
        if states is not None:
            states.put(slots, x_last, S_last)
        out = n @ p["out"]
        return (out, r, (y, r, rstd, x, z, xc, raw, g, o, n, stats, saved, x0, S0, cu_seqlens)) if save else (out, r)

    def token(self, u, residual, states, slots=None):
        """(out, r), both (B,E), for one token of each row's sequence; row i's
        state is entry slots[i] of the pool (i without slots), updated in place.
        Rows whose slot is not in the pool are idle."""
        p, C, D = self.p, self.mixed, self.heads * self.values
        y, r, _ = mg.rms_norm_fwd(u, p["norm_w"], residual)
        f = y @ p["in"]
        q, k, v = self._split(mg.causal_conv_step(f[..., :C], p["conv_w"], states.conv, p["conv_b"], slots=slots))
        o = mg.gated_scan_step(q, k, v, self._gates(f)[1], states.scan, slots=slots, scale=self.scale)
        n, _ = mg.group_norm_fwd(o.flatten(-2), p["out_w"], z=f[..., C:C + D], **self._norm())
        return n @ p["out"], r

    def backward(self, dout, dr, kept):
        """(du, gradients by parameter name) of sum(dout * out) + sum(dr * r); du is
        the gradient of u and of the residual alike."""
        y, r, rstd, x, z, xc, raw, gate, o, n, stats, saved, x0, S0, cu = kept
        p, g = self.p, {}

        def weight(a, b):   # a^T b over all rows
            return a.reshape(-1, a.shape[-1]).t() @ b.reshape(-1, b.shape[-1])

        g["out"] = weight(n, dout)
        do, g["out_w"], _, dz = mg.group_norm_bwd(dout @ p["out"].t(), stats, o, p["out_w"], z=z, **self._norm())
        do = do.unflatten(-1, (self.heads, self.values))
        dq, dk, dv, dg, _ = mg.gated_scan_bwd(do, saved, *self._split(xc), gate, S0, scale=self.scale, cu_seqlens=cu)
        g["A_log"] = (dg * gate).flatten(0, -2).sum(0)
        draw = dg * -torch.exp(p["A_log"]) * torch.sigmoid(raw)
        g["dt_bias"] = draw.flatten(0, -2).sum(0)
        dxc = torch.cat([dq.flatten(-2), dk.flatten(-2), dv.flatten(-2)], -1)
        dx, g["conv_w"], g["conv_b"], _ = mg.causal_conv_bwd(dxc, x, p["conv_w"], p["conv_b"], x0, cu_seqlens=cu)
        df = torch.cat([dx, dz, draw.to(self.dtype)], -1)
        g["in"] = weight(y, df)
        du, g["norm_w"] = mg.rms_norm_bwd(df @ p["in"].t(), rstd, r, p["norm_w"], dr)
        return du, g


def _selective():
    m = SelectiveMixer(width=256, channels=512)
    # prompts of 37, 1 and 90 tokens, packed; their states go to slots 2, 0, 3
    cu = torch.tensor([0, 37, 38, 128], device="cuda")
    u = torch.randn(1, 128, 256, device="cuda").to(m.dtype)
    states, slots = States(m, 4), torch.tensor([2, 0, 3], device="cuda")
    out = m.prompt(u, states, slots, cu_seqlens=cu)
    print("prompts:", tuple(out.shape), "mean square %.4f" % out.float().square().mean())
    for _ in range(3):   # three tokens each; the fourth row of the batch is idle
        row = torch.randn(4, 256, device="cuda").to(m.dtype)
        out = m.token(row, states, torch.cat([slots, slots.new_tensor([-1])]))
    print("tokens:", tuple(out.shape), "idle row's largest value %g" % out[3].abs().max())
    # a few steps of plain gradient descent on one batch
    u = torch.randn(4, 64, 256, device="cuda").to(m.dtype)
    target = torch.randn(4, 64, 256, device="cuda").to(m.dtype)
    for step in range(3):
        out, kept = m.prompt(u, save=True)
        err = out.float() - target.float()
        print("step %d: loss %.4f" % (step, err.square().mean()))
        _, grads = m.backward((2 * err).to(m.dtype), kept)
        for name, grad in grads.items():
            m.p[name] = (m.p[name].float() - 2e-4 * grad.float()).to(m.p[name].dtype)


def _gated():
    m = GatedMixer(width=256, heads=8, groups=2)
    # the same prompts, and a residual stream that the block adds to
    cu = torch.tensor([0, 37, 38, 128], device="cuda")
    u, stream = (torch.randn(1, 128, 256, device="cuda").to(m.dtype) for _ in range(2))
    states, slots = States(m, 4), torch.tensor([2, 0, 3], device="cuda")
    out, stream = m.prompt(u, stream, states, slots, cu_seqlens=cu)
    print("prompts:", tuple(out.shape), "mean square %.4f, of the stream %.4f" % (out.float().square().mean(), stream.float().square().mean()))
    for _ in range(3):
        row, stream = (torch.randn(4, 256, device="cuda").to(m.dtype) for _ in range(2))
        out, stream = m.token(row, stream, states, torch.cat([slots, slots.new_tensor([-1])]))
    print("tokens:", tuple(out.shape), "idle row's largest value %g" % out[3].abs().max())
    u, stream, target = (torch.randn(4, 64, 256, device="cuda").to(m.dtype) for _ in range(3))
    for step in range(3):
        out, r, kept = m.prompt(u, stream, save=True)
        err = out.float() + r.float() - target.float()
        print("step %d: mean square error %.4f" % (step, err.square().mean()))
        up = (2 * err).to(m.dtype)
        _, grads = m.backward(up, up, kept)
        for name, grad in grads.items():
            m.p[name] = (m.p[name].float() - 2e-4 * grad.float()).to(m.p[name].dtype)


def main():
    torch.manual_seed(0)
    print("selective mixer")
    _selective()
    print("gated block")
    _gated()
    mg.workspace_status()


if __name__ == "__main__":
    main()
