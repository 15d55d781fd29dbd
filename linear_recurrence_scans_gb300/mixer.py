"""A selective state space mixer layer, built from the library's operators.

    python -m linear_recurrence_scans_gb300.mixer

runs a small one through its three uses: packed prompts, single tokens out of a
pool of states, and a training step.

The layer maps u (B, T, E) to (B, T, E):

    x, z = u W_in                            (E -> 2 D, two halves)
    x    = causal_conv(x)                    short, depthwise, SiLU
    dt, B, C = x W_x, dt = dt W_dt           (D -> R + 2 G N, R -> D)
    y    = selective_scan(x, dt, A, B, C)    A = -exp(A_log)
    out  = group_norm(y, gate z) W_out       (D -> E)

The projections are torch's matrix products.  x, z, B and C are read by the
kernels where the projections left them, as slices of wider rows.
"""
from __future__ import annotations

import math

import torch

import linear_recurrence_scans_gb300 as mg


class States:
    """A pool of recurrent states: entry i belongs to one sequence.  Behind the
    pool lies an entry of zeros that stands for every slot outside it."""

    def __init__(self, mixer: "SelectiveMixer", count: int):
        m = mixer
        self._conv = torch.zeros(count + 1, m.taps - 1, m.channels, dtype=m.dtype, device=m.device)
        self._scan = torch.zeros(count + 1, m.channels, m.states, dtype=torch.float32, device=m.device)
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


def main():
    torch.manual_seed(0)
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
    mg.workspace_status()


if __name__ == "__main__":
    main()
