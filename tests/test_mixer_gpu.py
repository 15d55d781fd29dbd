"""The mixer layer built from the operators: tokens one by one against the
prompt, packed prompts against each alone, and its gradients against autograd
of the same formulas in 64 bits (row by row, on the CPU)."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu
F64 = torch.float64


def _mixer(**kw):
    from linear_recurrence_scans_gb300.mixer import SelectiveMixer
    return SelectiveMixer(**{**dict(width=24, channels=40, states=8, groups=2, rank=4, dtype=torch.float32, seed=1),
                             **kw})


def _plain(m, p, u):
    """The layer's formulas, float64 on the CPU, one row after another."""
    D, N, G, R, W = m.channels, m.states, m.groups, m.rank, m.taps
    silu = torch.nn.functional.silu
    B_, T, _ = u.shape
    xz = u @ p["in"]
    x, z = xz[..., :D], xz[..., D:]
    rows = torch.cat([torch.zeros(B_, W - 1, D, dtype=F64), x], 1)
    xc = silu(sum(rows[:, k:k + T] * p["conv_w"][:, k] for k in range(W)) + p["conv_b"])
    dbc = xc @ p["x"]
    dt = torch.nn.functional.softplus(dbc[..., :R] @ p["dt"] + p["dt_bias"])
    each = lambda v: v.unflatten(-1, (G, N)).repeat_interleave(D // G, -2)  # noqa: E731
    Bm, Cm, A = each(dbc[..., R:R + G * N]), each(dbc[..., R + G * N:]), -torch.exp(p["A_log"])
    h, ys = torch.zeros(B_, D, N, dtype=F64), []
    for t in range(T):
        h = torch.exp(dt[:, t, :, None] * A) * h + (dt[:, t] * xc[:, t])[..., None] * Bm[:, t]
        ys.append((h * Cm[:, t]).sum(-1) + p["D"] * xc[:, t])
    y = torch.stack(ys, 1)
    q = (y * silu(z) if m.norm["gate_first"] else y).unflatten(-1, (m.norm["groups"], -1))
    if not m.norm["rms"]:
        q = q - q.mean(-1, keepdim=True)
    o = (q / (q.square().mean(-1, keepdim=True) + 1e-5).sqrt()).flatten(-2) * p["norm_w"]
    return (o if m.norm["gate_first"] else o * silu(z)) @ p["out"]


@pytest.mark.parametrize("norm", [dict(), dict(norm_groups=5, rms=False, gate_first=False)], ids=["first", "after"])
def test_output_and_gradients_against_autograd(cuda_lib, norm):
    m = _mixer(**norm)
    p = {k: v.double().cpu().requires_grad_() for k, v in m.p.items()}
    torch.manual_seed(2)
    u, dout = torch.randn(2, 19, 24), torch.randn(2, 19, 24)
    u64 = u.double().requires_grad_()
    want = _plain(m, p, u64)
    want.backward(dout.double())
    out, kept = m.prompt(u.cuda(), save=True)
    du, g = m.backward(dout.cuda(), kept)
    # float32 through a dozen sums of up to 80 terms and 19 rows; torch's float32 products
    near = lambda a, b: torch.testing.assert_close(a.double().cpu(), b, rtol=1e-3, atol=1e-4 * float(b.abs().max()))  # noqa: E731
    near(out, want.detach())
    near(du, u64.grad)
    assert set(g) == set(m.p)
    for k in g:
        near(g[k], p[k].grad)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_tokens_continue_the_prompt(cuda_lib, dtype):
    from linear_recurrence_scans_gb300.mixer import States
    m = _mixer(width=64, channels=128, states=16, groups=1, dtype=dtype)
    torch.manual_seed(3)
    u = torch.randn(3, 20, 64).cuda().to(dtype)
    whole = m.prompt(u)
    states, slots = States(m, 5), torch.tensor([4, 1, 2], device="cuda")
    first = m.prompt(u[:, :12].contiguous(), states, slots)
    rest = torch.stack([m.token(u[:, t], states, slots) for t in range(12, 20)], 1)
    # the projections' products may be rounded differently for other shapes
    tol = 2e-4 if dtype == torch.float32 else 4e-2
    torch.testing.assert_close(torch.cat([first, rest], 1), whole, rtol=tol, atol=tol)
    assert (states.scan[[0, 3]] == 0).all()


def test_packed_prompts_are_the_prompts(cuda_lib):
    from linear_recurrence_scans_gb300.mixer import States
    m = _mixer(width=64, channels=128, states=16, groups=1)
    torch.manual_seed(4)
    u = torch.randn(1, 61, 64).cuda()
    cu = torch.tensor([0, 40, 40, 41, 61], device="cuda")
    states, slots = States(m, 4), torch.arange(4, device="cuda")
    packed = m.prompt(u, states, slots, cu_seqlens=cu)
    for i, (lo, hi) in enumerate(((0, 40), (40, 40), (40, 41), (41, 61))):
        if hi > lo:
            alone = States(m, 1)
            out = m.prompt(u[:, lo:hi].contiguous(), alone, slots[:1])
            torch.testing.assert_close(packed[:, lo:hi], out, rtol=2e-4, atol=2e-4)
            torch.testing.assert_close(states.scan[i], alone.scan[0], rtol=2e-4, atol=2e-4)
            torch.testing.assert_close(states.conv[i], alone.conv[0], rtol=2e-4, atol=2e-4)
    assert (states.scan[1] == 0).all() and (states.conv[1] == 0).all()


def test_example_runs(cuda_lib, capsys):
    from linear_recurrence_scans_gb300 import mixer
    mixer.main()
    said = capsys.readouterr().out
    losses = [float(x.split("loss ")[1]) for x in said.splitlines() if "loss" in x]
    assert len(losses) == 3 and losses[2] < losses[0] and "idle row's largest value 0" in said
