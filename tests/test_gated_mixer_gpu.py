"""The gated block built from the operators: tokens one by one against the
prompt, packed prompts against each alone, and its gradients against autograd
of the same formulas in 64 bits (row by row, on the CPU)."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu
F64 = torch.float64


def _mixer(**kw):
    from linear_recurrence_scans_gb300.mixer import GatedMixer
    return GatedMixer(**{**dict(width=24, heads=6, keys=8, values=12, groups=2, dtype=torch.float32, seed=1), **kw})


class _Rounded(torch.autograd.Function):
    """To bf16 and back, the gradient as well."""

    @staticmethod
    def forward(ctx, x):
        return x.bfloat16().double()

    @staticmethod
    def backward(ctx, g):
        return g.bfloat16().double()


def _plain(m, p, u, residual, at=lambda x: x):
    """The block's formulas, float64 on the CPU, one row after another; (out, r).
    `at` rounds what the block keeps in the activations' type."""
    H, G, N, P, W = m.heads, m.groups, m.keys, m.values, m.taps
    C, D, silu = m.mixed, H * P, torch.nn.functional.silu
    B_, T, _ = u.shape
    r = at(at(u) + residual)
    y = at(r / (r.square().mean(-1, keepdim=True) + 1e-5).sqrt() * p["norm_w"])
    f = at(y @ at(p["in"]))
    rows = torch.cat([torch.zeros(B_, W - 1, C, dtype=F64), f[..., :C]], 1)
    xc = at(silu(sum(rows[:, k:k + T] * p["conv_w"][:, k] for k in range(W)) + p["conv_b"]))
    g = -torch.exp(p["A_log"]) * torch.nn.functional.softplus(f[..., C + D:] + p["dt_bias"])
    each = lambda v: v.unflatten(-1, (G, N)).repeat_interleave(H // G, -2)  # noqa: E731
    q, k, v = each(xc[..., :G * N]), each(xc[..., G * N:2 * G * N]), xc[..., 2 * G * N:].unflatten(-1, (H, P))
    S, os = torch.zeros(B_, H, N, P, dtype=F64), []
    for t in range(T):
        S = torch.exp(g[:, t])[..., None, None] * S + k[:, t, :, :, None] * v[:, t, :, None, :]
        os.append(m.scale * (q[:, t, :, :, None] * S).sum(-2))
    o = at(torch.stack(os, 1)) * silu(f[..., C:C + D]).unflatten(-1, (H, P))
    n = at((o / (o.square().mean(-1, keepdim=True) + 1e-5).sqrt()).flatten(-2) * p["out_w"])
    return at(n @ at(p["out"])), r


@pytest.mark.parametrize("groups", [1, 2, 6])
def test_output_and_gradients_against_autograd(cuda_lib, groups):
    m = _mixer(groups=groups)
    p = {k: v.double().cpu().requires_grad_() for k, v in m.p.items()}
    torch.manual_seed(2)
    u, residual, dout, dr = (torch.randn(2, 19, 24) for _ in range(4))
    u64, res64 = u.double().requires_grad_(), residual.double().requires_grad_()
    want, want_r = _plain(m, p, u64, res64)
    torch.autograd.backward([want, want_r], [dout.double(), dr.double()])
    out, r, kept = m.prompt(u.cuda(), residual.cuda(), save=True)
    du, g = m.backward(dout.cuda(), dr.cuda(), kept)
    # float32 through a dozen sums of up to 130 terms and 19 rows; torch's float32 products
    near = lambda a, b: torch.testing.assert_close(a.double().cpu(), b, rtol=1e-3, atol=1e-4 * float(b.abs().max()))  # noqa: E731
    near(out, want.detach())
    near(r, want_r.detach())
    near(du, u64.grad)
    near(du, res64.grad)
    assert set(g) == set(m.p)
    for k in g:
        near(g[k], p[k].grad)


@pytest.mark.parametrize("keys,values", [(16, 16), (64, 128), (40, 24)])
def test_bf16_output_and_gradients(cuda_lib, keys, values):
    m = _mixer(width=64, heads=4, keys=keys, values=values, dtype=torch.bfloat16)
    p = {k: v.double().cpu().requires_grad_() for k, v in m.p.items()}
    torch.manual_seed(5)
    u, residual, dout, dr = (torch.randn(2, 150, 64).bfloat16() for _ in range(4))
    u64, res64 = u.double().requires_grad_(), residual.double().requires_grad_()
    want, want_r = _plain(m, p, u64, res64)
    torch.autograd.backward([want, want_r], [dout.double(), dr.double()])
    out, r, kept = m.prompt(u.cuda(), residual.cuda(), save=True)
    du, g = m.backward(dout.cuda(), dr.cuda(), kept)

    # What the roundings cost is told by the same formulas rounded at the same
    # places.  It is no fixed multiple of 2^-8: where the terms of a row's o nearly
    # cancel, o's norm is small against its error, and the normalisation divides
    # both by it; its gradient goes with 1 / norm, so those rows weigh most.  The
    # recurrence's products round one operand more in themselves (sqrt 2), and two
    # draws of an error that few rows make differ by a factor of 2: 3 in all.
    q = {k: v.detach().clone().requires_grad_() for k, v in p.items()}
    uq, resq = u.double().requires_grad_(), residual.double().requires_grad_()
    rounded = _plain(m, q, uq, resq, _Rounded.apply)
    torch.autograd.backward(rounded, [dout.double(), dr.double()])

    def near(a, b, c):
        a = a.double().cpu()
        assert a.shape == b.shape and torch.isfinite(a).all()
        assert float((a - b).square().mean()) <= 9 * float((c - b).square().mean())

    near(out, want.detach(), rounded[0].detach())
    near(r, want_r.detach(), rounded[1].detach())
    near(du, u64.grad, uq.grad)
    for k in ("in", "out", "conv_w", "out_w", "norm_w"):
        near(g[k], p[k].grad, q[k].grad)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_tokens_continue_the_prompt(cuda_lib, dtype):
    from linear_recurrence_scans_gb300.mixer import States
    m = _mixer(width=64, heads=4, keys=32, values=16, dtype=dtype)
    torch.manual_seed(3)
    u, residual = (torch.randn(3, 140, 64).cuda().to(dtype) for _ in range(2))
    whole, stream = m.prompt(u, residual)
    states, slots = States(m, 5), torch.tensor([4, 1, 2], device="cuda")
    first, r = m.prompt(u[:, :132].contiguous(), residual[:, :132].contiguous(), states, slots)
    rows = [m.token(u[:, t], residual[:, t], states, slots) for t in range(132, 140)]
    # the projections' products may be rounded differently for other shapes
    tol = 2e-4 if dtype == torch.float32 else 4e-2
    torch.testing.assert_close(torch.cat([first, torch.stack([o for o, _ in rows], 1)], 1), whole, rtol=tol, atol=tol)
    assert torch.equal(torch.cat([r, torch.stack([s for _, s in rows], 1)], 1), stream)
    assert (states.scan[[0, 3]] == 0).all() and (states.conv[[0, 3]] == 0).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_packed_prompts_are_the_prompts(cuda_lib, dtype):
    from linear_recurrence_scans_gb300.mixer import States
    m = _mixer(width=64, heads=4, keys=16, values=32, dtype=dtype)
    torch.manual_seed(4)
    ends = (0, 140, 140, 141, 181)
    u, residual = (torch.randn(1, 181, 64).cuda().to(dtype) for _ in range(2))
    cu = torch.tensor(ends, device="cuda")
    states, slots = States(m, 4), torch.arange(4, device="cuda")
    packed, r = m.prompt(u, residual, states, slots, cu_seqlens=cu)
    tol = 2e-4 if dtype == torch.float32 else 4e-2
    for i, (lo, hi) in enumerate(zip(ends, ends[1:])):
        if hi > lo:
            alone = States(m, 1)
            out, s = m.prompt(u[:, lo:hi].contiguous(), residual[:, lo:hi].contiguous(), alone, slots[:1])
            torch.testing.assert_close(packed[:, lo:hi], out, rtol=tol, atol=tol)
            assert torch.equal(r[:, lo:hi], s)
            torch.testing.assert_close(states.scan[i], alone.scan[0], rtol=tol, atol=tol)
            torch.testing.assert_close(states.conv[i], alone.conv[0], rtol=tol, atol=tol)
    assert (states.scan[1] == 0).all() and (states.conv[1] == 0).all()


def test_packed_gradients_are_the_prompts_sum(cuda_lib):
    m = _mixer(width=32, heads=4, keys=16, values=16)
    torch.manual_seed(6)
    ends = (0, 70, 71, 71, 140)
    u, residual, dout, dr = (torch.randn(1, 140, 32).cuda() for _ in range(4))
    _, _, kept = m.prompt(u, residual, cu_seqlens=torch.tensor(ends, device="cuda"), save=True)
    du, g = m.backward(dout, dr, kept)
    want = {k: torch.zeros_like(v, dtype=torch.float32) for k, v in m.p.items()}
    for lo, hi in zip(ends, ends[1:]):
        if hi > lo:
            rows = [t[:, lo:hi].contiguous() for t in (u, residual, dout, dr)]
            _, _, one = m.prompt(rows[0], rows[1], save=True)
            du_one, g_one = m.backward(rows[2], rows[3], one)
            torch.testing.assert_close(du[:, lo:hi], du_one, rtol=1e-3, atol=1e-4 * float(du.abs().max()))
            for k in want:
                want[k] += g_one[k]
    for k in want:
        torch.testing.assert_close(g[k].float(), want[k], rtol=1e-3, atol=1e-4 * float(want[k].abs().max()))


def test_a_token_step_in_a_graph(cuda_lib):
    """A captured step, replayed, goes on from the states that it left."""
    from linear_recurrence_scans_gb300.mixer import States
    m = _mixer(width=64, heads=4, keys=32, values=16, dtype=torch.bfloat16)
    torch.manual_seed(7)
    u, residual = (torch.randn(6, 2, 64).cuda().bfloat16() for _ in range(2))
    eager, states, slots = States(m, 3), States(m, 3), torch.tensor([2, 0], device="cuda")
    want = [m.token(u[t], residual[t], eager, slots) for t in range(6)]
    at, onto = u[0].clone(), residual[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m.token(at, onto, States(m, 3), slots)   # the products' handles and workspaces
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, r = m.token(at, onto, states, slots)
    for t in range(6):
        at.copy_(u[t]), onto.copy_(residual[t])
        graph.replay()
        torch.testing.assert_close(out, want[t][0], rtol=2e-2, atol=2e-2)
        assert torch.equal(r, want[t][1])
    torch.testing.assert_close(states.scan, eager.scan, rtol=2e-2, atol=2e-2)


def test_the_example_runs_both(cuda_lib, capsys):
    from linear_recurrence_scans_gb300 import mixer
    mixer.main()
    said = capsys.readouterr().out
    assert said.count("idle row's largest value 0") == 2 and said.count("step 2") == 2
