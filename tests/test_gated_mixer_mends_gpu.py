"""The gated block in bf16 against the same formulas rounded at the same places:
every output and the gradient of every parameter, the gates' among them."""
from __future__ import annotations

import pytest
import torch

from test_gated_mixer_gpu import _mixer, _plain, _Rounded

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,keys,values,groups", [(8, 16, 16, 2), (4, 64, 128, 1), (4, 40, 24, 4), (4, 72, 72, 2)])
def test_bf16_block_is_its_formulas_rounded_once_each(cuda_lib, heads, keys, values, groups):
    """The block rounds where `_plain` does with _Rounded, and nowhere else but to
    2^-16: of its roundings, at 2^-8, one in some 2^8 goes to the other side, so that
    the two results differ by some 2^-4 of the roundings' own error.  Half of it is
    ample; two draws of the same error would differ by 1.4 times it."""
    m = _mixer(width=64, heads=heads, keys=keys, values=values, groups=groups, dtype=torch.bfloat16)
    p = {k: v.double().cpu().requires_grad_() for k, v in m.p.items()}
    q = {k: v.detach().clone().requires_grad_() for k, v in p.items()}
    torch.manual_seed(8)
    u, residual, dout, dr = (torch.randn(2, 150, 64).bfloat16() for _ in range(4))
    results = []
    for params, at in ((p, lambda x: x), (q, _Rounded.apply)):
        x, y = u.double().requires_grad_(), residual.double().requires_grad_()
        outs = _plain(m, params, x, y, at)
        torch.autograd.backward(list(outs), [dout.double(), dr.double()])
        results.append([*(t.detach() for t in outs), x.grad, *(params[k].grad for k in sorted(params))])
    out, r, kept = m.prompt(u.cuda(), residual.cuda(), save=True)
    du, g = m.backward(dout.cuda(), dr.cuda(), kept)
    names = ["out", "r", "du", *sorted(p)]
    for name, a, exact, rounded in zip(names, [out, r, du, *(g[k] for k in sorted(p))], *results):
        a = a.double().cpu()
        assert a.shape == exact.shape and torch.isfinite(a).all()
        off, once = float((a - rounded).norm()), float((rounded - exact).norm())
        assert off <= 0.5 * once, (name, off / once)
