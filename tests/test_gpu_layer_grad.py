"""The norm and rope inside autograd Functions, as a training program wraps them: gradients against autograd's of the
formulas in binary64; refusals outside."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

EPS = 1e-5


def _functions(hq):
    class Norm(torch.autograd.Function):
        """(normalized rows as the codes stand for them, new residual); the codes' rounding passes gradients through."""

        @staticmethod
        def forward(ctx, x, r, w):
            o = hq.add_rmsnorm_fp8_k128(x, w, r, eps=EPS, want_rstd=True)
            ctx.save_for_backward(o["residual_out"], w, o["rstd"])
            y = (o["codes"].view(torch.float8_e4m3fn).float().unflatten(1, (-1, 128)) * o["scales"][..., None]).flatten(1)
            return y, o["residual_out"]

        @staticmethod
        def backward(ctx, dy, dres):
            h, w, rstd = ctx.saved_tensors
            dx, dw = hq.rmsnorm_backward(dy.contiguous(), h, w, rstd, dres=dres.contiguous())
            return dx, dx, dw

    class Rope(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, pos, inv):
            ctx.save_for_backward(pos, inv)
            return hq.rope(q, None, pos, inv, magnitude=1.25)[0]

        @staticmethod
        def backward(ctx, dy):
            pos, inv = ctx.saved_tensors
            return hq.rope(dy.contiguous(), None, pos, inv, magnitude=1.25, inverse=True)[0], None, None

    return Norm, Rope


def test_norm_and_rope_in_a_training_step(hq):
    Norm, Rope = _functions(hq)
    g = torch.Generator(device="cuda").manual_seed(5)
    M, K = 9, 256
    x, r, w = (torch.randn(s, generator=g, device="cuda").requires_grad_() for s in ((M, K), (M, K), (K,)))
    a, b = (torch.randn((M, K), generator=g, device="cuda") for _ in range(2))
    pos, inv = torch.arange(M, device="cuda") * 37, hq.rope_inv_freq(128)[0]
    y, h = Norm.apply(x, r, w)
    z = Rope.apply(y.unflatten(1, (2, 128)), pos, inv).flatten(1)
    got = torch.autograd.grad((z * a).sum() + (h * b).sum(), (x, r, w))

    x64, r64, w64 = (t.detach().double().requires_grad_() for t in (x, r, w))
    h64 = x64 + r64
    h64 = h64 + (h.detach().double() - h64.detach())  # the rounded sum
    y64 = h64 * (h64.square().mean(-1, keepdim=True) + EPS).rsqrt() * w64
    u, v = y64.unflatten(1, (2, 2, 64)).unbind(2)
    c, s = ((1.25 * f(pos.double()[:, None] * inv))[:, None] for f in (torch.cos, torch.sin))
    z64 = torch.cat((u * c - v * s, u * s + v * c), -1).flatten(1)
    want = torch.autograd.grad((z64 * a).sum() + (h64 * b).sum(), (x64, r64, w64))
    # dy: two products and a sum of 32-bit values of order 1 with cosines good to 1e-6 (5e-6 on values up to 4); dx and the
    # sums over 9 rows multiply it by at most 4 and add roundings of sums of 256 products (1e-5 in all)
    for x1, x2 in zip(got, want):
        assert float((x1.double() - x2).abs().max()) < 1e-4
    # the codes: half a step of E4M3 of the normalized rows, and the scales' rounding
    assert bool(((y.detach().double() - y64).abs() <= 0.0626 * y64.abs() + y64.abs().amax() / 448 / 512).all())


def test_a_recorded_backward_pass_is_refused(hq):
    """Second derivatives are not there: refused, not left out."""
    _, Rope = _functions(hq)
    q = torch.zeros((2, 1, 128), device="cuda", requires_grad=True)
    dy = torch.ones((2, 1, 128), device="cuda", requires_grad=True)
    out = Rope.apply(q, torch.arange(2, device="cuda"), hq.rope_inv_freq(128)[0])
    with pytest.raises(hq.HQError, match="no_grad"):
        torch.autograd.grad(out, q, dy, create_graph=True)
    for t in (q, q * 1):
        with pytest.raises(hq.HQError, match="no_grad"):
            hq.rope(t, None, torch.arange(2, device="cuda"), hq.rope_inv_freq(128)[0])
        with torch.no_grad():
            assert not hq.rope(t, None, torch.arange(2, device="cuda"), hq.rope_inv_freq(128)[0])[0].requires_grad
