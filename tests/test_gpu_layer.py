"""GPU parity of the attention-layer calls against plain forms in binary64 (exact simulations where results are whole
numbers, the oracle's bits for the cache).  u(t) is half a rounding step of a type relative to the value; every tolerance
counts roundings, as derived beside it."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import oracle
import synthetic as S
from _kv4 import attention64, decode, hadamard128, token_bytes

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: U32}
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape, dtype=F32, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


# ------------------------------------------------------------------- norm
def _depth(K):
    """Longest chain of FP32 additions behind a row's sum: at least 32 lanes share a row, then at most 5 + 32 joins."""
    return K / 32 + 40


def _check_norm(out, x, w, r, eps, transposed=False, ue8m0=False):
    M, K = x.shape
    h = x if r is None else (x.double() + r.double()).to(x.dtype) if x.dtype == F32 else (x.float() + r.float()).to(x.dtype)
    if r is not None:
        assert torch.equal(out["residual_out"], h)
    h = h.double()
    rstd = (h.square().mean(-1) + eps).rsqrt()
    # the sum of squares is off by (depth + 1) roundings at most, the root halves it; 4 more to the result
    tol = (_depth(K) / 2 + 4) * U32
    assert bool(((out["rstd"].double() - rstd).abs() <= tol * rstd).all())
    y = (h * rstd[:, None] * w.double()).unflatten(-1, (-1, 128))
    amax = y.abs().amax(-1)
    scales = out["scales"].double()
    scales = scales.t()[:M] if transposed else scales
    if "amax" in out:
        a = out["amax"].double()
        assert bool((((a.t()[:M] if transposed else a) - amax).abs() <= (tol + 2 * U32) * amax + 1e-37).all())
    want = amax.clamp(min=1e-10) / 448.0
    if ue8m0:
        assert bool((torch.frexp(scales)[0] == 0.5).all())  # powers of two
        assert bool((scales >= want * (1 - 8 * U32 - tol)).all()) and bool((scales < 2 * want * (1 + 8 * U32 + tol)).all())
    else:
        assert bool(((scales - want).abs() <= (tol + 5 * U32) * want).all())
    got = out["codes"].view(torch.float8_e4m3fn).double().unflatten(-1, (-1, 128)) * scales[..., None]
    # half a step of E4M3 (2^-4 of the value, 2^-10 of the scale below its normal range), of a value that is itself off
    # by the row's tol and four roundings
    half = torch.maximum(y.abs() * 2.0 ** -4, scales[..., None] * 2.0 ** -10)
    assert bool(((got - y).abs() <= half * (1 + 2.0 ** -20) + (tol + 4 * U32) * y.abs() * 1.07).all())


@pytest.mark.parametrize("M,K", [(1, 128), (3, 256), (37, 384), (5, 1152), (300, 2048), (19, 7168), (4, 8320), (2, 16512),
                                 (3, 32896), (2, 65536)])
@pytest.mark.parametrize("dtype,wdtype", [(BF16, BF16), (BF16, F32), (F16, F16), (F16, F32), (F32, F32)])
def test_add_rmsnorm(hq, M, K, dtype, wdtype):
    g = _gen(M * 7 + K)
    x, r = _normal(g, M, K, dtype=dtype), _normal(g, M, K, dtype=dtype, std=3.0)
    w = (1 + 0.2 * _normal(g, K)).to(wdtype)
    w[::5] *= -1
    out = hq.add_rmsnorm_fp8_k128(x, w, r, eps=1e-5, want_rstd=True, want_amax=True)
    _check_norm(out, x, w, r, 1e-5)
    out = hq.add_rmsnorm_fp8_k128(x, w, eps=1e-5, scale_layout=hq.HQ_SCALE_TRANSPOSED, scale_ld=M + 3, want_rstd=True)
    _check_norm(out, x, w, None, 1e-5, transposed=True)


def test_add_rmsnorm_many_rows(hq):
    g = _gen(5)
    x, r, w = _normal(g, 5000, 1024, dtype=BF16), _normal(g, 5000, 1024, dtype=BF16), _normal(g, 1024, dtype=BF16)
    out = hq.add_rmsnorm_fp8_k128(x, w, r, want_rstd=True, scale_layout=hq.HQ_SCALE_TRANSPOSED | hq.HQ_FP8_UE8M0)
    _check_norm(out, x, w, r, 1e-6, transposed=True, ue8m0=True)


def test_add_rmsnorm_padding_behind_transposed_scales_is_left(hq):
    g = _gen(6)
    x, w = _normal(g, 5, 256, dtype=BF16), _normal(g, 256, dtype=BF16)
    scales = torch.full((2, 9), 7.0, device="cuda")
    codes = torch.empty((5, 256), dtype=torch.uint8, device="cuda")
    hq.hq_add_rmsnorm_fp8_k128(hq.HQ_DT_BF16, x, 256, None, 0, w, hq.HQ_DT_BF16, 1e-6, 5, 256, None, codes, scales,
                               hq.HQ_SCALE_TRANSPOSED, 9)
    assert bool((scales[:, 5:] == 7.0).all()) and bool((scales[:, :5] != 7.0).all())


@pytest.mark.parametrize("K", [256, 4096, 8320])
def test_add_rmsnorm_in_place_and_strided(hq, K):
    g = _gen(K)
    wide = _normal(g, 11, K + 64, dtype=BF16)
    x = wide[:, 32:32 + K]  # rows of a wider matrix
    r, w = _normal(g, 11, K, dtype=BF16), _normal(g, K, dtype=BF16)
    want = hq.add_rmsnorm_fp8_k128(x.contiguous(), w, r, want_rstd=True)
    r2 = r.clone()
    got = hq.add_rmsnorm_fp8_k128(x, w, r2, want_rstd=True, residual_out=r2)
    assert got["residual_out"] is r2
    for k in want:
        assert torch.equal(got[k], want[k]), k
    x2 = x.contiguous().clone()
    got = hq.add_rmsnorm_fp8_k128(x2, w, r, want_rstd=True, residual_out=x2)
    for k in want:
        assert torch.equal(got[k], want[k]), k


def test_add_rmsnorm_rows_with_special_values(hq):
    K = 512
    g = _gen(9)
    x, w = _normal(g, 6, K, dtype=F32), torch.ones(K, device="cuda")
    clean = hq.add_rmsnorm_fp8_k128(x, w, want_rstd=True)
    x[1] = 0.0
    x[2, 5] = math.nan
    x[3, 7] = math.inf
    x[4] *= 1e-30
    out = hq.add_rmsnorm_fp8_k128(x, w, want_rstd=True)
    for m in (0, 5):  # other rows are not touched by their neighbours
        assert torch.equal(out["codes"][m], clean["codes"][m]) and out["rstd"][m] == clean["rstd"][m]
    v = out["codes"].view(torch.float8_e4m3fn).float()
    assert bool((v[1] == 0).all()) and bool((out["scales"][1] == np.float32(1e-10) * np.float32(1 / 448)).all())
    assert bool(torch.isnan(v[2]).all())                      # rstd is NaN: every value is
    assert bool(torch.isnan(v[3, 7])) and bool((v[3, :7] == 0).all()) and out["rstd"][3] == 0
    assert abs(float(out["rstd"][4]) - 1000.0) < 1e-2         # eps carries a row of vanishing values


def test_add_rmsnorm_empty(hq):
    x, w = torch.empty((0, 256), dtype=BF16, device="cuda"), torch.ones(256, dtype=BF16, device="cuda")
    out = hq.add_rmsnorm_fp8_k128(x, w, x)
    assert out["codes"].shape == (0, 256) and out["scales"].shape == (0, 2)


def _norm_grads64(dy, h, w, rstd, dres):
    g = dy.double() * w.double()
    h, rs = h.double(), rstd.double()[:, None]
    c = rs * rs * (g * h).mean(-1, keepdim=True)
    dx = rs * (g - h * c)
    terms = dy.double() * h * rs
    return (dx if dres is None else dx + dres.double()), terms.sum(0), terms.abs().sum(0), g, c, rs


@pytest.mark.parametrize("M,K", [(1, 128), (2, 256), (37, 384), (700, 1152), (333, 2048), (19, 7168), (5, 16512), (2, 65536)])
@pytest.mark.parametrize("dtype,wdtype", [(BF16, BF16), (F16, F32), (F32, F32)])
def test_rmsnorm_backward(hq, M, K, dtype, wdtype):
    g = _gen(M + 3 * K)
    dy, h = _normal(g, M, K, dtype=dtype, std=0.1), _normal(g, M, K, dtype=dtype, std=2.0)
    w = (1 + 0.2 * _normal(g, K)).to(wdtype)
    rstd = (h.float().square().mean(-1) + 1e-6).rsqrt()
    for dres in (None, _normal(g, M, K, dtype=dtype, std=0.1)):
        dx, dw = hq.rmsnorm_backward(dy, h, w, rstd, dres=dres)
        want, dw64, dw_abs, gg, c, rs = _norm_grads64(dy, h, w, rstd, dres)
        # c is off by the chain of its sum of products: depth + 4 roundings of sum |g h| / K; then 4 roundings of each
        # term and the result's own
        c_abs = rs * rs * (gg * h.double()).abs().mean(-1, keepdim=True)
        err = rs * h.double().abs() * c_abs * (_depth(K) + 8) * U32 + rs * gg.abs() * 6 * U32
        err = err + want.abs() * (U[dtype] + 2 * U32) + (0 if dres is None else dres.double().abs() * 2 * U32) + 1e-7 * (dtype == F16)
        assert bool(((dx.double() - want).abs() <= err).all())
        # each column's terms are off by 3 roundings, their sum by one for each addition of the longest chain (<= M + 8)
        assert bool(((dw.double() - dw64).abs() <= (M + 12) * U32 * dw_abs).all())


def test_rmsnorm_backward_against_differences(hq):
    """dx and dweight of a scalar loss against central differences of the forward formula in binary64."""
    g = _gen(12)
    M, K, eps = 2, 128, 1e-5
    h, w, dy = _normal(g, M, K), 1 + 0.3 * _normal(g, K), _normal(g, M, K)
    rstd = (h.double().square().mean(-1) + eps).rsqrt().float()
    dx, dw = hq.rmsnorm_backward(dy, h, w, rstd)

    def loss(h, w):
        return (h * (h.square().mean(-1, keepdim=True) + eps).rsqrt() * w * dy.double()).sum()

    h64, w64, step = h.double(), w.double(), 1e-5
    for i in range(0, M * K, 7):
        e = torch.zeros(M * K, dtype=torch.float64, device="cuda")
        e[i] = step
        e = e.view(M, K)
        d = (loss(h64 + e, w64) - loss(h64 - e, w64)) / (2 * step)
        # differences: step^2 of the third derivative (of order 1 here) and cancellation, below 1e-8; FP32 results:
        # values of order 1 through sums of 128 products, below 1e-5
        assert abs(float(d) - float(dx.flatten()[i])) < 2e-5
    for i in range(0, K, 5):
        e = torch.zeros(K, dtype=torch.float64, device="cuda")
        e[i] = step
        d = (loss(h64, w64 + e) - loss(h64, w64 - e)) / (2 * step)
        assert abs(float(d) - float(dw[i])) < 2e-5


def test_rmsnorm_backward_repeats_strides_in_place_and_empty(hq):
    g = _gen(13)
    M, K = 1021, 512
    both = _normal(g, M, 2 * K, dtype=BF16)
    dy, h = both[:, :K], both[:, K:]
    w, dres = _normal(g, K, dtype=BF16), _normal(g, M, K, dtype=BF16)
    rstd = (h.float().square().mean(-1) + 1e-6).rsqrt()
    dx, dw = hq.rmsnorm_backward(dy.contiguous(), h.contiguous(), w, rstd, dres=dres)
    ws = hq.rmsnorm_backward_workspace(M, K)
    ws.fill_(0xFF)  # any contents
    for _ in range(3):  # fixed order: the same bits every time
        dx2, dw2 = hq.rmsnorm_backward(dy, h, w, rstd, dres=dres, ws=ws)
        assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    d = dy.contiguous()
    dx3, dw3 = hq.rmsnorm_backward(d, h, w, rstd, dres=dres, dx=d)
    assert dx3 is d and torch.equal(dx3, dx) and torch.equal(dw3, dw)
    r = dres.clone()
    dx4, dw4 = hq.rmsnorm_backward(dy, h, w, rstd, dres=r, dx=r, want_dweight=False)
    assert dw4 is None and torch.equal(dx4, dx)
    dx0, dw0 = hq.rmsnorm_backward(dy[:0], h[:0], w, rstd[:0])
    assert dx0.shape == (0, K) and bool((dw0 == 0).all())


# ------------------------------------------------------------------- rope
def _rope64(x, pos, inv, offset, interleaved, mag, inverse):
    R = 2 * inv.numel()
    a = pos.double()[:, None] * inv
    c, s = (a.cos() * mag)[:, None], (a.sin() * mag * (-1 if inverse else 1))[:, None]
    y = x.double().clone()
    z = x.double()[..., offset:offset + R]
    u, v = (z[..., 0::2], z[..., 1::2]) if interleaved else (z[..., :R // 2], z[..., R // 2:])
    p, q = u * c - v * s, u * s + v * c
    size = u.abs() + v.abs()
    y[..., offset:offset + R] = torch.stack((p, q), -1).flatten(-2) if interleaved else torch.cat((p, q), -1)
    b = torch.zeros_like(y)
    b[..., offset:offset + R] = torch.stack((size, size), -1).flatten(-2) if interleaved else torch.cat((size, size), -1)
    return y, b * mag


@pytest.mark.parametrize("T,Hq,Hk,D,R,offset", [(1, 1, 1, 64, 64, 0), (3, 5, 2, 128, 64, 0), (17, 3, 1, 128, 128, 0),
                                                (5, 4, 4, 192, 64, 128), (2, 3, 2, 80, 20, 16), (9, 2, 1, 70, 70, 0),
                                                (4, 1, 0, 33, 2, 31), (64, 64, 8, 128, 64, 64), (3, 2, 2, 256, 200, 8)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_rope(hq, T, Hq, Hk, D, R, offset, interleaved, dtype):
    g = _gen(T + D + R)
    q = _normal(g, T, Hq, D, dtype=dtype)
    k = _normal(g, T, Hk, D, dtype=dtype) if Hk else None
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device="cuda")
    pos[0] = 0
    pos[-1] = -12345
    inv, _ = hq.rope_inv_freq(R)
    layout = hq.HQ_ROPE_INTERLEAVED if interleaved else hq.HQ_ROPE_HALVES
    for mag, inverse in ((1.0, False), (1.25, True)):
        got = hq.rope(q, k, pos, inv, offset=offset, layout=layout, magnitude=mag, inverse=inverse)
        for x, y in zip((q, k), got):
            if x is None:
                assert y is None
                continue
            want, size = _rope64(x, pos, inv, offset, interleaved, mag, inverse)
            # cos and sin: 4e-7 of the angle + 2^20 2^-50, 2 ulp of the functions, the magnitude's rounding; two products
            # and a sum; then the result's own rounding
            assert bool(((y.double() - want).abs() <= U[dtype] * want.abs() + 1e-6 * size + 6e-8 * (dtype == F16)).all())


def test_rope_far_positions_and_back(hq):
    g = _gen(21)
    q = _normal(g, 6, 2, 128)
    pos = torch.tensor([0, 1, 1 << 24, (1 << 31) + 7, -(1 << 31), 1 << 40], device="cuda")
    inv, mag = hq.rope_inv_freq(128, 1e6, hq.HQ_ROPE_PARTS, 16.0, 8192)
    got, _ = hq.rope(q, None, pos, inv, magnitude=mag)
    # whole turns taken off in exact arithmetic: position * frequency as rationals of the doubles
    from fractions import Fraction
    pi = Fraction(314159265358979323846264338327950288419716939937510582097494459, 10 ** 62)
    for t, p in enumerate(pos.tolist()):
        for i, f in enumerate(inv.tolist()):
            x = Fraction(p) * Fraction(f) / (2 * pi)
            a = float((x - math.floor(x)) * 2 * pi)
            u, v = float(q[t, 0, i]), float(q[t, 0, i + 64])
            # the stated bound on the angle, and roundings as above
            tol = mag * (abs(u) + abs(v)) * (1e-6 + abs(p) * f * 2.0 ** -50)
            assert abs(float(got[t, 0, i]) - mag * (u * math.cos(a) - v * math.sin(a))) <= tol, (p, i)
            assert abs(float(got[t, 0, i + 64]) - mag * (u * math.sin(a) + v * math.cos(a))) <= tol, (p, i)


def test_rope_gradient_is_the_inverse(hq):
    """<rope(x), dy> == <x, rope(dy, inverse)>: the transpose, for any magnitude; and differences along a direction."""
    g = _gen(22)
    x, dy, step = _normal(g, 7, 3, 128), _normal(g, 7, 3, 128), 0.25
    pos = torch.randint(0, 5000, (7,), generator=g, device="cuda")
    inv, _ = hq.rope_inv_freq(96)
    kw = dict(offset=16, layout=hq.HQ_ROPE_INTERLEAVED, magnitude=1.3)
    y, _ = hq.rope(x, None, pos, inv, **kw)
    dx, _ = hq.rope(dy, None, pos, inv, inverse=True, **kw)
    # 2688 products of order 1, each off by about 3e-7 relative to its pair
    assert abs(float((y.double() * dy.double()).sum() - (x.double() * dx.double()).sum())) < 2688 * 4e-6
    e = _normal(g, 7, 3, 128)
    up, _ = hq.rope(x + step * e, None, pos, inv, **kw)
    down, _ = hq.rope(x - step * e, None, pos, inv, **kw)
    d = ((up.double() - down.double()) * dy.double()).sum() / (2 * step)  # linear: no truncation error
    assert abs(float(d - (e.double() * dx.double()).sum())) < 2688 * 2e-5


@pytest.mark.parametrize("D,R,offset", [(128, 64, 64), (128, 128, 0), (72, 36, 4)])
def test_rope_strided_and_in_place(hq, D, R, offset):
    g = _gen(23)
    T, Hq, Hk = 33, 8, 2
    qkv = _normal(g, T, (Hq + 2 * Hk) * D, dtype=BF16)
    q, k = qkv[:, :Hq * D].unflatten(1, (Hq, D)), qkv[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D))
    pos = torch.randint(0, 9999, (T,), generator=g, device="cuda")
    inv, _ = hq.rope_inv_freq(R)
    want = hq.rope(q.contiguous(), k.contiguous(), pos, inv, offset=offset)
    got = hq.rope(q, k, pos, inv, offset=offset)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    rest = qkv[:, (Hq + Hk) * D:].clone()
    hq.rope(q, k, pos, inv, offset=offset, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(qkv[:, (Hq + Hk) * D:], rest)


def test_rope_without_heads_on_one_side(hq):
    """q without heads but with pointers, k in place; and the other way round."""
    g = _gen(24)
    T, H, D, R = 5, 3, 256, 88
    x, pos = _normal(g, T, H, D, dtype=BF16), torch.randint(0, 9999, (T,), generator=g, device="cuda")
    inv, _ = hq.rope_inv_freq(R)
    other = torch.full_like(x, 7.0)
    for layout in (hq.HQ_ROPE_HALVES, hq.HQ_ROPE_INTERLEAVED):
        want, _ = hq.rope(x, None, pos, inv, layout=layout)
        for heads in ((0, H), (H, 0)):
            y = x.clone()
            side = [(y, H * D, D, n, y) if n else (other, H * D, D, 0, x) for n in heads]
            hq.hq_rope(hq.HQ_DT_BF16, *side[0][:4], *side[1][:4], T, D, pos, inv, R, 0, layout, 1.0, 0, side[0][4], H * D, D,
                       side[1][4], H * D, D)
            assert torch.equal(y, want) and bool((other == 7.0).all())


# ------------------------------------------------------------------- slots
def _slots_by_hand(lens, new, table, stack, count, page, n_slots):
    B, W = table.shape
    cap, bad = len(stack), 0
    pages = lambda n: -(-n // page)  # noqa: E731
    for n, a in zip(lens, new):
        if n < 0 or n > W * page:
            bad |= 8
        elif a >= 0 and n + a > W * page:
            bad |= 4
    good = [0 <= n <= W * page and not (a >= 0 and n + a > W * page) for n, a in zip(lens, new)]
    back = sum(pages(n) for n, a, g in zip(lens, new, good) if g and a < 0)
    need = sum(pages(n + a) - pages(n) for n, a, g in zip(lens, new, good) if g and a >= 0)
    total = sum(a for a, g in zip(new, good) if g and a > 0)
    if not 0 <= count <= cap or count + back > cap:
        bad |= 8
    if need > count + back:
        bad |= 1
    if total > n_slots:
        bad |= 2
    if bad:
        return lens, [0] * (B + 1), [-1] * n_slots, [0] * n_slots, table, stack, count, bad
    table, stack, top = table.copy(), list(stack), count
    for b, (n, a) in enumerate(zip(lens, new)):
        if a < 0:
            for i in range(pages(n)):
                stack[top] = int(table[b, i])
                top += 1
    cu, slots, pos, out = [0], [], [], []
    for b, (n, a) in enumerate(zip(lens, new)):
        if a >= 0:
            for i in range(pages(n), pages(n + a)):
                top -= 1
                table[b, i] = stack[top]
            for t in range(n, n + a):
                slots.append(int(table[b, t // page]) * page + t % page)
                pos.append(t)
        out.append(0 if a < 0 else n + a)
        cu.append(len(slots))
    pad = n_slots - len(slots)
    return out, cu, slots + [-1] * pad, pos + [0] * pad, table, stack, top, 0


def _slots_case(hq, lens, new, width, page, n_slots, spare, seed=0, in_place=False):
    rng = np.random.RandomState(seed)
    held = [max(0, -(-n // page)) if n <= width * page else 0 for n in lens]
    order = rng.permutation(sum(held) + spare).astype(np.int32)
    table = np.full((len(lens), width), -7, np.int32)
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = order[at:at + h]
        at += h
    stack = list(order[at:]) + [-9] * at
    want = _slots_by_hand(list(lens), list(new), table, stack, spare, page, n_slots)
    i32 = dict(dtype=torch.int32, device="cuda")
    t_lens, t_new = torch.tensor(lens, **i32), torch.tensor(new, **i32)
    t_table, t_stack, t_count = torch.tensor(table, **i32).view(len(lens), width), torch.tensor(np.array(stack), **i32), torch.tensor([spare], **i32)
    kw = dict(lens_out=t_lens, free_count_out=t_count) if in_place else {}
    o = hq.kv_slots(t_lens, t_new, t_table, t_stack, t_count, page, n_slots, **kw)
    got = (o["lens"], o["cu_new"], o["slots"], o["positions"], t_table, t_stack, o["free_count"], o["status"])
    for name, g, w in zip(("lens", "cu", "slots", "positions", "table", "stack", "count", "status"), got, want):
        assert np.array_equal(g.cpu().numpy().reshape(-1), np.array(w).reshape(-1)), name
    return want[-1]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,page,longest,new,ended", [(1, 16, 50, 1, 0), (3, 16, 100, 5, 0.4), (64, 64, 3000, 1, 0.1),
                                                      (257, 32, 900, 40, 0.2), (1025, 128, 500, 3, 0.1),
                                                      (4096, 16, 64, 2, 0.3), (7, 1024, 5000, 9000, 0), (5, 16, 0, 1, 0)])
def test_kv_slots(hq, B, page, longest, new, ended, in_place):
    rng = np.random.RandomState(B + page)
    lens = rng.randint(0, longest + 1, B).tolist()
    add = [-1 if rng.rand() < ended else int(rng.randint(0, new + 1)) for _ in range(B)]
    width = (longest + new) // page + 2
    total = sum(max(a, 0) for a in add)
    assert _slots_case(hq, lens, add, width, page, total + 13, sum((a + page) // page for a in add if a >= 0) + 1, B,
                       in_place) == 0
    assert _slots_case(hq, lens, add, width, page, total, B * ((new + page) // page) + 5, B, in_place) == 0


def test_kv_slots_refusals_leave_everything(hq):
    # too few pages, too few rows, a row of the table outgrown, lengths out of range; each alone and together
    assert _slots_case(hq, [16, 32, 5], [1, 1, 30], 8, 16, 64, 3) == hq.HQ_KV_NO_PAGES
    assert _slots_case(hq, [16, 32, 5], [1, 1, 30], 8, 16, 31, 9) == hq.HQ_KV_NO_ROWS
    assert _slots_case(hq, [16, 32, 5], [1, 1, 30], 2, 16, 64, 9) == hq.HQ_KV_NO_WIDTH
    assert _slots_case(hq, [-1, 32, 5], [1, 1, 30], 8, 16, 64, 9) == hq.HQ_KV_BAD_STATE
    assert _slots_case(hq, [1, 32, 129], [1, 1, -1], 8, 16, 64, 9) == hq.HQ_KV_BAD_STATE
    assert _slots_case(hq, [1, 128, 129], [1, 1, 500], 8, 16, 1, 0) & hq.HQ_KV_NO_WIDTH
    # pages of an ended request serve the others of the same step
    assert _slots_case(hq, [64, 16], [-1, 40], 8, 16, 64, 0) == 0
    # sums of new tokens beyond 32 bits do not wrap
    assert _slots_case(hq, [0] * 4, [2 ** 30] * 4, 2 ** 21, 1024, 8, 5) & hq.HQ_KV_NO_ROWS


# ------------------------------------------------------------------- cache
def _bf16_bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


@pytest.mark.parametrize("N,H,page,rotate", [(1, 1, 16, 128), (5, 2, 16, 0), (40, 3, 32, 128), (64, 8, 64, 128),
                                             (300, 1, 128, 128), (33, 5, 1024, 0), (100, 4, 16, 128)])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_kv4_append_has_the_oracles_bits(hq, N, H, page, rotate, dtype):
    """Every byte of the written tokens against the oracle's NVFP4 form of the 128-vectors; every other byte as it was."""
    g = _gen(N + page)
    pages = -(-N // page) + 3
    # values that BF16 holds, so that the oracle's input is the same in every type (FP16: from its normal range)
    k, v = _normal(g, N, H, 128, dtype=BF16), (_normal(g, N, H, 128) * torch.exp(_normal(g, N, H, 1))).to(BF16)
    k[0, 0] = 0
    if dtype == F16:
        k, v = (torch.where(t.abs() < 2.0 ** -10, torch.zeros_like(t), t) for t in (k, v))
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:N]
    cache = torch.randint(0, 256, (pages, H, page // 16, 2432), generator=g, device="cuda", dtype=torch.uint8)
    before = cache.cpu().numpy().copy()
    hq.kv4_append(k.to(dtype), v.to(dtype), slots, cache, hadamard_n=rotate)
    after = cache.cpu().numpy()
    touched = np.zeros(after.shape, bool)
    for value, x in ((False, k), (True, v)):
        want = oracle.cat_rotate_nvfp4(_bf16_bits(x), None, N, H, rotate)
        for i, s in enumerate(slots.cpu().tolist()):
            for h in range(H):
                at = (s // page, h, s % page // 16)
                codes, sf, dec = token_bytes(after[at], s % 16, value)
                assert np.array_equal(codes, want["codes"][i, 64 * h:64 * h + 64]), (i, h, value)
                assert np.array_equal(sf, want["block_sf"][i, 8 * h:8 * h + 8])
                assert dec.view(np.uint32) == want["sdec"][i, h].view(np.uint32)
                mark = np.arange(2432)
                first = (2368 if value else 2304) + 4 * (s % 16)
                touched[at][first:first + 4] = True
                for b in range(8):
                    r = s % 16
                    touched[at][2176 + 64 * (r // 8) + 16 * (r % 8 // 2) + 2 * b + r % 2 if value else 2048 + 8 * r + b] = True
                    for p in range(8):
                        touched[at][1024 + 512 * (r // 8) + 64 * p + 16 * (r % 8 // 2) + 8 * (r % 2) + b if value
                                    else 64 * r + 16 * (p // 2) + 2 * b + p % 2] = True
                assert mark.size == 2432
    assert np.array_equal(after[~touched], before[~touched])


def test_kv4_append_skips_slots_outside_and_takes_strides(hq):
    g = _gen(31)
    N, H, page, pages = 50, 4, 32, 5
    kv = _normal(g, N, 3, H, 128, dtype=BF16)
    k, v = kv[:, 0], kv[:, 2]
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:N]
    want = hq.kv4_cache(pages, page, H)
    hq.kv4_append(k[3:].contiguous(), v[3:].contiguous(), slots[3:].contiguous(), want)
    slots[0], slots[1], slots[2] = -1, pages * page, -(1 << 40)
    got = hq.kv4_cache(pages, page, H)
    hq.kv4_append(k, v, slots, got)
    assert torch.equal(got, want)
    hq.kv4_append(k[:0], v[:0], slots[:0], got)
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("rotate", [0, 128])
def test_kv4_gather(hq, dtype, rotate):
    g = _gen(32)
    N, H, page, pages = 70, 3, 64, 3
    cache = hq.kv4_cache(pages, page, H)
    k, v = _normal(g, N, H, 128, dtype=BF16), _normal(g, N, H, 128, dtype=BF16)
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:N]
    hq.kv4_append(k, v, slots, cache)
    ask = torch.cat((slots, slots[:5], torch.tensor([-1, pages * page], device="cuda")))
    got = hq.kv4_gather(cache, ask, dtype=dtype, hadamard_n=rotate)
    h = torch.from_numpy(hadamard128()).cuda()
    for value, y, x in ((False, got[0], k), (True, got[1], v)):
        all_ = decode(cache, value).permute(0, 2, 3, 1, 4).reshape(pages * page, H, 128)[ask.clamp(0, pages * page - 1)]
        all_[-2:] = 0
        want = all_ @ h if rotate else all_
        # one product's rounding as stored (code * block scale is exact); rotated: 7 additions and a product more, of
        # sums no larger than the 1-norm; then the type's own rounding
        size = all_.abs().sum(-1, keepdim=True) / 128 ** 0.5 if rotate else all_.abs()
        assert bool(((y.double() - want).abs() <= U[dtype] * want.abs() + 10 * U32 * size + 6e-8 * (dtype == F16)).all())
        if rotate:  # what was written comes back, off by the 4-bit rounding: at most a sixth of a block's largest value,
            # about 0.1 of the vector's norm for normal data; a permuted or mis-signed element would be off by more than 1
            rel = (y[:N].double() - x.double()).norm() / x.double().norm()
            assert float(rel) < 0.2


# --------------------------------------------------------------- attention
def _filled(hq, g, B, Hkv, page, lens, rotate, spare=2):
    """A cache with B requests of given lengths on shuffled pages: (cache, table [B, W], lens)."""
    held = [-(-n // page) for n in lens]
    pages, W = sum(held) + spare, max(max(held), 1)
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    cache = torch.randint(0, 256, (pages, Hkv, page // 16, 2432), generator=g, device="cuda", dtype=torch.uint8)
    table = torch.full((B, W), -1, dtype=torch.int32, device="cuda")
    at, slots = 0, []
    for b, n in enumerate(held):
        table[b, :n] = order[at:at + n]
        at += n
        t = torch.arange(lens[b], device="cuda")
        slots.append(table[b].long()[t // page] * page + t % page)
    slots = torch.cat(slots)
    k = _normal(g, len(slots), Hkv, 128, dtype=BF16)
    v = _normal(g, len(slots), Hkv, 128, dtype=BF16)
    if len(slots):
        hq.kv4_append(k, v, slots, cache, hadamard_n=rotate)
    return cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda")


def _check_attention(got, lse, q, cache, table, lens, rows, scale, window, sinks, rotate):
    want, lse64, weight, peak = attention64(q, cache, table, lens, rows, scale, window, sinks, rotate)
    used = torch.zeros(q.shape[0], dtype=torch.bool, device="cuda")
    for a, b in rows:
        used[a:b] = True
    assert bool(torch.isfinite(got[used]).all())
    # score: |q| |k| bounds the products' sum; a 128-term FP32 chain and the query's two parts: 2^-17 of it
    norms = q.double().norm(dim=-1, keepdim=True) * 16.0 * scale  # |k| < 16: normal data of 128 dimensions
    ds = 2.0 ** -17 * norms
    # a weight: one FP16 rounding (2^-11; the bound leaves room for two), the score's error, exp; below FP16's normal range
    # 2^-25 of the largest weight each, on values below 8 (their rotation back adds up to sqrt(128) of them); the sums in FP32
    n = float(lens.max())
    tol = U[q.dtype] * want.abs() + weight * (2.0 ** -10 + 2.0 ** -13 + 2 * ds) + 1e-6
    tol = tol + n * peak * 2.0 ** -25 * 8 * (11.4 if rotate else 1)
    err = (got.double() - want).abs()
    assert bool((err <= tol)[used].all()), float((err / tol)[used].max())
    if lse is not None:
        fin = torch.isfinite(lse64) & used[:, None]
        assert bool(((lse.double() - lse64).abs() <= ds[..., 0] + 2.0 ** -20 * (1 + lse64.abs()))[fin].all())
        assert bool((lse[~torch.isfinite(lse64) & used[:, None]] == -math.inf).all())
        assert bool((got[~torch.isfinite(lse64) & used[:, None]] == 0).all())


ATTN_CASES = [  # B, Hkv, group, page, lens, q_len, window, sinks
    (1, 1, 1, 16, [1], 1, 0, 0),
    (2, 2, 8, 16, [17, 64], 1, 0, 0),
    (3, 1, 4, 32, [0, 1, 33], 1, 0, 0),              # an empty request: zeros
    (4, 8, 4, 16, [700, 65, 63, 128], 1, 0, 0),
    (2, 4, 16, 64, [1000, 129], 1, 0, 0),
    (2, 2, 5, 128, [300, 4097], 1, 0, 0),
    (1, 2, 8, 64, [20001], 1, 0, 0),                 # one long request: split over the GPU
    (5, 1, 12, 1024, [1023, 1024, 1025, 5, 2048], 1, 0, 0),
    (3, 2, 7, 16, [2, 40, 300], 4, 0, 0),            # more queries than tokens: the first see nothing
    (2, 1, 3, 64, [500, 77], 33, 0, 0),              # a chunk of a prefill
    (3, 2, 4, 32, [500, 31, 9], 1, 7, 0),
    (3, 2, 4, 32, [900, 64, 300], 2, 100, 4),
    (2, 1, 8, 16, [1500, 700], 3, 130, 70),          # sinks of more than a tile
    (2, 1, 8, 64, [800, 10], 1, 5000, 3),            # a window wider than the request
    (2, 2, 32, 64, [200, 100], 2, 64, 200),          # sinks reach past the window
]


@pytest.mark.parametrize("case", ATTN_CASES, ids=[str(i) for i in range(len(ATTN_CASES))])
@pytest.mark.parametrize("dtype,rotate", [(BF16, 128), (F16, 0), (F16, 128)])
def test_kv4_attention(hq, case, dtype, rotate):
    B, Hkv, group, page, lens, q_len, window, sinks = case
    g = _gen(sum(lens) + group)
    cache, table, t_lens = _filled(hq, g, B, Hkv, page, lens, rotate)
    q = _normal(g, B * q_len, Hkv * group, 128, dtype=dtype, std=1.5)
    ws = hq.kv4_attention_workspace()
    for scale in (128 ** -0.5, 0.5):
        out, lse = hq.kv4_attention(q, cache, table, t_lens, q_len=q_len, scale=scale, window=window, sinks=sinks,
                                    hadamard_n=rotate, ws=ws, want_lse=True)
        rows = [(b * q_len, (b + 1) * q_len) for b in range(B)]
        _check_attention(out, lse, q, cache, table, t_lens, rows, scale, window, sinks, rotate != 0)
        again = hq.kv4_attention(q, cache, table, t_lens, q_len=q_len, scale=scale, window=window, sinks=sinks,
                                 hadamard_n=rotate, ws=ws)
        assert torch.equal(out, again)  # the same bits every time, and the workspace is at rest again
    assert hq.hq_get_error(ws) == 0


@pytest.mark.parametrize("group,window,sinks", [(1, 0, 0), (4, 0, 0), (10, 50, 3)])
def test_kv4_attention_ragged_rows_and_padding(hq, group, window, sinks):
    g = _gen(41 + group)
    lens, counts, page, Hkv = [300, 0, 1, 77, 512, 9], [3, 0, 1, 0, 5, 2], 32, 2
    cache, table, t_lens = _filled(hq, g, len(lens), Hkv, page, lens, 128)
    cu = torch.tensor(np.concatenate(([0], np.cumsum(counts))), dtype=torch.int32, device="cuda")
    total = sum(counts)
    wide = _normal(g, total + 4, Hkv * group + 3, 128, dtype=BF16)
    q = wide[:, 1:1 + Hkv * group]  # heads of a wider row, and padding rows behind the last request
    out = torch.full((total + 4, Hkv * group, 128), 3.0, dtype=BF16, device="cuda")
    hq.kv4_attention(q, cache, table, t_lens, cu_q=cu, q_len=5, window=window, sinks=sinks, out=out)
    rows = [(int(cu[b]), int(cu[b + 1])) for b in range(len(lens))]
    _check_attention(out, None, q, cache, table, t_lens, rows, 128 ** -0.5, window, sinks, True)
    assert bool((out[total:] == 3.0).all())


def test_kv4_attention_bad_pages_are_reported_and_not_read(hq):
    g = _gen(51)
    lens, page, Hkv = [200, 300, 64], 16, 2
    cache, table, t_lens = _filled(hq, g, 3, Hkv, page, lens, 128)
    q = _normal(g, 3, Hkv * 4, 128, dtype=BF16)
    ws = hq.kv4_attention_workspace()
    hq.kv4_attention(q, cache, table, t_lens, ws=ws)
    assert hq.hq_get_error(ws) == 0
    table[0, 3], table[1, 0], table[1, 7] = -5, cache.shape[0], 2 ** 31 - 1
    out, lse = hq.kv4_attention(q, cache, table, t_lens, ws=ws, want_lse=True)
    _check_attention(out, lse, q, cache, table, t_lens, [(0, 1), (1, 2), (2, 3)], 128 ** -0.5, 0, 0, True)
    assert hq.hq_get_error(ws) == hq.HQ_ERR_PAGE and hq.hq_get_error(ws) == 0
    # a length beyond the row of the table: what the row holds counts
    cache, table, t_lens = _filled(hq, g, 2, 1, 16, [64, 64], 128)
    q = _normal(g, 2, 4, 128, dtype=BF16)
    long = torch.tensor([64, 100], dtype=torch.int32, device="cuda")
    out, lse = hq.kv4_attention(q, cache, table, long, ws=ws, want_lse=True)
    _check_attention(out, lse, q, cache, table, t_lens, [(0, 1), (1, 2)], 128 ** -0.5, 0, 0, True)
    assert hq.hq_get_error(ws) == hq.HQ_ERR_PAGE
    neg = torch.tensor([-3, 64], dtype=torch.int32, device="cuda")
    out, lse = hq.kv4_attention(q, cache, table, neg, ws=ws, want_lse=True)
    assert bool((out[0] == 0).all()) and bool((lse[0] == -math.inf).all())


def test_kv4_attention_rows_that_are_not_there_are_reported(hq):
    g = _gen(53)
    cache, table, lens = _filled(hq, g, 2, 1, 16, [40, 50], 128)
    q, ws = _normal(g, 4, 4, 128, dtype=BF16), hq.kv4_attention_workspace()
    want = hq.kv4_attention(q[:2].contiguous(), cache, table, lens, ws=ws)
    assert hq.hq_get_error(ws) == 0
    for cu in ([0, 1, 9], [-3, 1, 2], [0, 1, 4]):  # beyond the rows of q; before them; more than q_len
        out = torch.full_like(q, 5.0)
        hq.kv4_attention(q, cache, table, lens, cu_q=torch.tensor(cu, dtype=torch.int32, device="cuda"), q_len=1, ws=ws, out=out)
        assert hq.hq_get_error(ws) == hq.HQ_ERR_SHAPE, cu
        assert torch.equal(out[:2], want) and bool((out[2:] == 5.0).all()), cu


def test_kv4_attention_graphs_share_a_workspace(hq):
    """Two captured calls on one workspace, replayed in turn: each leaves it at rest for the other."""
    g = _gen(54)
    ws = hq.kv4_attention_workspace()
    cases = []
    for lens in ([3000, 10], [700, 4000, 1]):
        cache, table, t_lens = _filled(hq, g, len(lens), 2, 16, lens, 128)
        q = _normal(g, len(lens), 8, 128, dtype=BF16)
        want = hq.kv4_attention(q, cache, table, t_lens, ws=ws)
        out = torch.empty_like(q)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            hq.kv4_attention(q, cache, table, t_lens, ws=ws, out=out)
        cases.append((graph, out, want, q, cache, table, t_lens))
    for _ in range(3):
        for graph, out, want, *_ in cases:
            out.fill_(9.0)
            graph.replay()
            assert torch.equal(out, want)
    assert hq.hq_get_error(ws) == 0


def test_kv4_attention_columns_do_not_touch_each_other(hq):
    """NaN and infinite queries stay in their own rows."""
    g = _gen(55)
    cache, table, lens = _filled(hq, g, 2, 1, 32, [300, 70], 128)
    q = _normal(g, 2, 8, 128, dtype=F16)
    want = hq.kv4_attention(q, cache, table, lens)
    q[0, 2, 5], q[0, 6, 7], q[1, 0, 0] = math.nan, math.inf, -math.inf
    out, lse = hq.kv4_attention(q, cache, table, lens, want_lse=True)
    bad = torch.zeros((2, 8), dtype=torch.bool, device="cuda")
    bad[0, 2] = bad[0, 6] = bad[1, 0] = True
    assert torch.equal(out[~bad], want[~bad]) and bool(torch.isfinite(lse[~bad]).all())
    assert bool(torch.isnan(out[bad]).all())


def test_single_rows_with_any_stride(hq):
    """A dimension of one entry has no stride to check."""
    g = _gen(59)
    cache, table, lens = _filled(hq, g, 1, 1, 16, [40], 128)
    wide = [_normal(g, 1, 1, 131, dtype=BF16)[..., :128] for _ in range(3)]
    whole = [t.contiguous() for t in wide]
    assert wide[0].stride(0) == 131
    c2, slot = cache.clone(), torch.tensor([7], device="cuda")
    hq.kv4_append(wide[0], wide[1], slot, cache)
    hq.kv4_append(whole[0], whole[1], slot, c2)
    assert torch.equal(cache, c2)
    assert torch.equal(hq.kv4_attention(wide[2], cache, table, lens), hq.kv4_attention(whole[2], cache, table, lens))


def test_out_of_memory_is_the_frameworks_error(hq):
    x = torch.zeros((1, 65536), dtype=BF16, device="cuda").expand(2 ** 31 - 1, -1)  # 2^47 bytes of codes
    with pytest.raises(torch.OutOfMemoryError):
        hq.add_rmsnorm_fp8_k128(x, x[0].contiguous())


def test_a_tensor_on_the_host_is_refused_on_a_stream_too(hq):
    x, w = torch.zeros((2, 128), dtype=BF16, device="cuda"), torch.zeros(128, dtype=BF16)
    for kw in ({}, {"stream": torch.cuda.Stream()}):
        with pytest.raises(hq.HQError):
            hq.add_rmsnorm_fp8_k128(x, w, **kw)


def test_kv4_attention_lse_of_nan_scores(hq):
    g = _gen(56)
    cache, table, lens = _filled(hq, g, 1, 1, 16, [40], 128)
    q = _normal(g, 1, 8, 128, dtype=BF16)
    q[0, 3, 1] = math.nan
    _, lse = hq.kv4_attention(q, cache, table, lens, want_lse=True)
    assert bool(torch.isnan(lse[0, 3])) and int(torch.isnan(lse).sum()) == 1


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 3, 1 << 30])
def test_kv4_attention_widest_windows(hq, window):
    """More queries than tokens under a window as wide as the type allows: as without a window."""
    g = _gen(57)
    cache, table, lens = _filled(hq, g, 2, 1, 16, [2, 70], 128)
    q = _normal(g, 10, 4, 128, dtype=BF16)
    want = hq.kv4_attention(q, cache, table, lens, q_len=5, want_lse=True)
    got = hq.kv4_attention(q, cache, table, lens, q_len=5, window=window, want_lse=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_kv4_attention_largest_queries(hq):
    """Queries of 2^100 to the type's largest power of two, the scale their inverse: as the queries brought down before."""
    g = _gen(58)
    cache, table, lens = _filled(hq, g, 1, 1, 16, [300], 0)
    q = _normal(g, 1, 8, 128, dtype=BF16).clamp(-1.9, 1.9)
    want = hq.kv4_attention(q, cache, table, lens, scale=0.125, hadamard_n=0, want_lse=True)
    for e in (100, 112, 126, 127):
        up = q * 2.0 ** e
        assert bool(torch.isfinite(up).all())
        got = hq.kv4_attention(up, cache, table, lens, scale=2.0 ** (-3 - e), hadamard_n=0, want_lse=True)
        # powers of two only; at 2^127 the column's power is one too small: FP16 parts of twice the size, the same bits
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), e


def test_kv4_attention_extreme_scores(hq):
    """Scores of thousands: the running maximum carries them; one token takes all the weight."""
    g = _gen(52)
    cache, table, lens = _filled(hq, g, 1, 1, 16, [500], 128)
    q = _normal(g, 1, 8, 128, dtype=BF16, std=300.0)
    out, lse = hq.kv4_attention(q, cache, table, lens, want_lse=True)
    want, lse64, weight, _ = attention64(q, cache, table, lens, [(0, 1)], 128 ** -0.5, 0, 0, True)
    assert bool(torch.isfinite(out).all())
    ds = 2.0 ** -17 * q.double().norm(dim=-1, keepdim=True) * 16.0 * 128 ** -0.5  # as in _check_attention: about 0.4
    assert bool(((lse.double() - lse64).abs() <= ds[..., 0] + 2.0 ** -20 * (1 + lse64.abs())).all())
    tol = U[BF16] * want.abs() + weight * (2.0 ** -10 + 2.0 ** -13 + torch.expm1(2 * ds)) + 1e-4
    assert bool(((out.double() - want).abs() <= tol).all())


# ------------------------------------------------------ as used together
def _decode_step(hq, st, x, r, new, w_qkv, w_norm, inv, mag, Hq, Hkv, page, n_rows):
    """One serving step of an attention layer: norm + FP8, the product, rope, slots, cache, attention."""
    n = hq.add_rmsnorm_fp8_k128(x, w_norm, r)
    y = (n["codes"].view(torch.float8_e4m3fn).to(F32).unflatten(1, (-1, 128)) * n["scales"][..., None]).flatten(1)
    qkv = (y @ w_qkv).to(BF16)
    q, k, v = (qkv[:, a * 128:b * 128].unflatten(1, (b - a, 128)) for a, b in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
    s = hq.kv_slots(st["lens"], new, st["table"], st["free"], st["count"], page, n_rows, lens_out=st["lens"],
                    free_count_out=st["count"])
    q, k = hq.rope(q, k, s["positions"], inv, magnitude=mag, q_out=q, k_out=k)
    hq.kv4_append(k, v, s["slots"], st["cache"])
    out = torch.zeros((n_rows, Hq, 128), dtype=BF16, device="cuda")
    hq.kv4_attention(q, st["cache"], st["table"], s["lens"], cu_q=s["cu_new"], q_len=n_rows, ws=st["ws"], out=out)
    return {"q": q, "k": k, "v": v, "out": out, **{a: s[a] for a in ("cu_new", "slots", "positions", "status")}}


def _serving_state(hq, B, Hkv, page, pages, width):
    i32 = dict(dtype=torch.int32, device="cuda")
    return {"lens": torch.zeros(B, **i32), "table": torch.full((B, width), -1, **i32), "free": torch.arange(pages, **i32),
            "count": torch.tensor([pages], **i32), "cache": hq.kv4_cache(pages, page, Hkv), "ws": hq.kv4_attention_workspace()}


@pytest.mark.parametrize("captured", [False, True])
def test_serving_steps(hq, captured):
    """A prefill and decoding steps with requests ending and growing, eagerly and as one captured graph, against dense
    attention over the values that each request's tokens were stored as."""
    B, Hq, Hkv, page, pages, width, K, n_rows = 4, 8, 2, 16, 24, 12, 256, 64
    g = _gen(61)
    st = _serving_state(hq, B, Hkv, page, pages, width)
    w_qkv, w_norm = _normal(g, K, (Hq + 2 * Hkv) * 128) / K ** 0.5, 1 + 0.1 * _normal(g, K)
    inv, mag = hq.rope_inv_freq(128, 1e4, hq.HQ_ROPE_PARTS, 4.0, 4096)
    x, r = torch.zeros((n_rows, K), dtype=BF16, device="cuda"), torch.zeros((n_rows, K), dtype=BF16, device="cuda")
    new = torch.zeros(B, dtype=torch.int32, device="cuda")
    args = (hq, st, x, r, new, w_qkv, w_norm.to(BF16), inv, mag, Hq, Hkv, page, n_rows)
    if captured:
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            _decode_step(*args)  # warm-up: no new tokens
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            captured_out = _decode_step(*args)
    h = torch.from_numpy(hadamard128()).cuda()
    lens = [0] * B
    for step in ([20, 7, 0, 33], [1, 1, 1, 1], [1, 1, 5, 1], [-1, 1, 1, 2], [16, 1, 1, 1]):
        x.copy_(_normal(g, n_rows, K, dtype=BF16))
        r.copy_(_normal(g, n_rows, K, dtype=BF16))
        new.copy_(torch.tensor(step, dtype=torch.int32))
        if captured:
            graph.replay()
            o = captured_out
        else:
            o = _decode_step(*args)
        torch.cuda.synchronize()
        assert int(o["status"]) == 0
        lens = [0 if a < 0 else n + a for n, a in zip(lens, step)]
        assert st["lens"].tolist() == lens
        assert int(st["count"]) == pages - sum(-(-n // page) for n in lens)
        rows = [(int(o["cu_new"][b]), int(o["cu_new"][b + 1])) for b in range(B)]
        assert [b - a for a, b in rows] == [max(a, 0) for a in step]
        _check_attention(o["out"], None, o["q"], st["cache"], st["table"], st["lens"], rows, 128 ** -0.5, 0, 0, True)
        # the newest token's key is stored as the 4-bit form of what rope returned
        for b, (a, e) in enumerate(rows):
            if e > a:
                slot = int(o["slots"][e - 1])
                got = decode(st["cache"][slot // page, :, slot % page // 16], False)[:, slot % 16] @ h
                assert float((got - o["k"][e - 1].double()).norm() / o["k"][e - 1].double().norm()) < 0.2
    assert hq.hq_get_error(st["ws"]) == 0


def test_calls_on_another_stream(hq):
    g = _gen(71)
    side = torch.cuda.Stream()
    cache, table, lens = _filled(hq, g, 2, 2, 16, [100, 50], 128)
    q = _normal(g, 2, 8, 128, dtype=BF16)
    x, w = _normal(g, 64, 512, dtype=BF16), _normal(g, 512, dtype=BF16)
    pos, inv = torch.arange(2, device="cuda"), hq.rope_inv_freq(128)[0]
    want = (hq.kv4_attention(q, cache, table, lens), hq.add_rmsnorm_fp8_k128(x, w)["codes"], hq.rope(q, None, pos, inv)[0],
            hq.kv4_gather(cache, pos)[0])
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        got = (hq.kv4_attention(q, cache, table, lens, stream=stream), hq.add_rmsnorm_fp8_k128(x, w, stream=stream)["codes"],
               hq.rope(q, None, pos, inv, stream=stream)[0], hq.kv4_gather(cache, pos, stream=stream)[0])
        side.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


# ------------------------------------------------------- sizes and neighbours
@pytest.mark.parametrize("heads", [4, 16])
def test_kv4_attention_of_many_requests(hq, heads):
    """More requests than a block has threads, most of them tiny, some empty."""
    g = _gen(81)
    B, page = 3001, 16
    lens = torch.randint(0, 40, (B,), generator=torch.Generator().manual_seed(5)).tolist()
    lens[1234] = 2000
    cache, table, t_lens = _filled(hq, g, B, 1, page, lens, 128)
    q = _normal(g, B, heads, 128, dtype=BF16)
    out, lse = hq.kv4_attention(q, cache, table, t_lens, want_lse=True)
    for b in list(range(0, B, 211)) + [1233, 1234, 1235, B - 1]:
        rows = [(0, 0)] * b + [(b, b + 1)] + [(0, 0)] * (B - b - 1)
        want, lse64, weight, _ = attention64(q, cache, table, lens, rows, 128 ** -0.5, 0, 0, True)
        tol = U[BF16] * want[b].abs() + weight[b] * (2.0 ** -10 + 2.0 ** -12) + 1e-5  # as in _check_attention
        assert bool(((out[b].double() - want[b]).abs() <= tol).all()), b
        if lens[b]:
            assert bool(((lse[b].double() - lse64[b]).abs() < 1e-3).all()), b
    empty = t_lens == 0
    assert bool((out[empty] == 0).all()) and bool((lse[empty] == -math.inf).all())


def test_kv4_cache_beyond_32_bit_offsets(hq):
    """Pages whose bytes lie behind 2^32: the same results as in a small cache."""
    g = _gen(82)
    H, page, pages = 8, 64, 60_000  # 4.7 GB
    big = torch.empty((pages, H, page // 16, 2432), dtype=torch.uint8, device="cuda")
    small = hq.kv4_cache(4, page, H)
    n = 200
    k, v = _normal(g, n, H, 128, dtype=BF16), _normal(g, n, H, 128, dtype=BF16)
    where = torch.tensor([pages - 1, pages - 3, 57_000, pages - 2], device="cuda")
    t = torch.arange(n, device="cuda")
    hq.kv4_append(k, v, t, small)
    hq.kv4_append(k, v, where[t // page] * page + t % page, big)
    assert torch.equal(hq.kv4_gather(small, t)[0], hq.kv4_gather(big, where[t // page] * page + t % page)[0])
    q, lens = _normal(g, 1, 4 * H, 128, dtype=BF16), torch.tensor([n], dtype=torch.int32, device="cuda")
    a = hq.kv4_attention(q, small, torch.arange(4, dtype=torch.int32, device="cuda")[None], lens)
    assert torch.equal(a, hq.kv4_attention(q, big, where.to(torch.int32)[None], lens))


def test_norm_and_rope_beyond_32_bit_offsets(hq):
    """Tensors of more than 2^31 elements: the last rows as in a call on them alone."""
    g = _gen(83)
    M, K = 70_001, 32_768
    x = torch.zeros((M, K), dtype=BF16, device="cuda")
    x[-3:] = _normal(g, 3, K, dtype=BF16)
    w = _normal(g, K, dtype=BF16)
    out, last = hq.add_rmsnorm_fp8_k128(x, w, want_rstd=True), hq.add_rmsnorm_fp8_k128(x[-3:].contiguous(), w, want_rstd=True)
    for name in last:
        assert torch.equal(out[name][-3:], last[name]), name
    rstd = out["rstd"]
    del out
    dx, dw = hq.rmsnorm_backward(x, x, w, rstd)
    dx3, dw3 = hq.rmsnorm_backward(x[-3:].contiguous(), x[-3:].contiguous(), w, rstd[-3:].contiguous())
    assert torch.equal(dx[-3:], dx3) and torch.equal(dw, dw3)  # (the other rows add zeros)
    del dx
    q = x.view(M, 256, 128)
    pos, (inv, _) = torch.arange(M, device="cuda"), hq.rope_inv_freq(128)
    y, _ = hq.rope(q, None, pos, inv)
    assert torch.equal(y[-3:], hq.rope(q[-3:].contiguous(), None, pos[-3:].contiguous(), inv)[0])


def test_calls_on_two_streams_at_once(hq):
    """Calls that share no workspace do not disturb each other."""
    g = _gen(84)
    streams, sets = [torch.cuda.Stream() for _ in range(2)], []
    for k in range(2):
        cache, table, lens = _filled(hq, g, 3, 2, 32, [900 + 500 * k, 33, 2000], 128)
        sets.append((_normal(g, 3, 8, 128, dtype=BF16), cache, table, lens, hq.kv4_attention_workspace(),
                     _normal(g, 300, 1024, dtype=BF16), _normal(g, 1024, dtype=BF16), hq.rmsnorm_backward_workspace(300, 1024)))
    rstd = torch.ones(300, device="cuda")

    def calls(s):
        q, cache, table, lens, ws, x, w, ws2 = s
        return [hq.kv4_attention(q, cache, table, lens, ws=ws), *hq.rmsnorm_backward(x, x, w, rstd, ws=ws2)]

    want = [calls(s) for s in sets]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                got[k].append(calls(sets[k]))
    torch.cuda.synchronize()
    for k in range(2):
        for outs in got[k]:
            for a, b in zip(outs, want[k]):
                assert torch.equal(a, b)
