"""Host-side checks of the attention-layer calls (no GPU needed): argument errors of the C functions with pointers that
are never dereferenced, refusals of the Python conveniences, rotary frequencies."""
from __future__ import annotations

import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

import _kv4

import nvfp4_quantization_group_b200 as hq

FAKE = 0x10000
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def L():
    return hq.lib()


def test_add_rmsnorm_argument_errors(L):
    def call(dt=0, x=FAKE, xs=256, r=FAKE, rs=256, w=FAKE, wd=0, eps=1e-6, M=4, K=256, h=FAKE, out=FAKE, sc=FAKE,
             layout=0, ld=4, rstd=FAKE, amax=None):
        return L.hq_add_rmsnorm_fp8_k128(dt, P(x), xs, P(r), rs, P(w), wd, eps, M, K, P(h), P(out), P(sc), layout, ld,
                                         P(rstd), P(amax), None)
    assert call(dt=3) == hq.HQ_ERR_UNSUPPORTED
    assert call(dt=0, wd=1) == hq.HQ_ERR_UNSUPPORTED               # a weight of the rows' type or FP32
    assert call(layout=2) == hq.HQ_ERR_UNSUPPORTED
    assert call(layout=hq.HQ_SF_SWIZZLED) == hq.HQ_ERR_UNSUPPORTED
    assert call(eps=-1.0) == hq.HQ_ERR_UNSUPPORTED
    assert call(eps=math.nan) == hq.HQ_ERR_UNSUPPORTED
    assert call(M=-1) == hq.HQ_ERR_SHAPE
    assert call(K=0) == hq.HQ_ERR_SHAPE
    assert call(K=hq.HQ_NORM_MAX_K + 128, xs=1 << 20, rs=1 << 20) == hq.HQ_ERR_SHAPE
    assert call(K=200) == hq.HQ_ERR_ALIGN
    assert call(M=0, x=0) == hq.HQ_OK
    assert call(x=0) == hq.HQ_ERR_NULL
    assert call(w=0) == hq.HQ_ERR_NULL
    assert call(h=0) == hq.HQ_ERR_NULL                             # a residual without residual_out
    assert call(xs=128) == hq.HQ_ERR_SHAPE
    assert call(rs=128) == hq.HQ_ERR_SHAPE
    assert call(layout=1, ld=3) == hq.HQ_ERR_SHAPE
    assert call(xs=512, x=FAKE * 2, h=FAKE * 2) == hq.HQ_ERR_SHAPE  # in place on strided rows
    assert call(rs=512) == hq.HQ_ERR_SHAPE                         # the same for the residual (r == h here)
    assert call(xs=260, x=FAKE * 2) == hq.HQ_ERR_ALIGN
    assert call(x=FAKE + 8) == hq.HQ_ERR_ALIGN
    assert call(out=FAKE + 4) == hq.HQ_ERR_ALIGN
    assert call(rstd=FAKE + 2) == hq.HQ_ERR_ALIGN
    assert call(layout=1 | hq.HQ_FP8_UE8M0, ld=3) == hq.HQ_ERR_SHAPE


def test_rmsnorm_backward_argument_errors(L):
    n = hq.hq_rmsnorm_backward_workspace_size(4, 256)
    assert n > 0 and n % 256 == 0
    assert hq.hq_rmsnorm_backward_workspace_size(4, 200) == 0
    assert hq.hq_rmsnorm_backward_workspace_size(-1, 256) == 0

    def call(dt=0, dy=FAKE, ds=256, h=FAKE, hs=256, w=FAKE, wd=2, rstd=FAKE, dres=0, rs=256, M=4, K=256, dx=FAKE * 2,
             dw=FAKE, ws=FAKE, nws=n):
        return L.hq_rmsnorm_backward(dt, P(dy), ds, P(h), hs, P(w), wd, P(rstd), P(dres), rs, M, K, P(dx), P(dw), P(ws),
                                     nws, None)
    assert call(dt=-1) == hq.HQ_ERR_UNSUPPORTED
    assert call(dt=0, wd=1) == hq.HQ_ERR_UNSUPPORTED
    assert call(K=130) == hq.HQ_ERR_ALIGN
    assert call(M=0, dw=0) == hq.HQ_OK
    assert call(dy=0) == hq.HQ_ERR_NULL
    assert call(rstd=0) == hq.HQ_ERR_NULL
    assert call(ws=0) == hq.HQ_ERR_NULL
    assert call(nws=n - 1) == hq.HQ_ERR_WORKSPACE
    assert call(hs=128) == hq.HQ_ERR_SHAPE
    assert call(dx=FAKE, ds=512) == hq.HQ_ERR_SHAPE
    assert call(dres=FAKE * 2, rs=512) == hq.HQ_ERR_SHAPE
    assert call(ds=258) == hq.HQ_ERR_ALIGN
    assert call(dw=FAKE + 4) == hq.HQ_ERR_ALIGN


def test_rope_argument_errors(L):
    def call(dt=0, q=FAKE, k=FAKE, Hq=4, Hk=2, T=3, D=128, pos=FAKE, inv=FAKE, R=64, off=0, layout=0, qo=FAKE * 2,
             ko=FAKE * 2, qs=512):
        return L.hq_rope(dt, P(q), qs, 128, Hq, P(k), 256, 128, Hk, T, D, P(pos), P(inv), R, off, layout, 1.0, 0, P(qo),
                         512, 128, P(ko), 256, 128, None)
    assert call(dt=5) == hq.HQ_ERR_UNSUPPORTED
    assert call(layout=2) == hq.HQ_ERR_UNSUPPORTED
    assert call(R=63) == hq.HQ_ERR_SHAPE
    assert call(R=0) == hq.HQ_ERR_SHAPE
    assert call(R=130) == hq.HQ_ERR_SHAPE
    assert call(off=65) == hq.HQ_ERR_SHAPE
    assert call(off=-1) == hq.HQ_ERR_SHAPE
    assert call(D=1 << 14, R=64) == hq.HQ_ERR_SHAPE
    assert call(T=-1) == hq.HQ_ERR_SHAPE
    assert call(T=0, q=0) == hq.HQ_OK
    assert call(Hq=0, Hk=0) == hq.HQ_OK
    assert call(q=0) == hq.HQ_ERR_NULL
    assert call(ko=0) == hq.HQ_ERR_NULL
    assert call(inv=0) == hq.HQ_ERR_NULL
    assert call(qo=FAKE, qs=1024) == hq.HQ_ERR_SHAPE               # in place with other strides
    assert call(q=FAKE + 1) == hq.HQ_ERR_ALIGN
    assert call(dt=2, q=FAKE + 2) == hq.HQ_ERR_ALIGN
    assert call(pos=FAKE + 4) == hq.HQ_ERR_ALIGN


def test_rope_frequencies():
    base, R, trained = 10000.0, 64, 4096.0
    plain, m = hq.rope_inv_freq(R, base, device="cpu")
    want = torch.tensor([base ** (-2 * i / R) for i in range(R // 2)], dtype=torch.float64)
    # pow is correct to an ulp or so on both sides: 2^-50 leaves 4 of them
    assert torch.allclose(plain, want, rtol=2.0 ** -50, atol=0) and m == 1.0
    lin, m = hq.rope_inv_freq(R, base, hq.HQ_ROPE_LINEAR, 8.0, device="cpu")
    assert torch.allclose(lin, want / 8, rtol=2.0 ** -50, atol=0) and m == 1.0
    ntk, _ = hq.rope_inv_freq(R, base, hq.HQ_ROPE_NTK, 8.0, device="cpu")
    assert ntk[0] == 1.0 and abs(ntk[-1] / (want[-1] / 8) - 1) < 1e-12  # the slowest pair is divided by the factor
    parts, m = hq.rope_inv_freq(R, base, hq.HQ_ROPE_PARTS, 32.0, trained, device="cpu")
    turns = trained * want / (2 * math.pi)
    assert abs(m - (0.1 * math.log(32.0) + 1)) < 1e-15
    assert torch.equal(parts[turns > 40], plain[turns > 40])
    assert torch.allclose(parts[turns < 0.7], want[turns < 0.7] / 32, rtol=2.0 ** -50, atol=0)
    assert bool((parts[1:] < parts[:-1]).all())
    bands, m = hq.rope_inv_freq(R, base, hq.HQ_ROPE_BANDS, 8.0, trained, device="cpu")
    assert m == 1.0
    for i in range(R // 2):
        f, wave = float(want[i]), 2 * math.pi / float(want[i])
        if wave < trained / 4:
            w = f
        elif wave > trained / 1:
            w = f / 8
        else:
            s = (trained / wave - 1) / (4 - 1)
            w = (1 - s) * f / 8 + s * f
        assert abs(float(bands[i]) / w - 1) < 1e-12, i


def test_rope_frequency_errors():
    def status(*a, **k):
        with pytest.raises(hq.HQError) as e:
            hq.rope_inv_freq(*a, device="cpu", **k)
        return e.value.status
    assert status(63) == hq.HQ_ERR_SHAPE
    assert status(0) == hq.HQ_ERR_SHAPE
    assert status(2, 1e4, hq.HQ_ROPE_NTK, 2.0) == hq.HQ_ERR_SHAPE
    assert status(64, 1e4, 5) == hq.HQ_ERR_UNSUPPORTED
    assert status(64, 1.0) == hq.HQ_ERR_UNSUPPORTED
    assert status(64, 1e4, hq.HQ_ROPE_LINEAR, 0.5) == hq.HQ_ERR_UNSUPPORTED
    assert status(64, 1e4, hq.HQ_ROPE_PARTS, 2.0) == hq.HQ_ERR_UNSUPPORTED            # needs a trained length
    assert status(64, 1e4, hq.HQ_ROPE_PARTS, 2.0, 4096, p1=1.0, p2=2.0) == hq.HQ_ERR_UNSUPPORTED
    assert status(64, 1e4, hq.HQ_ROPE_BANDS, 2.0, 4096, p1=4.0, p2=1.0) == hq.HQ_ERR_UNSUPPORTED


def test_kv_slots_argument_errors(L):
    def call(B=4, lens=FAKE, new=FAKE, tab=FAKE, width=8, pages=FAKE, cap=32, cnt=FAKE, page=16, n=64, lo=FAKE, cu=FAKE,
             slots=FAKE, pos=FAKE, co=FAKE, st=FAKE):
        return L.hq_kv_slots(B, P(lens), P(new), P(tab), width, P(pages), cap, P(cnt), page, n, P(lo), P(cu), P(slots),
                             P(pos), P(co), P(st), None)
    for page in (0, 8, 24, 2048, -16):
        assert call(page=page) == hq.HQ_ERR_UNSUPPORTED
    assert call(B=-1) == hq.HQ_ERR_SHAPE
    assert call(B=hq.HQ_KV_MAX_REQUESTS + 1) == hq.HQ_ERR_SHAPE
    assert call(width=-1) == hq.HQ_ERR_SHAPE
    assert call(cap=-1) == hq.HQ_ERR_SHAPE
    assert call(n=-1) == hq.HQ_ERR_SHAPE
    for name in ("lens", "new", "tab", "pages", "cnt", "lo", "cu", "slots", "pos", "co", "st"):
        assert call(**{name: 0}) == hq.HQ_ERR_NULL, name
        assert call(**{name: FAKE + 2}) == hq.HQ_ERR_ALIGN, name
    assert call(slots=FAKE + 4) == hq.HQ_ERR_ALIGN


def test_kv4_argument_errors(L):
    assert hq.hq_kv4_cache_bytes(3, 64, 2) == 3 * 2 * 4 * 2432
    for bad in ((0, 64, 2), (3, 48, 2), (3, 64, 0), (1 << 40, 64, 8), (-1, 64, 2)):
        assert hq.hq_kv4_cache_bytes(*bad) == 0

    def call(f, dt=0, k=FAKE, v=FAKE, s=128, slots=FAKE, N=4, H=2, hn=128, cache=FAKE, pages=3, page=16):
        if f == "append":
            return L.hq_kv4_append(dt, P(k), 256, s, P(v), 256, s, P(slots), N, H, hn, P(cache), pages, page, None)
        return L.hq_kv4_gather(dt, P(cache), pages, page, P(slots), N, H, hn, P(k), 256, s, P(v), 256, s, None)
    for f in ("append", "gather"):
        assert call(f, dt=3) == hq.HQ_ERR_UNSUPPORTED
        assert call(f, hn=64) == hq.HQ_ERR_UNSUPPORTED
        assert call(f, page=8) == hq.HQ_ERR_UNSUPPORTED
        assert call(f, N=-1) == hq.HQ_ERR_SHAPE
        assert call(f, H=0) == hq.HQ_ERR_SHAPE
        assert call(f, pages=0) == hq.HQ_ERR_SHAPE
        assert call(f, N=0, k=0) == hq.HQ_OK
        assert call(f, k=0) == hq.HQ_ERR_NULL
        assert call(f, slots=0) == hq.HQ_ERR_NULL
        assert call(f, cache=0) == hq.HQ_ERR_NULL
        assert call(f, s=132) == hq.HQ_ERR_ALIGN
        assert call(f, v=FAKE + 8) == hq.HQ_ERR_ALIGN
        assert call(f, cache=FAKE + 8) == hq.HQ_ERR_ALIGN
        assert call(f, slots=FAKE + 4) == hq.HQ_ERR_ALIGN


def test_kv4_attention_argument_errors(L):
    n = hq.hq_kv4_attention_workspace_size()
    assert n > 0 and n % 256 == 0

    def call(dt=0, q=FAKE, s=128, Tq=4, Hq=8, cache=FAKE, pages=3, page=16, Hkv=2, tab=FAKE, width=8, B=4, lens=FAKE,
             cu=0, q_len=1, scale=0.1, window=0, sinks=0, hn=128, out=FAKE, lse=0, ws=FAKE, nws=n):
        return L.hq_kv4_attention(dt, P(q), 1024, s, Tq, Hq, P(cache), pages, page, Hkv, P(tab), width, B, P(lens), P(cu),
                                  q_len, scale, window, sinks, hn, P(out), 1024, 128, P(lse), P(ws), nws, None)
    assert call(dt=2) == hq.HQ_ERR_UNSUPPORTED                      # FP32 queries
    assert call(hn=16) == hq.HQ_ERR_UNSUPPORTED
    assert call(page=20) == hq.HQ_ERR_UNSUPPORTED
    assert call(window=-1) == hq.HQ_ERR_UNSUPPORTED
    assert call(sinks=-1) == hq.HQ_ERR_UNSUPPORTED
    assert call(scale=math.inf) == hq.HQ_ERR_UNSUPPORTED
    assert call(scale=math.nan) == hq.HQ_ERR_UNSUPPORTED
    assert call(Hq=9) == hq.HQ_ERR_SHAPE
    assert call(Hkv=0) == hq.HQ_ERR_SHAPE
    assert call(q_len=0) == hq.HQ_ERR_SHAPE
    assert call(B=5) == hq.HQ_ERR_SHAPE                             # fewer rows than B * q_len
    assert call(B=hq.HQ_KV_MAX_REQUESTS + 1, Tq=1 << 20) == hq.HQ_ERR_SHAPE
    assert call(q_len=1 << 17, Tq=1 << 20, cu=FAKE) == hq.HQ_ERR_SHAPE
    assert call(pages=0) == hq.HQ_ERR_SHAPE
    assert call(ws=0) == hq.HQ_ERR_NULL
    assert call(ws=FAKE + 4) == hq.HQ_ERR_ALIGN
    assert call(nws=n - 1) == hq.HQ_ERR_WORKSPACE
    assert call(Tq=0, B=0) == hq.HQ_OK
    assert call(q=0) == hq.HQ_ERR_NULL
    assert call(lens=0) == hq.HQ_ERR_NULL
    assert call(tab=0) == hq.HQ_ERR_NULL
    assert call(s=132) == hq.HQ_ERR_ALIGN
    assert call(out=FAKE + 8) == hq.HQ_ERR_ALIGN
    assert call(lse=FAKE + 2) == hq.HQ_ERR_ALIGN


def test_conveniences_refuse_before_any_launch():
    """Tensors that are not on a GPU, and shapes, types and strides that do not fit."""
    x, w = torch.zeros((2, 128), dtype=torch.bfloat16), torch.zeros(128, dtype=torch.bfloat16)
    i32, i64 = torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int64)
    cache = torch.zeros((2, 1, 1, hq.HQ_KV4_GROUP_BYTES), dtype=torch.uint8)
    qkv = torch.zeros((2, 1, 128), dtype=torch.bfloat16)
    calls = [lambda: hq.add_rmsnorm_fp8_k128(x, w), lambda: hq.rmsnorm_backward(x, x, w, torch.zeros(2)),
             lambda: hq.rope(qkv, None, i64, torch.zeros(64, dtype=torch.float64)),
             lambda: hq.kv_slots(i32, i32, torch.zeros((2, 4), dtype=torch.int32), i32, i32[:1], 16, 4),
             lambda: hq.kv4_append(qkv, qkv, i64, cache), lambda: hq.kv4_gather(cache, i64),
             lambda: hq.kv4_attention(qkv, cache, torch.zeros((2, 4), dtype=torch.int32), i32)]
    for f in calls:
        with pytest.raises(hq.HQError) as e:
            f()
        assert e.value.status == hq.HQ_ERR_UNSUPPORTED
    with pytest.raises(hq.HQError):
        hq.kv4_cache(4, 24, 2, device="cpu")
    assert hq.kv4_cache(4, 32, 2, device="cpu").shape == (4, 2, 2, hq.HQ_KV4_GROUP_BYTES)
    with pytest.raises(hq.HQError):
        hq.rmsnorm_backward_workspace(4, 100, device="cpu")


def test_cache_layout_of_the_document():
    """FORMAT.md's offsets fill a group's 2432 bytes exactly once and are those that the GPU tests read with."""
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "FORMAT.md")
    text = open(path, encoding="utf-8").read()
    part = text[text.index("### 6.5 "):]
    rows = dict(re.findall(r"^\| ([KV][a-z ]+?)(?: \(float\))? \| [^|]+ \| `([^`]+)` \|$", part[:part.index("## 7.")], flags=re.M))
    assert len(rows) == 6
    used = np.zeros(hq.HQ_KV4_GROUP_BYTES, int)
    group = np.arange(hq.HQ_KV4_GROUP_BYTES) % 251
    group = group.astype(np.uint8)
    for value, name in ((False, "K"), (True, "V")):
        at = lambda what, r, j=0: eval(rows[f"{name} {what}"], {"__builtins__": {}}, {"r": r, "j": j})  # noqa: E731
        for r in range(16):
            codes, sf, dec = _kv4.token_bytes(group, r, value)
            for j in range(0, 128, 2):
                used[at("codes", r, j)] += 1
                assert group[at("codes", r, j)] == codes[j // 2]
            for j in range(0, 128, 16):
                used[at("block scales", r, j)] += 1
                assert group[at("block scales", r, j)] == sf[j // 16]
            first = at("decode scale", r)
            used[first:first + 4] += 1
            assert group[first:first + 4].view(np.float32)[0] == dec
    assert (used == 1).all()
