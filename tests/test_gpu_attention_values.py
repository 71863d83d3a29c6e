"""Attention over caches whose values (and scores) differ in size from token to token: vectors of zeros, vectors many
powers of two larger than the others, tiny and huge ones.  Against binary64 sums over what the cache holds, with
tolerances that are relative to what each token adds to an output."""
from __future__ import annotations

import math

import pytest
import torch

from _kv4 import hadamard128, request_kv

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
U = {BF16: 2.0 ** -8, F16: 2.0 ** -11}  # half a rounding step of the outputs
SCALE = 128 ** -0.5


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _directed(g, n, heads, powers, dtype):
    """Queries [1, heads, 128] along one direction and keys [n, 1, 128] whose scores with the first query lie near
    `powers` [n] powers of two (4-bit keys: within about a tenth of the power)."""
    d = _normal(g, 128)
    d = d / d.norm()
    q = 8.0 * d * (1 + 0.05 * torch.arange(heads, device="cuda")[:, None])
    k = powers.float()[:, None] * (math.log(2.0) / (8.0 * SCALE)) * d + 0.05 * _normal(g, n, 128)
    return q[None].to(dtype), k[:, None].contiguous()


def _check(hq, q, k, v, rotate, window=0, sinks=0, page=16, scale=SCALE, q_len=1):
    """One request of one key/value head: k, v FP32 [n, 1, 128], q [q_len, heads, 128].  Returns (out, want)."""
    n, heads = k.shape[0], q.shape[1]
    pages = -(-n // page)
    cache = hq.kv4_cache(pages + 1, page, 1)
    table = torch.randperm(pages + 1, generator=torch.Generator().manual_seed(n)).to(torch.int32)[None, :pages].cuda()
    t = torch.arange(n, device="cuda")
    hq.kv4_append(k, v, table[0].long()[t // page] * page + t % page, cache, hadamard_n=rotate)
    lens, ws = torch.tensor([n], dtype=torch.int32, device="cuda"), hq.kv4_attention_workspace()
    out, lse = hq.kv4_attention(q, cache, table, lens, q_len=q_len, scale=scale, window=window, sinks=sinks,
                                hadamard_n=rotate, ws=ws, want_lse=True)
    again = hq.kv4_attention(q, cache, table, lens, q_len=q_len, scale=scale, window=window, sinks=sinks,
                             hadamard_n=rotate, ws=ws)
    assert torch.equal(out, again) and hq.hq_get_error(ws) == 0

    k64, v64 = (x[0] for x in request_kv(cache, table[0], n))
    h = torch.from_numpy(hadamard128()).cuda()
    x = q.double() @ h if rotate else q.double()
    s = torch.einsum("qhd,td->qht", x, k64) * scale
    p = torch.arange(n - q_len, n, device="cuda")[:, None]
    see = t[None] <= p
    if window:
        see &= (p - t[None] < window) | (t[None] < sinks)
    s = s.masked_fill(~see[:, None], -torch.inf)
    w = torch.softmax(s, -1)
    want = w @ v64
    # a score is off by 2^-17 |q| |k| scale at most: q's two parts keep 2^-23 of its largest element (times sqrt(128) for
    # the 1-norm of k: 2^-19.5), the sixteen steps of the product and its scaling 2^-23 each of |q| |k| (2^-19), a
    # rotation of q seven roundings (2^-21)
    ds = 2.0 ** -17 * x.norm(dim=-1)[..., None] * k64.norm(dim=-1) * scale
    mean_ds = (w * ds).sum(-1, keepdim=True)
    lse64 = torch.logsumexp(s, -1)
    assert bool(((lse.double() - lse64).abs() <= mean_ds[..., 0] * 1.01 + 2.0 ** -20 * (1 + lse64.abs())).all())
    # a token's weight: half a step of FP16 (2^-11), or two parts of it (2^-22); its score's error and the mean of all
    # (the sum below the line); 2^-15 for ex2 and the 32-bit sums (at most 2^8 steps of 2^-23)
    part = 2.0 ** -11 if q.dtype == BF16 else 2.0 ** -22
    rel = (w * (part + 2.0 ** -15 + 1.05 * (ds + mean_ds))) @ v64.abs()
    # below FP16's normal range a weight is off by 2^-25 where the largest contribution counts at least 2^9
    largest = (w * v64.abs().amax(-1)).amax(-1, keepdim=True)
    err = rel + see.sum(-1)[:, None, None] * 2.0 ** -34 * largest
    # weights are 32-bit: 2^(s - m) with m below the largest score + 1 is zero for s < m - 126, which leaves out a weight
    # below 2^-125 of the largest (it shows where a value is 2^125 times the winner's)
    err = err + 2.0 ** -125 * w.amax(-1, keepdim=True) * (see[:, None].double() @ v64.abs())
    if rotate:  # rotated back: at most the 2-norm of the errors, and seven roundings of 2^-24 of the 2-norm
        err = err.norm(dim=-1, keepdim=True) + 2.0 ** -21 * want.norm(dim=-1, keepdim=True)
        want = want @ h
    tol = U[q.dtype] * want.abs() + err
    tol = tol + (2.0 ** -25 if q.dtype == F16 else 2.0 ** -134)  # half a step of the outputs' subnormals
    bad = (out.double() - want).abs() / tol
    assert bool(torch.isfinite(out).all()) and float(bad.max()) <= 1.0, float(bad.max())
    return out, want


FORMS = [(BF16, 4, 128), (F16, 8, 0), (BF16, 16, 0), (F16, 16, 128)]  # type, query heads (8 and 16 columns), rotation


@pytest.mark.parametrize("dtype,heads,rotate", FORMS)
@pytest.mark.parametrize("power", [10, 17, 23, 30, 40])
@pytest.mark.parametrize("n", [70, 2048])
def test_a_large_value_without_weight(hq, dtype, heads, rotate, power, n):
    """A token whose value is 2^power times the others' and whose score is 60 powers of two below them."""
    g = _gen(1000 + power)
    powers = _normal(g, n) * 0.5
    powers[n // 3] = -60.0
    q, k = _directed(g, n, heads, powers, dtype)
    v = _normal(g, n, 1, 128)
    v[n // 3] *= 2.0 ** power
    _check(hq, q, k, v, rotate)


@pytest.mark.parametrize("dtype,heads,rotate", FORMS)
@pytest.mark.parametrize("std", [1.0, 2.0 ** -7, 1e-4, 2.0 ** -40, 2.0 ** 60])
def test_zero_values_among_small_ones(hq, dtype, heads, rotate, std):
    """Tokens whose value is zero, some of them with the largest scores, beside values of any size."""
    if dtype == F16 and std > 1.0:
        std = 2.0 ** 9  # outputs that the type holds
    g = _gen(1100)
    n = 1500
    powers = _normal(g, n)
    zero = torch.randperm(n, generator=g, device="cuda")[:400]
    powers[zero[:50]] += 12.0
    powers[zero[50]] = 40.0
    q, k = _directed(g, n, heads, powers, dtype)
    v = std * _normal(g, n, 1, 128)
    v[zero] = 0.0
    _check(hq, q, k, v, rotate)
    v[:] = 0.0
    out, _ = _check(hq, q, k, v, rotate)
    assert bool((out == 0).all())


@pytest.mark.parametrize("dtype,heads,rotate", FORMS)
def test_outputs_scale_with_the_values(hq, dtype, heads, rotate):
    """Values times a power of two have the same codes: the outputs are the same ones times it, to their rounding."""
    g = _gen(1200)
    n = 900
    q, k = _directed(g, n, heads, _normal(g, n), dtype)
    v = _normal(g, n, 1, 128)
    v[::7] = 0.0
    one, want = _check(hq, q, k, v, rotate)
    for power in (-7, -3, 5) if dtype == F16 else (-100, -14, -7, 20, 100):
        got, _ = _check(hq, q, k, v * 2.0 ** power, rotate)
        # twice the bound on one of them: what is held in 32 bits may round in another place
        assert bool(((got.double() * 2.0 ** -power - one.double()).abs() <= 2.2 * U[dtype] * want.abs() + 2.0 ** -9).all())


@pytest.mark.parametrize("dtype,heads,rotate", FORMS)
@pytest.mark.parametrize("window,sinks", [(100, 0), (333, 5)])
def test_large_values_outside_a_window(hq, dtype, heads, rotate, window, sinks):
    """Tokens just outside the window, in a group of 16 that is partly inside, with values 2^30 times the others'."""
    g = _gen(1300 + window)
    n = 1003
    for q_len in (1, 3):
        q, k = _directed(g, n, heads, _normal(g, n) * 0.5, dtype)
        q = q.expand(q_len, -1, -1).contiguous()
        v = _normal(g, n, 1, 128)
        v[sinks:n - q_len - window + 1] *= 2.0 ** 30
        _check(hq, q, k, v, rotate, window=window, sinks=sinks, q_len=q_len)


@pytest.mark.parametrize("dtype,heads,rotate", FORMS)
@pytest.mark.parametrize("n", [333, 2048])
def test_value_sizes_over_2_to_30(hq, dtype, heads, rotate, n):
    """Sizes spread evenly over 2^30 in any order, and rising or falling against the scores so that all weigh alike."""
    g = _gen(1400 + n)
    top = 0.0 if dtype == BF16 else -8.0  # outputs that the type holds
    size = torch.rand(n, generator=g, device="cuda") * 30.0 - 22.0 + top
    for powers, order in ((_normal(g, n), size), (-size, size), (-size.sort().values, size.sort().values),
                          (-size.sort(descending=True).values, size.sort(descending=True).values)):
        q, k = _directed(g, n, heads, powers, dtype)
        _check(hq, q, k, _normal(g, n, 1, 128) * torch.exp2(order)[:, None, None], rotate)


@pytest.mark.parametrize("rotate", [0, 128])
@pytest.mark.parametrize("heads", [1, 16])
def test_value_sizes_over_the_whole_range(hq, heads, rotate):
    """FP32 values from 2^-100 to 2^100, the scores against their sizes: a weight of 2^-100 on a value of 2^100 counts."""
    g = _gen(1500)
    n = 600
    size = torch.rand(n, generator=g, device="cuda") * 200.0 - 100.0
    for powers in (-0.5 * size, -size.clamp(min=-20.0, max=60.0), torch.zeros(n, device="cuda")):
        q, k = _directed(g, n, heads, powers, BF16)
        _check(hq, q, k, _normal(g, n, 1, 128) * torch.exp2(size)[:, None, None], rotate)


@pytest.mark.parametrize("dtype,heads,rotate", FORMS)
def test_a_long_request_in_many_shares(hq, dtype, heads, rotate):
    """20,001 tokens split over the GPU, whose shares differ in size by up to 2^30: the joins keep the small ones."""
    g = _gen(1600)
    n = 20_001
    size = torch.where(torch.arange(n, device="cuda") % 5000 < 2500, -20.0, 8.0)
    powers = torch.where(size > 0, -28.0, 0.0) + 0.3 * _normal(g, n)
    q, k = _directed(g, n, heads, powers, dtype)
    v = _normal(g, n, 1, 128) * torch.exp2(size)[:, None, None]
    v[4000:4100] = 0.0
    _check(hq, q, k, v, rotate, page=64)


@pytest.mark.parametrize("dtype,heads,rotate", FORMS)
@pytest.mark.parametrize("std", [2.0 ** -8, 1.0])
def test_a_score_far_above_the_others(hq, dtype, heads, rotate, std):
    """Scores of hundreds and thousands, one 40 and more above the rest: the output is that token's stored value, rounded."""
    g = _gen(1700)
    n = 500
    for top in (100.0, 1000.0, 8000.0, 100000.0):  # powers of two of the largest score
        d = torch.sign(_normal(g, 128)) / 128 ** 0.5
        q = (16.0 * d).expand(1, heads, 128).to(dtype).contiguous()
        powers = torch.rand(n, generator=g, device="cuda") * 0.5 * top
        powers[123] = top
        k = powers[:, None, None] * (math.log(2.0) / (16.0 * SCALE)) * d
        v = std * _normal(g, n, 1, 128)
        out, want = _check(hq, q, k, v, rotate)
        # whatever the scores' errors: the weight's rounding and 2^-15 as in _check, of the winner's value.  The other
        # weights are below 2^-39 (margins of 50 and more in powers of two, keys off by a fifth at most) and off by less
        # than a tenth of themselves: it shows where the winner's value is zero
        rest = n * 0.1 * 2.0 ** -39 * float(v.abs().max())
        size = want.abs() if not rotate else want.norm(dim=-1, keepdim=True)
        part = 2.0 ** -11 if dtype == BF16 else 2.0 ** -22
        assert bool(((out.double() - want).abs() <= U[dtype] * want.abs() + (part + 2.0 ** -15) * size
                     + (2.0 ** -25 if dtype == F16 else 0.0) + rest * (128 ** 0.5 if rotate else 1)).all()), top


# --------------------------------------------------------- calls without a workspace
def _small(hq, g):
    cache = hq.kv4_cache(8, 16, 2)
    t = torch.arange(128, device="cuda")
    hq.kv4_append(_normal(g, 128, 2, 128), _normal(g, 128, 2, 128), t, cache)
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
    return _normal(g, 2, 8, 128).to(BF16), cache, table, torch.tensor([64, 50], dtype=torch.int32, device="cuda")


def test_errors_of_a_call_without_a_workspace(hq):
    """The device's report comes back with want_error, with a workspace or without, captured or not."""
    q, cache, table, lens = _small(hq, _gen(1800))
    want = hq.kv4_attention(q, cache, table, lens)
    ws, side = hq.kv4_attention_workspace(), torch.cuda.Stream()
    bad = table.clone()
    bad[1, 2] = 8
    cu = torch.tensor([0, 1, 9], dtype=torch.int32, device="cuda")
    for kw in ({}, {"ws": ws}, {"stream": side}):
        for args, status in (({}, 0), ({"block_table": bad}, hq.HQ_ERR_PAGE), ({"cu_q": cu}, hq.HQ_ERR_SHAPE), ({}, 0)):
            torch.cuda.synchronize()
            o, lse, error = hq.kv4_attention(**{"q": q, "cache": cache, "block_table": table, "seq_lens": lens, **args}, **kw,
                                             want_lse=True, want_error=True)
            torch.cuda.synchronize()
            assert error.dtype == torch.int32 and error.tolist() == [status]
            assert torch.equal(o[0], want[0]) and lse.shape == (2, 8)
            if "ws" in kw:
                assert hq.hq_get_error(ws) == status
    o, error = hq.kv4_attention(q, cache, table, lens, want_error=True)
    assert torch.equal(o, want) and int(error) == 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, error = hq.kv4_attention(q, cache, table, lens, want_error=True)
    for entry, status in ((8, hq.HQ_ERR_PAGE), (6, 0), (-1, hq.HQ_ERR_PAGE)):
        table[1, 2] = entry
        graph.replay()
        assert int(error) == status and torch.equal(o[0], want[0])


def test_a_workspace_of_the_calls_own_from_used_memory(hq):
    q, cache, table, lens = _small(hq, _gen(1900))
    ws = hq.kv4_attention_workspace()
    want = hq.kv4_attention(q, cache, table, lens, ws=ws)
    for byte in (0xFF, 0x01, 0x7F):
        used = torch.full((hq.hq_kv4_attention_workspace_size(),), byte, dtype=torch.uint8, device="cuda")
        del used
        o, error = hq.kv4_attention(q, cache, table, lens, want_error=True)
        assert torch.equal(o, want) and int(error) == 0
    # of a workspace only the stated part has to be zero
    ws.fill_(0xFF)
    ws[:hq.HQ_KV4_ATTENTION_STATE_BYTES] = 0
    for _ in range(2):
        assert torch.equal(hq.kv4_attention(q, cache, table, lens, ws=ws), want)
    assert hq.hq_get_error(ws) == 0
