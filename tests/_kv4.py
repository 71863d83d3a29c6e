"""An independent reading of the cache layout and binary64 forms of the attention-layer operators, for the tests."""
from __future__ import annotations

import numpy as np
import torch

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def hadamard128() -> np.ndarray:
    h = np.ones((1, 1))
    while h.shape[0] < 128:
        h = np.block([[h, h], [h, -h]])
    return h / np.sqrt(128.0)


def token_bytes(group: np.ndarray, r: int, value: bool):
    """(codes [64] in natural order, block scales [8], decode scale) of token r of a 2432-byte group."""
    codes, sf = np.empty(64, np.uint8), np.empty(8, np.uint8)
    for b in range(8):
        for pair in range(8):  # elements 16 b + 2 pair, + 1
            if value:
                at = 1024 + 512 * (r // 8) + 64 * pair + 16 * (r % 8 // 2) + 8 * (r % 2) + b
            else:
                at = 64 * r + 16 * (pair // 2) + 2 * b + pair % 2
            codes[8 * b + pair] = group[at]
        sf[b] = group[2176 + 64 * (r // 8) + 16 * (r % 8 // 2) + 2 * b + r % 2] if value else group[2048 + 8 * r + b]
    first = (2368 if value else 2304) + 4 * r
    return codes, sf, group[first:first + 4].copy().view(np.float32)[0]


_PLACES = None


def _places():
    global _PLACES
    if _PLACES is None:
        mark = np.arange(2432, dtype=np.int64)
        place = np.empty((2, 16, 72), np.int64)
        for v in (0, 1):
            for r in range(16):
                for b in range(8):
                    for pair in range(8):
                        place[v, r, 8 * b + pair] = (1024 + 512 * (r // 8) + 64 * pair + 16 * (r % 8 // 2) + 8 * (r % 2) + b
                                                     if v else 64 * r + 16 * (pair // 2) + 2 * b + pair % 2)
                    place[v, r, 64 + b] = (2176 + 64 * (r // 8) + 16 * (r % 8 // 2) + 2 * b + r % 2 if v
                                           else 2048 + 8 * r + b)
        assert mark[place].max() < 2304
        _PLACES = torch.from_numpy(place)
    return _PLACES


def decode(groups: torch.Tensor, value: bool) -> torch.Tensor:
    """Values [..., 16, 128] (float64) of groups uint8 [..., 2432]."""
    place = _places()[int(value)].to(groups.device)
    by = groups[..., place[:, :64]].long()
    grid = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64, device=groups.device)
    v = torch.stack((grid[by & 15], grid[by >> 4]), -1).flatten(-2)
    sf = groups[..., place[:, 64:]].contiguous().view(torch.float8_e4m3fn).double()
    first = 2368 if value else 2304
    dec = groups[..., first:first + 64].contiguous().view(torch.float32).double()
    return v * sf.repeat_interleave(16, -1) * dec[..., None]


def request_kv(cache: torch.Tensor, pages: torch.Tensor, n: int):
    """Keys and values [heads, n, 128] (float64, as stored) of the first n tokens on `pages`."""
    g = cache[pages.long()].transpose(0, 1).flatten(1, 2)
    return decode(g, False).flatten(1, 2)[:, :n], decode(g, True).flatten(1, 2)[:, :n]


def attention64(q, cache, table, lens, q_rows, scale, window, sinks, rotate):
    """float64 (out, lse, weight, peak) of the attention: q_rows[b] = (first, last + 1) rows of q; weight is sum_d sum_t
    p_t |v_td| of the stored values over sqrt(128) (or the per-dimension sums without rotation): what a relative error of
    every weight can do to an output; peak the largest weight of a row."""
    Tq, Hq, _ = q.shape
    page = cache.shape[2] * 16
    out = torch.zeros((Tq, Hq, 128), dtype=torch.float64, device=q.device)
    lse = torch.full((Tq, Hq), -torch.inf, dtype=torch.float64, device=q.device)
    weight = torch.zeros((Tq, Hq, 128), dtype=torch.float64, device=q.device)
    peak = torch.zeros((Tq, Hq, 1), dtype=torch.float64, device=q.device)
    h = torch.from_numpy(hadamard128()).to(q.device)
    H = cache.shape[1]
    for b, (r0, r1) in enumerate(q_rows):
        n = int(lens[b])
        if r1 <= r0 or n <= 0:
            continue
        pages = table[b, : -(-n // page)]
        ok = ((pages >= 0) & (pages < cache.shape[0])).repeat_interleave(page)[:n]
        k, v = request_kv(cache, pages.clamp(0, cache.shape[0] - 1), n)
        x = q[r0:r1].double()
        x = (x @ h if rotate else x).reshape(r1 - r0, H, Hq // H, 128)
        s = torch.einsum("qhgd,htd->qhgt", x, k) * scale
        t = torch.arange(n, device=q.device)[None]
        p = torch.arange(n - (r1 - r0), n, device=q.device)[:, None]
        see = (t <= p) & ok[None]
        if window:
            see &= (p - t < window) | (t < sinks)
        s = s.masked_fill(~see[:, None, None], -torch.inf)
        some = see.any(1)
        l = torch.logsumexp(s, -1)
        w = torch.exp(s - torch.where(some[:, None, None], l, torch.zeros_like(l))[..., None])
        o = torch.einsum("qhgt,htd->qhgd", w, v).reshape(r1 - r0, Hq, 128)
        a = torch.einsum("qhgt,htd->qhgd", w, v.abs()).reshape(r1 - r0, Hq, 128)
        out[r0:r1] = o @ h if rotate else o
        weight[r0:r1] = a.sum(-1, keepdim=True) / 128 ** 0.5 if rotate else a
        lse[r0:r1] = l.reshape(r1 - r0, Hq)
        peak[r0:r1] = w.amax(-1).reshape(r1 - r0, Hq, 1)
    return out, lse, weight, peak
