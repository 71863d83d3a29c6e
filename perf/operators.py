"""The operators of an attention layer around the quantizers, as cases to measure.

Per step of a serving loop: the residual's addition with the root-mean-square norm and K128 FP8 codes (and the norm's
backward pass, for training), rotary positions of q and k, block tables and slot maps from request lengths, the paged
NVFP4 key/value cache (write, read back), and attention of the newest tokens over that cache.

With `own` false, run() computes the operators in their plain form with elementary torch operations; with `own` true it
calls the package's entry points.  exact() gives the same results from the definitions in binary64.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
HEAD = 128          # dimension of a cached head: one rotated 128-vector
GROUP = 16          # tokens of a cache group
GROUP_BYTES = 2432  # 16 tokens x (64 + 64 code bytes, 8 + 8 block scales, 4 + 4 bytes of vector scales)
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a decoding step of 16 requests: latency
        {"name": "norm_decode_16x7168", "op": "norm", "M": 16, "K": 7168, "dtype": "bf16", "residual": True,
         "transposed": False},
        # the rows of a whole prefill batch (the grouped cast's workload), scales as a following product reads them
        {"name": "norm_prefill_16384x7168", "op": "norm", "M": 16384, "K": 7168, "dtype": "bf16", "residual": True,
         "transposed": True},
        # the norm's gradients in a training step, with the gradient that arrives through the residual
        {"name": "norm_back_8191x4096", "op": "norm_back", "M": 8191, "K": 4096, "dtype": "bf16", "dres": True},
        # one token each of 64 requests, half of every head rotated (the indexer's 64 + 64), far positions
        {"name": "rope_decode_64", "op": "rope", "T": 64, "Hq": 64, "Hk": 8, "D": 128, "R": 64, "offset": 0,
         "interleaved": True, "dtype": "bf16", "far": 1 << 20, "factor": 32.0, "inverse": False},
        # a prefill of 8192 tokens, whole heads, the two-halves layout
        {"name": "rope_prefill_8192", "op": "rope", "T": 8192, "Hq": 64, "Hk": 8, "D": 128, "R": 128, "offset": 0,
         "interleaved": False, "dtype": "bf16", "far": 8192, "factor": 1.0, "inverse": False},
        # bookkeeping of a decoding step: 256 requests with one token each, some of them ended
        {"name": "slots_decode_256", "op": "slots", "B": 256, "page": 64, "width": 256, "longest": 16000, "new": 1,
         "ended": 0.05, "salt": 1},
        # bookkeeping of a prefill: 64 new requests of up to 2048 tokens
        {"name": "slots_prefill_64", "op": "slots", "B": 64, "page": 16, "width": 512, "longest": 4096, "new": 2048,
         "ended": 0.1, "salt": 2},
        # the new tokens of a decoding step into the cache, and the same tokens read back
        {"name": "cache_decode_64", "op": "cache", "N": 64, "H": 8, "page": 64, "pages": 512, "rotate": True,
         "dtype": "bf16"},
        # a prefill's tokens into the cache, and read back as a later chunk's attention takes them
        {"name": "cache_prefill_16384", "op": "cache", "N": 16384, "H": 8, "page": 64, "pages": 300, "rotate": True,
         "dtype": "bf16"},
        # a small decoding batch of short requests: latency
        {"name": "attend_4x700", "op": "attend", "B": 4, "Hq": 32, "Hkv": 8, "shortest": 17, "longest": 700, "page": 16,
         "q_len": 1, "ragged": False, "window": 0, "sinks": 0, "rotate": True, "dtype": "bf16", "salt": 3},
        # a full decoding batch of long requests
        {"name": "attend_32x16384", "op": "attend", "B": 32, "Hq": 64, "Hkv": 8, "shortest": 8000, "longest": 16384,
         "page": 64, "q_len": 1, "ragged": False, "window": 0, "sinks": 0, "rotate": True, "dtype": "bf16", "salt": 4},
        # drafted tokens verified, 1 to 4 a request, over a sliding window with a few first tokens kept
        {"name": "attend_verify_window", "op": "attend", "B": 48, "Hq": 20, "Hkv": 4, "shortest": 1, "longest": 9001,
         "page": 32, "q_len": 4, "ragged": True, "window": 2047, "sinks": 4, "rotate": True, "dtype": "f16", "salt": 5},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_back", "rope", "slots", "cache", "attend", "attend"])
    if op in ("norm", "norm_back"):
        K = 128 * _log_int(rng, 1, 64)
        M = _log_int(rng, 1, min(16384, (16384 * 7168 // 2) // K))
        c = {"op": op, "M": M, "K": K, "dtype": rng.choice(["bf16", "bf16", "f16", "f32"])}
        if op == "norm":
            return {**c, "residual": rng.random() < 0.8, "transposed": rng.random() < 0.5}
        return {**c, "dres": rng.random() < 0.8}
    if op == "rope":
        D = rng.choice([64, 80, 128, 192])
        R = 2 * rng.randint(8, D // 2)
        return {"op": op, "T": _log_int(rng, 1, 8192), "Hq": rng.randint(1, 64), "Hk": rng.randint(1, 8), "D": D, "R": R,
                "offset": rng.choice([0, D - R]), "interleaved": rng.random() < 0.5,
                "dtype": rng.choice(["bf16", "f16", "f32"]), "far": _log_int(rng, 64, 1 << 20),
                "factor": rng.choice([1.0, 4.0, 32.0]), "inverse": rng.random() < 0.3}
    if op == "slots":
        page = rng.choice([16, 32, 64, 128])
        longest = _log_int(rng, page, 16000)
        new = rng.choice([1, rng.randint(2, 8), _log_int(rng, 16, 1024)])
        B = _log_int(rng, 1, max(1, min(1024, 65536 // new)))
        return {"op": op, "B": B, "page": page, "width": (longest + new) // page + 1 + rng.randint(0, 9),
                "longest": longest, "new": new, "ended": rng.choice([0.0, 0.1, 0.3]), "salt": rng.randrange(1 << 30)}
    if op == "cache":
        N, page = _log_int(rng, 1, 16384), rng.choice([16, 32, 64, 128])
        return {"op": op, "N": N, "H": rng.randint(1, 8), "page": page, "pages": N // page + rng.randint(1, 100),
                "rotate": rng.random() < 0.8, "dtype": rng.choice(["bf16", "f16", "f32"])}
    Hkv, g = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 7, 8, 16])
    longest = _log_int(rng, 20, 65536)
    B = _log_int(rng, 1, max(1, min(64, 32 * 16384 * 8 // (2 * longest * Hkv))))
    window = rng.choice([0, 0, rng.randint(1, longest)])
    return {"op": op, "B": B, "Hq": g * Hkv, "Hkv": Hkv, "shortest": rng.choice([0, 1, longest // 2]), "longest": longest,
            "page": rng.choice([16, 32, 64, 128]), "q_len": rng.choice([1, 1, 2, 5, 8]), "ragged": rng.random() < 0.3,
            "window": window, "sinks": rng.choice([0, 4, 17]) if window else 0, "rotate": rng.random() < 0.8,
            "dtype": rng.choice(["bf16", "f16"]), "salt": rng.randrange(1 << 30)}


def _lens(c):
    """Cached tokens (the new ones among them) and new tokens of each request of an `attend` case."""
    rng = random.Random(c["salt"])
    q = [rng.randint(0, c["q_len"]) if c["ragged"] else c["q_len"] for _ in range(c["B"])]
    n = [max(rng.randint(c["shortest"], c["longest"]), k) for k in q]
    n[rng.randrange(c["B"])] = max(c["longest"], c["q_len"])
    if sum(q) == 0:
        q[0], n[0] = 1, max(n[0], 1)
    return n, q


def _visible(c, n, q):
    """Tokens that at least one query of a request sees: a window and the first tokens, or all."""
    if q == 0:
        return 0
    lo = max(0, n - q - c["window"] + 1) if c["window"] else 0
    return n - lo + min(lo, c["sinks"])


def _requests(c):
    """Lengths before the step and new tokens (-1: the request ended) of a `slots` case."""
    rng = random.Random(c["salt"])
    lens = [rng.randint(0, c["longest"]) for _ in range(c["B"])]
    new = [-1 if rng.random() < c["ended"] else (1 if c["new"] == 1 else rng.randint(0, c["new"])) for _ in lens]
    return lens, new


def _capacity(c):
    return c["B"] * c["new"]  # rows of the slot map, as a captured step has them; fewer are in use


def work(c):
    op = c["op"]
    if op == "norm":
        e, n = SIZE[c["dtype"]], c["M"] * c["K"]
        return {"bytes": n * (e * (3 if c["residual"] else 1) + 1) + n // 32 + 4 * c["M"] + e * c["K"], "flops": 8 * n}
    if op == "norm_back":
        e, n = SIZE[c["dtype"]], c["M"] * c["K"]
        return {"bytes": n * e * (4 if c["dres"] else 3) + 4 * c["M"] + (e + 4) * c["K"], "flops": 10 * n}
    if op == "rope":
        n = c["T"] * (c["Hq"] + c["Hk"])
        return {"bytes": 2 * n * c["D"] * SIZE[c["dtype"]] + 8 * c["T"], "flops": 3 * n * c["R"]}
    if op == "slots":
        lens, new = _requests(c)
        total = sum(max(v, 0) for v in new)
        pages = sum((n + max(v, 0)) // c["page"] + 1 for n, v in zip(lens, new))
        return {"bytes": 16 * c["B"] + 16 * _capacity(c) + 4 * pages, "flops": 4 * total}
    if op == "cache":
        n = c["N"] * c["H"]
        return {"bytes": n * (4 * HEAD * SIZE[c["dtype"]] + 2 * 152) + 8 * c["N"], "flops": n * HEAD * 30}
    n, q = _lens(c)
    seen = sum(_visible(c, a, b) for a, b in zip(n, q))
    pairs = sum(_visible(c, a, b) * b for a, b in zip(n, q))
    return {"bytes": seen * c["Hkv"] * 152 + 2 * sum(q) * c["Hq"] * HEAD * SIZE[c["dtype"]],
            "flops": 4 * HEAD * pairs * c["Hq"]}


# ----------------------------------------------------------------- inputs
def _inv_freq(c):
    """Frequencies of the rotated pairs (radians a position) and the magnitude of the rotation, scaled for a context
    `factor` times the trained one by parts: fast pairs keep theirs, slow ones are divided, a ramp between."""
    base, R, f, trained = 10000.0, c["R"], c["factor"], 4096
    inv = torch.tensor([base ** (-2 * i / R) for i in range(R // 2)], dtype=torch.float64)
    if f == 1.0:
        return inv, 1.0

    def pair(turns):
        return R * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(base))

    lo = max(math.floor(pair(32.0)), 0)
    hi = min(math.ceil(pair(1.0)), R - 1)
    ramp = ((torch.arange(R // 2, dtype=torch.float64) - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
    return inv / f * ramp + inv * (1 - ramp), 0.1 * math.log(f) + 1.0


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = "cuda"

    def normal(*shape, std=1.0, dtype="f32"):
        return (torch.randn(shape, generator=g, device=dev) * std).to(DTYPES[dtype])

    op = c["op"]
    if op in ("norm", "norm_back"):
        M, K, t = c["M"], c["K"], c["dtype"]
        s = {"case": c, "w": (1 + 0.1 * torch.randn(K, generator=g, device=dev)).to(DTYPES[t])}
        channel = torch.exp(0.5 * torch.randn(K, generator=g, device=dev))  # some channels are larger than others
        if op == "norm":
            s["x"] = normal(M, K, dtype=t)
            s["r"] = (torch.randn((M, K), generator=g, device=dev) * channel).to(DTYPES[t]) if c["residual"] else None
            return s
        s["dy"] = normal(M, K, std=1e-2, dtype=t)
        s["h"] = (torch.randn((M, K), generator=g, device=dev) * channel).to(DTYPES[t])
        s["rstd"] = 1.0 / torch.sqrt(s["h"].float().square().mean(-1) + 1e-6)
        s["dres"] = normal(M, K, std=1e-2, dtype=t) if c["dres"] else None
        return s
    if op == "rope":
        T, Hq, Hk, D = c["T"], c["Hq"], c["Hk"], c["D"]
        qkv = normal(T, (Hq + 2 * Hk) * D, dtype=c["dtype"])  # q and k are parts of one product's rows
        inv, magnitude = _inv_freq(c)
        return {"case": c, "q": qkv[:, :Hq * D].unflatten(1, (Hq, D)), "k": qkv[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D)),
                "pos": torch.randint(0, c["far"], (T,), generator=g, device=dev), "inv": inv.to(dev), "mag": magnitude}
    if op == "slots":
        lens, new = _requests(c)
        P, W = c["page"], c["width"]
        held = [-(-n // P) for n in lens]
        total = sum(held) + sum(-(-max(v, 0) // P) + 1 for v in new) + 7
        order = torch.randperm(total, generator=g, device=dev).to(torch.int32)
        lens_t = torch.tensor(lens, dtype=torch.int32, device=dev)
        held_t = torch.tensor(held, device=dev)
        at = torch.arange(W, device=dev)[None, :]
        first = (held_t.cumsum(0) - held_t)[:, None]
        table = torch.where(at < held_t[:, None], order[(first + at).clamp(max=total - 1)], 0).to(torch.int32)
        stack = torch.zeros(total, dtype=torch.int32, device=dev)
        n_free = total - sum(held)
        stack[:n_free] = order[sum(held):]
        return {"case": c, "lens": lens_t, "new": torch.tensor(new, dtype=torch.int32, device=dev), "table": table,
                "stack": stack, "count": torch.tensor([n_free], dtype=torch.int32, device=dev)}
    if op == "cache":
        N, H, P, t = c["N"], c["H"], c["page"], c["dtype"]
        channel = torch.exp(0.7 * torch.randn((H, HEAD), generator=g, device=dev))
        kv = torch.randn((N, 2, H, HEAD), generator=g, device=dev)
        kv[:, 0] *= channel
        kv = kv.to(DTYPES[t])
        slots = torch.randperm(c["pages"] * P, generator=g, device=dev)[:N]
        if N >= 8 * P:  # a prefill fills whole pages in order
            pages = torch.randperm(c["pages"], generator=g, device=dev)[: -(-N // P)]
            slots = (pages[:, None] * P + torch.arange(P, device=dev)[None, :]).flatten()[:N].contiguous()
        return {"case": c, "k": kv[:, 0], "v": kv[:, 1], "slots": slots,
                "cache": torch.zeros((c["pages"], H, P // GROUP, GROUP_BYTES), dtype=torch.uint8, device=dev)}
    n, q = _lens(c)
    B, H, P = c["B"], c["Hkv"], c["page"]
    held = [-(-v // P) for v in n]
    pages, W = sum(held) + 3, max(held)
    cache = torch.empty((pages, H, P // GROUP, GROUP_BYTES), dtype=torch.uint8, device=dev)
    channel = torch.exp(0.4 * torch.randn((H, 1, 1, HEAD), generator=g, device=dev))
    step = max(1, (1 << 27) // (H * P * HEAD))
    for p in range(0, pages, step):
        m = min(step, pages - p)
        k = torch.randn((m, H, P // GROUP, GROUP, HEAD), generator=g, device=dev) * channel
        v = torch.randn((m, H, P // GROUP, GROUP, HEAD), generator=g, device=dev)
        cache[p:p + m] = _pack(*_nvfp4(k, c["rotate"]), *_nvfp4(v, c["rotate"]))
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    held_t = torch.tensor(held, device=dev)
    at = torch.arange(W, device=dev)[None, :]
    table = torch.where(at < held_t[:, None], order[((held_t.cumsum(0) - held_t)[:, None] + at).clamp(max=pages - 1)], -1)
    cu = torch.tensor([0] + q, device=dev).cumsum(0).to(torch.int32)
    return {"case": c, "q": normal(sum(q), c["Hq"], HEAD, std=1.5, dtype=c["dtype"]), "cache": cache,
            "table": table.to(torch.int32), "lens": torch.tensor(n, dtype=torch.int32, device=dev),
            "cu": cu if c["ragged"] else None}


# ------------------------------------------------- the plain forms' parts
def _hadamard(x):
    """128-point orthonormal Hadamard rotation of the last dimension: Sylvester order, ascending stages, one scaling."""
    n = 1
    while n < HEAD:
        y = x.unflatten(-1, (HEAD // (2 * n), 2, n))
        a, b = y[..., 0, :], y[..., 1, :]
        x = torch.stack((a + b, a - b), dim=-2).flatten(-3)
        n *= 2
    return x * (2.0 ** -3.5)


def _nvfp4(x, rotate):
    """(E2M1 codes two a byte [..., 64], E4M3 block scales [..., 8] as bytes, decode scales [...]) of 128-vectors."""
    y = _hadamard(x.float()) if rotate else x.float()
    blocks = y.unflatten(-1, (8, 16))
    per_block = blocks.abs().amax(-1)
    amax = per_block.amax(-1)
    enc = torch.full_like(amax, 2688.0) / amax
    enc = torch.where((amax > 0) & torch.isfinite(enc), enc, torch.ones_like(enc))
    sf8 = (per_block / torch.full_like(per_block, 6.0) * enc[..., None]).to(torch.float8_e4m3fn)
    sf = sf8.float()
    mul = torch.where(sf > 0, enc[..., None] / sf, torch.zeros_like(sf))
    v = blocks * mul[..., None]
    a = v.abs()
    code = (a > 0.25).to(torch.uint8)
    for edge, tie_up in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (a >= edge) if tie_up else (a > edge)
    code += torch.signbit(v).to(torch.uint8) * 8
    code = code.flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), sf8.view(torch.uint8), torch.ones_like(enc) / enc


def _pack(kc, ks, kd, vc, vs, vd):
    """Cache groups [..., 2432] of 16 tokens from codes [..., 16, 64], block scales [..., 16, 8], scales [..., 16]."""
    k1 = kc.unflatten(-1, (8, 4, 2)).transpose(-3, -2).flatten(-4)                      # token, quad, block, byte
    v1 = vc.unflatten(-1, (8, 8)).unflatten(-3, (2, 4, 2))                               # half, pair, odd, block, byte
    v1 = v1.permute(*range(v1.dim() - 5), -5, -1, -4, -3, -2).flatten(-5)                # half, byte, pair, odd, block
    s1 = vs.unflatten(-2, (2, 4, 2)).transpose(-2, -1).flatten(-4)                       # half, pair, block, odd
    return torch.cat((k1, v1, ks.flatten(-2), s1, kd.contiguous().view(torch.uint8), vd.contiguous().view(torch.uint8)), -1)


def _unpack(c):
    """The inverse of _pack."""
    kc = c[..., :1024].unflatten(-1, (16, 4, 8, 2)).transpose(-3, -2).flatten(-3)
    vc = c[..., 1024:2048].unflatten(-1, (2, 8, 4, 2, 8))
    vc = vc.permute(*range(vc.dim() - 5), -5, -3, -2, -1, -4).flatten(-2).flatten(-4, -2)
    vs = c[..., 2176:2304].unflatten(-1, (2, 4, 8, 2)).transpose(-2, -1).flatten(-4, -2)
    return (kc, c[..., 2048:2176].unflatten(-1, (16, 8)), c[..., 2304:2368].contiguous().view(torch.float32),
            vc, vs, c[..., 2368:].contiguous().view(torch.float32))


def _values(codes, sf, scale):
    """Values of codes [..., 64], block scales [..., 8] and scales [...] in binary32."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    pairs = torch.stack((lut.repeat(16), lut.repeat_interleave(16)), -1)
    v = pairs[codes.int()].flatten(-2).unflatten(-1, (8, 16))
    return ((v * sf.contiguous().view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)) * scale[..., None]


def _addresses(device):
    """Bytes of a token's codes and block scales in its group: K codes, V codes [16, 64], K scales, V scales [16, 8]."""
    t, b = torch.arange(16, device=device)[:, None], torch.arange(64, device=device)[None, :]
    kc = t * 64 + (b % 8 // 2) * 16 + b // 8 * 2 + b % 2
    vc = 1024 + t // 8 * 512 + (b % 8 * 4 + t % 8 // 2) * 16 + t % 2 * 8 + b // 8
    s = torch.arange(8, device=device)[None, :]
    return kc, vc, 2048 + t * 8 + s, 2176 + t // 8 * 64 + t % 8 // 2 * 16 + s * 2 + t % 2


def _group_base(slots, cache):
    """First byte of the group of each slot and head [N, H], and the slot's place in it [N]."""
    pages, H, G, n = cache.shape
    page, at = slots // (16 * G), slots % (16 * G)
    return ((page[:, None] * H + torch.arange(H, device=slots.device)) * G + (at // 16)[:, None]) * n, at % 16


# -------------------------------------------------------------------- run
def run(s):
    return _own(s) if own else _plain(s)


def _plain(s):
    return {"norm": _plain_norm, "norm_back": _plain_norm_back, "rope": _plain_rope, "slots": _plain_slots,
            "cache": _plain_cache, "attend": _plain_attend}[s["case"]["op"]](s)


def _plain_norm(s):
    c, x = s["case"], s["x"]
    h = x if s["r"] is None else (x.float() + s["r"].float()).to(x.dtype)
    hf = h.float()
    rstd = 1.0 / torch.sqrt(hf.square().mean(-1) + 1e-6)
    y = (hf * rstd[:, None] * s["w"].float()).unflatten(-1, (-1, 128))
    scale = y.abs().amax(-1).clamp(min=1e-10) * (1.0 / 448.0)
    codes = (y / scale[..., None]).to(torch.float8_e4m3fn).flatten(-2)
    out = {"codes": codes, "scales": scale.t().contiguous() if c["transposed"] else scale, "rstd": rstd}
    return out if s["r"] is None else {**out, "h": h}


def _plain_norm_back(s):
    dy, h, rstd = s["dy"].float(), s["h"].float(), s["rstd"][:, None]
    g = dy * s["w"].float()
    dx = rstd * (g - h * (rstd * rstd * (g * h).mean(-1, keepdim=True)))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return {"dx": dx.to(s["dy"].dtype), "dw": (dy * h * rstd).sum(0)}


def _plain_rope(s):
    c = s["case"]
    angle = s["pos"].double()[:, None] * s["inv"]
    cos, sin = (angle.cos() * s["mag"]).float()[:, None], (angle.sin() * s["mag"]).float()[:, None]
    if c["inverse"]:
        sin = -sin

    def turn(x):
        y, R, o = x.float(), c["R"], c["offset"]
        z = y[..., o:o + R]
        a, b = (z[..., 0::2], z[..., 1::2]) if c["interleaved"] else (z[..., :R // 2], z[..., R // 2:])
        u, v = a * cos - b * sin, a * sin + b * cos
        z = torch.stack((u, v), -1).flatten(-2) if c["interleaved"] else torch.cat((u, v), -1)
        return torch.cat((y[..., :o], z, y[..., o + R:]), -1).to(x.dtype)

    return turn(s["q"]), turn(s["k"])


def _plain_slots(s):
    c, lens, new, table, stack = s["case"], s["lens"].long(), s["new"].long(), s["table"], s["stack"]
    P, n_slots = c["page"], _capacity(c)
    ended = new < 0
    add = new.clamp(min=0)
    held = (lens + P - 1) // P
    after = torch.where(ended, 0, lens + add)
    need = torch.where(ended, 0, (after + P - 1) // P - held)
    back = torch.where(ended, held, 0)
    top = s["count"].long() + back.sum()
    at = torch.arange(table.shape[1], device=table.device)[None, :]
    # pages of ended requests go onto the stack in order, then new pages come off its top in order
    put = (s["count"] + back.cumsum(0) - back)[:, None] + at
    freed = at < back[:, None]
    stack[put[freed]] = table[freed]
    take = top - 1 - ((need.cumsum(0) - need - held)[:, None] + at)
    fresh = (at >= held[:, None]) & (at < (held + need)[:, None])
    table[fresh] = stack[take[fresh]]
    cu = torch.cat((torch.zeros_like(add[:1]), add.cumsum(0)))
    row = torch.arange(n_slots, device=table.device)
    req = torch.searchsorted(cu[1:], row, right=True).clamp(max=c["B"] - 1)
    used = row < cu[-1]
    pos = torch.where(used, lens[req] + row - cu[req], 0)
    slot = torch.where(used, table[req, pos // P].long() * P + pos % P, -1)
    count = (top - need.sum()).to(torch.int32)
    return {"table": table, "stack": stack, "count": count, "lens": after.to(torch.int32), "cu": cu.to(torch.int32),
            "slots": slot, "positions": pos, "status": torch.zeros_like(count)}


def _plain_cache(s):
    c, cache = s["case"], s["cache"]
    base, r = _group_base(s["slots"], cache)
    places = _addresses(cache.device)
    flat = cache.view(-1)
    scales = flat.view(torch.float32)
    got = []
    for j, x in enumerate((s["k"], s["v"])):  # keys, values
        at_codes, at_sf = base[..., None] + places[j][r][:, None], base[..., None] + places[2 + j][r][:, None]
        at_scale = base // 4 + (576 + 16 * j) + r[:, None]
        codes, sf, scale = _nvfp4(x, c["rotate"])
        flat[at_codes], flat[at_sf], scales[at_scale] = codes, sf, scale
        y = _values(flat[at_codes], flat[at_sf], scales[at_scale])
        got.append(y.to(x.dtype))
    return got


def _plain_attend(s):
    c, cache = s["case"], s["cache"]
    B, H, g, P, W = c["B"], c["Hkv"], c["Hq"] // c["Hkv"], c["page"], s["table"].shape[1]
    Q, N = c["q_len"], P * W
    lens = s["lens"].long()
    cu = torch.arange(B + 1, device=cache.device) * Q if s["cu"] is None else s["cu"].long()
    kc, ks, kd, vc, vs, vd = _unpack(cache[s["table"].clamp(min=0).long()].transpose(1, 2))  # [B, H, W, G, ...]
    row = cu[:-1, None] + torch.arange(Q, device=cache.device)                                # rows of q [B, Q]
    real = row < cu[1:, None]
    q = s["q"].float()[row.clamp(max=s["q"].shape[0] - 1)].unflatten(2, (H, g)).permute(0, 2, 3, 1, 4)  # [B, H, g, Q, 128]
    if c["rotate"]:
        q = _hadamard(q)
    score = q.flatten(2, 3) @ _values(kc, ks, kd).flatten(2, 4).transpose(-1, -2) / math.sqrt(HEAD)     # [B, H, gQ, N]
    pos = (lens - (cu[1:] - cu[:-1]))[:, None] + torch.arange(Q, device=cache.device)                    # [B, Q]
    t = torch.arange(N, device=cache.device)
    see = (t <= pos[..., None]) & real[..., None]
    if c["window"]:
        see &= (pos[..., None] - t < c["window"]) | (t < c["sinks"])
    score = score.unflatten(2, (g, Q)).masked_fill(~see[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    o = p.flatten(2, 3) @ _values(vc, vs, vd).flatten(2, 4)
    o = o.unflatten(2, (g, Q)) / total.clamp(min=1e-30)
    if c["rotate"]:
        o = _hadamard(o)
    lse = (top + torch.log(total))[..., 0]
    return {"out": o.permute(0, 3, 1, 2, 4).flatten(2, 3)[real].to(s["q"].dtype),
            "lse": lse.permute(0, 3, 1, 2).flatten(2, 3)[real]}


# ---------------------------------------------------- the package's calls
def _own(s):
    import nvfp4_quantization_group_b200 as hq

    c = s["case"]
    op = c["op"]
    if op == "norm":
        out = hq.add_rmsnorm_fp8_k128(s["x"], s["w"], s["r"], eps=1e-6, want_rstd=True,
                                      scale_layout=hq.HQ_SCALE_TRANSPOSED if c["transposed"] else hq.HQ_SCALE_ROWMAJOR)
        got = {"codes": out["codes"].view(torch.float8_e4m3fn), "scales": out["scales"], "rstd": out["rstd"]}
        return got if s["r"] is None else {**got, "h": out["residual_out"]}
    if op == "norm_back":
        if "ws" not in s:  # kept by the program from step to step
            s["ws"] = hq.rmsnorm_backward_workspace(c["M"], c["K"])
        dx, dw = hq.rmsnorm_backward(s["dy"], s["h"], s["w"], s["rstd"], dres=s["dres"], ws=s["ws"])
        return {"dx": dx, "dw": dw}
    if op == "rope":
        return hq.rope(s["q"], s["k"], s["pos"], s["inv"], offset=c["offset"], magnitude=s["mag"], inverse=c["inverse"],
                       layout=hq.HQ_ROPE_INTERLEAVED if c["interleaved"] else hq.HQ_ROPE_HALVES)
    if op == "slots":
        o = hq.kv_slots(s["lens"], s["new"], s["table"], s["stack"], s["count"], c["page"], _capacity(c))
        return {"table": s["table"], "stack": s["stack"], "count": o["free_count"], "lens": o["lens"], "cu": o["cu_new"],
                "slots": o["slots"], "positions": o["positions"], "status": o["status"]}
    n = 128 if c["rotate"] else 0
    if op == "cache":
        hq.kv4_append(s["k"], s["v"], s["slots"], s["cache"], hadamard_n=n)
        return list(hq.kv4_gather(s["cache"], s["slots"], dtype=s["k"].dtype, hadamard_n=0))
    if "ws" not in s:  # kept by the program from step to step
        s["ws"] = hq.kv4_attention_workspace()
    o, lse = hq.kv4_attention(s["q"], s["cache"], s["table"], s["lens"], cu_q=s["cu"], q_len=c["q_len"],
                              window=c["window"], sinks=c["sinks"], hadamard_n=n, ws=s["ws"], want_lse=True)
    return {"out": o, "lse": lse}


# ------------------------------------------------------------- in 64 bits
def _h128():
    i = torch.arange(HEAD)
    bits = (i[:, None] & i[None, :])
    parity = sum((bits >> k) & 1 for k in range(7)) % 2
    return ((1 - 2 * parity).double() * 2.0 ** -3.5).cuda()


def _exact_vectors(x, rotate):
    """The values that the NVFP4 form of 128-vectors stands for, and no rotation back."""
    y = x.double() @ _h128() if rotate else x.double()
    b = y.unflatten(-1, (8, 16))
    # the binary32 steps of the scales are part of the format (ties are common among the values of narrow inputs)
    amax = y.abs().amax(-1)[..., None].float()
    enc = torch.where(amax > 0, torch.div(torch.full_like(amax, 2688.0), amax), torch.ones_like(amax))
    per_block = b.abs().amax(-1).float()
    sf = (torch.div(per_block, torch.full_like(per_block, 6.0)) * enc).to(torch.float8_e4m3fn).float()
    mul = torch.where(sf > 0, enc / sf, torch.zeros_like(sf))
    v = (b * mul[..., None].double()).float().double()
    sf, enc = sf.double(), enc.double()
    grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    i = torch.searchsorted(grid, v.abs().clamp(max=6.0), right=True).clamp(max=8) - 1
    up = (i + 1).clamp(max=7)
    d, e = v.abs().clamp(max=6.0) - grid[i], grid[up] - v.abs().clamp(max=6.0)
    i = torch.where((e < d) | ((e == d) & (i % 2 == 1)), up, i)
    return (torch.where(v < 0, -grid[i], grid[i]) * sf[..., None]).flatten(-2) / enc


def exact(c, seed):
    s = prepare(c, seed)
    op = c["op"]
    if op == "norm":
        h = s["x"] if s["r"] is None else (s["x"].double() + s["r"].double()).to(s["x"].dtype)
        rstd = (h.double().pow(2).sum(-1) / c["K"] + 1e-6).pow(-0.5)
        y = torch.einsum("mk,m,k->mk", h.double(), rstd, s["w"].double()).reshape(c["M"], -1, 128)
        scale = torch.maximum(y.abs().amax(-1), torch.tensor(1e-10, dtype=torch.float64, device=y.device)) / 448.0
        codes = (y / scale.unsqueeze(-1)).float().to(torch.float8_e4m3fn).double().reshape(c["M"], c["K"])
        out = {"codes": codes, "scales": scale.mT.contiguous() if c["transposed"] else scale, "rstd": rstd}
        return out if s["r"] is None else {**out, "h": h.double()}
    if op == "norm_back":
        dy, h, w, rstd = s["dy"].double(), s["h"].double(), s["w"].double(), s["rstd"].double()
        n = h * rstd[:, None]
        dn = dy * w
        dx = (dn - n * (dn * n).sum(-1, keepdim=True) / c["K"]) * rstd[:, None]
        return {"dx": dx if s["dres"] is None else dx + s["dres"].double(), "dw": torch.einsum("mk,mk->k", dy, n)}
    if op == "rope":
        z = torch.polar(torch.full((), s["mag"], dtype=torch.float64, device="cuda"), s["pos"].double()[:, None] * s["inv"])
        z = (z.conj() if c["inverse"] else z)[:, None]
        got = []
        for x in (s["q"], s["k"]):
            y = x.double().clone()
            part = y[..., c["offset"]:c["offset"] + c["R"]]
            pairs = part.reshape(*part.shape[:2], -1, 2) if c["interleaved"] else part.reshape(*part.shape[:2], 2, -1).mT
            turned = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * z)
            part.copy_(turned.reshape(part.shape) if c["interleaved"] else turned.mT.reshape(part.shape))
            got.append(y)
        return tuple(got)
    if op == "slots":
        return None
    if op == "cache":
        return [_exact_vectors(s["k"], c["rotate"]), _exact_vectors(s["v"], c["rotate"])]
    n, q = _lens(c)
    H, P = c["Hkv"], c["page"]
    grid = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device="cuda")
    kc, vc, ka, va = (a.cuda() for a in _addresses("cpu"))
    outs, lses, at = [], [], 0
    for b in range(c["B"]):
        if q[b] == 0:
            continue
        groups = s["cache"][s["table"][b, : -(-n[b] // P)].long()].transpose(0, 1).reshape(H, -1, GROUP_BYTES)

        def vectors(codes, scales, first):
            by = groups[..., codes].long()
            y = torch.stack((grid[by & 15], grid[by >> 4]), -1).reshape(H, -1, 16, 8, 16)
            y = y * groups[..., scales].contiguous().view(torch.float8_e4m3fn).double()[..., None]
            d = groups[..., first:first + 64].contiguous().view(torch.float32).double()
            return (y * d[..., None, None]).reshape(H, -1, HEAD)[:, : n[b]]

        k, v = vectors(kc, ka, 2304), vectors(vc, va, 2368)
        x = s["q"][at:at + q[b]].double()
        x = (x @ _h128() if c["rotate"] else x).reshape(q[b], H, -1, HEAD)
        dots = torch.einsum("qhgd,htd->qhgt", x, k) * HEAD ** -0.5
        t = torch.arange(n[b], device="cuda")[None, :]
        p = torch.arange(n[b] - q[b], n[b], device="cuda")[:, None]
        hide = t > p
        if c["window"]:
            hide |= (p - t >= c["window"]) & (t >= c["sinks"])
        dots = dots.masked_fill(hide[:, None, None, :], -math.inf)
        lses.append(torch.logsumexp(dots, -1).reshape(q[b], -1))
        o = torch.einsum("qhgt,htd->qhgd", torch.softmax(dots, -1), v).reshape(q[b], -1, HEAD)
        outs.append(o @ _h128() if c["rotate"] else o)
        at += q[b]
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
