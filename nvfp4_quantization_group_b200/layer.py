"""The attention layer around the quantizers: residual + RMS norm with FP8 codes, rotary positions, slot maps, the NVFP4
key/value cache and attention over it (the second half of include/hq.h).

``hq_*`` functions take caller-allocated tensors like the C calls; the others check types, shapes, strides and devices,
allocate what they return and call them.  Tensors may lie on any CUDA device (all of one call on the same); the work
goes to that device's current stream, or to `stream`.  With `stream` the outputs are allocated on it and the inputs
recorded on it, so that they may be dropped as soon as the call returns.  A refused call raises HQError, as in the rest
of the package.
"""
from __future__ import annotations

import ctypes

import torch

from . import (HQ_ERR_ALIGN, HQ_ERR_NULL, HQ_ERR_SHAPE, HQ_ERR_UNSUPPORTED, HQ_FP8_UE8M0, HQ_SCALE_ROWMAJOR,
               HQ_SCALE_TRANSPOSED, HQError, _check, _p, _stream, hq_workspace_init, lib)

HQ_DT_BF16, HQ_DT_F16, HQ_DT_F32 = 0, 1, 2
HQ_ROPE_HALVES, HQ_ROPE_INTERLEAVED = 0, 1
HQ_ROPE_PLAIN, HQ_ROPE_LINEAR, HQ_ROPE_NTK, HQ_ROPE_PARTS, HQ_ROPE_BANDS = range(5)
HQ_NORM_MAX_K = 65536
HQ_KV_MAX_REQUESTS = 4096
HQ_KV_NO_PAGES, HQ_KV_NO_ROWS, HQ_KV_NO_WIDTH, HQ_KV_BAD_STATE = 1, 2, 4, 8
HQ_KV4_HEAD, HQ_KV4_GROUP_TOKENS, HQ_KV4_GROUP_BYTES = 128, 16, 2432

_DTYPE = {torch.bfloat16: HQ_DT_BF16, torch.float16: HQ_DT_F16, torch.float32: HQ_DT_F32}

_P, _I64, _SZ, _INT, _F, _D = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int, ctypes.c_float,
                               ctypes.c_double)
# name: (result, arguments)
SIGNATURES = {
    "hq_add_rmsnorm_fp8_k128": (_INT, [_INT, _P, _I64, _P, _I64, _P, _INT, _F, _I64, _I64, _P, _P, _P, _INT, _I64, _P,
                                       _P, _P]),
    "hq_rmsnorm_backward_workspace_size": (_SZ, [_I64, _I64]),
    "hq_rmsnorm_backward": (_INT, [_INT, _P, _I64, _P, _I64, _P, _INT, _P, _P, _I64, _I64, _I64, _P, _P, _P, _SZ, _P]),
    "hq_rope_inv_freq": (_INT, [_INT, _D, _INT, _D, _D, _D, _D, _P, _P]),
    "hq_rope": (_INT, [_INT, _P, _I64, _I64, _INT, _P, _I64, _I64, _INT, _I64, _INT, _P, _P, _INT, _INT, _INT, _F, _INT,
                       _P, _I64, _I64, _P, _I64, _I64, _P]),
    "hq_kv_slots": (_INT, [_INT, _P, _P, _P, _I64, _P, _I64, _P, _INT, _I64, _P, _P, _P, _P, _P, _P, _P]),
    "hq_kv4_cache_bytes": (_SZ, [_I64, _INT, _INT]),
    "hq_kv4_append": (_INT, [_INT, _P, _I64, _I64, _P, _I64, _I64, _P, _I64, _INT, _INT, _P, _I64, _INT, _P]),
    "hq_kv4_gather": (_INT, [_INT, _P, _I64, _INT, _P, _I64, _INT, _INT, _P, _I64, _I64, _P, _I64, _I64, _P]),
    "hq_kv4_attention_workspace_size": (_SZ, []),
    "hq_kv4_attention": (_INT, [_INT, _P, _I64, _I64, _I64, _INT, _P, _I64, _INT, _INT, _P, _I64, _INT, _P, _P, _INT, _F,
                                _INT, _INT, _INT, _P, _I64, _I64, _P, _P, _SZ, _P]),
}


def _need(ok: bool, status: int, what: str) -> None:
    if not ok:
        raise HQError(status, what)


def _same_device(what: str, first: torch.Tensor, *others) -> torch.device:
    _need(first.is_cuda, HQ_ERR_UNSUPPORTED, what + ": a CUDA tensor is needed")
    for t in others:
        _need(t is None or t.device == first.device, HQ_ERR_UNSUPPORTED, what + ": tensors on different devices")
    return first.device


def _launch(device: torch.device, stream, inputs, call):
    """call(stream handle) with `device` current, allocations on the stream that the work goes to."""
    if stream is None:
        if device.index == torch.cuda.current_device():
            return call(torch.cuda.current_stream(device).cuda_stream)
        with torch.cuda.device(device):
            return call(torch.cuda.current_stream(device).cuda_stream)
    s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream), device)
    with torch.cuda.device(device), torch.cuda.stream(s):
        for t in inputs:
            if t is not None:
                t.record_stream(s)
        return call(s.cuda_stream)


# ------------------------------------------------------------------- norm
def hq_add_rmsnorm_fp8_k128(dtype, x, x_row_stride, residual, residual_row_stride, weight, w_dtype, eps, M, K,
                            residual_out, out_fp8, scales, scale_layout, scale_ld, rstd_opt=None, amax_opt=None,
                            stream=None) -> None:
    _check(lib().hq_add_rmsnorm_fp8_k128(int(dtype), _p(x), int(x_row_stride), _p(residual), int(residual_row_stride),
                                         _p(weight), int(w_dtype), float(eps), int(M), int(K), _p(residual_out),
                                         _p(out_fp8), _p(scales), int(scale_layout), int(scale_ld), _p(rstd_opt),
                                         _p(amax_opt), _stream(stream)), "hq_add_rmsnorm_fp8_k128")


def hq_rmsnorm_backward_workspace_size(M: int, K: int) -> int:
    return int(lib().hq_rmsnorm_backward_workspace_size(int(M), int(K)))


def hq_rmsnorm_backward(dtype, dy, dy_row_stride, h, h_row_stride, weight, w_dtype, rstd, dres, dres_row_stride, M, K,
                        dx, dweight, ws, stream=None) -> None:
    _check(lib().hq_rmsnorm_backward(int(dtype), _p(dy), int(dy_row_stride), _p(h), int(h_row_stride), _p(weight),
                                     int(w_dtype), _p(rstd), _p(dres), int(dres_row_stride), int(M), int(K), _p(dx),
                                     _p(dweight), _p(ws), 0 if ws is None else ws.numel() * ws.element_size(),
                                     _stream(stream)), "hq_rmsnorm_backward")


def _rows(what: str, name: str, t: torch.Tensor, like: torch.Tensor) -> int:
    """Row stride of a [M, K] tensor of `like`'s type and shape with contiguous rows."""
    _need(t.shape == like.shape, HQ_ERR_SHAPE, f"{what}: {name}'s shape")
    _need(t.dtype == like.dtype, HQ_ERR_UNSUPPORTED, f"{what}: {name}'s type")
    _need(t.stride(1) == 1, HQ_ERR_ALIGN, f"{what}: {name}'s rows are not contiguous")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _weight(what: str, w: torch.Tensor, x: torch.Tensor) -> int:
    _need(w.shape == (x.shape[1],) and w.is_contiguous(), HQ_ERR_SHAPE, what + ": weight's shape")
    _need(w.dtype == x.dtype or w.dtype == torch.float32, HQ_ERR_UNSUPPORTED, what + ": weight's type")
    return _DTYPE[w.dtype]


def add_rmsnorm_fp8_k128(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, eps: float = 1e-6,
                         scale_layout: int = HQ_SCALE_ROWMAJOR, scale_ld: int | None = None, want_rstd: bool = False,
                         want_amax: bool = False, residual_out: torch.Tensor | None = None, stream=None) -> dict:
    """Residual addition, RMS norm and K128 FP8 codes of [M, K] rows (see hq.h) -> dict with codes [M, K], scales,
    residual_out (with a residual: what the norm read; into `residual_out` where given, which may be x or residual
    itself) and, when asked, rstd [M] and amax."""
    what = "add_rmsnorm_fp8_k128"
    _need(x.dim() == 2, HQ_ERR_SHAPE, what + ": x is [M, K]")
    _need(x.dtype in _DTYPE, HQ_ERR_UNSUPPORTED, what + ": x's type")
    dev = _same_device(what, x, weight, residual, residual_out)
    M, K = x.shape
    xs, rs = _rows(what, "x", x, x), 0 if residual is None else _rows(what, "residual", residual, x)
    wd = _weight(what, weight, x)
    if residual_out is not None:
        _need(residual is not None, HQ_ERR_NULL, what + ": residual_out without a residual")
        _rows(what, "residual_out", residual_out, x)
        _need(residual_out.is_contiguous(), HQ_ERR_ALIGN, what + ": residual_out is not contiguous")
    groups = K // 128

    def call(s):
        out = {"codes": torch.empty((M, K), dtype=torch.uint8, device=dev)}
        if (scale_layout & ~HQ_FP8_UE8M0) == HQ_SCALE_TRANSPOSED:
            ld = M if scale_ld is None else scale_ld
            out["scales"] = torch.empty((groups, ld), dtype=torch.float32, device=dev)
        else:
            ld = groups
            out["scales"] = torch.empty((M, groups), dtype=torch.float32, device=dev)
        if residual is not None:
            out["residual_out"] = torch.empty((M, K), dtype=x.dtype, device=dev) if residual_out is None else residual_out
        if want_rstd:
            out["rstd"] = torch.empty(M, dtype=torch.float32, device=dev)
        if want_amax:
            out["amax"] = torch.empty_like(out["scales"])
        hq_add_rmsnorm_fp8_k128(_DTYPE[x.dtype], x, xs, residual, rs, weight, wd, eps, M, K, out.get("residual_out"),
                                out["codes"], out["scales"], scale_layout, ld, out.get("rstd"), out.get("amax"), s)
        return out

    return _launch(dev, stream, (x, weight, residual, residual_out), call)


def rmsnorm_backward_workspace(M: int, K: int, device="cuda") -> torch.Tensor:
    """Workspace of rmsnorm_backward for [M, K]; any contents."""
    nbytes = hq_rmsnorm_backward_workspace_size(M, K)
    _need(nbytes > 0, HQ_ERR_SHAPE, "rmsnorm_backward_workspace")
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def rmsnorm_backward(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                     dres: torch.Tensor | None = None, want_dweight: bool = True, ws: torch.Tensor | None = None,
                     dx: torch.Tensor | None = None, stream=None):
    """Gradients of the norm (see hq.h): dy the gradient of the normalized rows, h what the norm read (residual_out, or x
    without a residual), dres the gradient that reaches h along the residual -> (dx [M, K], dweight FP32 [K] or None).
    dx is written into `dx` where given (it may be dy or dres itself)."""
    what = "rmsnorm_backward"
    _need(dy.dim() == 2, HQ_ERR_SHAPE, what + ": dy is [M, K]")
    _need(dy.dtype in _DTYPE, HQ_ERR_UNSUPPORTED, what + ": dy's type")
    dev = _same_device(what, dy, h, weight, rstd, dres, ws, dx)
    M, K = dy.shape
    gs, hs = _rows(what, "dy", dy, dy), _rows(what, "h", h, dy)
    rs = 0 if dres is None else _rows(what, "dres", dres, dy)
    wd = _weight(what, weight, dy)
    _need(rstd.shape == (M,) and rstd.is_contiguous(), HQ_ERR_SHAPE, what + ": rstd's shape")
    _need(rstd.dtype == torch.float32, HQ_ERR_UNSUPPORTED, what + ": rstd's type")
    if dx is not None:
        _rows(what, "dx", dx, dy)
        _need(dx.is_contiguous(), HQ_ERR_ALIGN, what + ": dx is not contiguous")

    def call(s):
        out = torch.empty((M, K), dtype=dy.dtype, device=dev) if dx is None else dx
        dw = torch.empty(K, dtype=torch.float32, device=dev) if want_dweight else None
        w = rmsnorm_backward_workspace(M, K, dev) if want_dweight and ws is None else ws
        hq_rmsnorm_backward(_DTYPE[dy.dtype], dy, gs, h, hs, weight, wd, rstd, dres, rs, M, K, out, dw, w, s)
        return out, dw

    return _launch(dev, stream, (dy, h, weight, rstd, dres, ws, dx), call)


# ------------------------------------------------------------------- rope
def hq_rope_inv_freq(rotary_dim, base, scaling, factor, trained_len, p1, p2, inv_freq, magnitude) -> None:
    _check(lib().hq_rope_inv_freq(int(rotary_dim), float(base), int(scaling), float(factor), float(trained_len),
                                  float(p1), float(p2), inv_freq, magnitude), "hq_rope_inv_freq")


def hq_rope(dtype, q, q_token_stride, q_head_stride, Hq, k, k_token_stride, k_head_stride, Hk, T, D, positions, inv_freq,
            rotary_dim, offset, layout, magnitude, inverse, q_out, q_out_token_stride, q_out_head_stride, k_out,
            k_out_token_stride, k_out_head_stride, stream=None) -> None:
    _check(lib().hq_rope(int(dtype), _p(q), int(q_token_stride), int(q_head_stride), int(Hq), _p(k), int(k_token_stride),
                         int(k_head_stride), int(Hk), int(T), int(D), _p(positions), _p(inv_freq), int(rotary_dim),
                         int(offset), int(layout), float(magnitude), int(inverse), _p(q_out), int(q_out_token_stride),
                         int(q_out_head_stride), _p(k_out), int(k_out_token_stride), int(k_out_head_stride),
                         _stream(stream)), "hq_rope")


def rope_inv_freq(rotary_dim: int, base: float = 10000.0, scaling: int = HQ_ROPE_PLAIN, factor: float = 1.0,
                  trained_len: float = 0.0, p1: float | None = None, p2: float | None = None, device="cuda"):
    """Rotary frequencies (see hq.h) -> (float64 [rotary_dim / 2] on `device`, magnitude).  p1, p2: turns 32 and 1 for
    HQ_ROPE_PARTS, 1 and 4 for HQ_ROPE_BANDS unless given."""
    d1, d2 = (1.0, 4.0) if scaling == HQ_ROPE_BANDS else (32.0, 1.0)
    host = (ctypes.c_double * max(1, int(rotary_dim) // 2))()
    mag = ctypes.c_double(1.0)
    hq_rope_inv_freq(rotary_dim, base, scaling, factor, trained_len, d1 if p1 is None else p1, d2 if p2 is None else p2,
                     ctypes.cast(host, _P), ctypes.cast(ctypes.byref(mag), _P))
    return torch.tensor(list(host), dtype=torch.float64, device=device), mag.value


def rope(q: torch.Tensor, k: torch.Tensor | None, positions: torch.Tensor, inv_freq: torch.Tensor, offset: int = 0,
         layout: int = HQ_ROPE_HALVES, magnitude: float = 1.0, inverse: bool = False, q_out: torch.Tensor | None = None,
         k_out: torch.Tensor | None = None, stream=None):
    """Rotary positions (see hq.h) of q [T, Hq, D] and k [T, Hk, D] (or None) -> (q_out, k_out), contiguous new tensors
    unless given (q and k themselves: in place).  The rotated part is 2 * len(inv_freq) wide, from dimension `offset`;
    inverse=True is the gradient with respect to the inputs."""
    what = "rope"
    _need(q.dim() == 3, HQ_ERR_SHAPE, what + ": q is [T, heads, D]")
    _need(q.dtype in _DTYPE, HQ_ERR_UNSUPPORTED, what + ": q's type")
    dev = _same_device(what, q, k, positions, inv_freq, q_out, k_out)
    T, Hq, D = q.shape
    for name, t, like in (("q", q, q), ("k", k, None if k is None else k), ("q_out", q_out, q), ("k_out", k_out, k)):
        if t is None:
            continue
        _need(like is not None and t.shape == like.shape and t.dim() == 3 and t.shape[0] == T and t.shape[2] == D,
              HQ_ERR_SHAPE, f"{what}: {name}'s shape")
        _need(t.dtype == q.dtype, HQ_ERR_UNSUPPORTED, f"{what}: {name}'s type")
        _need(D <= 1 or t.stride(2) == 1, HQ_ERR_ALIGN, f"{what}: {name}'s rows are not contiguous")
    _need(positions.shape == (T,) and positions.is_contiguous(), HQ_ERR_SHAPE, what + ": positions' shape")
    _need(positions.dtype == torch.int64, HQ_ERR_UNSUPPORTED, what + ": positions' type")
    _need(inv_freq.dim() == 1 and inv_freq.is_contiguous(), HQ_ERR_SHAPE, what + ": inv_freq's shape")
    _need(inv_freq.dtype == torch.float64, HQ_ERR_UNSUPPORTED, what + ": inv_freq's type")
    Hk = 0 if k is None else k.shape[1]

    def call(s):
        qo = torch.empty((T, Hq, D), dtype=q.dtype, device=dev) if q_out is None else q_out
        ko = k_out
        if k is not None and ko is None:
            ko = torch.empty((T, Hk, D), dtype=q.dtype, device=dev)
        ks, kos = (0, 0) if k is None else (k.stride(0), k.stride(1)), (0, 0) if k is None else (ko.stride(0), ko.stride(1))
        hq_rope(_DTYPE[q.dtype], q, q.stride(0), q.stride(1), Hq, k, ks[0], ks[1], Hk, T, D, positions, inv_freq,
                2 * inv_freq.shape[0], offset, layout, magnitude, bool(inverse), qo, qo.stride(0), qo.stride(1), ko,
                kos[0], kos[1], s)
        return qo, ko

    return _launch(dev, stream, (q, k, positions, inv_freq, q_out, k_out), call)


# ------------------------------------------------------------ slots, cache
def hq_kv_slots(B, lens, new_tokens, block_table, table_width, free_pages, free_capacity, free_count, page_size, n_slots,
                lens_out, cu_new, slots, positions, free_count_out, status, stream=None) -> None:
    _check(lib().hq_kv_slots(int(B), _p(lens), _p(new_tokens), _p(block_table), int(table_width), _p(free_pages),
                             int(free_capacity), _p(free_count), int(page_size), int(n_slots), _p(lens_out), _p(cu_new),
                             _p(slots), _p(positions), _p(free_count_out), _p(status), _stream(stream)), "hq_kv_slots")


def kv_slots(lens: torch.Tensor, new_tokens: torch.Tensor, block_table: torch.Tensor, free_pages: torch.Tensor,
             free_count: torch.Tensor, page_size: int, n_slots: int, lens_out: torch.Tensor | None = None,
             free_count_out: torch.Tensor | None = None, stream=None) -> dict:
    """Block tables and slot maps of one step (see hq.h): block_table and free_pages are updated in place; returns a dict
    of new tensors lens, cu_new, slots, positions, free_count, status.  Pass lens_out=lens and
    free_count_out=free_count to update those in place too."""
    what = "kv_slots"
    dev = _same_device(what, lens, new_tokens, block_table, free_pages, free_count, lens_out, free_count_out)
    B = lens.shape[0] if lens.dim() == 1 else -1
    for name, t, shape in (("lens", lens, (B,)), ("new_tokens", new_tokens, (B,)), ("free_count", free_count, (1,)),
                           ("lens_out", lens_out, (B,)), ("free_count_out", free_count_out, (1,)),
                           ("free_pages", free_pages, (free_pages.numel(),)),
                           ("block_table", block_table, (B, block_table.shape[-1] if block_table.dim() else 0))):
        if t is None:
            continue
        _need(t.shape == shape and t.is_contiguous(), HQ_ERR_SHAPE, f"{what}: {name}'s shape")
        _need(t.dtype == torch.int32, HQ_ERR_UNSUPPORTED, f"{what}: {name}'s type")

    def call(s):
        i32, i64 = dict(dtype=torch.int32, device=dev), dict(dtype=torch.int64, device=dev)
        out = {"lens": torch.empty(B, **i32) if lens_out is None else lens_out, "cu_new": torch.empty(B + 1, **i32),
               "slots": torch.empty(n_slots, **i64), "positions": torch.empty(n_slots, **i64),
               "free_count": torch.empty(1, **i32) if free_count_out is None else free_count_out,
               "status": torch.empty(1, **i32)}
        hq_kv_slots(B, lens, new_tokens, block_table, block_table.shape[1], free_pages, free_pages.numel(), free_count,
                    page_size, n_slots, out["lens"], out["cu_new"], out["slots"], out["positions"], out["free_count"],
                    out["status"], s)
        return out

    return _launch(dev, stream, (lens, new_tokens, block_table, free_pages, free_count, lens_out, free_count_out), call)


def hq_kv4_cache_bytes(num_pages: int, page_size: int, H: int) -> int:
    return int(lib().hq_kv4_cache_bytes(int(num_pages), int(page_size), int(H)))


def kv4_cache(num_pages: int, page_size: int, H: int, device="cuda") -> torch.Tensor:
    """An empty NVFP4 key/value cache: uint8 [num_pages, H, page_size / 16, 2432]."""
    _need(hq_kv4_cache_bytes(num_pages, page_size, H) > 0, HQ_ERR_SHAPE, "kv4_cache")
    return torch.zeros((num_pages, H, page_size // HQ_KV4_GROUP_TOKENS, HQ_KV4_GROUP_BYTES), dtype=torch.uint8,
                       device=device)


def _cache_shape(what: str, cache: torch.Tensor):
    """(pages, page_size, heads) of a cache."""
    _need(cache.dim() == 4 and cache.shape[3] == HQ_KV4_GROUP_BYTES and cache.is_contiguous(), HQ_ERR_SHAPE,
          what + ": the cache is [pages, heads, page_size / 16, 2432], contiguous")
    _need(cache.dtype == torch.uint8, HQ_ERR_UNSUPPORTED, what + ": the cache's type")
    return cache.shape[0], cache.shape[2] * HQ_KV4_GROUP_TOKENS, cache.shape[1]


def hq_kv4_append(dtype, k, k_token_stride, k_head_stride, v, v_token_stride, v_head_stride, slots, N, H, hadamard_n,
                  cache, num_pages, page_size, stream=None) -> None:
    _check(lib().hq_kv4_append(int(dtype), _p(k), int(k_token_stride), int(k_head_stride), _p(v), int(v_token_stride),
                               int(v_head_stride), _p(slots), int(N), int(H), int(hadamard_n), _p(cache), int(num_pages),
                               int(page_size), _stream(stream)), "hq_kv4_append")


def hq_kv4_gather(dtype, cache, num_pages, page_size, slots, N, H, hadamard_n, k_out, k_token_stride, k_head_stride,
                  v_out, v_token_stride, v_head_stride, stream=None) -> None:
    _check(lib().hq_kv4_gather(int(dtype), _p(cache), int(num_pages), int(page_size), _p(slots), int(N), int(H),
                               int(hadamard_n), _p(k_out), int(k_token_stride), int(k_head_stride), _p(v_out),
                               int(v_token_stride), int(v_head_stride), _stream(stream)), "hq_kv4_gather")


def _slots_arg(what: str, slots: torch.Tensor) -> int:
    _need(slots.dim() == 1 and slots.is_contiguous(), HQ_ERR_SHAPE, what + ": slots' shape")
    _need(slots.dtype == torch.int64, HQ_ERR_UNSUPPORTED, what + ": slots' type")
    return slots.shape[0]


def kv4_append(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, cache: torch.Tensor, hadamard_n: int = 128,
               stream=None) -> None:
    """Quantize keys and values [N, H, 128] into the cache's slots (see hq.h); slots outside the cache are skipped."""
    what = "kv4_append"
    dev = _same_device(what, cache, k, v, slots)
    pages, page, H = _cache_shape(what, cache)
    N = _slots_arg(what, slots)
    for name, t in (("k", k), ("v", v)):
        _need(t.shape == (N, H, HQ_KV4_HEAD), HQ_ERR_SHAPE, f"{what}: {name}'s shape")
        _need(t.dtype == k.dtype and t.dtype in _DTYPE, HQ_ERR_UNSUPPORTED, f"{what}: {name}'s type")
        _need(t.stride(2) == 1, HQ_ERR_ALIGN, f"{what}: {name}'s rows are not contiguous")

    def call(s):
        hq_kv4_append(_DTYPE[k.dtype], k, k.stride(0), k.stride(1), v, v.stride(0), v.stride(1), slots, N, H, hadamard_n,
                      cache, pages, page, s)

    _launch(dev, stream, (k, v, slots, cache), call)


def kv4_gather(cache: torch.Tensor, slots: torch.Tensor, dtype: torch.dtype = torch.bfloat16, hadamard_n: int = 128,
               stream=None):
    """Keys and values [N, H, 128] of the cache's slots (see hq.h), rotated back with hadamard_n 128 -> (k, v)."""
    what = "kv4_gather"
    dev = _same_device(what, cache, slots)
    pages, page, H = _cache_shape(what, cache)
    N = _slots_arg(what, slots)
    _need(dtype in _DTYPE, HQ_ERR_UNSUPPORTED, what + ": dtype")

    def call(s):
        k = torch.empty((N, H, HQ_KV4_HEAD), dtype=dtype, device=dev)
        v = torch.empty_like(k)
        hq_kv4_gather(_DTYPE[dtype], cache, pages, page, slots, N, H, hadamard_n, k, k.stride(0), k.stride(1), v,
                      v.stride(0), v.stride(1), s)
        return k, v

    return _launch(dev, stream, (cache, slots), call)


# -------------------------------------------------------------- attention
def hq_kv4_attention_workspace_size() -> int:
    return int(lib().hq_kv4_attention_workspace_size())


def hq_kv4_attention(dtype, q, q_token_stride, q_head_stride, Tq, Hq, cache, num_pages, page_size, Hkv, block_table,
                     table_width, B, seq_lens, cu_q, q_len, scale, window, sinks, hadamard_n, out, out_token_stride,
                     out_head_stride, lse_opt, ws, stream=None) -> None:
    _check(lib().hq_kv4_attention(int(dtype), _p(q), int(q_token_stride), int(q_head_stride), int(Tq), int(Hq), _p(cache),
                                  int(num_pages), int(page_size), int(Hkv), _p(block_table), int(table_width), int(B),
                                  _p(seq_lens), _p(cu_q), int(q_len), float(scale), int(window), int(sinks),
                                  int(hadamard_n), _p(out), int(out_token_stride), int(out_head_stride), _p(lse_opt),
                                  _p(ws), 0 if ws is None else ws.numel() * ws.element_size(), _stream(stream)),
           "hq_kv4_attention")


def kv4_attention_workspace(device="cuda", stream=None) -> torch.Tensor:
    """A workspace of kv4_attention in its rest state; for any shapes, one call at a time."""
    ws = torch.empty(hq_kv4_attention_workspace_size(), dtype=torch.uint8, device=device)
    _launch(ws.device, stream, (ws,), lambda s: hq_workspace_init(ws, s))
    return ws


def kv4_attention(q: torch.Tensor, cache: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                  cu_q: torch.Tensor | None = None, q_len: int = 1, scale: float | None = None, window: int = 0,
                  sinks: int = 0, hadamard_n: int = 128, ws: torch.Tensor | None = None, out: torch.Tensor | None = None,
                  want_lse: bool = False, stream=None):
    """Attention of q [Tq, Hq, 128], the newest tokens of each request, over the cache (see hq.h) -> out, or (out, lse
    [Tq, Hq]) with want_lse.  Rows behind the last request's are left as they were (uninitialized in a new tensor).
    scale: 1 / sqrt(128) unless given."""
    what = "kv4_attention"
    dev = _same_device(what, q, cache, block_table, seq_lens, cu_q, ws, out)
    pages, page, Hkv = _cache_shape(what, cache)
    _need(q.dim() == 3 and q.shape[2] == HQ_KV4_HEAD, HQ_ERR_SHAPE, what + ": q is [Tq, heads, 128]")
    _need(q.dtype in (torch.bfloat16, torch.float16), HQ_ERR_UNSUPPORTED, what + ": q's type")
    _need(q.stride(2) == 1, HQ_ERR_ALIGN, what + ": q's rows are not contiguous")
    Tq, Hq, _ = q.shape
    B = seq_lens.shape[0] if seq_lens.dim() == 1 else -1
    _need(block_table.dim() == 2 and block_table.shape[0] == B and block_table.is_contiguous(), HQ_ERR_SHAPE,
          what + ": block_table's shape")
    for name, t, n in (("seq_lens", seq_lens, B), ("cu_q", cu_q, B + 1)):
        if t is not None:
            _need(t.shape == (n,) and t.is_contiguous(), HQ_ERR_SHAPE, f"{what}: {name}'s shape")
            _need(t.dtype == torch.int32, HQ_ERR_UNSUPPORTED, f"{what}: {name}'s type")
    _need(block_table.dtype == torch.int32, HQ_ERR_UNSUPPORTED, what + ": block_table's type")
    if out is not None:
        _need(out.shape == q.shape, HQ_ERR_SHAPE, what + ": out's shape")
        _need(out.dtype == q.dtype, HQ_ERR_UNSUPPORTED, what + ": out's type")
        _need(out.stride(2) == 1, HQ_ERR_ALIGN, what + ": out's rows are not contiguous")

    def call(s):
        o = torch.empty((Tq, Hq, HQ_KV4_HEAD), dtype=q.dtype, device=dev) if out is None else out
        lse = torch.empty((Tq, Hq), dtype=torch.float32, device=dev) if want_lse else None
        w = kv4_attention_workspace(dev) if ws is None else ws
        hq_kv4_attention(_DTYPE[q.dtype], q, q.stride(0), q.stride(1), Tq, Hq, cache, pages, page, Hkv, block_table,
                         block_table.shape[1], B, seq_lens, cu_q, q_len, HQ_KV4_HEAD ** -0.5 if scale is None else scale,
                         window, sinks, hadamard_n, o, o.stride(0), o.stride(1), lse, w, s)
        return (o, lse) if want_lse else o

    return _launch(dev, stream, (q, cache, block_table, seq_lens, cu_q, ws, out), call)


__all__ = [n for n in dir() if n.startswith(("HQ_DT_", "HQ_ROPE_", "HQ_NORM_", "HQ_KV", "hq_add_", "hq_rms", "hq_rope",
                                              "hq_kv"))]
__all__ += ["add_rmsnorm_fp8_k128", "rmsnorm_backward", "rmsnorm_backward_workspace", "rope", "rope_inv_freq", "kv_slots",
            "kv4_cache", "kv4_append", "kv4_gather", "kv4_attention", "kv4_attention_workspace"]
