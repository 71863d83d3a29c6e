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


def _need(ok: bool, status: int, *what: str) -> None:
    if not ok:
        raise HQError(status, ": ".join(what))


# handle of a device's current stream (the direct call saves a microsecond of building a Stream object)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda d: torch.cuda.current_stream(d).cuda_stream)


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _vector(what: str, name: str, t: torch.Tensor, n: int, dtype) -> None:
    """Refuses anything but a contiguous [n] tensor of the type."""
    if t.dtype == dtype and t.dim() == 1 and t.shape[0] == n and t.is_contiguous():
        return
    raise HQError(HQ_ERR_UNSUPPORTED if t.dtype != dtype else HQ_ERR_SHAPE, f"{what}: {name}'s type or shape")


def _table(what: str, t: torch.Tensor, B: int) -> int:
    """Width of a contiguous int32 [B, width] block table."""
    if t.dtype == torch.int32 and t.dim() == 2 and t.shape[0] == B and t.is_contiguous():
        return t.shape[1]
    raise HQError(HQ_ERR_UNSUPPORTED if t.dtype != torch.int32 else HQ_ERR_SHAPE, f"{what}: block_table's type or shape")


def _device(what: str, first: torch.Tensor, *others) -> int:
    """Index of the CUDA device that all tensors are on."""
    d = first.get_device()
    if d < 0:
        raise HQError(HQ_ERR_UNSUPPORTED, what + ": a CUDA tensor is needed")
    for t in others:
        if t is not None and t.get_device() != d:
            raise HQError(HQ_ERR_UNSUPPORTED, what + ": tensors on different devices")
    return d


def _launch(device: int, stream, inputs, call):
    """call(stream handle) with `device` current, allocations on the stream that the work goes to."""
    if stream is None:
        if device == torch.cuda.current_device():
            return call(_raw_stream(device))
        with torch.cuda.device(device):
            return call(_raw_stream(device))
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


def _rows(what: str, name: str, t: torch.Tensor, shape, dtype) -> int:
    """Row stride of a tensor of the given [M, K] and type with contiguous rows."""
    if t.shape != shape or t.dtype != dtype:
        raise HQError(HQ_ERR_SHAPE if t.dtype == dtype else HQ_ERR_UNSUPPORTED, f"{what}: {name}'s type or shape")
    row, one = t.stride()
    if one != 1:
        raise HQError(HQ_ERR_ALIGN, f"{what}: {name}'s rows are not contiguous")
    return row if shape[0] > 1 else shape[1]


def _weight(what: str, w: torch.Tensor, K: int, dtype) -> int:
    _vector(what, "weight", w, K, dtype if w.dtype == dtype else torch.float32)
    return _DTYPE[w.dtype]


def add_rmsnorm_fp8_k128(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, eps: float = 1e-6,
                         scale_layout: int = HQ_SCALE_ROWMAJOR, scale_ld: int | None = None, want_rstd: bool = False,
                         want_amax: bool = False, residual_out: torch.Tensor | None = None, stream=None) -> dict:
    """Residual addition, RMS norm and K128 FP8 codes of [M, K] rows (see hq.h) -> dict with codes [M, K], scales,
    residual_out (with a residual: what the norm read; into `residual_out` where given, which may be x or residual
    itself) and, when asked, rstd [M] and amax."""
    what = "add_rmsnorm_fp8_k128"
    shape, dtype = x.shape, x.dtype
    if len(shape) != 2 or dtype not in _DTYPE:
        raise HQError(HQ_ERR_SHAPE if dtype in _DTYPE else HQ_ERR_UNSUPPORTED, what + ": x is [M, K]")
    dev = _device(what, x, weight, residual, residual_out)
    M, K = shape
    xs, rs = _rows(what, "x", x, shape, dtype), 0 if residual is None else _rows(what, "residual", residual, shape, dtype)
    wd = _weight(what, weight, K, dtype)
    if residual_out is not None:
        _need(residual is not None, HQ_ERR_NULL, what, "residual_out without a residual")
        _rows(what, "residual_out", residual_out, shape, dtype)
        _need(residual_out.is_contiguous(), HQ_ERR_ALIGN, what, "residual_out is not contiguous")
    groups = K // 128

    def call(s):
        out = {"codes": x.new_empty(shape, dtype=torch.uint8)}
        if (scale_layout & ~HQ_FP8_UE8M0) == HQ_SCALE_TRANSPOSED:
            ld = M if scale_ld is None else scale_ld
            scales = x.new_empty((groups, ld), dtype=torch.float32)
        else:
            ld = groups
            scales = x.new_empty((M, groups), dtype=torch.float32)
        out["scales"] = scales
        if residual is not None:
            out["residual_out"] = x.new_empty(shape) if residual_out is None else residual_out
        if want_rstd:
            out["rstd"] = x.new_empty((M,), dtype=torch.float32)
        if want_amax:
            out["amax"] = torch.empty_like(scales)
        _check(lib().hq_add_rmsnorm_fp8_k128(
            _DTYPE[dtype], x.data_ptr(), xs, _ptr(residual), rs, weight.data_ptr(), wd, eps, M, K,
            _ptr(out.get("residual_out")), out["codes"].data_ptr(), scales.data_ptr(), scale_layout, ld,
            _ptr(out.get("rstd")), _ptr(out.get("amax")), s), what)
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
    shape, dtype = dy.shape, dy.dtype
    if len(shape) != 2 or dtype not in _DTYPE:
        raise HQError(HQ_ERR_SHAPE if dtype in _DTYPE else HQ_ERR_UNSUPPORTED, what + ": dy is [M, K]")
    dev = _device(what, dy, h, weight, rstd, dres, ws, dx)
    M, K = shape
    gs, hs = _rows(what, "dy", dy, shape, dtype), _rows(what, "h", h, shape, dtype)
    rs = 0 if dres is None else _rows(what, "dres", dres, shape, dtype)
    wd = _weight(what, weight, K, dtype)
    _vector(what, "rstd", rstd, M, torch.float32)
    if dx is not None:
        _rows(what, "dx", dx, shape, dtype)
        _need(dx.is_contiguous(), HQ_ERR_ALIGN, what, "dx is not contiguous")

    def call(s):
        out = dy.new_empty(shape) if dx is None else dx
        dw = dy.new_empty((K,), dtype=torch.float32) if want_dweight else None
        w = rmsnorm_backward_workspace(M, K, dy.device) if want_dweight and ws is None else ws
        _check(lib().hq_rmsnorm_backward(
            _DTYPE[dtype], dy.data_ptr(), gs, h.data_ptr(), hs, weight.data_ptr(), wd, rstd.data_ptr(), _ptr(dres), rs, M,
            K, out.data_ptr(), _ptr(dw), _ptr(w), 0 if w is None else w.nbytes, s), what)
        return out, dw

    return _launch(dev, stream, (dy, h, weight, rstd, dres, ws, dx), call)


def _heads(what: str, name: str, t: torch.Tensor, shape, dtype):
    """Token and head strides of a [T, heads, D] tensor of the given shape and type with contiguous rows."""
    if t.shape != shape or t.dtype != dtype:
        raise HQError(HQ_ERR_SHAPE if t.dtype == dtype else HQ_ERR_UNSUPPORTED, f"{what}: {name}'s type or shape")
    token, head, one = t.stride()
    if one != 1 and shape[2] > 1:
        raise HQError(HQ_ERR_ALIGN, f"{what}: {name}'s rows are not contiguous")
    return token, head


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
    shape, dtype = q.shape, q.dtype
    if len(shape) != 3 or dtype not in _DTYPE:
        raise HQError(HQ_ERR_SHAPE if dtype in _DTYPE else HQ_ERR_UNSUPPORTED, what + ": q is [T, heads, D]")
    dev = _device(what, q, k, positions, inv_freq, q_out, k_out)
    T, Hq, D = shape
    qs = _heads(what, "q", q, shape, dtype)
    kshape, ks, Hk = None, (0, 0), 0
    if k is not None:
        kshape = k.shape
        if len(kshape) != 3 or kshape[0] != T or kshape[2] != D:
            raise HQError(HQ_ERR_SHAPE, what + ": k's shape")
        ks, Hk = _heads(what, "k", k, kshape, dtype), kshape[1]
    elif k_out is not None:
        raise HQError(HQ_ERR_SHAPE, what + ": k_out without k")
    _vector(what, "positions", positions, T, torch.int64)
    half = inv_freq.shape[0] if inv_freq.dim() == 1 else -1
    _vector(what, "inv_freq", inv_freq, half, torch.float64)
    qos = (Hq * D, D) if q_out is None else _heads(what, "q_out", q_out, shape, dtype)
    kos = (Hk * D, D) if k_out is None else _heads(what, "k_out", k_out, kshape, dtype)

    def call(s):
        qo = q.new_empty(shape) if q_out is None else q_out
        ko = k.new_empty(kshape) if k is not None and k_out is None else k_out
        _check(lib().hq_rope(_DTYPE[dtype], q.data_ptr(), qs[0], qs[1], Hq, _ptr(k), ks[0], ks[1], Hk, T, D,
                             positions.data_ptr(), inv_freq.data_ptr(), 2 * half, offset, layout, magnitude,
                             1 if inverse else 0, qo.data_ptr(), qos[0], qos[1], _ptr(ko), kos[0], kos[1], s), what)
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
    dev = _device(what, lens, new_tokens, block_table, free_pages, free_count, lens_out, free_count_out)
    B = lens.shape[0] if lens.dim() == 1 else -1
    i32 = torch.int32
    _vector(what, "lens", lens, B, i32)
    _vector(what, "new_tokens", new_tokens, B, i32)
    width = _table(what, block_table, B)
    capacity = free_pages.numel()
    _vector(what, "free_pages", free_pages, capacity, i32)
    _vector(what, "free_count", free_count, 1, i32)
    if lens_out is not None:
        _vector(what, "lens_out", lens_out, B, i32)
    if free_count_out is not None:
        _vector(what, "free_count_out", free_count_out, 1, i32)
    _need(n_slots >= 0, HQ_ERR_SHAPE, what, "n_slots")

    def call(s):
        lo = torch.empty_like(lens) if lens_out is None else lens_out
        count = torch.empty_like(free_count) if free_count_out is None else free_count_out
        cu, status = lens.new_empty((B + 1,)), torch.empty_like(free_count)
        slots = lens.new_empty((n_slots,), dtype=torch.int64)
        positions = torch.empty_like(slots)
        _check(lib().hq_kv_slots(B, lens.data_ptr(), new_tokens.data_ptr(), block_table.data_ptr(), width,
                                 free_pages.data_ptr(), capacity, free_count.data_ptr(), page_size, n_slots,
                                 lo.data_ptr(), cu.data_ptr(), slots.data_ptr(), positions.data_ptr(), count.data_ptr(),
                                 status.data_ptr(), s), what)
        return {"lens": lo, "cu_new": cu, "slots": slots, "positions": positions, "free_count": count, "status": status}

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
    shape = cache.shape
    if len(shape) != 4 or shape[3] != HQ_KV4_GROUP_BYTES or cache.dtype != torch.uint8 or not cache.is_contiguous():
        raise HQError(HQ_ERR_SHAPE if cache.dtype == torch.uint8 else HQ_ERR_UNSUPPORTED,
                      what + ": the cache is uint8 [pages, heads, page_size / 16, 2432], contiguous")
    return shape[0], shape[2] * HQ_KV4_GROUP_TOKENS, shape[1]


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
    n = slots.numel()
    _vector(what, "slots", slots, n, torch.int64)
    return n


def kv4_append(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, cache: torch.Tensor, hadamard_n: int = 128,
               stream=None) -> None:
    """Quantize keys and values [N, H, 128] into the cache's slots (see hq.h); slots outside the cache are skipped."""
    what = "kv4_append"
    dev = _device(what, cache, k, v, slots)
    pages, page, H = _cache_shape(what, cache)
    N, dtype = _slots_arg(what, slots), k.dtype
    _need(dtype in _DTYPE, HQ_ERR_UNSUPPORTED, what, "k's type")
    shape = (N, H, HQ_KV4_HEAD)
    (kt, kh), (vt, vh) = _heads(what, "k", k, shape, dtype), _heads(what, "v", v, shape, dtype)

    def call(s):
        _check(lib().hq_kv4_append(_DTYPE[dtype], k.data_ptr(), kt, kh, v.data_ptr(), vt, vh, slots.data_ptr(), N, H,
                                   hadamard_n, cache.data_ptr(), pages, page, s), what)

    _launch(dev, stream, (k, v, slots, cache), call)


def kv4_gather(cache: torch.Tensor, slots: torch.Tensor, dtype: torch.dtype = torch.bfloat16, hadamard_n: int = 128,
               stream=None):
    """Keys and values [N, H, 128] of the cache's slots (see hq.h), rotated back with hadamard_n 128 -> (k, v)."""
    what = "kv4_gather"
    dev = _device(what, cache, slots)
    pages, page, H = _cache_shape(what, cache)
    N = _slots_arg(what, slots)
    _need(dtype in _DTYPE, HQ_ERR_UNSUPPORTED, what, "dtype")

    def call(s):
        k = cache.new_empty((N, H, HQ_KV4_HEAD), dtype=dtype)
        v = torch.empty_like(k)
        t = H * HQ_KV4_HEAD
        _check(lib().hq_kv4_gather(_DTYPE[dtype], cache.data_ptr(), pages, page, slots.data_ptr(), N, H, hadamard_n,
                                   k.data_ptr(), t, HQ_KV4_HEAD, v.data_ptr(), t, HQ_KV4_HEAD, s), what)
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
    _launch(_device("kv4_attention_workspace", ws), stream, (ws,), lambda s: hq_workspace_init(ws, s))
    return ws


def kv4_attention(q: torch.Tensor, cache: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                  cu_q: torch.Tensor | None = None, q_len: int = 1, scale: float | None = None, window: int = 0,
                  sinks: int = 0, hadamard_n: int = 128, ws: torch.Tensor | None = None, out: torch.Tensor | None = None,
                  want_lse: bool = False, stream=None):
    """Attention of q [Tq, Hq, 128], the newest tokens of each request, over the cache (see hq.h) -> out, or (out, lse
    [Tq, Hq]) with want_lse.  Rows behind the last request's are left as they were (uninitialized in a new tensor).
    scale: 1 / sqrt(128) unless given."""
    what = "kv4_attention"
    dev = _device(what, q, cache, block_table, seq_lens, cu_q, ws, out)
    pages, page, Hkv = _cache_shape(what, cache)
    shape, dtype = q.shape, q.dtype
    if len(shape) != 3 or shape[2] != HQ_KV4_HEAD or (dtype != torch.bfloat16 and dtype != torch.float16):
        raise HQError(HQ_ERR_UNSUPPORTED if len(shape) == 3 and shape[2] == HQ_KV4_HEAD else HQ_ERR_SHAPE,
                      what + ": q is BF16 or FP16 [Tq, heads, 128]")
    Tq, Hq, _ = shape
    qs = _heads(what, "q", q, shape, dtype)
    os = (Hq * HQ_KV4_HEAD, HQ_KV4_HEAD) if out is None else _heads(what, "out", out, shape, dtype)
    B = seq_lens.shape[0] if seq_lens.dim() == 1 else -1
    width = _table(what, block_table, B)
    _vector(what, "seq_lens", seq_lens, B, torch.int32)
    if cu_q is not None:
        _vector(what, "cu_q", cu_q, B + 1, torch.int32)

    def call(s):
        o = q.new_empty(shape) if out is None else out
        lse = q.new_empty((Tq, Hq), dtype=torch.float32) if want_lse else None
        w = kv4_attention_workspace(q.device) if ws is None else ws
        _check(lib().hq_kv4_attention(_DTYPE[dtype], q.data_ptr(), qs[0], qs[1], Tq, Hq, cache.data_ptr(), pages, page, Hkv,
                                      block_table.data_ptr(), width, B, seq_lens.data_ptr(), _ptr(cu_q), q_len,
                                      HQ_KV4_HEAD ** -0.5 if scale is None else scale, window, sinks, hadamard_n,
                                      o.data_ptr(), os[0], os[1], _ptr(lse), w.data_ptr(), w.nbytes, s), what)
        return (o, lse) if want_lse else o

    return _launch(dev, stream, (q, cache, block_table, seq_lens, cu_q, ws, out), call)


__all__ = [n for n in dir() if n.startswith(("HQ_DT_", "HQ_ROPE_", "HQ_NORM_", "HQ_KV", "hq_add_", "hq_rms", "hq_rope",
                                              "hq_kv"))]
__all__ += ["add_rmsnorm_fp8_k128", "rmsnorm_backward", "rmsnorm_backward_workspace", "rope", "rope_inv_freq", "kv_slots",
            "kv4_cache", "kv4_append", "kv4_gather", "kv4_attention", "kv4_attention_workspace"]
