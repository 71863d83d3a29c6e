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


def _elsewhere(device: int, stream, tensors, call):
    """call() with `device` and `stream` current: outputs are allocated on the stream, inputs recorded on it."""
    with torch.cuda.device(device):
        if stream is None:
            return call()
        s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream), device)
        with torch.cuda.stream(s):
            for t in tensors:
                if t is not None:
                    t.record_stream(s)
            return call()


def _apart(device: int, stream) -> bool:
    """Whether a call has to make its device or stream current first."""
    return stream is not None or device != torch.cuda.current_device()


# The conveniences below test everything in a few long conditions, one per status: a call's own time counts in a step of
# few tokens.
def _refuse(status: int, what: str):
    raise HQError(status, what)


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


def add_rmsnorm_fp8_k128(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, eps: float = 1e-6,
                         scale_layout: int = HQ_SCALE_ROWMAJOR, scale_ld: int | None = None, want_rstd: bool = False,
                         want_amax: bool = False, residual_out: torch.Tensor | None = None, stream=None) -> dict:
    """Residual addition, RMS norm and K128 FP8 codes of [M, K] rows (see hq.h) -> dict with codes [M, K], scales,
    residual_out (with a residual: what the norm read; into `residual_out` where given, which may be x or residual
    itself) and, when asked, rstd [M] and amax."""
    what = "add_rmsnorm_fp8_k128"
    dev, dtype, wtype, shape = x.get_device(), x.dtype, weight.dtype, x.shape
    if not (dev >= 0 and weight.get_device() == dev and dtype in _DTYPE and (wtype == dtype or wtype == torch.float32)
            and (residual is None or (residual.get_device() == dev and residual.dtype == dtype))
            and (residual_out is None or (residual_out.get_device() == dev and residual_out.dtype == dtype))):
        _refuse(HQ_ERR_UNSUPPORTED, what + ": tensors of one CUDA device and type (the weight may be FP32) are needed")
    if not (len(shape) == 2 and weight.dim() == 1 and weight.shape[0] == shape[1]
            and (residual is None or residual.shape == shape) and (residual_out is None or residual_out.shape == shape)):
        _refuse(HQ_ERR_SHAPE, what + ": x, residual and residual_out are [M, K], weight is [K]")
    if residual is None and residual_out is not None:
        _refuse(HQ_ERR_NULL, what + ": residual_out without a residual")
    M, K = shape
    xs, rs = x.stride(), (K, 1) if residual is None else residual.stride()
    if not (xs[1] == 1 and rs[1] == 1 and weight.is_contiguous() and (residual_out is None or residual_out.is_contiguous())):
        _refuse(HQ_ERR_ALIGN, what + ": rows, weight and residual_out have to be contiguous")
    if _apart(dev, stream):
        return _elsewhere(dev, stream, (x, weight, residual, residual_out), lambda: add_rmsnorm_fp8_k128(
            x, weight, residual, eps, scale_layout, scale_ld, want_rstd, want_amax, residual_out))
    groups = K // 128
    codes = x.new_empty(shape, dtype=torch.uint8)
    if (scale_layout & ~HQ_FP8_UE8M0) == HQ_SCALE_TRANSPOSED:
        ld = M if scale_ld is None else scale_ld
        scales = x.new_empty((groups, ld), dtype=torch.float32)
    else:
        ld = groups
        scales = x.new_empty((M, groups), dtype=torch.float32)
    out = {"codes": codes, "scales": scales}
    h = rstd = amax = None
    if residual is not None:
        h = out["residual_out"] = x.new_empty(shape) if residual_out is None else residual_out
    if want_rstd:
        rstd = out["rstd"] = x.new_empty((M,), dtype=torch.float32)
    if want_amax:
        amax = out["amax"] = torch.empty_like(scales)
    _check(lib().hq_add_rmsnorm_fp8_k128(
        _DTYPE[dtype], x.data_ptr(), xs[0] if M > 1 else K, _ptr(residual), rs[0] if M > 1 else K, weight.data_ptr(),
        _DTYPE[wtype], eps, M, K, _ptr(h), codes.data_ptr(), scales.data_ptr(), scale_layout, ld, _ptr(rstd), _ptr(amax),
        _raw_stream(dev)), what)
    return out


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
    dev, dtype, wtype, shape = dy.get_device(), dy.dtype, weight.dtype, dy.shape
    f32 = torch.float32
    if not (dev >= 0 and h.get_device() == dev and weight.get_device() == dev and rstd.get_device() == dev and dtype in _DTYPE
            and h.dtype == dtype and (wtype == dtype or wtype == f32) and rstd.dtype == f32
            and (dres is None or (dres.get_device() == dev and dres.dtype == dtype))
            and (dx is None or (dx.get_device() == dev and dx.dtype == dtype)) and (ws is None or ws.get_device() == dev)):
        _refuse(HQ_ERR_UNSUPPORTED, what + ": tensors of one CUDA device and type (weight and rstd FP32) are needed")
    if not (len(shape) == 2 and h.shape == shape and weight.dim() == 1 and weight.shape[0] == shape[1] and rstd.dim() == 1
            and rstd.shape[0] == shape[0] and (dres is None or dres.shape == shape) and (dx is None or dx.shape == shape)):
        _refuse(HQ_ERR_SHAPE, what + ": dy, h, dres and dx are [M, K], weight is [K], rstd is [M]")
    M, K = shape
    gs, hs, rs = dy.stride(), h.stride(), (K, 1) if dres is None else dres.stride()
    if not (gs[1] == 1 and hs[1] == 1 and rs[1] == 1 and weight.is_contiguous() and rstd.is_contiguous()
            and (dx is None or dx.is_contiguous()) and (ws is None or ws.is_contiguous())):
        _refuse(HQ_ERR_ALIGN, what + ": rows, weight, rstd, dx and the workspace have to be contiguous")
    if _apart(dev, stream):
        return _elsewhere(dev, stream, (dy, h, weight, rstd, dres, ws, dx), lambda: rmsnorm_backward(
            dy, h, weight, rstd, dres, want_dweight, ws, dx))
    out = dy.new_empty(shape) if dx is None else dx
    dw, nbytes = None, 0
    if want_dweight:
        dw = dy.new_empty((K,), dtype=f32)
        if ws is None:
            ws = rmsnorm_backward_workspace(M, K, dy.device)
        nbytes = ws.nbytes
    one = M <= 1
    _check(lib().hq_rmsnorm_backward(
        _DTYPE[dtype], dy.data_ptr(), K if one else gs[0], h.data_ptr(), K if one else hs[0], weight.data_ptr(),
        _DTYPE[wtype], rstd.data_ptr(), _ptr(dres), K if one else rs[0], M, K, out.data_ptr(), _ptr(dw), _ptr(ws), nbytes,
        _raw_stream(dev)), what)
    return out, dw


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
    dev, dtype, shape = q.get_device(), q.dtype, q.shape
    if not (dev >= 0 and positions.get_device() == dev and inv_freq.get_device() == dev and dtype in _DTYPE
            and positions.dtype == torch.int64 and inv_freq.dtype == torch.float64
            and (k is None or (k.get_device() == dev and k.dtype == dtype))
            and (q_out is None or (q_out.get_device() == dev and q_out.dtype == dtype))
            and (k_out is None or (k_out.get_device() == dev and k_out.dtype == dtype))):
        _refuse(HQ_ERR_UNSUPPORTED, what + ": tensors of one CUDA device and type, int64 positions, float64 inv_freq are needed")
    kshape = (*shape[:1], 0, *shape[-1:]) if k is None else k.shape
    if not (len(shape) == 3 and len(kshape) == 3 and kshape[0] == shape[0] and kshape[2] == shape[2] and positions.dim() == 1
            and positions.shape[0] == shape[0] and inv_freq.dim() == 1 and (q_out is None or q_out.shape == shape)
            and (k_out is None or (k is not None and k_out.shape == kshape))):
        _refuse(HQ_ERR_SHAPE, what + ": q is [T, Hq, D], k is [T, Hk, D], positions is [T]")
    T, Hq, D = shape
    Hk = kshape[1]
    qs, qos = q.stride(), (Hq * D, D, 1) if q_out is None else q_out.stride()
    ks, kos = (0, 0, 1) if k is None else k.stride(), (Hk * D, D, 1) if k_out is None else k_out.stride()
    if not ((D == 1 or (qs[2] == 1 and ks[2] == 1 and qos[2] == 1 and kos[2] == 1)) and positions.is_contiguous()
            and inv_freq.is_contiguous()):
        _refuse(HQ_ERR_ALIGN, what + ": heads, positions and inv_freq have to be contiguous")
    if _apart(dev, stream):
        return _elsewhere(dev, stream, (q, k, positions, inv_freq, q_out, k_out), lambda: rope(
            q, k, positions, inv_freq, offset, layout, magnitude, inverse, q_out, k_out))
    if q_out is None:
        q_out = q.new_empty(shape)
    if k is not None and k_out is None:
        k_out = k.new_empty(kshape)
    _check(lib().hq_rope(_DTYPE[dtype], q.data_ptr(), qs[0], qs[1], Hq, _ptr(k), ks[0], ks[1], Hk, T, D,
                         positions.data_ptr(), inv_freq.data_ptr(), 2 * inv_freq.shape[0], offset, layout, magnitude,
                         1 if inverse else 0, q_out.data_ptr(), qos[0], qos[1], _ptr(k_out), kos[0], kos[1],
                         _raw_stream(dev)), what)
    return q_out, k_out


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
    dev, i32 = lens.get_device(), torch.int32
    if not (dev >= 0 and new_tokens.get_device() == dev and block_table.get_device() == dev and free_pages.get_device() == dev
            and free_count.get_device() == dev and lens.dtype == i32 and new_tokens.dtype == i32 and block_table.dtype == i32
            and free_pages.dtype == i32 and free_count.dtype == i32
            and (lens_out is None or (lens_out.get_device() == dev and lens_out.dtype == i32))
            and (free_count_out is None or (free_count_out.get_device() == dev and free_count_out.dtype == i32))):
        _refuse(HQ_ERR_UNSUPPORTED, what + ": int32 tensors of one CUDA device are needed")
    if not (lens.dim() == 1 and new_tokens.shape == lens.shape and block_table.dim() == 2
            and block_table.shape[0] == lens.shape[0] and free_pages.dim() == 1 and free_count.numel() == 1
            and (lens_out is None or lens_out.shape == lens.shape)
            and (free_count_out is None or free_count_out.numel() == 1) and n_slots >= 0):
        _refuse(HQ_ERR_SHAPE, what + ": lens and new_tokens are [B], block_table is [B, width], free_count is [1]")
    if not (lens.is_contiguous() and new_tokens.is_contiguous() and block_table.is_contiguous() and free_pages.is_contiguous()
            and (lens_out is None or lens_out.is_contiguous())):
        _refuse(HQ_ERR_ALIGN, what + ": tensors have to be contiguous")
    if _apart(dev, stream):
        return _elsewhere(dev, stream, (lens, new_tokens, block_table, free_pages, free_count, lens_out, free_count_out),
                          lambda: kv_slots(lens, new_tokens, block_table, free_pages, free_count, page_size, n_slots,
                                           lens_out, free_count_out))
    B = lens.shape[0]
    lo = torch.empty_like(lens) if lens_out is None else lens_out
    count = torch.empty_like(free_count) if free_count_out is None else free_count_out
    cu, status = lens.new_empty((B + 1,)), torch.empty_like(free_count)
    slots = lens.new_empty((n_slots,), dtype=torch.int64)
    positions = torch.empty_like(slots)
    _check(lib().hq_kv_slots(B, lens.data_ptr(), new_tokens.data_ptr(), block_table.data_ptr(), block_table.shape[1],
                             free_pages.data_ptr(), free_pages.shape[0], free_count.data_ptr(), page_size, n_slots,
                             lo.data_ptr(), cu.data_ptr(), slots.data_ptr(), positions.data_ptr(), count.data_ptr(),
                             status.data_ptr(), _raw_stream(dev)), what)
    return {"lens": lo, "cu_new": cu, "slots": slots, "positions": positions, "free_count": count, "status": status}


def hq_kv4_cache_bytes(num_pages: int, page_size: int, H: int) -> int:
    return int(lib().hq_kv4_cache_bytes(int(num_pages), int(page_size), int(H)))


def kv4_cache(num_pages: int, page_size: int, H: int, device="cuda") -> torch.Tensor:
    """An empty NVFP4 key/value cache: uint8 [num_pages, H, page_size / 16, 2432]."""
    _need(hq_kv4_cache_bytes(num_pages, page_size, H) > 0, HQ_ERR_SHAPE, "kv4_cache")
    return torch.zeros((num_pages, H, page_size // HQ_KV4_GROUP_TOKENS, HQ_KV4_GROUP_BYTES), dtype=torch.uint8,
                       device=device)


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


def kv4_append(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, cache: torch.Tensor, hadamard_n: int = 128,
               stream=None) -> None:
    """Quantize keys and values [N, H, 128] into the cache's slots (see hq.h); slots outside the cache are skipped."""
    what = "kv4_append"
    dev, dtype, shape, cshape = cache.get_device(), k.dtype, k.shape, cache.shape
    if not (dev >= 0 and k.get_device() == dev and v.get_device() == dev and slots.get_device() == dev and dtype in _DTYPE
            and v.dtype == dtype and slots.dtype == torch.int64 and cache.dtype == torch.uint8):
        _refuse(HQ_ERR_UNSUPPORTED, what + ": k and v of one type, int64 slots and a uint8 cache on one CUDA device are needed")
    if not (len(cshape) == 4 and cshape[3] == HQ_KV4_GROUP_BYTES and len(shape) == 3 and shape[1] == cshape[1]
            and shape[2] == HQ_KV4_HEAD and v.shape == shape and slots.dim() == 1 and slots.shape[0] == shape[0]):
        _refuse(HQ_ERR_SHAPE, what + ": k and v are [N, H, 128], slots is [N], the cache [pages, H, page_size / 16, 2432]")
    ks, vs = k.stride(), v.stride()
    if not (ks[2] == 1 and vs[2] == 1 and slots.is_contiguous() and cache.is_contiguous()):
        _refuse(HQ_ERR_ALIGN, what + ": heads, slots and the cache have to be contiguous")
    if _apart(dev, stream):
        return _elsewhere(dev, stream, (k, v, slots, cache), lambda: kv4_append(k, v, slots, cache, hadamard_n))
    _check(lib().hq_kv4_append(_DTYPE[dtype], k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1], slots.data_ptr(),
                               shape[0], shape[1], hadamard_n, cache.data_ptr(), cshape[0],
                               cshape[2] * HQ_KV4_GROUP_TOKENS, _raw_stream(dev)), what)


def kv4_gather(cache: torch.Tensor, slots: torch.Tensor, dtype: torch.dtype = torch.bfloat16, hadamard_n: int = 128,
               stream=None):
    """Keys and values [N, H, 128] of the cache's slots (see hq.h), rotated back with hadamard_n 128 -> (k, v)."""
    what = "kv4_gather"
    dev, cshape = cache.get_device(), cache.shape
    if not (dev >= 0 and slots.get_device() == dev and dtype in _DTYPE and slots.dtype == torch.int64
            and cache.dtype == torch.uint8):
        _refuse(HQ_ERR_UNSUPPORTED, what + ": int64 slots and a uint8 cache on one CUDA device are needed")
    if not (len(cshape) == 4 and cshape[3] == HQ_KV4_GROUP_BYTES and slots.dim() == 1):
        _refuse(HQ_ERR_SHAPE, what + ": slots is [N], the cache [pages, H, page_size / 16, 2432]")
    if not (slots.is_contiguous() and cache.is_contiguous()):
        _refuse(HQ_ERR_ALIGN, what + ": slots and the cache have to be contiguous")
    if _apart(dev, stream):
        return _elsewhere(dev, stream, (cache, slots), lambda: kv4_gather(cache, slots, dtype, hadamard_n))
    N, H = slots.shape[0], cshape[1]
    k = cache.new_empty((N, H, HQ_KV4_HEAD), dtype=dtype)
    v = torch.empty_like(k)
    t = H * HQ_KV4_HEAD
    _check(lib().hq_kv4_gather(_DTYPE[dtype], cache.data_ptr(), cshape[0], cshape[2] * HQ_KV4_GROUP_TOKENS, slots.data_ptr(),
                               N, H, hadamard_n, k.data_ptr(), t, HQ_KV4_HEAD, v.data_ptr(), t, HQ_KV4_HEAD,
                               _raw_stream(dev)), what)
    return k, v


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
    dev = ws.get_device()
    if dev < 0:
        _refuse(HQ_ERR_UNSUPPORTED, "kv4_attention_workspace: a CUDA device is needed")
    _elsewhere(dev, stream, (ws,), lambda: hq_workspace_init(ws, _raw_stream(dev)))
    return ws


def kv4_attention(q: torch.Tensor, cache: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                  cu_q: torch.Tensor | None = None, q_len: int = 1, scale: float | None = None, window: int = 0,
                  sinks: int = 0, hadamard_n: int = 128, ws: torch.Tensor | None = None, out: torch.Tensor | None = None,
                  want_lse: bool = False, stream=None):
    """Attention of q [Tq, Hq, 128], the newest tokens of each request, over the cache (see hq.h) -> out, or (out, lse
    [Tq, Hq]) with want_lse.  Rows behind the last request's are left as they were (uninitialized in a new tensor).
    scale: 1 / sqrt(128) unless given."""
    what = "kv4_attention"
    dev, dtype, shape, cshape, i32 = q.get_device(), q.dtype, q.shape, cache.shape, torch.int32
    if not (dev >= 0 and cache.get_device() == dev and block_table.get_device() == dev and seq_lens.get_device() == dev
            and (dtype == torch.bfloat16 or dtype == torch.float16) and cache.dtype == torch.uint8 and block_table.dtype == i32
            and seq_lens.dtype == i32 and (cu_q is None or (cu_q.get_device() == dev and cu_q.dtype == i32))
            and (out is None or (out.get_device() == dev and out.dtype == dtype)) and (ws is None or ws.get_device() == dev)):
        _refuse(HQ_ERR_UNSUPPORTED, what + ": BF16 or FP16 q and out, a uint8 cache, int32 tables on one CUDA device are needed")
    B = seq_lens.numel()
    if not (len(shape) == 3 and shape[2] == HQ_KV4_HEAD and len(cshape) == 4 and cshape[3] == HQ_KV4_GROUP_BYTES
            and seq_lens.dim() == 1 and block_table.dim() == 2 and block_table.shape[0] == B
            and (cu_q is None or (cu_q.dim() == 1 and cu_q.shape[0] == B + 1)) and (out is None or out.shape == shape)):
        _refuse(HQ_ERR_SHAPE, what + ": q and out are [Tq, Hq, 128], the cache [pages, Hkv, page_size / 16, 2432], block_table "
                                     "[B, width], seq_lens [B], cu_q [B + 1]")
    Tq, Hq, _ = shape
    qs, os = q.stride(), (Hq * HQ_KV4_HEAD, HQ_KV4_HEAD, 1) if out is None else out.stride()
    if not (qs[2] == 1 and os[2] == 1 and cache.is_contiguous() and block_table.is_contiguous() and seq_lens.is_contiguous()
            and (cu_q is None or cu_q.is_contiguous()) and (ws is None or ws.is_contiguous())):
        _refuse(HQ_ERR_ALIGN, what + ": heads, the cache, tables and the workspace have to be contiguous")
    if _apart(dev, stream):
        return _elsewhere(dev, stream, (q, cache, block_table, seq_lens, cu_q, ws, out), lambda: kv4_attention(
            q, cache, block_table, seq_lens, cu_q, q_len, scale, window, sinks, hadamard_n, ws, out, want_lse))
    if out is None:
        out = q.new_empty(shape)
    lse = q.new_empty((Tq, Hq), dtype=torch.float32) if want_lse else None
    if ws is None:
        ws = kv4_attention_workspace(q.device)
    _check(lib().hq_kv4_attention(_DTYPE[dtype], q.data_ptr(), qs[0], qs[1], Tq, Hq, cache.data_ptr(), cshape[0],
                                  cshape[2] * HQ_KV4_GROUP_TOKENS, cshape[1], block_table.data_ptr(), block_table.shape[1], B,
                                  seq_lens.data_ptr(), _ptr(cu_q), q_len, HQ_KV4_HEAD ** -0.5 if scale is None else scale,
                                  window, sinks, hadamard_n, out.data_ptr(), os[0], os[1], _ptr(lse), ws.data_ptr(),
                                  ws.nbytes, _raw_stream(dev)), what)
    return (out, lse) if want_lse else out


__all__ = [n for n in dir() if n.startswith(("HQ_DT_", "HQ_ROPE_", "HQ_NORM_", "HQ_KV", "hq_add_", "hq_rms", "hq_rope",
                                              "hq_kv"))]
__all__ += ["add_rmsnorm_fp8_k128", "rmsnorm_backward", "rmsnorm_backward_workspace", "rope", "rope_inv_freq", "kv_slots",
            "kv4_cache", "kv4_append", "kv4_gather", "kv4_attention", "kv4_attention_workspace"]
