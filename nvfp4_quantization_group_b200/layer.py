"""The attention layer around the quantizers: residual + RMS norm with FP8 codes, rotary positions, slot maps, the NVFP4
key/value cache and attention over it (the second half of include/hq.h).

``hq_*`` functions take caller-allocated tensors like the C calls; the others check types, shapes, strides and devices,
allocate what they return and call the same C functions (in csrc/hq_torch.cpp, compiled beside the library: a step of few
tokens is bound by the host's part of a call).  Tensors may lie on any CUDA device (all of one call on the same); the
work goes to that device's current stream, or to `stream`.  With `stream` the outputs are allocated on it and the inputs
recorded on it, so that they may be dropped as soon as the call returns.  A refused call raises HQError, as in the rest
of the package.

None of them records gradients.  Rows that require a gradient (and the norm's weight) are refused while autograd records,
so that none is lost unseen: call them under torch.no_grad() or inside an autograd.Function, whose backward pass is
rmsnorm_backward or rope(..., inverse=True).
"""
from __future__ import annotations

import ctypes

import torch

from . import HQ_ERR_SHAPE, HQ_ERR_UNSUPPORTED, HQ_SCALE_ROWMAJOR, HQError, _check, _p, _stream, hq_workspace_init, lib

HQ_DT_BF16, HQ_DT_F16, HQ_DT_F32 = 0, 1, 2
HQ_ROPE_HALVES, HQ_ROPE_INTERLEAVED = 0, 1
HQ_ROPE_PLAIN, HQ_ROPE_LINEAR, HQ_ROPE_NTK, HQ_ROPE_PARTS, HQ_ROPE_BANDS = range(5)
HQ_NORM_MAX_K = 65536
HQ_KV_MAX_REQUESTS = 4096
HQ_KV_NO_PAGES, HQ_KV_NO_ROWS, HQ_KV_NO_WIDTH, HQ_KV_BAD_STATE = 1, 2, 4, 8
HQ_KV4_HEAD, HQ_KV4_GROUP_TOKENS, HQ_KV4_GROUP_BYTES = 128, 16, 2432
HQ_KV4_ATTENTION_STATE_BYTES = 2304

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


_torch_calls = None


def _x():
    """The compiled conveniences, bound to the loaded library (raises if they have not been built: there is no fallback)."""
    global _torch_calls
    if _torch_calls is None:
        from . import _build
        if not _build.torch_lib_fits():
            raise OSError(f"{_build.TORCH_LIB} is missing or was built for another torch or Python: run "
                          "nvfp4_quantization_group_b200/_build.py")
        from . import _hq_torch
        L = lib()
        _hq_torch.bind({n: ctypes.cast(getattr(L, n), _P).value for n in (*SIGNATURES, "hq_workspace_init")})
        _torch_calls = _hq_torch
    return _torch_calls


def _on(stream, tensors, call):
    """call() with the first tensor's device and `stream` current: outputs are allocated on the stream, inputs recorded."""
    device = tensors[0].get_device()
    if device < 0:
        return call()  # refuses
    s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream), device)
    with torch.cuda.device(device), torch.cuda.stream(s):
        for t in tensors:
            if t is not None and t.is_cuda:
                t.record_stream(s)
        return call()


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
    itself) and, when asked, rstd [M] and amax (up to 32 KB of scales share an allocation with them)."""
    if stream is not None:
        return _on(stream, (x, weight, residual, residual_out), lambda: add_rmsnorm_fp8_k128(
            x, weight, residual, eps, scale_layout, scale_ld, want_rstd, want_amax, residual_out))
    codes, scales, h, rstd, amax = _x().add_rmsnorm(x, weight, residual, eps, scale_layout, scale_ld, want_rstd, want_amax,
                                                    residual_out)
    out = {"codes": codes, "scales": scales}
    if h is not None:
        out["residual_out"] = h
    if want_rstd:
        out["rstd"] = rstd
    if want_amax:
        out["amax"] = amax
    return out


def rmsnorm_backward_workspace(M: int, K: int, device="cuda") -> torch.Tensor:
    """Workspace of rmsnorm_backward for [M, K]; any contents."""
    nbytes = hq_rmsnorm_backward_workspace_size(M, K)
    if nbytes == 0:
        raise HQError(HQ_ERR_SHAPE, "rmsnorm_backward_workspace")
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def rmsnorm_backward(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                     dres: torch.Tensor | None = None, want_dweight: bool = True, ws: torch.Tensor | None = None,
                     dx: torch.Tensor | None = None, stream=None):
    """Gradients of the norm (see hq.h): dy the gradient of the normalized rows, h what the norm read (residual_out, or x
    without a residual), dres the gradient that reaches h along the residual -> (dx [M, K], dweight FP32 [K] or None).
    dx is written into `dx` where given (it may be dy or dres itself)."""
    if stream is not None:
        return _on(stream, (dy, h, weight, rstd, dres, ws, dx), lambda: rmsnorm_backward(
            dy, h, weight, rstd, dres, want_dweight, ws, dx))
    return _x().rmsnorm_backward(dy, h, weight, rstd, dres, want_dweight, ws, dx)


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
    if stream is not None:
        return _on(stream, (q, k, positions, inv_freq, q_out, k_out), lambda: rope(
            q, k, positions, inv_freq, offset, layout, magnitude, inverse, q_out, k_out))
    return _x().rope(q, k, positions, inv_freq, offset, layout, magnitude, bool(inverse), q_out, k_out)


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
    if stream is not None:
        return _on(stream, (lens, new_tokens, block_table, free_pages, free_count, lens_out, free_count_out),
                   lambda: kv_slots(lens, new_tokens, block_table, free_pages, free_count, page_size, n_slots, lens_out,
                                    free_count_out))
    lo, cu, slots, positions, count, status = _x().kv_slots(lens, new_tokens, block_table, free_pages, free_count, page_size,
                                                            n_slots, lens_out, free_count_out)
    return {"lens": lo, "cu_new": cu, "slots": slots, "positions": positions, "free_count": count, "status": status}


def hq_kv4_cache_bytes(num_pages: int, page_size: int, H: int) -> int:
    return int(lib().hq_kv4_cache_bytes(int(num_pages), int(page_size), int(H)))


def kv4_cache(num_pages: int, page_size: int, H: int, device="cuda") -> torch.Tensor:
    """An empty NVFP4 key/value cache: uint8 [num_pages, H, page_size / 16, 2432]."""
    if hq_kv4_cache_bytes(num_pages, page_size, H) == 0:
        raise HQError(HQ_ERR_SHAPE, "kv4_cache")
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
    if stream is not None:
        return _on(stream, (cache, k, v, slots), lambda: kv4_append(k, v, slots, cache, hadamard_n))
    _x().kv4_append(k, v, slots, cache, hadamard_n)


def kv4_gather(cache: torch.Tensor, slots: torch.Tensor, dtype: torch.dtype = torch.bfloat16, hadamard_n: int = 128,
               stream=None):
    """Keys and values [N, H, 128] of the cache's slots (see hq.h), rotated back with hadamard_n 128 -> (k, v)."""
    if stream is not None:
        return _on(stream, (cache, slots), lambda: kv4_gather(cache, slots, dtype, hadamard_n))
    return _x().kv4_gather(cache, slots, dtype, hadamard_n)


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
    if not ws.is_cuda:
        raise HQError(HQ_ERR_UNSUPPORTED, "kv4_attention_workspace: a CUDA device is needed")
    _on(torch.cuda.current_stream(ws.device) if stream is None else stream, (ws,), lambda: hq_workspace_init(ws))
    return ws


def kv4_attention(q: torch.Tensor, cache: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                  cu_q: torch.Tensor | None = None, q_len: int = 1, scale: float | None = None, window: int = 0,
                  sinks: int = 0, hadamard_n: int = 128, ws: torch.Tensor | None = None, out: torch.Tensor | None = None,
                  want_lse: bool = False, stream=None, want_error: bool = False):
    """Attention of q [Tq, Hq, 128], the newest tokens of each request, over the cache (see hq.h) -> out; with want_lse
    (out, lse [Tq, Hq]), with want_error also an int32 [1] on the device, last.  Rows behind the last request's are left
    as they were (uninitialized in a new tensor).  scale: 1 / sqrt(128) unless given.

    A page or length outside the cache, rows outside q and a wait that gave up are found on the device; the call returns
    all the same, and what they concern counts as not seen or is not written.  They are reported by hq_get_error(ws), or
    by want_error: the workspace's error word after the call (0: none).  Without either the report is lost: a call without
    `ws` uses a workspace of its own (also slower: allocated and cleared each time)."""
    if stream is not None:
        return _on(stream, (q, cache, block_table, seq_lens, cu_q, ws, out), lambda: kv4_attention(
            q, cache, block_table, seq_lens, cu_q, q_len, scale, window, sinks, hadamard_n, ws, out, want_lse,
            want_error=want_error))
    o, lse, error = _x().kv4_attention(q, cache, block_table, seq_lens, cu_q, q_len, scale, window, sinks, hadamard_n, ws, out,
                                       want_lse, want_error)
    if want_error:
        return (o, lse, error) if want_lse else (o, error)
    return (o, lse) if want_lse else o


__all__ = [n for n in dir() if n.startswith(("HQ_DT_", "HQ_ROPE_", "HQ_NORM_", "HQ_KV", "hq_add_", "hq_rms", "hq_rope",
                                              "hq_kv"))]
__all__ += ["add_rmsnorm_fp8_k128", "rmsnorm_backward", "rmsnorm_backward_workspace", "rope", "rope_inv_freq", "kv_slots",
            "kv4_cache", "kv4_append", "kv4_gather", "kv4_attention", "kv4_attention_workspace"]
