// hq_torch.cpp -- the attention-layer conveniences of layer.py on torch
// tensors: checks of types, shapes and strides, allocation of the outputs, and
// one call of the C ABI each (include/hq.h).  No step of the computation runs
// here.  It is C++ because a step of few tokens is bound by the host: the same
// work in Python took 14 to 20 us a call, two to four times the kernels.
//
// The C functions are reached through the addresses that bind() is given (the
// library that the package has loaded); refusals become the package's HQError.
#include <ATen/ATen.h>
#include <ATen/core/grad_mode.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/utils/pybind.h>

#include <optional>
#include <string>
#include <tuple>

#include "hq.h"

namespace py = pybind11;
using at::Tensor;
using Maybe = std::optional<Tensor>;

namespace {

struct Refusal {
    int status;
    std::string what;
};
inline void need(bool ok, int status, const char* what) {
    if (!ok) throw Refusal{status, what};
}

struct Calls {
    decltype(&hq_add_rmsnorm_fp8_k128) norm = nullptr;
    decltype(&hq_rmsnorm_backward_workspace_size) norm_back_ws = nullptr;
    decltype(&hq_rmsnorm_backward) norm_back = nullptr;
    decltype(&hq_rope) rope = nullptr;
    decltype(&hq_kv_slots) slots = nullptr;
    decltype(&hq_kv4_append) append = nullptr;
    decltype(&hq_kv4_gather) gather = nullptr;
    decltype(&hq_kv4_attention_workspace_size) attention_ws = nullptr;
    decltype(&hq_kv4_attention) attention = nullptr;
    decltype(&hq_workspace_init) ws_init = nullptr;
} call;

template <typename F> void take(F& f, const py::dict& d, const char* name) {
    f = reinterpret_cast<F>(d[name].cast<uintptr_t>());
}
void bind(const py::dict& d) {
    take(call.norm, d, "hq_add_rmsnorm_fp8_k128");
    take(call.norm_back_ws, d, "hq_rmsnorm_backward_workspace_size");
    take(call.norm_back, d, "hq_rmsnorm_backward");
    take(call.rope, d, "hq_rope");
    take(call.slots, d, "hq_kv_slots");
    take(call.append, d, "hq_kv4_append");
    take(call.gather, d, "hq_kv4_gather");
    take(call.attention_ws, d, "hq_kv4_attention_workspace_size");
    take(call.attention, d, "hq_kv4_attention");
    take(call.ws_init, d, "hq_workspace_init");
}

inline int type_of(at::ScalarType t) {  // HQ_DT_*, or -1
    return t == at::kBFloat16 ? HQ_DT_BF16 : t == at::kHalf ? HQ_DT_F16 : t == at::kFloat ? HQ_DT_F32 : -1;
}
inline void* ptr(const Maybe& t) { return t ? t->data_ptr() : nullptr; }
// On `like`'s device and of its type; of a given type.
inline bool fits(const Tensor& t, const Tensor& like) { return t.device() == like.device() && t.scalar_type() == like.scalar_type(); }
inline bool fits(const Maybe& t, const Tensor& like) { return !t || fits(*t, like); }
inline bool is(const Tensor& t, const Tensor& like, at::ScalarType s) { return t.device() == like.device() && t.scalar_type() == s; }
inline bool is(const Maybe& t, const Tensor& like, at::ScalarType s) { return !t || is(*t, like, s); }
inline bool shaped(const Maybe& t, const Tensor& like) { return !t || t->sizes() == like.sizes(); }
inline bool vector_of(const Tensor& t, int64_t n) { return t.dim() == 1 && t.size(0) == n; }
inline bool rows_whole(const Maybe& t) { return !t || t->size(-1) <= 1 || t->stride(-1) == 1; }
// Stride of dimension d, 0 where it has one entry (its stride may be anything then).
inline int64_t step(const Tensor& t, int64_t d) { return t.size(d) > 1 ? t.stride(d) : 0; }
inline int64_t step(const Maybe& t, int64_t d) { return t ? step(*t, d) : 0; }
inline bool whole(const Maybe& t) { return !t || t->is_contiguous(); }
inline Tensor make(at::IntArrayRef shape, const Tensor& like, at::ScalarType s) {
    return Tensor(at::detail::empty_cuda(shape, s, like.device(), std::nullopt));
}

// A vector's entries from `at` on, as a tensor of its own on the same memory (one allocation for the small outputs
// of a call: an allocation costs more than the rest of the bookkeeping).
inline Tensor part(const Tensor& t, int64_t at, at::IntArrayRef shape) {
    Tensor r = at::detail::make_tensor<c10::TensorImpl>(c10::TensorImpl::VIEW, c10::Storage(t.storage()), t.key_set(), t.dtype());
    r.unsafeGetTensorImpl()->set_storage_offset(at);
    r.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
    return r;
}

// These calls record no gradients: an input that wants one while autograd records would lose it unseen.
inline bool tracked(const Tensor& t) { return t.requires_grad(); }
inline bool tracked(const Maybe& t) { return t && t->requires_grad(); }
template <typename... T> inline void untracked(const char* what, const T&... t) {
    need(!(at::GradMode::is_enabled() && (tracked(t) || ...)), HQ_ERR_UNSUPPORTED, what);
}

// Makes the tensors' device current and gives its current stream.
struct On {
    c10::cuda::CUDAGuard guard;
    void* stream;
    explicit On(const Tensor& t)
        : guard(t.device()), stream(c10::cuda::getCurrentCUDAStream(t.device().index()).stream()) {}
};

// ------------------------------------------------------------------- norm
std::tuple<Tensor, Tensor, Maybe, Maybe, Maybe> add_rmsnorm(const Tensor& x, const Tensor& weight, const Maybe& residual,
                                                            double eps, int layout, std::optional<int64_t> scale_ld,
                                                            bool want_rstd, bool want_amax, const Maybe& residual_out) {
    const char* const what = "add_rmsnorm_fp8_k128";
    const int dt = type_of(x.scalar_type()), wt = type_of(weight.scalar_type());
    untracked("add_rmsnorm_fp8_k128 records no gradients: call it under torch.no_grad() (they are rmsnorm_backward's)", x, weight,
              residual, residual_out);
    need(x.is_cuda() && dt >= 0 && weight.device() == x.device() && (wt == dt || wt == HQ_DT_F32) && fits(residual, x) &&
             fits(residual_out, x),
         HQ_ERR_UNSUPPORTED, "add_rmsnorm_fp8_k128: tensors of one CUDA device and type (the weight may be FP32) are needed");
    need(x.dim() == 2 && vector_of(weight, x.size(-1)) && shaped(residual, x) && shaped(residual_out, x), HQ_ERR_SHAPE,
         "add_rmsnorm_fp8_k128: x, residual and residual_out are [M, K], weight is [K]");
    need(residual || !residual_out, HQ_ERR_NULL, "add_rmsnorm_fp8_k128: residual_out without a residual");
    need(rows_whole(x) && rows_whole(residual) && weight.is_contiguous() && whole(residual_out), HQ_ERR_ALIGN,
         "add_rmsnorm_fp8_k128: rows, weight and residual_out have to be contiguous");
    const int64_t M = x.size(0), K = x.size(1), groups = K / 128;
    const On on(x);
    Tensor codes = make({M, K}, x, at::kByte);
    const bool transposed = (layout & ~HQ_FP8_UE8M0) == HQ_SCALE_TRANSPOSED;
    const int64_t ld = transposed ? scale_ld.value_or(M) : groups;
    need(ld >= 0 && ld <= INT32_MAX, HQ_ERR_SHAPE, "add_rmsnorm_fp8_k128: scale_ld");
    const int64_t rows = transposed ? groups : M, n = rows * ld;  // of scales
    // A backward pass keeps rstd, and must not keep a large batch's scales by it.  Up to 32 KB of scales (amax likewise)
    // lie in one allocation with it: [128, 7168] takes 7.4 us of host time a call, [147, 7168] 7.9.
    const bool apart = n > 8192;
    const int64_t n_amax = want_amax && !apart ? n : 0, n_rstd = want_rstd && !apart ? M : 0;
    const Tensor floats = make({n + n_amax + n_rstd}, x, at::kFloat);
    Tensor scales = part(floats, 0, {rows, ld});
    Maybe h, rstd, amax;
    if (residual) h = residual_out ? *residual_out : make({M, K}, x, x.scalar_type());
    if (want_amax) amax = apart ? make({rows, ld}, x, at::kFloat) : part(floats, n, {rows, ld});
    if (want_rstd) rstd = apart ? make({M}, x, at::kFloat) : part(floats, n + n_amax, {M});
    const int s = call.norm(dt, x.data_ptr(), M > 1 ? x.stride(0) : K, ptr(residual), residual && M > 1 ? residual->stride(0) : K,
                            weight.data_ptr(), wt, (float)eps, M, K, ptr(h), static_cast<uint8_t*>(codes.data_ptr()),
                            static_cast<float*>(scales.data_ptr()), layout, ld, static_cast<float*>(ptr(rstd)),
                            static_cast<float*>(ptr(amax)), on.stream);
    need(s == HQ_OK, s, what);
    return {codes, scales, h, rstd, amax};
}

std::tuple<Tensor, Maybe> rmsnorm_backward(const Tensor& dy, const Tensor& h, const Tensor& weight, const Tensor& rstd,
                                           const Maybe& dres, bool want_dweight, const Maybe& ws_in, const Maybe& dx_in) {
    const char* const what = "rmsnorm_backward";
    const int dt = type_of(dy.scalar_type()), wt = type_of(weight.scalar_type());
    untracked("rmsnorm_backward records no gradients of its own: call it under torch.no_grad()", dy, h, dres, dx_in);
    need(dy.is_cuda() && dt >= 0 && fits(h, dy) && weight.device() == dy.device() && (wt == dt || wt == HQ_DT_F32) &&
             is(rstd, dy, at::kFloat) && fits(dres, dy) && fits(dx_in, dy) && (!ws_in || ws_in->device() == dy.device()),
         HQ_ERR_UNSUPPORTED, "rmsnorm_backward: tensors of one CUDA device and type (weight and rstd FP32) are needed");
    need(dy.dim() == 2 && h.sizes() == dy.sizes() && vector_of(weight, dy.size(-1)) && vector_of(rstd, dy.size(0)) &&
             shaped(dres, dy) && shaped(dx_in, dy),
         HQ_ERR_SHAPE, "rmsnorm_backward: dy, h, dres and dx are [M, K], weight is [K], rstd is [M]");
    need(rows_whole(dy) && rows_whole(h) && rows_whole(dres) && weight.is_contiguous() && rstd.is_contiguous() && whole(dx_in) &&
             whole(ws_in),
         HQ_ERR_ALIGN, "rmsnorm_backward: rows, weight, rstd, dx and the workspace have to be contiguous");
    const int64_t M = dy.size(0), K = dy.size(1);
    const On on(dy);
    Tensor dx = dx_in ? *dx_in : make({M, K}, dy, dy.scalar_type());
    Maybe dw, ws = ws_in;
    if (want_dweight) {
        dw = make({K}, dy, at::kFloat);
        if (!ws) ws = make({(int64_t)call.norm_back_ws(M, K)}, dy, at::kByte);
    }
    auto row = [&](const Tensor& t) { return M > 1 ? t.stride(0) : K; };
    const int s = call.norm_back(dt, dy.data_ptr(), row(dy), h.data_ptr(), row(h), weight.data_ptr(), wt,
                                 static_cast<const float*>(rstd.data_ptr()), ptr(dres), dres ? row(*dres) : K, M, K, dx.data_ptr(),
                                 static_cast<float*>(ptr(dw)), want_dweight ? ptr(ws) : nullptr, want_dweight ? ws->nbytes() : 0,
                                 on.stream);
    need(s == HQ_OK, s, what);
    return {dx, dw};
}

// ------------------------------------------------------------------- rope
std::tuple<Tensor, Maybe> rope(const Tensor& q, const Maybe& k, const Tensor& positions, const Tensor& inv_freq, int offset,
                               int layout, double magnitude, bool inverse, const Maybe& q_out, const Maybe& k_out) {
    const char* const what = "rope";
    const int dt = type_of(q.scalar_type());
    untracked("rope records no gradients: call it under torch.no_grad() (they are rope's with inverse)", q, k, q_out, k_out);
    need(q.is_cuda() && dt >= 0 && fits(k, q) && is(positions, q, at::kLong) && is(inv_freq, q, at::kDouble) && fits(q_out, q) &&
             fits(k_out, q),
         HQ_ERR_UNSUPPORTED, "rope: tensors of one CUDA device and type, int64 positions, float64 inv_freq are needed");
    need(q.dim() == 3 && (!k || (k->dim() == 3 && k->size(0) == q.size(0) && k->size(2) == q.size(2))) &&
             vector_of(positions, q.size(0)) && inv_freq.dim() == 1 && shaped(q_out, q) && (k || !k_out) && (!k || shaped(k_out, *k)),
         HQ_ERR_SHAPE, "rope: q is [T, Hq, D], k is [T, Hk, D], positions is [T]");
    need(rows_whole(q) && rows_whole(k) && rows_whole(q_out) && rows_whole(k_out) && positions.is_contiguous() &&
             inv_freq.is_contiguous(),
         HQ_ERR_ALIGN, "rope: heads, positions and inv_freq have to be contiguous");
    const int64_t T = q.size(0), Hq = q.size(1), D = q.size(2), Hk = k ? k->size(1) : 0;
    need(Hq <= INT32_MAX && Hk <= INT32_MAX && D <= INT32_MAX && inv_freq.size(0) <= INT32_MAX / 2, HQ_ERR_SHAPE, "rope: sizes");
    const On on(q);
    Tensor qo = q_out ? *q_out : make({T, Hq, D}, q, q.scalar_type());
    Maybe ko = k_out;
    if (k && !ko) ko = make({T, Hk, D}, q, q.scalar_type());
    const int s = call.rope(dt, q.data_ptr(), step(q, 0), step(q, 1), (int)Hq, ptr(k), step(k, 0), step(k, 1),
                            (int)Hk, T, (int)D, static_cast<const int64_t*>(positions.data_ptr()),
                            static_cast<const double*>(inv_freq.data_ptr()), (int)(2 * inv_freq.size(0)), offset, layout,
                            (float)magnitude, inverse, qo.data_ptr(), step(qo, 0), step(qo, 1), ptr(ko), step(ko, 0), step(ko, 1),
                            on.stream);
    need(s == HQ_OK, s, what);
    return {qo, ko};
}

// ------------------------------------------------------------ slots, cache
std::tuple<Tensor, Tensor, Tensor, Tensor, Tensor, Tensor> kv_slots(const Tensor& lens, const Tensor& add, const Tensor& table,
                                                                    const Tensor& pages, const Tensor& count, int page_size,
                                                                    int64_t n_slots, const Maybe& lens_out,
                                                                    const Maybe& count_out) {
    const char* const what = "kv_slots";
    need(lens.is_cuda() && lens.scalar_type() == at::kInt && fits(add, lens) && fits(table, lens) && fits(pages, lens) &&
             fits(count, lens) && fits(lens_out, lens) && fits(count_out, lens),
         HQ_ERR_UNSUPPORTED, "kv_slots: int32 tensors of one CUDA device are needed");
    need(lens.dim() == 1 && add.sizes() == lens.sizes() && table.dim() == 2 && table.size(0) == lens.size(0) && pages.dim() == 1 &&
             count.numel() == 1 && shaped(lens_out, lens) && (!count_out || count_out->numel() == 1) && n_slots >= 0 && n_slots <= INT32_MAX &&
             lens.size(0) <= INT32_MAX,
         HQ_ERR_SHAPE, "kv_slots: lens and new_tokens are [B], block_table is [B, width], free_count is [1]");
    need(lens.is_contiguous() && add.is_contiguous() && table.is_contiguous() && pages.is_contiguous() && whole(lens_out),
         HQ_ERR_ALIGN, "kv_slots: tensors have to be contiguous");
    const int64_t B = lens.size(0);
    const On on(lens);
    const Tensor words = make({2 * B + 3}, lens, at::kInt), rows = make({2 * n_slots}, lens, at::kLong);
    Tensor cu = part(words, 0, {B + 1}), status = part(words, B + 1, {1});
    Tensor lo = lens_out ? *lens_out : part(words, B + 3, {B}), co = count_out ? *count_out : part(words, B + 2, {1});
    Tensor slots = part(rows, 0, {n_slots}), positions = part(rows, n_slots, {n_slots});
    auto i32 = [](const Tensor& t) { return static_cast<int32_t*>(t.data_ptr()); };
    auto i64 = [](const Tensor& t) { return static_cast<int64_t*>(t.data_ptr()); };
    const int s = call.slots((int)B, i32(lens), i32(add), i32(table), table.size(1), i32(pages), pages.size(0), i32(count), page_size,
                             n_slots, i32(lo), i32(cu), i64(slots), i64(positions), i32(co), i32(status), on.stream);
    need(s == HQ_OK, s, what);
    return {lo, cu, slots, positions, co, status};
}

inline bool cache_shape(const Tensor& c) { return c.dim() == 4 && c.size(3) == HQ_KV4_GROUP_BYTES && c.size(1) <= INT32_MAX; }
inline int cache_page(const Tensor& c) { return (int)std::min<int64_t>(c.size(2) * HQ_KV4_GROUP_TOKENS, INT32_MAX); }

void kv4_append(const Tensor& k, const Tensor& v, const Tensor& slots, const Tensor& cache, int hadamard_n) {
    const char* const what = "kv4_append";
    const int dt = type_of(k.scalar_type());
    untracked("kv4_append records no gradients: call it under torch.no_grad()", k, v);
    need(cache.is_cuda() && cache.scalar_type() == at::kByte && k.device() == cache.device() && dt >= 0 && fits(v, k) &&
             is(slots, k, at::kLong),
         HQ_ERR_UNSUPPORTED, "kv4_append: k and v of one type, int64 slots and a uint8 cache on one CUDA device are needed");
    need(cache_shape(cache) && k.dim() == 3 && k.size(1) == cache.size(1) && k.size(2) == HQ_KV4_HEAD && v.sizes() == k.sizes() &&
             vector_of(slots, k.size(0)),
         HQ_ERR_SHAPE, "kv4_append: k and v are [N, H, 128], slots is [N], the cache [pages, H, page_size / 16, 2432]");
    need(rows_whole(k) && rows_whole(v) && slots.is_contiguous() && cache.is_contiguous(), HQ_ERR_ALIGN,
         "kv4_append: heads, slots and the cache have to be contiguous");
    const On on(cache);
    const int s = call.append(dt, k.data_ptr(), step(k, 0), step(k, 1), v.data_ptr(), step(v, 0), step(v, 1),
                              static_cast<const int64_t*>(slots.data_ptr()), k.size(0), (int)k.size(1), hadamard_n,
                              static_cast<uint8_t*>(cache.data_ptr()), cache.size(0), cache_page(cache), on.stream);
    need(s == HQ_OK, s, what);
}

std::tuple<Tensor, Tensor> kv4_gather(const Tensor& cache, const Tensor& slots, at::ScalarType dtype, int hadamard_n) {
    const char* const what = "kv4_gather";
    const int dt = type_of(dtype);
    need(cache.is_cuda() && cache.scalar_type() == at::kByte && is(slots, cache, at::kLong) && dt >= 0, HQ_ERR_UNSUPPORTED,
         "kv4_gather: int64 slots and a uint8 cache on one CUDA device are needed");
    need(cache_shape(cache) && slots.dim() == 1, HQ_ERR_SHAPE,
         "kv4_gather: slots is [N], the cache [pages, H, page_size / 16, 2432]");
    need(slots.is_contiguous() && cache.is_contiguous(), HQ_ERR_ALIGN, "kv4_gather: slots and the cache have to be contiguous");
    const int64_t N = slots.size(0), H = cache.size(1);
    const On on(cache);
    Tensor k = make({N, H, HQ_KV4_HEAD}, cache, dtype), v = make({N, H, HQ_KV4_HEAD}, cache, dtype);
    const int64_t t = H * HQ_KV4_HEAD;
    const int s = call.gather(dt, static_cast<const uint8_t*>(cache.data_ptr()), cache.size(0), cache_page(cache),
                              static_cast<const int64_t*>(slots.data_ptr()), N, (int)H, hadamard_n, k.data_ptr(), t, HQ_KV4_HEAD,
                              v.data_ptr(), t, HQ_KV4_HEAD, on.stream);
    need(s == HQ_OK, s, what);
    return {k, v};
}

// -------------------------------------------------------------- attention
std::tuple<Tensor, Maybe, Maybe> kv4_attention(const Tensor& q, const Tensor& cache, const Tensor& table, const Tensor& lens,
                                        const Maybe& cu_q, int q_len, std::optional<double> scale, int window, int sinks,
                                        int hadamard_n, const Maybe& ws_in, const Maybe& out_in, bool want_lse, bool want_error) {
    const char* const what = "kv4_attention";
    const int dt = type_of(q.scalar_type());
    untracked("kv4_attention records no gradients: call it under torch.no_grad()", q, out_in);
    need(q.is_cuda() && (dt == HQ_DT_BF16 || dt == HQ_DT_F16) && is(cache, q, at::kByte) && is(table, q, at::kInt) &&
             is(lens, q, at::kInt) && is(cu_q, q, at::kInt) && fits(out_in, q) && (!ws_in || ws_in->device() == q.device()),
         HQ_ERR_UNSUPPORTED, "kv4_attention: BF16 or FP16 q and out, a uint8 cache, int32 tables on one CUDA device are needed");
    need(q.dim() == 3 && q.size(2) == HQ_KV4_HEAD && q.size(1) <= INT32_MAX && cache_shape(cache) && lens.dim() == 1 &&
             table.dim() == 2 && table.size(0) == lens.size(0) && lens.size(0) < INT32_MAX &&
             (!cu_q || vector_of(*cu_q, lens.size(0) + 1)) && shaped(out_in, q),
         HQ_ERR_SHAPE, "kv4_attention: q and out are [Tq, Hq, 128], the cache [pages, Hkv, page_size / 16, 2432], block_table "
                       "[B, width], seq_lens [B], cu_q [B + 1]");
    need(rows_whole(q) && rows_whole(out_in) && cache.is_contiguous() && table.is_contiguous() && lens.is_contiguous() &&
             whole(cu_q) && whole(ws_in),
         HQ_ERR_ALIGN, "kv4_attention: heads, the cache, tables and the workspace have to be contiguous");
    const int64_t Tq = q.size(0), Hq = q.size(1);
    const On on(q);
    Tensor out = out_in ? *out_in : make({Tq, Hq, HQ_KV4_HEAD}, q, q.scalar_type());
    Maybe lse, error, ws = ws_in;
    if (want_lse) lse = make({Tq, Hq}, q, at::kFloat);
    if (!ws) {
        ws = make({(int64_t)call.attention_ws()}, q, at::kByte);
        const int s = call.ws_init(ws->data_ptr(), HQ_KV4_ATTENTION_STATE_BYTES, on.stream);
        need(s == HQ_OK, s, what);
    }
    const int s = call.attention(dt, q.data_ptr(), step(q, 0), step(q, 1), Tq, (int)Hq, static_cast<const uint8_t*>(cache.data_ptr()),
                                 cache.size(0), cache_page(cache), (int)cache.size(1), static_cast<const int32_t*>(table.data_ptr()),
                                 table.size(1), (int)lens.size(0), static_cast<const int32_t*>(lens.data_ptr()),
                                 static_cast<const int32_t*>(ptr(cu_q)), q_len,
                                 scale ? (float)*scale : 0.08838834764831845f /* 1 / sqrt(128) */, window, sinks, hadamard_n,
                                 out.data_ptr(), step(out, 0), step(out, 1), static_cast<float*>(ptr(lse)), ws->data_ptr(),
                                 ws->nbytes(), on.stream);
    need(s == HQ_OK, s, what);
    if (want_error) {  // (a copy: the caller need not keep the workspace, nor does the next call change it)
        error = make({1}, q, at::kInt);
        error->copy_(at::from_blob(static_cast<char*>(ws->data_ptr()) + 8, {1}, error->options()));
    }
    return {out, lse, error};
}

}  // namespace

PYBIND11_MODULE(_hq_torch, m) {
    py::register_exception_translator([](std::exception_ptr p) {
        try {
            if (p) std::rethrow_exception(p);
        } catch (const Refusal& r) {
            const py::object type = py::module_::import("nvfp4_quantization_group_b200").attr("HQError");
            const py::object error = type(r.status, r.what);
            PyErr_SetObject(type.ptr(), error.ptr());
        } catch (const c10::OutOfMemoryError& e) {
            PyErr_SetString(py::module_::import("torch").attr("OutOfMemoryError").ptr(), e.what_without_backtrace());
        }
    });
    // (the allocator may wait for the device: other Python threads run meanwhile)
    const py::call_guard<py::gil_scoped_release> free;
    m.attr("built_for") = HQ_BUILT_FOR;  // (the build looks for it in the file)
    m.def("bind", &bind);
    m.def("add_rmsnorm", &add_rmsnorm, free);
    m.def("rmsnorm_backward", &rmsnorm_backward, free);
    m.def("rope", &rope, free);
    m.def("kv_slots", &kv_slots, free);
    m.def("kv4_append", &kv4_append, free);
    m.def("kv4_gather", &kv4_gather, free);
    m.def("kv4_attention", &kv4_attention, free);
}
