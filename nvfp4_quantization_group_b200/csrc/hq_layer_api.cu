// hq_layer_api.cu -- extern "C" entry points of the attention-layer calls of
// include/hq.h: argument checks, parameter blocks, launches.  No allocation, no
// synchronization, no environment reads.
#include <math.h>
#include <string.h>

#include <mutex>

#include "hq_layer.h"

using namespace hq;

namespace hq {

int device_sms() {
    constexpr int kMaxDevices = 64;
    static int sms[kMaxDevices];
    static std::once_flag once[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
    std::call_once(once[dev], [dev] {
        if (cudaDeviceGetAttribute(&sms[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) sms[dev] = 0;
    });
    return sms[dev];
}

}  // namespace hq

namespace {

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool known_type(int t) { return t == HQ_DT_BF16 || t == HQ_DT_F16 || t == HQ_DT_F32; }
inline uintptr_t type_bytes(int t) { return t == HQ_DT_F32 ? 4 : 2; }
inline hq_status launch_status() {
    return cudaPeekAtLastError() == cudaSuccess ? HQ_OK : (cudaGetLastError(), HQ_ERR_CUDA);
}
constexpr int64_t kMaxRows = ((int64_t)1 << 31) - 1;

int page_shift_of(int page_size) {  // -1: not a power of two from 16 to 1024
    for (int s = 4; s <= 10; ++s)
        if (page_size == 1 << s) return s;
    return -1;
}

}  // namespace

extern "C" {

// ------------------------------------------------------------------- norm
hq_status hq_add_rmsnorm_fp8_k128(int dtype, const void* x, int64_t x_row_stride, const void* residual,
                                  int64_t residual_row_stride, const void* weight, int w_dtype, float eps, int64_t M,
                                  int64_t K, void* residual_out, uint8_t* out_fp8, float* scales, int scale_layout,
                                  int64_t scale_ld, float* rstd_opt, float* amax_opt, void* stream) {
    const bool ue8m0 = (scale_layout & HQ_FP8_UE8M0) != 0;
    scale_layout &= ~HQ_FP8_UE8M0;
    if (!known_type(dtype) || (w_dtype != dtype && w_dtype != HQ_DT_F32)) return HQ_ERR_UNSUPPORTED;
    if (scale_layout != HQ_SCALE_ROWMAJOR && scale_layout != HQ_SCALE_TRANSPOSED) return HQ_ERR_UNSUPPORTED;
    if (!(eps >= 0.0f)) return HQ_ERR_UNSUPPORTED;
    if (M < 0 || M > kMaxRows || K <= 0 || K > HQ_NORM_MAX_K) return HQ_ERR_SHAPE;
    if (K % 128) return HQ_ERR_ALIGN;
    if (M == 0) return HQ_OK;
    if (!x || !weight || !out_fp8 || !scales || (residual && !residual_out)) return HQ_ERR_NULL;
    if (x_row_stride < K || (residual && residual_row_stride < K)) return HQ_ERR_SHAPE;
    if (scale_layout == HQ_SCALE_TRANSPOSED && scale_ld < M) return HQ_ERR_SHAPE;
    if (residual && ((residual_out == x && x_row_stride != K) || (residual_out == residual && residual_row_stride != K)))
        return HQ_ERR_SHAPE;
    if (x_row_stride % 8 || (residual && residual_row_stride % 8)) return HQ_ERR_ALIGN;
    if (!aligned(x, 16) || !aligned(weight, 16) || !aligned(out_fp8, 16) || !aligned(scales, 4) ||
        !aligned(rstd_opt, 4) || !aligned(amax_opt, 4) || (residual && (!aligned(residual, 16) || !aligned(residual_out, 16))))
        return HQ_ERR_ALIGN;
    const int sms = device_sms();
    if (!sms) return HQ_ERR_CUDA;
    NormParams p;
    p.x = x;
    p.r = residual;
    p.w = weight;
    p.x_stride = x_row_stride;
    p.r_stride = residual_row_stride;
    p.M = M;
    p.K = K;
    p.eps = eps;
    p.h = residual ? residual_out : nullptr;
    p.out = out_fp8;
    p.scales = scales;
    p.rstd = rstd_opt;
    p.amax = amax_opt;
    p.scale_ld = scale_ld;
    p.transposed = scale_layout == HQ_SCALE_TRANSPOSED;
    p.ue8m0 = ue8m0;
    launch_norm(dtype, w_dtype, p, sms, (cudaStream_t)stream);
    return launch_status();
}

size_t hq_rmsnorm_backward_workspace_size(int64_t M, int64_t K) {
    if (M < 0 || M > kMaxRows || K <= 0 || K > HQ_NORM_MAX_K || K % 128) return 0;
    return (norm_back_partial_floats(M, K) * sizeof(float) + 255) & ~(size_t)255;
}

hq_status hq_rmsnorm_backward(int dtype, const void* dy, int64_t dy_row_stride, const void* h, int64_t h_row_stride,
                              const void* weight, int w_dtype, const float* rstd, const void* dres,
                              int64_t dres_row_stride, int64_t M, int64_t K, void* dx, float* dweight, void* ws,
                              size_t ws_bytes, void* stream) {
    if (!known_type(dtype) || (w_dtype != dtype && w_dtype != HQ_DT_F32)) return HQ_ERR_UNSUPPORTED;
    if (M < 0 || M > kMaxRows || K <= 0 || K > HQ_NORM_MAX_K) return HQ_ERR_SHAPE;
    if (K % 128) return HQ_ERR_ALIGN;
    if (M == 0 && !dweight) return HQ_OK;
    if (M > 0 && (!dy || !h || !weight || !rstd || !dx)) return HQ_ERR_NULL;
    if (dweight && !ws) return HQ_ERR_NULL;
    if (M > 0 && (dy_row_stride < K || h_row_stride < K || (dres && dres_row_stride < K))) return HQ_ERR_SHAPE;
    if (M > 0 && ((dx == dy && dy_row_stride != K) || (dres && dx == dres && dres_row_stride != K))) return HQ_ERR_SHAPE;
    if (dy_row_stride % 8 || h_row_stride % 8 || (dres && dres_row_stride % 8)) return HQ_ERR_ALIGN;
    if (!aligned(dy, 16) || !aligned(h, 16) || !aligned(weight, 16) || !aligned(dx, 16) || !aligned(dres, 16) ||
        !aligned(rstd, 4) || !aligned(dweight, 16) || !aligned(ws, 16))
        return HQ_ERR_ALIGN;
    if (dweight && ws_bytes < hq_rmsnorm_backward_workspace_size(M, K)) return HQ_ERR_WORKSPACE;
    const int sms = device_sms();
    if (!sms) return HQ_ERR_CUDA;
    NormBackParams p;
    p.dy = dy;
    p.h = h;
    p.w = weight;
    p.dres = dres;
    p.rstd = rstd;
    p.dy_stride = dy_row_stride;
    p.h_stride = h_row_stride;
    p.dres_stride = dres_row_stride;
    p.M = M;
    p.K = K;
    p.dx = dx;
    p.dw = dweight;
    p.partial = static_cast<float*>(ws);
    launch_norm_back(dtype, w_dtype, p, sms, (cudaStream_t)stream);
    return launch_status();
}

// ------------------------------------------------------------------- rope
hq_status hq_rope_inv_freq(int rotary_dim, double base, int scaling, double factor, double trained_len, double p1,
                           double p2, double* inv_freq, double* magnitude) {
    const double two_pi = 6.283185307179586477;
    if (scaling < HQ_ROPE_PLAIN || scaling > HQ_ROPE_BANDS) return HQ_ERR_UNSUPPORTED;
    if (!(base > 1.0) || !(factor >= 1.0) || isinf(base) || isinf(factor)) return HQ_ERR_UNSUPPORTED;
    if ((scaling == HQ_ROPE_PARTS || scaling == HQ_ROPE_BANDS) && (!(trained_len > 0.0) || !(p1 > 0.0) || !(p2 > 0.0)))
        return HQ_ERR_UNSUPPORTED;
    if (scaling == HQ_ROPE_PARTS && !(p1 > p2)) return HQ_ERR_UNSUPPORTED;
    if (scaling == HQ_ROPE_BANDS && !(p2 > p1)) return HQ_ERR_UNSUPPORTED;
    if (rotary_dim < 2 || rotary_dim % 2 || (scaling == HQ_ROPE_NTK && rotary_dim < 4)) return HQ_ERR_SHAPE;
    if (!inv_freq) return HQ_ERR_NULL;
    const int half = rotary_dim / 2;
    const double R = rotary_dim;
    if (scaling == HQ_ROPE_NTK) base *= pow(factor, R / (R - 2.0));
    if (magnitude) *magnitude = scaling == HQ_ROPE_PARTS && factor > 1.0 ? 0.1 * log(factor) + 1.0 : 1.0;
    // pair index that turns `turns` times within trained_len
    auto pair_of = [&](double turns) { return R * log(trained_len / (turns * two_pi)) / (2.0 * log(base)); };
    double lo = 0.0, hi = 0.0;
    if (scaling == HQ_ROPE_PARTS) {
        lo = fmax(floor(pair_of(p1)), 0.0);
        hi = fmin(ceil(pair_of(p2)), R - 1.0);
    }
    for (int i = 0; i < half; ++i) {
        const double f = pow(base, -2.0 * i / R);
        double mix = 0.0;  // share of the divided frequency
        if (scaling == HQ_ROPE_LINEAR) mix = 1.0;
        if (scaling == HQ_ROPE_PARTS) mix = fmin(fmax((i - lo) / fmax(hi - lo, 1e-3), 0.0), 1.0);
        if (scaling == HQ_ROPE_BANDS) {
            const double turns = trained_len * f / two_pi;  // trained_len / wavelength
            mix = fmin(fmax((p2 - turns) / (p2 - p1), 0.0), 1.0);
        }
        inv_freq[i] = f / factor * mix + f * (1.0 - mix);
    }
    return HQ_OK;
}

hq_status hq_rope(int dtype, const void* q, int64_t q_token_stride, int64_t q_head_stride, int Hq, const void* k,
                  int64_t k_token_stride, int64_t k_head_stride, int Hk, int64_t T, int D, const int64_t* positions,
                  const double* inv_freq, int rotary_dim, int offset, int layout, float magnitude, int inverse,
                  void* q_out, int64_t q_out_token_stride, int64_t q_out_head_stride, void* k_out,
                  int64_t k_out_token_stride, int64_t k_out_head_stride, void* stream) {
    if (!known_type(dtype)) return HQ_ERR_UNSUPPORTED;
    if (layout != HQ_ROPE_HALVES && layout != HQ_ROPE_INTERLEAVED) return HQ_ERR_UNSUPPORTED;
    if (T < 0 || T > kMaxRows || Hq < 0 || Hk < 0 || Hq > 65535 || Hk > 65535 || D <= 0 || D > 8192) return HQ_ERR_SHAPE;
    if (rotary_dim < 2 || rotary_dim % 2 || offset < 0 || offset > D - rotary_dim) return HQ_ERR_SHAPE;
    if (T == 0 || Hq + Hk == 0) return HQ_OK;
    if ((Hq && (!q || !q_out)) || (Hk && (!k || !k_out)) || !positions || !inv_freq) return HQ_ERR_NULL;
    if ((Hq && q == q_out && (q_token_stride != q_out_token_stride || q_head_stride != q_out_head_stride)) ||
        (Hk && k == k_out && (k_token_stride != k_out_token_stride || k_head_stride != k_out_head_stride)))
        return HQ_ERR_SHAPE;
    const uintptr_t e = type_bytes(dtype);
    if (!aligned(q, e) || !aligned(k, e) || !aligned(q_out, e) || !aligned(k_out, e) || !aligned(positions, 8) ||
        !aligned(inv_freq, 8))
        return HQ_ERR_ALIGN;
    const int sms = device_sms();
    if (!sms) return HQ_ERR_CUDA;
    RopeParams p;
    // (a tensor without heads counts as in place, whatever its pointers: the kernels' units per head depend on it)
    p.t[0] = RopeTensor{q, Hq ? q_out : const_cast<void*>(q), q_token_stride, q_head_stride, q_out_token_stride, q_out_head_stride, Hq};
    p.t[1] = RopeTensor{k, Hk ? k_out : const_cast<void*>(k), k_token_stride, k_head_stride, k_out_token_stride, k_out_head_stride, Hk};
    p.T = T;
    p.D = D;
    p.R = rotary_dim;
    p.offset = offset;
    p.interleaved = layout == HQ_ROPE_INTERLEAVED;
    p.inverse = inverse != 0;
    // whole, aligned chunks of 8 elements everywhere, at most 256 to a head
    p.vec = offset % 8 == 0 && D % 8 == 0 && D <= 2048 && rotary_dim % (p.interleaved ? 8 : 16) == 0;
    for (const RopeTensor& x : p.t)
        if (x.heads)
            p.vec = p.vec && aligned(x.in, 16) && aligned(x.out, 16) && x.in_ts % 8 == 0 && x.in_hs % 8 == 0 &&
                    x.out_ts % 8 == 0 && x.out_hs % 8 == 0;
    p.pos = positions;
    p.inv_freq = inv_freq;
    p.magnitude = magnitude;
    launch_rope(dtype, p, sms, (cudaStream_t)stream);
    return launch_status();
}

// ------------------------------------------------------------ slots, cache
hq_status hq_kv_slots(int B, const int32_t* lens, const int32_t* new_tokens, int32_t* block_table, int64_t table_width,
                      int32_t* free_pages, int64_t free_capacity, const int32_t* free_count, int page_size,
                      int64_t n_slots, int32_t* lens_out, int32_t* cu_new, int64_t* slots, int64_t* positions,
                      int32_t* free_count_out, int32_t* status, void* stream) {
    const int shift = page_shift_of(page_size);
    if (shift < 0) return HQ_ERR_UNSUPPORTED;
    if (B < 0 || B > HQ_KV_MAX_REQUESTS || table_width < 0 || table_width > kMaxRows || free_capacity < 0 ||
        free_capacity > kMaxRows || n_slots < 0 || n_slots > kMaxRows)
        return HQ_ERR_SHAPE;
    if ((B && (!lens || !new_tokens || !lens_out)) || (B && table_width && !block_table) ||
        (free_capacity && !free_pages) || !free_count || !cu_new || (n_slots && (!slots || !positions)) ||
        !free_count_out || !status)
        return HQ_ERR_NULL;
    if (!aligned(lens, 4) || !aligned(new_tokens, 4) || !aligned(block_table, 4) || !aligned(free_pages, 4) ||
        !aligned(free_count, 4) || !aligned(lens_out, 4) || !aligned(cu_new, 4) || !aligned(slots, 8) ||
        !aligned(positions, 8) || !aligned(free_count_out, 4) || !aligned(status, 4))
        return HQ_ERR_ALIGN;
    const int sms = device_sms();
    if (!sms) return HQ_ERR_CUDA;
    SlotParams p;
    p.B = B;
    p.page_shift = shift;
    p.lens = lens;
    p.add = new_tokens;
    p.table = block_table;
    p.width = table_width;
    p.stack = free_pages;
    p.capacity = free_capacity;
    p.count = free_count;
    p.n_slots = n_slots;
    p.lens_out = lens_out;
    p.cu = cu_new;
    p.slots = slots;
    p.positions = positions;
    p.count_out = free_count_out;
    p.status = status;
    launch_slots(p, sms, (cudaStream_t)stream);
    return launch_status();
}

size_t hq_kv4_cache_bytes(int64_t num_pages, int page_size, int H) {
    if (page_shift_of(page_size) < 0 || num_pages <= 0 || num_pages > kMaxRows || H <= 0 || H > 65535) return 0;
    const int64_t per_page = (int64_t)H * (page_size / HQ_KV4_GROUP_TOKENS) * HQ_KV4_GROUP_BYTES;
    if (num_pages > ((int64_t)1 << 32) * HQ_KV4_GROUP_BYTES / per_page - 1) return 0;  // groups have 32-bit numbers
    return (size_t)(num_pages * per_page);
}

// Checks and parameters that append and gather share.
static hq_status kv4_params(int dtype, const void* k, int64_t k_ts, int64_t k_hs, const void* v, int64_t v_ts,
                            int64_t v_hs, const int64_t* slots, int64_t N, int H, int hadamard_n, const uint8_t* cache,
                            int64_t num_pages, int page_size, KvParams& p) {
    if (!known_type(dtype) || (hadamard_n != 0 && hadamard_n != 128)) return HQ_ERR_UNSUPPORTED;
    const int shift = page_shift_of(page_size);
    if (shift < 0) return HQ_ERR_UNSUPPORTED;
    if (N < 0 || N > kMaxRows || H <= 0 || !hq_kv4_cache_bytes(num_pages, page_size, H)) return HQ_ERR_SHAPE;
    if (N == 0) return HQ_OK;
    if (!k || !v || !slots || !cache) return HQ_ERR_NULL;
    if (k_ts % 8 || k_hs % 8 || v_ts % 8 || v_hs % 8) return HQ_ERR_ALIGN;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(cache, 16) || !aligned(slots, 8)) return HQ_ERR_ALIGN;
    p.k = const_cast<void*>(k);
    p.v = const_cast<void*>(v);
    p.k_ts = k_ts;
    p.k_hs = k_hs;
    p.v_ts = v_ts;
    p.v_hs = v_hs;
    p.slots = slots;
    p.N = N;
    p.H = H;
    p.rotate = hadamard_n == 128;
    p.cache = const_cast<uint8_t*>(cache);
    p.n_slots = num_pages << shift;
    p.page_shift = shift;
    p.wide = aligned(k, 32) && aligned(v, 32) && k_ts % 16 == 0 && k_hs % 16 == 0 && v_ts % 16 == 0 && v_hs % 16 == 0;
    return HQ_OK;
}

hq_status hq_kv4_append(int dtype, const void* k, int64_t k_token_stride, int64_t k_head_stride, const void* v,
                        int64_t v_token_stride, int64_t v_head_stride, const int64_t* slots, int64_t N, int H,
                        int hadamard_n, uint8_t* cache, int64_t num_pages, int page_size, void* stream) {
    KvParams p;
    const hq_status r = kv4_params(dtype, k, k_token_stride, k_head_stride, v, v_token_stride, v_head_stride, slots, N,
                                   H, hadamard_n, cache, num_pages, page_size, p);
    if (r != HQ_OK || N == 0) return r;
    const int sms = device_sms();
    if (!sms) return HQ_ERR_CUDA;
    launch_append(dtype, p, sms, (cudaStream_t)stream);
    return launch_status();
}

hq_status hq_kv4_gather(int dtype, const uint8_t* cache, int64_t num_pages, int page_size, const int64_t* slots,
                        int64_t N, int H, int hadamard_n, void* k_out, int64_t k_token_stride, int64_t k_head_stride,
                        void* v_out, int64_t v_token_stride, int64_t v_head_stride, void* stream) {
    KvParams p;
    const hq_status r = kv4_params(dtype, k_out, k_token_stride, k_head_stride, v_out, v_token_stride, v_head_stride,
                                   slots, N, H, hadamard_n, cache, num_pages, page_size, p);
    if (r != HQ_OK || N == 0) return r;
    const int sms = device_sms();
    if (!sms) return HQ_ERR_CUDA;
    launch_gather(dtype, p, sms, (cudaStream_t)stream);
    return launch_status();
}

// -------------------------------------------------------------- attention
size_t hq_kv4_attention_workspace_size(void) { return (attn_workspace_bytes() + 255) & ~(size_t)255; }

hq_status hq_kv4_attention(int dtype, const void* q, int64_t q_token_stride, int64_t q_head_stride, int64_t Tq, int Hq,
                           const uint8_t* cache, int64_t num_pages, int page_size, int Hkv, const int32_t* block_table,
                           int64_t table_width, int B, const int32_t* seq_lens, const int32_t* cu_q, int q_len,
                           float scale, int window, int sinks, int hadamard_n, void* out, int64_t out_token_stride,
                           int64_t out_head_stride, float* lse_opt, void* ws, size_t ws_bytes, void* stream) {
    if (dtype != HQ_DT_BF16 && dtype != HQ_DT_F16) return HQ_ERR_UNSUPPORTED;
    if (hadamard_n != 0 && hadamard_n != 128) return HQ_ERR_UNSUPPORTED;
    const int shift = page_shift_of(page_size);
    if (shift < 0 || window < 0 || sinks < 0 || !(fabsf(scale) <= 1e30f)) return HQ_ERR_UNSUPPORTED;
    if (Tq < 0 || Tq > kMaxRows || B < 0 || B > HQ_KV_MAX_REQUESTS || Hkv <= 0 || Hq <= 0 || Hq % Hkv || q_len < 1 ||
        table_width < 0 || table_width > (1 << 26) || (table_width << shift) > (1 << 30))
        return HQ_ERR_SHAPE;
    if ((int64_t)q_len * (Hq / Hkv) > 65536 || !hq_kv4_cache_bytes(num_pages, page_size, Hkv)) return HQ_ERR_SHAPE;
    if (!cu_q && Tq < (int64_t)B * q_len) return HQ_ERR_SHAPE;
    if (!ws) return HQ_ERR_NULL;
    if (!aligned(ws, 16)) return HQ_ERR_ALIGN;
    if (ws_bytes < hq_kv4_attention_workspace_size()) return HQ_ERR_WORKSPACE;
    if (Tq == 0 || B == 0) return HQ_OK;
    if (!q || !cache || !seq_lens || !out || (table_width && !block_table)) return HQ_ERR_NULL;
    if (q_token_stride % 8 || q_head_stride % 8 || out_token_stride % 8 || out_head_stride % 8) return HQ_ERR_ALIGN;
    if (!aligned(q, 16) || !aligned(cache, 16) || !aligned(out, 16) || !aligned(block_table, 4) ||
        !aligned(seq_lens, 4) || !aligned(cu_q, 4) || !aligned(lse_opt, 4))
        return HQ_ERR_ALIGN;
    const int sms = device_sms();
    if (!sms) return HQ_ERR_CUDA;
    AttnParams p;
    p.q = q;
    p.out = out;
    p.lse = lse_opt;
    p.q_ts = q_token_stride;
    p.q_hs = q_head_stride;
    p.o_ts = out_token_stride;
    p.o_hs = out_head_stride;
    p.Tq = Tq;
    p.cache = cache;
    p.num_pages = num_pages;
    p.table = block_table;
    p.width = table_width;
    p.lens = seq_lens;
    p.cu_q = cu_q;
    p.B = B;
    p.Hkv = Hkv;
    p.group = Hq / Hkv;
    p.q_len = q_len;
    p.page_shift = shift;
    p.scale = scale;
    p.window = window < (1 << 30) ? window : 1 << 30;  // (no token is farther back: position - window stays in 32 bits)
    p.sinks = sinks;
    p.rotate = hadamard_n == 128;
    p.ws = static_cast<uint32_t*>(ws);
    if (launch_attn(dtype, p, sms, (cudaStream_t)stream) != (int)cudaSuccess) return (cudaGetLastError(), HQ_ERR_CUDA);
    return HQ_OK;
}

}  // extern "C"
