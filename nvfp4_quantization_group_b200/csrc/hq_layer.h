// hq_layer.h -- parameter blocks and launchers of the attention-layer calls
// (norm + FP8 codes, rotary positions, slot maps, NVFP4 key/value cache,
// attention over it), shared by hq_layer_api.cu and the kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "hq.h"

namespace hq {

int device_sms();  // SM count of the current device, 0 on failure (hq_layer_api.cu)

// ------------------------------------------------------------------- norm
struct NormParams {
    const void* x;
    const void* r;  // residual or NULL
    const void* w;
    int64_t x_stride, r_stride;  // elements
    int64_t M, K;
    float eps;
    void* h;  // residual_out (NULL without a residual)
    uint8_t* out;
    float* scales;
    float* rstd;  // or NULL
    float* amax;  // or NULL
    int64_t scale_ld;
    int transposed, ue8m0;
};
struct NormBackParams {
    const void *dy, *h, *w, *dres;
    const float* rstd;
    int64_t dy_stride, h_stride, dres_stride;
    int64_t M, K;
    void* dx;
    float* dw;
    float* partial;  // [row blocks, K]
};
void launch_norm(int dtype, int w_dtype, const NormParams& p, int sms, cudaStream_t st);
size_t norm_back_partial_floats(int64_t M, int64_t K);
void launch_norm_back(int dtype, int w_dtype, const NormBackParams& p, int sms, cudaStream_t st);

// ------------------------------------------------------------------- rope
struct RopeTensor {
    const void* in;
    void* out;
    int64_t in_ts, in_hs, out_ts, out_hs;  // token and head strides, elements
    int heads;
};
struct RopeParams {
    RopeTensor t[2];  // q, k
    int64_t T;
    int D, R, offset, interleaved, inverse;
    int vec;  // rows and parts are whole, aligned chunks of 8 elements
    const int64_t* pos;
    const double* inv_freq;
    float magnitude;
};
void launch_rope(int dtype, const RopeParams& p, int sms, cudaStream_t st);

// ------------------------------------------------------------ slots, cache
struct SlotParams {
    int B, page_shift;
    const int32_t *lens, *add;
    int32_t* table;
    int64_t width;
    int32_t* stack;
    int64_t capacity;
    const int32_t* count;
    int64_t n_slots;
    int32_t *lens_out, *cu;
    int64_t *slots, *positions;
    int32_t *count_out, *status;
};
void launch_slots(const SlotParams& p, int sms, cudaStream_t st);

// Byte places inside a 16-token group of one head (see hq.h).
constexpr int KV_K_CODES = 0, KV_V_CODES = 1024, KV_K_SF = 2048, KV_V_SF = 2176, KV_K_DEC = 2304, KV_V_DEC = 2368;
constexpr int KV_GROUP_BYTES = HQ_KV4_GROUP_BYTES;
static_assert(KV_V_DEC + 64 == KV_GROUP_BYTES, "group layout");

struct KvParams {
    void *k, *v;  // append: read; gather: written
    int64_t k_ts, k_hs, v_ts, v_hs;
    const int64_t* slots;
    int64_t N;
    int H;
    int rotate;
    uint8_t* cache;
    int64_t n_slots;  // num_pages * page_size
    int page_shift;
    int wide;  // k and v: 32-byte aligned vectors
};
void launch_append(int dtype, const KvParams& p, int sms, cudaStream_t st);
void launch_gather(int dtype, const KvParams& p, int sms, cudaStream_t st);

// -------------------------------------------------------------- attention
struct AttnParams {
    const void* q;
    void* out;
    float* lse;
    int64_t q_ts, q_hs, o_ts, o_hs, Tq;
    const uint8_t* cache;
    int64_t num_pages;
    const int32_t* table;
    int64_t width;
    const int32_t *lens, *cu_q;
    int B, Hkv, group, q_len, page_shift;
    float scale;
    int window, sinks, rotate;
    uint32_t* ws;  // [2] sticky error word
};
size_t attn_workspace_bytes();
int launch_attn(int dtype, const AttnParams& p, int sms, cudaStream_t st);  // cudaError_t

}  // namespace hq
