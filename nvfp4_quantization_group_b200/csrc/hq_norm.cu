// hq_norm.cu -- residual addition + RMS norm + K128 FP8 codes, and the norm's
// gradients (sm_100a).
#include "hq_layer.cuh"

namespace hq {

constexpr int NORM_THREADS = 256;

// Sum over the block (every thread gets it); one barrier before the read, one
// after, so that it can be called again.
__device__ __forceinline__ float block_sum(float v, float* red) {
    v = warp_sum(v);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.0f;
    for (int i = 0; i < (int)blockDim.x / 32; ++i) s = __fadd_rn(s, red[i]);
    __syncthreads();
    return s;
}

// One block per row; a half-warp holds one group of 128 columns (16 lanes x 8).
template <int DT, int WDT>
__global__ void __launch_bounds__(NORM_THREADS) add_rmsnorm_fp8_kernel(NormParams p) {
    __shared__ float red[32];
    const int64_t m = blockIdx.x;
    const int chunks = (int)(p.K / 8), l = threadIdx.x & 15;
    float sum = 0.0f;
    for (int c = threadIdx.x; c < chunks; c += NORM_THREADS) {
        float h[8];
        unpack8<DT>(load_chunk<DT>(p.x, m * p.x_stride + 8 * c), h);
        if (p.r) {
            float r[8];
            unpack8<DT>(load_chunk<DT>(p.r, m * p.r_stride + 8 * c), r);
#pragma unroll
            for (int i = 0; i < 8; ++i) h[i] = __fadd_rn(h[i], r[i]);
            const Chunk<DT> hc = pack8<DT>(h);
            store_chunk<DT>(p.h, m * p.K + 8 * c, hc);
            unpack8<DT>(hc, h);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = __fmaf_rn(h[i], h[i], sum);
    }
    sum = block_sum(sum, red);
    const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(sum, (float)p.K), p.eps)));
    if (p.rstd && threadIdx.x == 0) p.rstd[m] = rstd;
    const int rounds = (chunks + NORM_THREADS - 1) / NORM_THREADS;
    for (int j = 0; j < rounds; ++j) {
        const int c = j * NORM_THREADS + threadIdx.x;
        const bool ok = c < chunks;  // the same for all lanes of a half-warp
        float y[8] = {};
        if (ok) {
            float w[8];
            // h as the first loop wrote it (the same thread), or x
            unpack8<DT>(p.r ? load_chunk<DT>(p.h, m * p.K + 8 * c) : load_chunk<DT>(p.x, m * p.x_stride + 8 * c), y);
            unpack8<WDT>(load_chunk<WDT>(p.w, 8 * c), w);
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = __fmul_rn(__fmul_rn(y[i], rstd), w[i]);
        }
        float a = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) a = absmax3(a, y[2 * i], y[2 * i + 1]);
#pragma unroll
        for (int o = 8; o >= 1; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
        if (!ok) continue;
        const float s = p.ue8m0 ? ue8m0_up(fp8_group_scale(a)) : fp8_group_scale(a);
        *reinterpret_cast<uint2*>(p.out + m * p.K + 8 * c) = fp8_codes8(y, s);
        if (l == 0) {
            const int64_t at = p.transposed ? (c / 16) * p.scale_ld + m : m * (p.K / 128) + c / 16;
            p.scales[at] = s;
            if (p.amax) p.amax[at] = a;
        }
    }
}

// dx, one block per row.
template <int DT, int WDT>
__global__ void __launch_bounds__(NORM_THREADS) rmsnorm_dx_kernel(NormBackParams p) {
    __shared__ float red[32];
    const int64_t m = blockIdx.x;
    const int chunks = (int)(p.K / 8);
    float sum = 0.0f;
    for (int c = threadIdx.x; c < chunks; c += NORM_THREADS) {
        float g[8], h[8], w[8];
        unpack8<DT>(load_chunk<DT>(p.dy, m * p.dy_stride + 8 * c), g);
        unpack8<DT>(load_chunk<DT>(p.h, m * p.h_stride + 8 * c), h);
        unpack8<WDT>(load_chunk<WDT>(p.w, 8 * c), w);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = __fmaf_rn(__fmul_rn(g[i], w[i]), h[i], sum);
    }
    sum = block_sum(sum, red);
    const float rstd = p.rstd[m];
    const float c1 = __fmul_rn(__fmul_rn(rstd, rstd), __fdiv_rn(sum, (float)p.K));
    for (int c = threadIdx.x; c < chunks; c += NORM_THREADS) {
        float g[8], h[8], w[8], d[8] = {};
        unpack8<DT>(load_chunk<DT>(p.dy, m * p.dy_stride + 8 * c), g);
        unpack8<DT>(load_chunk<DT>(p.h, m * p.h_stride + 8 * c), h);
        unpack8<WDT>(load_chunk<WDT>(p.w, 8 * c), w);
        if (p.dres) unpack8<DT>(load_chunk<DT>(p.dres, m * p.dres_stride + 8 * c), d);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = __fmaf_rn(rstd, __fmaf_rn(-h[i], c1, __fmul_rn(g[i], w[i])), d[i]);
        store_chunk<DT>(p.dx, m * p.K + 8 * c, pack8<DT>(d));
    }
}

// dweight, one thread per column, rows in order.
template <int DT> __global__ void rmsnorm_dw_kernel(NormBackParams p) {
    const int64_t k = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (k >= p.K) return;
    const typename Elem<DT>::T* dy = static_cast<const typename Elem<DT>::T*>(p.dy);
    const typename Elem<DT>::T* h = static_cast<const typename Elem<DT>::T*>(p.h);
    float s = 0.0f;
    for (int64_t m = 0; m < p.M; ++m)
        s = __fmaf_rn(to_f32(dy[m * p.dy_stride + k]), __fmul_rn(to_f32(h[m * p.h_stride + k]), p.rstd[m]), s);
    p.dw[k] = s;
}

template <int DT, int WDT> static void norm_t(const NormParams& p, cudaStream_t st) {
    add_rmsnorm_fp8_kernel<DT, WDT><<<(unsigned)p.M, NORM_THREADS, 0, st>>>(p);
}
void launch_norm(int dtype, int w_dtype, const NormParams& p, int sms, cudaStream_t st) {
    (void)sms;
    if (dtype == HQ_DT_F32) norm_t<HQ_DT_F32, HQ_DT_F32>(p, st);
    else if (dtype == HQ_DT_BF16) w_dtype == HQ_DT_F32 ? norm_t<HQ_DT_BF16, HQ_DT_F32>(p, st) : norm_t<HQ_DT_BF16, HQ_DT_BF16>(p, st);
    else w_dtype == HQ_DT_F32 ? norm_t<HQ_DT_F16, HQ_DT_F32>(p, st) : norm_t<HQ_DT_F16, HQ_DT_F16>(p, st);
}

size_t norm_back_partial_floats(int64_t M, int64_t K) {
    (void)M;
    (void)K;
    return 4;
}
template <int DT, int WDT> static void norm_back_t(const NormBackParams& p, cudaStream_t st) {
    // dw first: dx may be written over dy
    if (p.dw) rmsnorm_dw_kernel<DT><<<(unsigned)((p.K + 127) / 128), 128, 0, st>>>(p);
    if (p.M > 0) rmsnorm_dx_kernel<DT, WDT><<<(unsigned)p.M, NORM_THREADS, 0, st>>>(p);
}
void launch_norm_back(int dtype, int w_dtype, const NormBackParams& p, int sms, cudaStream_t st) {
    (void)sms;
    if (dtype == HQ_DT_F32) norm_back_t<HQ_DT_F32, HQ_DT_F32>(p, st);
    else if (dtype == HQ_DT_BF16) w_dtype == HQ_DT_F32 ? norm_back_t<HQ_DT_BF16, HQ_DT_F32>(p, st) : norm_back_t<HQ_DT_BF16, HQ_DT_BF16>(p, st);
    else w_dtype == HQ_DT_F32 ? norm_back_t<HQ_DT_F16, HQ_DT_F32>(p, st) : norm_back_t<HQ_DT_F16, HQ_DT_F16>(p, st);
}

}  // namespace hq
