// hq_norm.cu -- residual addition + RMS norm + K128 FP8 codes, and the norm's
// gradients (sm_100a).
//
// Forward, per row: h = RN(x + r), rstd = 1 / sqrt(mean(h^2) + eps),
// y = (h rstd) w, then the K128 FP8 rule.  Backward, per row: g = dy w,
// c = rstd^2 mean(g h), dx = rstd (g - h c) + dres, and over the rows
// dw = sum dy h rstd.  A handful of operations per element: bound by the bytes.
// Up to K = 8192 every input byte is read once and every output byte written once: a
// row stays in registers between its sum and its second use, and the loads of a
// thread's next row are in flight meanwhile.  Longer rows are held too, but nothing is
// loaded ahead and part of them spills (forward 220 to 1472 bytes a thread; the
// gradients up to 352 at 16384, 1.7 to 2.6 KB beyond), and beyond 16384 the gradients
// read dy and h twice.  Times are of thirty replays; called for a second the largest
// cases take 5 to 15 % more (the clocks go down).
#include "hq_layer.cuh"

namespace hq {

// Sum over the block of one value per thread; every thread gets it.  `red` has
// one float per warp; two of them are used in turn (one barrier per sum).
__device__ __forceinline__ float block_sum(float v, float* red) {
    v = warp_sum(v);
    const int w = threadIdx.x >> 5, n = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) red[w] = v;
    __syncthreads();
    v = (threadIdx.x & 31) < n ? red[threadIdx.x & 31] : 0.0f;
    return warp_sum(v);
}

// ----------------------------------------------------------------- forward
// A row is held by a warp (WARP) or a block of at most T threads, J chunks of
// 8 columns a thread, chunk j of thread i being i + j * threads: a half-warp
// holds one group of 128 columns.
template <int DT, int WDT, int J, int T, int MINB, bool WARP, bool AHEAD>
__global__ void __launch_bounds__(T, MINB) add_rmsnorm_fp8_kernel(NormParams p) {
    __shared__ float red[2][32];
    const int lane = threadIdx.x & 31, nt = WARP ? 32 : (int)blockDim.x, i = WARP ? lane : (int)threadIdx.x;
    const int chunks = (int)(p.K / 8);
    const int64_t step = WARP ? (int64_t)gridDim.x * (blockDim.x >> 5) : gridDim.x;
    int64_t m = WARP ? (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
    Chunk<WDT> w[J];
    Chunk<DT> x[J], r[J];
#pragma unroll
    for (int j = 0; j < J; ++j)
        if (i + j * nt < chunks) w[j] = load_chunk<WDT>(p.w, 8 * (i + j * nt));
    auto load = [&](int64_t row) {
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int c = i + j * nt;
            if (c < chunks && row < p.M) {
                x[j] = load_chunk<DT>(p.x, row * p.x_stride + 8 * c);
                if (p.r) r[j] = load_chunk<DT>(p.r, row * p.r_stride + 8 * c);
            }
        }
    };
    load(m);
    const float inv_k = 1.0f / (float)p.K;
    for (int k = 0; m < p.M; m += step, k ^= 1) {
        Chunk<DT> h[J];
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int c = i + j * nt;
            if (c >= chunks) continue;
            float a[8];
            unpack8<DT>(x[j], a);
            h[j] = x[j];
            if (p.r) {
                float b[8];
                unpack8<DT>(r[j], b);
#pragma unroll
                for (int e = 0; e < 8; ++e) a[e] = __fadd_rn(a[e], b[e]);
                h[j] = pack8<DT>(a);
                store_chunk<DT>(p.h, m * p.K + 8 * c, h[j]);
                unpack8<DT>(h[j], a);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) sum = __fmaf_rn(a[e], a[e], sum);
        }
        if constexpr (AHEAD) load(m + step);
        sum = WARP ? warp_sum(sum) : block_sum(sum, red[k]);
        const float rstd = __frsqrt_rn(__fmaf_rn(sum, inv_k, p.eps));
        if (p.rstd && i == 0) p.rstd[m] = rstd;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int c = i + j * nt;
            const bool ok = c < chunks;  // the same for all lanes of a half-warp
            float y[8] = {};
            if (ok) {
                float v[8];
                unpack8<DT>(h[j], y);
                unpack8<WDT>(w[j], v);
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = __fmul_rn(__fmul_rn(y[e], rstd), v[e]);
            }
            float a = 0.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e) a = absmax3(a, y[2 * e], y[2 * e + 1]);
#pragma unroll
            for (int o = 8; o >= 1; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
            if (!ok) continue;
            const float s = p.ue8m0 ? ue8m0_up(fp8_group_scale(a)) : fp8_group_scale(a);
            *reinterpret_cast<uint2*>(p.out + m * p.K + 8 * c) = fp8_codes8(y, s);
            if ((lane & 15) == 0) {
                const int64_t at = p.transposed ? (int64_t)(c >> 4) * p.scale_ld + m : m * (chunks >> 4) + (c >> 4);
                p.scales[at] = s;
                if (p.amax) p.amax[at] = a;
            }
        }
        if constexpr (!AHEAD) load(m + step);
    }
}

template <int DT, int WDT, int J, int T, int MINB, bool WARP, bool AHEAD>
static void norm_launch(const NormParams& p, int threads, int sms, cudaStream_t st) {
    auto kernel = add_rmsnorm_fp8_kernel<DT, WDT, J, T, MINB, WARP, AHEAD>;
    static std::atomic<int> per_sm{0};  // resident blocks of T threads (the same on every sm_100a GPU)
    if (!per_sm) {
        int n = 0;
        per_sm = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, T, 0) == cudaSuccess && n > 0 ? n : 1;
    }
    const int rows = WARP ? threads / 32 : 1;
    const int64_t blocks = (p.M + rows - 1) / rows, cap = (int64_t)sms * per_sm * (T / threads);
    kernel<<<(unsigned)(blocks < cap ? blocks : cap), threads, 0, st>>>(p);
}

// Who holds a row.  Few rows: one chunk a thread, for the shortest chain.  Many:
// two chunks a thread with two blocks of 512 threads an SM, so that 57 KB of the
// next rows are in flight on each while one is worked on ([16384, 7168] BF16 with
// a residual: 148 us, 5.6 TB/s; four chunks in blocks of 256 179 us, without the
// loads ahead 196 us, one chunk in blocks of 1024 204 us).  An FP32 weight leaves
// room for one block an SM: 273 us there; FP32 rows [8192, 7168] 170 us for 118 of
// copying.  [8192, 16384] BF16 255 us for 146, FP32 [4096, 16384] 302 for 135.
template <int DT, int WDT> static void norm_t(const NormParams& p, int sms, cudaStream_t st) {
    constexpr int TWO = DT == HQ_DT_F32 || WDT == HQ_DT_F32 ? 1 : 2;  // (FP32 chunks need the registers of both)
    const int chunks = (int)(p.K / 8);
    auto block = [&](int j) { return ((chunks + j - 1) / j + 31) / 32 * 32; };
    if (chunks <= 128 && p.M > sms)
        norm_launch<DT, WDT, 4, 256, 1, true, true>(p, 256, sms, st);
    else if (chunks <= 1024 && p.M <= 2 * sms)
        norm_launch<DT, WDT, 1, 1024, 1, false, false>(p, block(1), sms, st);
    else if (chunks <= 1024)
        norm_launch<DT, WDT, 2, 512, TWO, false, true>(p, block(2), sms, st);
    else if (chunks <= 4096)
        norm_launch<DT, WDT, 8, 512, 1, false, false>(p, block(8), sms, st);
    else
        norm_launch<DT, WDT, 8, 1024, 1, false, false>(p, block(8), sms, st);
}
void launch_norm(int dtype, int w_dtype, const NormParams& p, int sms, cudaStream_t st) {
    const bool wf = w_dtype == HQ_DT_F32;
    if (dtype == HQ_DT_F32) norm_t<HQ_DT_F32, HQ_DT_F32>(p, sms, st);
    else if (dtype == HQ_DT_BF16) wf ? norm_t<HQ_DT_BF16, HQ_DT_F32>(p, sms, st) : norm_t<HQ_DT_BF16, HQ_DT_BF16>(p, sms, st);
    else wf ? norm_t<HQ_DT_F16, HQ_DT_F32>(p, sms, st) : norm_t<HQ_DT_F16, HQ_DT_F16>(p, sms, st);
}

// ---------------------------------------------------------------- backward
// Rows of the partial sums of dw: as many as blocks.
constexpr int64_t NORM_PARTS = 592;
size_t norm_back_partial_floats(int64_t M, int64_t K) {
    return (size_t)((M < NORM_PARTS ? M : NORM_PARTS) * K) + 4;
}

// dx, and each block's sum of dw over its rows, in row order.  Rows are held
// as in the forward kernel; a thread keeps the sums of its own columns.
template <int DT, int WDT, int J, int T, int MINB, bool WARP>
__global__ void __launch_bounds__(T, MINB) rmsnorm_back_kernel(NormBackParams p) {
    __shared__ float red[2][32];
    extern __shared__ float sums[];  // WARP: [K]
    const int lane = threadIdx.x & 31, nt = WARP ? 32 : (int)blockDim.x, i = WARP ? lane : (int)threadIdx.x;
    const int chunks = (int)(p.K / 8);
    const int64_t step = WARP ? (int64_t)gridDim.x * (blockDim.x >> 5) : gridDim.x;
    int64_t m = WARP ? (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
    Chunk<WDT> w[J];
    Chunk<DT> dy[J], h[J];
    float dw[J][8];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        if (i + j * nt < chunks) w[j] = load_chunk<WDT>(p.w, 8 * (i + j * nt));
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[j][e] = 0.0f;
    }
    float rstd = 0.0f;
    auto load = [&](int64_t row) {
        if (row >= p.M) return;
        rstd = p.rstd[row];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int c = i + j * nt;
            if (c < chunks) {
                dy[j] = load_chunk<DT>(p.dy, row * p.dy_stride + 8 * c);
                h[j] = load_chunk<DT>(p.h, row * p.h_stride + 8 * c);
            }
        }
    };
    load(m);
    const float inv_k = 1.0f / (float)p.K;
    for (int k = 0; m < p.M; m += step, k ^= 1) {
        Chunk<DT> d[J];
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int c = i + j * nt;
            if (c >= chunks) continue;
            if (p.dres) d[j] = load_chunk<DT>(p.dres, m * p.dres_stride + 8 * c);
            float g[8], a[8], v[8];
            unpack8<DT>(dy[j], g);
            unpack8<DT>(h[j], a);
            unpack8<WDT>(w[j], v);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float t = __fmul_rn(g[e], a[e]);
                dw[j][e] = __fmaf_rn(t, rstd, dw[j][e]);
                sum = __fmaf_rn(t, v[e], sum);
            }
        }
        sum = WARP ? warp_sum(sum) : block_sum(sum, red[k]);
        const float rs = rstd, c1 = __fmul_rn(__fmul_rn(rs, rs), __fmul_rn(sum, inv_k));
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int c = i + j * nt;
            if (c >= chunks) continue;
            float g[8], a[8], v[8], o[8] = {};
            unpack8<DT>(dy[j], g);
            unpack8<DT>(h[j], a);
            unpack8<WDT>(w[j], v);
            if (p.dres) unpack8<DT>(d[j], o);
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = __fmaf_rn(rs, __fmaf_rn(-a[e], c1, __fmul_rn(g[e], v[e])), o[e]);
            store_chunk<DT>(p.dx, m * p.K + 8 * c, pack8<DT>(o));
        }
        load(m + step);
    }
    if (!p.dw) return;
    let_next();
    float* const part = p.partial + (int64_t)blockIdx.x * p.K;
    if constexpr (WARP) {
        for (int x = 0; x < (int)blockDim.x / 32; ++x) {  // the warps in order
            if (x == (int)(threadIdx.x >> 5)) {
#pragma unroll
                for (int j = 0; j < J; ++j)
                    if (i + j * 32 < chunks) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            float& s = sums[8 * (i + j * 32) + e];
                            s = x ? __fadd_rn(s, dw[j][e]) : dw[j][e];
                        }
                    }
            }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < (int)p.K; c += blockDim.x) part[c] = sums[c];
    } else {
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int c = i + j * nt;
            if (c >= chunks) continue;
            float4* o = reinterpret_cast<float4*>(part + 8 * c);
            o[0] = make_float4(dw[j][0], dw[j][1], dw[j][2], dw[j][3]);
            o[1] = make_float4(dw[j][4], dw[j][5], dw[j][6], dw[j][7]);
        }
    }
}

// dw alone, for rows too long to be held: 256 columns a block (blockIdx.x), the
// rows blockIdx.y, + gridDim.y, ...
template <int DT> __global__ void __launch_bounds__(256) rmsnorm_dw_kernel(NormBackParams p) {
    typedef typename Elem<DT>::T E;
    const int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (k >= p.K) return;
    const E* dy = static_cast<const E*>(p.dy);
    const E* h = static_cast<const E*>(p.h);
    float s = 0.0f;
    for (int64_t m = blockIdx.y; m < p.M; m += gridDim.y)
        s = __fmaf_rn(__fmul_rn(to_f32(dy[m * p.dy_stride + k]), to_f32(h[m * p.h_stride + k])), p.rstd[m], s);
    p.partial[(int64_t)blockIdx.y * p.K + k] = s;
}

// Sum of `parts` rows of partial sums: 32 columns a block, thread row y takes
// rows y, y + 32, ... (eight of them in flight), then the 32 of them in order.
__global__ void __launch_bounds__(1024) rmsnorm_dw_join_kernel(const float* partial, float* dw, int64_t K, int parts) {
    __shared__ float s[32][33];
    const int64_t k = (int64_t)blockIdx.x * 32 + threadIdx.x;
    float a = 0.0f;
    after_previous();
    for (int r0 = threadIdx.y; r0 < parts; r0 += 32 * 8) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int r = r0 + 32 * j;
            v[j] = r < parts ? __ldcg(partial + (int64_t)r * K + k) : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) a = __fadd_rn(a, v[j]);
    }
    s[threadIdx.y][threadIdx.x] = a;
    __syncthreads();
    const float b = warp_sum(s[threadIdx.x][threadIdx.y]);  // column y's 32 sums
    if (threadIdx.x == 0) dw[(int64_t)blockIdx.x * 32 + threadIdx.y] = b;
}

template <int DT, int WDT, int J, int T, int MINB, bool WARP>
static int norm_back_launch(const NormBackParams& p, int threads, int sms, cudaStream_t st) {
    auto kernel = rmsnorm_back_kernel<DT, WDT, J, T, MINB, WARP>;
    static std::atomic<int> per_sm{0};
    if (!per_sm) {
        int n = 0;
        per_sm = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, T, 0) == cudaSuccess && n > 0 ? n : 1;
    }
    const int rows = WARP ? threads / 32 : 1;
    const int64_t blocks = (p.M + rows - 1) / rows;
    int64_t cap = (int64_t)sms * per_sm * (T / threads);
    if (cap > NORM_PARTS) cap = NORM_PARTS;
    const int grid = (int)(blocks < cap ? blocks : cap);
    kernel<<<grid, threads, WARP ? sizeof(float) * (size_t)p.K : 0, st>>>(p);
    return grid;
}
// Two chunks a thread and two blocks of 512 threads an SM ([8191, 4096] BF16 with
// dres: 52 us, 5.2 TB/s; one block an SM 61 us, four chunks a thread 54 us, one 72 us;
// FP32 100 us for 83 of copying).  [4096, 16384] 104 us for 83 in BF16, 307 for 166 in
// FP32; [2048, 32768] BF16 582 for 83.
template <int DT, int WDT> static void norm_back_t(const NormBackParams& p, int sms, cudaStream_t st) {
    constexpr int TWO = DT == HQ_DT_F32 || WDT == HQ_DT_F32 ? 1 : 2;
    const int chunks = (int)(p.K / 8);
    auto block = [&](int j) { return ((chunks + j - 1) / j + 31) / 32 * 32; };
    int parts = 0;
    if (p.M == 0) {
        cudaMemsetAsync(p.dw, 0, sizeof(float) * (size_t)p.K, st);
        return;
    }
    if (chunks <= 64) {
        parts = norm_back_launch<DT, WDT, 2, 256, 1, true>(p, 256, sms, st);
    } else if (chunks <= 1024) {
        parts = norm_back_launch<DT, WDT, 2, 512, TWO, false>(p, block(2), sms, st);
    } else if (chunks <= 2048) {
        parts = norm_back_launch<DT, WDT, 4, 512, 1, false>(p, block(4), sms, st);
    } else {
        // (a row's sums of dw do not fit in registers; dx, which may be dy, is
        // written after dw has been taken)
        parts = (int)(p.M < 64 ? p.M : 64);
        if (p.dw)
            rmsnorm_dw_kernel<DT><<<dim3((unsigned)((p.K + 255) / 256), (unsigned)parts), 256, 0, st>>>(p);
        NormBackParams q = p;
        q.dw = nullptr;
        norm_back_launch<DT, WDT, 8, 1024, 1, false>(q, block(8), sms, st);
    }
    if (p.dw) launch_next(rmsnorm_dw_join_kernel, dim3((unsigned)(p.K / 32)), dim3(32, 32), 0, st, p.partial, p.dw, p.K, parts);
}
void launch_norm_back(int dtype, int w_dtype, const NormBackParams& p, int sms, cudaStream_t st) {
    const bool wf = w_dtype == HQ_DT_F32;
    if (dtype == HQ_DT_F32) norm_back_t<HQ_DT_F32, HQ_DT_F32>(p, sms, st);
    else if (dtype == HQ_DT_BF16) wf ? norm_back_t<HQ_DT_BF16, HQ_DT_F32>(p, sms, st) : norm_back_t<HQ_DT_BF16, HQ_DT_BF16>(p, sms, st);
    else wf ? norm_back_t<HQ_DT_F16, HQ_DT_F32>(p, sms, st) : norm_back_t<HQ_DT_F16, HQ_DT_F16>(p, sms, st);
}

}  // namespace hq
