// hq_rope.cu -- rotary positions of q and k in one launch (sm_100a).
//
// Pair i of a token's every head turns by the same angle, position *
// inv_freq[i]: a block takes a few tokens, one thread per (token, pair) forms
// cosine and sine once into shared memory, and the heads stream past them.
// Bound by the bytes, each read and written once in 16-byte pieces.
#include "hq_layer.cuh"

namespace hq {

constexpr int ROPE_THREADS = 256;

// cos and sin of position * inv_freq, the angle reduced to turns in FP64: the
// product keeps 53 bits, so its distance to the nearest whole turn is good to
// |turns| 2^-52, and only that distance is rounded to FP32.
__device__ __forceinline__ float2 rope_cos_sin(int64_t pos, double inv_freq, float magnitude, bool inverse) {
    const double turns = (double)pos * (inv_freq * 0.15915494309189533577);
    const float t = (float)(turns - rint(turns));
    float s, c;
    sincospif(2.0f * t, &s, &c);
    return make_float2(__fmul_rn(c, magnitude), __fmul_rn(inverse ? -s : s, magnitude));
}

__device__ __forceinline__ void rope_turn(float& u, float& v, float2 r) {
    const float a = __fsub_rn(__fmul_rn(u, r.x), __fmul_rn(v, r.y));
    v = __fadd_rn(__fmul_rn(u, r.y), __fmul_rn(v, r.x));
    u = a;
}

// Quotient and remainder by a divisor below 2^16 with m = floor((2^32 - 1) / d).
__device__ __forceinline__ uint32_t rope_div(uint32_t x, uint32_t d, uint32_t m, uint32_t& r) {
    uint32_t q = __umulhi(x, m);
    r = x - q * d;
    while (r >= d) {
        ++q;
        r -= d;
    }
    return q;
}

// ------------------------------------------------------------- wide chunks
// TT tokens a block (blockIdx.x), the heads' units split over blockIdx.y.  A
// unit is 8 pairs (two chunks of 8 elements, HALVES), 4 pairs (one chunk,
// INTERLEAVED) or a chunk passed through; a thread has UN of them in flight.
template <int DT, bool INTER, int TT>
__global__ void __launch_bounds__(ROPE_THREADS) rope_vec_kernel(RopeParams p) {
    constexpr int UN = DT == HQ_DT_F32 ? 2 : 4;
    extern __shared__ float2 cs[];  // [TT][R / 2]
    const int half = p.R / 2;
    const int64_t t0 = (int64_t)blockIdx.x * TT;
    const int tokens = p.T - t0 < TT ? (int)(p.T - t0) : TT;
    for (int n = threadIdx.x; n < tokens * half; n += ROPE_THREADS) {
        const int t = n / half, i = n - t * half;
        cs[n] = rope_cos_sin(p.pos[t0 + t], p.inv_freq[i], p.magnitude, p.inverse != 0);
    }
    __syncthreads();
    const uint32_t turned = INTER ? p.R / 8 : p.R / 16, before = p.offset / 8;
#pragma unroll 1
    for (int z = 0; z < 2; ++z) {
        const RopeTensor& x = p.t[z];
        if (x.heads == 0) continue;
        const uint32_t per_head = turned + (x.in != x.out ? (p.D - p.R) / 8 : 0);
        const uint32_t per_token = per_head * x.heads, total = per_token * tokens;
        const uint32_t head_m = 0xFFFFFFFFu / per_head, token_m = 0xFFFFFFFFu / per_token;
        for (uint32_t n0 = blockIdx.y * ROPE_THREADS + threadIdx.x; n0 < total; n0 += gridDim.y * ROPE_THREADS * UN) {
            Chunk<DT> a[UN], b[UN];
            int64_t at[UN];   // output element of the first chunk
            int unit[UN];     // unit of the head; token << 16
#pragma unroll
            for (int k = 0; k < UN; ++k) {
                const uint32_t n = n0 + k * gridDim.y * ROPE_THREADS;
                unit[k] = -1;
                if (n >= total) continue;
                uint32_t in_token, u;
                const uint32_t t = TT == 1 ? (in_token = n, 0u) : rope_div(n, per_token, token_m, in_token);
                const uint32_t head = rope_div(in_token, per_head, head_m, u);
                uint32_t e;  // first element
                if (u < turned) e = p.offset + 8 * u;
                else e = u - turned < before ? 8 * (u - turned) : 8 * (u - turned) + p.R;
                const int64_t src = (t0 + t) * x.in_ts + (int64_t)head * x.in_hs + e;
                at[k] = (t0 + t) * x.out_ts + (int64_t)head * x.out_hs + e;
                a[k] = load_chunk<DT>(x.in, src);
                if (!INTER && u < turned) b[k] = load_chunk<DT>(x.in, src + half);
                unit[k] = (int)(t << 16 | u);
            }
#pragma unroll
            for (int k = 0; k < UN; ++k) {
                if (unit[k] < 0) continue;
                const uint32_t u = unit[k] & 0xFFFF, t = (uint32_t)unit[k] >> 16;
                if (u < turned) {
                    float f[8];
                    unpack8<DT>(a[k], f);
                    const float4* r = reinterpret_cast<const float4*>(cs + t * half + (INTER ? 4 : 8) * u);
                    if constexpr (INTER) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float4 v = r[e];
                            rope_turn(f[4 * e], f[4 * e + 1], make_float2(v.x, v.y));
                            rope_turn(f[4 * e + 2], f[4 * e + 3], make_float2(v.z, v.w));
                        }
                    } else {
                        float g[8];
                        unpack8<DT>(b[k], g);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float4 v = r[e];
                            rope_turn(f[2 * e], g[2 * e], make_float2(v.x, v.y));
                            rope_turn(f[2 * e + 1], g[2 * e + 1], make_float2(v.z, v.w));
                        }
                        store_chunk<DT>(x.out, at[k] + half, pack8<DT>(g));
                    }
                    store_chunk<DT>(x.out, at[k], pack8<DT>(f));
                } else {
                    store_chunk<DT>(x.out, at[k], a[k]);
                }
            }
        }
    }
}

// ---------------------------------------------------------- any other shape
// One block per token, one element pair (or one passed-through element) a step.
template <int DT>
__global__ void __launch_bounds__(ROPE_THREADS) rope_kernel(RopeParams p) {
    typedef typename Elem<DT>::T T;
    extern __shared__ float2 cs[];  // [R / 2]
    const int64_t t = blockIdx.x;
    const int half = p.R / 2;
    for (int i = threadIdx.x; i < half; i += ROPE_THREADS)
        cs[i] = rope_cos_sin(p.pos[t], p.inv_freq[i], p.magnitude, p.inverse != 0);
    __syncthreads();
    for (int z = 0; z < 2; ++z) {
        const RopeTensor& x = p.t[z];
        const int rest = x.in != x.out ? p.D - p.R : 0, per_head = half + rest;
        const T* in = static_cast<const T*>(x.in) + t * x.in_ts;
        T* out = static_cast<T*>(x.out) + t * x.out_ts;
        for (int n = threadIdx.x; n < x.heads * per_head; n += ROPE_THREADS) {
            const int head = n / per_head, i = n % per_head;
            const T* a = in + head * x.in_hs;
            T* b = out + head * x.out_hs;
            if (i < half) {
                const int e = p.offset + (p.interleaved ? 2 * i : i), f = e + (p.interleaved ? 1 : half);
                float u = to_f32(a[e]), v = to_f32(a[f]);
                rope_turn(u, v, cs[i]);
                b[e] = from_f32<DT>(u);
                b[f] = from_f32<DT>(v);
            } else {
                const int e = i - half < p.offset ? i - half : i - half + p.R;
                b[e] = a[e];
            }
        }
    }
}

template <int DT, int TT> static void rope_vec(const RopeParams& p, int split, cudaStream_t st) {
    const dim3 grid((unsigned)((p.T + TT - 1) / TT), (unsigned)split);
    const size_t smem = sizeof(float2) * (size_t)(p.R / 2) * TT;
    if (p.interleaved) rope_vec_kernel<DT, true, TT><<<grid, ROPE_THREADS, smem, st>>>(p);
    else rope_vec_kernel<DT, false, TT><<<grid, ROPE_THREADS, smem, st>>>(p);
}
template <int DT> static void rope_t(const RopeParams& p, int sms, cudaStream_t st) {
    if (!p.vec) {
        rope_kernel<DT><<<(unsigned)p.T, ROPE_THREADS, sizeof(float2) * (size_t)(p.R / 2), st>>>(p);
        return;
    }
    // Many tokens: four a block, so that every thread has an angle to form.  Few:
    // the heads of a token over several blocks, up to two per SM.
    if (p.T >= 4 * sms && p.R <= 1024) {
        rope_vec<DT, 4>(p, 1, st);
    } else {
        const int64_t units = ((int64_t)p.t[0].heads + p.t[1].heads) * (p.D / 8);
        int64_t split = (2 * sms + p.T - 1) / p.T, most = (units + ROPE_THREADS - 1) / ROPE_THREADS;
        if (split > most) split = most;
        rope_vec<DT, 1>(p, (int)(split < 1 ? 1 : split), st);
    }
}
void launch_rope(int dtype, const RopeParams& p, int sms, cudaStream_t st) {
    if (dtype == HQ_DT_BF16) rope_t<HQ_DT_BF16>(p, sms, st);
    else if (dtype == HQ_DT_F16) rope_t<HQ_DT_F16>(p, sms, st);
    else rope_t<HQ_DT_F32>(p, sms, st);
}

}  // namespace hq
