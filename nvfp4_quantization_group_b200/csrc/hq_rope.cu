// hq_rope.cu -- rotary positions of q and k in one launch (sm_100a).
//
// Pair i of a token's every head turns by the same angle, position *
// inv_freq[i]: a block takes a few tokens, one thread per (token, pair) forms
// cosine and sine once into shared memory, and the heads stream past them.
// Bound by the bytes, each read and written once in 16-byte pieces: 8192 tokens of
// 64 + 8 BF16 heads of 128 take 56 us, 5.4 TB/s (84 % of the measured copy rate), FP32
// 103 us (91 %); 64 tokens 2.7 us, a launch and one chain of loads.  Shapes without
// whole chunks go element by element: heads of 80 with dimensions 16 to 35 turned take
// 130 us where the bytes need 29, bound by instructions on 2-byte accesses.
#include "hq_layer.cuh"

namespace hq {

constexpr int ROPE_THREADS = 256;

// cos and sin of position * inv_freq, the angle reduced to turns in FP64: the
// product keeps 53 bits, so its distance to the nearest whole turn is good to
// |turns| 2^-52.  That distance is rounded to FP32 (t), and the rest of it (d, in
// radians, below 2 pi 2^-26) put right to first order: cos - d sin, sin + d cos.
__device__ __forceinline__ float2 rope_cos_sin(int64_t pos, double inv_freq, float magnitude, bool inverse) {
    const double turns = (double)pos * (inv_freq * 0.15915494309189533577), part = turns - rint(turns);
    const float t = (float)part, d = (float)(part - (double)t) * 6.2831853f;
    float s, c;
    sincospif(2.0f * t, &s, &c);
    const float c2 = __fmaf_rn(-d, s, c), s2 = __fmaf_rn(d, c, s);
    return make_float2(__fmul_rn(c2, magnitude), __fmul_rn(inverse ? -s2 : s2, magnitude));
}

__device__ __forceinline__ void rope_turn(float& u, float& v, float2 r) {
    const float a = __fsub_rn(__fmul_rn(u, r.x), __fmul_rn(v, r.y));
    v = __fadd_rn(__fmul_rn(u, r.y), __fmul_rn(v, r.x));
    u = a;
}

// ------------------------------------------------------------- wide chunks
// A unit is 8 pairs (two chunks of 8 elements, HALVES), 4 pairs (one chunk,
// INTERLEAVED) or a chunk passed through.  A thread has the same unit of every
// head that it takes, so blockDim.x is a multiple of the units per head; the
// heads of q and k of TT tokens (blockIdx.x) go round over the threads' groups and
// blockIdx.y.  UN units of a thread are in flight, the first ones while the
// angles are formed.
template <int DT, bool INTER, int TT>
__global__ void __launch_bounds__(ROPE_THREADS) rope_vec_kernel(RopeParams p) {
    constexpr int UN = DT == HQ_DT_F32 ? 2 : 4, V4 = INTER ? 2 : 4;  // float4s of cosines and sines per unit
    extern __shared__ float4 cs[];  // [TT][V4][units turned]: no bank conflicts between a warp's units
    const int64_t t0 = (int64_t)blockIdx.x * TT;
    const int tokens = p.T - t0 < TT ? (int)(p.T - t0) : TT, half = p.R / 2;
    const int turned = half / (2 * V4), rest = (p.D - p.R) / 8;
    const bool copy[2] = {p.t[0].in != p.t[0].out, p.t[1].heads && p.t[1].in != p.t[1].out};
    const int per_head = turned + (copy[0] || copy[1] ? rest : 0), groups = blockDim.x / per_head;
    const int u = threadIdx.x % per_head, heads = p.t[0].heads + p.t[1].heads;
    const bool turn = u < turned;
    int e = p.offset + 8 * u;  // first element
    if (!turn) e = u - turned < p.offset / 8 ? 8 * (u - turned) : 8 * (u - turned) + p.R;
    // the thread's next (token, head), as token * heads + head
    int head = blockIdx.y * groups + threadIdx.x / per_head, t = 0;
    const int step = gridDim.y * groups;
    auto settle = [&] {
        while (head >= heads) {
            head -= heads;
            ++t;
        }
    };
    settle();
    Chunk<DT> a[UN], b[UN];
    int64_t at[UN];  // output element of the first chunk
    int tok[UN];     // token; bit 8: k; -1: none
    auto load = [&] {
#pragma unroll
        for (int k = 0; k < UN; ++k) {
            tok[k] = -1;
            if (t >= tokens) continue;
            const bool z = head >= p.t[0].heads;
            const RopeTensor& x = p.t[z];
            const int64_t h = z ? head - p.t[0].heads : head;
            if (turn || copy[z]) {
                const int64_t src = (t0 + t) * x.in_ts + h * x.in_hs + e;
                at[k] = (t0 + t) * x.out_ts + h * x.out_hs + e;
                a[k] = load_chunk<DT>(x.in, src);
                if (!INTER && turn) b[k] = load_chunk<DT>(x.in, src + half);
                tok[k] = t | (z ? 256 : 0);
            }
            head += step;
            settle();
        }
    };
    load();
    for (int n = threadIdx.x; n < tokens * half; n += blockDim.x) {
        const int q = n / half, i = n - q * half;
        const float2 v = rope_cos_sin(p.pos[t0 + q], p.inv_freq[i], p.magnitude, p.inverse != 0);
        const int at4 = (q * V4 + i % (2 * V4) / 2) * turned + i / (2 * V4);
        reinterpret_cast<float2*>(cs)[2 * at4 + (i & 1)] = v;
    }
    __syncthreads();
    for (bool more = true; more;) {
        more = t < tokens;
#pragma unroll
        for (int k = 0; k < UN; ++k) {
            if (tok[k] < 0) continue;
            void* const out = p.t[tok[k] >> 8].out;
            if (!turn) {
                store_chunk<DT>(out, at[k], a[k]);
                continue;
            }
            const float4* const r = cs + (tok[k] & 255) * V4 * turned + u;
            float f[8];
            unpack8<DT>(a[k], f);
            if constexpr (INTER) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float4 v = r[i * turned];
                    rope_turn(f[4 * i], f[4 * i + 1], make_float2(v.x, v.y));
                    rope_turn(f[4 * i + 2], f[4 * i + 3], make_float2(v.z, v.w));
                }
            } else {
                float g[8];
                unpack8<DT>(b[k], g);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 v = r[i * turned];
                    rope_turn(f[2 * i], g[2 * i], make_float2(v.x, v.y));
                    rope_turn(f[2 * i + 1], g[2 * i + 1], make_float2(v.z, v.w));
                }
                store_chunk<DT>(out, at[k] + half, pack8<DT>(g));
            }
            store_chunk<DT>(out, at[k], pack8<DT>(f));
        }
        if (more) load();
    }
}

// ---------------------------------------------------------- any other shape
// One block per token, one element pair (or one passed-through element) a step.
template <int DT>
__global__ void __launch_bounds__(ROPE_THREADS) rope_kernel(RopeParams p) {
    typedef typename Elem<DT>::T T;
    extern __shared__ float2 angles[];  // [R / 2]
    const int64_t t = blockIdx.x;
    const int half = p.R / 2;
    for (int i = threadIdx.x; i < half; i += ROPE_THREADS)
        angles[i] = rope_cos_sin(p.pos[t], p.inv_freq[i], p.magnitude, p.inverse != 0);
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
                rope_turn(u, v, angles[i]);
                b[e] = from_f32<DT>(u);
                b[f] = from_f32<DT>(v);
            } else {
                const int e = i - half < p.offset ? i - half : i - half + p.R;
                b[e] = a[e];
            }
        }
    }
}

template <int DT, int TT> static void rope_vec(const RopeParams& p, int threads, int split, cudaStream_t st) {
    const dim3 grid((unsigned)((p.T + TT - 1) / TT), (unsigned)split);
    const size_t smem = sizeof(float2) * (size_t)(p.R / 2) * TT;
    if (p.interleaved) rope_vec_kernel<DT, true, TT><<<grid, threads, smem, st>>>(p);
    else rope_vec_kernel<DT, false, TT><<<grid, threads, smem, st>>>(p);
}
template <int DT> static void rope_t(const RopeParams& p, int sms, cudaStream_t st) {
    if (!p.vec) {
        rope_kernel<DT><<<(unsigned)p.T, ROPE_THREADS, sizeof(float2) * (size_t)(p.R / 2), st>>>(p);
        return;
    }
    bool copy = false;
    for (const RopeTensor& x : p.t) copy = copy || (x.heads && x.in != x.out);
    const int per_head = p.R / (p.interleaved ? 8 : 16) + (copy ? (p.D - p.R) / 8 : 0), groups = ROPE_THREADS / per_head;
    // Many tokens: four a block, so that a thread has an angle or more to form.
    // Few: the heads of a token over several blocks, up to two blocks per SM.
    if (p.T >= 4 * sms) {
        rope_vec<DT, 4>(p, groups * per_head, 1, st);
    } else {
        const int64_t most = (p.t[0].heads + p.t[1].heads + groups - 1) / groups;
        int64_t split = (2 * sms + p.T - 1) / p.T;
        if (split > most) split = most;
        rope_vec<DT, 1>(p, groups * per_head, (int)split, st);
    }
}
void launch_rope(int dtype, const RopeParams& p, int sms, cudaStream_t st) {
    if (dtype == HQ_DT_BF16) rope_t<HQ_DT_BF16>(p, sms, st);
    else if (dtype == HQ_DT_F16) rope_t<HQ_DT_F16>(p, sms, st);
    else rope_t<HQ_DT_F32>(p, sms, st);
}

}  // namespace hq
