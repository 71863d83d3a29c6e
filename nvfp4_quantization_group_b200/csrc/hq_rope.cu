// hq_rope.cu -- rotary positions of q and k in one launch (sm_100a).
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

// One block per token; its angles once into shared memory, then one element
// pair (or one passed-through element) per step.
template <int DT>
__global__ void __launch_bounds__(ROPE_THREADS) rope_kernel(RopeParams p) {
    typedef typename Elem<DT>::T T;
    extern __shared__ float2 cs[];  // [R / 2]
    const int64_t t = blockIdx.x;
    const int half = p.R / 2;
    for (int i = threadIdx.x; i < half; i += ROPE_THREADS)
        cs[i] = rope_cos_sin(p.pos[t], p.inv_freq[i], p.magnitude, p.inverse != 0);
    __syncthreads();
    const int rest = p.copy ? p.D - p.R : 0, per_head = half + rest;
    for (int z = 0; z < 2; ++z) {
        const RopeTensor& x = p.t[z];
        const T* in = static_cast<const T*>(x.in) + t * x.in_ts;
        T* out = static_cast<T*>(x.out) + t * x.out_ts;
        for (int n = threadIdx.x; n < x.heads * per_head; n += ROPE_THREADS) {
            const int head = n / per_head, i = n % per_head;
            const T* a = in + head * x.in_hs;
            T* b = out + head * x.out_hs;
            if (i < half) {
                const int e = p.offset + (p.interleaved ? 2 * i : i), f = e + (p.interleaved ? 1 : half);
                const float u = to_f32(a[e]), v = to_f32(a[f]);
                const float2 r = cs[i];
                b[e] = from_f32<DT>(__fsub_rn(__fmul_rn(u, r.x), __fmul_rn(v, r.y)));
                b[f] = from_f32<DT>(__fadd_rn(__fmul_rn(u, r.y), __fmul_rn(v, r.x)));
            } else {
                const int e = i - half < p.offset ? i - half : i - half + p.R;
                b[e] = a[e];
            }
        }
    }
}

void launch_rope(int dtype, const RopeParams& p, int sms, cudaStream_t st) {
    (void)sms;
    const size_t smem = sizeof(float2) * (size_t)(p.R / 2);
    if (dtype == HQ_DT_BF16) rope_kernel<HQ_DT_BF16><<<(unsigned)p.T, ROPE_THREADS, smem, st>>>(p);
    else if (dtype == HQ_DT_F16) rope_kernel<HQ_DT_F16><<<(unsigned)p.T, ROPE_THREADS, smem, st>>>(p);
    else rope_kernel<HQ_DT_F32><<<(unsigned)p.T, ROPE_THREADS, smem, st>>>(p);
}

}  // namespace hq
