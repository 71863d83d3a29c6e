// hq_layer.cuh -- device helpers of the attention-layer kernels: element
// types, 8-element chunks, warp reductions.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "hq_device.cuh"
#include "hq_layer.h"

namespace hq {

template <int DT> struct Elem;
template <> struct Elem<HQ_DT_BF16> { typedef __nv_bfloat16 T; };
template <> struct Elem<HQ_DT_F16> { typedef __half T; };
template <> struct Elem<HQ_DT_F32> { typedef float T; };

__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }
template <int DT> __device__ __forceinline__ typename Elem<DT>::T from_f32(float v);
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<HQ_DT_BF16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f32<HQ_DT_F16>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ float from_f32<HQ_DT_F32>(float v) { return v; }

// 16-byte load that may read what this kernel writes elsewhere (no read-only
// path: outputs may be the inputs themselves).
__device__ __forceinline__ uint4 ld_v4(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}

// A chunk of 8 elements as loaded: 16 bytes, or 32 for FP32.
template <int DT> struct Chunk { uint4 w[DT == HQ_DT_F32 ? 2 : 1]; };

template <int DT> __device__ __forceinline__ Chunk<DT> load_chunk(const void* base, int64_t elem) {
    Chunk<DT> c;
    const typename Elem<DT>::T* p = static_cast<const typename Elem<DT>::T*>(base) + elem;
    c.w[0] = ld_v4(p);
    if constexpr (DT == HQ_DT_F32) c.w[1] = ld_v4(p + 4);
    return c;
}
template <int DT> __device__ __forceinline__ void store_chunk(void* base, int64_t elem, const Chunk<DT>& c) {
    uint4* p = reinterpret_cast<uint4*>(static_cast<typename Elem<DT>::T*>(base) + elem);
    p[0] = c.w[0];
    if constexpr (DT == HQ_DT_F32) p[1] = c.w[1];
}
// Sixteen elements: where they are 32-byte aligned (the caller's word for it), as
// 32-byte accesses, a whole sector each.
template <int DT> __device__ __forceinline__ void load_pair(const void* base, int64_t elem, bool wide, Chunk<DT> (&c)[2]) {
    const typename Elem<DT>::T* const p = static_cast<const typename Elem<DT>::T*>(base) + elem;
    if (!wide) {
        c[0] = load_chunk<DT>(base, elem);
        c[1] = load_chunk<DT>(base, elem + 8);
    } else if constexpr (DT == HQ_DT_F32) {
        ld_nc_v8(p, c[0].w[0], c[0].w[1]);
        ld_nc_v8(p + 8, c[1].w[0], c[1].w[1]);
    } else {
        ld_nc_v8(p, c[0].w[0], c[1].w[0]);
    }
}
__device__ __forceinline__ void st_v8(void* p, const uint4& a, const uint4& b) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 :: "l"(p), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w) : "memory");
}
template <int DT> __device__ __forceinline__ void store_pair(void* base, int64_t elem, bool wide, const Chunk<DT> (&c)[2]) {
    typename Elem<DT>::T* const p = static_cast<typename Elem<DT>::T*>(base) + elem;
    if (!wide) {
        store_chunk<DT>(base, elem, c[0]);
        store_chunk<DT>(base, elem + 8, c[1]);
    } else if constexpr (DT == HQ_DT_F32) {
        st_v8(p, c[0].w[0], c[0].w[1]);
        st_v8(p + 8, c[1].w[0], c[1].w[1]);
    } else {
        st_v8(p, c[0].w[0], c[1].w[0]);
    }
}
template <int DT> __device__ __forceinline__ void unpack8(const Chunk<DT>& c, float (&f)[8]) {
    if constexpr (DT == HQ_DT_F32) {
        const uint32_t u[8] = {c.w[0].x, c.w[0].y, c.w[0].z, c.w[0].w, c.w[1].x, c.w[1].y, c.w[1].z, c.w[1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(u[i]);
    } else {
        const uint32_t u[4] = {c.w[0].x, c.w[0].y, c.w[0].z, c.w[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (DT == HQ_DT_BF16) {
                f[2 * i] = bf16_lo(u[i]);
                f[2 * i + 1] = bf16_hi(u[i]);
            } else {
                const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
                f[2 * i] = v.x;
                f[2 * i + 1] = v.y;
            }
        }
    }
}
// One rounding of each value to the type.
template <int DT> __device__ __forceinline__ Chunk<DT> pack8(const float (&f)[8]) {
    Chunk<DT> c;
    uint32_t u[DT == HQ_DT_F32 ? 8 : 4];
    if constexpr (DT == HQ_DT_F32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = __float_as_uint(f[i]);
        c.w[1] = make_uint4(u[4], u[5], u[6], u[7]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (DT == HQ_DT_BF16) {
                const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
                u[i] = *reinterpret_cast<const uint32_t*>(&v);
            } else {
                const __half2 v = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
                u[i] = *reinterpret_cast<const uint32_t*>(&v);
            }
        }
    }
    c.w[0] = make_uint4(u[0], u[1], u[2], u[3]);
    return c;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}

// E4M3(y / s) of 8 values by the FP8 rule's correctly rounded quotient
// (element 0 in the low byte of x); s = +inf takes plain IEEE division.
__device__ __forceinline__ uint2 fp8_codes8(const float (&y)[8], float s) {
    uint32_t c[4];
    if (!isinf(s)) {
        const Recip d = make_recip(s);
        const f2 b2 = pack2(d.b, d.b), nr2 = pack2(d.nr, d.nr);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a, b;
            unpack2(div2_rn_neg(pack2(-y[2 * i], -y[2 * i + 1]), b2, nr2), a, b);
            c[i] = e4m3x2(a, b);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = e4m3x2(__fdiv_rn(y[2 * i], s), __fdiv_rn(y[2 * i + 1], s));
    }
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// A kernel of the same call that follows another one: its blocks may be placed
// while the first one's last blocks run, and wait for its end (and its writes)
// in after_previous().  The first kernel says let_next() where it no longer
// matters when the next one's blocks take room.
__device__ __forceinline__ void let_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <typename... P, typename... A>
void launch_next(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, A... args) {
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c = {};
    c.gridDim = grid;
    c.blockDim = block;
    c.dynamicSmemBytes = smem;
    c.stream = st;
    c.attrs = at;
    c.numAttrs = 1;
    cudaLaunchKernelEx(&c, kernel, static_cast<P>(args)...);
}

// Lets a kernel use `bytes` of dynamic shared memory on the current device;
// asked once per kernel and device.  Returns a cudaError_t.
template <typename K> int allow_shared(K* kernel, size_t bytes) {
    constexpr int kMaxDevices = 64;
    static std::atomic<const void*> done[kMaxDevices][4];  // (kernels of one signature share this table)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return (int)e;
    const void* const key = reinterpret_cast<const void*>(kernel);
    if (dev >= 0 && dev < kMaxDevices)
        for (auto& d : done[dev])
            if (d.load(std::memory_order_acquire) == key) return (int)cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return (int)e;
    if (dev >= 0 && dev < kMaxDevices)
        for (auto& d : done[dev]) {
            const void* none = nullptr;
            if (d.compare_exchange_strong(none, key) || none == key) break;
        }
    return (int)cudaSuccess;
}

}  // namespace hq
