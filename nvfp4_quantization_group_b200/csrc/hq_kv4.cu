// hq_kv4.cu -- block tables and slot maps, and the NVFP4 key/value cache:
// write new tokens, read tokens back (sm_100a).
#include "hq_layer.cuh"

namespace hq {

// ------------------------------------------------------------------- slots
constexpr int SLOT_THREADS = 1024;

// Sum of v over the threads before this one, and over all (in `total`).
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int& total) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, s, o);
        if (lane >= o) s += u;
    }
    if (lane == 31) warp_sums[w] = s;
    __syncthreads();
    if (w == 0) {
        int t = warp_sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xFFFFFFFFu, t, o);
            if (lane >= o) t += u;
        }
        warp_sums[lane] = t;
    }
    __syncthreads();
    const int before = w ? warp_sums[w - 1] : 0;
    total = warp_sums[31];
    __syncthreads();
    return before + s - v;
}

struct SlotShared {
    // running sums over the requests: pages given back, pages taken, new tokens
    int back[HQ_KV_MAX_REQUESTS + 1], need[HQ_KV_MAX_REQUESTS + 1], cu[HQ_KV_MAX_REQUESTS + 1];
    int lens[HQ_KV_MAX_REQUESTS];
    int warp_sums[32];
    int bad;
    long long total[3];
};

// One block.  The sums are taken first (64-bit totals, so that no sum of
// 32-bit lengths wraps unseen), the step is refused or carried out after.
__global__ void __launch_bounds__(SLOT_THREADS) kv_slots_kernel(SlotParams p) {
    extern __shared__ char raw[];
    SlotShared& sh = *reinterpret_cast<SlotShared*>(raw);
    const int tid = threadIdx.x, P = 1 << p.page_shift;
    const long long row_tokens = p.width << p.page_shift;
    if (tid == 0) {
        sh.bad = 0;
        sh.total[0] = sh.total[1] = sh.total[2] = 0;
        sh.back[0] = sh.need[0] = sh.cu[0] = 0;
    }
    __syncthreads();
    const long long count = *p.count;
    int back0 = 0, need0 = 0, cu0 = 0;
    for (int b0 = 0; b0 < p.B; b0 += SLOT_THREADS) {
        const int b = b0 + tid;
        int back = 0, need = 0, add = 0;
        if (b < p.B) {
            const long long n = p.lens[b], a = p.add[b];
            sh.lens[b] = (int)n;
            if (n < 0 || n > row_tokens) {
                atomicOr(&sh.bad, HQ_KV_BAD_STATE);
            } else if (a < 0) {
                back = (int)((n + P - 1) >> p.page_shift);
            } else if (n + a > row_tokens || n + a > 0x7FFFFFFF) {
                atomicOr(&sh.bad, HQ_KV_NO_WIDTH);
            } else {
                need = (int)(((n + a + P - 1) >> p.page_shift) - ((n + P - 1) >> p.page_shift));
                add = (int)a;
            }
            atomicAdd(reinterpret_cast<unsigned long long*>(&sh.total[0]), (unsigned long long)back);
            atomicAdd(reinterpret_cast<unsigned long long*>(&sh.total[1]), (unsigned long long)need);
            atomicAdd(reinterpret_cast<unsigned long long*>(&sh.total[2]), (unsigned long long)add);
        }
        int t0, t1, t2;
        const int e0 = block_scan(back, sh.warp_sums, t0), e1 = block_scan(need, sh.warp_sums, t1),
                  e2 = block_scan(add, sh.warp_sums, t2);
        if (b < p.B) {
            sh.back[b + 1] = back0 + e0 + back;
            sh.need[b + 1] = need0 + e1 + need;
            sh.cu[b + 1] = cu0 + e2 + add;
        }
        back0 += t0;
        need0 += t1;
        cu0 += t2;
    }
    __syncthreads();
    int bad = sh.bad;
    if (count < 0 || count > p.capacity || count + sh.total[0] > p.capacity) bad |= HQ_KV_BAD_STATE;
    if (sh.total[1] > count + sh.total[0]) bad |= HQ_KV_NO_PAGES;
    if (sh.total[2] > p.n_slots) bad |= HQ_KV_NO_ROWS;
    if (bad) {
        for (int b = tid; b < p.B; b += SLOT_THREADS) {
            p.lens_out[b] = sh.lens[b];
            p.cu[b + 1] = 0;
        }
        if (tid == 0) {
            p.cu[0] = 0;
            *p.count_out = (int)count;
            *p.status = bad;
        }
        for (int64_t i = tid; i < p.n_slots; i += SLOT_THREADS) {
            p.slots[i] = -1;
            p.positions[i] = 0;
        }
        return;
    }
    const int lane = tid & 31, w = tid >> 5;
    // pages of ended requests onto the stack
    for (int b = w; b < p.B; b += SLOT_THREADS / 32) {
        const int at = (int)count + sh.back[b], n = sh.back[b + 1] - sh.back[b];
        for (int i = lane; i < n; i += 32) p.stack[at + i] = p.table[b * p.width + i];
    }
    __syncthreads();
    // new pages off its top
    const int top = (int)count + (int)sh.total[0];
    for (int b = w; b < p.B; b += SLOT_THREADS / 32) {
        const int first = sh.need[b], n = sh.need[b + 1] - first;
        if (n == 0) continue;
        const int held = (int)(((long long)sh.lens[b] + P - 1) >> p.page_shift);
        for (int i = lane; i < n; i += 32) p.table[b * p.width + held + i] = p.stack[top - 1 - first - i];
    }
    for (int b = tid; b < p.B; b += SLOT_THREADS) {
        const bool ended = sh.back[b + 1] > sh.back[b];
        p.lens_out[b] = ended ? 0 : sh.lens[b] + sh.cu[b + 1] - sh.cu[b];
        p.cu[b + 1] = sh.cu[b + 1];
    }
    if (tid == 0) {
        p.cu[0] = 0;
        *p.count_out = top - (int)sh.total[1];
        *p.status = 0;
    }
    __syncthreads();
    const int total = (int)sh.total[2];
    for (int64_t i = tid; i < p.n_slots; i += SLOT_THREADS) {
        int64_t slot = -1, pos = 0;
        if (i < total) {
            int lo = 0, hi = p.B - 1;  // the request with cu[lo] <= i < cu[lo + 1]
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (sh.cu[mid + 1] > i) hi = mid;
                else lo = mid + 1;
            }
            pos = (int64_t)sh.lens[lo] + (i - sh.cu[lo]);
            slot = ((int64_t)p.table[lo * p.width + (pos >> p.page_shift)] << p.page_shift) + (pos & (P - 1));
        }
        p.slots[i] = slot;
        p.positions[i] = pos;
    }
}

void launch_slots(const SlotParams& p, int sms, cudaStream_t st) {
    (void)sms;
    cudaFuncSetAttribute(kv_slots_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(SlotShared));
    kv_slots_kernel<<<1, SLOT_THREADS, sizeof(SlotShared), st>>>(p);
}

// ------------------------------------------------------------ append, gather
// One warp per 128-vector, lane l with elements 4 l .. 4 l + 3 (block l / 4,
// quad l % 4 of it).  Hadamard stages 1 and 2 in the lane, 4 .. 64 by
// exchanges, ascending: the values of hq_cat_rotate_nvfp4 bit for bit.
__device__ __forceinline__ void hadamard128_warp(float (&y)[4], int lane) {
    float a = y[0], b = y[1], c = y[2], d = y[3];
    y[0] = __fadd_rn(a, b);
    y[1] = __fsub_rn(a, b);
    y[2] = __fadd_rn(c, d);
    y[3] = __fsub_rn(c, d);
    a = y[0], b = y[1], c = y[2], d = y[3];
    y[0] = __fadd_rn(a, c);
    y[1] = __fadd_rn(b, d);
    y[2] = __fsub_rn(a, c);
    y[3] = __fsub_rn(b, d);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float other = __shfl_xor_sync(0xFFFFFFFFu, y[i], o);
            y[i] = lane & o ? __fsub_rn(other, y[i]) : __fadd_rn(y[i], other);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = __fmul_rn(y[i], __uint_as_float(0x3DB504F3u));  // RN(1 / sqrt(128))
}

// Group of slot s and head h in the cache.
__device__ __forceinline__ uint8_t* kv_group(const KvParams& p, int64_t s, int h) {
    const int64_t page = s >> p.page_shift;
    const int groups = 1 << (p.page_shift - 4), at = (int)(s & ((1 << p.page_shift) - 1));
    return p.cache + ((page * p.H + h) * groups + at / 16) * KV_GROUP_BYTES;
}

template <int DT> __global__ void __launch_bounds__(256) kv4_append_kernel(KvParams p) {
    typedef typename Elem<DT>::T T;
    __shared__ float2 vr[128];  // per E4M3 code {value, -RN(1 / value)}
    if (threadIdx.x < 128) {
        const bool zc = threadIdx.x == 0 || threadIdx.x == 127;
        const float v = zc ? 0.0f : e4m3_value(threadIdx.x);
        vr[threadIdx.x] = make_float2(v, zc ? -0.0f : -__frcp_rn(v));
    }
    __syncthreads();
    const int lane = threadIdx.x & 31, quad = lane & 3, blk = lane >> 2;
    const int64_t per_token = 2 * p.H, n = p.N * per_token, warps = (int64_t)gridDim.x * 8;
    for (int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); i < n; i += warps) {
        const int64_t tok = i / per_token, s = p.slots[tok];
        if (s < 0 || s >= p.n_slots) continue;
        const int z = (int)(i % per_token) / p.H, h = (int)(i % p.H);
        const T* x = z ? static_cast<const T*>(p.v) + tok * p.v_ts + h * p.v_hs
                       : static_cast<const T*>(p.k) + tok * p.k_ts + h * p.k_hs;
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = to_f32(x[4 * lane + e]);
        if (p.rotate) hadamard128_warp(y, lane);
        float ab = max3(fmaxf(fabsf(y[0]), fabsf(y[1])), fabsf(y[2]), fabsf(y[3]));
        ab = fmaxf(ab, __shfl_xor_sync(0xFFFFFFFFu, ab, 1));
        ab = fmaxf(ab, __shfl_xor_sync(0xFFFFFFFFu, ab, 2));
        float amax = ab;
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
        const float S = global_encode(amax);
        const uint32_t sf = block_sf(ab, S);
        const float enc = block_enc(vr, sf, S, slow_scale(S));
        const uint32_t codes = e2m1x8(__fmul_rn(y[0], enc), __fmul_rn(y[1], enc), __fmul_rn(y[2], enc),
                                      __fmul_rn(y[3], enc), 0.0f, 0.0f, 0.0f, 0.0f);
        uint8_t* g = kv_group(p, s, h);
        const int r = (int)(s & 15), half = r >> 3, pair = (r & 7) >> 1, odd = r & 1;
        if (z == 0) {
            *reinterpret_cast<uint16_t*>(g + KV_K_CODES + r * 64 + quad * 16 + blk * 2) = (uint16_t)codes;
            if (quad == 0) g[KV_K_SF + r * 8 + blk] = (uint8_t)sf;
            if (lane == 0) reinterpret_cast<float*>(g + KV_K_DEC)[r] = __fdiv_rn(1.0f, S);
        } else {
            uint8_t* o = g + KV_V_CODES + half * 512 + pair * 16 + odd * 8 + blk;
            o[(2 * quad) * 64] = (uint8_t)codes;
            o[(2 * quad + 1) * 64] = (uint8_t)(codes >> 8);
            if (quad == 0) g[KV_V_SF + half * 64 + pair * 16 + blk * 2 + odd] = (uint8_t)sf;
            if (lane == 0) reinterpret_cast<float*>(g + KV_V_DEC)[r] = __fdiv_rn(1.0f, S);
        }
    }
}

// Value of an E2M1 nibble.
__device__ __forceinline__ float e2m1_value(uint32_t c) {
    const uint32_t m = c & 7u;
    const float v = m < 2u ? 0.5f * (float)m : __uint_as_float(((m >> 1) + 126u) << 23 | (m & 1u) << 22);
    return c & 8u ? -v : v;
}

template <int DT> __global__ void __launch_bounds__(256) kv4_gather_kernel(KvParams p) {
    typedef typename Elem<DT>::T T;
    const int lane = threadIdx.x & 31, quad = lane & 3, blk = lane >> 2;
    const int64_t per_token = 2 * p.H, n = p.N * per_token, warps = (int64_t)gridDim.x * 8;
    for (int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); i < n; i += warps) {
        const int64_t tok = i / per_token, s = p.slots[tok];
        const int z = (int)(i % per_token) / p.H, h = (int)(i % p.H);
        T* x = z ? static_cast<T*>(p.v) + tok * p.v_ts + h * p.v_hs : static_cast<T*>(p.k) + tok * p.k_ts + h * p.k_hs;
        float y[4] = {};
        if (s >= 0 && s < p.n_slots) {
            const uint8_t* g = kv_group(p, s, h);
            const int r = (int)(s & 15), half = r >> 3, pair = (r & 7) >> 1, odd = r & 1;
            uint32_t codes, sf;
            float dec;
            if (z == 0) {
                codes = *reinterpret_cast<const uint16_t*>(g + KV_K_CODES + r * 64 + quad * 16 + blk * 2);
                sf = g[KV_K_SF + r * 8 + blk];
                dec = reinterpret_cast<const float*>(g + KV_K_DEC)[r];
            } else {
                const uint8_t* o = g + KV_V_CODES + half * 512 + pair * 16 + odd * 8 + blk;
                codes = o[(2 * quad) * 64] | (uint32_t)o[(2 * quad + 1) * 64] << 8;
                sf = g[KV_V_SF + half * 64 + pair * 16 + blk * 2 + odd];
                dec = reinterpret_cast<const float*>(g + KV_V_DEC)[r];
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
                y[e] = __fmul_rn(__fmul_rn(e2m1_value(codes >> (4 * e)), e4m3_value(sf)), dec);
            if (p.rotate) hadamard128_warp(y, lane);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) x[4 * lane + e] = from_f32<DT>(y[e]);
    }
}

static int kv_grid(const KvParams& p, int sms) {
    const int64_t blocks = (p.N * 2 * p.H + 7) / 8, cap = (int64_t)sms * 8;
    return (int)(blocks < cap ? blocks : cap);
}
void launch_append(int dtype, const KvParams& p, int sms, cudaStream_t st) {
    const int grid = kv_grid(p, sms);
    if (dtype == HQ_DT_BF16) kv4_append_kernel<HQ_DT_BF16><<<grid, 256, 0, st>>>(p);
    else if (dtype == HQ_DT_F16) kv4_append_kernel<HQ_DT_F16><<<grid, 256, 0, st>>>(p);
    else kv4_append_kernel<HQ_DT_F32><<<grid, 256, 0, st>>>(p);
}
void launch_gather(int dtype, const KvParams& p, int sms, cudaStream_t st) {
    const int grid = kv_grid(p, sms);
    if (dtype == HQ_DT_BF16) kv4_gather_kernel<HQ_DT_BF16><<<grid, 256, 0, st>>>(p);
    else if (dtype == HQ_DT_F16) kv4_gather_kernel<HQ_DT_F16><<<grid, 256, 0, st>>>(p);
    else kv4_gather_kernel<HQ_DT_F32><<<grid, 256, 0, st>>>(p);
}

}  // namespace hq
