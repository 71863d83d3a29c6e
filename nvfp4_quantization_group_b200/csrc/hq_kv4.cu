// hq_kv4.cu -- block tables and slot maps, and the NVFP4 key/value cache:
// write new tokens, read tokens back (sm_100a).
#include "hq_layer.cuh"

namespace hq {

// ------------------------------------------------------------------- slots
// Three running sums over the requests (pages given back, pages taken, new
// tokens), 64 bits wide so that no sum of 32-bit lengths wraps unseen; then
// every page and every token finds its request by bisection of them.  Latency
// counts: one block, one barrier per dependent step, nothing per request that
// is longer than its share.
constexpr int SLOT_THREADS = 1024;
constexpr int SLOT_ROWS = 8192;  // slot maps up to this many rows are filled by the same block

struct SlotShared {
    long long warp_sums[3][32];
    int bad;
    // then int [B + 1] each: back, need, cu (sums before each request), and int [B] lens
};

// The request b with sum[b] <= i < sum[b + 1] (i below the last sum).
__device__ __forceinline__ int slot_request(const int* sum, int B, int i) {
    int lo = 0, hi = B - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (sum[mid + 1] > i) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

__global__ void __launch_bounds__(SLOT_THREADS) kv_slots_kernel(SlotParams p, int rows_here) {
    extern __shared__ __align__(16) char raw[];
    SlotShared& sh = *reinterpret_cast<SlotShared*>(raw);
    int* const back = reinterpret_cast<int*>(raw + sizeof(SlotShared));
    int* const need = back + p.B + 1;
    int* const cu = need + p.B + 1;
    int* const lens = cu + p.B + 1;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, P = 1 << p.page_shift;
    const long long row_tokens = p.width << p.page_shift;
    const long long count = *p.count;
    if (tid == 0) {
        sh.bad = 0;
        back[0] = need[0] = cu[0] = 0;
    }
    __syncthreads();
    long long before[3] = {0, 0, 0};
    for (int b0 = 0; b0 < p.B; b0 += SLOT_THREADS) {
        const int b = b0 + tid;
        long long v[3] = {0, 0, 0};
        if (b < p.B) {
            const long long n = p.lens[b], a = p.add[b];
            lens[b] = (int)n;
            if (n < 0 || n > row_tokens) {
                atomicOr(&sh.bad, HQ_KV_BAD_STATE);
            } else if (a < 0) {
                v[0] = (n + P - 1) >> p.page_shift;
            } else if (n + a > row_tokens || n + a > 0x7FFFFFFF) {
                atomicOr(&sh.bad, HQ_KV_NO_WIDTH);
            } else {
                v[1] = ((n + a + P - 1) >> p.page_shift) - ((n + P - 1) >> p.page_shift);
                v[2] = a;
            }
        }
        long long s[3];
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            s[k] = v[k];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long u = __shfl_up_sync(0xFFFFFFFFu, s[k], o);
                if (lane >= o) s[k] += u;
            }
            if (lane == 31) sh.warp_sums[k][w] = s[k];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            long long t = sh.warp_sums[k][lane];  // every warp sums the warps' sums for itself
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long u = __shfl_up_sync(0xFFFFFFFFu, t, o);
                if (lane >= o) t += u;
            }
            const long long mine = __shfl_sync(0xFFFFFFFFu, t, w ? w - 1 : 0);
            s[k] += before[k] + (w ? mine : 0);
            before[k] += __shfl_sync(0xFFFFFFFFu, t, 31);
        }
        if (b < p.B) {  // (truncated sums are not used: such a step is refused)
            back[b + 1] = (int)s[0];
            need[b + 1] = (int)s[1];
            cu[b + 1] = (int)s[2];
        }
        __syncthreads();
    }
    int bad = sh.bad;
    if (count < 0 || count > p.capacity || count + before[0] > p.capacity) bad |= HQ_KV_BAD_STATE;
    if (before[1] > count + before[0]) bad |= HQ_KV_NO_PAGES;
    if (before[2] > p.n_slots) bad |= HQ_KV_NO_ROWS;
    const int top = (int)(count + before[0]), taken = bad ? 0 : (int)before[1], total = bad ? 0 : (int)before[2];
    // pages of ended requests onto the stack
    if (!bad && before[0] > 0) {
        for (int i = tid; i < (int)before[0]; i += SLOT_THREADS) {
            const int b = slot_request(back, p.B, i);
            p.stack[(int)count + i] = p.table[b * p.width + (i - back[b])];
        }
        __syncthreads();
    }
    // new pages off its top
    for (int i = tid; i < taken; i += SLOT_THREADS) {
        const int b = slot_request(need, p.B, i);
        const int held = (int)(((long long)lens[b] + P - 1) >> p.page_shift);
        p.table[b * p.width + held + (i - need[b])] = p.stack[top - 1 - i];
    }
    for (int b = tid; b < p.B; b += SLOT_THREADS) {
        p.lens_out[b] = bad ? lens[b] : back[b + 1] > back[b] ? 0 : lens[b] + cu[b + 1] - cu[b];
        p.cu[b + 1] = bad ? 0 : cu[b + 1];
    }
    if (tid == 0) {
        p.cu[0] = 0;
        *p.count_out = bad ? (int)count : top - taken;
        *p.status = bad;
    }
    // slots and positions (a page taken in this step is read from the stack, where it still lies)
    for (int i = tid; i < rows_here; i += SLOT_THREADS) {
        int64_t slot = -1, pos = 0;
        if (i < total) {
            const int b = slot_request(cu, p.B, i);
            pos = (int64_t)lens[b] + (i - cu[b]);
            const int held = (int)(((long long)lens[b] + P - 1) >> p.page_shift), k = (int)(pos >> p.page_shift);
            const int page = k < held ? p.table[b * p.width + k] : p.stack[top - 1 - need[b] - (k - held)];
            slot = ((int64_t)page << p.page_shift) + (pos & (P - 1));
        }
        p.slots[i] = slot;
        p.positions[i] = pos;
    }
}

// The rest of a long slot map, from what kv_slots_kernel left (a refused step
// left sums of zero: no row is in use).
__global__ void __launch_bounds__(256) kv_slot_rows_kernel(SlotParams p) {
    extern __shared__ __align__(16) int sums[];  // [B + 1]
    for (int b = threadIdx.x; b <= p.B; b += 256) sums[b] = p.cu[b];
    __syncthreads();
    const int total = sums[p.B], P = 1 << p.page_shift;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < p.n_slots; i += (int64_t)gridDim.x * 256) {
        int64_t slot = -1, pos = 0;
        if (i < total) {
            const int b = slot_request(sums, p.B, (int)i);
            pos = (int64_t)p.lens_out[b] - (sums[b + 1] - i);
            slot = ((int64_t)p.table[b * p.width + (pos >> p.page_shift)] << p.page_shift) + (pos & (P - 1));
        }
        p.slots[i] = slot;
        p.positions[i] = pos;
    }
}

void launch_slots(const SlotParams& p, int sms, cudaStream_t st) {
    auto bytes = [](int B) { return sizeof(SlotShared) + sizeof(int) * (4 * (size_t)B + 3); };
    allow_shared(kv_slots_kernel, bytes(HQ_KV_MAX_REQUESTS));
    const bool rows = p.n_slots > SLOT_ROWS;
    kv_slots_kernel<<<1, SLOT_THREADS, bytes(p.B), st>>>(p, rows ? 0 : (int)p.n_slots);
    if (rows) {
        const int64_t blocks = (p.n_slots + 1023) / 1024, cap = 2 * (int64_t)sms;
        kv_slot_rows_kernel<<<(unsigned)(blocks < cap ? blocks : cap), 256, sizeof(int) * ((size_t)p.B + 1), st>>>(p);
    }
}

// ------------------------------------------------------------ append, gather
// A tile is 16 consecutive tokens of one head, keys and values: 32 vectors, four
// threads each.  A thread has 32 consecutive elements on the side of the
// vectors and, on the side of the cache, elements 16 b + 4 i .. + 3 of every
// block b (i the thread of the four): the 16 bytes of keys' codes, or two times
// 8 bytes of values' codes, that lie together in a group.  The tokens of a tile
// usually fill one group, whose sectors are then written whole.
constexpr int KV_THREADS = 128;

struct KvShared {
    // a vector's 32 chunks of four elements, chunk k of thread j (elements 32 j + 4 k ..) at 8 j + ((k + 2 j) & 7);
    // 33 per vector: two vectors of a quarter-warp hit different banks on both sides
    float4 t[32][33];
};
__device__ __forceinline__ int kv_chunk(int c) {  // place of chunk c (elements 4 c .. 4 c + 3)
    const int j = c >> 3, k = c & 7;
    return 8 * j + ((k + 2 * j) & 7);
}

// Stages h = 1, 2, .. of a butterfly over N values held by one thread.
template <int N> __device__ __forceinline__ void butterfly(float (&y)[32], int first, int last) {
#pragma unroll
    for (int h = 1; h < N; h <<= 1) {
        if (h < first || h > last) continue;
#pragma unroll
        for (int e = 0; e < N; ++e)
            if ((e & h) == 0) {
                const float a = y[e], b = y[e + h];
                y[e] = __fadd_rn(a, b);
                y[e + h] = __fsub_rn(a, b);
            }
    }
}

// Group of slot s and head h in the cache.
__device__ __forceinline__ uint8_t* kv_group(const KvParams& p, int64_t s, int h) {
    const int64_t page = s >> p.page_shift;
    const int groups = 1 << (p.page_shift - 4), at = (int)(s & ((1 << p.page_shift) - 1));
    return p.cache + ((page * p.H + h) * groups + at / 16) * KV_GROUP_BYTES;
}

// Quantizes as hq_cat_rotate_nvfp4, bit for bit: stages in ascending order, the
// same scales and conversions.
template <int DT> __global__ void __launch_bounds__(KV_THREADS) kv4_append_kernel(KvParams p) {
    __shared__ KvShared sh;
    __shared__ float2 vr[128];  // per E4M3 code {value, -RN(1 / value)}
    const int tid = threadIdx.x;
    {
        const bool zc = tid == 0 || tid == 127;
        const float v = zc ? 0.0f : e4m3_value(tid);
        vr[tid] = make_float2(v, zc ? -0.0f : -__frcp_rn(v));
    }
    __syncthreads();
    const int vec = tid >> 2, i = tid & 3, z = vec >> 4;
    float4* const row = sh.t[vec];
    const int64_t tiles = (p.N + 15) / 16 * p.H;
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int h = (int)(tile % p.H);
        const int64_t tok = tile / p.H * 16 + (vec & 15);
        const int64_t s = tok < p.N ? p.slots[tok] : -1;
        const bool ok = s >= 0 && s < p.n_slots;  // (the four threads of a vector agree)
        float y[32];
        if (ok) {
            const void* const x = z ? p.v : p.k;
            const int64_t at = z ? tok * p.v_ts + h * p.v_hs : tok * p.k_ts + h * p.k_hs;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                float f[8];
                unpack8<DT>(load_chunk<DT>(x, at + 32 * i + 8 * c), f);
#pragma unroll
                for (int e = 0; e < 8; ++e) y[8 * c + e] = f[e];
            }
        } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) y[e] = 0.0f;
        }
        if (p.rotate) butterfly<32>(y, 1, 16);
        __syncwarp();  // the last tile's reads are done
#pragma unroll
        for (int k = 0; k < 8; ++k) row[kv_chunk(8 * i + k)] = make_float4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
        __syncwarp();
#pragma unroll
        for (int b = 0; b < 8; ++b) {  // y[4 b + e]: element 16 b + 4 i + e
            const float4 v = row[kv_chunk(4 * b + i)];
            y[4 * b] = v.x;
            y[4 * b + 1] = v.y;
            y[4 * b + 2] = v.z;
            y[4 * b + 3] = v.w;
        }
        if (p.rotate) {
            butterfly<32>(y, 8, 16);  // elements 32 and 64 apart: two and four blocks
#pragma unroll
            for (int e = 0; e < 32; ++e) y[e] = __fmul_rn(y[e], __uint_as_float(0x3DB504F3u));  // RN(1 / sqrt(128))
        }
        float ab[8], amax = 0.0f;
#pragma unroll
        for (int b = 0; b < 8; ++b) {
            float a = max3(fmaxf(fabsf(y[4 * b]), fabsf(y[4 * b + 1])), fabsf(y[4 * b + 2]), fabsf(y[4 * b + 3]));
            a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, 1));
            ab[b] = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, 2));
            amax = fmaxf(amax, ab[b]);
        }
        const float S = global_encode(amax);
        const bool slow = slow_scale(S);
        uint32_t codes[8], sf[2] = {0u, 0u};  // four nibbles of each block; the blocks' scales
#pragma unroll
        for (int b = 0; b < 8; b += 2) {
            const uint32_t f0 = block_sf(ab[b], S), f1 = block_sf(ab[b + 1], S);
            const float e0 = block_enc(vr, f0, S, slow), e1 = block_enc(vr, f1, S, slow);
            const uint32_t c = e2m1x8(__fmul_rn(y[4 * b], e0), __fmul_rn(y[4 * b + 1], e0), __fmul_rn(y[4 * b + 2], e0),
                                      __fmul_rn(y[4 * b + 3], e0), __fmul_rn(y[4 * b + 4], e1), __fmul_rn(y[4 * b + 5], e1),
                                      __fmul_rn(y[4 * b + 6], e1), __fmul_rn(y[4 * b + 7], e1));
            codes[b / 2] = c;  // bytes: block b pairs 0, 1; block b + 1 pairs 0, 1
            sf[b / 4] |= (f0 | f1 << 8) << (8 * (b & 3));
        }
        if (!ok) continue;
        uint8_t* const g = kv_group(p, s, h);
        const int r = (int)(s & 15), half = r >> 3, pair = (r & 7) >> 1, odd = r & 1;
        if (z == 0) {
            *reinterpret_cast<uint4*>(g + KV_K_CODES + r * 64 + i * 16) = make_uint4(codes[0], codes[1], codes[2], codes[3]);
            if (i == 0) *reinterpret_cast<uint2*>(g + KV_K_SF + r * 8) = make_uint2(sf[0], sf[1]);
            if (i == 1) reinterpret_cast<float*>(g + KV_K_DEC)[r] = __fdiv_rn(1.0f, S);
        } else {
            // byte pairs 2 i and 2 i + 1 of the eight blocks
            uint8_t* const o = g + KV_V_CODES + half * 512 + 2 * i * 64 + pair * 16 + odd * 8;
            *reinterpret_cast<uint2*>(o) = make_uint2(__byte_perm(codes[0], codes[1], 0x6420), __byte_perm(codes[2], codes[3], 0x6420));
            *reinterpret_cast<uint2*>(o + 64) = make_uint2(__byte_perm(codes[0], codes[1], 0x7531), __byte_perm(codes[2], codes[3], 0x7531));
            uint8_t* const f = g + KV_V_SF + half * 64 + pair * 16 + odd + 4 * i;  // blocks 2 i, 2 i + 1
            const uint32_t two = (i & 2 ? sf[1] : sf[0]) >> (16 * (i & 1));
            f[0] = (uint8_t)two;
            f[2] = (uint8_t)(two >> 8);
            if (i == 1) reinterpret_cast<float*>(g + KV_V_DEC)[r] = __fdiv_rn(1.0f, S);
        }
    }
}

// Four E2M1 nibbles (the low 16 bits) as FP32.
__device__ __forceinline__ void e2m1x4_to_f32(uint32_t c, float& a, float& b, float& d, float& e) {
    uint32_t lo, hi;
    asm("{\n\t.reg .b8 p, q, r, s;\n\tmov.b32 {p, q, r, s}, %2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, p;\n\tcvt.rn.f16x2.e2m1x2 %1, q;\n\t}" : "=r"(lo), "=r"(hi) : "r"(c));
    const float2 u = __half22float2(*reinterpret_cast<const __half2*>(&lo)), v = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    a = u.x;
    b = u.y;
    d = v.x;
    e = v.y;
}

template <int DT> __global__ void __launch_bounds__(KV_THREADS) kv4_gather_kernel(KvParams p) {
    __shared__ KvShared sh;
    const int tid = threadIdx.x, vec = tid >> 2, i = tid & 3, z = vec >> 4;
    float4* const row = sh.t[vec];
    const int64_t tiles = (p.N + 15) / 16 * p.H;
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int h = (int)(tile % p.H);
        const int64_t tok = tile / p.H * 16 + (vec & 15);
        const int64_t s = tok < p.N ? p.slots[tok] : -1;
        float y[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) y[e] = 0.0f;
        if (s >= 0 && s < p.n_slots) {
            const uint8_t* const g = kv_group(p, s, h);
            const int r = (int)(s & 15), half = r >> 3, pair = (r & 7) >> 1, odd = r & 1;
            uint32_t codes[4], sf[2];  // as in the append kernel
            float dec;
            if (z == 0) {
                const uint4 c = *reinterpret_cast<const uint4*>(g + KV_K_CODES + r * 64 + i * 16);
                codes[0] = c.x;
                codes[1] = c.y;
                codes[2] = c.z;
                codes[3] = c.w;
                const uint2 f = *reinterpret_cast<const uint2*>(g + KV_K_SF + r * 8);
                sf[0] = f.x;
                sf[1] = f.y;
                dec = reinterpret_cast<const float*>(g + KV_K_DEC)[r];
            } else {
                const uint8_t* const o = g + KV_V_CODES + half * 512 + 2 * i * 64 + pair * 16 + odd * 8;
                const uint2 lo = *reinterpret_cast<const uint2*>(o), hi = *reinterpret_cast<const uint2*>(o + 64);
                codes[0] = __byte_perm(lo.x, hi.x, 0x5140);
                codes[1] = __byte_perm(lo.x, hi.x, 0x7362);
                codes[2] = __byte_perm(lo.y, hi.y, 0x5140);
                codes[3] = __byte_perm(lo.y, hi.y, 0x7362);
                const uint4 f = *reinterpret_cast<const uint4*>(g + KV_V_SF + half * 64 + pair * 16);
                const uint32_t pick = odd ? 0x7531 : 0x6420;
                sf[0] = __byte_perm(f.x, f.y, pick);
                sf[1] = __byte_perm(f.z, f.w, pick);
                dec = reinterpret_cast<const float*>(g + KV_V_DEC)[r];
            }
#pragma unroll
            for (int b = 0; b < 8; ++b) {
                float* const v = y + 4 * b;
                e2m1x4_to_f32(codes[b / 2] >> (16 * (b & 1)), v[0], v[1], v[2], v[3]);
                const float f = e4m3_value((sf[b / 4] >> (8 * (b & 3))) & 0xFFu);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = __fmul_rn(__fmul_rn(v[e], f), dec);
            }
        }
        // stages 1, 2 and, between blocks, 16, 32, 64 here; 4 and 8 after the exchange
        if (p.rotate) butterfly<32>(y, 1, 16);
        __syncwarp();
#pragma unroll
        for (int b = 0; b < 8; ++b) row[kv_chunk(4 * b + i)] = make_float4(y[4 * b], y[4 * b + 1], y[4 * b + 2], y[4 * b + 3]);
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float4 v = row[kv_chunk(8 * i + k)];
            y[4 * k] = v.x;
            y[4 * k + 1] = v.y;
            y[4 * k + 2] = v.z;
            y[4 * k + 3] = v.w;
        }
        if (p.rotate) {
            butterfly<32>(y, 4, 8);
#pragma unroll
            for (int e = 0; e < 32; ++e) y[e] = __fmul_rn(y[e], __uint_as_float(0x3DB504F3u));
        }
        if (tok >= p.N) continue;
        void* const x = z ? p.v : p.k;
        const int64_t at = z ? tok * p.v_ts + h * p.v_hs : tok * p.k_ts + h * p.k_hs;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = y[8 * c + e];
            store_chunk<DT>(x, at + 32 * i + 8 * c, pack8<DT>(f));
        }
    }
}

static int kv_grid(const KvParams& p, int sms) {
    const int64_t tiles = (p.N + 15) / 16 * p.H, cap = (int64_t)sms * 8;
    return (int)(tiles < cap ? tiles : cap);
}
void launch_append(int dtype, const KvParams& p, int sms, cudaStream_t st) {
    const int grid = kv_grid(p, sms);
    if (dtype == HQ_DT_BF16) kv4_append_kernel<HQ_DT_BF16><<<grid, KV_THREADS, 0, st>>>(p);
    else if (dtype == HQ_DT_F16) kv4_append_kernel<HQ_DT_F16><<<grid, KV_THREADS, 0, st>>>(p);
    else kv4_append_kernel<HQ_DT_F32><<<grid, KV_THREADS, 0, st>>>(p);
}
void launch_gather(int dtype, const KvParams& p, int sms, cudaStream_t st) {
    const int grid = kv_grid(p, sms);
    if (dtype == HQ_DT_BF16) kv4_gather_kernel<HQ_DT_BF16><<<grid, KV_THREADS, 0, st>>>(p);
    else if (dtype == HQ_DT_F16) kv4_gather_kernel<HQ_DT_F16><<<grid, KV_THREADS, 0, st>>>(p);
    else kv4_gather_kernel<HQ_DT_F32><<<grid, KV_THREADS, 0, st>>>(p);
}

}  // namespace hq
