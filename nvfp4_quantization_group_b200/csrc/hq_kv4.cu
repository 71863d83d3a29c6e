// hq_kv4.cu -- block tables and slot maps, and the NVFP4 key/value cache:
// write new tokens, read tokens back (sm_100a).
#include "hq_layer.cuh"

namespace hq {

// ------------------------------------------------------------------- slots
// Three running sums over the requests (pages given back, pages taken, new
// tokens), 64 bits wide so that no sum of 32-bit lengths wraps unseen; then
// every page and every token finds its request by bisection of them.  Latency
// counts: one block, one barrier per dependent step, nothing per request that
// is longer than its share.  256 requests with a token each take 5.9 us, 64 with up
// to 2048 each 8.9 (a long slot map is filled by a second kernel over the GPU).
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
    let_next();  // (one block: the rest of the GPU is free for kv_slot_rows_kernel's)
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
    after_previous();
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
        launch_next(kv_slot_rows_kernel, dim3((unsigned)(blocks < cap ? blocks : cap)), dim3(256),
                    sizeof(int) * ((size_t)p.B + 1), st, p);
    }
}

// ------------------------------------------------------------ append, gather
// A tile is 16 consecutive tokens of one head, keys and values: 32 vectors, four
// threads each.  A thread has 32 consecutive elements on the side of the
// vectors and, on the side of the cache, elements 16 b + 4 i .. + 3 of every
// block b (i the thread of the four): the 16 bytes of keys' codes, or two times
// 8 bytes of values' codes, that lie together in a group.  The tokens of a tile
// usually fill one group, whose sectors are then written whole.  Append is bound by
// its instructions (issue slots 70 % busy): butterflies, exact quotients, conversions.
// Gather is not (57 %, 66 % of the copy rate as stored): with one tile in flight and a
// third of an SM's warps it waits for its loads.  16384 tokens x 8 heads in BF16: append
// 27 us (21 without the rotation), gather 24 rotated back and 20 as stored, where the
// bytes need 13.5 each; in FP32 42 (152 bytes spilled under the cap below), 40, 40 and
// 39 for 24.  Times are of twenty to thirty replays; append and gather called for a
// second take 49 us where they take 46 replayed.
constexpr int KV_THREADS = 128;
// Resident blocks that the registers are capped for: 16384 tokens x 8 heads
// written and read back take 46 us with 6, 48 uncapped (4 to 5), 54 with 5 or 7,
// 58 with 8 (spills).
constexpr int KV_BLOCKS = 6;

struct KvShared {
    // a vector's 32 chunks of four elements, chunk k of thread j (elements 32 j + 4 k ..) at 8 j + ((k + j) & 7); 36
    // per vector: the eight lanes of a quarter-warp (two vectors) hit different banks on both sides
    float4 t[32][36];
};
__device__ __forceinline__ int kv_chunk(int c) {  // place of chunk c (elements 4 c .. 4 c + 3)
    const int j = c >> 3, k = c & 7;
    return 8 * j + ((k + j) & 7);
}

// Stages h = first, 2 first, .. last of a butterfly over 32 values held as pairs
// (value 2 k, 2 k + 1 in y[k]).
__device__ __forceinline__ void butterfly(f2 (&y)[16], int first, int last) {
    if (first <= 1) {
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            float a, b;
            unpack2(y[k], a, b);
            y[k] = pack2(__fadd_rn(a, b), __fsub_rn(a, b));
        }
    }
#pragma unroll
    for (int h = 2; h < 32; h <<= 1) {
        if (h < first || h > last) continue;
#pragma unroll
        for (int k = 0; k < 16; ++k)
            if ((2 * k & h) == 0) {
                const f2 a = y[k], b = y[k + h / 2];
                y[k] = add2(a, b);
                y[k + h / 2] = sub2(a, b);
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
// same scales and conversions.  blockIdx.y is the head.
template <int DT> __global__ void __launch_bounds__(KV_THREADS, KV_BLOCKS) kv4_append_kernel(KvParams p) {
    __shared__ KvShared sh;
    __shared__ float2 vr[128];  // per E4M3 code {value, -RN(1 / value)}
    const int tid = threadIdx.x;
    {
        const bool zc = tid == 0 || tid == 127;
        const float v = zc ? 0.0f : e4m3_value(tid);
        vr[tid] = make_float2(v, zc ? -0.0f : -__frcp_rn(v));
    }
    __syncthreads();
    const int vec = tid >> 2, i = tid & 3, z = vec >> 4, h = blockIdx.y;
    float4* const row = sh.t[vec];
    const void* const x = z ? p.v : p.k;
    const int64_t ts = z ? p.v_ts : p.k_ts, first = (z ? p.v_hs : p.k_hs) * h + 32 * i;
    // the vector of the next tile is on its way while one is worked on (loaded whether its slot is in use or not)
    int64_t tok = (int64_t)blockIdx.x * 16 + (vec & 15), s = -1;
    Chunk<DT> u[2][2] = {};
    auto load = [&] {
        s = -1;
        if (tok >= p.N) return;
        s = p.slots[tok];
#pragma unroll
        for (int c = 0; c < 2; ++c) load_pair<DT>(x, tok * ts + first + 16 * c, p.wide, u[c]);
    };
    load();
    while (tok - (vec & 15) < p.N) {
        const int64_t slot = s;
        const bool ok = slot >= 0 && slot < p.n_slots;  // (the four threads of a vector agree)
        f2 y[16];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float f[8];
                unpack8<DT>(u[c][k], f);
#pragma unroll
                for (int e = 0; e < 4; ++e) y[8 * c + 4 * k + e] = pack2(f[2 * e], f[2 * e + 1]);
            }
        }
        tok += (int64_t)gridDim.x * 16;
        load();
        if (p.rotate) butterfly(y, 1, 16);
        __syncwarp();  // the last tile's reads are done
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            float4 v;
            unpack2(y[2 * k], v.x, v.y);
            unpack2(y[2 * k + 1], v.z, v.w);
            row[kv_chunk(8 * i + k)] = v;
        }
        __syncwarp();
#pragma unroll
        for (int b = 0; b < 8; ++b) {  // y[2 b], y[2 b + 1]: elements 16 b + 4 i .. + 3
            const float4 v = row[kv_chunk(4 * b + i)];
            y[2 * b] = pack2(v.x, v.y);
            y[2 * b + 1] = pack2(v.z, v.w);
        }
        if (p.rotate) {
            butterfly(y, 8, 16);  // elements 32 and 64 apart: two and four blocks
            const f2 c = pack2(__uint_as_float(0x3DB504F3u), __uint_as_float(0x3DB504F3u));  // RN(1 / sqrt(128))
#pragma unroll
            for (int k = 0; k < 16; ++k) y[k] = mul2(y[k], c);
        }
        float ab[8];
#pragma unroll
        for (int b = 0; b < 8; ++b) {
            float a0, a1, a2, a3;
            unpack2(y[2 * b], a0, a1);
            unpack2(y[2 * b + 1], a2, a3);
            ab[b] = absmax3(fmaxf(fabsf(a0), fabsf(a1)), a2, a3);
        }
        // the four threads' maxima of each block, thread i ending with blocks 2 i and 2 i + 1
        float m4[4], m2[2];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float mine = i & 2 ? ab[4 + k] : ab[k], other = i & 2 ? ab[k] : ab[4 + k];
            m4[k] = fmaxf(mine, __shfl_xor_sync(0xFFFFFFFFu, other, 2));
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float mine = i & 1 ? m4[2 + k] : m4[k], other = i & 1 ? m4[k] : m4[2 + k];
            m2[k] = fmaxf(mine, __shfl_xor_sync(0xFFFFFFFFu, other, 1));
        }
        float amax = fmaxf(m2[0], m2[1]);
        amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
        const float S = global_encode(amax);
        const bool slow = slow_scale(S);
        const uint32_t sf0 = block_sf(m2[0], S), sf1 = block_sf(m2[1], S);
        const float enc[2] = {block_enc(vr, sf0, S, slow), block_enc(vr, sf1, S, slow)};
        uint32_t codes[4];
#pragma unroll
        for (int b = 0; b < 8; b += 2) {
            float q[8];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float f = __shfl_sync(0xFFFFFFFFu, enc[k], b / 2, 4);
                const f2 f22 = pack2(f, f);
                unpack2(mul2(y[2 * (b + k)], f22), q[4 * k], q[4 * k + 1]);
                unpack2(mul2(y[2 * (b + k) + 1], f22), q[4 * k + 2], q[4 * k + 3]);
            }
            // bytes: block b pairs 0, 1; block b + 1 pairs 0, 1
            codes[b / 2] = e2m1x8(q[0], q[1], q[2], q[3], q[4], q[5], q[6], q[7]);
        }
        if (!ok) continue;
        uint8_t* const g = kv_group(p, slot, h);
        const int r = (int)(slot & 15), half = r >> 3, pair = (r & 7) >> 1, odd = r & 1;
        if (z == 0) {
            *reinterpret_cast<uint4*>(g + KV_K_CODES + r * 64 + i * 16) = make_uint4(codes[0], codes[1], codes[2], codes[3]);
            *reinterpret_cast<uint16_t*>(g + KV_K_SF + r * 8 + 2 * i) = (uint16_t)(sf0 | sf1 << 8);
            if (i == 1) reinterpret_cast<float*>(g + KV_K_DEC)[r] = __fdiv_rn(1.0f, S);
        } else {
            // byte pairs 2 i and 2 i + 1 of the eight blocks
            uint8_t* const o = g + KV_V_CODES + half * 512 + 2 * i * 64 + pair * 16 + odd * 8;
            *reinterpret_cast<uint2*>(o) = make_uint2(__byte_perm(codes[0], codes[1], 0x6420), __byte_perm(codes[2], codes[3], 0x6420));
            *reinterpret_cast<uint2*>(o + 64) = make_uint2(__byte_perm(codes[0], codes[1], 0x7531), __byte_perm(codes[2], codes[3], 0x7531));
            uint8_t* const f = g + KV_V_SF + half * 64 + pair * 16 + odd + 4 * i;  // blocks 2 i, 2 i + 1
            f[0] = (uint8_t)sf0;
            f[2] = (uint8_t)sf1;
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

template <int DT> __global__ void __launch_bounds__(KV_THREADS, KV_BLOCKS) kv4_gather_kernel(KvParams p) {
    __shared__ KvShared sh;
    const int tid = threadIdx.x, vec = tid >> 2, i = tid & 3, z = vec >> 4, h = blockIdx.y;
    float4* const row = sh.t[vec];
    void* const x = z ? p.v : p.k;
    const int64_t ts = z ? p.v_ts : p.k_ts, first = (z ? p.v_hs : p.k_hs) * h + 32 * i;
    // a tile's codes and scales are on their way while the one before is worked on, and the slot of the one after
    const int64_t step = (int64_t)gridDim.x * 16;
    int64_t tok = (int64_t)blockIdx.x * 16 + (vec & 15), s = tok < p.N ? p.slots[tok] : -1;
    uint4 codes, sf;  // keys: 16 bytes, 8 bytes; values: twice 8 bytes, 16 bytes with both tokens of the pair
    float dec;
    int odd;
    auto load = [&] {  // of slot s, then the next slot
        codes = sf = make_uint4(0u, 0u, 0u, 0u);
        dec = 0.0f;
        odd = (int)(s & 1);
        if (s >= 0 && s < p.n_slots) {
            const uint8_t* const g = kv_group(p, s, h);
            const int r = (int)(s & 15), half = r >> 3, pair = (r & 7) >> 1;
            if (z == 0) {
                codes = *reinterpret_cast<const uint4*>(g + KV_K_CODES + r * 64 + i * 16);
                const uint2 f = *reinterpret_cast<const uint2*>(g + KV_K_SF + r * 8);
                sf.x = f.x;
                sf.y = f.y;
            } else {
                const uint8_t* const o = g + KV_V_CODES + half * 512 + 2 * i * 64 + pair * 16 + odd * 8;
                const uint2 lo = *reinterpret_cast<const uint2*>(o), hi = *reinterpret_cast<const uint2*>(o + 64);
                codes = make_uint4(lo.x, lo.y, hi.x, hi.y);
                sf = *reinterpret_cast<const uint4*>(g + KV_V_SF + half * 64 + pair * 16);
            }
            dec = reinterpret_cast<const float*>(g + (z ? KV_V_DEC : KV_K_DEC))[r];
        }
        s = tok + step < p.N ? p.slots[tok + step] : -1;
    };
    load();
    while (tok - (vec & 15) < p.N) {
        f2 y[16];
        {
            uint32_t c[4] = {codes.x, codes.y, codes.z, codes.w}, f8[2] = {sf.x, sf.y};  // in the append kernel's order
            if (z) {
                c[0] = __byte_perm(codes.x, codes.z, 0x5140);
                c[1] = __byte_perm(codes.x, codes.z, 0x7362);
                c[2] = __byte_perm(codes.y, codes.w, 0x5140);
                c[3] = __byte_perm(codes.y, codes.w, 0x7362);
                const uint32_t pick = odd ? 0x7531 : 0x6420;
                f8[0] = __byte_perm(sf.x, sf.y, pick);
                f8[1] = __byte_perm(sf.z, sf.w, pick);
            }
            const f2 d2 = pack2(dec, dec);
#pragma unroll
            for (int b = 0; b < 8; ++b) {
                float v[4];
                e2m1x4_to_f32(c[b / 2] >> (16 * (b & 1)), v[0], v[1], v[2], v[3]);
                const float f = e4m3_value((f8[b / 4] >> (8 * (b & 3))) & 0xFFu);
                const f2 f22 = pack2(f, f);
                y[2 * b] = mul2(mul2(pack2(v[0], v[1]), f22), d2);
                y[2 * b + 1] = mul2(mul2(pack2(v[2], v[3]), f22), d2);
            }
        }
        const int64_t here = tok;
        tok += step;
        load();
        // stages 1, 2 and, between blocks, 16, 32, 64 here; 4 and 8 after the exchange
        if (p.rotate) butterfly(y, 1, 16);
        __syncwarp();
#pragma unroll
        for (int b = 0; b < 8; ++b) {
            float4 v;
            unpack2(y[2 * b], v.x, v.y);
            unpack2(y[2 * b + 1], v.z, v.w);
            row[kv_chunk(4 * b + i)] = v;
        }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float4 v = row[kv_chunk(8 * i + k)];
            y[2 * k] = pack2(v.x, v.y);
            y[2 * k + 1] = pack2(v.z, v.w);
        }
        if (p.rotate) {
            butterfly(y, 4, 8);
            const f2 c = pack2(__uint_as_float(0x3DB504F3u), __uint_as_float(0x3DB504F3u));
#pragma unroll
            for (int k = 0; k < 16; ++k) y[k] = mul2(y[k], c);
        }
        if (here >= p.N) continue;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            Chunk<DT> u[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float f[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) unpack2(y[8 * c + 4 * k + e], f[2 * e], f[2 * e + 1]);
                u[k] = pack8<DT>(f);
            }
            store_pair<DT>(x, here * ts + first + 16 * c, p.wide, u);
        }
    }
}

static dim3 kv_grid(const KvParams& p, int sms) {
    const int64_t tiles = (p.N + 15) / 16, cap = ((int64_t)sms * 2 * KV_BLOCKS + p.H - 1) / p.H;
    return dim3((unsigned)(tiles < cap ? tiles : cap), (unsigned)p.H);
}
void launch_append(int dtype, const KvParams& p, int sms, cudaStream_t st) {
    const dim3 grid = kv_grid(p, sms);
    if (dtype == HQ_DT_BF16) kv4_append_kernel<HQ_DT_BF16><<<grid, KV_THREADS, 0, st>>>(p);
    else if (dtype == HQ_DT_F16) kv4_append_kernel<HQ_DT_F16><<<grid, KV_THREADS, 0, st>>>(p);
    else kv4_append_kernel<HQ_DT_F32><<<grid, KV_THREADS, 0, st>>>(p);
}
void launch_gather(int dtype, const KvParams& p, int sms, cudaStream_t st) {
    const dim3 grid = kv_grid(p, sms);
    if (dtype == HQ_DT_BF16) kv4_gather_kernel<HQ_DT_BF16><<<grid, KV_THREADS, 0, st>>>(p);
    else if (dtype == HQ_DT_F16) kv4_gather_kernel<HQ_DT_F16><<<grid, KV_THREADS, 0, st>>>(p);
    else kv4_gather_kernel<HQ_DT_F32><<<grid, KV_THREADS, 0, st>>>(p);
}

}  // namespace hq
