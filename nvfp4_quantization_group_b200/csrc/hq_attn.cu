// hq_attn.cu -- attention of the newest tokens over the NVFP4 cache (sm_100a).
#include "hq_layer.cuh"

namespace hq {

constexpr int ATTN_COLS = 8, ATTN_WARPS = 4;

__device__ __forceinline__ float e2m1_value4(uint32_t c) {
    const uint32_t m = c & 7u;
    const float v = m < 2u ? 0.5f * (float)m : __uint_as_float(((m >> 1) + 126u) << 23 | (m & 1u) << 22);
    return c & 8u ? -v : v;
}

// Unnormalised 128-point butterfly over a warp, lane l with elements 4 l ..
// 4 l + 3, and the factor 1 / sqrt(128).
__device__ __forceinline__ void rotate_warp(float (&y)[4], int lane) {
    const float a = y[0] + y[1], b = y[0] - y[1], c = y[2] + y[3], d = y[2] - y[3];
    y[0] = a + c;
    y[1] = b + d;
    y[2] = a - c;
    y[3] = b - d;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float other = __shfl_xor_sync(0xFFFFFFFFu, y[i], o);
            y[i] = lane & o ? other - y[i] : y[i] + other;
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] *= 0.08838834764831845f;
}

// One block per (request, key/value head, 8 columns); a column is one query
// head of one query token.  A warp takes every fourth token, a lane four
// dimensions of it.
template <int DT> __global__ void __launch_bounds__(32 * ATTN_WARPS) kv4_attention_kernel(AttnParams p) {
    typedef typename Elem<DT>::T T;
    __shared__ float so[ATTN_WARPS][ATTN_COLS][128], sm[ATTN_WARPS][ATTN_COLS], sl[ATTN_WARPS][ATTN_COLS];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, quad = lane & 3, blk = lane >> 2;
    const int b = blockIdx.x, kvh = blockIdx.y, col0 = blockIdx.z * ATTN_COLS;
    int64_t q0 = p.cu_q ? p.cu_q[b] : (int64_t)b * p.q_len, q1 = p.cu_q ? p.cu_q[b + 1] : q0 + p.q_len;
    if (q0 < 0) q0 = 0;
    if (q1 > p.Tq) q1 = p.Tq;
    const int nq = (int)(q1 - q0 < 0 ? 0 : (q1 - q0 > p.q_len ? p.q_len : q1 - q0)), cols = nq * p.group;
    if (col0 >= cols) return;
    const int64_t row_tokens = p.width << p.page_shift;
    int len = p.lens[b];
    bool bad = false;
    if (len > row_tokens) {
        bad = true;
        len = (int)row_tokens;
    }
    const int pos_last = p.lens[b] - 1;
    const int groups = 1 << (p.page_shift - 4);
    float q[ATTN_COLS][4], o[ATTN_COLS][4] = {}, m[ATTN_COLS], l[ATTN_COLS] = {};
    int pos[ATTN_COLS];
#pragma unroll
    for (int c = 0; c < ATTN_COLS; ++c) {
        const int col = col0 + c;
        m[c] = -INFINITY;
        pos[c] = -1;
        if (col < cols) {
            const int j = col / p.group;
            const T* x = static_cast<const T*>(p.q) + (q0 + j) * p.q_ts + (kvh * p.group + col % p.group) * p.q_hs;
            pos[c] = pos_last - (nq - 1 - j);
#pragma unroll
            for (int e = 0; e < 4; ++e) q[c][e] = to_f32(x[4 * lane + e]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) q[c][e] = 0.0f;
        }
        if (p.rotate) rotate_warp(q[c], lane);
    }
    for (int t = w; t < len; t += ATTN_WARPS) {
        const int page = p.table[b * p.width + (t >> p.page_shift)];
        if (page < 0 || page >= p.num_pages) {
            bad = true;
            continue;
        }
        const uint8_t* g = p.cache + (((int64_t)page * p.Hkv + kvh) * groups + ((t & ((1 << p.page_shift) - 1)) >> 4)) * KV_GROUP_BYTES;
        const int r = t & 15, half = r >> 3, pair = (r & 7) >> 1, odd = r & 1;
        const uint32_t kc = *reinterpret_cast<const uint16_t*>(g + KV_K_CODES + r * 64 + quad * 16 + blk * 2);
        const float ks = e4m3_value(g[KV_K_SF + r * 8 + blk]) * reinterpret_cast<const float*>(g + KV_K_DEC)[r];
        const uint8_t* vo = g + KV_V_CODES + half * 512 + pair * 16 + odd * 8 + blk;
        const uint32_t vc = vo[(2 * quad) * 64] | (uint32_t)vo[(2 * quad + 1) * 64] << 8;
        const float vs = e4m3_value(g[KV_V_SF + half * 64 + pair * 16 + blk * 2 + odd]) * reinterpret_cast<const float*>(g + KV_V_DEC)[r];
        float k[4], v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            k[e] = e2m1_value4(kc >> (4 * e)) * ks;
            v[e] = e2m1_value4(vc >> (4 * e)) * vs;
        }
#pragma unroll
        for (int c = 0; c < ATTN_COLS; ++c) {
            float s = 0.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e) s = __fmaf_rn(q[c][e], k[e], s);
            s = warp_sum(s) * p.scale;
            const bool see = t <= pos[c] && (p.window == 0 || pos[c] - t < p.window || t < p.sinks);
            if (!see) continue;
            const float mn = fmaxf(m[c], s), a = expf(m[c] - mn), e = expf(s - mn);
            m[c] = mn;
            l[c] = l[c] * a + e;
#pragma unroll
            for (int i = 0; i < 4; ++i) o[c][i] = __fmaf_rn(o[c][i], a, e * v[i]);
        }
    }
    if (bad && lane == 0) p.ws[2] = HQ_ERR_PAGE;
#pragma unroll
    for (int c = 0; c < ATTN_COLS; ++c) {
#pragma unroll
        for (int i = 0; i < 4; ++i) so[w][c][4 * lane + i] = o[c][i];
        if (lane == 0) {
            sm[w][c] = m[c];
            sl[w][c] = l[c];
        }
    }
    __syncthreads();
    for (int c = w; c < ATTN_COLS; c += ATTN_WARPS) {
        const int col = col0 + c;
        if (col >= cols) continue;
        float mx = -INFINITY, total = 0.0f, y[4] = {};
        for (int i = 0; i < ATTN_WARPS; ++i) mx = fmaxf(mx, sm[i][c]);
        for (int i = 0; i < ATTN_WARPS; ++i) {
            if (sl[i][c] == 0.0f) continue;
            const float a = expf(sm[i][c] - mx);
            total += sl[i][c] * a;
            for (int e = 0; e < 4; ++e) y[e] += so[i][c][4 * lane + e] * a;
        }
        for (int e = 0; e < 4; ++e) y[e] = total > 0.0f ? y[e] / total : 0.0f;
        if (p.rotate) rotate_warp(y, lane);
        const int j = col / p.group, head = kvh * p.group + col % p.group;
        T* out = static_cast<T*>(p.out) + (q0 + j) * p.o_ts + head * p.o_hs;
        for (int e = 0; e < 4; ++e) out[4 * lane + e] = from_f32<DT>(y[e]);
        if (p.lse && lane == 0)
            p.lse[(q0 + j) * (int64_t)(p.Hkv * p.group) + head] = total > 0.0f ? mx + logf(total) : -INFINITY;
    }
}

size_t attn_workspace_bytes() { return 256; }

int launch_attn(int dtype, const AttnParams& p, int sms, cudaStream_t st) {
    (void)sms;
    const dim3 grid((unsigned)p.B, (unsigned)p.Hkv, (unsigned)((p.q_len * p.group + ATTN_COLS - 1) / ATTN_COLS));
    if (dtype == HQ_DT_BF16) kv4_attention_kernel<HQ_DT_BF16><<<grid, 32 * ATTN_WARPS, 0, st>>>(p);
    else kv4_attention_kernel<HQ_DT_F16><<<grid, 32 * ATTN_WARPS, 0, st>>>(p);
    return (int)cudaPeekAtLastError();
}

}  // namespace hq
