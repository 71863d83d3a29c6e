// hq_attn.cu -- attention of the newest tokens over the NVFP4 cache (sm_100a).
//
// For the columns n of one (request, key/value head) -- a column is one query
// head of one query token, NC = 8 or 16 of them at a time -- and its tokens t
//   s_tn = scale * q_n . k_t,  o_n = sum_t exp(s_tn - m_n) v_t,  l_n = sum_t exp(s_tn - m_n).
// A warp takes groups of 16 tokens.  Both products are m16n8k16 matrix
// instructions with the columns as their n side, so that 8 query heads of one
// key/value head fill them:
//   S^T [16 tokens, n] = K [16, 128] q^T     (8 instructions a part of q)
//   O^T [16 d,      n] += V^T [16 d, 16 t] P^T  (8 instructions, one per 16-element block)
// A code times its block scale has 6 significant bits and lies within FP16's
// range, subnormals included: both operands are widened exactly.  (A block scale
// covers exactly one instruction's depth, K, or height, V.)  The decode scales
// multiply the scores and the weights in FP32.  q is split into two FP16 parts
// (hi + lo, 22 bits), so scores are FP32-like.  The weights P are rounded to FP16
// once for BF16 outputs, whose own rounding is eight times as coarse; for FP16
// outputs they too go in two parts (the error against 64 bits is then the output's
// own, 2.1e-4, where one part gives 2.9e-4; 117 -> 122 us at the sizes below).
// The cache's byte order gives each lane its operands of a group as 16-byte
// pieces (four for the codes, three for the block scales).  A warp takes one
// or two groups (a unit) at a time, copied into its own ring by bulk copies that
// run one unit ahead, so warps never wait for one another inside a row; both
// groups of a unit that every column sees go through one stretch of code.
//
// The running maximum moves only when a lane's weights exceed 64, so the usual
// group needs no exchange between lanes.  The decode scales of V are folded into
// the weights: what goes into FP16 is c = weight * decode scale, times a power of
// two per column that follows the largest c of the tokens that the column sees (as
// the maximum does, 2^9 to 2^15), never a token's scale alone: a large value without
// weight, outside the window, or a vector of zeros (its decode scale is 1) leaves the
// others their bits.  A c is good to 2^-11 down to 2^-23 of that largest one, to
// 2^-34 of it below.
//
// Bound: the codes and scales are 152 bytes per token and key/value head, but a
// group also costs about 370 warp instructions, 64 of them conversions of code
// pairs at half rate.  32 requests of 8000 to 16384 tokens, 64 query and 8
// key/value heads: 117 us replayed 30 times, 4.1 TB/s (63 % of the measured copy
// rate), 126 to 128 us called for a second.  Nothing is full (issue slots 58 % busy,
// ALU 52 %, matrix 30 %): what limits it now is latency at four warps a scheduler
// (128 registers each, 40 bytes of them spilled; 96 would spill more).  Steps there:
// one group a turn 166, two 133, look-ups by whole lanes 121, both groups' scores
// together 114, contributions in place of decode scales 118, their range checked
// once a unit 117.  (These
// matrix instructions, not tcgen05: that one reads its operands from shared memory,
// where K and V would have to be widened first: 512 bytes per token and head
// written and read again, 8 clocks of an SM's shared memory beside the 2.4 of the
// codes, where the whole loop takes 10.)
#include "hq_layer.cuh"

namespace hq {

constexpr int ATTN_STAGES = 2;       // units in flight per warp
// Units that a row's start and end (its q, the joins) are worth.  48 requests with
// a window of 2047 tokens and up to 20 columns take 39.4 us with 10, 36.6 with 16,
// 36.0 with 24, 35.5 with 28; 16 requests of 12000 tokens 41.1, 39.5, 38.2, 38.3; a
// batch of 4 short requests 10.8, 10.7, 11.0, 11.0 (a cost that goes by the units'
// size takes a register too many: 115 us instead of 114 for the largest batch).
constexpr int ATTN_ROW_COST = 24;
constexpr int ATTN_MAX_CTAS = 512;   // workspace: CTAs of a launch at most
constexpr int ATTN_MAX_NC = 16;
constexpr int ATTN_PART = ATTN_MAX_NC * (128 + 4);  // floats of one partial result: sums, {maximum, sum, power of two}
constexpr float ATTN_NONE = -1e30f;  // running maximum before any token

// ---------------------------------------------------------------- schedule
// Units of one or two groups (16 << us tokens, us = 0 or 1) are numbered request
// by request, then (head, column tile) row by row, then in the order of the
// tokens.  Each row counts ATTN_ROW_COST units more than it has, in front of them:
// what starting and ending a row costs.  CTA c of G takes units [U c / G,
// U (c + 1) / G), a cut in a row's front part (or right behind it) moved to the
// row's start: about the same load for every CTA whatever the lengths.
struct Request {
    int q0, nq;       // first row of q, query tokens
    int len;          // tokens (clamped to the block table's row)
    int last;         // position of the last query
    int tiles;        // column tiles
    int sink_units;   // units of the first tokens, before the window's
    int first_unit;   // the window's first unit
    int n;            // units per row, ATTN_ROW_COST among them (no tokens: one more)
    bool bad;         // the length exceeds the block table's row
};

__device__ __forceinline__ Request attn_request(const AttnParams& p, int b, int nc, int us) {
    Request r;
    const int ut = 16 << us;
    int64_t a = p.cu_q ? p.cu_q[b] : (int64_t)b * p.q_len, e = p.cu_q ? p.cu_q[b + 1] : a + p.q_len;
    a = a < 0 ? 0 : a;
    e = e > p.Tq ? p.Tq : e;
    r.q0 = (int)a;
    r.nq = (int)(e - a < 0 ? 0 : (e - a > p.q_len ? p.q_len : e - a));
    const int64_t row = p.width << p.page_shift;
    const int len = p.lens[b];
    r.last = len - 1;
    r.bad = len > row;
    r.len = len < 0 ? 0 : (r.bad ? (int)row : len);
    r.tiles = (r.nq * p.group + nc - 1) / nc;
    // the window's first token (lengths are below 2^30: host check)
    const int64_t first = (int64_t)r.last - r.nq + 1 - p.window + 1;
    const int lo = p.window > 0 && first > 0 ? (int)min(first, (int64_t)r.len) : 0;
    r.first_unit = lo >> (4 + us);
    r.sink_units = min((min(p.sinks, lo) + ut - 1) >> (4 + us), r.first_unit);
    r.n = r.nq ? ATTN_ROW_COST + max(1, r.sink_units + ((r.len + ut - 1) >> (4 + us)) - r.first_unit) : 0;
    return r;
}

// A CTA's walk over its pieces: a piece is a run of units of one row.
struct Walk {
    Request r;
    int b, row, head;     // request, row (head, column tile) of it, the row's head
    int ja, jb;           // units of the piece: [ja, jb) of r.n (the first ATTN_ROW_COST have no tokens)
    uint64_t at, end;     // next unit, end of the CTA's units
    bool live;
};

struct Sched {
    uint64_t U;
    uint32_t G;
};

// The CTA that holds unit u of a row's own units.
__device__ __forceinline__ uint32_t cta_of(const Sched& s, uint64_t u) { return (uint32_t)(((u + 1) * s.G - 1) / s.U); }
// The request that holds unit u: pre[b] <= u < pre[b + 1].
__device__ __forceinline__ int request_of(const AttnParams& p, const uint64_t* pre, uint64_t u) {
    int lo = 0, hi = p.B - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (pre[mid + 1] > u) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}
__device__ __forceinline__ void walk_piece(const uint64_t* pre, Walk& w) {
    w.live = w.at < w.end;
    if (!w.live) return;
    const uint64_t in = w.at - pre[w.b];
    w.row = (int)(in / (uint32_t)w.r.n);
    w.head = w.row / w.r.tiles;
    w.ja = (int)(in - (uint64_t)w.row * w.r.n);
    const uint64_t left = w.end - w.at;
    w.jb = left < (uint64_t)(w.r.n - w.ja) ? w.ja + (int)left : w.r.n;
}
// The first unit of CTA c (U for c == G), and where it lies (only for c < G): w.at, b, r, row, ja.
__device__ __forceinline__ void walk_cut(const AttnParams& p, const uint64_t* pre, int nc, int us, const Sched& s, uint32_t c,
                                         Walk& w) {
    w.at = s.U * c / s.G;
    if (c == s.G) return;
    w.b = request_of(p, pre, w.at);
    w.r = attn_request(p, w.b, nc, us);
    const uint64_t in = w.at - pre[w.b];
    w.row = (int)(in / (uint32_t)w.r.n);
    w.ja = (int)(in - (uint64_t)w.row * w.r.n);
    if (w.ja <= ATTN_ROW_COST) {
        w.at -= w.ja;
        w.ja = 0;
    }
}
// The rest of the piece that starts there, up to unit `end` at most.
__device__ __forceinline__ void walk_start(Walk& w, uint64_t end) {
    w.end = end;
    w.live = w.at < end;
    if (!w.live) return;
    w.head = w.row / w.r.tiles;
    const uint64_t left = end - w.at;
    w.jb = left < (uint64_t)(w.r.n - w.ja) ? w.ja + (int)left : w.r.n;
}
__device__ __forceinline__ void walk_next(const AttnParams& p, const uint64_t* pre, int nc, int us, Walk& w) {
    w.at += (uint64_t)(w.jb - w.ja);
    if (w.at < w.end && w.at >= pre[w.b + 1]) {
        do ++w.b;
        while (w.at >= pre[w.b + 1]);
        w.r = attn_request(p, w.b, nc, us);
    }
    walk_piece(pre, w);
}

// ------------------------------------------------------------------ device
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// Four bytes of E2M1 pairs -> four FP16 pairs (low nibble in the low half).
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(w));
}
// Two pairs of E4M3 bytes -> two FP16 pairs (exact).
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}" : "=r"(lo), "=r"(hi) : "r"(w));
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same with a zero addend.
__device__ __forceinline__ void mma16816_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ uint32_t hmul2u(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// A pair times the low (HI: high) half of `f`.
template <bool HI> __device__ __forceinline__ uint32_t hmul2_half(uint32_t a, uint32_t f) {
    const __half2 s = *reinterpret_cast<const __half2*>(&f);
    const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), HI ? __high2half2(s) : __low2half2(s));
    return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ float2 h2f(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2*>(&v)); }
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 :: "r"(dst), "l"(src), "r"(bytes), "r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void mbar_arrive_expect(uint64_t* bar, uint32_t bytes) {
    asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;\n\t}"
                 :: "r"(smem_u32(bar)), "r"(bytes) : "memory");
}

__device__ __forceinline__ uint32_t arrive(uint32_t* p) {
    uint32_t r;
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(r) : "l"(p) : "memory");
    return r;
}

// 128-point butterfly over a warp, lane l with elements 4 l .. 4 l + 3, and
// the factor 1 / sqrt(128).
__device__ __forceinline__ void rotate_warp(float (&y)[4], int lane) {
    const float a = __fadd_rn(y[0], y[1]), b = __fsub_rn(y[0], y[1]), c = __fadd_rn(y[2], y[3]), d = __fsub_rn(y[2], y[3]);
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
    for (int i = 0; i < 4; ++i) y[i] = __fmul_rn(y[i], 0.08838834764831845f);
}

// Shared memory of a CTA of W warps with NC columns.
template <int NT, int W> struct AttnShared {
    static constexpr int NC = 8 * NT, OS = 132;  // columns; padded row of the merge buffer (free of bank conflicts)
    alignas(128) uint8_t ring[W][ATTN_STAGES][2 * KV_GROUP_BYTES];
    union {  // one after the other within a row
        uint4 q[NT][8][32];               // per block and lane: hi and lo parts of its four elements of column lane / 4
        float4 frag[W / 2][NT * 8][32];   // accumulators of the upper half's warps
        float o[W / 2][NC][OS];           // results of the lower half's warps
    };
    float2 mz[W][NC];  // a warp's maximum and power of two of each column
    float l[W][NC];
    float qs[NC];  // factor of a column's scores, in powers of two
    int pos[NC];   // a column's position
    Walk cw, nw;   // the CTA's current piece and the one after it
    Walk lw[W];    // the piece of each warp's next load
    uint64_t full[W][ATTN_STAGES];
    ulonglong2 warp_sums[W];
    int last;
    // then the units before each request, uint64_t [B + 1]
};

// What a lane carries through a row.
template <int NT> struct AttnState {
    float o[NT][8][4];  // O^T: block b, rows d = 16 b + 2 g (0, 1) and + 1 (2, 3), columns 2 i, 2 i + 1
    float m[NT][2], l[NT][2];  // m: an integer, so that what moves with it are powers of two
    float cz[NT][2];           // power of two that the second product's weights carry
    float qs[NT][2];
};
constexpr float ATTN_CZ_MOST = 8.507059173023462e37f;  // 2^126, before any contribution
__device__ __forceinline__ int pow2_of(float x) { return (int)(__float_as_uint(x) >> 23) - 127; }  // x: normal, > 0
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }  // e: -126 .. 127

// Scores (in powers of two) of the group at `grp`: rows g, g + 8, columns 2 i,
// 2 i + 1.
template <int NT>
__device__ __forceinline__ void attn_scores(const uint8_t* grp, const uint4 (*q)[8][32], const AttnState<NT>& a, int lane,
                                            float (&s)[NT][4]) {
    const int g = lane >> 2;
    const uint4 k0 = *reinterpret_cast<const uint4*>(grp + KV_K_CODES + lane * 16);
    const uint4 k1 = *reinterpret_cast<const uint4*>(grp + KV_K_CODES + lane * 16 + 512);
    const uint2 f0 = *reinterpret_cast<const uint2*>(grp + KV_K_SF + g * 8);
    const uint2 f1 = *reinterpret_cast<const uint2*>(grp + KV_K_SF + g * 8 + 64);
    const uint32_t kw0[4] = {k0.x, k0.y, k0.z, k0.w}, kw1[4] = {k1.x, k1.y, k1.z, k1.w};
    uint32_t sf0[4], sf1[4];
    e4m3x4_to_f16(f0.x, sf0[0], sf0[1]);
    e4m3x4_to_f16(f0.y, sf0[2], sf0[3]);
    e4m3x4_to_f16(f1.x, sf1[0], sf1[1]);
    e4m3x4_to_f16(f1.y, sf1[2], sf1[3]);
    // four running products (hi and lo parts, even and odd pairs of blocks): short chains
    float c[NT][4][4];
#pragma unroll
    for (int b2 = 0; b2 < 4; ++b2) {  // blocks 2 b2, 2 b2 + 1
        uint32_t a0[4], a1[4];
        e2m1x8_to_f16(kw0[b2], a0);
        e2m1x8_to_f16(kw1[b2], a1);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint32_t m0 = k ? hmul2_half<true>(a0[2], sf0[b2]) : hmul2_half<false>(a0[0], sf0[b2]);
            const uint32_t m1 = k ? hmul2_half<true>(a1[2], sf1[b2]) : hmul2_half<false>(a1[0], sf1[b2]);
            const uint32_t m2 = k ? hmul2_half<true>(a0[3], sf0[b2]) : hmul2_half<false>(a0[1], sf0[b2]);
            const uint32_t m3 = k ? hmul2_half<true>(a1[3], sf1[b2]) : hmul2_half<false>(a1[1], sf1[b2]);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint4 f = q[n][2 * b2 + k][lane];
                const int z = 2 * (b2 & 1);
                if (b2 < 2 && k == 0) {
                    mma16816_first(c[n][z], m0, m1, m2, m3, f.x, f.y);
                    mma16816_first(c[n][z + 1], m0, m1, m2, m3, f.z, f.w);
                } else {
                    mma16816(c[n][z], m0, m1, m2, m3, f.x, f.y);
                    mma16816(c[n][z + 1], m0, m1, m2, m3, f.z, f.w);
                }
            }
        }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] = (c[n][0][e] + c[n][2][e]) + (c[n][1][e] + c[n][3][e]);
    const float d0 = *reinterpret_cast<const float*>(grp + KV_K_DEC + 4 * g);
    const float d1 = *reinterpret_cast<const float*>(grp + KV_K_DEC + 4 * g + 32);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        s[n][0] = __fmul_rn(s[n][0], __fmul_rn(d0, a.qs[n][0]));
        s[n][1] = __fmul_rn(s[n][1], __fmul_rn(d0, a.qs[n][1]));
        s[n][2] = __fmul_rn(s[n][2], __fmul_rn(d1, a.qs[n][0]));
        s[n][3] = __fmul_rn(s[n][3], __fmul_rn(d1, a.qs[n][1]));
    }
}

// The same of the two groups of a unit, block by block: q is read once for both,
// and one running product each is enough (two each: 117 us at the sizes above, the
// groups one after the other with four: 118).
template <int NT>
__device__ __forceinline__ void attn_scores2(const uint8_t* unit, const uint4 (*q)[8][32], const AttnState<NT>& a, int lane,
                                             float (&s)[2][NT][4]) {
    const int g = lane >> 2;
    uint32_t kw[2][2][4], sf[2][2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const uint8_t* grp = unit + h * KV_GROUP_BYTES;
            const uint4 k = *reinterpret_cast<const uint4*>(grp + KV_K_CODES + lane * 16 + 512 * r);
            const uint2 f = *reinterpret_cast<const uint2*>(grp + KV_K_SF + g * 8 + 64 * r);
            kw[h][r][0] = k.x;
            kw[h][r][1] = k.y;
            kw[h][r][2] = k.z;
            kw[h][r][3] = k.w;
            e4m3x4_to_f16(f.x, sf[h][r][0], sf[h][r][1]);
            e4m3x4_to_f16(f.y, sf[h][r][2], sf[h][r][3]);
        }
    float c[2][NT][4];
#pragma unroll
    for (int b2 = 0; b2 < 4; ++b2) {
        uint32_t a0[2][4], a1[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            e2m1x8_to_f16(kw[h][0][b2], a0[h]);
            e2m1x8_to_f16(kw[h][1][b2], a1[h]);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            uint4 f[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) f[n] = q[n][2 * b2 + k][lane];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t x0 = sf[h][0][b2], x1 = sf[h][1][b2];
                const uint32_t m0 = k ? hmul2_half<true>(a0[h][2], x0) : hmul2_half<false>(a0[h][0], x0);
                const uint32_t m1 = k ? hmul2_half<true>(a1[h][2], x1) : hmul2_half<false>(a1[h][0], x1);
                const uint32_t m2 = k ? hmul2_half<true>(a0[h][3], x0) : hmul2_half<false>(a0[h][1], x0);
                const uint32_t m3 = k ? hmul2_half<true>(a1[h][3], x1) : hmul2_half<false>(a1[h][1], x1);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if (b2 == 0 && k == 0) {
                        mma16816_first(c[h][n], m0, m1, m2, m3, f[n].x, f[n].y);
                        mma16816(c[h][n], m0, m1, m2, m3, f[n].z, f[n].w);
                    } else {
                        mma16816(c[h][n], m0, m1, m2, m3, f[n].x, f[n].y);
                        mma16816(c[h][n], m0, m1, m2, m3, f[n].z, f[n].w);
                    }
                }
            }
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint8_t* grp = unit + h * KV_GROUP_BYTES;
        const float d0 = *reinterpret_cast<const float*>(grp + KV_K_DEC + 4 * g);
        const float d1 = *reinterpret_cast<const float*>(grp + KV_K_DEC + 4 * g + 32);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            s[h][n][0] = __fmul_rn(c[h][n][0], __fmul_rn(d0, a.qs[n][0]));
            s[h][n][1] = __fmul_rn(c[h][n][1], __fmul_rn(d0, a.qs[n][1]));
            s[h][n][2] = __fmul_rn(c[h][n][2], __fmul_rn(d1, a.qs[n][0]));
            s[h][n][3] = __fmul_rn(c[h][n][3], __fmul_rn(d1, a.qs[n][1]));
        }
    }
}

// Weights of N groups (the first at `grp`) from their scores s and decode scales v
// (of rows g, g + 8), as FP16 pairs u (FINE: their rest in lo) for the second
// product; the weights are summed.  Where a lane's weights or contributions leave
// their range, the running maxima go up to the scores, and the columns' powers of
// two to where the largest contribution is 2^9 to 2^10.
template <int NT, int N, bool FINE>
__device__ __forceinline__ void attn_weigh(AttnState<NT>& a, const float (&s)[N][NT][4], float (&v)[N][2], const uint8_t* grp,
                                           int lane, uint32_t (&u)[N][NT][2], uint32_t (&lo)[N][NT][2]) {
    float sum[NT][2];
    auto weigh = [&] {  // returns the largest of what goes into FP16
        float most = 0.0f;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int h = 0; h < N; ++h) {
                const float e0 = ex2(s[h][n][0] - a.m[n][0]), e1 = ex2(s[h][n][1] - a.m[n][1]);
                const float e2 = ex2(s[h][n][2] - a.m[n][0]), e3 = ex2(s[h][n][3] - a.m[n][1]);
                sum[n][0] = h ? sum[n][0] + (e0 + e2) : e0 + e2;
                sum[n][1] = h ? sum[n][1] + (e1 + e3) : e1 + e3;
                const float w0 = e0 * v[h][0] * a.cz[n][0], w1 = e1 * v[h][0] * a.cz[n][1];
                const float w2 = e2 * v[h][1] * a.cz[n][0], w3 = e3 * v[h][1] * a.cz[n][1];
                most = max3(max3(most, w0, w1), w2, w3);
                u[h][n][0] = pack_h2(w0, w1);
                u[h][n][1] = pack_h2(w2, w3);
                if constexpr (FINE) {
                    const float2 a0 = h2f(u[h][n][0]), a1 = h2f(u[h][n][1]);
                    lo[h][n][0] = pack_h2(w0 - a0.x, w1 - a0.y);
                    lo[h][n][1] = pack_h2(w2 - a1.x, w3 - a1.y);
                }
            }
        return most;
    };
    bool big = weigh() > 32768.0f;
#pragma unroll
    for (int n = 0; n < NT; ++n) big |= fmaxf(sum[n][0], sum[n][1]) > 64.0f;
    if (__any_sync(0xFFFFFFFFu, big)) {
        // vectors of zeros contribute nothing: all eight block scales of the token are zero
        const int g = lane >> 2;
#pragma unroll
        for (int h = 0; h < N; ++h)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const uint4 f = *reinterpret_cast<const uint4*>(grp + h * KV_GROUP_BYTES + KV_V_SF + 64 * r + 16 * (g >> 1));
                if (((f.x | f.y | f.z | f.w) & 0x00FF00FFu << 8 * (g & 1)) == 0) v[h][r] = 0.0f;
            }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float t = fmaxf(s[0][n][k], s[0][n][2 + k]);
#pragma unroll
                for (int h = 1; h < N; ++h) t = max3(t, s[h][n][k], s[h][n][2 + k]);
#pragma unroll
                for (int y = 4; y <= 16; y <<= 1) t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, y));
                t = fmaxf(a.m[n][k], ceilf(t));
                const float d = a.m[n][k] - t;
                a.m[n][k] = t;
                a.l[n][k] *= ex2(d);
                float c = 0.0f;
#pragma unroll
                for (int h = 0; h < N; ++h) c = max3(c, ex2(s[h][n][k] - t) * v[h][0], ex2(s[h][n][2 + k] - t) * v[h][1]);
#pragma unroll
                for (int y = 4; y <= 16; y <<= 1) c = fmaxf(c, __shfl_xor_sync(0xFFFFFFFFu, c, y));
                // the accumulators' own power of two moves against the maximum (e), but not above 2^126 or to where the
                // largest contribution leaves FP16's range; the rest falls to them
                const float e = (float)pow2_of(a.cz[n][k]) - d, z = fminf(fminf(e, 126.0f), (float)(9 - pow2_of(c)));
                const float f = ex2(z - e);
                a.cz[n][k] = pow2((int)z);
#pragma unroll
                for (int b = 0; b < 8; ++b) {
                    a.o[n][b][k] *= f;
                    a.o[n][b][2 + k] *= f;
                }
            }
        weigh();
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        a.l[n][0] += sum[n][0];
        a.l[n][1] += sum[n][1];
    }
}

// Adds the group's weighted values.  u, lo: its weights (attn_weigh); keep0, keep1:
// the bytes to keep of the block scales of the lane's tokens 2 i, 2 i + 1 and
// 2 i + 8, + 9.
template <int NT, bool MASK, bool FINE>
__device__ __forceinline__ void attn_values(const uint8_t* grp, AttnState<NT>& a, const uint32_t (&u)[NT][2],
                                            const uint32_t (&lo)[NT][2], uint32_t keep0, uint32_t keep1, int lane) {
    uint4 vf0 = *reinterpret_cast<const uint4*>(grp + KV_V_SF + (lane & 3) * 16);
    uint4 vf1 = *reinterpret_cast<const uint4*>(grp + KV_V_SF + (lane & 3) * 16 + 64);
    if constexpr (MASK) {
        vf0 = make_uint4(vf0.x & keep0, vf0.y & keep0, vf0.z & keep0, vf0.w & keep0);
        vf1 = make_uint4(vf1.x & keep1, vf1.y & keep1, vf1.z & keep1, vf1.w & keep1);
    }
    uint32_t pb[NT][2], pl[NT][2];  // weights as the n side: column g, tokens 2 i, 2 i + 1 and 2 i + 8, + 9; FINE: their rest
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        pb[n][0] = transpose8x8(u[n][0]);
        pb[n][1] = transpose8x8(u[n][1]);
        if constexpr (FINE) {
            pl[n][0] = transpose8x8(lo[n][0]);
            pl[n][1] = transpose8x8(lo[n][1]);
        }
    }
    const uint4 c0 = *reinterpret_cast<const uint4*>(grp + KV_V_CODES + lane * 16);
    const uint4 c1 = *reinterpret_cast<const uint4*>(grp + KV_V_CODES + lane * 16 + 512);
    const uint32_t ev0[2] = {c0.x, c0.y}, od0[2] = {c0.z, c0.w}, ev1[2] = {c1.x, c1.y}, od1[2] = {c1.z, c1.w};
    const uint32_t fw0[4] = {vf0.x, vf0.y, vf0.z, vf0.w}, fw1[4] = {vf1.x, vf1.y, vf1.z, vf1.w};
#pragma unroll
    for (int q = 0; q < 2; ++q) {  // blocks 4 q .. 4 q + 3
        uint32_t ea[4], oa[4], eb[4], ob[4], x0[4], x1[4];
        e2m1x8_to_f16(ev0[q], ea);
        e2m1x8_to_f16(od0[q], oa);
        e2m1x8_to_f16(ev1[q], eb);
        e2m1x8_to_f16(od1[q], ob);
        e4m3x4_to_f16(fw0[2 * q], x0[0], x0[1]);
        e4m3x4_to_f16(fw0[2 * q + 1], x0[2], x0[3]);
        e4m3x4_to_f16(fw1[2 * q], x1[0], x1[1]);
        e4m3x4_to_f16(fw1[2 * q + 1], x1[2], x1[3]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t a0 = hmul2u(__byte_perm(ea[k], oa[k], 0x5410), x0[k]);
            const uint32_t a1 = hmul2u(__byte_perm(ea[k], oa[k], 0x7632), x0[k]);
            const uint32_t a2 = hmul2u(__byte_perm(eb[k], ob[k], 0x5410), x1[k]);
            const uint32_t a3 = hmul2u(__byte_perm(eb[k], ob[k], 0x7632), x1[k]);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                mma16816(a.o[n][4 * q + k], a0, a1, a2, a3, pb[n][0], pb[n][1]);
                if constexpr (FINE) mma16816(a.o[n][4 * q + k], a0, a1, a2, a3, pl[n][0], pl[n][1]);
            }
        }
    }
}

template <int DT, int NT, int W, int MINB>
__global__ void __launch_bounds__(32 * W, MINB) kv4_attention_kernel(AttnParams p) {
    typedef typename Elem<DT>::T T;
    typedef AttnShared<NT, W> Shared;
    constexpr int NC = 8 * NT, S = ATTN_STAGES;
    constexpr bool FINE = DT == HQ_DT_F16;  // weights in two parts
    extern __shared__ __align__(128) uint8_t raw[];
    Shared& sh = *reinterpret_cast<Shared*>(raw);
    uint64_t* const pre = reinterpret_cast<uint64_t*>(raw + sizeof(Shared));
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, g = lane >> 2, i4 = lane & 3;

    if (lane < S) mbar_init(&sh.full[w][lane], 1);
    // ---- units before each request: units of one group while there are few
    // (latency counts), of two otherwise (fewer turns of the loops)
    // (both are summed at once; the second pass is only for more requests than threads)
    Sched sc;
    int us = 0;
    for (bool again = true; again;) {
        unsigned long long carry[2] = {0, 0}, mine[2] = {0, 0};
        for (int b0 = 0; b0 < p.B; b0 += 32 * W) {
            const int b = b0 + tid;
            unsigned long long v[2] = {0, 0}, s[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                if (b < p.B) {
                    const Request r = attn_request(p, b, NC, k);
                    v[k] = (unsigned long long)r.tiles * p.Hkv * r.n;
                }
                s[k] = v[k];
            }
#pragma unroll
            for (int o = 1; o < 32; o <<= 1)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const unsigned long long u = __shfl_up_sync(0xFFFFFFFFu, s[k], o);
                    if (lane >= o) s[k] += u;
                }
            if (lane == 31) sh.warp_sums[w] = make_ulonglong2(s[0], s[1]);
            __syncthreads();
            mine[0] = carry[0] + s[0] - v[0];
            mine[1] = carry[1] + s[1] - v[1];
#pragma unroll
            for (int k = 0; k < W; ++k) {
                const ulonglong2 t = sh.warp_sums[k];
                if (k < w) {
                    mine[0] += t.x;
                    mine[1] += t.y;
                }
                carry[0] += t.x;
                carry[1] += t.y;
            }
            if (b < p.B) pre[b] = us ? mine[1] : mine[0];
            __syncthreads();
        }
        sc.U = us ? carry[1] : carry[0];
        again = false;
        if (us == 0 && sc.U > 2ull * W * gridDim.x) {
            us = 1;
            sc.U = carry[1];
            again = p.B > 32 * W;
            if (!again && tid < p.B) pre[tid] = mine[1];
        }
    }
    if (tid == 0) pre[p.B] = sc.U;
    fence_mbar_init();
    __syncthreads();
    if (blockIdx.x == 0)
        for (int b = tid; b < p.B; b += 32 * W) {
            if (p.cu_q && (p.cu_q[b] < 0 || p.cu_q[b + 1] > p.Tq || (int64_t)p.cu_q[b + 1] - p.cu_q[b] > p.q_len))
                p.ws[2] = HQ_ERR_SHAPE;
            const Request r = attn_request(p, b, NC, 0);
            if (r.bad && r.nq) p.ws[2] = HQ_ERR_PAGE;
        }
    if (sc.U == 0) return;
    {  // at least one unit per warp of a CTA
        const uint64_t most = (sc.U + W - 1) / W;
        sc.G = most < gridDim.x ? (uint32_t)most : gridDim.x;
    }
    if (blockIdx.x >= sc.G) return;

    // ---- the warp's loads run ahead of its arithmetic, across pieces.  (The
    // pieces' records live in shared memory: they are read once per unit, and in
    // registers they would push the accumulators out.)
    Walk& cw = sh.cw;
    Walk& lw = sh.lw[w];
    {
        // (lanes 0 and 1 find the two ends side by side)
        Walk t;
        walk_cut(p, pre, NC, us, sc, blockIdx.x + (lane & 1), t);
        walk_start(t, __shfl_sync(0xFFFFFFFFu, t.at, 1));  // (lane 0's is the CTA's)
        if (tid == 0) cw = t;
        if (lane == 0) lw = t;
    }
    __syncthreads();
    if (!cw.live) return;  // (a CTA whose units all lie in front of a row)
    // column c of a piece's q, four elements a lane
    constexpr int CPW = (NC + W - 1) / W;  // columns per warp
    uint2 qraw[CPW];
    auto load_q = [&](const Walk& k) {
#pragma unroll
        for (int x = 0; x < CPW; ++x) {
            qraw[x] = make_uint2(0u, 0u);
            const int c = w + x * W, col = (k.row - k.head * k.r.tiles) * NC + c;
            if (c < NC && col < k.r.nq * p.group) {
                const int j = col / p.group, hh = col - j * p.group;
                const T* q = static_cast<const T*>(p.q) + (int64_t)(k.r.q0 + j) * p.q_ts + (int64_t)(k.head * p.group + hh) * p.q_hs;
                qraw[x] = *reinterpret_cast<const uint2*>(q + 4 * lane);
            }
        }
    };
    load_q(cw);
    const int groups_shift = p.page_shift - 4;
    const bool small_pages = groups_shift == 0;  // a unit's two groups lie on two pages
    auto own = [](const Walk& k) { return max(k.ja, ATTN_ROW_COST); };
    auto unit_of = [](const Walk& k, int j) {
        const int t = j - ATTN_ROW_COST;
        return t < k.r.sink_units ? t : k.r.first_unit + (t - k.r.sink_units);
    };
    // Up to 32 of the warp's next units in a piece are looked up at once, one by
    // each lane, which keeps where its unit lies and starts its copy when its
    // turn comes; masks tell all lanes which of them have their groups.
    int lj = own(lw) + w;      // the batch's first unit in lw's piece
    int turn = 32;             // lane whose unit is loaded next; 32: a new batch
    int count = 0;             // units of the batch
    uint32_t has0 = 0, has1 = 0;
    uint32_t src = 0, src1 = 0;  // the lane's unit: its two groups' numbers in the cache
    uint32_t stage_ok = 0;     // bits 2 s, 2 s + 1: stage s holds its groups
    auto batch = [&]() {
        has0 = has1 = 0;
        turn = 0;
        count = 0;
        if (!lw.live) return;
        if (lj >= lw.jb) {  // on to the next piece with a unit for this warp
            Walk t = lw;
            while (t.live && lj >= t.jb) {
                walk_next(p, pre, NC, us, t);
                lj = own(t) + w;
            }
            __syncwarp();
            if (lane == 0) lw = t;
            __syncwarp();
            if (!lw.live) return;
        }
        count = min(32, (lw.jb - lj + W - 1) / W);
        const int len = lw.r.len, g0 = unit_of(lw, lj + lane * W) << us;  // first group
        const bool in0 = lane < count && 16 * g0 < len, in1 = us && lane < count && 16 * g0 + 16 < len;
        const int32_t* const row = p.table + (int64_t)lw.b * p.width;
        const int pg0 = in0 ? row[g0 >> groups_shift] : -1;
        const int pg1 = in1 ? (small_pages ? row[g0 + 1] : pg0) : -1;
        const bool ok0 = (uint32_t)pg0 < (uint64_t)p.num_pages, ok1 = (uint32_t)pg1 < (uint64_t)p.num_pages;  // (not -1)
        if (in0 != ok0 || in1 != ok1) p.ws[2] = HQ_ERR_PAGE;
        const uint32_t page_groups = (uint32_t)p.Hkv << groups_shift, head = (uint32_t)lw.head << groups_shift;
        src = (uint32_t)pg0 * page_groups + head + ((uint32_t)g0 & ((1u << groups_shift) - 1));
        src1 = (uint32_t)pg1 * page_groups + head;  // (read with pages of one group only)
        has0 = __ballot_sync(0xFFFFFFFFu, ok0);
        has1 = __ballot_sync(0xFFFFFFFFu, ok1);
        lj += W * count;
    };
    // load the next unit into stage st
    auto issue = [&](int st) {
        if (turn >= count) batch();
        const uint32_t ok = (has0 >> turn & 1u) | (has1 >> turn & 1u) << 1;
        stage_ok = (stage_ok & ~(3u << (2 * st))) | ok << (2 * st);
        if (lane == turn && ok) {
            const uint32_t dst = smem_u32(sh.ring[w][st]);
            mbar_arrive_expect(&sh.full[w][st], ok == 3 ? 2 * KV_GROUP_BYTES : KV_GROUP_BYTES);
            const uint8_t* const a = p.cache + (uint64_t)src * KV_GROUP_BYTES;
            if (!small_pages) {
                bulk_load(dst, a, ok == 3 ? 2 * KV_GROUP_BYTES : KV_GROUP_BYTES, &sh.full[w][st]);
            } else {
                if (ok & 1) bulk_load(dst, a, KV_GROUP_BYTES, &sh.full[w][st]);
                if (ok & 2)
                    bulk_load(dst + KV_GROUP_BYTES, p.cache + (uint64_t)src1 * KV_GROUP_BYTES, KV_GROUP_BYTES, &sh.full[w][st]);
            }
        }
        ++turn;
    };
#pragma unroll 1
    for (int s = 0; s < S; ++s) issue(s);
    int st = 0;
    uint32_t phases = 0;  // bit s: parity of stage s's next completion

    while (cw.live) {
        const int head = cw.head, col0 = (cw.row - head * cw.r.tiles) * NC, cols = cw.r.nq * p.group;
        const int tile_cols = min(NC, cols - col0);
        // ---- q: rotate, split into two FP16 parts, relative to the column's largest power of two
#pragma unroll
        for (int x = 0; x < CPW; ++x) {
            const int c = w + x * W;
            if (c >= NC) break;
            float y[4];
            const T* h = reinterpret_cast<const T*>(&qraw[x]);
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = to_f32(h[e]);
            if (p.rotate) rotate_warp(y, lane);
            float a = max3(fmaxf(fabsf(y[0]), fabsf(y[1])), fabsf(y[2]), fabsf(y[3]));
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
            // 2^e in (a / 2, a] (at most 2^126, whose inverse is normal); a column below 2^-111 keeps its values
            const uint32_t ebits = min(__float_as_uint(a) & 0x7F800000u, 0x7E800000u);
            const bool plain = ebits < 0x08000000u;
            const float up = plain ? 1.0f : __uint_as_float(ebits), down = plain ? 1.0f : __uint_as_float(0x7F000000u - ebits);
            float hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float v = __fmul_rn(y[e], down);
                hi[e] = __half2float(__float2half_rn(v));
                lo[e] = __fsub_rn(v, hi[e]);
            }
            // elements 4 lane .. + 3: block lane / 4, quad lane % 4 of column c
            sh.q[c >> 3][lane >> 2][(c & 7) * 4 + (lane & 3)] =
                make_uint4(pack_h2(hi[0], hi[1]), pack_h2(hi[2], hi[3]), pack_h2(lo[0], lo[1]), pack_h2(lo[2], lo[3]));
            if (lane == 0) {
                sh.qs[c] = up * p.scale * 1.4426950408889634f;
                sh.pos[c] = cw.r.last - (cw.r.nq - 1 - min(col0 + c, cols - 1) / p.group);
            }
        }
        __syncthreads();
        if (tid == 32 * (W - 1)) {  // the next piece (read after the loop; the last warp has the fewest units)
            Walk t = cw;
            walk_next(p, pre, NC, us, t);
            sh.nw = t;
        }
        AttnState<NT> a;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int c = 8 * n + 2 * i4 + k;
                a.qs[n][k] = sh.qs[c];
                a.m[n][k] = ATTN_NONE;
                a.l[n][k] = 0.0f;
                a.cz[n][k] = ATTN_CZ_MOST;
            }
#pragma unroll
            for (int b = 0; b < 8; ++b)
#pragma unroll
                for (int e = 0; e < 4; ++e) a.o[n][b][e] = 0.0f;
        }

        for (int j = own(cw) + w; j < cw.jb; j += W) {
            const int cur = st;
            st = st + 1 == S ? 0 : st + 1;
            const uint32_t ok = stage_ok >> (2 * cur) & 3u;
            if (ok) {  // (no page: the tokens count as not seen)
                // a copy ends by itself; the limit (about 2 s) only keeps the wait from being endless
                if (!mbar_wait_bounded(&sh.full[w][cur], phases >> cur & 1u, 2000000u)) p.ws[2] = HQ_ERR_TIMEOUT;
                phases ^= 1u << cur;
                const uint8_t* const unit = sh.ring[w][cur];
                const int t0 = unit_of(cw, j) << (4 + us);
                // (read again for every unit: as loop constants they cost the accumulators their registers)
                const int pos_min = *const_cast<volatile int*>(&sh.pos[0]), pos_max = *const_cast<volatile int*>(&sh.pos[NC - 1]);
                if (ok == 3u && t0 + 31 <= pos_min && (p.window == 0 || pos_max - t0 < p.window || t0 + 31 < p.sinks)) {
                    // every column sees every token
                    float s[2][NT][4], v[2][2];
                    attn_scores2<NT>(unit, sh.q, a, lane, s);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint8_t* grp = unit + h * KV_GROUP_BYTES;
                        v[h][0] = *reinterpret_cast<const float*>(grp + KV_V_DEC + 4 * g);
                        v[h][1] = *reinterpret_cast<const float*>(grp + KV_V_DEC + 4 * g + 32);
                    }
                    uint32_t u[2][NT][2], lo[2][NT][2];
                    attn_weigh<NT, 2, FINE>(a, s, v, unit, lane, u, lo);
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        attn_values<NT, false, FINE>(unit + h * KV_GROUP_BYTES, a, u[h], lo[h], 0u, 0u, lane);
                } else if (t0 <= pos_max && !(p.window > 0 && t0 + 31 <= pos_min - p.window && t0 >= p.sinks)) {
                    // some do (in a chunk of a prefill, a unit may be ahead of all of these columns, or behind their window)
#pragma unroll 1
                    for (int h = 0; h < 2; ++h) {
                        if (!(ok >> h & 1u)) continue;
                        const uint8_t* grp = unit + h * KV_GROUP_BYTES;
                        float s[1][NT][4], v[1][2];
                        attn_scores<NT>(grp, sh.q, a, lane, s[0]);
                        const int t1 = t0 + 16 * h, ta = t1 + g, tb = ta + 8;
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const int q = sh.pos[8 * n + 2 * i4 + k];
                                if (!(ta <= q && (p.window == 0 || q - ta < p.window || ta < p.sinks))) s[0][n][k] = -INFINITY;
                                if (!(tb <= q && (p.window == 0 || q - tb < p.window || tb < p.sinks))) s[0][n][2 + k] = -INFINITY;
                            }
                        // tokens behind the last query's position may hold anything: their value scales count as zero
                        v[0][0] = ta > pos_max ? 0.0f : *reinterpret_cast<const float*>(grp + KV_V_DEC + 4 * g);
                        v[0][1] = tb > pos_max ? 0.0f : *reinterpret_cast<const float*>(grp + KV_V_DEC + 4 * g + 32);
                        const int e = pos_max - t1 - 2 * i4;  // the lane's even token is real if e >= 0, the odd one if e >= 1
                        const uint32_t keep0 = (e >= 0 ? 0x00FF00FFu : 0u) | (e >= 1 ? 0xFF00FF00u : 0u);
                        const uint32_t keep1 = (e >= 8 ? 0x00FF00FFu : 0u) | (e >= 9 ? 0xFF00FF00u : 0u);
                        uint32_t u[1][NT][2], lo[1][NT][2];
                        attn_weigh<NT, 1, FINE>(a, s, v, grp, lane, u, lo);
                        attn_values<NT, true, FINE>(grp, a, u[0], lo[0], keep0, keep1, lane);
                    }
                }
            }
            __syncwarp();  // every lane has read the unit before its stage is filled again
            issue(cur);
        }

        // ---- join the warps: common references, then the upper half's accumulators into the lower half's
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float t = a.l[n][k];
#pragma unroll
                for (int x = 4; x <= 16; x <<= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, x);
                if (g == 0) {
                    sh.mz[w][8 * n + 2 * i4 + k] = make_float2(a.m[n][k], (float)-pow2_of(a.cz[n][k]));
                    sh.l[w][8 * n + 2 * i4 + k] = t;
                }
            }
        __syncthreads();
        if (sh.nw.live) load_q(sh.nw);
        // a warp's accumulators are relative to 2^(m + z); in common: the largest of these
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int c = 8 * n + 2 * i4 + k;
                float M = ATTN_NONE, Z = ATTN_NONE;
#pragma unroll
                for (int x = 0; x < W; ++x) M = fmaxf(M, sh.mz[x][c].x);
#pragma unroll
                for (int x = 0; x < W; ++x) Z = fmaxf(Z, sh.mz[x][c].y + (sh.mz[x][c].x - M));
                const float f = ex2((float)-pow2_of(a.cz[n][k]) + (a.m[n][k] - M) - Z);
#pragma unroll
                for (int b = 0; b < 8; ++b) {
                    a.o[n][b][k] *= f;
                    a.o[n][b][2 + k] *= f;
                }
            }
            if (w >= W / 2) {
#pragma unroll
                for (int b = 0; b < 8; ++b)
                    sh.frag[w - W / 2][8 * n + b][lane] = make_float4(a.o[n][b][0], a.o[n][b][1], a.o[n][b][2], a.o[n][b][3]);
            }
        }
        __syncthreads();
        if (w < W / 2) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int b = 0; b < 8; ++b) {
                    const float4 v = sh.frag[w][8 * n + b][lane];
                    a.o[n][b][0] += v.x;
                    a.o[n][b][1] += v.y;
                    a.o[n][b][2] += v.z;
                    a.o[n][b][3] += v.w;
                }
        }
        __syncthreads();
        if (w < W / 2) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int b = 0; b < 8; ++b)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        *reinterpret_cast<float2*>(&sh.o[w][8 * n + 2 * i4 + k][16 * b + 2 * g]) =
                            make_float2(a.o[n][b][k], a.o[n][b][2 + k]);
        }
        __syncthreads();
        const bool complete = cw.ja == 0 && cw.jb == cw.r.n;
        const uint64_t u0 = pre[cw.b] + (uint64_t)cw.row * cw.r.n;  // the row's first unit
        float* const parts = reinterpret_cast<float*>(p.ws + 64 + ATTN_MAX_CTAS);
        auto store = [&](int c, float (&y)[4], float mx, float L, float Z) {  // Z: -126 .. 126
            const float inv = L > 0.0f ? __fdiv_rn(1.0f, L) : 0.0f, scale = ex2(Z);
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = y[e] * inv * scale;
            if (p.rotate) rotate_warp(y, lane);
            const int j = (col0 + c) / p.group, hq_ = head * p.group + (col0 + c) - j * p.group;
            const int64_t row = cw.r.q0 + j;
            T* out = static_cast<T*>(p.out) + row * p.o_ts + (int64_t)hq_ * p.o_hs;
            const T h[4] = {from_f32<DT>(y[0]), from_f32<DT>(y[1]), from_f32<DT>(y[2]), from_f32<DT>(y[3])};
            *reinterpret_cast<uint2*>(out + 4 * lane) = *reinterpret_cast<const uint2*>(h);
            if (p.lse && lane == 0)
                p.lse[row * ((int64_t)p.Hkv * p.group) + hq_] = L != 0.0f ? (mx + log2f(L)) * 0.6931471805599453f : -INFINITY;  // (NaN stays)
        };
        // partial results: CTA c's slot 0 for a row that began before it, slot 1 for one that goes on after it
        float* const mine = parts + (size_t)(2 * blockIdx.x + (cw.ja == 0 ? 1 : 0)) * ATTN_PART;
        for (int c = w; c < tile_cols; c += W) {
            float mx = ATTN_NONE, Z = ATTN_NONE, L = 0.0f, y[4] = {};
#pragma unroll
            for (int k = 0; k < W; ++k) mx = fmaxf(mx, sh.mz[k][c].x);
#pragma unroll
            for (int k = 0; k < W; ++k) {
                const float2 v = sh.mz[k][c];
                const float d = v.x - mx;
                L += ex2(d) * sh.l[k][c];
                Z = fmaxf(Z, v.y + d);
            }
#pragma unroll
            for (int k = 0; k < W / 2; ++k) {
                const float4 v = *reinterpret_cast<const float4*>(&sh.o[k][c][4 * lane]);
                y[0] += v.x;
                y[1] += v.y;
                y[2] += v.z;
                y[3] += v.w;
            }
            if (complete) {
                store(c, y, mx, L, Z);
            } else {
                __stcg(reinterpret_cast<float4*>(mine + c * 128 + 4 * lane), make_float4(y[0], y[1], y[2], y[3]));
                if (lane == 0) __stcg(reinterpret_cast<float4*>(mine + ATTN_MAX_NC * 128 + 4 * c), make_float4(mx, L, Z, 0.0f));
            }
        }
        if (!complete) {
            // the CTA that arrives last joins the row's partial results, in the order of its CTAs
            const uint32_t first = cta_of(sc, u0 + ATTN_ROW_COST), last = cta_of(sc, u0 + cw.r.n - 1);
            // (one thread releases what all wrote before the barrier, and acquires for all after the next one)
            __syncthreads();
            if (tid == 0) {
                const uint32_t seen = arrive(p.ws + 64 + first);
                sh.last = seen == last - first;
                if (sh.last) p.ws[64 + first] = 0;  // rest state
            }
            __syncthreads();
            if (sh.last) {
                float mx[CPW], L[CPW], Z[CPW], y[CPW][4];
#pragma unroll
                for (int x = 0; x < CPW; ++x) {
                    mx[x] = Z[x] = ATTN_NONE;
                    L[x] = y[x][0] = y[x][1] = y[x][2] = y[x][3] = 0.0f;
                }
                for (uint32_t k0 = first; k0 <= last; k0 += 4) {  // four results of the warp's columns on their way at a time
                    float4 ml[CPW][4];
                    float4 v[CPW][4];
#pragma unroll
                    for (int x = 0; x < CPW; ++x)
#pragma unroll
                        for (int z = 0; z < 4; ++z) {
                            const uint32_t k = k0 + z;
                            const int c = w + x * W;
                            const float* part = parts + (size_t)(2 * k + (k == first ? 1 : 0)) * ATTN_PART;
                            ml[x][z] = make_float4(ATTN_NONE, 0.0f, ATTN_NONE, 0.0f);
                            v[x][z] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                            if (k <= last && c < tile_cols) {
                                ml[x][z] = __ldcg(reinterpret_cast<const float4*>(part + ATTN_MAX_NC * 128 + 4 * c));
                                v[x][z] = __ldcg(reinterpret_cast<const float4*>(part + c * 128 + 4 * lane));
                            }
                        }
#pragma unroll
                    for (int x = 0; x < CPW; ++x) {
                        float t = mx[x];
#pragma unroll
                        for (int z = 0; z < 4; ++z) t = fmaxf(t, ml[x][z].x);
                        const float za = Z[x] + (mx[x] - t);
                        float zt = za;
#pragma unroll
                        for (int z = 0; z < 4; ++z) zt = fmaxf(zt, ml[x][z].z + (ml[x][z].x - t));
                        const float fa = ex2(za - zt);
                        L[x] *= ex2(mx[x] - t);
#pragma unroll
                        for (int e = 0; e < 4; ++e) y[x][e] *= fa;
#pragma unroll
                        for (int z = 0; z < 4; ++z) {
                            const float d = ml[x][z].x - t, fb = ex2(ml[x][z].z + d - zt);
                            L[x] += ml[x][z].y * ex2(d);
                            y[x][0] += v[x][z].x * fb;
                            y[x][1] += v[x][z].y * fb;
                            y[x][2] += v[x][z].z * fb;
                            y[x][3] += v[x][z].w * fb;
                        }
                        mx[x] = t;
                        Z[x] = zt;
                    }
                }
#pragma unroll
                for (int x = 0; x < CPW; ++x)
                    if (w + x * W < tile_cols) store(w + x * W, y[x], mx[x], L[x], Z[x]);
            }
        }
        __syncthreads();  // the merge buffer, q and the piece's record are free again
        if (tid == 0) cw = sh.nw;
        __syncthreads();
    }
}

// ------------------------------------------------------------------ launch
// Words: [0..3] as the grouped call's workspace (only [2], the error word, is
// used), [64 ..] arrivals per CTA, then two partial results per CTA.
static_assert(4 * (64 + ATTN_MAX_CTAS) == HQ_KV4_ATTENTION_STATE_BYTES, "the words that are zero at rest");
size_t attn_workspace_bytes() { return 4 * (64 + (size_t)ATTN_MAX_CTAS + 2 * (size_t)ATTN_MAX_CTAS * ATTN_PART); }

template <int DT, int NT, int W, int MINB> static int launch_t(const AttnParams& p, int sms, cudaStream_t st) {
    auto kernel = kv4_attention_kernel<DT, NT, W, MINB>;
    constexpr size_t base = sizeof(AttnShared<NT, W>);
    const int e = allow_shared(kernel, base + 8 * (HQ_KV_MAX_REQUESTS + 1));
    if (e != (int)cudaSuccess) return e;
    const int grid = sms * MINB < ATTN_MAX_CTAS ? sms * MINB : ATTN_MAX_CTAS;
    kernel<<<grid, 32 * W, base + 8 * ((size_t)p.B + 1), st>>>(p);
    return (int)cudaPeekAtLastError();
}

int launch_attn(int dtype, const AttnParams& p, int sms, cudaStream_t st) {
    // Two column tiles of 8 in one pass cost about 1.7 times one (64 requests of
    // 12000 tokens, 4 key/value heads: 165 us against 211 one by one; a prefill's
    // chunks of up to 128 tokens 149 against 187; a batch of 4 short requests 16
    // against 12), so they are paired when their number is even.  (Up to 20
    // columns, three tiles, of 48 verifying requests: 44 us paired, half a pass
    // empty, against 38.)  Six warps a block, as one of eight with 255 registers
    // or two blocks of four take 172 and 167 us there.  (As measured when chosen;
    // 163 us there now.  168 registers spill about 200 bytes a thread.)
    const bool wide = ((int64_t)p.q_len * p.group + 7) / 8 % 2 == 0;
    if (dtype == HQ_DT_BF16)
        return wide ? launch_t<HQ_DT_BF16, 2, 6, 2>(p, sms, st) : launch_t<HQ_DT_BF16, 1, 8, 2>(p, sms, st);
    return wide ? launch_t<HQ_DT_F16, 2, 6, 2>(p, sms, st) : launch_t<HQ_DT_F16, 1, 8, 2>(p, sms, st);
}

}  // namespace hq
