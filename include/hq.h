/*
 * hq.h -- C ABI of the hq library: Hadamard rotation fused with block-scaled
 * low-precision quantization (NVFP4 and FP8 E4M3) on NVIDIA B200 (sm_100a).
 *
 * Conventions for every call below:
 *  - Pointers are CUDA device pointers owned by the caller, unless a comment
 *    says "host".  The library allocates no memory, never synchronizes the
 *    stream (hq_get_error excepted) and reads no environment variables.
 *  - `stream` is a cudaStream_t passed as void* (NULL = legacy default).
 *  - Every argument is checked before anything is launched; a violation
 *    returns a nonzero hq_status and leaves all outputs untouched.  There is no
 *    fallback path: an unsupported request is an error.
 *  - Calls are asynchronous: a status of HQ_OK means the work was enqueued.
 *  - BF16 tensors are passed as their 16-bit patterns, FP8 E4M3 codes as
 *    bytes, NVFP4 E2M1 codes two per byte (element 2k in the low nibble).
 *
 * Sources for the operations (page titles):
 *  [GRP] TransformerEngine PR #2564 "[NVFP4][MOE] Bug Fix for NVFP4 Grouped
 *        Quant": the grouped row-cast / column-Hadamard-transform-cast kernel
 *        over MoE split sections, and its caller-provided 4-byte tile
 *        scheduler workspace (replacing a per-call cudaMallocAsync), plus the
 *        reviewers' request for a workspace-size query.
 *  [FUS] TransformerEngine PR #2555 review comments: split_section % 128
 *        fusion rule, rht_matrix, rowwise-only output needs no RHT, the RHT'd
 *        columnwise output is the transposed [cols, rows] tensor.
 *  [DSA] TensorRT-LLM PR #15158 "[#13061][bugfix] Add rotate_activation to DSA
 *        fused_cat_fp8 path": cat([pe, nope]) -> Hadamard rotation ->
 *        fp8_quantize_1x128, scales transposed.
 *  [QMOE] onnxruntime PR #33644 (QMoE activation_quantization="dynamic_fp8"),
 *        Description: K128 groups, saturating nearest-even E4M3,
 *        max(amax, 1e-10) * float32(1/448) scales, FP32 SiLU/SwiGLU before
 *        the second quantizer, explicit errors instead of fallbacks.
 */
#ifndef HQ_H
#define HQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum hq_status {
    HQ_OK = 0,
    HQ_ERR_NULL = 1,        /* a required pointer is NULL */
    HQ_ERR_SHAPE = 2,       /* sizes negative, inconsistent or too large */
    HQ_ERR_ALIGN = 3,       /* pointer/stride not 16-byte aligned, or a size
                               not a multiple of the required block */
    HQ_ERR_WORKSPACE = 4,   /* workspace missing or smaller than the query */
    HQ_ERR_UNSUPPORTED = 5, /* unknown flag, mode, layout or transform size */
    HQ_ERR_CUDA = 6,        /* the CUDA runtime reported an error */
    HQ_ERR_TIMEOUT = 7,     /* a bounded device-side wait gave up */
    HQ_ERR_PAGE = 8         /* a block table or a length points outside the cache
                               (device error word of hq_kv4_attention) */
} hq_status;

/* hq_group_rht_quant flags */
#define HQ_ROWWISE 1u      /* rowwise NVFP4 output (plain cast along K) */
#define HQ_COLWISE 2u      /* columnwise NVFP4 output (RHT16 along M, transposed) */
#define HQ_ROW_RHT 4u      /* with HQ_ROWWISE: the rowwise output casts the RHT16
                              of each 16-column block along K instead of x */
#define HQ_ROW_SR 32u      /* hq_group_rht_quant_sr: rowwise codes round stochastically */
#define HQ_COL_SR 64u      /* hq_group_rht_quant_sr: columnwise codes round stochastically */
#define HQ_AMAX_GIVEN 16u  /* amax_row / amax_col are inputs: the caller's section
                              amax values; one pass, no amax computation */
#define HQ_SF_SWIZZLED 128u /* row_sf and each section's col_sf block in the
                              interleaved 128 x 4 tiles that block-scaled
                              tcgen05 MMAs read (see below) */
#define HQ_TWO_PASS 8u     /* schedule: amax pass and cast pass as two launches
                              (without HQ_ROW_RHT the amax pass is a streaming
                              kernel of its own) instead of one launch in which
                              each section's cast follows its amax while the
                              rows are still in L2.  A call whose only
                              non-empty section fills the grid at least once,
                              without HQ_ROW_RHT, takes two launches without
                              the flag too (its casts wait for the whole amax
                              pass either way).  Results are identical. */

/* hq_cat_rotate_fp8 scale layouts */
#define HQ_SCALE_ROWMAJOR 0   /* scale of group (t, g) at scales[t * G + g] */
#define HQ_SCALE_TRANSPOSED 1 /* scale of group (t, g) at scales[g * scale_ld + t] */

/*
 * Scale formats for GEMMs that consume the outputs directly (the TensorRT-LLM
 * PR #15158 review asks for a use_ue8m0 option of the 1x128 quantizer;
 * DeepGEMM issue #320 discusses the tcgen05 data-path layouts of scales).
 *
 * HQ_FP8_UE8M0, added to scale_layout of hq_cat_rotate_fp8 or to mode of
 * hq_swiglu_fp8_k128: each group's FP32 scale s is rounded up to the smallest
 * power of two not below it, and the codes are E4M3(y / that power of two).
 * The stored scale is that FP32 power of two; its UE8M0 byte is the binary32
 * exponent field (bits 30..23).
 *
 * HQ_SF_SWIZZLED (hq_group_rht_quant* flags; added to scale_layout of
 * hq_cat_rotate_nvfp4): E4M3 block scales in tiles of 128 rows x 4 columns
 * of the [rows, cols] scale matrix, 512 bytes each, stored tile-row major;
 * element (r, c) at byte
 *   ((r / 128) * (cols / 4) + c / 4) * 512 + (r % 32) * 16 + ((r % 128) / 32) * 4 + c % 4.
 * The grouped cast's row_sf is [M, K/16]; each section's col_sf block is
 * [K, M_s/16] at its usual byte K * r0 / 16 (every dimension a multiple of the
 * tile: a permutation of the plain layout, same size).  The FP4 DSA call's
 * block_sf is [M, G * 8] and needs M % 128 == 0 (HQ_ERR_ALIGN otherwise).
 */
#define HQ_FP8_UE8M0 256

/* hq_swiglu_fp8_k128 modes (+ HQ_FP8_UE8M0) */
#define HQ_ACT_NONE_BF16 0  /* in: BF16 [M, K_out] */
#define HQ_ACT_NONE_F32 1   /* in: FP32 [M, K_out] */
#define HQ_ACT_SWIGLU_F32 2 /* in: FP32 [M, 2*K_out], gate = cols [0, K_out),
                               up = cols [K_out, 2*K_out); value SiLU(gate)*up */

/* hq_convert formats */
#define HQ_FMT_E4M3 0 /* one E4M3 code per output byte */
#define HQ_FMT_E2M1 1 /* one E2M1 code per output byte (low nibble) */

#define HQ_MAX_SECTIONS 256

/* Library version, (major << 16) | minor. */
int hq_version(void);

/* Static description of a status code. */
const char *hq_status_string(hq_status s);

/*
 * Workspace bytes hq_group_rht_quant needs for `num_sections` sections
 * (1 <= num_sections <= HQ_MAX_SECTIONS; 0 otherwise).  The first 4 bytes
 * are the tile-scheduler counter of [GRP]; an exit count, an error word, an
 * abort flag, then per section an amax accumulator per direction and a count
 * of its completed amax tiles follow (16 + 12 * S bytes, rounded up to 256).
 * The size query is the reviewers' proposal in [GRP].
 */
size_t hq_group_rht_quant_workspace_size(int num_sections);

/*
 * Put a workspace into its rest state (all zero).  Call once after
 * allocating it (an enqueued memset on `stream`).  Every hq_group_rht_quant
 * call leaves the workspace in the rest state again, so no per-call memset
 * is needed.  Two calls that share one workspace must not overlap in time
 * (same stream, or ordered by events).
 * Errors: HQ_ERR_NULL, HQ_ERR_ALIGN (ws not 16-byte aligned), HQ_ERR_CUDA.
 */
hq_status hq_workspace_init(void *ws, size_t ws_bytes, void *stream);

/*
 * Read and clear the workspace's device error word.  Synchronizes `stream`.
 * *err_out (host) receives 0, or HQ_ERR_TIMEOUT if a bounded device wait of
 * an earlier call gave up (that call's outputs are then incomplete).
 */
hq_status hq_get_error(void *ws, size_t ws_bytes, uint32_t *err_out, void *stream);

/*
 * Grouped random-Hadamard-transform + NVFP4 cast over MoE split sections
 * [GRP], [FUS].
 *
 *  x          BF16 [M, K] row major.  16-byte aligned.
 *  M, K       rows, columns.  K > 0 and K % 128 == 0.
 *  split_rows HOST int64 [S]: rows per section, each >= 0 and a multiple of
 *             128 ([FUS] fusion rule), summing to M.  Empty sections allowed.
 *  S          number of sections, 1 <= S <= HQ_MAX_SECTIONS.
 *  sign_mask  the random sign vector of the 16-point RHT: bit i set means
 *             sigma_i = -1 for position i of each 16-row block (and, with
 *             HQ_ROW_RHT, of each 16-column block of a row).
 *  flags      HQ_ROWWISE | HQ_COLWISE (at least one), optionally HQ_ROW_RHT
 *             (only with HQ_ROWWISE; the grouped-quant pages speak of the RHT
 *             on both outputs, their fused kernel rotates only the columns),
 *             HQ_AMAX_GIVEN, HQ_TWO_PASS (ignored with HQ_AMAX_GIVEN) and
 *             HQ_SF_SWIZZLED.
 *
 * For section s (rows [r0, r0 + M_s)) and each requested direction:
 *   A_s = max |v| over the section's values (v = x rowwise, the RHT16 output
 *   along K with HQ_ROW_RHT; v = RHT16 output columnwise), or with
 *   HQ_AMAX_GIVEN the caller's amax_*[s]; S_enc = 2688 / A_s (1 when A_s is
 *   not positive or the quotient is not finite),
 *   sdec = 1 / S_enc; for each block of 16 values along the quantized
 *   direction: sf = E4M3((a_b / 6) * S_enc), code_i = E2M1(v_i * S_enc / sf)
 *   (0 when sf == 0); saturating round-to-nearest-even conversions.
 *   RHT16 of a block: v = 0.25 * H16 * diag(sigma) * x, H16 the Sylvester
 *   Hadamard matrix.
 *
 * Outputs (device; each 16-byte aligned; amax/sdec 4-byte aligned):
 *  row_codes  uint8 [M, K/2]     rowwise E2M1 codes          (HQ_ROWWISE)
 *  row_sf     uint8 [M, K/16]    rowwise E4M3 block scales   (HQ_ROWWISE)
 *  col_codes  uint8 [M*K/2]      per section s: [K, M_s/2] at byte K*r0/2
 *  col_sf     uint8 [M*K/16]     per section s: [K, M_s/16] at byte K*r0/16
 *  amax_row, sdec_row  float [S] (HQ_ROWWISE)
 *  amax_col, sdec_col  float [S] (HQ_COLWISE)
 *  With HQ_AMAX_GIVEN amax_row / amax_col are inputs (device, read only, set
 *  before the call in stream order) and only sdec_* is written; the call then
 *  reads x once (the cast pass alone).
 *  Pointers of a direction not requested may be NULL, and so may the code
 *  and block-scale buffers when M == 0.
 *
 *  ws, ws_bytes  caller workspace, >= hq_group_rht_quant_workspace_size(S),
 *                16-byte aligned, in the rest state (hq_workspace_init).
 * Errors: HQ_ERR_NULL, HQ_ERR_SHAPE, HQ_ERR_ALIGN, HQ_ERR_WORKSPACE,
 *         HQ_ERR_UNSUPPORTED, HQ_ERR_CUDA.
 * Inputs must be finite (NaN/inf are outside the NVFP4 contract).
 */
hq_status hq_group_rht_quant(const void *x, int64_t M, int64_t K,
                             const int64_t *split_rows, int S, uint16_t sign_mask,
                             unsigned flags,
                             uint8_t *row_codes, uint8_t *row_sf,
                             uint8_t *col_codes, uint8_t *col_sf,
                             float *amax_row, float *amax_col,
                             float *sdec_row, float *sdec_col,
                             void *ws, size_t ws_bytes, void *stream);

/*
 * hq_group_rht_quant with stochastic rounding of the E2M1 codes (the grouped
 * pages' review discusses the Philox generator and deterministic offsets of
 * stochastic rounding for this cast; it gives no rounding rule).  flags may
 * add HQ_ROW_SR (with HQ_ROWWISE) and HQ_COL_SR (with HQ_COLWISE); block
 * scales, amax and sdec are as without.  A code rounds |v| (v = value *
 * encode factor, as for nearest-even) up to the next E2M1 value iff its
 * random byte r < floor(256 f), f the fraction of |v| above the E2M1 value
 * below it in grid steps (0.5 below 2, 1 below 4, 2 below 6); |v| >= 6
 * saturates; the sign is kept.  r of output element e (its index in
 * row_codes' [M, K] order, or in col_codes' element order) is byte
 * offset + e of the stream of bytes B_i = byte (i % 4) of word (i / 4) % 4
 * of Philox4x32-10(counter = {i / 16 low 32 bits, i / 16 high 32 bits, 0, 0},
 * key = {k low, k high}), k = seed for rowwise codes and seed + 1 for
 * columnwise codes, so results depend only on (seed, offset), not on the
 * launch.  offset must be a multiple of 16 (HQ_ERR_ALIGN).  Other arguments,
 * outputs and errors as hq_group_rht_quant (which rejects the SR flags).
 */
hq_status hq_group_rht_quant_sr(const void *x, int64_t M, int64_t K,
                                const int64_t *split_rows, int S, uint16_t sign_mask,
                                unsigned flags, uint64_t seed, uint64_t offset,
                                uint8_t *row_codes, uint8_t *row_sf,
                                uint8_t *col_codes, uint8_t *col_sf,
                                float *amax_row, float *amax_col,
                                float *sdec_row, float *sdec_col,
                                void *ws, size_t ws_bytes, void *stream);

/*
 * The grouped cast with x and every output in HOST memory: the rows are
 * copied to the device, cast and copied back in groups of whole sections, so
 * the copies of one group overlap the cast of the next and the copies in the
 * other direction (page-locked host buffers are needed for the overlap;
 * pageable ones give the same results, copied without overlap).  The codes
 * and scales are those of hq_group_rht_quant_sr on the whole tensor (without
 * HQ_ROW_SR / HQ_COL_SR, those of hq_group_rht_quant); a section's amax never
 * crosses groups, and the random byte streams keep their element indices.
 *  x, row_codes, row_sf, col_codes, col_sf, amax_row, amax_col, sdec_row,
 *  sdec_col      host buffers with the layouts of hq_group_rht_quant; with
 *                HQ_AMAX_GIVEN amax_* are read (host) and copied in.
 *  seed, offset  as hq_group_rht_quant_sr (ignored without the SR flags).
 *  dev_buf, dev_buf_bytes  device staging memory, >=
 *                hq_group_rht_quant_host_device_bytes(M, K, S), 256-byte
 *                aligned; it holds x, the outputs and the workspace (kept in
 *                its rest state by the calls; zero it once before the first).
 *  groups        section groups (1..HQ_HOST_MAX_GROUPS); 0 picks 16.  Groups
 *                are cut at section boundaries only (a section's amax needs
 *                all its rows), so S sections give at most S groups and a
 *                single section is copied, cast and copied back in sequence.
 *  stream        the cast runs here; the call is ordered after the work
 *                already on it, and work enqueued on it afterwards runs after
 *                the last copy back (synchronize it before reading outputs).
 *  h2d_stream, d2h_stream  two further streams for the copies (distinct from
 *                stream and from each other).
 * A fixed set of CUDA events per device is created on the first call and
 * kept for the life of the process; calls from several host threads are
 * serialized while they enqueue.
 * Errors: as hq_group_rht_quant_sr, HQ_ERR_WORKSPACE when dev_buf is too
 *         small, HQ_ERR_UNSUPPORTED for a bad group count or stream set.
 *         Argument errors are found before anything is enqueued; a CUDA
 *         error after the first group was enqueued returns HQ_ERR_CUDA with
 *         the earlier groups' copies and casts still in flight.
 */
#define HQ_HOST_MAX_GROUPS 32
size_t hq_group_rht_quant_host_device_bytes(int64_t M, int64_t K, int S);
hq_status hq_group_rht_quant_host(const void *x, int64_t M, int64_t K,
                                  const int64_t *split_rows, int S, uint16_t sign_mask,
                                  unsigned flags, uint64_t seed, uint64_t offset,
                                  uint8_t *row_codes, uint8_t *row_sf,
                                  uint8_t *col_codes, uint8_t *col_sf,
                                  float *amax_row, float *amax_col,
                                  float *sdec_row, float *sdec_col,
                                  void *dev_buf, size_t dev_buf_bytes, int groups,
                                  void *stream, void *h2d_stream, void *d2h_stream);

/*
 * hq_group_rht_quant without a caller workspace, for callers that cannot
 * allocate device memory where they quantize (plugins whose host framework
 * owns all device memory, allocation-free runtimes).  The paper has no
 * counterpart.
 *
 * Arguments, outputs and errors are those of hq_group_rht_quant without
 * ws / ws_bytes.  The scratch words live in a fixed array inside the library
 * (3328 bytes, room for HQ_MAX_SECTIONS = 256 sections; S > 256 returns
 * HQ_ERR_SHAPE), present on every GPU that loads the library until the
 * process exits.  The call allocates nothing: it clears the array with an
 * enqueued memset and launches the kernel.  The first call on a device looks
 * up the array's device address (cudaGetSymbolAddress) and so should come
 * before any stream capture; a lookup that fails returns HQ_ERR_CUDA and is
 * tried again by the next call.  All calls on a device share the one array:
 * calls that overlap on the GPU (different streams without ordering) race
 * and give wrong results.  A bounded device wait that gives up is not
 * reported by this entry point (there is no workspace to read it from).
 */
hq_status hq_group_rht_quant_noalloc(const void *x, int64_t M, int64_t K,
                                     const int64_t *split_rows, int S, uint16_t sign_mask,
                                     unsigned flags,
                                     uint8_t *row_codes, uint8_t *row_sf,
                                     uint8_t *col_codes, uint8_t *col_sf,
                                     float *amax_row, float *amax_col,
                                     float *sdec_row, float *sdec_col, void *stream);

/*
 * Concatenate -> 128-point Hadamard rotation -> FP8 E4M3 1x128 quantization
 * [DSA] (the DSA indexer's q/k preparation), with the scale rule of [QMOE].
 *
 *  a          BF16; element j of group g of row t is
 *             a[t * a_row_stride + g * a_width + j], 0 <= j < a_width.
 *  b          BF16 or NULL (when b_width == 0); same indexing with b_*.
 *             The 128-vector of (t, g) is a-part followed by b-part
 *             ([pe, nope]); a_width + b_width == 128, both multiples of 8.
 *  M, G       rows (tokens) and groups (heads) per row.
 *  hadamard_n 128 (rotate by H128 / sqrt(128), Sylvester order) or 0 (none).
 *  out_fp8    uint8 [M, G*128] codes: (t, g, j) at (t * G + g) * 128 + j.
 *  scales     float: group scale s = max(amax, 1e-10) * float32(1/448),
 *             codes = E4M3(y / s) (IEEE division, saturating RNE).
 *             scale_layout HQ_SCALE_ROWMAJOR: [M, G] (scale_ld ignored);
 *             HQ_SCALE_TRANSPOSED: [G, scale_ld], scale_ld >= M; either may
 *             add HQ_FP8_UE8M0.
 *  amax_opt   float, NULL or each group's amax = max |y| (y the rotated
 *             128-vector), in the scales' layout; 4-byte aligned.
 *  ws, ws_bytes  unused: hq_cat_rotate_fp8_workspace_size() is 0 (may be
 *             NULL / 0).
 * Alignment: a, b, out 16 bytes; strides multiples of 8 elements.
 * Errors: HQ_ERR_NULL, HQ_ERR_SHAPE, HQ_ERR_ALIGN, HQ_ERR_UNSUPPORTED,
 *         HQ_ERR_CUDA.
 */
hq_status hq_cat_rotate_fp8(const void *a, int64_t a_row_stride, int a_width,
                            const void *b, int64_t b_row_stride, int b_width,
                            int64_t M, int G, int hadamard_n,
                            uint8_t *out_fp8, float *scales, int scale_layout,
                            int64_t scale_ld, float *amax_opt,
                            void *ws, size_t ws_bytes, void *stream);

/* Workspace bytes hq_cat_rotate_fp8 needs: 0 (none). */
size_t hq_cat_rotate_fp8_workspace_size(void);

/*
 * The DSA indexer prep with an NVFP4 output (the FP4 path [DSA] names as
 * lacking the rotation; the pages give no FP4 format, the reading is the
 * two-level NVFP4 scheme of hq_group_rht_quant with the 128-vector in place
 * of a section): concat and optional rotation exactly as hq_cat_rotate_fp8,
 * then for each vector (t, g) with rotated values y:
 *   A = max |y| over the vector, S_enc = 2688 / A (1 when A is 0 or the
 *   quotient is not finite); per block of 16 consecutive values
 *   sf = E4M3((a_b / 6) * S_enc), code_i = E2M1(y_i * S_enc / sf) (0 when
 *   sf == 0); saturating round-to-nearest-even conversions.
 *
 *  a, b, a_width, b_width, strides, M, G, hadamard_n, scale_layout,
 *  scale_ld   as hq_cat_rotate_fp8.
 *  codes      uint8 [M, G*64]: vector (t, g) at (t * G + g) * 64, two E2M1
 *             codes per byte, element 2k in the low nibble.  16-byte aligned.
 *  block_sf   uint8 [M, G*8] E4M3 block scales.
 *  sdec       float, per vector 1 / S_enc, in the FP8 scales' layouts
 *             ([M, G] or [G, scale_ld]).  4-byte aligned.
 *  amax_opt   float, NULL or A per vector, in the same layout.
 *  ws, ws_bytes  unused: hq_cat_rotate_nvfp4_workspace_size() is 0.
 * Errors: HQ_ERR_NULL, HQ_ERR_SHAPE, HQ_ERR_ALIGN, HQ_ERR_UNSUPPORTED,
 *         HQ_ERR_CUDA.  Inputs must be finite.  scale_layout may add
 *         HQ_SF_SWIZZLED (block_sf in the interleaved tiles, M % 128 == 0).
 */
hq_status hq_cat_rotate_nvfp4(const void *a, int64_t a_row_stride, int a_width,
                              const void *b, int64_t b_row_stride, int b_width,
                              int64_t M, int G, int hadamard_n,
                              uint8_t *codes, uint8_t *block_sf, float *sdec,
                              int scale_layout, int64_t scale_ld, float *amax_opt,
                              void *ws, size_t ws_bytes, void *stream);

/* Workspace bytes hq_cat_rotate_nvfp4 needs: 0 (none). */
size_t hq_cat_rotate_nvfp4_workspace_size(void);

/*
 * QMoE dynamic FP8 activation quantizer [QMOE]: each row of K_out values is
 * split into consecutive groups of 128; each group gets the FP8 rule above.
 *  mode     HQ_ACT_NONE_BF16, HQ_ACT_NONE_F32 or HQ_ACT_SWIGLU_F32 (the value
 *           quantized is SiLU(gate) * up computed in FP32, SiLU(g) =
 *           g / (1 + exp(-g)), with no narrower rounding in between); any
 *           mode may add HQ_FP8_UE8M0.
 *  in       see the modes; row stride K_out (or 2*K_out for SwiGLU).
 *  out_fp8  uint8 [M, K_out];  scales float [M, K_out/128] row major.
 *  amax_opt float [M, K_out/128] or NULL: each group's amax = max |y|.
 *  K_out    multiple of 128.   ws, ws_bytes unused:
 *           hq_swiglu_fp8_k128_workspace_size() is 0 (may be NULL / 0).
 * Alignment: in and out 16 bytes, scales and amax_opt 4 bytes.
 * Errors: HQ_ERR_NULL, HQ_ERR_SHAPE, HQ_ERR_ALIGN, HQ_ERR_UNSUPPORTED,
 *         HQ_ERR_CUDA.
 */
hq_status hq_swiglu_fp8_k128(int mode, const void *in, int64_t M, int64_t K_out,
                             uint8_t *out_fp8, float *scales, float *amax_opt,
                             void *ws, size_t ws_bytes, void *stream);

/* Workspace bytes hq_swiglu_fp8_k128 needs: 0 (none). */
size_t hq_swiglu_fp8_k128_workspace_size(void);

/*
 * Element-wise conversion of FP32 values with the library's own device
 * conversion routines (the ones every kernel above uses): E4M3 (saturating,
 * nearest even) or E2M1 (one nibble per byte).  n >= 0; in and out may have
 * any alignment.
 * Errors: HQ_ERR_NULL, HQ_ERR_SHAPE, HQ_ERR_UNSUPPORTED, HQ_ERR_CUDA.
 */
hq_status hq_convert(int fmt, const float *in, uint8_t *out, int64_t n, void *stream);

/*
 * Element-wise stochastic E2M1 conversion with the device routine of
 * hq_group_rht_quant_sr: out[i] (low nibble) is the code of in[i] rounded
 * with random byte rnd[i] by that call's rule (|v| up to the next E2M1 value
 * iff rnd[i] < floor(256 f); |v| >= 6 saturates; sign kept).  n >= 0; any
 * alignment.  Errors: HQ_ERR_NULL, HQ_ERR_SHAPE, HQ_ERR_CUDA.
 */
hq_status hq_convert_e2m1_sr(const float *in, const uint8_t *rnd, uint8_t *out, int64_t n, void *stream);

/* ======================================================================
 * The attention layer around the quantizers: residual + RMS norm with FP8
 * codes, rotary positions, slot maps, the NVFP4 key/value cache and
 * attention over it.
 *
 * Common rules of these calls: element types are HQ_DT_*; strides are in
 * elements; rows (the last dimension) are contiguous; tensors of one call are
 * on the current device.  Checks come before any launch; nothing is allocated
 * and nothing synchronizes.  Outputs must not overlap inputs except where a
 * call says so.
 * ====================================================================== */

/* element types */
#define HQ_DT_BF16 0
#define HQ_DT_F16 1
#define HQ_DT_F32 2

#define HQ_NORM_MAX_K 65536

/*
 * Residual addition, root-mean-square norm and K128 FP8 codes in one pass over
 * the rows (the activation quantizer's rule, hq_swiglu_fp8_k128, applied to
 * the normalized row):
 *   h = x + r rounded to the type (h = x without a residual),
 *   rstd = 1 / sqrt(mean(h^2) + eps), y = (h * rstd) * w in FP32,
 *   per group of 128 columns: s = max(amax, 1e-10) * float32(1/448),
 *   code = E4M3(y / s).
 *
 *  dtype      type of x, residual and residual_out; w_dtype: dtype or HQ_DT_F32.
 *  x, residual  [M, K], row strides given; residual NULL: none.
 *  weight     [K].   eps  >= 0 (0: a row of zeros has NaN codes).
 *  residual_out [M, K] contiguous: h (needed with a residual, else ignored).
 *             May be x or residual itself where that is contiguous.
 *  out_fp8    uint8 [M, K].
 *  scales     float: HQ_SCALE_ROWMAJOR [M, K/128], or HQ_SCALE_TRANSPOSED
 *             [K/128, scale_ld] (scale_ld >= M; columns behind M are left as
 *             they were); either may add HQ_FP8_UE8M0.
 *  rstd_opt   float [M] or NULL (the backward pass reads it).
 *  amax_opt   float, the groups' max |y| in the scales' layout, or NULL.
 *  K          multiple of 128, at most HQ_NORM_MAX_K.
 * A row with a NaN or an infinity has codes that are NaN wherever y is; the
 * group rule skips NaNs.  Squares are summed in FP32: |h| above 1e19 gives
 * rstd = 0.
 * Alignment: 16 bytes (rstd, scales, amax: 4), strides multiples of 8.
 * Errors: HQ_ERR_NULL, HQ_ERR_SHAPE, HQ_ERR_ALIGN, HQ_ERR_UNSUPPORTED,
 *         HQ_ERR_CUDA.
 */
hq_status hq_add_rmsnorm_fp8_k128(int dtype, const void *x, int64_t x_row_stride,
                                  const void *residual, int64_t residual_row_stride,
                                  const void *weight, int w_dtype, float eps, int64_t M, int64_t K,
                                  void *residual_out, uint8_t *out_fp8, float *scales, int scale_layout,
                                  int64_t scale_ld, float *rstd_opt, float *amax_opt, void *stream);

/*
 * The norm's gradients (the codes' rounding passes them straight through):
 *   g = dy * w, c = rstd^2 * mean(g * h), dx = rstd * (g - h * c) + dres,
 *   dweight = sum over the rows of dy * h * rstd.
 * dx is the gradient of x and of the residual alike.
 *  dtype      type of dy, h, dres and dx; w_dtype: dtype or HQ_DT_F32.
 *  dy, h, dres  [M, K] with row strides (dres NULL: none); rstd float [M].
 *  dx         [M, K] contiguous; may be dy or dres itself where contiguous.
 *  dweight    float [K], or NULL.
 *  ws         >= hq_rmsnorm_backward_workspace_size(M, K) bytes, 16-byte
 *             aligned, any contents (unused without dweight: may be NULL).
 *             Calls that share one must not overlap in time.
 * The sum over the rows is taken in a fixed order: equal inputs give equal
 * bits on one GPU model.  M == 0 gives dweight = 0.
 * Alignment and errors as above, and HQ_ERR_WORKSPACE.
 */
size_t hq_rmsnorm_backward_workspace_size(int64_t M, int64_t K);
hq_status hq_rmsnorm_backward(int dtype, const void *dy, int64_t dy_row_stride, const void *h,
                              int64_t h_row_stride, const void *weight, int w_dtype, const float *rstd,
                              const void *dres, int64_t dres_row_stride, int64_t M, int64_t K, void *dx,
                              float *dweight, void *ws, size_t ws_bytes, void *stream);

/* hq_rope layouts: which two elements of the rotated part make pair i */
#define HQ_ROPE_HALVES 0      /* i and i + rotary_dim / 2 */
#define HQ_ROPE_INTERLEAVED 1 /* 2 i and 2 i + 1 */

/* hq_rope_inv_freq scalings */
#define HQ_ROPE_PLAIN 0  /* base^(-2 i / rotary_dim) */
#define HQ_ROPE_LINEAR 1 /* divided by factor */
#define HQ_ROPE_NTK 2    /* base * factor^(rotary_dim / (rotary_dim - 2)) */
#define HQ_ROPE_PARTS 3  /* by parts: pairs that turn more than p1 times within
                            trained_len keep their frequency, those below p2
                            turns are divided by factor, a linear ramp over the
                            pair index between (its ends rounded outwards);
                            magnitude 0.1 ln(factor) + 1 */
#define HQ_ROPE_BANDS 4  /* by wavelength L: L < trained_len / p2 keeps, L >
                            trained_len / p1 is divided by factor, between the
                            two are mixed linearly in trained_len / L (p2 > p1) */

/*
 * Rotary frequencies in radians per position, on the host, in FP64:
 * inv_freq[rotary_dim / 2] and *magnitude (may be NULL), the factor that
 * hq_rope multiplies both cosine and sine with.  factor >= 1; trained_len, p1,
 * p2 (> 0) are read by HQ_ROPE_PARTS and HQ_ROPE_BANDS.
 * Errors: HQ_ERR_NULL, HQ_ERR_SHAPE (rotary_dim odd or < 2; NTK: < 4),
 *         HQ_ERR_UNSUPPORTED (unknown scaling, parameters out of range).
 */
hq_status hq_rope_inv_freq(int rotary_dim, double base, int scaling, double factor, double trained_len,
                           double p1, double p2, double *inv_freq, double *magnitude);

/*
 * Rotary positions of q and k in one launch: dimensions [offset, offset +
 * rotary_dim) of each head are turned pair by pair by the angle
 * position * inv_freq[i]; the others are passed through.
 *   (a, b) -> m (a cos - b sin), m (a sin + b cos), FP32, rounded once.
 * inverse != 0 turns by minus the angle (the gradient: the transpose of the
 * rotation, times the same magnitude).
 *  q, k       [T, Hq, D], [T, Hk, D]; strides of token and head; k may be NULL
 *             (Hk == 0).
 *  positions  int64 [T], any value (angles are reduced in FP64: absolute error
 *             below 4e-7 + |position| * inv_freq * 2^-50 radians).
 *  inv_freq   device double [rotary_dim / 2].
 *  q_out, k_out  same shapes, own strides; may be q and k themselves (same
 *             strides).
 * Any D, rotary_dim (even), offset and strides; 16-byte aligned rows with
 * whole chunks of 8 elements take wide loads, others element by element.
 * Alignment: to the element (positions, inv_freq 8 bytes).
 * Errors: HQ_ERR_NULL, HQ_ERR_SHAPE, HQ_ERR_ALIGN, HQ_ERR_UNSUPPORTED,
 *         HQ_ERR_CUDA.
 */
hq_status hq_rope(int dtype, const void *q, int64_t q_token_stride, int64_t q_head_stride, int Hq,
                  const void *k, int64_t k_token_stride, int64_t k_head_stride, int Hk, int64_t T, int D,
                  const int64_t *positions, const double *inv_freq, int rotary_dim, int offset, int layout,
                  float magnitude, int inverse, void *q_out, int64_t q_out_token_stride,
                  int64_t q_out_head_stride, void *k_out, int64_t k_out_token_stride,
                  int64_t k_out_head_stride, void *stream);

/*
 * Block tables and slot maps of one step, on the GPU.  Pages of page_size
 * tokens are held by requests (block_table) or lie on a stack (free_pages,
 * its height *free_count).
 *  lens        int32 [B], tokens cached so far.
 *  new_tokens  int32 [B], tokens to come in this step; < 0: the request has
 *              ended.
 *  block_table int32 [B, table_width], row stride table_width; entries below
 *              ceil(lens / page_size) are the request's pages.
 * In this order: the pages of ended requests go onto the stack (by request,
 * then page); the pages that the others need for lens + new_tokens come off
 * its top (by request, then page) into their rows.
 *  lens_out    int32 [B]: lens + new_tokens, 0 for ended requests.
 *  cu_new      int32 [B + 1]: running sum of the new tokens (0 where ended).
 *  slots, positions  int64 [n_slots]: for new token j of request b at row
 *              cu_new[b] + j its place in the cache, page * page_size +
 *              position % page_size, and its position lens[b] + j.  Rows
 *              behind the last token: slot -1, position 0.
 *  free_count_out  int32 [1].
 *  status      int32 [1]: 0, or a sum of HQ_KV_* reasons.  Then nothing is
 *              taken or given back: lens_out = lens, *free_count_out =
 *              *free_count, cu_new and positions 0, slots -1, block_table and
 *              free_pages unchanged.
 * lens_out may be lens, free_count_out may be free_count.  B <=
 * HQ_KV_MAX_REQUESTS; page_size a power of two from 16 to 1024.
 * Errors: HQ_ERR_NULL, HQ_ERR_SHAPE, HQ_ERR_ALIGN, HQ_ERR_UNSUPPORTED
 *         (page_size), HQ_ERR_CUDA.
 */
#define HQ_KV_MAX_REQUESTS 4096
#define HQ_KV_NO_PAGES 1   /* fewer free pages than the step needs */
#define HQ_KV_NO_ROWS 2    /* more new tokens than n_slots */
#define HQ_KV_NO_WIDTH 4   /* a request outgrows its row of the block table */
#define HQ_KV_BAD_STATE 8  /* a length is negative or does not fit its row, the stack's height is
                              outside [0, free_capacity], or its pages would not fit */
hq_status hq_kv_slots(int B, const int32_t *lens, const int32_t *new_tokens, int32_t *block_table,
                      int64_t table_width, int32_t *free_pages, int64_t free_capacity,
                      const int32_t *free_count, int page_size, int64_t n_slots, int32_t *lens_out,
                      int32_t *cu_new, int64_t *slots, int64_t *positions, int32_t *free_count_out,
                      int32_t *status, void *stream);

/*
 * The NVFP4 key/value cache: uint8 [num_pages, H, page_size / 16, 2432].  Keys
 * and values of HQ_KV4_HEAD = 128 dimensions are quantized one 128-vector at a
 * time as by hq_cat_rotate_nvfp4 (after the same 128-point Hadamard rotation
 * when hadamard_n is 128), 64 + 8 + 4 bytes each.  A group of 16 tokens of one
 * head holds, in bytes (token r, 16-element block b, element d = 16 b + e):
 *      0  K codes, pair (d, d + 1), e = 4 i + 2 j, i < 4, j < 2:
 *         64 r + 16 i + 2 b + j
 *   1024  V codes, pair (d, d + 1), e = 2 g, g < 8:
 *         512 (r / 8) + 64 g + 16 (r % 8 / 2) + 8 (r % 2) + b
 *   2048  K block scales (E4M3): 8 r + b
 *   2176  V block scales: 64 (r / 8) + 16 (r % 8 / 2) + 2 b + r % 2
 *   2304  K decode scales (float): 4 r
 *   2368  V decode scales (float): 4 r
 * so that a group is one contiguous copy and a lane of the attention kernel
 * finds the operands of its matrix instructions in 16-byte pieces.
 * Slot s is token s % page_size of page s / page_size.
 * page_size: a power of two from 16 to 1024.
 */
#define HQ_KV4_HEAD 128
#define HQ_KV4_GROUP_TOKENS 16
#define HQ_KV4_GROUP_BYTES 2432
/* bytes of a cache; 0 for sizes out of range */
size_t hq_kv4_cache_bytes(int64_t num_pages, int page_size, int H);

/*
 * Quantize new keys and values into the cache.
 *  k, v       [N, H, 128], strides of token and head, dtype HQ_DT_*.
 *  slots      int64 [N]; a slot outside [0, num_pages * page_size) is skipped
 *             (padding rows).  Slots of one call must differ: of a slot given
 *             twice the contents are undefined (no other slot is touched).
 *  hadamard_n 128 or 0.
 * Values must be finite.  Alignment: k, v 16 bytes, strides multiples of 8,
 * cache 16 bytes, slots 8.
 * Errors: HQ_ERR_NULL, HQ_ERR_SHAPE, HQ_ERR_ALIGN, HQ_ERR_UNSUPPORTED,
 *         HQ_ERR_CUDA.
 */
hq_status hq_kv4_append(int dtype, const void *k, int64_t k_token_stride, int64_t k_head_stride, const void *v,
                        int64_t v_token_stride, int64_t v_head_stride, const int64_t *slots, int64_t N, int H,
                        int hadamard_n, uint8_t *cache, int64_t num_pages, int page_size, void *stream);

/*
 * Read tokens back: k_out, v_out [N, H, 128] in dtype, each value code * block
 * scale * decode scale in FP32, rotated back (hadamard_n 128) or as stored (0),
 * rounded once.  A slot outside the cache gives zeros.  A slot may be given
 * more than once.  Other arguments and errors as hq_kv4_append.
 */
hq_status hq_kv4_gather(int dtype, const uint8_t *cache, int64_t num_pages, int page_size, const int64_t *slots,
                        int64_t N, int H, int hadamard_n, void *k_out, int64_t k_token_stride,
                        int64_t k_head_stride, void *v_out, int64_t v_token_stride, int64_t v_head_stride,
                        void *stream);

/*
 * Attention of the newest tokens of each request over the cache (their own
 * keys and values already appended).
 *  q, out     [Tq, Hq, 128], strides of token and head, dtype HQ_DT_BF16 or
 *             HQ_DT_F16.  Query head h reads key/value head h / (Hq / Hkv).
 *  block_table int32 [B, table_width], seq_lens int32 [B]: tokens in the cache,
 *             the queries' own among them.
 *  cu_q       int32 [B + 1] or NULL: request b's queries are rows [cu_q[b],
 *             cu_q[b + 1]), at most q_len of them; NULL: rows [b q_len,
 *             (b + 1) q_len).  Query j of n is at position seq_len - n + j.
 *  A query at position p sees the tokens t <= p, and with window > 0 only those
 *  with p - t < window or t < sinks.
 *   s_t = scale * q . k_t, out = sum_t softmax(s)_t v_t, lse = ln sum_t exp s_t
 *  over the tokens it sees; none: out = 0, lse = -inf.  (Scores times log2(e)
 *  below -1e30 count as not seen.  A query with a NaN or an infinity gets NaNs, in its
 *  own rows only.)
 *  hadamard_n the one that the cache was written with: q is rotated before,
 *             out rotated back after (rotations keep q . k).
 *  lse_opt    float [Tq, Hq] or NULL.
 *  Rows of out and lse behind the last request's are left as they were.
 *  ws         >= hq_kv4_attention_workspace_size() bytes, 16-byte aligned, in
 *             the rest state: the first HQ_KV4_ATTENTION_STATE_BYTES zero
 *             (hq_workspace_init), the others may hold anything; the call leaves
 *             it so.  Calls that share one must not overlap in time.
 * The workspace's error word (hq_get_error) is set to HQ_ERR_PAGE by a block-table
 * entry outside [0, num_pages) or a seq_len beyond the row's table_width *
 * page_size tokens (tokens without a page count as not seen), to HQ_ERR_SHAPE by a
 * request whose rows reach outside [0, Tq) or are more than q_len (those left out
 * are not written).
 * Arithmetic: scores in FP32 from FP16 keys (exact) and a query in two FP16 parts
 * (22 bits of an element, 2^-24 of its column's largest where that is more).  What
 * a token adds, its weight times its value's decode scale, is rounded to FP16 (BF16
 * outputs) or held in two FP16 parts (FP16 outputs) for the second product: 2^-11 or
 * 2^-22 of it, or 2^-34 of the largest such product among the tokens that the query
 * sees where that is more, whatever the sizes of the values.  Weights below 2^-125
 * of the row's largest may count as zero.  Sums in FP32.  Results do not
 * depend on anything but the inputs and the GPU's SM count.
 * Alignment: q, out, cache, ws 16 bytes, strides of q and out multiples of 8.
 * Errors: HQ_ERR_NULL, HQ_ERR_SHAPE (B > HQ_KV_MAX_REQUESTS, Hq not a multiple
 *         of Hkv, q_len * Hq / Hkv > 65536, a table row of more than 2^30
 *         tokens), HQ_ERR_ALIGN, HQ_ERR_WORKSPACE,
 *         HQ_ERR_UNSUPPORTED (dtype, hadamard_n, page_size, a negative window),
 *         HQ_ERR_CUDA.
 */
#define HQ_KV4_ATTENTION_STATE_BYTES 2304
size_t hq_kv4_attention_workspace_size(void);
hq_status hq_kv4_attention(int dtype, const void *q, int64_t q_token_stride, int64_t q_head_stride, int64_t Tq,
                           int Hq, const uint8_t *cache, int64_t num_pages, int page_size, int Hkv,
                           const int32_t *block_table, int64_t table_width, int B, const int32_t *seq_lens,
                           const int32_t *cu_q, int q_len, float scale, int window, int sinks, int hadamard_n,
                           void *out, int64_t out_token_stride, int64_t out_head_stride, float *lse_opt,
                           void *ws, size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* HQ_H */
