/*
 * qmoe.h -- C ABI of the GB300 (sm_103a) quantized Mixture-of-Experts expert
 * path: routed top-k pairs -> expert-sorted order -> grouped gate/up GEMM with
 * fused SwiGLU -> grouped down GEMM over packed low-bit expert weights ->
 * top-k-weighted combine in a fixed order.
 *
 * Sources the operations follow:
 *   [hip-ep]  "perf(qmoe): group prefill expert matmuls" -- description:
 *             grouped expert projections over symmetric int4 weights, one
 *             launch for all experts, deterministic scatter order.
 *   [gfx1151] "Evaluate native IU4/IU8 WMMA for grouped-INT MoE prefill on
 *             gfx1151" -- Problem (dequantise-then-dot for W4A16, decode is
 *             GEMV-like), Constraint (int8 x int8 -> int32 needs quantised
 *             activations: W8A8).
 *   [aiter]   the tuned grouped-fmoe config page for an MXFP4 model on
 *             gfx1250 -- Changes (fp8 activations, MXFP4 weights, two-stage
 *             grouped kernel), Test Plan (stage1/stage2 tiles, rel L2 check,
 *             K tiles larger than inter_dim excluded).
 *
 * Notation: T tokens, k = top_k, P = T*k routed pairs (pair p = t*k + j),
 * H hidden size, I intermediate size, E experts.  A "slot" is a position in
 * expert-sorted order; slot-ordered buffers hold one row per valid pair.
 *
 * Conventions for every call:
 *   - All array pointers are DEVICE pointers unless stated otherwise.  The
 *     caller owns every buffer, including the workspace; the library never
 *     allocates, frees or synchronises.
 *   - Calls are asynchronous on `stream` (NULL = the legacy default stream).
 *   - Host-side checks run before any launch: a NULL pointer, a dimension
 *     <= 0 (T may be 0), H or I not a multiple of 32, or a pointer not
 *     16-byte aligned returns QMOE_ERR_ARG; shapes beyond the kernels'
 *     limits return QMOE_ERR_UNSUPPORTED; a failed launch returns
 *     QMOE_ERR_LAUNCH.  Nothing is launched after an error.
 *   - Device-side errors never trap: a routing id outside [0, E) sets bit
 *     QMOE_DEV_BAD_EXPERT_ID of *dev_status (which the caller zeroes before
 *     the first call and reads after synchronising); that pair then takes no
 *     slot and contributes nothing to the output.  A tensor-core kernel whose
 *     pipeline wait exceeds its time limit sets QMOE_DEV_WAIT_TIMEOUT, stops
 *     and releases its resources; its outputs are then undefined.
 *   - Calls on different streams are independent when they use different
 *     output and workspace buffers.
 *
 * Storage formats (K = the reduction axis, always contiguous):
 *   bf16      uint16 bit patterns.
 *   int4      W [rows, K/2] bytes; element 2i in the low nibble of byte i,
 *             2i+1 in the high nibble; stored n = q + 8, value (n - 8) * s;
 *             scales fp16 [rows, K/32].  The W4A16 GEMMs take codes and
 *             scales pre-packed together (qmoe_prepack_int4_weights).
 *   E2M1      same nibble order; OCP MX element encoding; scales E8M0
 *             (value 2^(b-127)), one per 32 K elements.  The MXFP4 GEMMs take
 *             weights and scales pre-packed (qmoe_prepack_fp4_weights,
 *             qmoe_prepack_mx_scales).
 *   E4M3      OCP "fn" fp8 (max 448, no infinities).
 *   int8      W int8 [rows, K], fp32 scale per output row.
 * Weight tensors: W1 [E, 2I, H] (rows 0..I-1 gate, I..2I-1 up), W2 [E, H, I].
 */
#ifndef QMOE_H
#define QMOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t. */
typedef struct CUstream_st* qmoe_stream_t;

typedef enum {
    QMOE_OK = 0,
    QMOE_ERR_ARG = -1,
    QMOE_ERR_UNSUPPORTED = -2,
    QMOE_ERR_LAUNCH = -3,
    QMOE_ERR_CUDA = -4
} qmoe_status;

/* Bits of the device status word. */
enum { QMOE_DEV_BAD_EXPERT_ID = 1, QMOE_DEV_WAIT_TIMEOUT = 2, QMOE_DEV_BAD_OFFSETS = 4 };

typedef struct {
    int32_t T, k, H, I, E;
} qmoe_dims;

/* Human-readable name of a qmoe_status code (static string). */
const char* qmoe_status_str(int code);

/* Library version string (static). */
const char* qmoe_version(void);

/* ---------------------------------------------------------------- token-tile table
 *
 * Every call below cuts each expert's slots into token tiles of NMAX = 16, 112
 * or 224 rows (the activation tile layouts, the tile schedule qmoe_align_sort
 * writes, the GEMMs' work units).  Without rules NMAX is 224 when T*k > 96*E,
 * else 112.  A tuned table (the aiter tuned grouped-fmoe page, Changes: one
 * configuration row per model shape and token bucket) replaces that choice:
 *
 * qmoe_tile_rule -- matches dims with H, I, E, k equal to the rule's (0 = any)
 *   and t_min <= T <= t_max; nmax is 16, 112 or 224 (16 shrinks each
 *   pipeline slot of the MXFP4 GEMMs, so small batches keep more weight
 *   loads in flight).
 * qmoe_set_tile_rules -- replaces the table with rules[0..n) (n = 0 clears it);
 *   the first matching rule wins.  QMOE_ERR_ARG for a bad rule (table
 *   unchanged).  Host state shared by the process: set it before sizing
 *   buffers and workspaces for a shape, and not while calls for that shape are
 *   in flight, since every size and schedule of the shape follows NMAX.
 * qmoe_tile_nmax -- the NMAX the library uses for *d. */
typedef struct {
    int32_t H, I, E, k;
    int64_t t_min, t_max;
    int32_t nmax;
    int32_t reserved;
} qmoe_tile_rule;
int qmoe_set_tile_rules(const qmoe_tile_rule* rules, int n);
int qmoe_tile_nmax(const qmoe_dims* d);

/* ---------------------------------------------------------------- routing
 *
 * Bytes of device workspace the routing and GEMM calls need for dims *d
 * (scratch for per-chunk histograms, the GEMM tile schedule and each slot's
 * row in the token tiles). */
size_t qmoe_workspace_bytes(const qmoe_dims* d);

/* qmoe_align_sort -- expert-sorted permutation of the routed pairs.
 * [hip-ep] description (all experts grouped into one launch, the scatter
 * back kept in a deterministic order); [aiter] Changes (two-stage grouped
 * kernel over sorted tokens).
 *
 * in   topk_ids        int32 [T, k], expert id of pair p = t*k + j
 * out  counts          int32 [E], pairs routed to each expert
 * out  offsets         int32 [E+1], exclusive prefix sum of counts;
 *                      offsets[E] = number of valid pairs
 * out  sorted_pair_ids int32 [P]; slot s -> pair id, ascending p within an
 *                      expert (a stable sort); slots >= offsets[E] hold -1
 * out  pair_slot       int32 [P]; pair id -> slot, -1 for an invalid id
 * i/o  dev_status      int32 [1]; bit QMOE_DEV_BAD_EXPERT_ID is OR-ed in
 * ws   workspace of qmoe_workspace_bytes(d) bytes, 256-byte aligned; besides
 *      scratch it receives the token-tile schedule and each slot's token-tile
 *      row, which the permute, intermediate and GEMM calls read
 * The result is bit-identical run to run (no atomics decide an order).
 * qmoe_align_sort_routed -- the same, but for an id of -1: a pair that is meant to be
 *   routed nowhere, which is not reported. */
int qmoe_align_sort(const qmoe_dims* d, const int32_t* topk_ids, int32_t* counts, int32_t* offsets,
                    int32_t* sorted_pair_ids, int32_t* pair_slot, int32_t* dev_status, void* ws,
                    size_t ws_bytes, qmoe_stream_t stream);
int qmoe_align_sort_routed(const qmoe_dims* d, const int32_t* topk_ids, int32_t* counts, int32_t* offsets,
                           int32_t* sorted_pair_ids, int32_t* pair_slot, int32_t* dev_status, void* ws,
                           size_t ws_bytes, qmoe_stream_t stream);

/* qmoe_align_sort_static_scratch -- the same sort as qmoe_align_sort, for
 * callers that cannot allocate device memory.  The source pages have no
 * counterpart to this call; it exists for integrations where cudaMalloc is
 * not available when tokens are routed: a host framework that owns every
 * device allocation through its own pool, a plugin that may not allocate
 * after start-up, or a latency path where allocating is forbidden.
 *
 * The caller still passes every input and output (same meaning and layout as
 * qmoe_align_sort); the histogram scratch is a fixed array of
 * QMOE_STATIC_SCRATCH_BYTES inside the library, present on every GPU that
 * loads the library until the process exits.  No cudaMalloc, cudaFree or
 * other allocating call is made.
 *
 * Limits: E <= 4096 and ceil(T*k / 2048) * E * 4 <= QMOE_STATIC_SCRATCH_BYTES
 * (for example T*k <= 81920 with E = 512 uses 80 KiB); larger shapes return
 * QMOE_ERR_UNSUPPORTED before any launch -- use qmoe_align_sort with a
 * workspace for them.
 *
 * The first call on a device looks up the array's device address on the
 * current device (kept once it succeeds; a failed lookup returns
 * QMOE_ERR_CUDA and is tried again on the next call).  With lazy module
 * loading (the CUDA default) that lookup is also what loads the library's
 * device code onto the GPU and places the array there, so the first call is
 * not itself free of allocation: make it once per device at start-up, before
 * any region that must not allocate and before any stream capture.  Later
 * calls allocate nothing.  Every call on a device shares the one array and it keeps the last
 * call's contents; nothing in it needs to start at zero (each call rewrites
 * all it reads).  Calls whose executions overlap on the GPU (different
 * streams, or different host threads) race on the array: serialise them. */
#define QMOE_STATIC_SCRATCH_BYTES (1u << 20)
int qmoe_align_sort_static_scratch(const qmoe_dims* d, const int32_t* topk_ids, int32_t* counts, int32_t* offsets,
                                   int32_t* sorted_pair_ids, int32_t* pair_slot, int32_t* dev_status,
                                   qmoe_stream_t stream);

/* ---------------------------------------------------------------- activation quantisation
 *
 * qmoe_quant_act_mxfp8 -- bf16 rows to E4M3 codes with one E8M0 scale per 32
 * consecutive columns (the fp8 activations of [aiter] Changes).  Per block:
 * X = 2^(floor(log2 amax) - 8), code = nearest-even E4M3 of v / X saturated
 * to +-448; amax = 0 gives scale byte 127 and zero codes (OCP MX v1.0).
 * in x_bf16 [rows, cols]; out x_q uint8 [rows, cols], x_s uint8 [rows, cols/32].
 * cols must be a multiple of 32. */
int qmoe_quant_act_mxfp8(int64_t rows, int64_t cols, const uint16_t* x_bf16, uint8_t* x_q, uint8_t* x_s,
                         qmoe_stream_t stream);

/* MX activation tiles -- the layout in which the MXFP4 GEMMs take their
 * activations (x for stage 1, h for stage 2).  The valid slots of each expert
 * are cut into token tiles of NMAX rows (NMAX = qmoe_tile_nmax(d), see the
 * token-tile table; tile_start = prefix over experts of ceil(count / NMAX),
 * kept by qmoe_align_sort in its workspace).  For reduction length K the buffer holds,
 * per (tile t, K step kt of 128), a block of NMAX*128 + ceil(NMAX/128)*512
 * bytes at ((t * K/128) + kt) * that size:
 *   row r's 128 E4M3 codes at r*128, 16-byte chunk c at ((c ^ (r % 8)) * 16);
 *   then the E8M0 scales, row r / block b (0..3 of the step) at
 *   NMAX*128 + (r/128)*512 + 16*(r%32) + 4*((r%128)/32) + b.
 * Rows past a tile's token count are unspecified.
 *
 * qmoe_mx_tiles_bytes -- bytes of such a buffer for dims *d and length K. */
size_t qmoe_mx_tiles_bytes(const qmoe_dims* d, int64_t K);

/* qmoe_permute_quant_mxfp8 -- the expert-sorted permutation of the routed
 * activations and their MX quantisation (rule of qmoe_quant_act_mxfp8) in one
 * pass: for every pair p = t*k + j with pair_slot[p] >= 0 (the inverse
 * permutation from qmoe_align_sort), slot pair_slot[p] of its expert gets the
 * codes of token t, written as MX activation tiles with K = H.  Each token
 * row is read and quantised once and written to its k slots.
 * ws = the workspace qmoe_align_sort filled for this routing; the kernel
 * reads each pair's token-tile row from it (pair_slot and offsets must be
 * that call's outputs). */
int qmoe_permute_quant_mxfp8(const qmoe_dims* d, const uint16_t* x_bf16, const int32_t* pair_slot,
                             const int32_t* offsets, uint8_t* x_tiles, const void* ws, size_t ws_bytes,
                             qmoe_stream_t stream);

/* W4A16 activation tiles -- the layout in which the W4A16 GEMMs take their
 * activations: the token tiles of the MX layout above (same NMAX and
 * tile_start), per (tile t, K step kt of 64 elements) one block of NMAX*128
 * bytes at ((t * K/64) + kt) * NMAX*128, row r's 64 16-bit values at r*128
 * with 16-byte chunk c at ((c ^ (r % 8)) * 16); after the blocks a per-row
 * tail of fp32 values.  Two kinds:
 *   x tiles (K = H, stage-1 input): fp16 values v * 2^-e_r, where 2^-e_r is
 *     the power of two that moves the row's largest |v| into [2^14, 2^15)
 *     (e_r = 0 for a zero row; exact for bf16 inputs); tail: 2^e_r at
 *     (t*NMAX + r).  qmoe_w4a16_x_tiles_bytes(d) bytes.
 *   h tiles (K = I, stage-1 output / stage-2 input): bf16 values; tail: the
 *     largest |h| of each 32-column group at ((t*NMAX + r) * I/32 + g).
 *     qmoe_w4a16_h_tiles_bytes(d) bytes.
 * Rows past a tile's token count are unspecified. */
size_t qmoe_w4a16_x_tiles_bytes(const qmoe_dims* d);
size_t qmoe_w4a16_h_tiles_bytes(const qmoe_dims* d);

/* h16 tiles (K = I, stage-2 input): the x-tile form of h -- fp16 values
 * h * 2^-e_r with e_r chosen from the row's largest |h| as for x tiles, tail
 * 2^e_r at (t*NMAX + r).  qmoe_w4a16_h16_tiles_bytes(d) bytes (0 unless
 * I % 64 == 0).
 * qmoe_w4a16_h_to_f16 -- h tiles (from qmoe_gemm1_swiglu_w4a16) -> h16 tiles,
 * exactly for rows whose values stay within fp16's range after the scaling,
 * reading the group maxima of the h tail.  The input is not modified.  ws =
 * the workspace qmoe_align_sort filled for this routing. */
size_t qmoe_w4a16_h16_tiles_bytes(const qmoe_dims* d);
int qmoe_w4a16_h_to_f16(const qmoe_dims* d, const uint8_t* h_tiles, const int32_t* offsets, uint8_t* h16_tiles,
                        const void* ws, size_t ws_bytes, qmoe_stream_t stream);

/* qmoe_permute_x_f16 -- the expert-sorted permutation of the routed bf16
 * activations, written as W4A16 x tiles: slot s of expert e gets row
 * sorted_pair_ids[s] / k of x_bf16 [T, H] ([hip-ep] description: one grouped
 * launch over all experts' routed tokens).  H % 64 == 0.  ws = the workspace
 * qmoe_align_sort filled for this routing. */
int qmoe_permute_x_f16(const qmoe_dims* d, const uint16_t* x_bf16, const int32_t* sorted_pair_ids,
                       const int32_t* offsets, uint8_t* x_tiles, const void* ws, size_t ws_bytes,
                       qmoe_stream_t stream);

/* qmoe_quant_rows_int8_{bf16,f32} -- per-row symmetric int8 quantisation,
 * the activation-quantised W8A8 scheme of [gfx1151] Constraint: s = amax/127
 * (1 when amax = 0), q = clamp(rint(v / s), -127, 127), all in fp32.
 * in x [rows, cols] (bf16 bits or fp32); out q int8 [rows, cols], s fp32 [rows]. */
int qmoe_quant_rows_int8_bf16(int64_t rows, int64_t cols, const uint16_t* x, int8_t* q, float* s,
                              qmoe_stream_t stream);
int qmoe_quant_rows_int8_f32(int64_t rows, int64_t cols, const float* x, int8_t* q, float* s,
                             qmoe_stream_t stream);

/* W8A8 activation tiles -- the layout in which the W8A8 GEMMs take their
 * activations: the blocks of the W4A16 tiles above (same NMAX, tile_start,
 * 128-byte rows of 64 fp16 values, chunk swizzle), each value the fp16 equal
 * to an int8 code (exact); then a per-row tail of one fp32 scale s at
 * (t*NMAX + r); then, for each 112-row part h of a tile (ceil(NMAX/112)
 * parts; a 16-row tile is one short part) and each 128-element K step j, the
 * int32 max over the part's rows of sum |code| over the step, at
 * ((t*ceil(NMAX/112) + h) * K/128 + j): the GEMMs
 * bound their partial sums with it.  Rows past a tile's token count are
 * unspecified.
 * qmoe_w8a8_tiles_bytes -- bytes of such a buffer for dims *d and length K
 * (K % 128 == 0 and K <= 16384; 0 otherwise). */
size_t qmoe_w8a8_tiles_bytes(const qmoe_dims* d, int64_t K);

/* qmoe_permute_quant_int8 -- the expert-sorted permutation of the routed
 * activations and their per-token int8 quantisation (the rule of
 * qmoe_quant_rows_int8_bf16 applied to each token row of x_bf16 [T, H]) in
 * one pass: slot s gets the codes of token sorted_pair_ids[s] / k and its
 * scale, written as W8A8 tiles with K = H ([gfx1151] Constraint: W8A8 needs
 * quantised activations).  Each token row is read and quantised once and
 * written to its k slots.  H % 128 == 0, H <= 16384.  ws = the workspace
 * qmoe_align_sort filled for this routing; the kernel reads each pair's
 * token-tile row from it (sorted_pair_ids and offsets must be that call's
 * outputs). */
int qmoe_permute_quant_int8(const qmoe_dims* d, const uint16_t* x_bf16, const int32_t* sorted_pair_ids,
                            const int32_t* offsets, uint8_t* x_tiles, const void* ws, size_t ws_bytes,
                            qmoe_stream_t stream);

/* qmoe_quant_tiles_int8_f32 -- the W8A8 intermediate quantisation: each slot
 * row of h_f32 [P, I] (slot order, from qmoe_gemm1_swiglu_w8a8) quantised
 * with the rule of qmoe_quant_rows_int8_f32 and written as W8A8 tiles with
 * K = I.  I % 128 == 0, I <= 16384.  ws as above. */
int qmoe_quant_tiles_int8_f32(const qmoe_dims* d, const float* h_f32, const int32_t* offsets, uint8_t* h_tiles,
                              const void* ws, size_t ws_bytes, qmoe_stream_t stream);

/* ---------------------------------------------------------------- weight preparation
 *
 * qmoe_prepack_mx_scales -- one-time rearrangement of E8M0 weight scales
 * [rows, K/32] (row-major, one byte per 32 K elements) into the order the
 * block-scaled tensor-core MMA consumes: 512-byte atoms, one per (128-row
 * tile, group of 4 scale blocks), group index fastest; inside an atom, row r
 * (0..127) and block b (0..3) at byte 16*(r%32) + 4*(r/32) + b.  Padding rows
 * and blocks hold 127 (scale 1).  The MXFP4 GEMMs take their weight scales in
 * this form.  Output size: qmoe_mx_scales_packed_bytes(rows, K) bytes,
 * 16-byte aligned.  No counterpart on the pages: it is a storage-order
 * choice for this hardware, like any weight repacking at load time. */
size_t qmoe_mx_scales_packed_bytes(int64_t rows, int64_t K);
int qmoe_prepack_mx_scales(int64_t rows, int64_t K, const uint8_t* s_rowmajor, uint8_t* s_packed, qmoe_stream_t stream);

/* qmoe_prepack_fp4_weights -- one-time rearrangement of packed 4-bit weights
 * [rows, K/2 bytes] (element 2i in the low nibble of byte i) into tile-major
 * order: every 128-row x 128-element tile becomes one contiguous 8 KiB block,
 * tile (rt, kt) at (rt * ceil(K/128) + kt) * 8192, tile row r at r * 64 in it,
 * nibble order unchanged; padding is zero.  The MXFP4 GEMMs take their E2M1
 * weights in this form (a tile is then one contiguous read from HBM).
 * Output size: qmoe_fp4_weights_packed_bytes(rows, K), 32-byte aligned.  No
 * counterpart on the pages (a storage-order choice, made at load time). */
size_t qmoe_fp4_weights_packed_bytes(int64_t rows, int64_t K);
int qmoe_prepack_fp4_weights(int64_t rows, int64_t K, const uint8_t* w_rowmajor, uint8_t* w_packed,
                             qmoe_stream_t stream);

/* qmoe_prepack_int4_weights -- one-time rearrangement of symmetric int4
 * weights (codes [rows, K/2] bytes, nibble order as above, n = q + 8) and
 * their fp16 scales [rows, K/32] into the blocks the W4A16 GEMMs read: per
 * (128-row tile rt, 64-element K step kt) one 4608-byte block at
 * (rt * ceil(K/64) + kt) * 4608 holding row r's 32 code bytes at r*32 and
 * then, at 4096 + r*4, its two scales of the step as fp16(s * 2^p_r), where
 * 2^p_r is the power of two that moves the row's largest |s| into
 * [2^10, 2^11) (p_r = 0 for an all-zero row).  After all blocks, one fp32
 * 2^-p_r per row, ceil(rows/128)*128 of them.  Inside each 32-bit code word
 * (8 elements) the nibbles are reordered so that nibble j holds element 2j
 * and nibble 4+j element 2j+1 (j = 0..3).  Padding codes are 8 (value 0),
 * padding scales 0, padding rows' factors 1.  K % 32 == 0; packed 16-byte
 * aligned, codes 4-byte aligned.  Output size:
 * qmoe_int4_weights_packed_bytes(rows, K).  No counterpart on the pages (a
 * storage-order choice, made at load time). */
size_t qmoe_int4_weights_packed_bytes(int64_t rows, int64_t K);
int qmoe_prepack_int4_weights(int64_t rows, int64_t K, const uint8_t* w_rowmajor, const uint16_t* s_fp16,
                              uint8_t* packed, qmoe_stream_t stream);

/* ---------------------------------------------------------------- stage 1: gate/up + SwiGLU
 *
 * For every expert e and slot s in [offsets[e], offsets[e+1]), with
 * a = the activation row of token sorted_pair_ids[s] / k:
 *   g[n] = W1[e][n] . a,  u[n] = W1[e][I+n] . a,  h[s][n] = silu(g[n]) * u[n]
 * for n < I, silu(v) = v / (1 + exp(-v)); then h is quantised per scheme.
 * [hip-ep] description (grouped projections, all experts in one launch);
 * [aiter] Changes/Test Plan (stage 1 of the grouped a8w4 kernel).
 * Only slots < offsets[E] are written.
 *
 * W4A16 (tensor cores, fp16 MMAs; needs H % 256 == 0, I % 128 == 0,
 *        E <= 512): x_tiles = qmoe_permute_x_f16 output (K = H); w1 =
 *        qmoe_prepack_int4_weights of the int4 [E*2I, H/2] codes and their
 *        fp16 [E*2I, H/32] scales.  Each weight is dequantised on chip
 *        ([gfx1151] Problem: dequantise, then a 16-bit dot) to
 *        fp16((n - 8) * s * 2^p_r), one rounding of relative size <= 2^-11;
 *        products are summed in fp32 and the sums scaled back by
 *        2^(e_r - p_r), exactly; out h_tiles: h rounded to bf16 (nearest
 *        even), stored as W4A16 h tiles.  ws = the workspace that
 *        qmoe_align_sort filled for this routing. */
int qmoe_gemm1_swiglu_w4a16(const qmoe_dims* d, const uint8_t* x_tiles, const uint8_t* w1, const int32_t* offsets,
                            uint8_t* h_tiles, int32_t* dev_status, void* ws, size_t ws_bytes, qmoe_stream_t stream);

/* MXFP4 x FP8 (tensor cores; needs H % 256 == 0, I % 128 == 0, E <= 512):
 *        x_tiles = qmoe_permute_quant_mxfp8 output (MX activation tiles, K = H);
 *        w1 = qmoe_prepack_fp4_weights of the E2M1 [E*2I, H/2] bytes (32-byte
 *        aligned); w1_s = qmoe_prepack_mx_scales of the E8M0 [E*2I, H/32] scales;
 *        out h_tiles: the fp32 h quantised with the rule of
 *        qmoe_quant_act_mxfp8 along I, stored as MX activation tiles (K = I),
 *        qmoe_mx_tiles_bytes(d, I) bytes.  ws = the workspace that
 *        qmoe_align_sort filled for this routing (it holds the tile schedule). */
int qmoe_gemm1_swiglu_mxfp4(const qmoe_dims* d, const uint8_t* x_tiles, const uint8_t* w1, const uint8_t* w1_s,
                            const int32_t* offsets, uint8_t* h_tiles, int32_t* dev_status, void* ws,
                            size_t ws_bytes, qmoe_stream_t stream);

/* MXFP4 x FP8, gathering form: the same stage 1 (same weights, output, rules
 *        and limits) reading the activations token-major instead of from
 *        permuted tiles, as x plus the routing sort's order.  x_q uint8 [T, H]
 *        and x_s uint8 [T, H/32] = qmoe_quant_act_mxfp8 of x_bf16 [T, H]
 *        (16-byte aligned); sorted_pair_ids = the qmoe_align_sort output for
 *        this routing.  Row r of expert e's slots (slot offsets[e] + r) takes
 *        token sorted_pair_ids[offsets[e] + r] / k (an entry outside [0, T*k)
 *        is not read, and that row's output is undefined); the kernel copies that
 *        token's codes and scales into each pipeline step, so no expanded copy
 *        of x is written.  The result equals qmoe_gemm1_swiglu_mxfp4 on the
 *        qmoe_permute_quant_mxfp8 tiles of the same x, bit for bit ([aiter]
 *        Changes: fp8 activations into the stage-1 grouped GEMM). */
int qmoe_gemm1_swiglu_mxfp4_gather(const qmoe_dims* d, const uint8_t* x_q, const uint8_t* x_s,
                                   const int32_t* sorted_pair_ids, const uint8_t* w1, const uint8_t* w1_s,
                                   const int32_t* offsets, uint8_t* h_tiles, int32_t* dev_status, void* ws,
                                   size_t ws_bytes, qmoe_stream_t stream);

/* qmoe_mx_layer_gathers -- 1 if qmoe_moe_forward runs MXFP4 stage 1 in the
 *        gathering form for these dims (qmoe_quant_act_mxfp8, then
 *        qmoe_gemm1_swiglu_mxfp4_gather), 0 if through qmoe_permute_quant_mxfp8
 *        and qmoe_gemm1_swiglu_mxfp4; 0 for invalid dims.  Host only.  The two
 *        give the same bits; the choice is by speed: the gathering form when
 *        the token tile has 112 or 224 rows, I <= 512 and T*k >= 64*E. */
int qmoe_mx_layer_gathers(const qmoe_dims* d);

/* qmoe_forward_launches -- how many kernels one qmoe_moe_forward call with
 *        these dims and scheme launches (0 for invalid arguments).  Host only.
 *        The routing sort is one launch up to 2048 pairs and two above; then
 *        the activation quantisation, the two GEMMs, the W4A16 / integer
 *        intermediate pass, and the combine. */
int qmoe_forward_launches(const qmoe_dims* d, int scheme);

/* W8A8 (tensor cores; needs H % 256 == 0, I % 128 == 0, H and I <= 16384,
 *        E <= 512): x_tiles = qmoe_permute_quant_int8 output (K = H);
 *        w1 int8 [E, 2I, H] (row-major, as given; 16-byte aligned);
 *        w1_s fp32 [E, 2I].  The int8 x int8 products are summed exactly in
 *        int32 ([gfx1151] Constraint): the tensor cores take the codes as
 *        exact fp16 values and accumulate in fp32, and the epilogue carries
 *        the sum on in integers whenever the tiles' step maxima say a fp32
 *        partial sum could otherwise reach 2^24.  g = ((float)acc * s_x) *
 *        w1_s[e][n] in fp32, likewise u; out h fp32 [P, I] in slot order;
 *        dbg_acc (nullable, 16-byte aligned) int32 [P, 2I] receives the exact
 *        gate/up sums. */
int qmoe_gemm1_swiglu_w8a8(const qmoe_dims* d, const uint8_t* x_tiles, const int8_t* w1, const float* w1_s,
                           const int32_t* offsets, float* h, int32_t* dbg_acc, int32_t* dev_status, void* ws,
                           size_t ws_bytes, qmoe_stream_t stream);

/* W4A8 ([gfx1151] Constraint: int4 weights widened to 8-bit integers before
 *        the integer MMA, with int8 activations).  As W8A8 in every argument
 *        and rule except the weights: w1 holds int4 codes q in [-7, 7] as
 *        bytes [E, 2I, H/2] (byte i of a row: code 2i in the low nibble, code
 *        2i+1 in the high nibble, stored n = q + 8; 16-byte aligned), with
 *        one fp32 scale per output channel in w1_s [E, 2I].  The codes are
 *        widened on chip to exact fp16 integers; |q| <= 7 keeps every fp32
 *        partial sum below 2^24 for H, I <= 16384, so the sums are exact with
 *        no carry passes.  dbg_acc as for W8A8. */
int qmoe_gemm1_swiglu_w4a8(const qmoe_dims* d, const uint8_t* x_tiles, const uint8_t* w1, const float* w1_s,
                           const int32_t* offsets, float* h, int32_t* dbg_acc, int32_t* dev_status, void* ws,
                           size_t ws_bytes, qmoe_stream_t stream);

/* ---------------------------------------------------------------- stage 2: down projection
 *
 * y[s][c] = W2[e][c] . hq[s] for c < H, slots of expert e as above, summed
 * in fp32 and stored as bf16 (round to nearest even) [P, H] in slot order.  [aiter] Test Plan ("stage2 tiles"; K tiles larger
 * than inter_dim read out of bounds, so the kernels never let a K tile pass
 * the end of I).
 *
 * W4A16: h16_tiles from qmoe_w4a16_h_to_f16 (h rows already scaled into
 *        fp16 by powers of two); w2 = qmoe_prepack_int4_weights of the int4
 *        [E*H, I/2] codes and fp16 [E*H, I/32] scales, dequantised on chip as
 *        in stage 1; fp16 MMAs, fp32 sums scaled back by 2^(e_r - p_r); ws as
 *        for stage 1. */
int qmoe_gemm2_w4a16(const qmoe_dims* d, const uint8_t* h16_tiles, const uint8_t* w2, const int32_t* offsets,
                     uint16_t* y, int32_t* dev_status, void* ws, size_t ws_bytes, qmoe_stream_t stream);

/* MXFP4 x FP8: h_tiles from qmoe_gemm1_swiglu_mxfp4; w2 = qmoe_prepack_fp4_weights
 *        of the E2M1 [E*H, I/2] bytes; w2_s = qmoe_prepack_mx_scales of the
 *        E8M0 [E*H, I/32] scales; ws as for stage 1. */
int qmoe_gemm2_mxfp4(const qmoe_dims* d, const uint8_t* h_tiles, const uint8_t* w2, const uint8_t* w2_s,
                     const int32_t* offsets, uint16_t* y, int32_t* dev_status, void* ws, size_t ws_bytes,
                     qmoe_stream_t stream);

/* W8A8: h_tiles = qmoe_quant_tiles_int8_f32 output (K = I); w2 int8
 *        [E, H, I]; w2_s fp32 [E, H]; y = ((float)acc * s_h) * w2_s[e][c]
 *        with acc the exact int32 sum (as for stage 1); dbg_acc (nullable,
 *        16-byte aligned) int32 [P, H].  ws as for stage 1. */
int qmoe_gemm2_w8a8(const qmoe_dims* d, const uint8_t* h_tiles, const int8_t* w2, const float* w2_s,
                    const int32_t* offsets, uint16_t* y, int32_t* dbg_acc, int32_t* dev_status, void* ws,
                    size_t ws_bytes, qmoe_stream_t stream);

/* W4A8: as W8A8 stage 2 with w2 int4 codes [E, H, I/2] (layout of stage 1)
 *        and w2_s fp32 [E, H]. */
int qmoe_gemm2_w4a8(const qmoe_dims* d, const uint8_t* h_tiles, const uint8_t* w2, const float* w2_s,
                    const int32_t* offsets, uint16_t* y, int32_t* dbg_acc, int32_t* dev_status, void* ws,
                    size_t ws_bytes, qmoe_stream_t stream);

/* ---------------------------------------------------------------- combine
 *
 * qmoe_combine -- out[t][c] = bf16( sum_{j=0..k-1} topk_w[t][j] * y[pair_slot[t*k+j]][c] ),
 * summed in fp32 with j ascending from 0 (a fixed order, so the result is
 * reproducible bit for bit: [hip-ep] description, "deterministic scatter
 * order").  Pairs with pair_slot = -1 contribute nothing.
 * in y bf16 [P, H] (slot order), topk_w fp32 [T, k], pair_slot int32 [P];
 * out out_bf16 [T, H]. */
int qmoe_combine(const qmoe_dims* d, const uint16_t* y, const float* topk_w, const int32_t* pair_slot,
                 uint16_t* out_bf16, qmoe_stream_t stream);

/* ---------------------------------------------------------------- whole layer
 *
 * One call for the whole path: routing, activation quantisation (MXFP4,
 * W8A8, W4A8), stage 1, intermediate quantisation (W8A8, W4A8), stage 2 and
 * combine, all launched in order on `stream`.  scheme: 0 = W4A16, 1 = MXFP4
 * x FP8, 2 = W8A8, 3 = W4A8.  Weights and scales as for the per-stage calls (MXFP4 weights
 * and scales pre-packed; W4A16 weights pre-packed with their scales, so
 * w1_s and w2_s are ignored and may be NULL for scheme 0).  All
 * intermediates live in the caller's workspace of
 * qmoe_forward_workspace_bytes(d, scheme) bytes (256-byte aligned).
 * dev_status as for qmoe_align_sort. */
size_t qmoe_forward_workspace_bytes(const qmoe_dims* d, int scheme);
int qmoe_moe_forward(int scheme, const qmoe_dims* d, const uint16_t* x_bf16, const int32_t* topk_ids,
                     const float* topk_w, const void* w1, const void* w1_s, const void* w2, const void* w2_s,
                     uint16_t* out_bf16, int32_t* dev_status, void* ws, size_t ws_bytes, qmoe_stream_t stream);

/* ---------------------------------------------------------------- around the experts: norms
 *
 * The calls from here on take values of several types (qmoe_dtype) and rows
 * with a stride: ld* is the distance in elements between rows, at least the
 * columns; columns are contiguous.  Pointers need the alignment of their type
 * only; 16-byte aligned rows of a multiple of 8 columns run faster.  A type
 * code, mode or stride outside these rules returns QMOE_ERR_ARG, a shape
 * beyond a stated limit QMOE_ERR_UNSUPPORTED.  An output may not overlap an
 * input unless the call says so.  Zero rows are valid and write what sums over
 * no rows give.  The norms' waits for their own copies give up after some 2 s,
 * as only a fault of the machine makes them; the row then has NaN values. */
enum { QMOE_F32 = 0, QMOE_BF16 = 1, QMOE_F16 = 2 };

/* What a block's gate is one value for: nothing (no gate), a row (fp32 [rows]),
 * a column (fp32 [cols]) or an element (block type, [rows, cols] of row stride
 * ldg). */
enum { QMOE_GATE_NONE = 0, QMOE_GATE_ROW = 1, QMOE_GATE_COL = 2, QMOE_GATE_FULL = 3 };

/* qmoe_norm_pre -- the norm that opens a block:
 *   rstd[t] = 1 / sqrt(mean_c x[t][c]^2 + eps),  n[t][c] = x[t][c] * rstd[t] * w[c].
 * x has the stream's type, n the block's type: the same as the stream's, or a
 * 16-bit type beside an fp32 stream.  All arithmetic is fp32, rounded once.
 * cols <= 16384.  eps >= 0.
 * in x [rows, cols], w fp32 [cols];  out n [rows, cols], rstd fp32 [rows] (may
 * be NULL; the gradient needs it). */
int qmoe_norm_pre(int64_t rows, int64_t cols, int stream_dtype, int block_dtype, const void* x, int64_t ldx,
                  const float* w, float eps, void* n, int64_t ldn, float* rstd, qmoe_stream_t stream);

/* qmoe_norm_post -- the end of a block, and the norm that opens the next one:
 *   z = y * rstd * w  (w NULL: z = y, no norm),
 *   out = r + alpha * gate * z,
 *   n = out * rstd_next * w_next  (w_next NULL: not computed),
 * with rstd and rstd_next the reciprocal root mean squares of y and of out
 * (taken of the fp32 sum, before out is rounded).  r and out have the stream's
 * type, y, n and a full gate the block's.  out may be r.
 * rstd and rstd_next fp32 [rows], may be NULL. */
int qmoe_norm_post(int64_t rows, int64_t cols, int stream_dtype, int block_dtype, const void* r, int64_t ldr,
                   const void* y, int64_t ldy, const float* w, int gate_mode, const void* gate, int64_t ldg,
                   float alpha, const float* w_next, float eps, void* out, int64_t ldo, void* n, int64_t ldn,
                   float* rstd, float* rstd_next, qmoe_stream_t stream);

/* Gradients.  Column sums (dw, dw_next, a column gate's) are fp32, added in a
 * fixed order through the workspace of qmoe_norm_bwd_workspace_bytes(rows,
 * cols) bytes (256-byte aligned): the same inputs give the same bits.
 *
 * qmoe_norm_pre_backward -- dx = dres + d(n)/d(x) . dn (dres NULL: without it),
 *   dw[c] = sum_t dn[t][c] x[t][c] rstd[t].  dres and dx have the stream's type;
 *   dx may be dres.  rstd as qmoe_norm_pre gave it.
 *
 * qmoe_norm_post_backward -- with D = dout (NULL: 0) + d(n)/d(out) . dn (dn NULL:
 *   without it, and out, w_next, rstd_next, dw_next are ignored):
 *   dr = D;  dz = alpha * gate * D;  dy = d(z)/d(y) . dz;  dw = sum_t dz y rstd;
 *   dgate = alpha * z * D summed over what the gate is shared by (fp32, a full
 *   gate's in the block's type).  dout or dn must be given.  dw and dgate are
 *   written where w and gate are given, and may then not be NULL.  dr may be dout. */
size_t qmoe_norm_bwd_workspace_bytes(int64_t rows, int64_t cols);
int qmoe_norm_pre_backward(int64_t rows, int64_t cols, int stream_dtype, int block_dtype, const void* dn,
                           int64_t lddn, const void* x, int64_t ldx, const float* rstd, const float* w,
                           const void* dres, int64_t lddres, void* dx, int64_t lddx, float* dw, void* ws,
                           size_t ws_bytes, qmoe_stream_t stream);
int qmoe_norm_post_backward(int64_t rows, int64_t cols, int stream_dtype, int block_dtype, const void* dout,
                            int64_t lddout, const void* y, int64_t ldy, const float* w, const float* rstd,
                            int gate_mode, const void* gate, int64_t ldg, float alpha, const void* dn, int64_t lddn,
                            const void* out, int64_t ldo, const float* w_next, const float* rstd_next, void* dr,
                            int64_t lddr, void* dy, int64_t lddy, float* dw, void* dgate, int64_t lddg,
                            float* dw_next, void* ws, size_t ws_bytes, qmoe_stream_t stream);

/* ---------------------------------------------------------------- around the experts: routing
 *
 * qmoe_route_topk -- the k experts of each token, their weights, and the load
 *   statistics:
 *   p[t] = softmax(logits[t]);  ids[t] = the k experts of largest logit + bias
 *   (bias NULL: 0; an fp32 sum), largest first, the lower id first where equal;
 *   w[t][j] = scale * p[t][ids[t][j]], or with renorm scale * softmax over the
 *   k chosen logits.
 * The bias is added to the logit.  (Routers that balance their experts by a bias
 * on the score, the sigmoid or the softmax of the logit, choose otherwise: their
 * biases are not meant here, and there is no sigmoid score.)
 * A logit of -inf is an expert that is not available: it has p = 0 and is never
 * chosen; NaN counts as -inf, +inf as the largest finite fp32 value, whatever
 * the logits' type.  Places that no available expert fills hold id -1 and weight
 * 0.  A token whose mask byte is 0 (mask NULL: none) or whose logits are all -inf
 * is routed nowhere: ids -1, weights 0, lse -inf, no part in the statistics.  (An
 * id of -1 in topk_ids contributes nothing to qmoe_moe_forward and raises
 * QMOE_DEV_BAD_EXPERT_ID.)
 * Statistics (counts, probs, loss: all three or none), over the n routed tokens:
 *   counts[e] = pairs of expert e, counts[E] = n;  probs[e] = mean_t p[t][e];
 *   loss = coef * E * sum_e counts[e] / (k n) * probs[e]  (0 for n = 0).
 * E <= 1024, k <= min(E, 32).  scale > 0.
 * in logits [T, E] of row stride ld, bias fp32 [E], mask uint8 [T];  out ids
 * int32 [T, k], w fp32 [T, k], lse fp32 [T] (logsumexp of the logits; may be
 * NULL, the gradient needs it), counts int32 [E + 1], probs fp32 [E], loss fp32
 * [1].  ws of qmoe_route_workspace_bytes(T, E) bytes, 256-byte aligned, for the
 * statistics (else NULL). */
size_t qmoe_route_workspace_bytes(int64_t T, int E);
int qmoe_route_topk(int64_t T, int E, int k, int dtype, const void* logits, int64_t ld, const float* bias,
                    const uint8_t* mask, int renorm, float scale, int32_t* ids, float* w, float* lse, float coef,
                    int32_t* counts, float* probs, float* loss, void* ws, size_t ws_bytes, qmoe_stream_t stream);

/* qmoe_route_topk_backward -- dlogits [T, E] (the logits' type, row stride ldd)
 *   from dw fp32 [T, k] (gradient of the weights; NULL: none) and dloss fp32 [1]
 *   (gradient of the loss; NULL: none), one at least.  The counts and the
 *   choice of experts are constants.  logits, renorm, scale, coef as in the
 *   forward call, ids, w, lse, counts as it gave them. */
int qmoe_route_topk_backward(int64_t T, int E, int k, int dtype, const void* logits, int64_t ld, const int32_t* ids,
                             const float* w, const float* lse, int renorm, float scale, const float* dw, float coef,
                             const int32_t* counts, const float* dloss, void* dlogits, int64_t ldd,
                             qmoe_stream_t stream);

/* ---------------------------------------------------------------- around the experts: FP8 products
 *
 * E4M3 codes with one fp32 scale for each 128 values along the reduction axis
 * (of one row, or of 128 rows together).  A block of values v gets
 *   amax = max(max |v|, 2^-100),  code = E4M3(v * (448 / amax)),  scale = amax / 448
 * with fp32 divisions and products rounded to nearest and codes rounded to
 * nearest even, saturating; NaN keeps a NaN code, and a block with an infinity
 * gives NaN products.  The last block of an axis may be shorter.
 * Codes are uint8 [rows, cols], row stride ldq a multiple of 16, base 16-byte
 * aligned; bytes from cols to the next multiple of 16 may be overwritten.
 *
 * qmoe_fp8_quant_rows -- a scale for each 128 of a row.  x [rows, cols] of type
 *   dtype -> q, s fp32 [ceil(cols / 128), rows].
 * qmoe_fp8_quant_cols -- a scale for each 128 of a column, transposed: qt [cols,
 *   rows], st fp32 [ceil(rows / 128), cols]; where q is given also what
 *   qmoe_fp8_quant_rows gives (q, s), from the same read of x.
 * qmoe_fp8_quant_blocks -- a scale for each 128 x 128 block: q [rows, cols]
 *   and / or qt [cols, rows] (the same codes transposed), s fp32 [ceil(rows / 128),
 *   ceil(cols / 128)].  rows <= 8388480 for the last two. */
int qmoe_fp8_quant_rows(int64_t rows, int64_t cols, int dtype, const void* x, int64_t ldx, uint8_t* q, int64_t ldq,
                        float* s, qmoe_stream_t stream);
int qmoe_fp8_quant_cols(int64_t rows, int64_t cols, int dtype, const void* x, int64_t ldx, uint8_t* qt, int64_t ldqt,
                        float* st, uint8_t* q, int64_t ldq, float* s, qmoe_stream_t stream);
int qmoe_fp8_quant_blocks(int64_t rows, int64_t cols, int dtype, const void* x, int64_t ldx, uint8_t* q, int64_t ldq,
                          uint8_t* qt, int64_t ldqt, float* s, qmoe_stream_t stream);

/* A matrix of E4M3 codes: q [rows, K] of row stride ld (as above); the scale of
 * (row r, block b of 128 along K) is s[(r / s_rows) * s_row + b * s_blk], s_rows
 * 1 or 128. */
typedef struct {
    const uint8_t* q;
    int64_t ld;
    const float* s;
    int64_t s_row, s_blk;
    int32_t s_rows;
    int32_t reserved;
} qmoe_fp8_mat;

/* qmoe_fp8_matmul -- c[m][n] = sum over blocks of sa(m) sb(n) sum_k a[m][k] b[n][k]:
 *   each block of 128 is summed by the tensor core from zero, the scaled sums
 *   of the blocks in fp32 in a fixed order, and c (type c_dtype, row stride ldc)
 *   rounded once.  a [M, K], b [N, K].  dev_status int32 [1]: bit
 *   QMOE_DEV_WAIT_TIMEOUT is OR-ed in if a wait of the kernel runs out (c is
 *   then undefined).  QMOE_ERR_UNSUPPORTED for sizes above 2^30.
 * qmoe_fp8_linear -- y = x w^T: qmoe_fp8_quant_rows of x [M, K] (type x_dtype)
 *   into the workspace (qmoe_fp8_linear_workspace_bytes(M, K) bytes, 256-byte
 *   aligned), then qmoe_fp8_matmul. */
int qmoe_fp8_matmul(int64_t M, int64_t N, int64_t K, const qmoe_fp8_mat* a, const qmoe_fp8_mat* b, void* c,
                    int c_dtype, int64_t ldc, int32_t* dev_status, qmoe_stream_t stream);
size_t qmoe_fp8_linear_workspace_bytes(int64_t M, int64_t K);
int qmoe_fp8_linear(int64_t M, int64_t N, int64_t K, int x_dtype, const void* x, int64_t ldx, const qmoe_fp8_mat* w,
                    void* y, int y_dtype, int64_t ldy, int32_t* dev_status, void* ws, size_t ws_bytes,
                    qmoe_stream_t stream);

/* ---------------------------------------------------------------- training the experts: grouped products
 *
 * Rows in expert order (slots): expert e has the rows offsets[e] <= s <
 * offsets[e + 1] of P, as qmoe_align_sort gives them; rows from offsets[E] on
 * have no expert.  Weights [E, N, K], 16 bits (dtype QMOE_BF16 or QMOE_F16, of all
 * matrices of a call), row stride ldw, w_expert elements from expert to expert.
 *
 * qmoe_expert_linear -- y[s][n] = sum_k w[e][n][k] x[s][k].
 * qmoe_expert_linear_dx -- dx[s][k] = sum_n w[e][n][k] dy[s][n].
 * qmoe_expert_linear_dw -- dw[e][n][k] = sum_s dy[s][n] x[s][k], contiguous [E, N, K];
 *   zeros for an expert without rows.
 * Sums are fp32 and rounded once, to dtype or, where y_dtype, dx_dtype or dw_dtype
 * is QMOE_F32, not at all.  Rows of y and dx without an expert are zeros.  The same
 * inputs give the same bits.
 * pairs (may be NULL) int32 [P]: x has x_rows rows and the row of slot s is
 *   x[pairs[s] / k], as for sorted_pair_ids of qmoe_align_sort and x token by
 *   token; an entry below 0 or past x counts as a row of zeros.  Without pairs x
 *   has P rows, and k and x_rows are ignored.
 * offsets int32 [E + 1] from 0 to at most P, none below the one before it; else bit
 *   QMOE_DEV_BAD_OFFSETS of *dev_status is set, and which rows belong to which
 *   expert is undefined.  QMOE_DEV_WAIT_TIMEOUT as for qmoe_fp8_matmul.
 * ws (256-byte aligned; NULL where nothing is needed): qmoe_expert_workspace_bytes
 *   (op 0 for qmoe_expert_linear, 1 for ..._dx, 2 for ..._dw; pairs: whether they are
 *   given), and for each x, dy or w whose base or strides are no multiples of 16
 *   bytes, which is copied first, qmoe_expert_copy_bytes(rows, columns) (for w E * N
 *   rows; x with pairs as it lies).  But qmoe_expert_linear needs none at all where w is
 *   such and qmoe_expert_linear_in_place is 1: few rows, beside which w is read as it
 *   lies.
 * E <= 1024, other sizes <= 2^30. */
size_t qmoe_expert_copy_bytes(int64_t rows, int64_t cols);
size_t qmoe_expert_workspace_bytes(int64_t P, int E, int64_t N, int64_t K, int op, int pairs);
int qmoe_expert_linear_in_place(int64_t P, int E, int64_t N, int64_t K);
int qmoe_expert_linear(int64_t P, int E, int64_t N, int64_t K, int dtype, const void* x, int64_t ldx, int64_t x_rows,
                       const int32_t* pairs, int k, const void* w, int64_t ldw, int64_t w_expert,
                       const int32_t* offsets, void* y, int y_dtype, int64_t ldy, int32_t* dev_status, void* ws,
                       size_t ws_bytes, qmoe_stream_t stream);
int qmoe_expert_linear_dx(int64_t P, int E, int64_t N, int64_t K, int dtype, const void* dy, int64_t lddy,
                          const void* w, int64_t ldw, int64_t w_expert, const int32_t* offsets, void* dx, int dx_dtype,
                          int64_t lddx, int32_t* dev_status, void* ws, size_t ws_bytes, qmoe_stream_t stream);
int qmoe_expert_linear_dw(int64_t P, int E, int64_t N, int64_t K, int dtype, const void* dy, int64_t lddy,
                          const void* x, int64_t ldx, int64_t x_rows, const int32_t* pairs, int k,
                          const int32_t* offsets, void* dw, int dw_dtype, int32_t* dev_status, void* ws,
                          size_t ws_bytes, qmoe_stream_t stream);

/* ---------------------------------------------------------------- training the experts: SwiGLU, weighted sum
 *
 * qmoe_swiglu -- h = silu(g) u for rows gu = [g, u] [rows, 2 I], silu(v) = v s(v),
 *   s(v) = 1 / (1 + exp(-v)).  gu, h of type dtype.
 * qmoe_swiglu_backward -- dg = dh u s (1 + g (1 - s)), du = dh g s, dgu = [dg, du];
 *   h (NULL: not made) as qmoe_swiglu gives it.  dgu may be gu. */
int qmoe_swiglu(int64_t rows, int64_t I, int dtype, const void* gu, int64_t ldgu, void* h, int64_t ldh,
                qmoe_stream_t stream);
int qmoe_swiglu_backward(int64_t rows, int64_t I, int dtype, const void* dh, int64_t lddh, const void* gu, int64_t ldgu,
                         void* dgu, int64_t lddgu, void* h, int64_t ldh, qmoe_stream_t stream);

/* qmoe_weighted_sum -- qmoe_combine for any type, width and stride:
 *   out[t] = sum_j w[t][j] y[pair_slot[t][j]]  (w NULL: 1, the gradient of a gather),
 *   summed in fp32 with j ascending.  y [P, H], out [T, H] of type dtype; a slot
 *   outside [0, P) contributes nothing.
 * qmoe_weighted_sum_backward -- dy[pair_slot[t][j]] = w[t][j] dout[t], zeros in the
 *   rows of dy from *routed on (offsets + E of qmoe_align_sort); dw[t][j] =
 *   <y[pair_slot[t][j]], dout[t]>, 0 for a pair without a slot.  y and dw both or
 *   neither (NULL).  No slot may be there twice.  H <= 2^30, T * k < 2^31, P < 2^31. */
int qmoe_weighted_sum(int64_t T, int k, int64_t P, int64_t H, int dtype, const void* y, int64_t ldy, const float* w,
                      const int32_t* pair_slot, void* out, int64_t ldo, qmoe_stream_t stream);
int qmoe_weighted_sum_backward(int64_t T, int k, int64_t P, int64_t H, int dtype, const void* dout, int64_t lddout,
                               const void* y, int64_t ldy, const float* w, const int32_t* pair_slot,
                               const int32_t* routed, void* dy, int64_t lddy, float* dw, qmoe_stream_t stream);

/* ---------------------------------------------------------------- 4-bit products of few tokens
 *
 * Weights as the checkpoint holds them, not prepacked: codes uint8 [N, K / 2]
 * (16-byte aligned, rows and experts one behind the other; element 2i in the low
 * nibble of byte i) and a scale for each `group` values of a row.
 *   QMOE_W4_INT4  value (n - 8) s, s fp16 [N, K / group], group 32, 64 or 128;
 *   QMOE_W4_E2M1  E2M1 elements, s E8M0 bytes [N, K / 32], group 32.
 * K is a multiple of group.
 *
 * qmoe_w4_linear -- y[t] = W x[t], or with ids int32 [T, k] of E matrices the
 *   products of each token with its experts, y [T * k, N]:
 *   y[t k + j] = W[ids[t][j]] x[t]; a row whose id is outside [0, E) is zeros.
 *   (ids NULL: one matrix, E = k = 1; T * k <= 32768 with ids.)  A row of x with a NaN
 *   gives NaN, one with an infinity no finite value: NaN or an infinity; other rows are
 *   what they are without it.  Beside int4 codes x is below 2^117.
 *   x [T, K] and y of type dtype (QMOE_BF16 or QMOE_F16; y_dtype may be QMOE_F32).  No
 *   weight is rounded, sums are fp32: with ids, and up to QMOE_W4_FEW or some more
 *   tokens, codes are multiplied as they are and groups' sums by their scales; above it
 *   W is widened into the workspace, in dtype (int4: two matrices whose sum is W), for
 *   the grouped product.  Scales may be of any size their type holds: in fp16 each row
 *   of W is widened over a power of two (what is below 2^-39 of the row's largest is
 *   lost).
 * qmoe_w4_linear_dx -- dx = dy W for one matrix, W widened as above, in fp16 each
 *   column over a power of two.
 * ws of qmoe_w4_workspace_bytes(T, N, K, dx) bytes (dx 0 for the product, 1 for the
 * gradient; 0 bytes: NULL), 256-byte aligned, and dev_status as for
 * qmoe_expert_linear. */
enum { QMOE_W4_INT4 = 0, QMOE_W4_E2M1 = 1 };
#define QMOE_W4_FEW 16
size_t qmoe_w4_workspace_bytes(int64_t T, int64_t N, int64_t K, int dx);
int qmoe_w4_linear(int64_t T, int k, int E, int64_t N, int64_t K, int format, int group, int dtype, const void* x,
                   int64_t ldx, const uint8_t* w, const void* s, const int32_t* ids, void* y, int y_dtype, int64_t ldy,
                   int32_t* dev_status, void* ws, size_t ws_bytes, qmoe_stream_t stream);
int qmoe_w4_linear_dx(int64_t T, int64_t N, int64_t K, int format, int group, int dtype, const void* dy, int64_t lddy,
                      const uint8_t* w, const void* s, void* dx, int dx_dtype, int64_t lddx, int32_t* dev_status,
                      void* ws, size_t ws_bytes, qmoe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* QMOE_H */
