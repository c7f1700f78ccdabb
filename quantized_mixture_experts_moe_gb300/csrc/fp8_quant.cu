// FP8 (E4M3) quantisation with one fp32 scale for each 128 values:
// qmoe_fp8_quant_rows (128 along a row), qmoe_fp8_quant_cols (128 down a
// column, codes transposed; the row form besides), qmoe_fp8_quant_blocks
// (128 x 128; codes as they are and transposed).
//
//   amax = max(|block|, 2^-100),  q = E4M3(x * (448 / amax)) to nearest even,
//   saturating,  scale = amax / 448
//
// Both divisions and the product are correctly rounded fp32 operations, so a
// code does not depend on which of the kernels made it.  Each value is read
// once; HBM is the bound of the row form (2 bytes in and 1 out for each code of
// a 16-bit input).  The tile forms reach 0.57 of a copy's rate: a CTA has one
// tile, so its loads, sums and stores follow one another, and 512 or 1024 CTAs
// on 304 places end unevenly.
//
// 16-bit input: rows of 8192 x 4096 19.3 us, 5.2 TB/s (0.78 of a copy's rate);
// columns of 4096 x 4096 13.2 us, rows and columns from one read 17.7; 128 x 128
// blocks of 2048 x 4096 with both orders of the codes 8.8 us.  Rows off the
// 16-byte boundaries are read value by value: 8192 x 4095 31 us.
#include "row_ops.cuh"

namespace qmoe {
namespace fp8 {

constexpr float AMAX_MIN = 7.888609052210118e-31f;  // 2^-100

__device__ __forceinline__ float inverse_of(float amax) { return __fdiv_rn(448.f, amax); }
__device__ __forceinline__ float scale_of(float amax) { return __fdiv_rn(amax, 448.f); }
// 8 values of a row as they lie in memory.
template <typename T> using Raw8 = row::Raw<T, 8>;

// fmaxf drops a NaN; its own code is still NaN.
template <typename T>
__device__ __forceinline__ float amax8(const Raw8<T>& r, float m) {
    float v[8];
    row::widen<8>(r, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
    return m;
}
__device__ __forceinline__ uint2 codes8(const float (&v)[8], float inv) {
    uint2 q;
    q.x = (uint32_t)e4m3x2_from_float(__fmul_rn(v[0], inv), __fmul_rn(v[1], inv)) |
          ((uint32_t)e4m3x2_from_float(__fmul_rn(v[2], inv), __fmul_rn(v[3], inv)) << 16);
    q.y = (uint32_t)e4m3x2_from_float(__fmul_rn(v[4], inv), __fmul_rn(v[5], inv)) |
          ((uint32_t)e4m3x2_from_float(__fmul_rn(v[6], inv), __fmul_rn(v[7], inv)) << 16);
    return q;
}
template <typename T>
__device__ __forceinline__ uint2 codes8(const Raw8<T>& r, float inv) {
    float v[8];
    row::widen<8>(r, v);
    return codes8(v, inv);
}

__device__ __forceinline__ void set8(Raw8<float>& r, const float (&v)[8]) {
    r.a = make_float4(v[0], v[1], v[2], v[3]);
    r.b = make_float4(v[4], v[5], v[6], v[7]);
}
template <typename T>
__device__ __forceinline__ void set8(Raw8<T>& r, const float (&v)[8]) {
    r.v = make_uint4(row::pack2(v[0], v[1], T{}), row::pack2(v[2], v[3], T{}), row::pack2(v[4], v[5], T{}),
                     row::pack2(v[6], v[7], T{}));
}

// 8 values of a row from column c on; zeros past the row's end, and where the row is not `real`.
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* row, bool real, int64_t c, int64_t cols, Raw8<T>& r) {
    if (VEC && real && c < cols) {
        row::load_raw<8>(r, row + c);
        return;
    }
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = !VEC && real && c + i < cols ? row::to_f32(row[c + i]) : 0.f;
    set8(r, v);
}

// A warp takes 8 row blocks of 128 at a time (1024 columns of a row), two to a
// pass, a block for each half of the warp; the loads of all go out first.
constexpr int ROW_PASSES = 4;

template <typename T, bool VEC>
__global__ void __launch_bounds__(256)
quant_rows_kernel(const T* __restrict__ x, int64_t ldx, int64_t rows, int64_t cols, int chunks,
                  uint8_t* __restrict__ q, int64_t ldq, float* __restrict__ s) {
    const int lane = threadIdx.x & 31, half = lane >> 4;
    const int64_t n = rows * chunks;
    pdl_sync();
    for (int64_t u = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); u < n; u += (int64_t)gridDim.x * 8) {
        const int64_t r = n < (1ll << 31) ? (int64_t)((uint32_t)u / (uint32_t)chunks) : u / chunks;
        const int64_t c0 = (u - r * chunks) * (ROW_PASSES * 256) + lane * 8;
        Raw8<T> v[ROW_PASSES];
#pragma unroll
        for (int i = 0; i < ROW_PASSES; ++i) load8<T, VEC>(x + r * ldx, true, c0 + i * 256, cols, v[i]);
#pragma unroll
        for (int i = 0; i < ROW_PASSES; ++i) {
            const int64_t c = c0 + i * 256;
            float m = amax8<T>(v[i], AMAX_MIN);
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
            if (c < cols) *reinterpret_cast<uint2*>(q + r * ldq + c) = codes8<T>(v[i], inverse_of(m));
            if ((lane & 15) == 0 && c < cols) s[(c >> 7) * rows + r] = scale_of(m);
        }
    }
}

// A 128 x 128 tile a CTA of 512 threads; a thread holds 4 x 8 values (rows
// 4 (tid / 16) on, columns 8 (tid % 16) on), 16 registers of a 16-bit type, so
// that two CTAs' loads are in flight on an SM.  Row codes leave in 8-byte
// pieces; the transposed ones go through shared memory, 4 bytes a column and
// thread, exclusive-ored so that neither side's accesses share a bank, to leave
// in 16-byte pieces of whole rows.
//   MODE 0: column scales, codes transposed, and where q is given the row form
//   MODE 1: one scale, codes where q is given, transposed where qt is given
struct TileArgs {
    const void* x;
    int64_t ldx, rows, cols;
    uint8_t* q;
    int64_t ldq;
    float* s;
    uint8_t* qt;
    int64_t ldqt;
    float* st;
};
constexpr int TILE_THREADS = 512, TILE_WARPS = 16, TILE_ROWS = 4;

template <typename T, bool VEC, int MODE>
__global__ void __launch_bounds__(TILE_THREADS, 2)
quant_tile_kernel(const TileArgs a) {
    __shared__ __align__(16) uint32_t tile[128 * 32];  // [column][4-row piece ^ 2 (column / 8)]
    __shared__ float part[TILE_WARPS][128];
    __shared__ float col_inv[128];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rg = tid >> 4, cg = tid & 15;
    const int64_t r0 = (int64_t)blockIdx.y * 128, c0 = (int64_t)blockIdx.x * 128;
    const int64_t c = c0 + cg * 8;
    pdl_sync();
    Raw8<T> v[TILE_ROWS];
#pragma unroll
    for (int i = 0; i < TILE_ROWS; ++i) {
        const int64_t r = r0 + rg * TILE_ROWS + i;
        load8<T, VEC>(static_cast<const T*>(a.x) + r * a.ldx, r < a.rows, c, a.cols, v[i]);
    }
    float inv_c[8];
    if (MODE == 0) {
        float m[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) m[j] = AMAX_MIN;
#pragma unroll
        for (int i = 0; i < TILE_ROWS; ++i) {
            float t[8];
            row::widen<8>(v[i], t);
#pragma unroll
            for (int j = 0; j < 8; ++j) m[j] = fmaxf(m[j], fabsf(t[j]));
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) m[j] = fmaxf(m[j], __shfl_xor_sync(0xFFFFFFFFu, m[j], 16));
        if (lane < 16) {
            float4* to = reinterpret_cast<float4*>(&part[warp][cg * 8]);
            to[0] = make_float4(m[0], m[1], m[2], m[3]);
            to[1] = make_float4(m[4], m[5], m[6], m[7]);
        }
        __syncthreads();
        if (tid < 128) {
            float t = part[0][tid];
#pragma unroll
            for (int i = 1; i < TILE_WARPS; ++i) t = fmaxf(t, part[i][tid]);
            col_inv[tid] = inverse_of(t);
            if (c0 + tid < a.cols) a.st[(int64_t)blockIdx.y * a.cols + c0 + tid] = scale_of(t);
        }
        if (a.q) {
#pragma unroll
            for (int i = 0; i < TILE_ROWS; ++i) {
                const int64_t r = r0 + rg * TILE_ROWS + i;
                float t = amax8<T>(v[i], AMAX_MIN);
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, o));
                if (r < a.rows) {
                    if (c < a.cols) *reinterpret_cast<uint2*>(a.q + r * a.ldq + c) = codes8<T>(v[i], inverse_of(t));
                    if (cg == 0) a.s[(int64_t)blockIdx.x * a.rows + r] = scale_of(t);
                }
            }
        }
        __syncthreads();
        const float4* from = reinterpret_cast<const float4*>(&col_inv[cg * 8]);
        const float4 lo = from[0], hi = from[1];
        inv_c[0] = lo.x; inv_c[1] = lo.y; inv_c[2] = lo.z; inv_c[3] = lo.w;
        inv_c[4] = hi.x; inv_c[5] = hi.y; inv_c[6] = hi.z; inv_c[7] = hi.w;
    } else {
        float m = AMAX_MIN;
#pragma unroll
        for (int i = 0; i < TILE_ROWS; ++i) m = amax8<T>(v[i], m);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        if (lane == 0) part[0][warp] = m;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < TILE_WARPS; ++i) m = fmaxf(m, part[0][i]);
        if (tid == 0) a.s[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = scale_of(m);
        const float inv = inverse_of(m);
#pragma unroll
        for (int j = 0; j < 8; ++j) inv_c[j] = inv;
        if (a.q && c < a.cols) {
#pragma unroll
            for (int i = 0; i < TILE_ROWS; ++i) {
                const int64_t r = r0 + rg * TILE_ROWS + i;
                if (r < a.rows) *reinterpret_cast<uint2*>(a.q + r * a.ldq + c) = codes8<T>(v[i], inv);
            }
        }
    }
    if (!a.qt) return;
    float w[TILE_ROWS][8];
#pragma unroll
    for (int i = 0; i < TILE_ROWS; ++i) row::widen<8>(v[i], w[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j)
        tile[(cg * 8 + j) * 32 + (rg ^ (2 * cg))] =
            (uint32_t)e4m3x2_from_float(__fmul_rn(w[0][j], inv_c[j]), __fmul_rn(w[1][j], inv_c[j])) |
            ((uint32_t)e4m3x2_from_float(__fmul_rn(w[2][j], inv_c[j]), __fmul_rn(w[3][j], inv_c[j])) << 16);
    __syncthreads();
    // a column of the tile is 128 codes of one transposed row: 8 lanes of 16 bytes
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int col = i * 64 + (tid >> 3), g = tid & 7, x = col >> 3;
        const int64_t r = r0 + g * 16;
        uint4 q = *reinterpret_cast<const uint4*>(&tile[col * 32 + ((g ^ (x >> 1)) << 2)]);
        if (x & 1) q = make_uint4(q.z, q.w, q.x, q.y);
        if (c0 + col < a.cols && r < a.rows) *reinterpret_cast<uint4*>(a.qt + (c0 + col) * a.ldqt + r) = q;
    }
}

template <typename T>
int rows_launch(int64_t rows, int64_t cols, const T* x, int64_t ldx, uint8_t* q, int64_t ldq, float* s,
                cudaStream_t st) {
    const int chunks = (int)((cols + ROW_PASSES * 256 - 1) / (ROW_PASSES * 256));
    const int64_t ctas = (rows * chunks + 7) / 8, most = (int64_t)row::kSMs * 8;
    const unsigned grid = (unsigned)(ctas < most ? ctas : most);
    const bool vec = cols % 8 == 0 && aligned16(x) && (ldx * sizeof(T)) % 16 == 0;
    if (vec) return launch_pdl(quant_rows_kernel<T, true>, grid, 256, 0, st, x, ldx, rows, cols, chunks, q, ldq, s);
    return launch_pdl(quant_rows_kernel<T, false>, grid, 256, 0, st, x, ldx, rows, cols, chunks, q, ldq, s);
}

int quant_rows_launch(int64_t rows, int64_t cols, int dtype, const void* x, int64_t ldx, uint8_t* q, int64_t ldq,
                      float* s, cudaStream_t st) {
    if (dtype == QMOE_F32) return rows_launch(rows, cols, static_cast<const float*>(x), ldx, q, ldq, s, st);
    if (dtype == QMOE_BF16) return rows_launch(rows, cols, static_cast<const __nv_bfloat16*>(x), ldx, q, ldq, s, st);
    return rows_launch(rows, cols, static_cast<const __half*>(x), ldx, q, ldq, s, st);
}

template <int MODE, typename T>
int tile_launch(const TileArgs& a, bool vec, cudaStream_t st) {
    const dim3 grid((unsigned)((a.cols + 127) / 128), (unsigned)((a.rows + 127) / 128));
    if (vec) return launch_pdl(quant_tile_kernel<T, true, MODE>, grid, TILE_THREADS, 0, st, a);
    return launch_pdl(quant_tile_kernel<T, false, MODE>, grid, TILE_THREADS, 0, st, a);
}
template <int MODE>
int tile_run(int dtype, const TileArgs& a, cudaStream_t st) {
    const bool vec = a.cols % 8 == 0 && aligned16(a.x) && (a.ldx * row::dtype_size(dtype)) % 16 == 0;
    if (dtype == QMOE_F32) return tile_launch<MODE, float>(a, vec, st);
    if (dtype == QMOE_BF16) return tile_launch<MODE, __nv_bfloat16>(a, vec, st);
    return tile_launch<MODE, __half>(a, vec, st);
}

// Codes [rows, cols]: rows on 16-byte boundaries.
inline bool codes_ok(const uint8_t* q, int64_t ldq, int64_t cols) {
    return q && aligned16(q) && ldq >= cols && ldq % 16 == 0;
}
inline bool source_ok(int64_t rows, int64_t cols, int dtype, const void* x, int64_t ldx) {
    return rows == 0 || (x && ldx >= cols && row::type_aligned(x, row::dtype_size(dtype)));
}
inline bool fp32_ok(const float* s) { return s && row::type_aligned(s, 4); }

}  // namespace fp8
}  // namespace qmoe

using namespace qmoe;

extern "C" int qmoe_fp8_quant_rows(int64_t rows, int64_t cols, int dtype, const void* x, int64_t ldx, uint8_t* q,
                                   int64_t ldq, float* s, qmoe_stream_t stream) {
    if (rows < 0 || cols <= 0 || !row::dtype_ok(dtype) || !fp8::source_ok(rows, cols, dtype, x, ldx))
        return QMOE_ERR_ARG;
    if (rows == 0) return QMOE_OK;
    if (!fp8::codes_ok(q, ldq, cols) || !fp8::fp32_ok(s)) return QMOE_ERR_ARG;
    return fp8::quant_rows_launch(rows, cols, dtype, x, ldx, q, ldq, s, (cudaStream_t)stream);
}

extern "C" int qmoe_fp8_quant_cols(int64_t rows, int64_t cols, int dtype, const void* x, int64_t ldx, uint8_t* qt,
                                   int64_t ldqt, float* st, uint8_t* q, int64_t ldq, float* s, qmoe_stream_t stream) {
    if (rows < 0 || cols <= 0 || !row::dtype_ok(dtype) || !fp8::source_ok(rows, cols, dtype, x, ldx))
        return QMOE_ERR_ARG;
    if (rows == 0) return QMOE_OK;
    if (!fp8::codes_ok(qt, ldqt, rows) || !fp8::fp32_ok(st)) return QMOE_ERR_ARG;
    if (q && (!fp8::codes_ok(q, ldq, cols) || !fp8::fp32_ok(s))) return QMOE_ERR_ARG;
    if ((rows + 127) / 128 > 65535) return QMOE_ERR_UNSUPPORTED;
    const fp8::TileArgs a = {x, ldx, rows, cols, q, ldq, s, qt, ldqt, st};
    return fp8::tile_run<0>(dtype, a, (cudaStream_t)stream);
}

extern "C" int qmoe_fp8_quant_blocks(int64_t rows, int64_t cols, int dtype, const void* x, int64_t ldx, uint8_t* q,
                                     int64_t ldq, uint8_t* qt, int64_t ldqt, float* s, qmoe_stream_t stream) {
    if (rows < 0 || cols <= 0 || !row::dtype_ok(dtype) || !fp8::source_ok(rows, cols, dtype, x, ldx))
        return QMOE_ERR_ARG;
    if (rows == 0) return QMOE_OK;
    if ((!q && !qt) || !fp8::fp32_ok(s)) return QMOE_ERR_ARG;
    if ((q && !fp8::codes_ok(q, ldq, cols)) || (qt && !fp8::codes_ok(qt, ldqt, rows))) return QMOE_ERR_ARG;
    if ((rows + 127) / 128 > 65535) return QMOE_ERR_UNSUPPORTED;
    const fp8::TileArgs a = {x, ldx, rows, cols, q, ldq, s, qt, ldqt, nullptr};
    return fp8::tile_run<1>(dtype, a, (cudaStream_t)stream);
}
