// Products of few tokens with 4-bit weights (qmoe_w4_linear), and the layer's
// wider forms (qmoe_w4_linear for many tokens, qmoe_w4_linear_dx).
//
//   y[t][n] = sum over groups G of s[n][G] sum_{k in G} v(code[n][k]) x[t][k]
//
// Few tokens: the codes' bytes are what the product cannot do without, so they go
// straight from HBM to the tensor core's registers.  mma.sync m16n8k16 with 16
// rows of W and 8 tokens: a code becomes the 16-bit float 16 + n by two bit
// operations for two codes (n in the top mantissa bits of a float between 16 and
// 32), exactly, and the sum of a group starts from -24 sum x, so that it ends as
// the sum of (n - 8) x; E2M1 codes are shifted to a float's sign, exponent and top
// mantissa bit and multiplied by the power of two that is missing.  A group's sum
// is then scaled in fp32: nothing is rounded before the output but fp32 sums.
// The order of the reduction inside a group is free, so the codes of a 32-bit
// word are taken as they come (0 4 1 5 2 6 3 7), and x lies in shared memory in
// that order.
#include "row_ops.cuh"
#include "tc_ptx.cuh"
#include "tma_host.cuh"

namespace qmoe {
namespace w4 {

constexpr int WARPS = 8, THREADS = WARPS * 32;
constexpr int ROWS = 16;          // of W, of a CTA
constexpr int BLOCK = 256;        // values of a row in a stage (128 bytes)
constexpr int STAGE = ROWS * 128, DEPTH = 4;

struct Args {
    int T, k, E, N, K;
    int shift;  // log2 of the group
    const void* x;
    int64_t ldx;
    int x_wide;
    const void* s;
    const int32_t* ids;
    void* y;
    int64_t ldy;
    int ytype;
    int chunk;  // values of x in shared memory at once, a multiple of WARPS * BLOCK or all
    int32_t* status;
};

template <typename T> struct Num;
template <> struct Num<__half> {
    static constexpr uint32_t BASE = 0x4C004C00u;  // 16
    static constexpr int UP = 6;                   // from bit 0 to the top four mantissa bits
    static constexpr int E2M1 = 9;                 // from bits 0..2 to two exponent bits and a mantissa bit
    static __device__ __forceinline__ uint32_t rescale(uint32_t v) {  // by 2^14
        const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&v), __half2{__ushort_as_half(0x7400), __ushort_as_half(0x7400)});
        return *reinterpret_cast<const uint32_t*>(&r);
    }
    static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};
template <> struct Num<__nv_bfloat16> {
    static constexpr uint32_t BASE = 0x41804180u;  // 16
    static constexpr int UP = 3;
    static constexpr int E2M1 = 6;
    static __device__ __forceinline__ uint32_t rescale(uint32_t v) {  // by 2^126
        const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&v),
                                         __nv_bfloat162{__ushort_as_bfloat16(0x7E80), __ushort_as_bfloat16(0x7E80)});
        return *reinterpret_cast<const uint32_t*>(&r);
    }
    static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};

// Codes j and j + 4 of a word, as the two halves of a register: 16 + n, or E2M1
// values.
template <typename T, int FORMAT, int J>
__device__ __forceinline__ uint32_t pair_of(uint32_t word) {
    using M = Num<T>;
    if constexpr (FORMAT == QMOE_W4_INT4) {
        constexpr int by = M::UP - 4 * J;
        const uint32_t v = by >= 0 ? word << (by >= 0 ? by : 0) : word >> (by < 0 ? -by : 0);
        return (v & (0x000F000Fu << M::UP)) | M::BASE;
    } else {
        constexpr int by = M::E2M1 - 4 * J, sign = 12 - 4 * J;
        const uint32_t m = by >= 0 ? word << (by >= 0 ? by : 0) : word >> (by < 0 ? -by : 0);
        const uint32_t s = word << sign;
        return M::rescale((m & (0x00070007u << M::E2M1)) | (s & 0x80008000u));
    }
}

template <int FORMAT>
__device__ __forceinline__ float scale_at(const void* s, int64_t i) {
    if constexpr (FORMAT == QMOE_W4_INT4) return __half2float(static_cast<const __half*>(s)[i]);
    else return e8m0_to_float(static_cast<const uint8_t*>(s)[i]);
}

__device__ __forceinline__ void put(void* y, int type, int64_t at, float v) {
    if (type == QMOE_F32) static_cast<float*>(y)[at] = v;
    else if (type == QMOE_BF16) static_cast<__nv_bfloat16*>(y)[at] = __float2bfloat16_rn(v);
    else static_cast<__half*>(y)[at] = __float2half_rn(v);
}

// Bytes of a token's x in shared memory: rows of two neighbouring tokens fall into
// different halves of the banks.
__host__ __device__ constexpr int pitch_of(int chunk) { return chunk * 2 + 64; }

template <typename T, int FORMAT, int NT>  // NT: tiles of 8 tokens
__global__ void __launch_bounds__(THREADS) w4_few_kernel(const __grid_constant__ CUtensorMap map, const Args g) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t bars[WARPS * DEPTH];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = lane >> 2, quad = lane & 3;
    const int n0 = blockIdx.x * ROWS;
    uint8_t* const ring = smem + warp * DEPTH * STAGE;
    uint64_t* const bar = bars + warp * DEPTH;
    uint8_t* const xs = smem + WARPS * DEPTH * STAGE;
    const int tokens = g.ids ? 1 : g.T, pitch = pitch_of(g.chunk);
    float* const sums = reinterpret_cast<float*>(xs + tokens * pitch);  // [groups of 32 in a chunk][8 NT]

    pdl_wait();
    int e = 0;
    const int64_t t0 = g.ids ? blockIdx.y / g.k : 0;
    if (g.ids) {
        e = g.ids[blockIdx.y];
        if (e < 0 || e >= g.E) {
            pdl_trigger();
            if (threadIdx.x < ROWS && n0 + threadIdx.x < g.N) put(g.y, g.ytype, blockIdx.y * g.ldy + n0 + threadIdx.x, 0.f);
            return;
        }
    }
    const int blocks = (g.K + BLOCK - 1) / BLOCK;
    if (lane == 0) {
        for (int i = 0; i < DEPTH; ++i) tc::mbar_init(&bar[i], 1);
        tc::fence_barrier_init();
        for (int i = 0; i < DEPTH; ++i) {
            const int b = warp + i * WARPS;
            if (b < blocks) {
                tc::mbar_arrive_expect_tx(&bar[i], STAGE);
                tc::tma_load_3d(ring + i * STAGE, &map, &bar[i], b * (BLOCK / 2), n0, e);
            }
        }
    }
    pdl_trigger();
    const int per_row = g.K >> g.shift;
    const int64_t s_row = ((int64_t)e * g.N + n0 + row) * per_row;
    const bool there[2] = {n0 + row < g.N, n0 + row + 8 < g.N};
    // scales of groups 2 quad and 2 quad + 1 of a block, rows row and row + 8
    float sc[2][2];
    auto scales = [&](int b, float (&to)[2][2]) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int k = b * BLOCK + (2 * quad + i) * 32;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                to[h][i] = k < g.K && there[h] ? scale_at<FORMAT>(g.s, s_row + (int64_t)h * 8 * per_row + (k >> g.shift)) : 0.f;
        }
    };
    if (warp < blocks) scales(warp, sc);

    float acc[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
    bool ok = true;
    int it = 0;
    for (int c0 = 0; c0 < g.K; c0 += g.chunk) {
        // x of this chunk, zeros up to whole blocks, and the sum of each 32 values
        const int len = min(g.chunk, (g.K - c0 + BLOCK - 1) / BLOCK * BLOCK);
        if (c0) __syncthreads();
        for (int i = threadIdx.x; i < tokens * (len / 8); i += THREADS) {
            const int t = i / (len / 8), k = (i - t * (len / 8)) * 8;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (c0 + k < g.K) {
                const T* from = static_cast<const T*>(g.x) + (t0 + t) * g.ldx + c0 + k;
                if (g.x_wide) {
                    v = *reinterpret_cast<const uint4*>(from);
                } else {
                    uint32_t u[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) u[j] = reinterpret_cast<const uint16_t*>(from)[j];
                    v = make_uint4(u[0] | u[1] << 16, u[2] | u[3] << 16, u[4] | u[5] << 16, u[6] | u[7] << 16);
                }
            }
            const float2 a = row::unpack2(v.x, T{}), b = row::unpack2(v.y, T{}), c = row::unpack2(v.z, T{}), d = row::unpack2(v.w, T{});
            float sum = ((a.x + a.y) + (b.x + b.y)) + ((c.x + c.y) + (d.x + d.y));
            // len / 8 is a multiple of 32: the lanes of a warp hold one token's neighbouring values
            sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
            sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
            if (FORMAT == QMOE_W4_INT4 && (i & 3) == 0) sums[(k / 32) * (8 * NT) + t] = -24.f * sum;
            *reinterpret_cast<uint4*>(xs + t * pitch + k * 2) =
                make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632), __byte_perm(v.y, v.w, 0x5410),
                           __byte_perm(v.y, v.w, 0x7632));
        }
        __syncthreads();
        for (int b = c0 / BLOCK + warp; b < (c0 + len) / BLOCK && ok; b += WARPS, ++it) {
            const int slot = it % DEPTH;
            float next[2][2] = {};
            if (b + WARPS < blocks) scales(b + WARPS, next);
            ok = __all_sync(0xFFFFFFFFu, tc::mbar_wait(&bar[slot], it / DEPTH & 1));
            const uint8_t* st = ring + slot * STAGE + row * 128 + quad * 4;
            const uint8_t* xb = xs + (b * BLOCK - c0) * 2 + quad * 16;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t at = (j ^ (row & 7)) * 16;
                const uint32_t lo = *reinterpret_cast<const uint32_t*>(st + at);
                const uint32_t hi = *reinterpret_cast<const uint32_t*>(st + 1024 + at);
                const uint32_t a0[4] = {pair_of<T, FORMAT, 0>(lo), pair_of<T, FORMAT, 0>(hi), pair_of<T, FORMAT, 1>(lo),
                                        pair_of<T, FORMAT, 1>(hi)};
                const uint32_t a1[4] = {pair_of<T, FORMAT, 2>(lo), pair_of<T, FORMAT, 2>(hi), pair_of<T, FORMAT, 3>(lo),
                                        pair_of<T, FORMAT, 3>(hi)};
                const float f0 = __shfl_sync(0xFFFFFFFFu, sc[0][j & 1], (lane & 28) | (j >> 1));
                const float f1 = __shfl_sync(0xFFFFFFFFu, sc[1][j & 1], (lane & 28) | (j >> 1));
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const int t = min(i * 8 + row, tokens - 1);
                    const uint4 v = *reinterpret_cast<const uint4*>(xb + t * pitch + j * 64);
                    float d[4] = {0.f, 0.f, 0.f, 0.f};
                    if constexpr (FORMAT == QMOE_W4_INT4) {
                        const float2 z = *reinterpret_cast<const float2*>(sums + ((b * BLOCK - c0) / 32 + j) * (8 * NT) + i * 8 + quad * 2);
                        d[0] = d[2] = z.x;
                        d[1] = d[3] = z.y;
                    }
                    Num<T>::mma(d, a0, v.x, v.y);
                    Num<T>::mma(d, a1, v.z, v.w);
                    acc[i][0] = fmaf(f0, d[0], acc[i][0]);
                    acc[i][1] = fmaf(f0, d[1], acc[i][1]);
                    acc[i][2] = fmaf(f1, d[2], acc[i][2]);
                    acc[i][3] = fmaf(f1, d[3], acc[i][3]);
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 2; ++i) sc[h][i] = next[h][i];
            __syncwarp();
            if (lane == 0 && b + DEPTH * WARPS < blocks) {
                tc::mbar_arrive_expect_tx(&bar[slot], STAGE);
                tc::tma_load_3d(ring + slot * STAGE, &map, &bar[slot], (b + DEPTH * WARPS) * (BLOCK / 2), n0, e);
            }
        }
    }
    if (!ok && lane == 0) {
        atomicOr(g.status, QMOE_DEV_WAIT_TIMEOUT);
        // the blocks asked for and not waited for: no load outlives the CTA
        for (int i = it - 1; i < it - 1 + DEPTH; ++i)
            if (warp + i * WARPS < blocks) tc::mbar_wait(&bar[i % DEPTH], i / DEPTH & 1);
    }
    // the warps' sums, added in order
    __syncthreads();
    float* const part = reinterpret_cast<float*>(xs);
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        float* to = part + ((warp * NT + i) * 8 + quad * 2) * ROWS + row;
        to[0] = acc[i][0];
        to[ROWS] = acc[i][1];
        to[8] = acc[i][2];
        to[ROWS + 8] = acc[i][3];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < tokens * ROWS; i += THREADS) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) v += part[w * NT * 8 * ROWS + i];
        const int t = i / ROWS, n = n0 + i % ROWS;
        if (n < g.N) put(g.y, g.ytype, (g.ids ? (int64_t)blockIdx.y : t) * g.ldy + n, v);
    }
}

// W in 16 bits, [N, K], and {0, T} for the grouped product with one expert.
template <typename T, int FORMAT>
__global__ void __launch_bounds__(256) w4_widen_kernel(int64_t words, int per_row, int shift, const uint32_t* w, const void* s,
                                                       uint4* to, int32_t* offsets, int tokens) {
    pdl_wait();
    pdl_trigger();
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i == 0) {
        offsets[0] = 0;
        offsets[1] = tokens;
    }
    if (i >= words) return;
    const int64_t n = i / per_row, k = (i - n * per_row) * 8;
    const float f = scale_at<FORMAT>(s, n * ((int64_t)per_row * 8 >> shift) + (k >> shift));
    const uint32_t v = w[i];
    float d[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t c = v >> 4 * j & 15;
        d[j] = f * (FORMAT == QMOE_W4_INT4 ? (float)((int)c - 8) : e2m1_to_float(c));
    }
    row::store<8>(reinterpret_cast<T*>(to + i), d);
}

// ------------------------------------------------------------------ host side

template <typename T, int FORMAT, int NT>
static int few(const CUtensorMap& map, Args& g, int64_t pairs, cudaStream_t st) {
    const int tokens = g.ids ? 1 : g.T, all = (g.K + BLOCK - 1) / BLOCK * BLOCK;
    const int most = NT == 1 ? 4096 : 2048;
    g.chunk = all < most ? all : most;
    const int x = tokens * pitch_of(g.chunk) + g.chunk / 32 * 8 * NT * 4, part = WARPS * NT * 8 * ROWS * 4;
    const int smem = 1024 + WARPS * DEPTH * STAGE + (x > part ? x : part);
    constexpr int kMostSmem = 220 * 1024;
    const int rc = row::allow_smem<w4_few_kernel<T, FORMAT, NT>>(kMostSmem);
    if (rc != QMOE_OK) return rc;
    return launch_pdl(w4_few_kernel<T, FORMAT, NT>, dim3((unsigned)((g.N + ROWS - 1) / ROWS), (unsigned)pairs), dim3(THREADS),
                      (size_t)smem, st, map, g);
}
template <typename T, int FORMAT>
static int few_tokens(const CUtensorMap& map, Args& g, int64_t pairs, cudaStream_t st) {
    const int tokens = g.ids ? 1 : g.T;
    if (tokens <= 8) return few<T, FORMAT, 1>(map, g, pairs, st);
    if (tokens <= 16) return few<T, FORMAT, 2>(map, g, pairs, st);
    return few<T, FORMAT, 4>(map, g, pairs, st);
}

inline bool format_ok(int format, int group) {
    return (format == QMOE_W4_INT4 && (group == 32 || group == 64 || group == 128)) || (format == QMOE_W4_E2M1 && group == 32);
}
inline int log2_of(int group) { return group == 32 ? 5 : group == 64 ? 6 : 7; }
inline size_t up256(size_t n) { return (n + 255) / 256 * 256; }

template <typename T, int FORMAT>
static int widen(int64_t N, int64_t K, int group, const uint8_t* w, const void* s, uint8_t* ws, int32_t* offsets, int T_,
                 cudaStream_t st) {
    const int64_t words = N * (K / 8);
    return launch_pdl(w4_widen_kernel<T, FORMAT>, dim3((unsigned)((words + 255) / 256)), dim3(256), 0, st, words, (int)(K / 8),
                      log2_of(group), reinterpret_cast<const uint32_t*>(w), s, reinterpret_cast<uint4*>(ws), offsets, T_);
}
static int widen_any(int dtype, int format, int64_t N, int64_t K, int group, const uint8_t* w, const void* s, uint8_t* ws,
                     int32_t* offsets, int T, cudaStream_t st) {
    if (dtype == QMOE_BF16)
        return format == QMOE_W4_INT4 ? widen<__nv_bfloat16, QMOE_W4_INT4>(N, K, group, w, s, ws, offsets, T, st)
                                      : widen<__nv_bfloat16, QMOE_W4_E2M1>(N, K, group, w, s, ws, offsets, T, st);
    return format == QMOE_W4_INT4 ? widen<__half, QMOE_W4_INT4>(N, K, group, w, s, ws, offsets, T, st)
                                  : widen<__half, QMOE_W4_E2M1>(N, K, group, w, s, ws, offsets, T, st);
}

constexpr int64_t kMost = 1ll << 30;

static int check(int64_t T, int64_t N, int64_t K, int format, int group, int dtype, int out_dtype, int64_t ldo, int64_t cols) {
    if (T < 0 || N <= 0 || K <= 0 || !format_ok(format, group) || K % group || (dtype != QMOE_BF16 && dtype != QMOE_F16) ||
        (out_dtype != dtype && out_dtype != QMOE_F32) || ldo < cols)
        return QMOE_ERR_ARG;
    if (T > kMost || N > kMost || K > kMost || N * (K / 8) > (kMost << 6)) return QMOE_ERR_UNSUPPORTED;
    return QMOE_OK;
}
static bool arrays_ok(const void* x, int64_t ldx, int64_t cols, const uint8_t* w, const void* s, int format, const void* y,
                      int y_dtype, const int32_t* status) {
    return x && ldx >= cols && ldx < (1ll << 38) && row::type_aligned(x, 2) && w && aligned16(w) && s &&
           (format != QMOE_W4_INT4 || row::type_aligned(s, 2)) && y && row::type_aligned(y, row::dtype_size(y_dtype)) &&
           status && row::type_aligned(status, 4);
}

}  // namespace w4
}  // namespace qmoe

using namespace qmoe;

extern "C" size_t qmoe_w4_workspace_bytes(int64_t T, int64_t N, int64_t K, int dx) {
    if (T <= 0 || N <= 0 || K <= 0 || (!dx && T <= QMOE_W4_FEW)) return 0;
    return w4::up256((size_t)N * K * 2) + 256 + qmoe_expert_copy_bytes(T, dx ? N : K) +
           qmoe_expert_workspace_bytes(T, 1, N, K, dx ? 1 : 0, 0);
}

extern "C" int qmoe_w4_linear(int64_t T, int k, int E, int64_t N, int64_t K, int format, int group, int dtype, const void* x,
                              int64_t ldx, const uint8_t* w, const void* s, const int32_t* ids, void* y, int y_dtype,
                              int64_t ldy, int32_t* dev_status, void* ws, size_t ws_bytes, qmoe_stream_t stream) {
    int rc = w4::check(T, N, K, format, group, dtype, y_dtype, ldy, N);
    if (rc != QMOE_OK) return rc;
    if (k <= 0 || E <= 0 || (!ids && (k != 1 || E != 1))) return QMOE_ERR_ARG;
    if (T == 0) return QMOE_OK;
    if (!w4::arrays_ok(x, ldx, K, w, s, format, y, y_dtype, dev_status) || (ids && !row::type_aligned(ids, 4))) return QMOE_ERR_ARG;
    if (ids && (T * k > 65535 || (int64_t)E * N > w4::kMost)) return QMOE_ERR_UNSUPPORTED;
    cudaStream_t st = (cudaStream_t)stream;
    if (!ids && T > QMOE_W4_FEW) {
        if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < qmoe_w4_workspace_bytes(T, N, K, 0)) return QMOE_ERR_ARG;
        uint8_t* at = static_cast<uint8_t*>(ws);
        const size_t wide = w4::up256((size_t)N * K * 2);
        int32_t* offsets = reinterpret_cast<int32_t*>(at + wide);
        rc = w4::widen_any(dtype, format, N, K, group, w, s, at, offsets, (int)T, st);
        if (rc != QMOE_OK) return rc;
        return qmoe_expert_linear(T, 1, N, K, dtype, x, ldx, T, nullptr, 0, at, K, N * K, offsets, y, y_dtype, ldy, dev_status,
                                  at + wide + 256, ws_bytes - wide - 256, stream);
    }
    EncodeTiledFn enc = encode_tiled_fn();
    if (!enc) return QMOE_ERR_CUDA;
    CUtensorMap map;
    const cuuint64_t dim[3] = {(cuuint64_t)K / 2, (cuuint64_t)N, (cuuint64_t)E};
    const cuuint64_t stride[2] = {(cuuint64_t)K / 2, (cuuint64_t)(K / 2 * N)};
    const cuuint32_t box[3] = {128, w4::ROWS, 1};
    const cuuint32_t one[3] = {1, 1, 1};
    if (enc(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(w), dim, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return QMOE_ERR_UNSUPPORTED;
    w4::Args g = {(int)T, k, E, (int)N, (int)K, w4::log2_of(group), x, ldx, aligned16(x) && (ldx % 8 == 0 || T == 1), s, ids, y, ldy,
                  y_dtype, 0, dev_status};
    const int64_t pairs = ids ? T * k : 1;
    if (dtype == QMOE_BF16)
        return format == QMOE_W4_INT4 ? w4::few_tokens<__nv_bfloat16, QMOE_W4_INT4>(map, g, pairs, st)
                                      : w4::few_tokens<__nv_bfloat16, QMOE_W4_E2M1>(map, g, pairs, st);
    return format == QMOE_W4_INT4 ? w4::few_tokens<__half, QMOE_W4_INT4>(map, g, pairs, st)
                                  : w4::few_tokens<__half, QMOE_W4_E2M1>(map, g, pairs, st);
}

extern "C" int qmoe_w4_linear_dx(int64_t T, int64_t N, int64_t K, int format, int group, int dtype, const void* dy, int64_t lddy,
                                 const uint8_t* w, const void* s, void* dx, int dx_dtype, int64_t lddx, int32_t* dev_status,
                                 void* ws, size_t ws_bytes, qmoe_stream_t stream) {
    int rc = w4::check(T, N, K, format, group, dtype, dx_dtype, lddx, K);
    if (rc != QMOE_OK) return rc;
    if (T == 0) return QMOE_OK;
    if (!w4::arrays_ok(dy, lddy, N, w, s, format, dx, dx_dtype, dev_status) || !ws || (reinterpret_cast<uintptr_t>(ws) & 255u) ||
        ws_bytes < qmoe_w4_workspace_bytes(T, N, K, 1))
        return QMOE_ERR_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    uint8_t* at = static_cast<uint8_t*>(ws);
    const size_t wide = w4::up256((size_t)N * K * 2);
    int32_t* offsets = reinterpret_cast<int32_t*>(at + wide);
    rc = w4::widen_any(dtype, format, N, K, group, w, s, at, offsets, (int)T, st);
    if (rc != QMOE_OK) return rc;
    return qmoe_expert_linear_dx(T, 1, N, K, dtype, dy, lddy, at, K, N * K, offsets, dx, dx_dtype, lddx, dev_status,
                                 at + wide + 256, ws_bytes - wide - 256, stream);
}
