// Arguments and launch shapes shared by the forward and the backward kernels
// of the block norms (norm_block.cu, norm_block_bwd.cu).
#pragma once

#include "row_ops.cuh"
#include "tc_ptx.cuh"

namespace qmoe {
namespace norm {

constexpr int64_t MAX_COLS = 16384;

inline bool gate_mode_ok(int m) { return m >= QMOE_GATE_NONE && m <= QMOE_GATE_FULL; }

// Rows of 16-byte accesses: an aligned base and row stride.
inline bool row_aligned(const void* p, int64_t ld, int size) { return aligned16(p) && (ld * size) % 16 == 0; }

// How a row is cut: nv vectors of vec columns in each of `threads` threads, 8,
// 16 or 32 values each (the fewer a thread holds, the more threads share a
// row's loads and a single row is spread widest), at most 512 threads; rows of
// 32 threads go four to a CTA.
struct Shape {
    int vec, nv, threads, rows_per_cta;
    int values() const { return vec * nv; }
};

inline Shape shape_of(int64_t cols, bool vec) {
    Shape s;
    s.vec = vec ? 8 : 1;
    for (int values = 8;; values *= 2) {
        s.nv = values / s.vec;
        const int64_t per = (cols + values - 1) / values;
        s.threads = (int)((per + 31) / 32 * 32);
        if (s.threads <= 512 || values == 32) break;
    }
    s.rows_per_cta = s.threads == 32 ? 4 : 1;
    return s;
}

// ------------------------------------------------------------------ rows on their way
//
// A CTA's next rows are copied into a ring of shared memory stages with
// cp.async while it works on the present one: HBM wants some 40 KB in flight
// for each SM, more than the registers of the threads that share a row can
// hold beside their work.  Rows of 16-byte accesses (VEC = 8): a thread copies
// what it reads itself, so no barrier is needed.  Other rows: the threads copy
// the 16-byte granules that the row lies in, in step with their addresses,
// and meet at a barrier; a granule reaches past the row, but never past the
// first and the last value of the matrix (there its values are copied one by
// one).

// One matrix that a kernel reads: rows of `cols` values, at `off` in a stage.
struct Source {
    const void* p;  // null: not given
    int64_t ld;
    int off;
};

constexpr int MAX_STAGES = 6;

inline int stage_bytes(int64_t cols, int size) { return (int)((cols * size + 15) / 16 * 16 + 16); }

// Stages that fit in a CTA's share of an SM's shared memory.
inline int stages_of(int64_t bytes_per_stage, int64_t other_bytes, int ctas_per_sm) {
    const int64_t n = (226 * 1024 / ctas_per_sm - 2048 - other_bytes) / bytes_per_stage;
    return n > MAX_STAGES ? MAX_STAGES : n > 0 ? (int)n : 0;
}

template <int VEC, int NV, typename T>
__device__ __forceinline__ void copy_row(const Source& s, uint8_t* stage, int64_t row, int64_t rows, int cols) {
    if (!s.p) return;
    const T* src = static_cast<const T*>(s.p) + row * s.ld;
    uint8_t* dst = stage + s.off;
    if constexpr (VEC == 8) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * blockDim.x + threadIdx.x) * 8;
            if (c >= cols) continue;
#pragma unroll
            for (int i = 0; i < (int)sizeof(T) / 2; ++i)
                tc::cp_async_16(dst + c * sizeof(T) + i * 16, reinterpret_cast<const uint8_t*>(src + c) + i * 16);
        }
    } else {
        const uintptr_t g0 = reinterpret_cast<uintptr_t>(src), g1 = g0 + (uintptr_t)cols * sizeof(T);
        const uintptr_t lo = reinterpret_cast<uintptr_t>(s.p);
        const uintptr_t hi = lo + ((uintptr_t)(rows - 1) * s.ld + cols) * sizeof(T);
        const uintptr_t base = g0 & ~uintptr_t(15);
        for (uintptr_t a = base + threadIdx.x * 16; a < g1; a += blockDim.x * 16) {
            if (a >= lo && a + 16 <= hi) {
                tc::cp_async_16(dst + (a - base), reinterpret_cast<const void*>(a));
            } else {
                for (uintptr_t b = a > g0 ? a : g0; b < a + 16 && b < g1; b += sizeof(T))
                    *reinterpret_cast<T*>(dst + (b - base)) = *reinterpret_cast<const T*>(b);
            }
        }
    }
}

// This thread's values of a row, widened; zeros past the row's end.  RING: from
// a stage; else straight from the matrix.
template <int VEC, int NV, bool RING, typename T>
__device__ __forceinline__ void read_row(const Source& s, const uint8_t* stage, int64_t row, int cols, float* v) {
    const T* src = static_cast<const T*>(s.p) + row * s.ld;
    if (RING) src = reinterpret_cast<const T*>(stage + s.off + (VEC == 1 ? reinterpret_cast<uintptr_t>(src) & 15 : 0));
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * blockDim.x + threadIdx.x) * VEC;
        if (c < cols) {
            row::load<VEC>(src + c, &v[i * VEC]);
        } else {
#pragma unroll
            for (int j = 0; j < VEC; ++j) v[i * VEC + j] = 0.f;
        }
    }
}

// The threads of a row meet.
__device__ __forceinline__ void row_barrier() {
    if (blockDim.x == 32) __syncwarp();
    else __syncthreads();
}

// Waits for the present row, in stage `stage`, and sends for the row that is
// stages - 1 further on, into the stage that was read last time.  fetch(ahead,
// stage) commits one group.  With a single stage the row is fetched here.
template <int VEC, typename Fetch>
__device__ __forceinline__ void next_row(int stages, int stage, Fetch&& fetch) {
    if (stages > 1) {
        tc::cp_async_wait_dyn(stages - 2);
        if (VEC == 1) row_barrier();
        fetch(stages - 1, stage == 0 ? stages - 1 : stage - 1);
    } else {
        if (VEC == 1) row_barrier();
        fetch(0, 0);
        tc::cp_async_wait<0>();
        if (VEC == 1) row_barrier();
    }
}

// (stream type, block type): the same type twice, or a 16-bit block beside an
// fp32 stream.
template <template <typename, typename> class F, typename... A>
inline int by_types(int rt, int yt, A&&... a) {
    if (rt == QMOE_F32 && yt == QMOE_F32) return F<float, float>::go(a...);
    if (rt == QMOE_F32 && yt == QMOE_BF16) return F<float, __nv_bfloat16>::go(a...);
    if (rt == QMOE_F32 && yt == QMOE_F16) return F<float, __half>::go(a...);
    if (rt == QMOE_BF16 && yt == QMOE_BF16) return F<__nv_bfloat16, __nv_bfloat16>::go(a...);
    if (rt == QMOE_F16 && yt == QMOE_F16) return F<__half, __half>::go(a...);
    return QMOE_ERR_ARG;
}

inline bool types_ok(int rt, int yt) {
    return row::dtype_ok(rt) && row::dtype_ok(yt) && (rt == yt || rt == QMOE_F32);
}

}  // namespace norm
}  // namespace qmoe
