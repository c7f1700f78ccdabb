// Arguments and launch shapes shared by the forward and the backward kernels
// of the block norms (norm_block.cu, norm_block_bwd.cu).
#pragma once

#include "row_ops.cuh"

namespace qmoe {
namespace norm {

constexpr int64_t MAX_COLS = 16384;

inline bool gate_mode_ok(int m) { return m >= QMOE_GATE_NONE && m <= QMOE_GATE_FULL; }

// Rows of 16-byte accesses: an aligned base and row stride.
inline bool row_aligned(const void* p, int64_t ld, int size) { return aligned16(p) && (ld * size) % 16 == 0; }

// How a row is cut: nv vectors of vec columns in each of `threads` threads;
// rows of 32 threads go four to a CTA.
struct Shape {
    int vec, nv, threads, rows_per_cta;
};

// 8 columns a thread up to `most` threads, then 16 and 32: the fewer values a
// thread holds, the more rows' loads are in flight at once, and a single row
// is spread widest.  Without 16-byte rows 4 single columns a thread, then 16
// and 32 (kernels of up to 8 values a thread run up to 1024 threads, the
// others 512, so that their rows stay in registers).
inline Shape shape_of(int64_t cols, bool vec, int most) {
    Shape s;
    s.vec = vec ? 8 : 1;
    const int64_t n = vec ? cols / 8 : cols;
    const int nv[3] = {vec ? 1 : 4, vec ? 2 : 16, vec ? 4 : 32};
    const int limit[3] = {vec ? most : 1024, 512, 512};
    for (int i = 0; i < 3; ++i) {
        s.nv = nv[i];
        s.threads = (int)(((n + s.nv - 1) / s.nv + 31) / 32 * 32);
        if (s.threads <= limit[i]) break;
    }
    s.rows_per_cta = s.threads == 32 ? 4 : 1;
    return s;
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
