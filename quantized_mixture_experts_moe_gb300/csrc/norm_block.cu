// Norms before and after a block, forward (qmoe_norm_pre, qmoe_norm_post).
//
//   z = y rstd(y) w,  out = r + alpha g z,  n = out rstd(out) w_next,
//   rstd(v) = 1 / sqrt(mean v^2 + eps)
//
// One pass: a row lives in the registers of the threads that share it, so r
// and y are read once and out and n written once (8 bytes a column in 16-bit
// types), and the second sum runs on values already at hand.  The bound is
// HBM; what there is besides are the two sums of a row, each a latency of two
// shuffles' trees and a barrier.  A CTA therefore asks for its next row before
// it sums the present one.
#include "norm_block.cuh"

namespace qmoe {
namespace norm {

struct FwdArgs {
    int64_t rows;
    int cols;
    const void* r;  // the stream (norm_pre: x)
    int64_t ldr;
    const void* y;
    int64_t ldy;
    const float* w;
    int gate_mode;
    const void* gate;
    int64_t ldg;
    float alpha, eps;
    const float* w_next;
    void* out;
    int64_t ldo;
    void* n;
    int64_t ldn;
    float *rstd, *rstd_next;
};

// POST: y, its norm and gate; without it the kernel is norm_pre (out = r, not written).
template <typename RT, typename YT, int NV, int VEC, bool POST>
__global__ void __launch_bounds__(NV * VEC > 8 ? 512 : 1024)
norm_fwd_kernel(const FwdArgs a) {
    constexpr int E = NV * VEC;
    constexpr bool KEEP = E <= 8;  // the weights stay in registers from row to row
    __shared__ float2 sums[2][32];
    const int tx = threadIdx.x, step = blockDim.x * VEC, cols = a.cols;
    const int64_t stride = (int64_t)gridDim.x * blockDim.y;
    const float inv_cols = 1.f / (float)cols;
    int flip = 0;

    float w[KEEP ? E : 1], wn[KEEP ? E : 1], gc[KEEP ? E : 1];
    row::Raw<RT, VEC> rr[NV];
    row::Raw<YT, VEC> ry[NV];
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = v * step + tx * VEC;
            if (c >= cols) continue;
            if (POST) row::load_raw<VEC>(ry[v], static_cast<const YT*>(a.y) + row * a.ldy + c);
            row::load_raw<VEC>(rr[v], static_cast<const RT*>(a.r) + row * a.ldr + c);
        }
    };
    int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    pdl_sync();
    if (row < a.rows) fetch(row);
    if (KEEP) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = v * step + tx * VEC;
            if (c >= cols) continue;
            if (POST && a.w) row::load<VEC>(a.w + c, &w[v * VEC]);
            if (a.w_next) row::load<VEC>(a.w_next + c, &wn[v * VEC]);
            if (POST && a.gate_mode == QMOE_GATE_COL)
                row::load<VEC>(static_cast<const float*>(a.gate) + c, &gc[v * VEC]);
        }
    }
    for (; row < a.rows; row += stride) {
        float o[E], y[POST ? E : 1];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if (v * step + tx * VEC < cols) {
                row::widen<VEC>(rr[v], &o[v * VEC]);
                if (POST) row::widen<VEC>(ry[v], &y[v * VEC]);
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    o[v * VEC + i] = 0.f;
                    if (POST) y[v * VEC + i] = 0.f;
                }
            }
        }
        if (row + stride < a.rows) fetch(row + stride);
        if (POST) {
            float scale = a.alpha;
            if (a.w) {
                float s = 0.f;
#pragma unroll
                for (int i = 0; i < E; ++i) s = fmaf(y[i], y[i], s);
                const float rstd = rsqrtf(row::row_sum(s, 0.f, sums[flip]).x * inv_cols + a.eps);
                flip ^= 1;
                if (tx == 0 && a.rstd) a.rstd[row] = rstd;
                scale *= rstd;
            }
            if (a.gate_mode == QMOE_GATE_ROW) scale *= static_cast<const float*>(a.gate)[row];
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int c = v * step + tx * VEC;
                if (c >= cols) continue;
                float g[VEC];
                if (a.gate_mode == QMOE_GATE_FULL)
                    row::load<VEC>(static_cast<const YT*>(a.gate) + row * a.ldg + c, g);
                else if (!KEEP && a.gate_mode == QMOE_GATE_COL)
                    row::load<VEC>(static_cast<const float*>(a.gate) + c, g);
                float wv[VEC];
                if (!KEEP && a.w) row::load<VEC>(a.w + c, wv);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const int e = v * VEC + i;
                    float z = y[e] * scale;
                    if (a.w) z *= KEEP ? w[e] : wv[i];
                    if (a.gate_mode == QMOE_GATE_FULL) z *= g[i];
                    else if (a.gate_mode == QMOE_GATE_COL) z *= KEEP ? gc[e] : g[i];
                    o[e] += z;
                }
                row::store<VEC>(static_cast<RT*>(a.out) + row * a.ldo + c, &o[v * VEC]);
            }
        }
        if (a.w_next) {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < E; ++i) s = fmaf(o[i], o[i], s);
            const float rstd = rsqrtf(row::row_sum(s, 0.f, sums[flip]).x * inv_cols + a.eps);
            flip ^= 1;
            if (tx == 0 && a.rstd_next) a.rstd_next[row] = rstd;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int c = v * step + tx * VEC;
                if (c >= cols) continue;
                float wv[VEC];
                if (!KEEP) row::load<VEC>(a.w_next + c, wv);
                float n[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) n[i] = o[v * VEC + i] * rstd * (KEEP ? wn[v * VEC + i] : wv[i]);
                row::store<VEC>(static_cast<YT*>(a.n) + row * a.ldn + c, n);
            }
        }
    }
}

template <bool POST>
struct Fwd {
    template <typename RT, typename YT>
    struct Go {
        static int go(const FwdArgs& a, bool vec, cudaStream_t st) {
            const Shape s = shape_of(a.cols, vec, 512);
            const dim3 block(s.threads, s.rows_per_cta);
            const int64_t ctas = (a.rows + s.rows_per_cta - 1) / s.rows_per_cta;
            const int64_t fit = (int64_t)row::kSMs * (1024 / (s.threads * s.rows_per_cta));
            const dim3 grid((unsigned)(ctas < fit ? ctas : fit));
            if (s.vec == 8) {
                if (s.nv == 1) return launch_pdl(norm_fwd_kernel<RT, YT, 1, 8, POST>, grid, block, 0, st, a);
                if (s.nv == 2) return launch_pdl(norm_fwd_kernel<RT, YT, 2, 8, POST>, grid, block, 0, st, a);
                return launch_pdl(norm_fwd_kernel<RT, YT, 4, 8, POST>, grid, block, 0, st, a);
            }
            if (s.nv == 4) return launch_pdl(norm_fwd_kernel<RT, YT, 4, 1, POST>, grid, block, 0, st, a);
            if (s.nv == 16) return launch_pdl(norm_fwd_kernel<RT, YT, 16, 1, POST>, grid, block, 0, st, a);
            return launch_pdl(norm_fwd_kernel<RT, YT, 32, 1, POST>, grid, block, 0, st, a);
        }
    };
};
template <typename RT, typename YT> using PreGo = Fwd<false>::Go<RT, YT>;
template <typename RT, typename YT> using PostGo = Fwd<true>::Go<RT, YT>;

}  // namespace norm
}  // namespace qmoe

using namespace qmoe;

extern "C" int qmoe_norm_pre(int64_t rows, int64_t cols, int stream_dtype, int block_dtype, const void* x, int64_t ldx,
                             const float* w, float eps, void* n, int64_t ldn, float* rstd, qmoe_stream_t stream) {
    if (rows < 0 || cols <= 0 || !norm::types_ok(stream_dtype, block_dtype) || !(eps >= 0.f)) return QMOE_ERR_ARG;
    if (rows == 0) return QMOE_OK;
    if (!x || !w || !n || ldx < cols || ldn < cols) return QMOE_ERR_ARG;
    const int rs = row::dtype_size(stream_dtype), bs = row::dtype_size(block_dtype);
    if (!row::type_aligned(x, rs) || !row::type_aligned(n, bs) || !row::type_aligned(w, 4) ||
        !row::type_aligned(rstd, 4))
        return QMOE_ERR_ARG;
    if (cols > norm::MAX_COLS) return QMOE_ERR_UNSUPPORTED;
    norm::FwdArgs a = {};
    a.rows = rows;
    a.cols = (int)cols;
    a.r = x;
    a.ldr = ldx;
    a.w_next = w;
    a.eps = eps;
    a.n = n;
    a.ldn = ldn;
    a.rstd_next = rstd;
    const bool vec = cols % 8 == 0 && norm::row_aligned(x, ldx, rs) && norm::row_aligned(n, ldn, bs) && aligned16(w);
    return norm::by_types<norm::PreGo>(stream_dtype, block_dtype, a, vec, (cudaStream_t)stream);
}

extern "C" int qmoe_norm_post(int64_t rows, int64_t cols, int stream_dtype, int block_dtype, const void* r,
                              int64_t ldr, const void* y, int64_t ldy, const float* w, int gate_mode, const void* gate,
                              int64_t ldg, float alpha, const float* w_next, float eps, void* out, int64_t ldo,
                              void* n, int64_t ldn, float* rstd, float* rstd_next, qmoe_stream_t stream) {
    if (rows < 0 || cols <= 0 || !norm::types_ok(stream_dtype, block_dtype) || !(eps >= 0.f) ||
        !norm::gate_mode_ok(gate_mode))
        return QMOE_ERR_ARG;
    if (rows == 0) return QMOE_OK;
    if (!r || !y || !out || ldr < cols || ldy < cols || ldo < cols) return QMOE_ERR_ARG;
    if (gate_mode != QMOE_GATE_NONE && !gate) return QMOE_ERR_ARG;
    if (gate_mode == QMOE_GATE_FULL && ldg < cols) return QMOE_ERR_ARG;
    if (w_next && (!n || ldn < cols)) return QMOE_ERR_ARG;
    const int rs = row::dtype_size(stream_dtype), bs = row::dtype_size(block_dtype);
    if (!row::type_aligned(r, rs) || !row::type_aligned(out, rs) || !row::type_aligned(y, bs) ||
        (w_next && !row::type_aligned(n, bs)) || !row::type_aligned(w, 4) || !row::type_aligned(w_next, 4) ||
        (gate_mode != QMOE_GATE_NONE && !row::type_aligned(gate, gate_mode == QMOE_GATE_FULL ? bs : 4)) ||
        !row::type_aligned(rstd, 4) || !row::type_aligned(rstd_next, 4))
        return QMOE_ERR_ARG;
    if (cols > norm::MAX_COLS) return QMOE_ERR_UNSUPPORTED;
    norm::FwdArgs a = {};
    a.rows = rows;
    a.cols = (int)cols;
    a.r = r;
    a.ldr = ldr;
    a.y = y;
    a.ldy = ldy;
    a.w = w;
    a.gate_mode = gate_mode;
    a.gate = gate;
    a.ldg = ldg;
    a.alpha = alpha;
    a.eps = eps;
    a.w_next = w_next;
    a.out = out;
    a.ldo = ldo;
    a.n = n;
    a.ldn = ldn;
    a.rstd = w ? rstd : nullptr;
    a.rstd_next = rstd_next;
    bool vec = cols % 8 == 0 && norm::row_aligned(r, ldr, rs) && norm::row_aligned(y, ldy, bs) &&
               norm::row_aligned(out, ldo, rs) && aligned16(w) && aligned16(w_next);
    if (w_next) vec = vec && norm::row_aligned(n, ldn, bs);
    if (gate_mode == QMOE_GATE_FULL) vec = vec && norm::row_aligned(gate, ldg, bs);
    if (gate_mode == QMOE_GATE_COL) vec = vec && aligned16(gate);
    return norm::by_types<norm::PostGo>(stream_dtype, block_dtype, a, vec, (cudaStream_t)stream);
}
