// Norms before and after a block, forward (qmoe_norm_pre, qmoe_norm_post).
//
//   z = y rstd(y) w,  out = r + alpha g z,  n = out rstd(out) w_next,
//   rstd(v) = 1 / sqrt(mean v^2 + eps)
//
// One pass: a row lives in the registers of the threads that share it, so r
// and y are read once and out and n written once (8 bytes a column in 16-bit
// types), and the second sum runs on values already at hand.  The bound is
// HBM; what there is besides are the two sums of a row, each a latency of two
// shuffles' trees and a barrier, which the rows on their way hide.
#include "norm_block.cuh"

namespace qmoe {
namespace norm {

struct FwdArgs {
    int64_t rows;
    int cols, stages, stage_bytes;
    Source r, y, full_gate;  // r: the stream (norm_pre: x)
    const float* w;
    int gate_mode;
    const float* gate;
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
__global__ void __launch_bounds__(512, 1)
norm_fwd_kernel(const FwdArgs a) {
    constexpr int E = NV * VEC;
    constexpr bool KEEP = E <= 16;  // the weights stay in registers from row to row
    __shared__ __align__(16) float sums[2][2][16];
    __shared__ uint64_t full[MAX_ROWS][MAX_STAGES];
    extern __shared__ __align__(128) uint8_t dynamic[];
    const int tx = threadIdx.x, cols = a.cols;
    const int64_t stride = (int64_t)gridDim.x * blockDim.y;
    const float inv_cols = 1.f / (float)cols;
    int flip = 0;

    int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    Ring<VEC> ring = {full[threadIdx.y], dynamic + (int64_t)threadIdx.y * a.stages * a.stage_bytes, a.stages,
                      a.stage_bytes, a.rows, stride};
    int matrices = 0;
    ring.feed.take(a.r, sizeof(RT), matrices, tx, row, stride, cols);
    if (POST) ring.feed.take(a.y, sizeof(YT), matrices, tx, row, stride, cols);
    if (POST) ring.feed.take(a.full_gate, sizeof(YT), matrices, tx, row, stride, cols);
    if (tx == 0)
        for (int i = 0; i < MAX_STAGES; ++i) tc::mbar_init(&full[threadIdx.y][i], matrices);
    for (int i = tx; i < 64; i += blockDim.x) (&sums[0][0][0])[i] = 0.f;
    tc::fence_barrier_init();
    __syncthreads();
    pdl_sync();
    ring.begin(row);
    // what a column of y and of out is multiplied by: w and a column gate in one
    float wg[E], wn[E];
    auto col_factors = [&] {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * blockDim.x + tx) * VEC;
            if (c >= cols) continue;
#pragma unroll
            for (int i = 0; i < VEC; ++i) wg[v * VEC + i] = 1.f;
            if (a.w) row::load<VEC>(a.w + c, &wg[v * VEC]);
            if (a.gate_mode == QMOE_GATE_COL) {
                float g[VEC];
                row::load<VEC>(a.gate + c, g);
#pragma unroll
                for (int i = 0; i < VEC; ++i) wg[v * VEC + i] *= g[i];
            }
        }
    };
    auto next_weights = [&] {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * blockDim.x + tx) * VEC;
            if (c < cols && a.w_next) row::load<VEC>(a.w_next + c, &wn[v * VEC]);
        }
    };
    if (KEEP) {
        if (POST) col_factors();
        next_weights();
    }
    // a row's own scalars are asked for one row early
    const bool row_gate = POST && a.gate_mode == QMOE_GATE_ROW;
    float g_next = row_gate && row < a.rows ? a.gate[row] : 1.f;
    for (; row < a.rows; row += stride) {
        const float g_row = g_next;
        if (row_gate && row + stride < a.rows) g_next = a.gate[row + stride];
        const uint8_t* const from = ring.wait();
        bool met = false;
        float o[E];
        read_row<VEC, NV, true, RT>(a.r, from, row, cols, o);
        if (ring.lost) o[0] = NAN;
        if (POST) {
            float y[E];
            read_row<VEC, NV, true, YT>(a.y, from, row, cols, y);
            if (!KEEP) col_factors();
            float scale = a.alpha * g_row;
            if (a.w) {
                float s = 0.f;
#pragma unroll
                for (int i = 0; i < E; ++i) s = fmaf(y[i], y[i], s);
                const float rstd = rsqrtf(row::row_sum(s, sums[flip]) * inv_cols + a.eps);
                flip ^= 1;
                met = true;
                ring.refill(row);
                if (tx == 0 && a.rstd) a.rstd[row] = rstd;
                scale *= rstd;
            }
            if (a.gate_mode == QMOE_GATE_FULL) {
                float g[E];
                read_row<VEC, NV, true, YT>(a.full_gate, from, row, cols, g);
#pragma unroll
                for (int i = 0; i < E; ++i) y[i] *= g[i];
            }
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int c = (v * blockDim.x + tx) * VEC;
                if (c >= cols) continue;
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const int e = v * VEC + i;
                    o[e] = fmaf(y[e] * scale, wg[e], o[e]);
                }
                row::store<VEC>(static_cast<RT*>(a.out) + row * a.ldo + c, &o[v * VEC]);
            }
        }
        if (a.w_next) {
            if (!KEEP) next_weights();
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < E; ++i) s = fmaf(o[i], o[i], s);
            const float rstd = rsqrtf(row::row_sum(s, sums[flip]) * inv_cols + a.eps);
            flip ^= 1;
            if (!met) ring.refill(row);
            met = true;
            if (tx == 0 && a.rstd_next) a.rstd_next[row] = rstd;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int c = (v * blockDim.x + tx) * VEC;
                if (c >= cols) continue;
                float n[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) n[i] = o[v * VEC + i] * rstd * wn[v * VEC + i];
                row::store<VEC>(static_cast<YT*>(a.n) + row * a.ldn + c, n);
            }
        }
        if (!met || blockDim.x == 32) {
            row_barrier();
            if (!met) ring.refill(row);
        }
        if (a.stages == 1) {
            row_barrier();
            ring.post(row + stride, 0);
        }
        ring.next();
    }
}

template <auto Kernel>
inline int start(const Shape& s, FwdArgs& a, int row_bytes, cudaStream_t st) {
    const int threads = s.threads * s.rows_per_cta;
    const int64_t ctas = (a.rows + s.rows_per_cta - 1) / s.rows_per_cta;
    // one wave of 512 threads an SM; fewer CTAs where that leaves each two stages
    int per_sm = 512 / threads;
    a.stage_bytes = row_bytes;
    while (per_sm > 1 && stages_of((int64_t)row_bytes * s.rows_per_cta, 0, per_sm) < 2) --per_sm;
    a.stages = stages_of((int64_t)row_bytes * s.rows_per_cta, 0, per_sm);
    if (!a.stages) return QMOE_ERR_UNSUPPORTED;
    const int64_t fit = (int64_t)row::kSMs * per_sm;
    const size_t smem = (size_t)a.stages * row_bytes * s.rows_per_cta;
    if (smem > 47 * 1024) {
        const int rc = row::allow_smem<Kernel>(225 * 1024);
        if (rc != QMOE_OK) return rc;
    }
    return launch_pdl(Kernel, dim3((unsigned)(ctas < fit ? ctas : fit)), dim3(s.threads, s.rows_per_cta), smem, st, a);
}

template <bool POST>
struct Fwd {
    template <typename RT, typename YT>
    struct Go {
        static int go(FwdArgs& a, bool vec, cudaStream_t st) {
            constexpr int W = wide_vec<RT, YT>();
            const Shape s = shape_of(a.cols, vec ? W : 1, 16);
            const int rb = stage_bytes(a.cols, sizeof(RT)), yb = stage_bytes(a.cols, sizeof(YT));
            a.y.off = rb;
            a.full_gate.off = rb + yb;
            const int bytes = rb + (POST ? yb : 0) + (a.full_gate.p ? yb : 0);
            if (vec) {
                if (s.values() == 16) return start<norm_fwd_kernel<RT, YT, 16 / W, W, POST>>(s, a, bytes, st);
                return start<norm_fwd_kernel<RT, YT, 32 / W, W, POST>>(s, a, bytes, st);
            }
            if (s.values() == 16) return start<norm_fwd_kernel<RT, YT, 16, 1, POST>>(s, a, bytes, st);
            return start<norm_fwd_kernel<RT, YT, 32, 1, POST>>(s, a, bytes, st);
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
    a.r = {x, ldx, 0};
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
    a.r = {r, ldr, 0};
    a.y = {y, ldy, 0};
    a.w = w;
    a.gate_mode = gate_mode;
    if (gate_mode == QMOE_GATE_FULL) a.full_gate = {gate, ldg, 0};
    else a.gate = static_cast<const float*>(gate);
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
