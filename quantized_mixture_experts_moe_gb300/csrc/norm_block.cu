// Norms before and after a block, forward (qmoe_norm_pre, qmoe_norm_post).
//
//   z = y rstd(y) w,  out = r + alpha g z,  n = out rstd(out) w_next,
//   rstd(v) = 1 / sqrt(mean v^2 + eps)
//
// One pass: a row lives in the registers of the threads that share it, so r
// and y are read once and out and n written once (8 bytes a column in 16-bit
// types), and the second sum runs on values already at hand.  The bound is
// HBM; what there is besides are the two sums of a row, each a latency of two
// shuffles' trees and a barrier, which the rows on their way hide in part.
// T=4096, H=4096 with the next norm: 16-bit 26.5 us, 5.1 TB/s (0.76 of a copy's
// rate); fp32 stream 35 us, 5.7 TB/s; H=8192, 16-bit 49 us, 5.5 TB/s.  One row
// of T: 4 us, launch and two sums (2.7 us in a graph).
#include "norm_block.cuh"

namespace qmoe {
namespace norm {

struct FwdArgs {
    int64_t rows;
    int cols, stages, stage_bytes;
    int lie_base, lie_step;  // Lie
    bool fp32;               // Columns
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
template <typename RT, typename YT, int NV, int VEC, bool SHIFT, bool POST>
__global__ void __launch_bounds__(512, 1)
norm_fwd_kernel(const FwdArgs a) {
    constexpr int E = NV * VEC;
    constexpr bool KEEP = E <= 16;  // the weights stay in registers from row to row, y from sum to sum
    __shared__ __align__(16) float sums[2][2][16];
    __shared__ uint64_t full[MAX_ROWS][MAX_STAGES];
    extern __shared__ __align__(128) uint8_t dynamic[];
    const int tx = threadIdx.x, cols = a.cols;
    const int64_t stride = (int64_t)gridDim.x * blockDim.y;
    const float inv_cols = 1.f / (float)cols;
    int flip = 0;

    int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const int shift = SHIFT ? (int)((a.lie_base + row * a.lie_step) % VEC) : 0;
    const Columns<VEC, SHIFT> k = {cols, shift, a.fp32 && shift == 0};
    Ring<VEC != 1 && !SHIFT> ring = {full[threadIdx.y], dynamic + (int64_t)threadIdx.y * a.stages * a.stage_bytes, a.stages,
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
    constexpr int HELD = KEEP ? E : VEC;
    float wg[HELD], wn[HELD], y[HELD];
    auto col_factors = [&](int c, float* to) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) to[i] = 1.f;
        if (a.w) load_columns(k, a.w, c, to);
        if (a.gate_mode == QMOE_GATE_COL) {
            float g[VEC];
            load_columns(k, a.gate, c, g);
#pragma unroll
            for (int i = 0; i < VEC; ++i) to[i] *= g[i];
        }
    };
    if (KEEP) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = k.at(v);
            if (!k.live(c)) continue;
            if (POST) col_factors(c, &wg[v * VEC]);
            if (a.w_next) load_columns(k, a.w_next, c, &wn[v * VEC]);
        }
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
        read_row<NV, true, RT>(a.r, from, row, k, o);
        if (ring.lost) o[0] = NAN;
        if (POST) {
            if (KEEP) read_row<NV, true, YT>(a.y, from, row, k, y);
            // the v-th access of y; wide rows read it once more from the stage
            auto y_of = [&](int v) -> float* {
                if (KEEP) return &y[v * VEC];
                read_columns<true>(k, row_at<true, YT>(k, a.y, from, row), k.at(v), y);
                return y;
            };
            float scale = a.alpha * g_row;
            if (a.w) {
                float s = 0.f;
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    if (!k.live(k.at(v))) continue;
                    const float* const yv = y_of(v);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) s = fmaf(yv[i], yv[i], s);
                }
                const float rstd = rsqrtf(row::row_sum(s, sums[flip]) * inv_cols + a.eps);
                flip ^= 1;
                met = true;
                ring.refill(row);
                if (tx == 0 && a.rstd) a.rstd[row] = rstd;
                scale *= rstd;
            }
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int c = k.at(v);
                if (!k.live(c)) continue;
                float* const yv = y_of(v);
                if (a.gate_mode == QMOE_GATE_FULL) {
                    float g[VEC];
                    read_columns<true>(k, row_at<true, YT>(k, a.full_gate, from, row), c, g);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) yv[i] *= g[i];
                }
                if (!KEEP) col_factors(c, wg);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const int e = v * VEC + i;
                    o[e] = fmaf(yv[i] * scale, wg[KEEP ? e : i], o[e]);
                }
                clear_outside(k, c, &o[v * VEC]);  // 0 times a scale that is not finite
                store_columns(k, static_cast<RT*>(a.out) + row * a.ldo, c, &o[v * VEC]);
            }
        }
        if (a.w_next) {
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
                const int c = k.at(v);
                if (!k.live(c)) continue;
                float n[VEC];
                if (!KEEP) load_columns(k, a.w_next, c, wn);
#pragma unroll
                for (int i = 0; i < VEC; ++i) n[i] = o[v * VEC + i] * rstd * wn[KEEP ? v * VEC + i : i];
                store_columns(k, static_cast<YT*>(a.n) + row * a.ldn, c, n);
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

static_assert(3 * (int64_t)stage_bytes(MAX_COLS, 4) <= room_of(0, 1), "a stage of the widest rows: r, y and a full gate");

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
        static int go(FwdArgs& a, cudaStream_t st) {
            constexpr int W = wide_vec<RT, YT>();
            Lie lie = {W, a.cols};
            lie.add(a.r.p, a.r.ld, sizeof(RT));
            if (POST) lie.add(a.y.p, a.y.ld, sizeof(YT));
            if (a.full_gate.p) lie.add(a.full_gate.p, a.full_gate.ld, sizeof(YT));
            if (POST) lie.add(a.out, a.ldo, sizeof(RT));
            if (a.w_next) lie.add(a.n, a.ldn, sizeof(YT));
            a.lie_base = lie.base;
            a.lie_step = lie.step;
            a.fp32 = aligned16(a.w) && aligned16(a.w_next) && aligned16(a.gate_mode == QMOE_GATE_COL ? a.gate : nullptr);
            const bool at_zero = lie.at_zero() && a.fp32;
            // a warp more for the shift is worth it (T=4096, 16-bit: H=2047 21 us against 30 value by value, H=4095 50.5
            // against 56), twice the values a thread are not (H=8191 145 us against 105)
            Shape s = shape_of(a.cols, W, 16, false);
            const bool shifted = !at_zero && fits(s, lie);
            if (!at_zero && !shifted) s = shape_for(a.cols, 1, 16);
            const int rb = stage_bytes(a.cols, sizeof(RT)), yb = stage_bytes(a.cols, sizeof(YT));
            a.y.off = rb;
            a.full_gate.off = rb + yb;
            const int bytes = rb + (POST ? yb : 0) + (a.full_gate.p ? yb : 0);
            const bool few = s.values() == 16;
            if (at_zero)
                return few ? start<norm_fwd_kernel<RT, YT, 16 / W, W, false, POST>>(s, a, bytes, st)
                           : start<norm_fwd_kernel<RT, YT, 32 / W, W, false, POST>>(s, a, bytes, st);
            if (shifted)
                return few ? start<norm_fwd_kernel<RT, YT, 16 / W, W, true, POST>>(s, a, bytes, st)
                           : start<norm_fwd_kernel<RT, YT, 32 / W, W, true, POST>>(s, a, bytes, st);
            return few ? start<norm_fwd_kernel<RT, YT, 16, 1, false, POST>>(s, a, bytes, st)
                       : start<norm_fwd_kernel<RT, YT, 32, 1, false, POST>>(s, a, bytes, st);
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
    return norm::by_types<norm::PreGo>(stream_dtype, block_dtype, a, (cudaStream_t)stream);
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
    return norm::by_types<norm::PostGo>(stream_dtype, block_dtype, a, (cudaStream_t)stream);
}
