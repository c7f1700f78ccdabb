// Norms before and after a block, gradients (qmoe_norm_pre_backward,
// qmoe_norm_post_backward).
//
//   D  = dout + rstd_n (dn w_n - x mean(dn w_n x)),  x = out rstd_n
//   dz = alpha g D,  t = y rstd,  dy = rstd (dz w - t mean(dz w t))
//   dw_n = sum_t dn x,  dw = sum_t dz t,  dg = alpha z D  (z = t w)
//
// norm_pre's gradient is the first line alone.  As in the forward, a row lives
// in registers and is read and written once (6 values a column for the whole
// sandwich).  The sums over rows stay in registers (rows of up to 16 values a
// thread) or in shared memory words that one thread owns, over all the rows of
// a CTA; each CTA then writes one partial row, and a second launch adds the
// partial rows in a fixed order, so no atomic decides an order.
//
// HBM is the bound beside an fp32 stream: T=8192, H=4096, the whole sandwich
// 106 us, 5.7 TB/s (0.85 of a copy's rate).  With a 16-bit one it is not: an SM
// has one row of 4096 columns at a time, whose wait, two sums and barriers take
// as long for two thirds of the bytes: T=4096 58 us, 3.5 TB/s (0.52), H=8192
// 106 us (128 with a gate for each column); norm_pre's, one sum, 32 us (0.63)
// and 52.  Rows past 8192 columns (32 values a thread, spilled in part, no ring)
// run at 1.6 TB/s: T=4096, H=12288, 16-bit 374 us.
#include "norm_block.cuh"

namespace qmoe {
namespace norm {

struct BwdArgs {
    int64_t rows;
    int cols, stages, stage_bytes;
    int lie_base, lie_step;  // Lie
    bool fp32;               // Columns
    // dout (norm_pre: dres) and out (what the next norm read; norm_pre: x) have the stream's type, dn, y and a full
    // gate the block's; dn null: no next norm
    Source dout, dn, out, y, full_gate;
    const float* w_next;
    const float* rstd_next;
    const float* w;
    const float* rstd;
    int gate_mode;
    const float* gate;
    float alpha;
    void* dr;
    int64_t lddr;
    void* dy;
    int64_t lddy;
    void* dgate;
    int64_t lddg;
    float* part;  // [3][partial rows][cols]: dw_next, dw, column gate
    int64_t part_rows;
};

// Sums over rows that one thread owns: registers, or shared memory words laid
// out so that a warp's accesses hit distinct banks.
template <int E, bool SMEM>
struct ColSums {
    float r[SMEM ? 1 : E];
    float* s;
    __device__ __forceinline__ void init(float* smem) {
        if constexpr (SMEM) {
            s = smem;
#pragma unroll
            for (int e = 0; e < E; ++e) s[at(e)] = 0.f;
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) r[e] = 0.f;
        }
    }
    __device__ __forceinline__ static int at(int e) { return e * blockDim.x + threadIdx.x; }
    __device__ __forceinline__ void add(int e, float v) {
        if constexpr (SMEM) s[at(e)] += v;
        else r[e] += v;
    }
    __device__ __forceinline__ float get(int e) const {
        if constexpr (SMEM) return s[at(e)];
        else return r[e];
    }
};

// Where a kernel of E values a thread keeps things: 8: sums and weights in
// registers; 16: the weights in shared memory; 32: the sums there, and then no
// room for a ring, so rows and weights come straight from global memory.
// POST: the whole sandwich; without it the kernel is norm_pre's gradient.
template <typename RT, typename YT, int NV, int VEC, bool SHIFT, bool POST>
__global__ void __launch_bounds__(512, 1)
norm_bwd_kernel(const BwdArgs a) {
    constexpr int E = NV * VEC;
    constexpr bool SMEM = E > 16, RING = !SMEM, KEEP = E <= 8, W_SMEM = E == 16;
    __shared__ __align__(16) float sums[2][2][16];
    __shared__ uint64_t full[MAX_ROWS][MAX_STAGES];
    extern __shared__ __align__(128) uint8_t dynamic[];  // the ring; column sums or weights [w_next, w]
    const int tx = threadIdx.x, cols = a.cols;
    const int64_t stride = (int64_t)gridDim.x * blockDim.y;
    const float inv_cols = 1.f / (float)cols;
    const bool next = POST ? a.dn.p != nullptr : true;
    int flip = 0;

    float* const cols_smem = reinterpret_cast<float*>(dynamic + (int64_t)blockDim.y * a.stages * a.stage_bytes);
    ColSums<E, SMEM> sum_wn, sum_w, sum_g;
    sum_wn.init(cols_smem);
    if (POST) {
        sum_w.init(cols_smem + E * blockDim.x);
        sum_g.init(cols_smem + 2 * E * blockDim.x);
    }
    int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const int shift = SHIFT ? (int)((a.lie_base + row * a.lie_step) % VEC) : 0;
    const Columns<VEC, SHIFT> k = {cols, shift, a.fp32 && shift == 0};
    Ring<VEC != 1 && !SHIFT> ring = {full[threadIdx.y], dynamic + (int64_t)threadIdx.y * a.stages * a.stage_bytes, a.stages,
                                     a.stage_bytes, a.rows, stride};
    int matrices = 0;
    ring.feed.take(a.dout, sizeof(RT), matrices, tx, row, stride, cols);
    ring.feed.take(a.dn, sizeof(YT), matrices, tx, row, stride, cols);
    ring.feed.take(a.out, sizeof(RT), matrices, tx, row, stride, cols);
    if (POST) ring.feed.take(a.y, sizeof(YT), matrices, tx, row, stride, cols);
    if (POST) ring.feed.take(a.full_gate, sizeof(YT), matrices, tx, row, stride, cols);
    if (RING && tx == 0)
        for (int i = 0; i < MAX_STAGES; ++i) tc::mbar_init(&full[threadIdx.y][i], matrices);
    for (int i = tx; i < 64; i += blockDim.x) (&sums[0][0][0])[i] = 0.f;
    tc::fence_barrier_init();
    __syncthreads();
    pdl_sync();
    if (RING) ring.begin(row);
    float w[KEEP ? E : VEC], wn[KEEP ? E : VEC], gc[KEEP ? E : VEC];
    auto column = [&](int v) { return k.at(v); };
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = column(v);
        if (!k.live(c)) continue;
        if (KEEP) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) w[v * VEC + i] = gc[v * VEC + i] = 1.f;
            if (POST && a.w) load_columns(k, a.w, c, &w[v * VEC]);
            if (next) load_columns(k, a.w_next, c, &wn[v * VEC]);
            if (POST && a.gate_mode == QMOE_GATE_COL) load_columns(k, a.gate, c, &gc[v * VEC]);
        } else if (W_SMEM) {  // a thread reads back what it wrote itself
            float t[VEC];
            if (next) {
                load_columns(k, a.w_next, c, t);
                row::store<VEC>(cols_smem + c + k.shift, t);
            }
            if (POST && a.w) {
                load_columns(k, a.w, c, t);
                row::store<VEC>(cols_smem + E * blockDim.x + c + k.shift, t);
            }
        }
    }
    // a vector's weights, where they are not in registers from row to row
    auto weights_next = [&](int c, int v) -> const float* {
        if (KEEP) return &wn[v * VEC];
        if (W_SMEM) row::load<VEC>(cols_smem + c + k.shift, wn);
        else load_columns(k, a.w_next, c, wn);
        return wn;
    };
    // a row's own scalars are asked for one row early
    float rstd_n_ahead = 0.f, rstd_ahead = 1.f, g_ahead = 1.f;
    auto ahead = [&](int64_t r) {
        if (r >= a.rows) return;
        if (next) rstd_n_ahead = a.rstd_next[r];
        if (POST && a.w) rstd_ahead = a.rstd[r];
        if (POST && a.gate_mode == QMOE_GATE_ROW) g_ahead = a.gate[r];
    };
    ahead(row);
    for (; row < a.rows; row += stride) {
        const float rstd_n = rstd_n_ahead, rstd = rstd_ahead, g_row = g_ahead;
        ahead(row + stride);
        const uint8_t* const from = RING ? ring.wait() : nullptr;
        bool met = false;
        auto meet = [&] {  // the row's threads have met: what the last row's stage held is free
            if (RING && !met) ring.refill(row);
            met = true;
        };
        float d[E];
        if (a.dout.p) {
            read_row<NV, RING, RT>(a.dout, from, row, k, d);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) d[e] = 0.f;
        }
        if (RING && ring.lost) d[0] = NAN;
        if (next) {
            float x[E], dn[E], s = 0.f;
            read_row<NV, RING, YT>(a.dn, from, row, k, dn);
            read_row<NV, RING, RT>(a.out, from, row, k, x);
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                if (!k.live(column(v))) continue;
                const float* const wv = weights_next(column(v), v);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const int e = v * VEC + i;
                    x[e] *= rstd_n;
                    sum_wn.add(e, dn[e] * x[e]);
                    dn[e] *= wv[i];
                    s = fmaf(dn[e], x[e], s);
                }
            }
            const float mean = row::row_sum(s, sums[flip]) * inv_cols;
            flip ^= 1;
            meet();
#pragma unroll
            for (int e = 0; e < E; ++e) d[e] = fmaf(rstd_n, dn[e] - x[e] * mean, d[e]);
#pragma unroll
            for (int v = 0; v < NV; ++v) clear_outside(k, column(v), &d[v * VEC]);  // 0 times a mean that is not finite
        }
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (k.live(column(v)))
                store_columns(k, static_cast<RT*>(a.dr) + row * a.lddr, column(v), &d[v * VEC]);
        if (POST) {
            float t[E], s = 0.f, s_gate = 0.f;
            read_row<NV, RING, YT>(a.y, from, row, k, t);
            // t = y rstd; d becomes dz w
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int c = column(v);
                if (!k.live(c)) continue;
                float wt[VEC], g[VEC], dg[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    wt[i] = KEEP ? w[v * VEC + i] : 1.f;
                    g[i] = g_row;
                    if (KEEP) g[i] *= gc[v * VEC + i];
                }
                if (W_SMEM && a.w) row::load<VEC>(cols_smem + E * blockDim.x + c + k.shift, wt);
                if (!W_SMEM && !KEEP && a.w) load_columns(k, a.w, c, wt);
                if (!KEEP && a.gate_mode == QMOE_GATE_COL) load_columns(k, a.gate, c, g);
                if (a.gate_mode == QMOE_GATE_FULL)
                    read_columns<RING>(k, row_at<RING, YT>(k, a.full_gate, from, row), c, g);
                clear_outside(k, c, g);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const int e = v * VEC + i;
                    const float ad = a.alpha * d[e];
                    t[e] *= rstd;
                    const float dz = ad * g[i];
                    dg[i] = ad * (t[e] * wt[i]);
                    s_gate += dg[i];
                    sum_w.add(e, dz * t[e]);
                    d[e] = dz * wt[i];
                    s = fmaf(d[e], t[e], s);
                }
                if (a.gate_mode == QMOE_GATE_COL) {
#pragma unroll
                    for (int i = 0; i < VEC; ++i) sum_g.add(v * VEC + i, dg[i]);
                }
                if (a.gate_mode == QMOE_GATE_FULL)
                    store_columns(k, static_cast<YT*>(a.dgate) + row * a.lddg, c, dg);
            }
            if (a.w || a.gate_mode == QMOE_GATE_ROW) {
                if (a.gate_mode == QMOE_GATE_ROW) {
                    const float2 both = row::row_sums<true>(s, s_gate, sums[flip]);
                    s = both.x;
                    if (tx == 0) static_cast<float*>(a.dgate)[row] = both.y;
                } else {
                    s = row::row_sum(s, sums[flip]);
                }
                flip ^= 1;
                meet();
                s *= inv_cols;
            }
            if (a.w) {
#pragma unroll
                for (int e = 0; e < E; ++e) d[e] = rstd * (d[e] - t[e] * s);
            }
#pragma unroll
            for (int v = 0; v < NV; ++v)
                if (k.live(column(v)))
                    store_columns(k, static_cast<YT*>(a.dy) + row * a.lddy, column(v), &d[v * VEC]);
        }
        if (RING) {
            if (!met || blockDim.x == 32) {
                row_barrier();
                meet();
            }
            if (a.stages == 1) {
                row_barrier();
                ring.post(row + stride, 0);
            }
            ring.next();
        }
    }
    const int64_t part = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = column(v);
        if (!k.live(c)) continue;
        float t[VEC];
        auto put = [&](ColSums<E, SMEM>& s, int which) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) t[i] = s.get(v * VEC + i);
            float* to = a.part + (which * a.part_rows + part) * cols + c;
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                if (k.in(c + i)) to[i] = t[i];
        };
        if (next) put(sum_wn, 0);
        if (POST && a.w) put(sum_w, 1);
        if (POST && a.gate_mode == QMOE_GATE_COL) put(sum_g, 2);
    }
}

// out[j][c] = the sum of partial rows of output j, in row order within each of
// 32 interleaved groups, then over the groups.
struct SumArgs {
    const float* part;
    int64_t part_rows, used;
    int cols;
    float* out[3];
};
__global__ void __launch_bounds__(1024) norm_sum_kernel(const SumArgs a) {
    __shared__ float group[32][33];
    pdl_sync();
    float* out = a.out[blockIdx.y];
    if (!out) return;
    const int c = blockIdx.x * 32 + threadIdx.x;
    float s = 0.f;
    if (c < a.cols) {
        const float* p = a.part + (int64_t)blockIdx.y * a.part_rows * a.cols + c;
#pragma unroll 4
        for (int64_t i = threadIdx.y; i < a.used; i += 32) s += p[i * a.cols];
    }
    group[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    s = group[threadIdx.x][threadIdx.y];
    s = row::warp_sum(s);
    const int oc = blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x == 0 && oc < a.cols) out[oc] = s;
}

// The threads of a row go by the columns alone, not by the access.  No warp more
// for a shift: that would leave an SM fewer rows, and value by value is faster
// then (T=4096, 16-bit: H=2047 50 us against 67, H=4095 93 against 120).
inline Shape cut_of(int64_t cols) { return shape_of(cols, 8, 8, true); }
// CTAs of a launch: one wave of 512 threads an SM.
inline int per_sm_of(const Shape& s) { return 512 / (s.threads * s.rows_per_cta); }
inline int64_t bwd_ctas(const Shape& s, int64_t rows) {
    const int64_t ctas = (rows + s.rows_per_cta - 1) / s.rows_per_cta;
    const int64_t fit = (int64_t)row::kSMs * per_sm_of(s);
    return ctas < fit ? ctas : fit;
}
inline int64_t part_rows(int64_t rows, int64_t cols) {
    const Shape s = cut_of(cols);
    return bwd_ctas(s, rows) * s.rows_per_cta > 0 ? bwd_ctas(s, rows) * s.rows_per_cta : 1;
}

// Bytes beside the ring: sums (32 values a thread) or weights (16).
constexpr int64_t besides_of(int values, int threads, int sums) {
    return values == 32 ? (int64_t)sums * 32 * threads * 4 : values == 16 ? (int64_t)(sums == 3 ? 2 : 1) * 16 * threads * 4 : 0;
}
// Every width that goes through the ring has room for a stage of five fp32
// matrices (a full gate, dout and dn): at 8192 columns 432 bytes remain.
constexpr bool all_fit() {
    for (int threads = 32; threads <= 512; threads += 32) {
        const int rows = threads == 32 ? 4 : 1;
        if (5 * (int64_t)stage_bytes(8 * threads, 4) * rows > room_of(0, 512 / (threads * rows))) return false;
        if (threads > 256 && 5 * (int64_t)stage_bytes(16 * threads, 4) > room_of(besides_of(16, threads, 3), 1)) return false;
    }
    return true;
}
static_assert(all_fit(), "a stage of the widest rows");

template <auto Kernel>
inline int start(const Shape& s, BwdArgs& a, int sums, int row_bytes, int64_t ctas, cudaStream_t st) {
    const int64_t besides = besides_of(s.values(), s.threads, sums);
    a.stage_bytes = row_bytes;
    a.stages = s.values() == 32 ? 0 : stages_of((int64_t)row_bytes * s.rows_per_cta, besides, per_sm_of(s));
    if (s.values() < 32 && !a.stages) return QMOE_ERR_UNSUPPORTED;
    const size_t smem = (size_t)(besides + (int64_t)a.stages * row_bytes * s.rows_per_cta);
    if (smem > 47 * 1024) {
        const int rc = row::allow_smem<Kernel>(225 * 1024);
        if (rc != QMOE_OK) return rc;
    }
    return launch_pdl(Kernel, dim3((unsigned)ctas), dim3(s.threads, s.rows_per_cta), smem, st, a);
}

template <bool POST>
struct Bwd {
    template <typename RT, typename YT>
    struct Go {
        // WIDE, FEW: columns of an access for rows of 16 values a thread and more, and of 8
        template <int WIDE, int FEW, bool SHIFT>
        static int by_values(const Shape& s, BwdArgs& a, int bytes, int64_t ctas, cudaStream_t st) {
            constexpr int sums = POST ? 3 : 1;
            if (s.values() == 8)
                return start<norm_bwd_kernel<RT, YT, 8 / FEW, FEW, SHIFT, POST>>(s, a, sums, bytes, ctas, st);
            if (s.values() == 16)
                return start<norm_bwd_kernel<RT, YT, 16 / WIDE, WIDE, SHIFT, POST>>(s, a, sums, bytes, ctas, st);
            return start<norm_bwd_kernel<RT, YT, 32 / WIDE, WIDE, SHIFT, POST>>(s, a, sums, bytes, ctas, st);
        }
        static int go(BwdArgs& a, cudaStream_t st) {
            Shape s = cut_of(a.cols);
            // rows of 8 values a thread: in two accesses of 4 columns (T=4096, H=4096, 16-bit 59 us against 61 in one of 8,
            // H=1024 21 against 24); wider rows by 8 where the types allow it (H=8192: 117 us against 131; all when it was
            // chosen)
            constexpr int WIDE = wide_vec<RT, YT>();
            const int W = s.values() == 8 ? 4 : WIDE;
            Lie lie = {W, a.cols};
            auto lies = [&](const Source& m, int size) {
                if (m.p) lie.add(m.p, m.ld, size);
            };
            lies(a.dout, sizeof(RT));
            lies(a.dn, sizeof(YT));
            lies(a.out, sizeof(RT));
            lie.add(a.dr, a.lddr, sizeof(RT));
            if (POST) {
                lies(a.y, sizeof(YT));
                lies(a.full_gate, sizeof(YT));
                lie.add(a.dy, a.lddy, sizeof(YT));
                if (a.full_gate.p) lie.add(a.dgate, a.lddg, sizeof(YT));
            }
            a.lie_base = lie.base;
            a.lie_step = lie.step;
            a.fp32 = aligned16(a.w) && aligned16(a.w_next) && aligned16(a.gate_mode == QMOE_GATE_COL ? a.gate : nullptr);
            const bool at_zero = lie.at_zero() && a.fp32, shifted = !at_zero && fits(s, lie);
            const int vec = at_zero || shifted ? W : 1;
            s.nv = s.values() / vec;
            s.vec = vec;
            const int64_t ctas = bwd_ctas(s, a.rows);
            const int rb = stage_bytes(a.cols, sizeof(RT)), yb = stage_bytes(a.cols, sizeof(YT));
            int at = 0;
            auto place = [&](Source& src, int bytes) {
                src.off = at;
                if (src.p) at += bytes;
            };
            place(a.dout, rb);
            place(a.dn, yb);
            place(a.out, rb);
            place(a.y, yb);
            place(a.full_gate, yb);
            if (at_zero) return by_values<WIDE, 4, false>(s, a, at, ctas, st);
            if (shifted) return by_values<WIDE, 4, true>(s, a, at, ctas, st);
            return by_values<1, 1, false>(s, a, at, ctas, st);
        }
    };
};
template <typename RT, typename YT> using PreGo = Bwd<false>::Go<RT, YT>;
template <typename RT, typename YT> using PostGo = Bwd<true>::Go<RT, YT>;

template <template <typename, typename> class F>
inline int run(BwdArgs& a, int rt, int yt, float* const (&out)[3], void* ws, cudaStream_t st) {
    a.part = static_cast<float*>(ws);
    a.part_rows = part_rows(a.rows, a.cols);
    const Shape s = cut_of(a.cols);
    const int64_t ctas = bwd_ctas(s, a.rows);
    if (ctas > 0) {
        const int rc = by_types<F>(rt, yt, a, st);
        if (rc != QMOE_OK) return rc;
    }
    if (!out[0] && !out[1] && !out[2]) return QMOE_OK;
    SumArgs b = {a.part, a.part_rows, ctas * s.rows_per_cta, a.cols, {out[0], out[1], out[2]}};
    return launch_pdl(norm_sum_kernel, dim3((unsigned)((a.cols + 31) / 32), 3), dim3(32, 32), 0, st, b);
}

}  // namespace norm
}  // namespace qmoe

using namespace qmoe;

extern "C" size_t qmoe_norm_bwd_workspace_bytes(int64_t rows, int64_t cols) {
    if (rows < 0 || cols <= 0 || cols > norm::MAX_COLS) return 0;
    return (size_t)(3 * norm::part_rows(rows, cols) * cols * 4 + 255) / 256 * 256;
}

static bool ws_ok(int64_t rows, int64_t cols, const void* ws, size_t bytes) {
    return ws && (reinterpret_cast<uintptr_t>(ws) & 255u) == 0 && bytes >= qmoe_norm_bwd_workspace_bytes(rows, cols);
}

extern "C" int qmoe_norm_pre_backward(int64_t rows, int64_t cols, int stream_dtype, int block_dtype, const void* dn,
                                      int64_t lddn, const void* x, int64_t ldx, const float* rstd, const float* w,
                                      const void* dres, int64_t lddres, void* dx, int64_t lddx, float* dw, void* ws,
                                      size_t ws_bytes, qmoe_stream_t stream) {
    if (rows < 0 || cols <= 0 || !norm::types_ok(stream_dtype, block_dtype)) return QMOE_ERR_ARG;
    if (!w || !dw || !row::type_aligned(w, 4) || !row::type_aligned(dw, 4)) return QMOE_ERR_ARG;
    const int rs = row::dtype_size(stream_dtype), bs = row::dtype_size(block_dtype);
    if (rows > 0) {
        if (!dn || !x || !rstd || !dx || lddn < cols || ldx < cols || lddx < cols || (dres && lddres < cols))
            return QMOE_ERR_ARG;
        if (!row::type_aligned(dn, bs) || !row::type_aligned(x, rs) || !row::type_aligned(dx, rs) ||
            !row::type_aligned(dres, rs) || !row::type_aligned(rstd, 4))
            return QMOE_ERR_ARG;
    }
    if (cols > norm::MAX_COLS) return QMOE_ERR_UNSUPPORTED;
    if (!ws_ok(rows, cols, ws, ws_bytes)) return QMOE_ERR_ARG;
    norm::BwdArgs a = {};
    a.rows = rows;
    a.cols = (int)cols;
    a.dout = {dres, lddres, 0};
    a.dn = {dn, lddn, 0};
    a.out = {x, ldx, 0};
    a.w_next = w;
    a.rstd_next = rstd;
    a.dr = dx;
    a.lddr = lddx;
    return norm::run<norm::PreGo>(a, stream_dtype, block_dtype, {dw, nullptr, nullptr}, ws, (cudaStream_t)stream);
}

extern "C" int qmoe_norm_post_backward(int64_t rows, int64_t cols, int stream_dtype, int block_dtype, const void* dout,
                                       int64_t lddout, const void* y, int64_t ldy, const float* w, const float* rstd,
                                       int gate_mode, const void* gate, int64_t ldg, float alpha, const void* dn,
                                       int64_t lddn, const void* out, int64_t ldo, const float* w_next,
                                       const float* rstd_next, void* dr, int64_t lddr, void* dy, int64_t lddy,
                                       float* dw, void* dgate, int64_t lddg, float* dw_next, void* ws, size_t ws_bytes,
                                       qmoe_stream_t stream) {
    if (rows < 0 || cols <= 0 || !norm::types_ok(stream_dtype, block_dtype) || !norm::gate_mode_ok(gate_mode))
        return QMOE_ERR_ARG;
    const int rs = row::dtype_size(stream_dtype), bs = row::dtype_size(block_dtype);
    const bool full = gate_mode == QMOE_GATE_FULL, gated = gate_mode != QMOE_GATE_NONE;
    if (w && (!dw || !row::type_aligned(w, 4) || !row::type_aligned(dw, 4))) return QMOE_ERR_ARG;
    // a column gate's sum is written for zero rows too
    if (gated && (!gate || !dgate) && (rows > 0 || gate_mode == QMOE_GATE_COL)) return QMOE_ERR_ARG;
    if (gated && (!row::type_aligned(gate, full ? bs : 4) || !row::type_aligned(dgate, full ? bs : 4)))
        return QMOE_ERR_ARG;
    if (dn && (!w_next || !dw_next || !row::type_aligned(w_next, 4) || !row::type_aligned(dw_next, 4)))
        return QMOE_ERR_ARG;
    if (rows > 0) {
        if ((!dout && !dn) || !y || !dr || !dy || (dout && lddout < cols) || ldy < cols || lddr < cols || lddy < cols)
            return QMOE_ERR_ARG;
        if (dn && (!out || !rstd_next || lddn < cols || ldo < cols)) return QMOE_ERR_ARG;
        if (w && !rstd) return QMOE_ERR_ARG;
        if (full && (ldg < cols || lddg < cols)) return QMOE_ERR_ARG;
        if (!row::type_aligned(dout, rs) || !row::type_aligned(y, bs) || !row::type_aligned(dr, rs) ||
            !row::type_aligned(dy, bs) || !row::type_aligned(rstd, 4) || !row::type_aligned(dn, bs) ||
            (dn && (!row::type_aligned(out, rs) || !row::type_aligned(rstd_next, 4))))
            return QMOE_ERR_ARG;
    }
    if (cols > norm::MAX_COLS) return QMOE_ERR_UNSUPPORTED;
    if (!ws_ok(rows, cols, ws, ws_bytes)) return QMOE_ERR_ARG;
    norm::BwdArgs a = {};
    a.rows = rows;
    a.cols = (int)cols;
    a.dout = {dout, lddout, 0};
    a.y = {y, ldy, 0};
    a.w = w;
    a.rstd = rstd;
    a.gate_mode = gate_mode;
    if (full) a.full_gate = {gate, ldg, 0};
    else a.gate = static_cast<const float*>(gate);
    a.alpha = alpha;
    a.dr = dr;
    a.lddr = lddr;
    a.dy = dy;
    a.lddy = lddy;
    a.dgate = dgate;
    a.lddg = lddg;
    if (dn) {
        a.dn = {dn, lddn, 0};
        a.out = {out, ldo, 0};
        a.w_next = w_next;
        a.rstd_next = rstd_next;
    }
    float* const col_gate = gate_mode == QMOE_GATE_COL ? static_cast<float*>(dgate) : nullptr;
    return norm::run<norm::PostGo>(a, stream_dtype, block_dtype,
                                   {dn ? dw_next : nullptr, w ? dw : nullptr, col_gate}, ws, (cudaStream_t)stream);
}
