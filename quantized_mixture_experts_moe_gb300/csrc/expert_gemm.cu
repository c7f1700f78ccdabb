// Products of the routed experts' rows with 16-bit weights, and their
// gradients (qmoe_expert_linear, qmoe_expert_linear_dx, qmoe_expert_linear_dw):
//
//   y[s][n]     = sum_k w[e][n][k] x[s][k]      for the rows s of expert e
//   dx[s][k]    = sum_n w[e][n][k] dy[s][n]
//   dw[e][n][k] = sum_s dy[s][n] x[s][k]
//
// One persistent kernel for the three.  The 128 lanes of a tile are outputs of
// the layer (y), its inputs (dx) or rows of dw; the columns are up to NT rows s
// (y, dx) or columns of dw.  An operand whose reduction axis is contiguous in
// memory (w and x for y, dy for dx) is read as such; the others (w for dx, both
// for dw) lie in shared memory as they do in HBM, reduction rows of 64 values,
// and the tensor core transposes them as it reads.
#include "expert_gemm.cuh"

namespace qmoe {
namespace eg {

// Warps: the epilogue's, one that loads tiles, one that issues products, then
// those that gather.
constexpr int WARP_TMA = 8, WARP_MMA = 9;
constexpr int threads_of(bool gather) { return (10 + (gather ? GATHER_WARPS : 0)) * 32; }

template <int MODE, int NT>
struct Cfg {
    static constexpr int P_BYTES = 128 * STEP * 2, Q_BYTES = NT * STEP * 2, STAGE = P_BYTES + Q_BYTES;
    static constexpr int TMEM_COLS = 2 * NT < 32 ? 32 : 2 * NT;
    static constexpr int LIST = 2 * (MAX_E + 2) * 4;
    static constexpr int FIXED = EPI_WARPS * STAGE_OUT + (LIST + 15) / 16 * 16 + 512 + 1024;
    static constexpr int FIT = (232448 - FIXED) / STAGE;
    static constexpr int STAGES = FIT > 10 ? 10 : FIT;
    static constexpr int OUT_OFF = STAGES * STAGE;
    static constexpr int LIST_OFF = OUT_OFF + EPI_WARPS * STAGE_OUT;
    static constexpr int BAR_OFF = LIST_OFF + (LIST + 15) / 16 * 16;
    static constexpr int MISC_OFF = BAR_OFF + (2 * STAGES + 4) * 8;
    static constexpr int SMEM = MISC_OFF + 64 + 1024;
    static_assert(SMEM <= 232448 && STAGES >= 4, "shared memory per CTA");
};

template <int MODE, int NT, bool GATHER>
__global__ void __launch_bounds__(threads_of(GATHER), 1)
expert_gemm_kernel(const __grid_constant__ CUtensorMap map_p, const __grid_constant__ CUtensorMap map_q, const Args g) {
    using C = Cfg<MODE, NT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    int* off = reinterpret_cast<int*>(smem + C::LIST_OFF);
    int* base = off + MAX_E + 1;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
    uint64_t* empty = full + C::STAGES;
    uint64_t* acc_full = empty + C::STAGES;
    uint64_t* acc_empty = acc_full + 2;
    uint32_t* tmem_at = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::MISC_OFF + 8);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::STAGES; ++i) {
            tc::mbar_init(&full[i], 1);
            tc::mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&acc_full[i], 1);
            tc::mbar_init(&acc_empty[i], EPI_WARPS);
        }
        *abort_flag = 0;
        tc::fence_barrier_init();
    }
    if (warp == WARP_MMA) {
        tc::tmem_alloc(tmem_at, C::TMEM_COLS);
        tc::tmem_relinquish();
    }
    pdl_wait();
    read_offsets<MODE, 128, NT>(g, off, base);
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tm = *tmem_at;
    Walk<MODE, 128, NT, 16> walk(g, off, base);
    const int total = walk.total();

    if (warp == WARP_TMA) {
        int slot = 0, in_flight = 0;
        uint32_t phase = 0;
        for (int u = blockIdx.x; u < total && !*abort_flag; u += gridDim.x) {
            const Unit t = walk.at(u);
            const int boxes = GATHER ? 0 : (t.n + Q_BOX - 1) / Q_BOX;
            for (int s = 0; s < t.steps; ++s) {
                if (!warp_wait(&empty[slot], phase ^ 1, abort_flag, g.status)) break;
                uint8_t* st = smem + slot * C::STAGE;
                const int k0 = s * STEP;
                if (lane == 0) {
                    tc::mbar_arrive_expect_tx(&full[slot], C::P_BYTES + (GATHER ? (t.n + 3) / 4 * 512 : boxes * Q_BOX * 128));
                    if constexpr (MODE == FWD) {
                        tc::tma_load_3d(st, &map_p, &full[slot], k0, t.l0, t.e);
                    } else {
                        tc::tma_load_3d(st, &map_p, &full[slot], t.l0, k0, t.e);
                        tc::tma_load_3d(st + 8192, &map_p, &full[slot], t.l0 + 64, k0, t.e);
                    }
                }
                __syncwarp();
                if (lane < boxes)
                    tc::tma_load_2d(st + C::P_BYTES + lane * Q_BOX * 128, &map_q, &full[slot], k0, t.q0 + lane * Q_BOX);
                __syncwarp();
                if (in_flight < C::STAGES) ++in_flight;
                if (++slot == C::STAGES) { slot = 0; phase ^= 1; }
            }
        }
        if (*abort_flag && lane == 0)  // nobody may have waited for these: no load outlives the CTA
            for (; in_flight > 0; --in_flight) {
                if (slot == 0) { slot = C::STAGES; phase ^= 1; }
                --slot;
                tc::mbar_wait(&full[slot], phase);
            }
        __syncwarp();
    } else if (warp == WARP_MMA) {
        int slot = 0, buf = 0;
        uint32_t phase = 0, acc_phase = 0;
        int last = -1;
        uint32_t last_phase = 0;
        for (int u = blockIdx.x; u < total && !*abort_flag; u += gridDim.x) {
            const Unit t = walk.at(u);
            if (t.steps == 0) continue;  // zeros: no sums to wait for
            const uint32_t n16 = (uint32_t)(t.n + 15) & ~15u;
            const uint32_t idesc = g.idesc | (n16 >> 3) << 17 | (128u >> 4) << 24;
            bool ok = warp_wait(&acc_empty[buf], acc_phase ^ 1, abort_flag, g.status);
            for (int s = 0; s < t.steps && ok; ++s) {
                ok = warp_wait(&full[slot], phase, abort_flag, g.status);
                if (!ok) break;
                if (lane == 0) {
                    tc::tc_fence_after();
                    const uint32_t sa = tc::smem_u32(smem + slot * C::STAGE), sb = sa + C::P_BYTES;
                    const uint64_t da = MODE == FWD ? tc::sdesc_kmajor_sw128(sa) : sdesc_across(sa);
                    const uint64_t db = tc::sdesc_kmajor_sw128(sb);
                    constexpr int SA = MODE == FWD ? 2 : 128, SB = 2;  // of 16 values, in 16 bytes
#pragma unroll
                    for (int k = 0; k < STEP / 16; ++k)
                        tc::mma_f16(tm + buf * NT, da + SA * k, db + SB * k, idesc, s > 0 || k > 0);
                    tc::mma_commit(&empty[slot]);
                }
                __syncwarp();
                last = slot;
                last_phase = phase;
                if (++slot == C::STAGES) { slot = 0; phase ^= 1; }
            }
            if (!ok) break;
            if (lane == 0) tc::mma_commit(&acc_full[buf]);
            __syncwarp();
            if (++buf == 2) { buf = 0; acc_phase ^= 1; }
        }
        if (*abort_flag && last >= 0 && lane == 0)  // no product outlives the accumulators
            tc::mbar_wait(&empty[last], last_phase);
        __syncwarp();
    } else if (warp > WARP_MMA) {
        const int gw = warp - WARP_MMA - 1, turn = gw / GATHER_SHARE, share = gw % GATHER_SHARE;
        int it = 0;
        for (int u = blockIdx.x; u < total && !*abort_flag; u += gridDim.x) {
            const Unit t = walk.at(u);
            // lane j has the group share + 4 j of the tile
            const int group = share + GATHER_SHARE * lane;
            const bool mine = lane < NT / (4 * GATHER_SHARE) && group * 4 < t.n;
            GatherRows rows;
            if (t.steps > 0 && mine) {
                rows.read(g, t.q0, t.n, group);
                rows.to_rows(g);
            }
            for (int s = 0; s < t.steps; ++s, ++it) {
                if (it % GATHER_TURNS != turn) continue;
                const int slot = it % C::STAGES;
                if (!warp_wait(&empty[slot], (it / C::STAGES & 1) ^ 1, abort_flag, g.status)) break;
                if (mine)
                    tma_gather4(smem + slot * C::STAGE + C::P_BYTES + group * 512, &map_q, &full[slot], s * STEP, rows);
                __syncwarp();
            }
        }
    } else {
        const int quad = warp & 3, half = warp >> 2;
        uint8_t* const stage = smem + C::OUT_OFF + warp * STAGE_OUT;
        int buf = 0;
        uint32_t acc_phase = 0;
        for (int u = blockIdx.x; u < total && !*abort_flag; u += gridDim.x) {
            const Unit t = walk.at(u);
            const int l0 = t.l0 + quad * 32;
            if (t.steps > 0) {
                if (!warp_wait(&acc_full[buf], acc_phase, abort_flag, g.status)) break;
                tc::tc_fence_after();
            }
            for (int c = half * 32; c < t.n; c += 64) {
                uint32_t r[32];
                if (t.steps > 0) {
                    tmem_ld32(tm + ((uint32_t)(quad * 32) << 16) + buf * NT + c, r);
                    tc::tmem_ld_wait();
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) r[j] = 0;
                }
                put<MODE>(g, stage, t.e, l0, t.q0 + c, t.n - c, lane, r);
            }
            if (t.steps > 0) {
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&acc_empty[buf]);
                if (++buf == 2) { buf = 0; acc_phase ^= 1; }
            }
        }
    }
    __syncwarp();
    pdl_trigger();
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (warp == WARP_MMA) tc::tmem_dealloc(tm, C::TMEM_COLS);
}

// Rows of 16-bit values laid out for TMA: rows that start off the 16-byte
// boundaries, and rows of x in expert order.  A warp takes a row; a lane loads
// aligned pieces of 16 bytes, only such as hold values of the row, and takes what
// lies in the next piece from its neighbour.
struct RowCopy {
    const uint16_t* x;
    int64_t rows, inner, ld, outer;  // row r: (r / inner) * outer + (r % inner) * ld
    const int32_t* pairs;            // or the row of x of a slot
    int k, x_rows;
    int cols;
    uint16_t* to;
    int64_t ldt;
};
__device__ __forceinline__ uint4 shifted(uint4 v, uint4 w, int words, bool half) {
    uint32_t a, b, c, d, e;
    switch (words) {
        case 0: a = v.x; b = v.y; c = v.z; d = v.w; e = w.x; break;
        case 1: a = v.y; b = v.z; c = v.w; d = w.x; e = w.y; break;
        case 2: a = v.z; b = v.w; c = w.x; d = w.y; e = w.z; break;
        default: a = v.w; b = w.x; c = w.y; d = w.z; e = w.w; break;
    }
    if (!half) return make_uint4(a, b, c, d);
    return make_uint4(__byte_perm(a, b, 0x5432), __byte_perm(b, c, 0x5432), __byte_perm(c, d, 0x5432), __byte_perm(d, e, 0x5432));
}
__global__ void __launch_bounds__(256) copy_rows_kernel(const RowCopy c) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    constexpr int U = 4;  // pieces of a lane on their way
    for (int64_t r = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); r < c.rows; r += (int64_t)gridDim.x * 8) {
        const uint16_t* from;
        if (c.pairs) {
            const int p = c.pairs[r], t = p >= 0 ? p / c.k : c.x_rows;
            from = t < c.x_rows ? c.x + t * c.ld : nullptr;
        } else {
            from = c.x + r / c.inner * c.outer + r % c.inner * c.ld;
        }
        uint16_t* const to = c.to + r * c.ldt;
        const int pieces = (c.cols + 7) / 8;
        if (!from) {
            for (int i = lane; i < pieces; i += 32) *reinterpret_cast<uint4*>(to + i * 8) = make_uint4(0, 0, 0, 0);
            continue;
        }
        const int shift = (int)(reinterpret_cast<uintptr_t>(from) & 15);  // bytes
        const uint4* const base = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(from) - shift);
        const int there = (shift + c.cols * 2 + 15) / 16;  // pieces that hold values of the row
        for (int i0 = lane; i0 - lane < pieces; i0 += 32 * U) {
            uint4 v[U + 1];
#pragma unroll
            for (int j = 0; j < U; ++j) v[j] = i0 + j * 32 < there ? base[i0 + j * 32] : make_uint4(0, 0, 0, 0);
            if (shift) {
                // lane 31's neighbour is lane 0's next piece
                v[U] = lane == 0 && i0 + U * 32 < there ? base[i0 + U * 32] : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int j = 0; j < U; ++j) {
                    const uint4 mine = lane == 0 ? v[j + 1] : v[j];  // what the lane below wants
                    uint4 w;
                    w.x = __shfl_sync(0xFFFFFFFFu, mine.x, (lane + 1) & 31);
                    w.y = __shfl_sync(0xFFFFFFFFu, mine.y, (lane + 1) & 31);
                    w.z = __shfl_sync(0xFFFFFFFFu, mine.z, (lane + 1) & 31);
                    w.w = __shfl_sync(0xFFFFFFFFu, mine.w, (lane + 1) & 31);
                    if (i0 + j * 32 < pieces)
                        *reinterpret_cast<uint4*>(to + (i0 + j * 32) * 8) = shifted(v[j], w, shift >> 2, shift & 2);
                }
            } else {
#pragma unroll
                for (int j = 0; j < U; ++j)
                    if (i0 + j * 32 < pieces) *reinterpret_cast<uint4*>(to + (i0 + j * 32) * 8) = v[j];
            }
        }
    }
}

// ------------------------------------------------------------------ host side

// A matrix of 16-bit values, or one for each expert.
struct Mat {
    const void* p;
    int64_t rows, cols, ld, experts, stride;
};

inline size_t padded(int64_t rows, int64_t cols) { return ((size_t)rows * (size_t)((cols + 7) / 8 * 8) * 2 + 255) / 256 * 256; }
inline bool fits(const Mat& m) {
    return aligned16(m.p) && (m.rows == 1 || m.ld % 8 == 0) && (m.experts == 1 || m.stride % 8 == 0);
}

// Copies m (or its rows in the order of pairs) into the workspace.
static int copy_rows(Mat& m, const int32_t* pairs, int64_t P, int k, uint8_t*& ws, size_t& left, cudaStream_t st) {
    const int64_t rows = pairs ? P : m.rows * m.experts, ld = (m.cols + 7) / 8 * 8;
    const size_t need = padded(rows, m.cols);
    if (need > left) return QMOE_ERR_ARG;
    const RowCopy c = {static_cast<const uint16_t*>(m.p), rows, m.rows, m.ld, m.stride, pairs, k, (int)(pairs ? m.rows : 0),
                       (int)m.cols, reinterpret_cast<uint16_t*>(ws), ld};
    const int64_t grid = (rows + 7) / 8, most = 32 * row::kSMs;
    const int rc = launch_pdl(copy_rows_kernel, dim3((unsigned)(grid < most ? grid : most)), dim3(256), 0, st, c);
    m.p = ws;
    m.ld = ld;
    m.stride = ld * m.rows;
    if (pairs) m.rows = P;
    ws += need;
    left -= need;
    return rc;
}
static int as_tma(Mat& m, uint8_t*& ws, size_t& left, cudaStream_t st) {
    if (!fits(m)) return copy_rows(m, nullptr, 0, 0, ws, left, st);
    if (m.ld % 8) m.ld = (m.cols + 7) / 8 * 8;  // a single row: the stride is not used
    return QMOE_OK;
}

static int map_of(CUtensorMap* map, const Mat& m, int dtype, int box_cols, int box_rows, bool three) {
    EncodeTiledFn enc = encode_tiled_fn();
    if (!enc) return QMOE_ERR_CUDA;
    const cuuint64_t dim[3] = {(cuuint64_t)m.cols, (cuuint64_t)m.rows, (cuuint64_t)m.experts};
    const cuuint64_t stride[2] = {(cuuint64_t)m.ld * 2, (cuuint64_t)(m.experts > 1 ? m.stride : m.ld * m.rows) * 2};
    const cuuint32_t box[3] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows, 1};
    const cuuint32_t one[3] = {1, 1, 1};
    return enc(map, dtype == QMOE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
               three ? 3 : 2, const_cast<void*>(m.p), dim, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? QMOE_OK
               : QMOE_ERR_UNSUPPORTED;
}

template <int MODE, int NT, bool GATHER>
static int launch(const CUtensorMap& mp, const CUtensorMap& mq, const Args& g, int64_t most, cudaStream_t st) {
    using C = Cfg<MODE, NT>;
    const int rc = row::allow_smem<expert_gemm_kernel<MODE, NT, GATHER>>(C::SMEM);
    if (rc != QMOE_OK) return rc;
    const int64_t grid = most < row::kSMs ? most : row::kSMs;
    return launch_pdl(expert_gemm_kernel<MODE, NT, GATHER>, dim3((unsigned)grid), dim3(threads_of(GATHER)), (size_t)C::SMEM, st, mp, mq,
                      g);
}

// Few rows for each expert: narrow tiles, whose stages are almost all weight, so that more of them are in flight.
// Gathered rows of x are read as they lie for few rows an expert; for many they are
// laid out in expert order first: a tile's rows are read again for every 256
// outputs, and TMA's gather of four rows takes as long as a box of 128 (8192 x 8
// rows of 4096, 2816 outputs: 1136 us gathered in the product, 960 laid out).
inline int tile_of(int64_t P, int E) {
    const int64_t touched = P < E ? P : E;
    return P <= 16 * touched ? 32 : P <= 96 * touched ? 128 : 256;
}

template <int MODE, bool GATHER>
static int run_rows(Mat w, Mat q, Args& g, int dtype, cudaStream_t st) {
    const int nt = tile_of(g.P, g.E), lt = nt == 256 ? 256 : 128;
    CUtensorMap mp, mq;
    int rc = MODE == FWD ? map_of(&mp, w, dtype, STEP, 128, true) : map_of(&mp, w, dtype, 64, STEP, true);
    if (rc != QMOE_OK) return rc;
    rc = map_of(&mq, q, dtype, STEP, GATHER ? 1 : nt == 256 ? 128 : Q_BOX, false);
    if (rc != QMOE_OK) return rc;
    // no more units than this, whatever the offsets
    const int64_t parts = (g.P < g.E ? g.P : g.E) + 1 + g.P / nt, most = parts * ((g.lanes + lt - 1) / lt);
    if (most >= (1ll << 31)) return QMOE_ERR_UNSUPPORTED;
    switch (nt) {
        case 32: return launch<MODE, 32, GATHER>(mp, mq, g, most, st);
        case 128: return launch<MODE, 128, GATHER>(mp, mq, g, most, st);
        default: return GATHER ? QMOE_ERR_UNSUPPORTED : launch_pair<MODE>(mp, mq, g, most, st);
    }
}

constexpr int64_t kMost = 1ll << 30;

struct Call {
    int64_t P, N, K;
    int E, dtype;
    const int32_t *offsets, *pairs;
    int k;
    int64_t x_rows;
    int32_t* status;
};
static int check(const Call& c) {
    if (c.P < 0 || c.E <= 0 || c.N <= 0 || c.K <= 0 || (c.dtype != QMOE_BF16 && c.dtype != QMOE_F16)) return QMOE_ERR_ARG;
    if (c.pairs && (c.k <= 0 || c.x_rows < 0 || !row::type_aligned(c.pairs, 4))) return QMOE_ERR_ARG;
    if (c.P > kMost || c.N > kMost || c.K > kMost || c.E > MAX_E || (c.pairs && c.x_rows > kMost)) return QMOE_ERR_UNSUPPORTED;
    return QMOE_OK;
}
static bool mat_ok(const Mat& m, int size) {
    return m.p && row::type_aligned(m.p, size) && m.ld >= m.cols && m.ld < (1ll << 38) &&
           (m.experts == 1 || (m.stride >= m.ld * (m.rows - 1) + m.cols && m.stride < (1ll << 38)));
}
static bool word_ok(const void* p) { return p && row::type_aligned(p, 4); }

}  // namespace eg
}  // namespace qmoe

using namespace qmoe;

extern "C" size_t qmoe_expert_copy_bytes(int64_t rows, int64_t cols) {
    if (rows <= 0 || cols <= 0) return 0;
    return eg::padded(rows, cols);
}

extern "C" size_t qmoe_expert_gather_bytes(int64_t P, int E, int64_t K, int dw) {
    if (P <= 0 || E <= 0 || K <= 0 || (!dw && eg::tile_of(P, E) < 256)) return 0;
    return eg::padded(P, K);
}

extern "C" int qmoe_expert_linear(int64_t P, int E, int64_t N, int64_t K, int dtype, const void* x, int64_t ldx,
                                  int64_t x_rows, const int32_t* pairs, int k, const void* w, int64_t ldw, int64_t w_expert,
                                  const int32_t* offsets, void* y, int y_dtype, int64_t ldy, int32_t* dev_status, void* ws,
                                  size_t ws_bytes, qmoe_stream_t stream) {
    const eg::Call c = {P, N, K, E, dtype, offsets, pairs, k, x_rows, dev_status};
    int rc = eg::check(c);
    if (rc != QMOE_OK) return rc;
    if ((y_dtype != dtype && y_dtype != QMOE_F32) || ldy < N) return QMOE_ERR_ARG;
    if (P == 0) return QMOE_OK;
    if (pairs && x_rows == 0) return QMOE_ERR_ARG;
    eg::Mat mw = {w, N, K, ldw, E, w_expert}, mx = {x, pairs ? x_rows : P, K, ldx, 1, 0};
    if (!eg::mat_ok(mw, 2) || !eg::mat_ok(mx, 2) || !eg::word_ok(offsets) || !y ||
        !row::type_aligned(y, row::dtype_size(y_dtype)) || !eg::word_ok(dev_status))
        return QMOE_ERR_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    uint8_t* at = static_cast<uint8_t*>(ws);
    size_t left = ws && !(reinterpret_cast<uintptr_t>(ws) & 255u) ? ws_bytes : 0;
    if ((rc = eg::as_tma(mw, at, left, st)) != QMOE_OK) return rc;
    const bool lay_out = pairs && qmoe_expert_gather_bytes(P, E, K, 0);
    rc = lay_out ? eg::copy_rows(mx, pairs, P, k, at, left, st) : eg::as_tma(mx, at, left, st);
    if (rc != QMOE_OK) return rc;
    if (lay_out) pairs = nullptr;
    const int size = row::dtype_size(y_dtype);
    eg::Args g = {(int)P, E, (int)N, 0, (int)K, offsets, pairs, k, (int)mx.rows, y, ldy, 0, y_dtype,
                  aligned16(y) && ldy * size % 16 == 0,
                  dtype == QMOE_BF16 ? tc::idesc_bf16_f32(0, 0) : tc::idesc_f16_f32(0, 0), dev_status};
    return pairs ? eg::run_rows<eg::FWD, true>(mw, mx, g, dtype, st) : eg::run_rows<eg::FWD, false>(mw, mx, g, dtype, st);
}

extern "C" int qmoe_expert_linear_dx(int64_t P, int E, int64_t N, int64_t K, int dtype, const void* dy, int64_t lddy,
                                     const void* w, int64_t ldw, int64_t w_expert, const int32_t* offsets, void* dx,
                                     int dx_dtype, int64_t lddx, int32_t* dev_status, void* ws, size_t ws_bytes,
                                     qmoe_stream_t stream) {
    const eg::Call c = {P, N, K, E, dtype, offsets, nullptr, 0, 0, dev_status};
    int rc = eg::check(c);
    if (rc != QMOE_OK) return rc;
    if ((dx_dtype != dtype && dx_dtype != QMOE_F32) || lddx < K) return QMOE_ERR_ARG;
    if (P == 0) return QMOE_OK;
    eg::Mat mw = {w, N, K, ldw, E, w_expert}, my = {dy, P, N, lddy, 1, 0};
    if (!eg::mat_ok(mw, 2) || !eg::mat_ok(my, 2) || !eg::word_ok(offsets) || !dx ||
        !row::type_aligned(dx, row::dtype_size(dx_dtype)) || !eg::word_ok(dev_status))
        return QMOE_ERR_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    uint8_t* at = static_cast<uint8_t*>(ws);
    size_t left = ws && !(reinterpret_cast<uintptr_t>(ws) & 255u) ? ws_bytes : 0;
    if ((rc = eg::as_tma(mw, at, left, st)) != QMOE_OK || (rc = eg::as_tma(my, at, left, st)) != QMOE_OK) return rc;
    const int size = row::dtype_size(dx_dtype);
    eg::Args g = {(int)P, E, (int)K, 0, (int)N, offsets, nullptr, 0, (int)P, dx, lddx, 0, dx_dtype,
                  aligned16(dx) && lddx * size % 16 == 0,
                  (dtype == QMOE_BF16 ? tc::idesc_bf16_f32(0, 0) : tc::idesc_f16_f32(0, 0)) | 1u << 15, dev_status};
    return eg::run_rows<eg::DX, false>(mw, my, g, dtype, st);
}

extern "C" int qmoe_expert_linear_dw(int64_t P, int E, int64_t N, int64_t K, int dtype, const void* dy, int64_t lddy,
                                     const void* x, int64_t ldx, int64_t x_rows, const int32_t* pairs, int k,
                                     const int32_t* offsets, void* dw, int dw_dtype, int32_t* dev_status, void* ws,
                                     size_t ws_bytes, qmoe_stream_t stream) {
    const eg::Call c = {P, N, K, E, dtype, offsets, pairs, k, x_rows, dev_status};
    int rc = eg::check(c);
    if (rc != QMOE_OK) return rc;
    if (dw_dtype != dtype && dw_dtype != QMOE_F32) return QMOE_ERR_ARG;
    if (!eg::word_ok(offsets) || !dw || !row::type_aligned(dw, row::dtype_size(dw_dtype)) || !eg::word_ok(dev_status))
        return QMOE_ERR_ARG;
    const int64_t units = (int64_t)E * ((N + 255) / 256) * ((K + 255) / 256);
    if (units >= (1ll << 31)) return QMOE_ERR_UNSUPPORTED;
    const int size = row::dtype_size(dw_dtype);
    cudaStream_t st = (cudaStream_t)stream;
    if (P == 0)
        return cudaMemsetAsync(dw, 0, (size_t)E * N * K * size, st) == cudaSuccess ? QMOE_OK : QMOE_ERR_LAUNCH;
    if (pairs && x_rows == 0) return QMOE_ERR_ARG;
    eg::Mat my = {dy, P, N, lddy, 1, 0}, mx = {x, pairs ? x_rows : P, K, ldx, 1, 0};
    if (!eg::mat_ok(my, 2) || !eg::mat_ok(mx, 2)) return QMOE_ERR_ARG;
    uint8_t* at = static_cast<uint8_t*>(ws);
    size_t left = ws && !(reinterpret_cast<uintptr_t>(ws) & 255u) ? ws_bytes : 0;
    if ((rc = eg::as_tma(my, at, left, st)) != QMOE_OK) return rc;
    rc = pairs ? eg::copy_rows(mx, pairs, P, k, at, left, st) : eg::as_tma(mx, at, left, st);
    if (rc != QMOE_OK) return rc;
    eg::Args g = {(int)P, E, (int)N, (int)K, 0, offsets, nullptr, 0, (int)mx.rows, dw, K, N * K, dw_dtype,
                  aligned16(dw) && K * size % 16 == 0,
                  (dtype == QMOE_BF16 ? tc::idesc_bf16_f32(0, 0) : tc::idesc_f16_f32(0, 0)) | 3u << 15, dev_status};
    CUtensorMap mp, mq;
    rc = eg::map_of(&mp, my, dtype, 64, eg::STEP, false);
    if (rc != QMOE_OK) return rc;
    rc = eg::map_of(&mq, mx, dtype, 64, eg::STEP, false);
    if (rc != QMOE_OK) return rc;
    return eg::launch_pair<eg::DW>(mp, mq, g, units, st);
}
