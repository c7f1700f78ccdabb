// Products of the routed experts' rows with 16-bit weights, and their
// gradients (qmoe_expert_linear, qmoe_expert_linear_dx, qmoe_expert_linear_dw):
//
//   y[s][n]     = sum_k w[e][n][k] x[s][k]      for the rows s of expert e
//   dx[s][k]    = sum_n w[e][n][k] dy[s][n]
//   dw[e][n][k] = sum_s dy[s][n] x[s][k]
//
// Persistent kernels.  The lanes of a tile are outputs of the layer (y), its inputs
// (dx) or rows of dw; the columns are rows s (y, dx: a tile is no wider than its
// expert has rows, to the next 16) or columns of dw.  An operand whose reduction axis
// is contiguous in memory (w and x for y, dy for dx) is read as such; the others (w
// for dx, both for dw) lie in shared memory as they do in HBM, reduction rows of 64
// values, and the tensor core transposes them as it reads.
//
// Many rows an expert, and dw: 256 x 256 tiles of two CTAs (expert_gemm_pair.cu).
// Here: y and dx for fewer, 128 lanes and up to 32 or 128 columns (tile_of), so that the
// ring holds mostly weights, which bound it: 1024 pairs over 128 experts 2048 -> 1536
// 131 us, 6.1 TB/s; 64 x 16 rows 4096 -> 2816 230 us, 6.4 TB/s.  One token x 8 of
// 128 experts (50 MB) 15 us: 2.4 until the first load, 1.5 its latency, 9 the
// weights at 5.3 TB/s, 1.2 the stores.
#include <cmath>

#include "expert_gemm.cuh"

namespace qmoe {
namespace eg {

// Warps: the epilogue's, two that load tiles and two that issue products, each pair
// taking the steps in turn (each of the two that issue has a sum of its own), then
// those that gather.  With one warp of each: 16 tokens x 2 of 8 experts 4096 -> 2816
// 40.5 us for 38.4, one row 4096 -> 4096 14.9 for 14.0, but one token x 8 of 128
// experts 14.5 for 15.0.
constexpr int TURNS = 2, WARP_TMA = 8, WARP_MMA = WARP_TMA + TURNS, WARP_GATHER = WARP_MMA + TURNS;
constexpr int PIECE = TURNS * LONG;  // steps of a piece of a long sum
constexpr int threads_of(bool gather) { return (WARP_GATHER + (gather ? GATHER_WARPS : 0)) * 32; }

template <int MODE, int NT>
struct Cfg {
    static constexpr int P_BYTES = 128 * STEP * 2, Q_BYTES = NT * STEP * 2, STAGE = P_BYTES + Q_BYTES;
    static constexpr int TMEM_COLS = 2 * TURNS * NT;  // two tiles' sums of each warp that issues
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
    static_assert(TURNS == 2 && STAGES % TURNS == 0, "a stage has one warp that loads it and one that issues its products");
};

// What a CTA works on: whole tiles in turn; or, SPLIT, its even share of the steps
// of all tiles in one piece, so that few tiles keep all SMs busy.  The sums of a
// tile that starts or ends within the share go to the workspace, in fp32, and
// join_kernel adds the parts of a tile in the CTAs' order.
struct Segment {
    Unit t;
    int s0, s1;  // steps
    int part;    // -1: the whole tile; 0: it starts before the share, 1: it ends behind it
};
template <int MODE, int NT, bool SPLIT>
struct Segments {
    Walk<128, 16> walk;
    int64_t at, end;  // steps (SPLIT)
    // Of at least LEAST steps: a tile in many short parts takes longer to join than the steps do.  `each` is a share's
    // length, the first `more` have one step more.
    static constexpr int LEAST = 6;
    int64_t each;
    int more, ctas;
    int u, total, per;
    __device__ Segments(const Args& g, const int* off, const int* base) : walk(g, off, base, NT) {
        total = base[g.E + 1];
        per = g.steps;
        u = (SPLIT ? base[g.E] : 0) + blockIdx.x;
        if (SPLIT) {
            const int64_t steps = (int64_t)base[g.E] * per;
            ctas = (int)max((int64_t)1, min((int64_t)gridDim.x, steps / LEAST));
            each = steps < (1ll << 32) ? (uint32_t)steps / ctas : steps / ctas;
            more = (int)(steps - each * ctas);
            at = share(min((int)blockIdx.x, ctas));
            end = share(min((int)blockIdx.x + 1, ctas));
        }
    }
    __device__ __forceinline__ int64_t share(int i) const { return i * each + min(i, more); }
    __device__ __forceinline__ bool next(Segment& s) {
        if (SPLIT && at < end) {
            const int unit = (int)(at < (1ll << 32) ? (uint32_t)at / (uint32_t)per : at / per);
            s.t = walk.at(unit);
            s.s0 = (int)(at - (int64_t)unit * per);
            s.s1 = (int)min((int64_t)per, s.s0 + (end - at));
            s.part = s.s0 > 0 ? 0 : s.s1 < per ? 1 : -1;
            at += s.s1 - s.s0;
            return true;
        }
        if (u >= total) return false;
        s.t = walk.at(u);
        s.s0 = 0;
        s.s1 = s.t.steps;
        s.part = -1;
        u += gridDim.x;
        return true;
    }
    // CTAs after this one that have a part of the tile that it leaves unfinished
    __device__ __forceinline__ int others(const Segment& s) const {
        const int64_t last = end + per - s.s1;
        int n = 1;
        while ((int)blockIdx.x + n + 1 < ctas && share(blockIdx.x + n + 1) < last) ++n;
        return n;
    }
};

template <int MODE, int NT, bool GATHER, bool SPLIT, bool BY>
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
    if (threadIdx.x == 32) {
        tc::prefetch_tensormap(&map_p);
        tc::prefetch_tensormap(&map_q);
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::STAGES; ++i) {
            tc::mbar_init(&full[i], 1 + (GATHER ? GATHER_SHARE : 0));
            tc::mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&acc_full[i], TURNS);
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
    __shared__ int slot_rows[GATHER ? FEW_SLOTS : 1];
    if (GATHER && g.P <= FEW_SLOTS && threadIdx.x < g.P) slot_rows[threadIdx.x] = row_of(g, g.pairs[threadIdx.x]);
    read_offsets<128, NT, false>(g, off, base);
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tm = *tmem_at;
    Segments<MODE, NT, SPLIT> segments(g, off, base);
    Segment seg;
    const Unit& t = seg.t;
    if (SPLIT) pdl_trigger();  // join_kernel needs little, and waits

    if (warp >= WARP_TMA && warp < WARP_MMA) {
        int it = 0;
        while (!*abort_flag && segments.next(seg)) {
            const int boxes = GATHER ? 0 : (t.n + Q_BOX - 1) / Q_BOX;
            for (int s = seg.s0; s < seg.s1; ++s, ++it) {
                if (it % TURNS != warp - WARP_TMA) continue;
                const int slot = it % C::STAGES;
                if (!warp_wait(&empty[slot], (it / C::STAGES & 1) ^ 1, abort_flag, g.status)) break;
                uint8_t* st = smem + slot * C::STAGE;
                const int second = s >= g.per, k0 = (s - (second ? g.per : 0)) * STEP, z = t.e + second;
                if (lane == 0) {
                    tc::mbar_arrive_expect_tx(&full[slot], C::P_BYTES + (GATHER ? (t.n + 3) / 4 * 512 : boxes * Q_BOX * 128));
                    if constexpr (MODE == FWD) {
                        tc::tma_load_3d(st, &map_p, &full[slot], k0, t.l0, z);
                    } else {
                        tc::tma_load_3d(st, &map_p, &full[slot], t.l0, k0, z);
                        tc::tma_load_3d(st + 8192, &map_p, &full[slot], t.l0 + 64, k0, z);
                    }
                }
                __syncwarp();
                if (lane < boxes)
                    tc::tma_load_2d(st + C::P_BYTES + lane * Q_BOX * 128, &map_q, &full[slot], k0, t.q0 + lane * Q_BOX);
                __syncwarp();
            }
        }
        __syncwarp();
    } else if (warp >= WARP_MMA && warp < WARP_GATHER) {
        const int turn = warp - WARP_MMA;
        int it = 0, buf = 0;
        uint32_t acc_phase = 0;
        bool ok = true;  // after a wait that ran out no more products are issued and no more stages let go
        while (ok && segments.next(seg)) {
            if (seg.s1 == 0) continue;  // zeros: no sums to wait for
            const uint32_t n16 = (uint32_t)(t.n + 15) & ~15u;
            const uint32_t idesc = g.idesc | (n16 >> 3) << 17 | (128u >> 4) << 24;
            const int end = it + seg.s1 - seg.s0;
            while (it < end) {  // pieces of the sum, each in an accumulator of its own
                const uint32_t d = tm + (buf * TURNS + turn) * NT;
                if (!(ok = issue_wait(&acc_empty[buf], acc_phase ^ 1, abort_flag, g.status))) break;
                // every second step, a sum of its own: by the steps' count from the first tile's on, so that a stage is always one
                // warp's.  By turns within a tile, odd ones gave a stage to the other warp, which took a load that was two rounds
                // behind for one that had come: the parity of a barrier does not tell them apart.
                const int last = min(it + PIECE, end);
                uint32_t more = 0;
#pragma unroll 1
                for (int i = it + ((it ^ turn) & 1); i < last; i += TURNS) {
                    const int slot = i % C::STAGES;
                    if (!(ok = issue_wait(&full[slot], i / C::STAGES & 1, abort_flag, g.status))) break;
                    tc::tc_fence_after();
                    const uint32_t sa = tc::smem_u32(smem) + slot * C::STAGE, sb = sa + C::P_BYTES;
                    const uint64_t da = MODE == FWD ? tc::sdesc_kmajor_sw128(sa) : sdesc_across(sa);
                    const uint64_t db = tc::sdesc_kmajor_sw128(sb);
                    constexpr int SA = MODE == FWD ? 2 : 128, SB = 2;  // of 16 values, in 16 bytes
#pragma unroll
                    for (int k = 0; k < STEP / 16; ++k) tc::mma_f16_elect(d, da + SA * k, db + SB * k, idesc, k > 0 ? 1 : more);
                    tc::mma_commit_elect(&empty[slot]);
                    more = 1;
                }
                if (!ok) break;
                it = last;
                tc::mma_commit_elect(&acc_full[buf]);
                if (++buf == 2) { buf = 0; acc_phase ^= 1; }
            }
        }
        __syncwarp();
    } else if (warp >= WARP_GATHER) {
        const int gw = warp - WARP_GATHER, turn = gw / GATHER_SHARE, share = gw % GATHER_SHARE;
        int it = 0;
        while (!*abort_flag && segments.next(seg)) {
            // lane j has the group share + 4 j of the tile
            const int group = share + GATHER_SHARE * lane;
            const bool mine = lane < NT / (4 * GATHER_SHARE) && group * 4 < t.n;
            GatherRows rows;
            if (seg.s1 > 0 && mine) {
                if (g.P <= FEW_SLOTS) {
                    rows.take(g, slot_rows, t.q0, t.n, group);
                } else {
                    rows.read(g, t.q0, t.n, group);
                    rows.to_rows(g);
                }
            }
            for (int s = seg.s0; s < seg.s1; ++s, ++it) {
                if (it % GATHER_TURNS != turn) continue;
                const int slot = it % C::STAGES;
                if (!warp_wait(&empty[slot], (it / C::STAGES & 1) ^ 1, abort_flag, g.status)) break;
                if (mine)
                    tma_gather4(smem + slot * C::STAGE + C::P_BYTES + group * 512, &map_q, &full[slot], s * STEP, rows);
                __syncwarp();
                // A warp arrives also where none of the tile's rows are its own (12 rows and fewer).  Only with bytes to bring it
                // would be kept in step by them, and one without, a round behind, took empty's parity for the round it waited for,
                // and at the end waited for one that did not come.
                if (lane == 0) tc::mbar_arrive(&full[slot]);
            }
        }
    } else {
        const int quad = warp & 3, half = warp >> 2;
        int4 join = make_int4(0, 0, 0, 0);
        const bool matrices = by_matrices<MODE>(g);
        uint8_t* const stage = smem + C::OUT_OFF + warp * STAGE_OUT;
        int buf = 0, it = 0;
        uint32_t acc_phase = 0;
        while (!*abort_flag && segments.next(seg)) {
            const int l0 = t.l0 + quad * 32;
            if (SPLIT && seg.part == 1) join = make_int4(t.l0, t.q0, t.n, segments.others(seg));
            // where a sum lies in its accumulator: with the warp that has the first step, and (two) the other's
            const uint32_t all = tm + ((uint32_t)(quad * 32) << 16), one = (it & 1) * NT, other = (~it & 1) * NT;
            const int steps = seg.s1 - seg.s0;
            bool two = steps > 1, ok = true;
            if (seg.s1 > 0) {
                if (!warp_wait(&acc_full[buf], acc_phase, abort_flag, g.status)) break;
                tc::tc_fence_after();
#pragma unroll 1
                for (int left = steps - PIECE; left > 0; left -= PIECE) {
                    // the sum so far is added to the next piece's, in TMEM, and its accumulator let go
                    const int before = buf;
                    if (++buf == 2) { buf = 0; acc_phase ^= 1; }
                    if (!(ok = warp_wait(&acc_full[buf], acc_phase, abort_flag, g.status))) break;
                    tc::tc_fence_after();
#pragma unroll 1
                    for (int h = half * 32; h < t.n; h += h & 16 ? 48 : 16) {  // 16 columns at a time: few registers
                        const uint32_t from = all + before * TURNS * NT + h, to = all + buf * TURNS * NT + h;
                        uint32_t r[16], x[16];
                        auto plus = [&](uint32_t at) {
                            tc::tmem_ld_32x32b_x16(at, x);
                            tc::tmem_ld_wait();
#pragma unroll
                            for (int j = 0; j < 16; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) + __uint_as_float(x[j]));
                        };
                        tc::tmem_ld_32x32b_x16(from + one, r);
                        if (two) plus(from + other);
                        plus(to + one);
                        if (left > 1) plus(to + other);
                        tc::tmem_st_32x32b_x16(to + one, r);
                    }
                    tc::tmem_st_wait();
                    tc::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&acc_empty[before]);
                    two = false;
                }
                if (!ok) break;
            }
            for (int c = half * 32; c < t.n; c += 64) {
                uint32_t r[32];
                const bool part = SPLIT && seg.part >= 0;
                if (seg.s1 > 0) {
                    const uint32_t from = all + buf * TURNS * NT + c;
                    take<MODE>(matrices && !part, from + one, r);
                    tc::tmem_ld_wait();
                    if (two) {
                        uint32_t y[32];
                        take<MODE>(matrices && !part, from + other, y);
                        tc::tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) + __uint_as_float(y[j]));
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) r[j] = 0;
                }
                if (part) {
                    float* to = g.parts + (((int64_t)blockIdx.x * 2 + seg.part) * NT + c) * 128 + quad * 32 + lane;
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (c + j < t.n) to[j * 128] = __uint_as_float(r[j]);
                } else {
                    put<MODE, false, BY>(g, nullptr, matrices, stage, t.e, l0, t.q0 + c, t.n - c, lane, r);
                }
            }
            it += steps;
            if (seg.s1 > 0) {
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&acc_empty[buf]);
                if (++buf == 2) { buf = 0; acc_phase ^= 1; }
            }
        }
        if (SPLIT && threadIdx.x == 0) g.joins[blockIdx.x] = join;
    }
    __syncwarp();
    if (!SPLIT) pdl_trigger();
    tc::tc_fence_before();
    __syncthreads();
    wind_down(abort_flag);
    tc::tc_fence_after();
    if (warp == WARP_MMA) tc::tmem_dealloc(tm, C::TMEM_COLS);
}

// The tiles that Segments left in parts: block j has the one that starts within
// the share of CTA j and ends behind it.
template <int NT>
__global__ void __launch_bounds__(512) join_kernel(const Args g) {
    pdl_wait();
    pdl_trigger();
    const int4 t = g.joins[blockIdx.x];  // first lane, first row, rows, CTAs that go on
    const int l = threadIdx.x & 127;
    constexpr int U = 4;  // columns of a thread; the grid's y has 16 of a tile each
    const int c0 = blockIdx.y * 4 * U + (threadIdx.x >> 7) * U;
    if (c0 >= t.z) return;
    float sum[U];
#pragma unroll
    for (int j = 0; j < U; ++j) sum[j] = 0.f;
#pragma unroll 4
    for (int q = 0; q <= t.w; ++q) {
        const float* from = g.parts + (((int64_t)(blockIdx.x + q) * 2 + (q == 0)) * NT + c0) * 128 + l;
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (c0 + j < t.z) sum[j] += from[j * 128];
    }
#pragma unroll
    for (int j = 0; j < U; ++j)
        if (c0 + j < t.z && t.x + l < g.lanes)
            put_value(g.out, g.ctype, (int64_t)(t.y + c0 + j) * g.ld + t.x + l, g.by ? sum[j] * g.by[t.x + l] : sum[j]);
}

// Rows of 16-bit values laid out for TMA: rows that start off the 16-byte
// boundaries, and rows of x in expert order.  Up to a warp takes a row; a lane loads
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
    const int32_t* offsets;          // of the experts whose rows (inner of each) these are: those without rows are left out
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
template <int LANES>  // that take a row
__global__ void __launch_bounds__(256) copy_rows_kernel(const RowCopy c) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & (LANES - 1), first = (threadIdx.x & 31) & ~(LANES - 1);
    const uint32_t mask = LANES == 32 ? 0xFFFFFFFFu : ((1u << LANES) - 1) << first;
    constexpr int U = 4, ROWS = 256 / LANES;  // pieces of a lane on their way; rows of a CTA
    for (int64_t r = (int64_t)blockIdx.x * ROWS + threadIdx.x / LANES; r < c.rows; r += (int64_t)gridDim.x * ROWS) {
        const uint16_t* from;
        if (c.pairs) {
            const int p = c.pairs[r], t = p >= 0 ? p / c.k : c.x_rows;
            from = t < c.x_rows ? c.x + t * c.ld : nullptr;
        } else {
            const int64_t e = c.rows < (1ll << 31) ? (uint32_t)r / (uint32_t)c.inner : r / c.inner;
            if (c.offsets && c.offsets[e + 1] <= c.offsets[e]) continue;
            from = c.x + e * c.outer + (r - e * c.inner) * c.ld;
        }
        uint16_t* const to = c.to + r * c.ldt;
        const int pieces = (c.cols + 7) / 8;
        if (!from) {
            for (int i = lane; i < pieces; i += LANES) *reinterpret_cast<uint4*>(to + i * 8) = make_uint4(0, 0, 0, 0);
            continue;
        }
        const int shift = (int)(reinterpret_cast<uintptr_t>(from) & 15);  // bytes
        const uint4* const base = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(from) - shift);
        const int there = (shift + c.cols * 2 + 15) / 16;  // pieces that hold values of the row
        for (int i0 = lane; i0 - lane < pieces; i0 += LANES * U) {
            uint4 v[U + 1];
#pragma unroll
            for (int j = 0; j < U; ++j) v[j] = i0 + j * LANES < there ? base[i0 + j * LANES] : make_uint4(0, 0, 0, 0);
            if (shift) {
                // the last lane's neighbour is the first one's next piece
                v[U] = lane == 0 && i0 + U * LANES < there ? base[i0 + U * LANES] : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int j = 0; j < U; ++j) {
                    const uint4 mine = lane == 0 ? v[j + 1] : v[j];  // what the lane below wants
                    const int above = first + ((lane + 1) & (LANES - 1));
                    uint4 w;
                    w.x = __shfl_sync(mask, mine.x, above);
                    w.y = __shfl_sync(mask, mine.y, above);
                    w.z = __shfl_sync(mask, mine.z, above);
                    w.w = __shfl_sync(mask, mine.w, above);
                    if (i0 + j * LANES < pieces)
                        *reinterpret_cast<uint4*>(to + (i0 + j * LANES) * 8) = shifted(v[j], w, shift >> 2, shift & 2);
                }
            } else {
#pragma unroll
                for (int j = 0; j < U; ++j)
                    if (i0 + j * LANES < pieces) *reinterpret_cast<uint4*>(to + (i0 + j * LANES) * 8) = v[j];
            }
        }
    }
}

// ------------------------------------------------------------------ host side

inline size_t padded(int64_t rows, int64_t cols) { return ((size_t)rows * (size_t)((cols + 7) / 8 * 8) * 2 + 255) / 256 * 256; }
// Copies m (or its rows in the order of pairs) into the workspace.
static int copy_rows(Mat& m, const int32_t* pairs, int64_t P, int k, const int32_t* offsets, uint8_t*& ws, size_t& left,
                     cudaStream_t st) {
    const int64_t rows = pairs ? P : m.rows * m.experts, ld = (m.cols + 7) / 8 * 8;
    const size_t need = padded(rows, m.cols);
    if (need > left) return QMOE_ERR_ARG;
    const RowCopy c = {static_cast<const uint16_t*>(m.p), rows, m.rows, m.ld, m.stride, pairs, k, (int)(pairs ? m.rows : 0),
                       (int)m.cols, reinterpret_cast<uint16_t*>(ws), ld, offsets};
    // a lane for each piece of a narrow row
    const int lanes = m.cols <= 64 ? 8 : m.cols <= 128 ? 16 : 32;
    const int64_t grid = (rows * lanes + 255) / 256, most = 32 * row::kSMs;
    const int rc = launch_pdl(lanes == 8 ? copy_rows_kernel<8> : lanes == 16 ? copy_rows_kernel<16> : copy_rows_kernel<32>,
                              dim3((unsigned)(grid < most ? grid : most)), dim3(256), 0, st, c);
    m.p = ws;
    m.ld = ld;
    m.stride = ld * m.rows;
    if (pairs) m.rows = P;
    ws += need;
    left -= need;
    return rc;
}
inline size_t copy_need(const Mat& m) { return fits(m) ? 0 : padded(m.rows * m.experts, m.cols); }
static int as_tma(Mat& m, const int32_t* offsets, uint8_t*& ws, size_t& left, cudaStream_t st) {
    if (!fits(m)) return copy_rows(m, nullptr, 0, 0, offsets, ws, left, st);
    if (m.ld % 8) m.ld = (m.cols + 7) / 8 * 8;  // a single row: the stride is not used
    return QMOE_OK;
}

// store: a box's rows have 32 values, elsewhere 128 bytes.
static int map_of(CUtensorMap* map, const Mat& m, int dtype, int box_cols, int box_rows, bool three, bool store = false) {
    EncodeTiledFn enc = encode_tiled_fn();
    if (!enc) return QMOE_ERR_CUDA;
    const cuuint64_t size = (cuuint64_t)row::dtype_size(dtype);
    const cuuint64_t dim[3] = {(cuuint64_t)m.cols, (cuuint64_t)m.rows, (cuuint64_t)m.experts};
    const cuuint64_t stride[2] = {(cuuint64_t)m.ld * size, (cuuint64_t)(m.experts > 1 ? m.stride : m.ld * m.rows) * size};
    const cuuint32_t box[3] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows, 1};
    const cuuint32_t one[3] = {1, 1, 1};
    const CUtensorMapDataType type = dtype == QMOE_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                     : dtype == QMOE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                          : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    return enc(map, type, three ? 3 : 2, const_cast<void*>(m.p), dim, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
               store && size == 2 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? QMOE_OK
               : QMOE_ERR_UNSUPPORTED;
}

template <int MODE, int NT, bool GATHER, bool BY, bool SPLIT>
static int launch_as(const CUtensorMap& mp, const CUtensorMap& mq, const Args& g, int64_t most, cudaStream_t st) {
    using C = Cfg<MODE, NT>;
    const auto kernel = expert_gemm_kernel<MODE, NT, GATHER, SPLIT, BY>;
    int rc = row::allow_smem<expert_gemm_kernel<MODE, NT, GATHER, SPLIT, BY>>(C::SMEM);
    if (rc != QMOE_OK) return rc;
    const int64_t grid = SPLIT || most > row::kSMs ? row::kSMs : most;
    rc = launch_pdl(kernel, dim3((unsigned)grid), dim3(threads_of(GATHER)), (size_t)C::SMEM, st, mp, mq, g);
    if (rc != QMOE_OK || !SPLIT) return rc;
    return launch_pdl(join_kernel<NT>, dim3((unsigned)grid, NT / 16), dim3(512), 0, st, g);
}

// Columns of a tile, by the rows an expert has on average (the offsets are not known
// here).  Few: narrow tiles, whose stages are almost all weight, so that more of them
// are in flight.  Many: tiles of two CTAs.  Between 24 and 96, these for weights that take
// some 8 us to read and fill pairs' lanes about as well, in sums of some length, else
// tiles of 128; also for one matrix, whose few tiles the SMs share, which pairs do not.
// us of y with tiles of 32, 128 and 256, rows an expert: 64 experts 4096 -> 2816, 16 rows
// 230 276 261, 32 rows 233 279 262, 48 rows 296 280 264, 96 rows - 287 269; 32 experts
// 2048 -> 1536, 32 rows 38 47 44, 40 rows 48 48 44; one matrix 4096 -> 4096, 32 rows 14.3
// 16.0 21.9, 64 rows 18.4 16.4 22.2, 192 rows - 21.5 23.6; 128 and 256: 16 experts 64 ->
// 1024, 54 rows 5.5 6.4; 512 experts 256 -> 545 (640 and 768 lanes), 72 rows 42 52; 128
// experts 128 -> 1408, 62 rows 20.8 24.2.  Between 24 and 32 rows uneven loads decide
// (Zipf's law of the given exponent, largest expert): 64 experts 4096 -> 2816, 25 rows,
// 0.8, 144 rows 257 278 260, 32 rows, 1.2, 245 rows 281 279 262, all to one expert 123 66
// 42; 512 experts 2048 -> 1024, 20 rows, 1.2, 964 rows 380 390 349, 16 rows and a quarter
// of all for one 354 394 362.
//
// Gathered rows of x are read as they lie for few rows an expert; for many they are
// laid out in expert order first: a tile's rows are read again for every 256
// outputs, and TMA's gather of four rows takes as long as a box of 128 (8192 x 8
// rows of 4096, 2816 outputs: 1136 us gathered in the product, 960 laid out).
inline int tile_of(int64_t P, int E, int64_t lanes, int64_t red) {
    const int64_t touched = P < E ? P : E;
    if (touched == 1) return P <= 32 ? 32 : P <= 192 ? 128 : 256;
    if (P <= 24 * touched) return 32;
    const bool fills = (lanes + 255) / 256 * 256 * 10 <= (lanes + 127) / 128 * 128 * 11;
    return P > 96 * touched || (fills && red >= 512 && touched * lanes * red >= 20000000) ? 256 : 128;
}

// No more tiles than this, whatever the offsets.
inline int64_t most_tiles(int64_t P, int E, int64_t lanes, int nt) {
    const int lt = nt == 256 ? 256 : 128;
    return ((P < E ? P : E) + 1 + P / nt) * ((lanes + lt - 1) / lt);
}
// Whether the SMs share the steps of all tiles evenly, and a second kernel joins the
// parts, by a model of the time in us fitted to GB300: beside some 7.5 of either form
// (offsets, the first loads' latency, the last stores) a step of 64 x 128 weights takes
// 0.39 where all SMs load (HBM), 0.25 where few do; the join 2.5.  Whole and shared:
// 10 experts 4096 -> 2048 (160 tiles of 64 steps) 57 and 37 (by the model 57 and 36), 8
// experts 2048 -> 1536 (96 of 32) 15.3 and 16.3 (15.5 and 17.9), 16 experts (192 of 32)
// 26.7 and 24.4, one matrix 4096 -> 4096 (32 of 64) 21.2 and 14.7 (23.5 and 15.3), 1408
// of 2048 by 6 experts (66 of 32) 14.4 and 15.0.
inline bool split(int64_t P, int E, int64_t lanes, int64_t per, int nt) {
    if (nt == 256) return false;
    const int64_t tiles = ((P < E ? P : E) + P / nt) * ((lanes + 127) / 128);
    if (tiles > 2 * row::kSMs) return false;  // measured no faster, up to a fifth slower, with more
    const float busy = tiles < row::kSMs ? (float)tiles / row::kSMs : 1.f;
    const float whole = (float)((tiles + row::kSMs - 1) / row::kSMs) * per * (0.39f * busy > 0.25f ? 0.39f * busy : 0.25f);
    const float ctas = (float)(tiles * per / 6 < row::kSMs ? tiles * per / 6 + 1 : row::kSMs);
    const float share = (float)tiles * per / ctas;
    return share * (0.39f * ctas / row::kSMs > 0.25f ? 0.39f * ctas / row::kSMs : 0.25f) + 2.5f < whole;
}
inline size_t part_bytes(int nt) { return (size_t)row::kSMs * 2 * nt * 128 * 4 + (row::kSMs * 16 + 255) / 256 * 256; }

// Whether y is better made by expert_few_kernel, for weights off the 16-byte
// boundaries: by a model of the times in us fitted to GB300, for as many experts with
// rows as P rows spread over E by chance reach.  In place: 3 and, shared by all SMs, 16.5
// ns for each CTA of 16 rows of an expert's w and 1024 of their values, 5 ns for one
// whose row is not its expert's first.  Copied: 10, a look at every row of w, the copy of
// the experts that have rows (6 TB/s) and the product that reads it (5.3 TB/s).  In place
// and copied, tokens x experts: 1 x 8 of 128, 2047 -> 1536, 22 and 41; 4 x 8 101 and
// 104; 1 x 8, 513 -> 767, 7.5 and 18, 4 x 8 29 and 26; 16 x 7 of 256, 1095 -> 1408, 242
// and 152; 6 x 9 of 64, 1957 -> 2816, 182 and 162; 1 x 10 of 512, 4095 -> 2047, 69 and
// 131; 1, 4 and 16 rows of one matrix, 4095 -> 4096, 16 20 41 and 24 29 29.
inline bool few(int64_t P, int E, int64_t N, int64_t K) {
    if (P > 65535) return false;
    const double touched = E * (1 - std::pow(1 - 1.0 / E, (double)P)), tiles = (double)((N + 15) / 16);
    const double in_place = 3 + touched * tiles * 0.0165 * (double)((K + 1023) / 1024) + (P - touched) * tiles * 0.005;
    return in_place < 10 + 3e-5 * E * N + touched * N * K * (4 / 6e6 + 2 / 5.3e6);
}

template <int MODE, bool GATHER, bool BY>
static int run_rows(Mat w, Mat q, Args& g, int dtype, uint8_t* ws, size_t left, cudaStream_t st) {
    const int nt = tile_of(g.P, g.E, g.lanes, g.red);
    CUtensorMap mp, mq;
    int rc = MODE == FWD ? map_of(&mp, w, dtype, STEP, 128, true) : map_of(&mp, w, dtype, 64, STEP, true);
    if (rc != QMOE_OK) return rc;
    rc = map_of(&mq, q, dtype, STEP, GATHER ? 1 : nt == 256 ? 128 : Q_BOX, false);
    if (rc != QMOE_OK) return rc;
    const int64_t most = most_tiles(g.P, g.E, g.lanes, nt);
    if (most >= (1ll << 31)) return QMOE_ERR_UNSUPPORTED;
    const bool shares = split(g.P, g.E, g.lanes, g.steps, nt);
    if (shares) {
        if (left < part_bytes(nt)) return QMOE_ERR_ARG;  // asked for above
        g.parts = reinterpret_cast<float*>(ws);
        g.joins = reinterpret_cast<int4*>(ws + (size_t)row::kSMs * 2 * nt * 128 * 4);
    }
    switch (nt) {
        case 32:
            return shares ? launch_as<MODE, 32, GATHER, BY, true>(mp, mq, g, most, st)
                          : launch_as<MODE, 32, GATHER, BY, false>(mp, mq, g, most, st);
        case 128:
            return shares ? launch_as<MODE, 128, GATHER, BY, true>(mp, mq, g, most, st)
                          : launch_as<MODE, 128, GATHER, BY, false>(mp, mq, g, most, st);
        default: return GATHER ? QMOE_ERR_UNSUPPORTED : launch_pair<MODE, false, BY>(mp, mq, mq, g, most, st);
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
    int parts = 1;              // of w, whose products are summed up (E is 1)
    const float* by = nullptr;  // a factor of each output (y) or input (dx) of the layer
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

static size_t product_bytes(int64_t P, int E, int64_t N, int64_t K, int op, int pairs, int parts) {
    if (P <= 0 || E <= 0 || N <= 0 || K <= 0 || op < 0 || op > 2 || P > eg::kMost || N > eg::kMost || K > eg::kMost) return 0;
    if (op == eg::DW) return pairs ? eg::padded(P, K) : 0;
    const int64_t lanes = op == eg::FWD ? N : K, red = op == eg::FWD ? K : N;
    const int nt = eg::tile_of(P, E, lanes, red);
    if (nt == 256) return pairs && op == eg::FWD ? eg::padded(P, K) : 0;
    return eg::split(P, E, lanes, (int64_t)parts * eg::steps_of(red), nt) ? eg::part_bytes(nt) : 0;
}
extern "C" size_t qmoe_expert_workspace_bytes(int64_t P, int E, int64_t N, int64_t K, int op, int pairs) {
    return product_bytes(P, E, N, K, op, pairs, 1);
}
extern "C" int qmoe_expert_linear_in_place(int64_t P, int E, int64_t N, int64_t K) {
    return P >= 0 && E > 0 && N > 0 && K > 0 && eg::few(P, E, N, K);
}

namespace qmoe {
namespace eg {

static int linear(const Call& c, const void* x, int64_t ldx, const void* w, int64_t ldw, int64_t w_expert, void* y, int y_dtype,
                  int64_t ldy, void* ws, size_t ws_bytes, cudaStream_t st) {
    int rc = check(c);
    if (rc != QMOE_OK) return rc;
    if ((y_dtype != c.dtype && y_dtype != QMOE_F32) || ldy < c.N) return QMOE_ERR_ARG;
    if (c.P == 0) return QMOE_OK;
    if (c.pairs && c.x_rows == 0) return QMOE_ERR_ARG;
    Mat mw = {w, c.N, c.K, ldw, c.E * c.parts, w_expert}, mx = {x, c.pairs ? c.x_rows : c.P, c.K, ldx, 1, 0};
    if (!mat_ok(mw, 2) || !mat_ok(mx, 2) || !word_ok(c.offsets) || !y || !row::type_aligned(y, row::dtype_size(y_dtype)) ||
        !word_ok(c.status))
        return QMOE_ERR_ARG;
    uint8_t* at = static_cast<uint8_t*>(ws);
    size_t left = ws && !(reinterpret_cast<uintptr_t>(ws) & 255u) ? ws_bytes : 0;
    const int size = row::dtype_size(y_dtype);
    Args g = {(int)c.P, c.E, (int)c.N, 0, (int)c.K, c.offsets, c.pairs, c.k, (int)mx.rows, y, ldy, 0, y_dtype,
              aligned16(y) && ldy * size % 16 == 0, c.dtype == QMOE_BF16 ? tc::idesc_bf16_f32(0, 0) : tc::idesc_f16_f32(0, 0), c.status,
              nullptr, nullptr, c.by, steps_of(c.K), steps_of(c.K) * c.parts};
    if (!fits(mw) && few(c.P, c.E, c.N, c.K)) return launch_few(mw, mx, g, c.dtype, st);
    const bool lay_out = c.pairs && tile_of(c.P, c.E, c.N, c.K) == 256;
    const size_t need = product_bytes(c.P, c.E, c.N, c.K, FWD, c.pairs != nullptr, c.parts);
    if (left < need + copy_need(mw) + (lay_out ? 0 : copy_need(mx))) return QMOE_ERR_ARG;
    if ((rc = as_tma(mw, c.offsets, at, left, st)) != QMOE_OK) return rc;
    rc = lay_out ? copy_rows(mx, c.pairs, c.P, c.k, nullptr, at, left, st) : as_tma(mx, nullptr, at, left, st);
    if (rc != QMOE_OK) return rc;
    if (lay_out) g.pairs = nullptr;
    if (g.pairs) return run_rows<FWD, true, false>(mw, mx, g, c.dtype, at, left, st);
    return c.by ? run_rows<FWD, false, true>(mw, mx, g, c.dtype, at, left, st) : run_rows<FWD, false, false>(mw, mx, g, c.dtype, at, left, st);
}

static int linear_dx(const Call& c, const void* dy, int64_t lddy, const void* w, int64_t ldw, int64_t w_expert, void* dx, int dx_dtype,
                     int64_t lddx, void* ws, size_t ws_bytes, cudaStream_t st) {
    int rc = check(c);
    if (rc != QMOE_OK) return rc;
    if ((dx_dtype != c.dtype && dx_dtype != QMOE_F32) || lddx < c.K) return QMOE_ERR_ARG;
    if (c.P == 0) return QMOE_OK;
    Mat mw = {w, c.N, c.K, ldw, c.E * c.parts, w_expert}, my = {dy, c.P, c.N, lddy, 1, 0};
    if (!mat_ok(mw, 2) || !mat_ok(my, 2) || !word_ok(c.offsets) || !dx || !row::type_aligned(dx, row::dtype_size(dx_dtype)) ||
        !word_ok(c.status))
        return QMOE_ERR_ARG;
    uint8_t* at = static_cast<uint8_t*>(ws);
    size_t left = ws && !(reinterpret_cast<uintptr_t>(ws) & 255u) ? ws_bytes : 0;
    if (left < product_bytes(c.P, c.E, c.N, c.K, DX, 0, c.parts) + copy_need(mw) + copy_need(my)) return QMOE_ERR_ARG;
    if ((rc = as_tma(mw, c.offsets, at, left, st)) != QMOE_OK || (rc = as_tma(my, nullptr, at, left, st)) != QMOE_OK) return rc;
    const int size = row::dtype_size(dx_dtype);
    Args g = {(int)c.P, c.E, (int)c.K, 0, (int)c.N, c.offsets, nullptr, 0, (int)c.P, dx, lddx, 0, dx_dtype,
              aligned16(dx) && lddx * size % 16 == 0,
              (c.dtype == QMOE_BF16 ? tc::idesc_bf16_f32(0, 0) : tc::idesc_f16_f32(0, 0)) | 1u << 15, c.status, nullptr, nullptr, c.by,
              steps_of(c.N), steps_of(c.N) * c.parts};
    return c.by ? run_rows<DX, false, true>(mw, my, g, c.dtype, at, left, st) : run_rows<DX, false, false>(mw, my, g, c.dtype, at, left, st);
}

size_t scaled_bytes(int64_t T, int64_t N, int64_t K, int parts, int dx) {
    return qmoe_expert_copy_bytes(T, dx ? N : K) + product_bytes(T, 1, N, K, dx ? DX : FWD, 0, parts);
}
static Call call_of(const Scaled& c) { return {c.T, c.N, c.K, 1, c.dtype, c.offsets, nullptr, 0, c.T, c.status, c.parts, c.by}; }
int scaled_linear(const Scaled& c, const void* x, int64_t ldx, void* y, int y_dtype, int64_t ldy, cudaStream_t st) {
    return linear(call_of(c), x, ldx, c.w, c.K, c.N * c.K, y, y_dtype, ldy, c.ws, c.ws_bytes, st);
}
int scaled_linear_dx(const Scaled& c, const void* dy, int64_t lddy, void* dx, int dx_dtype, int64_t lddx, cudaStream_t st) {
    return linear_dx(call_of(c), dy, lddy, c.w, c.K, c.N * c.K, dx, dx_dtype, lddx, c.ws, c.ws_bytes, st);
}

}  // namespace eg
}  // namespace qmoe

extern "C" int qmoe_expert_linear(int64_t P, int E, int64_t N, int64_t K, int dtype, const void* x, int64_t ldx,
                                  int64_t x_rows, const int32_t* pairs, int k, const void* w, int64_t ldw, int64_t w_expert,
                                  const int32_t* offsets, void* y, int y_dtype, int64_t ldy, int32_t* dev_status, void* ws,
                                  size_t ws_bytes, qmoe_stream_t stream) {
    return eg::linear({P, N, K, E, dtype, offsets, pairs, k, x_rows, dev_status}, x, ldx, w, ldw, w_expert, y, y_dtype, ldy, ws,
                      ws_bytes, (cudaStream_t)stream);
}

extern "C" int qmoe_expert_linear_dx(int64_t P, int E, int64_t N, int64_t K, int dtype, const void* dy, int64_t lddy,
                                     const void* w, int64_t ldw, int64_t w_expert, const int32_t* offsets, void* dx,
                                     int dx_dtype, int64_t lddx, int32_t* dev_status, void* ws, size_t ws_bytes,
                                     qmoe_stream_t stream) {
    return eg::linear_dx({P, N, K, E, dtype, offsets, nullptr, 0, 0, dev_status}, dy, lddy, w, ldw, w_expert, dx, dx_dtype, lddx,
                         ws, ws_bytes, (cudaStream_t)stream);
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
    if (left < (pairs ? eg::padded(P, K) : eg::copy_need(mx)) + eg::copy_need(my)) return QMOE_ERR_ARG;
    if ((rc = eg::as_tma(my, nullptr, at, left, st)) != QMOE_OK) return rc;
    rc = pairs ? eg::copy_rows(mx, pairs, P, k, nullptr, at, left, st) : eg::as_tma(mx, nullptr, at, left, st);
    if (rc != QMOE_OK) return rc;
    eg::Args g = {(int)P, E, (int)N, (int)K, 0, offsets, nullptr, 0, (int)mx.rows, dw, K, N * K, dw_dtype,
                  aligned16(dw) && K * size % 16 == 0,
                  (dtype == QMOE_BF16 ? tc::idesc_bf16_f32(0, 0) : tc::idesc_f16_f32(0, 0)) | 3u << 15, dev_status, nullptr, nullptr, nullptr, 0, 0};
    CUtensorMap mp, mq;
    rc = eg::map_of(&mp, my, dtype, 64, eg::STEP, false);
    if (rc != QMOE_OK) return rc;
    rc = eg::map_of(&mq, mx, dtype, 64, eg::STEP, false);
    if (rc != QMOE_OK) return rc;
    if (!g.wide || P > (size == 4 ? 32ll : 256ll) * E) return eg::launch_pair<eg::DW>(mp, mq, mq, g, units, st);
    // few rows an expert: put_dw has both sides
    CUtensorMap mo;
    const eg::Mat out = {dw, N, K, K, E, N * K};
    rc = eg::map_of(&mo, out, dw_dtype, 32, 32, true, true);
    if (rc != QMOE_OK) return rc;
    return eg::launch_pair<eg::DW, true>(mp, mq, mo, g, units, st);
}
