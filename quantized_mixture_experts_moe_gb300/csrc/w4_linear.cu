// Products of few tokens with 4-bit weights (qmoe_w4_linear), and the layer's
// wider forms (qmoe_w4_linear for many tokens, qmoe_w4_linear_dx).
//
//   y[t][n] = sum over groups G of s[n][G] sum_{k in G} v(code[n][k]) x[t][k]
//
// Few tokens: the codes' bytes are what the product cannot do without, and turning
// them into numbers is what it spends its instructions on.  mma.sync m16n8k16 with
// 16 rows of W and 8 tokens.  An int4 code becomes the 16-bit float 16 + n by two
// bit operations for two codes (n in the top mantissa bits of a float between 16
// and 32), exactly, and the sum of 32 values starts from -24 sum x, so that it ends
// as the sum of (n - 8) x.  The order of the reduction inside such a sum is free, so
// the codes of a word are taken as they come (0 4 1 5 2 6 3 7), and x lies in shared
// memory in that order.  E2M1 codes are converted to fp16, two by an instruction; x
// is then taken to fp16 too, each 32 values of a token by the power of two that
// moves the largest into [2^14, 2^15) (exact for values above 2^-28 of it).  Sums of
// 32 values are scaled in fp32.
//
// Up to 4 tokens leave columns of the tensor core's 8 unused.  These then keep GC
// groups of 32 values apart: a lane takes 32 GC / 4 contiguous codes of its row, all of
// one group, and column (token, group) has x where the lane's group is its own, and
// zeros elsewhere.  A scale is then applied once for GC groups, by the lane that has
// both, and codes come 16 bytes (GC = 4) or 8 at a time.
//
// Persistent CTAs, two an SM as x leaves room: each takes a run of (matrix, rows)
// tiles, and a warp of its own keeps the next four blocks of 16 rows x 256 codes of
// each of the eight others on the way, over the ends of tiles too.  One CTA a tile
// spent 9 us on each, waiting for ids, codes, x and scales in turn.  With ids, pairs
// of the same expert share its codes: the CTAs put the pairs in expert order.
//
// What bounds it: the conversion.  Four tokens x 10 of 512 experts 4096 -> 2048 (E2M1,
// 178 MB): 56 us, 3.1 TB/s, with 53% of the issue slots busy and the integer pipe,
// which converts, in the way; int4 64 us (104 at first, a CTA a tile and eight
// operations for two E2M1 codes).  One token 2048 -> 2816, int4: 4.1 us, latency.
#include <algorithm>
#include <type_traits>

#include "expert_gemm.cuh"

namespace qmoe {
namespace w4 {

constexpr int WARPS = 8, THREADS = (WARPS + 1) * 32;  // of products, and one that sends for codes
constexpr int ROWS = 16;          // of W, of a warp
constexpr int BLOCK = 256;        // values of a row in a stage (128 bytes)
constexpr int STAGE = ROWS * 128, DEPTH = 4;
constexpr int MOST_PAIRS = 256;   // that are put in expert order, or of a CTA's run

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
    int chunk;   // values of x in shared memory at once, a multiple of WARPS * BLOCK or all
    int tiles;   // of a matrix, of ROWS * WARPS / kw rows
    int units;   // tiles of all pairs
    int kw_log;  // warps that share a reduction
    int two;     // scales of two neighbouring groups can be read at once
    int pairs;   // rows of y with ids, 0: without
    int share;   // most tokens that share a tile: pairs of one expert (1: each by itself)
    int32_t* status;
};

template <typename T> struct Num;
template <> struct Num<__half> {
    static constexpr uint32_t BASE = 0x4C004C00u;  // 16
    static constexpr int UP = 6;                   // from bit 0 to the top four mantissa bits
};
template <> struct Num<__nv_bfloat16> {
    static constexpr uint32_t BASE = 0x41804180u;  // 16
    static constexpr int UP = 3;
};
// Codes of a word as numbers in the halves of a register.  int4: codes j and j + 4,
// as 16 + n.  E2M1: codes 2 j and 2 j + 1.
template <typename T, int FORMAT, int J>
__device__ __forceinline__ uint32_t pair_of(uint32_t word) {
    if constexpr (FORMAT == QMOE_W4_INT4) {
        using M = Num<T>;
        constexpr int by = M::UP - 4 * J;
        const uint32_t v = by >= 0 ? word << (by >= 0 ? by : 0) : word >> (by < 0 ? -by : 0);
        return (v & (0x000F000Fu << M::UP)) | M::BASE;
    } else {
        uint32_t v;
        asm("{\n\t.reg .b8 b<4>;\n\tmov.b32 {b0, b1, b2, b3}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b%2;\n\t}" : "=r"(v) : "r"(word), "n"(J));
        return v;
    }
}

// A scale as it lies in memory, and what it stands for.
template <int FORMAT> struct Scale { typedef uint8_t Raw; };
template <> struct Scale<QMOE_W4_INT4> { typedef uint16_t Raw; };
template <int FORMAT>
__device__ __forceinline__ float scale_of(uint32_t raw) {
    if constexpr (FORMAT == QMOE_W4_INT4) return __half2float(__ushort_as_half((unsigned short)raw));
    else return e8m0_to_float((uint8_t)raw);
}
template <int FORMAT>
__device__ __forceinline__ float scale_at(const void* s, int64_t i) {
    return scale_of<FORMAT>(static_cast<const typename Scale<FORMAT>::Raw*>(s)[i]);
}

// Bytes of a token's x in shared memory: rows of two neighbouring tokens fall into
// different halves of the banks.
__host__ __device__ constexpr int pitch_of(int chunk) { return chunk * 2 + 64; }
// Shared memory: rings, then x, a number for each 32 values of a token, the sums
// of the warps (two tiles' for up to 8 tokens), and the sets of pairs.
constexpr int RING = WARPS * DEPTH * STAGE;
constexpr int LISTS = (3 * MOST_PAIRS + 16) * 4;  // sets of pairs, and their pairs
__host__ __device__ constexpr int bufs_of(int nt) { return nt == 1 ? 2 : 1; }
inline int smem_of(int tokens, int chunk, int nt) {
    return 1024 + RING + tokens * pitch_of(chunk) + chunk / 32 * 8 * nt * 4 + bufs_of(nt) * WARPS * nt * 8 * ROWS * 4 + LISTS;
}

// Whether a phase is over, without waiting for it.
__device__ __forceinline__ bool is_over(uint64_t* bar, uint32_t parity) {
    uint32_t over;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(over)
        : "r"(tc::smem_u32(bar)), "r"(parity)
        : "memory");
    return over != 0;
}
// A barrier of the warps of products.
__device__ __forceinline__ void products_sync() { asm volatile("bar.sync 1, %0;" ::"n"(WARPS * 32) : "memory"); }

// x of a set's tokens (without ids of all) in [c0, c0 + len), zeros up to whole blocks; and for each 32
// values of a token -24 times their sum (int4), or the power of two that they were
// divided by (E2M1).
template <typename T, int FORMAT, int NT, int GC>
__device__ __forceinline__ void stage_x(const Args& g, uint8_t* xs, float* sums, int pitch, const int* pairs, int tokens, int c0, int len) {
    // pieces of a thread on their way: one at a time took 16 tokens 4096 -> 4096 int4 18.0 us for 14.5, 8 tokens 11.5 for
    // 10.2; for one or two tokens four cost half a microsecond (2048 -> 2816 4.1 for 4.7), in code that has to be fetched
    constexpr int U = GC == 4 ? 1 : 4 * NT;
    const int per = len / 8, n = tokens * per;
    for (int i0 = threadIdx.x; i0 < n; i0 += U * WARPS * 32) {
        uint4 raw[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int i = i0 + j * WARPS * 32, t = i / per, k = (i - t * per) * 8;
            raw[j] = make_uint4(0, 0, 0, 0);
            if (i < n && c0 + k < g.K) {
                const T* from = static_cast<const T*>(g.x) + (int64_t)(pairs ? pairs[t] / g.k : t) * g.ldx + c0 + k;
                if (g.x_wide) {
                    raw[j] = *reinterpret_cast<const uint4*>(from);
                } else {
                    uint32_t u[8];
#pragma unroll
                    for (int q = 0; q < 8; ++q) u[q] = reinterpret_cast<const uint16_t*>(from)[q];
                    raw[j] = make_uint4(u[0] | u[1] << 16, u[2] | u[3] << 16, u[4] | u[5] << 16, u[6] | u[7] << 16);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int i = i0 + j * WARPS * 32, t = i / per, k = (i - t * per) * 8;
            if (i >= n) break;
            uint4 v = raw[j];
            const float2 a = row::unpack2(v.x, T{}), b = row::unpack2(v.y, T{}), c = row::unpack2(v.z, T{}), d = row::unpack2(v.w, T{});
            // len / 8 is a multiple of 32: the lanes of a warp hold one token's neighbouring values
            float of;
            if constexpr (FORMAT == QMOE_W4_INT4) {
                of = ((a.x + a.y) + (b.x + b.y)) + ((c.x + c.y) + (d.x + d.y));
                of += __shfl_xor_sync(0xFFFFFFFFu, of, 1);
                of += __shfl_xor_sync(0xFFFFFFFFu, of, 2);
                of *= -24.f;
            } else {
                float m = fmaxf(fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(b.x), fabsf(b.y))),
                                fmaxf(fmaxf(fabsf(c.x), fabsf(c.y)), fmaxf(fabsf(d.x), fabsf(d.y))));
                m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
                m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
                const int e = f16_row_exponent(m);
                const float by = exp2i(-e);
                v = make_uint4(row::pack2(a.x * by, a.y * by, __half{}), row::pack2(b.x * by, b.y * by, __half{}),
                               row::pack2(c.x * by, c.y * by, __half{}), row::pack2(d.x * by, d.y * by, __half{}));
                of = exp2i(e);
            }
            if ((i & 3) == 0) sums[GC ? t * (g.chunk / 32) + k / 32 : (k / 32) * (8 * NT) + t] = of;
            if constexpr (FORMAT == QMOE_W4_INT4)  // in the order of the codes
                v = make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632), __byte_perm(v.y, v.w, 0x5410),
                               __byte_perm(v.y, v.w, 0x7632));
            *reinterpret_cast<uint4*>(xs + t * pitch + k * 2) = v;
        }
    }
    if (GC && threadIdx.x < 4) *reinterpret_cast<uint4*>(xs + g.chunk * 2 + threadIdx.x * 16) = make_uint4(0, 0, 0, 0);
}

template <typename T, int FORMAT, int NT, int GC, bool IDS>  // NT: tiles of 8 tokens; GC 0: columns are tokens
__global__ void __launch_bounds__(THREADS, NT == 1 ? 2 : 1) w4_few_kernel(const __grid_constant__ CUtensorMap map, const Args g) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t bars[2 * WARPS * DEPTH];  // full and empty stages of each warp's ring
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quad = lane & 3, col = lane >> 2;
    // the row of W of a lane: with GC the lanes that read shared memory together have rows 4 apart, whose swizzles differ
    const int row = GC ? (col >> 1) | (col & 1) << 2 : col;
    const int kw = 1 << g.kw_log, part = warp & (kw - 1), rows = ROWS * (WARPS >> g.kw_log);
    const int first_row = (warp >> g.kw_log) * ROWS;  // of this warp in a tile
    uint8_t* const xs = smem + RING;
    const int most = IDS ? g.share : g.T, pitch = pitch_of(g.chunk);  // tokens of a tile
    float* const sums = reinterpret_cast<float*>(xs + most * pitch);  // [groups of 32 in a chunk][8 NT], with GC [token][groups]
    float* const parts = sums + g.chunk / 32 * 8 * NT;                // [bufs][WARPS][8 NT][ROWS]
    // sets of pairs of one expert: the expert (-1: none), the first of its pairs in `order`; order: the pairs
    int* const experts = reinterpret_cast<int*>(parts + bufs_of(NT) * WARPS * NT * 8 * ROWS);
    int *const starts = experts + MOST_PAIRS, *const order = starts + MOST_PAIRS + 1, *const marks = order + MOST_PAIRS;
    const int blocks = (g.K + BLOCK - 1) / BLOCK, mine = (blocks - part + kw - 1) >> g.kw_log;  // of a tile, of this warp

    if (threadIdx.x == 0) tc::prefetch_tensormap(&map);
    pdl_wait();
    if (threadIdx.x < 2 * WARPS * DEPTH) {
        tc::mbar_init(&bars[threadIdx.x], 1);
        tc::fence_barrier_init();
    }
    int units = g.tiles, p0 = 0;  // of all sets; the first set that is listed
    if (IDS && g.share > 1) {
        // The pairs in expert order, those of no expert last, cut into sets of `share`: by every CTA for itself.
        const int p = threadIdx.x;
        auto key = [&](int e) { return e >= 0 && e < g.E ? e : g.E; };
        int e = g.E;
        if (p < g.pairs) experts[p] = e = key(g.ids[p]);
        __syncthreads();
        int rank = 0, less = 0;  // pairs before this one, pairs of experts before its
        if (p < g.pairs)
            for (int q = 0; q < g.pairs; ++q) {
                const int f = experts[q];
                less += f < e;
                rank += f < e || (f == e && q < p);
            }
        __syncthreads();
        if (p < g.pairs) {
            order[rank] = p;
            experts[rank] = e;
        }
        if (p < 9) marks[p] = 0;
        // where a set starts, by its place in the order: bits of words of 32
        __syncthreads();
        if (p < g.pairs && (rank - less) % g.share == 0) atomicOr(&marks[rank >> 5], 1 << (rank & 31));
        __syncthreads();
        int sets = 0, before = 0, sorted = g.E;
        const bool first_of = p < g.pairs && (marks[p >> 5] >> (p & 31) & 1);
        if (p < g.pairs) sorted = experts[p];
        for (int w = 0; w * 32 < g.pairs; ++w) {
            const int n = __popc(marks[w]);
            if (w < (p >> 5)) before += n;
            sets += n;
        }
        if (p < g.pairs) before += __popc(marks[p >> 5] & ((1 << (p & 31)) - 1));
        __syncthreads();
        if (first_of) {
            starts[before] = p;
            experts[before] = sorted < g.E ? sorted : -1;
        }
        if (p == 0) starts[sets] = g.pairs;
        units = sets * g.tiles;
    } else if (IDS) {
        units = g.units;
    }
    // this CTA's run
    const int u0 = (int)((int64_t)units * blockIdx.x / gridDim.x), u1 = (int)((int64_t)units * (blockIdx.x + 1) / gridDim.x);
    if (IDS && g.share == 1 && u0 < u1) {
        p0 = u0 / g.tiles;
        const int n = (u1 - 1) / g.tiles - p0 + 1;
        for (int i = threadIdx.x; i < n; i += THREADS) {
            const int e = g.ids[p0 + i];
            experts[i] = e >= 0 && e < g.E ? e : -1;
            starts[i] = i;
            order[i] = p0 + i;
            if (i == n - 1) starts[n] = n;
        }
    }
    __syncthreads();
    pdl_trigger();
    // a place in the run: unit, set, tile and the set's expert (-1: none)
    struct Place {
        int u, pair, tile, e;
    };
    auto look = [&](Place& p) { p.e = p.u < u1 ? (IDS ? experts[p.pair - p0] : 0) : -1; };
    auto step = [&](Place& p) {
        ++p.u;
        if (++p.tile == g.tiles) {
            p.tile = 0;
            ++p.pair;
            look(p);
        } else if (p.u >= u1) {
            p.e = -1;
        }
    };
    auto settle = [&](Place& p) {  // at p or the next unit of an expert
        while (p.e < 0 && p.u < u1) step(p);
    };
    Place start = {u0, u0 / g.tiles, u0 % g.tiles, 0};
    look(start);
    if (warp == WARPS) {
        // lane i sends for warp i: block j of its part of unit `at`
        const int of = lane & (kw - 1), first = (lane >> g.kw_log) * ROWS, n = (blocks - of + kw - 1) >> g.kw_log;
        Place at = start;
        settle(at);
        int j = 0, slot = 0;
        uint32_t phase = 1;
        bool more = lane < WARPS && at.e >= 0;
        long long since = clock64();
        while (__any_sync(0xFFFFFFFFu, more)) {
            uint64_t* const full = &bars[(lane * DEPTH + slot) & (WARPS * DEPTH - 1)];
            const bool free = more && is_over(full + WARPS * DEPTH, phase);
            if (free) {
                tc::mbar_arrive_expect_tx(full, STAGE);
                tc::tma_load_3d(smem + (lane * DEPTH + slot) * STAGE, &map, full, (of + j * kw) * (BLOCK / 2), at.tile * rows + first, at.e);
                if (++slot == DEPTH) { slot = 0; phase ^= 1; }
                if (++j == n) {
                    j = 0;
                    step(at);
                    settle(at);
                    more = at.e >= 0;
                }
            }
            if (__any_sync(0xFFFFFFFFu, free)) {
                since = clock64();
                continue;
            }
            __nanosleep(64);  // a stage lasts a warp some 1500
            if (clock64() - since > 4000000000ll) {
                if (lane == 0) atomicOr(g.status, QMOE_DEV_WAIT_TIMEOUT);
                break;
            }
        }
        return;
    }

    // Scales, a block ahead: rows row and row + 8; with GC the groups of this lane's columns 2 quad and 2 quad + 1 in each
    // span of GC groups, else groups 2 quad and 2 quad + 1 of the block, which the lanes of a quad share.  Behind the
    // last row and the last group the last ones are read: those rows are not stored, and x is zero there.
    typedef typename Scale<FORMAT>::Raw Raw;
    typedef typename std::conditional<sizeof(Raw) == 2, uint32_t, uint16_t>::type Two;
    constexpr int SPANS = GC ? 8 / GC : 1, RAW_BITS = 8 * sizeof(Raw);
    const int per_row = g.K >> g.shift, g0 = GC == 4 ? 2 * (quad & 1) : GC == 2 ? 0 : 2 * quad;
    Place later = start;
    settle(later);
    const Raw* at_row[2] = {};
    int later_j = 0;
    uint32_t raw[SPANS][2];
    auto find_rows = [&]() {
        const int n = later.tile * rows + first_row + row;
        const Raw* const of = static_cast<const Raw*>(g.s) + (int64_t)later.e * g.N * per_row;
        at_row[0] = of + (int64_t)min(n, g.N - 1) * per_row;
        at_row[1] = of + (int64_t)min(n + 8, g.N - 1) * per_row;
    };
    auto fetch = [&]() {
        if (later.e < 0) return;
        const int b = part + later_j * kw;
        if (g.two && (b + 1) * BLOCK <= g.K) {  // both in one word
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const Two* const from = reinterpret_cast<const Two*>(at_row[h] + b * 8 + g0);
#pragma unroll
                for (int s = 0; s < SPANS; ++s) raw[s][h] = from[s * GC / 2];
            }
        } else {
#pragma unroll
            for (int s = 0; s < SPANS; ++s) {
                const int k0 = b * BLOCK + (s * GC + g0) * 32;
                const int i0 = min(k0, g.K - 32) >> g.shift, i1 = min(k0 + 32, g.K - 32) >> g.shift;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t one = at_row[h][i0];
                    raw[s][h] = one | (i1 == i0 ? one : (uint32_t)at_row[h][i1]) << RAW_BITS;
                }
            }
        }
        if (++later_j == mine) {
            later_j = 0;
            step(later);
            settle(later);
            if (later.e >= 0) find_rows();
        }
    };
    if (later.e >= 0) find_rows();
    fetch();

    // after a wait that ran out a warp frees no more stages (the one that sends gives up by itself) and only keeps the others'
    // barriers company
    bool ok = true;
    int slot = 0, buf = 0, staged_c = -1;
    uint32_t phase = 0;
    int staged_set = -1;
    for (Place at = start; at.u < u1; step(at)) {
        const int n0 = at.tile * rows;
        const int* const set = IDS ? order + starts[at.pair - p0] : nullptr;
        const int tokens = IDS ? starts[at.pair - p0 + 1] - starts[at.pair - p0] : g.T;
        auto row_of = [&](int t) { return (int64_t)(set ? set[t] : t) * g.ldy; };  // of y
        if (at.e < 0) {
            for (int t = 0; t < tokens; ++t)
                for (int i = threadIdx.x; i < rows; i += WARPS * 32)
                    if (n0 + i < g.N) eg::put_value(g.y, g.ytype, row_of(t) + n0 + i, 0.f);
            continue;
        }
        float acc[NT][4];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
        int j0 = 0;
        for (int c0 = 0; c0 < g.K; c0 += g.chunk) {
            const int len = min(g.chunk, (g.K - c0 + BLOCK - 1) / BLOCK * BLOCK);
            if (staged_c != c0 || staged_set != at.pair) {
                if (staged_c >= 0) products_sync();
                stage_x<T, FORMAT, NT, GC>(g, xs, sums, pitch, set, tokens, c0, len);
                staged_c = c0;
                staged_set = at.pair;
                products_sync();
            }
            for (; j0 < mine && (part + j0 * kw) * BLOCK < c0 + len; ++j0) {
                const int b = part + j0 * kw;
                float sc[SPANS][2][2];
#pragma unroll
                for (int s = 0; s < SPANS; ++s)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int i = 0; i < 2; ++i) sc[s][h][i] = scale_of<FORMAT>(raw[s][h] >> i * RAW_BITS & (Raw)~Raw(0));
                fetch();
                if (ok) ok = __all_sync(0xFFFFFFFFu, tc::mbar_wait(&bars[warp * DEPTH + slot], phase));
                constexpr bool INT4 = FORMAT == QMOE_W4_INT4, BF16 = INT4 && std::is_same<T, __nv_bfloat16>::value;
                if constexpr (GC > 0) {
                    const uint8_t* st = smem + (warp * DEPTH + slot) * STAGE + row * 128;
                    // this lane's column's x, or zeros; its columns' numbers
                    const bool own_x = col % GC == quad * GC / 4 && col / GC < tokens;
                    const uint8_t* xp = own_x ? xs + col / GC * pitch + (b * BLOCK - c0) * 2 + quad * GC * 16 : xs + g.chunk * 2;
                    const int x_step = own_x ? GC * 64 : 0;
                    const int t = min(GC == 4 ? quad >> 1 : quad, tokens - 1);
                    const float* zp = sums + t * (g.chunk / 32) + (b * BLOCK - c0) / 32 + g0;
#pragma unroll
                    for (int s = 0; s < SPANS; ++s) {
                        uint32_t lo[GC], hi[GC];
                        if constexpr (GC == 4) {
                            const uint32_t at = ((s * 4 + quad) ^ (row & 7)) * 16;
                            *reinterpret_cast<uint4*>(lo) = *reinterpret_cast<const uint4*>(st + at);
                            *reinterpret_cast<uint4*>(hi) = *reinterpret_cast<const uint4*>(st + 1024 + at);
                        } else {
                            const uint32_t at = ((s * 2 + (quad >> 1)) ^ (row & 7)) * 16 + (quad & 1) * 8;
                            *reinterpret_cast<uint2*>(lo) = *reinterpret_cast<const uint2*>(st + at);
                            *reinterpret_cast<uint2*>(hi) = *reinterpret_cast<const uint2*>(st + 1024 + at);
                        }
                        const float2 z = *reinterpret_cast<const float2*>(zp + s * GC);
                        float d[4] = {INT4 ? z.x : 0.f, INT4 ? z.y : 0.f, INT4 ? z.x : 0.f, INT4 ? z.y : 0.f};
#pragma unroll
                        for (int i = 0; i < GC; ++i) {
                            const uint4 v = *reinterpret_cast<const uint4*>(xp + i * 16);
                            const uint32_t a0[4] = {pair_of<T, FORMAT, 0>(lo[i]), pair_of<T, FORMAT, 0>(hi[i]),
                                                    pair_of<T, FORMAT, 1>(lo[i]), pair_of<T, FORMAT, 1>(hi[i])};
                            const uint32_t a1[4] = {pair_of<T, FORMAT, 2>(lo[i]), pair_of<T, FORMAT, 2>(hi[i]),
                                                    pair_of<T, FORMAT, 3>(lo[i]), pair_of<T, FORMAT, 3>(hi[i])};
                            tc::mma_sync<BF16>(d, a0[0], a0[1], a0[2], a0[3], v.x, v.y);
                            tc::mma_sync<BF16>(d, a1[0], a1[1], a1[2], a1[3], v.z, v.w);
                        }
                        xp += x_step;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            acc[0][2 * h] = fmaf(sc[s][h][0], INT4 ? d[2 * h] : d[2 * h] * z.x, acc[0][2 * h]);
                            acc[0][2 * h + 1] = fmaf(sc[s][h][1], INT4 ? d[2 * h + 1] : d[2 * h + 1] * z.y, acc[0][2 * h + 1]);
                        }
                    }
                } else {
                    const uint8_t* st = smem + (warp * DEPTH + slot) * STAGE + row * 128 + quad * 4;
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
                        const float f0 = __shfl_sync(0xFFFFFFFFu, sc[0][0][j & 1], (lane & 28) | (j >> 1));
                        const float f1 = __shfl_sync(0xFFFFFFFFu, sc[0][1][j & 1], (lane & 28) | (j >> 1));
#pragma unroll
                        for (int i = 0; i < NT; ++i) {
                            const int t = min(i * 8 + col, tokens - 1);
                            const uint4 v = *reinterpret_cast<const uint4*>(xb + t * pitch + j * 64);
                            const float2 z = *reinterpret_cast<const float2*>(sums + ((b * BLOCK - c0) / 32 + j) * (8 * NT) + i * 8 + quad * 2);
                            float d[4] = {INT4 ? z.x : 0.f, INT4 ? z.y : 0.f, INT4 ? z.x : 0.f, INT4 ? z.y : 0.f};
                            tc::mma_sync<BF16>(d, a0[0], a0[1], a0[2], a0[3], v.x, v.y);
                            tc::mma_sync<BF16>(d, a1[0], a1[1], a1[2], a1[3], v.z, v.w);
                            if constexpr (!INT4) {
                                d[0] *= z.x;
                                d[1] *= z.y;
                                d[2] *= z.x;
                                d[3] *= z.y;
                            }
                            acc[i][0] = fmaf(f0, d[0], acc[i][0]);
                            acc[i][1] = fmaf(f0, d[1], acc[i][1]);
                            acc[i][2] = fmaf(f1, d[2], acc[i][2]);
                            acc[i][3] = fmaf(f1, d[3], acc[i][3]);
                        }
                    }
                }
                __syncwarp();
                if (ok && lane == 0) tc::mbar_arrive(&bars[WARPS * DEPTH + warp * DEPTH + slot]);
                if (++slot == DEPTH) { slot = 0; phase ^= 1; }
            }
        }
        if constexpr (GC > 0) {  // a token's groups, into acc[0][0] and acc[0][2]
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float v = acc[0][2 * h] + acc[0][2 * h + 1];
                if (GC == 4) v += __shfl_xor_sync(0xFFFFFFFFu, v, 1);
                acc[0][2 * h] = v;
            }
        }
        // this lane's sums: token, row of the warp, value
        auto each = [&](auto f) {
            if constexpr (GC > 0) {
                if (GC == 2 || (quad & 1) == 0) {
                    f(GC == 4 ? quad >> 1 : quad, row, acc[0][0]);
                    f(GC == 4 ? quad >> 1 : quad, row + 8, acc[0][2]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) f(i * 8 + quad * 2 + (j & 1), row + (j >> 1) * 8, acc[i][j]);
            }
        };
        if (kw == 1) {  // all of them
            each([&](int t, int r, float v) {
                const int n = n0 + first_row + r;
                if (t < tokens && n < g.N) eg::put_value(g.y, g.ytype, row_of(t) + n, v);
            });
            continue;
        }
        // the warps' sums, added in order
        float* const to = parts + (buf * WARPS + warp) * NT * 8 * ROWS;
        each([&](int t, int r, float v) { to[t * ROWS + r] = v; });
        products_sync();
        for (int i = threadIdx.x; i < tokens * rows; i += WARPS * 32) {
            const int row_log = 7 - g.kw_log, t = i >> row_log, n = i & (rows - 1);
            const float* from = parts + (buf * WARPS + (n / ROWS) * kw) * NT * 8 * ROWS + t * ROWS + n % ROWS;
            float v = 0.f;
            for (int w = 0; w < kw; ++w) v += from[w * NT * 8 * ROWS];
            if (n0 + n < g.N) eg::put_value(g.y, g.ytype, row_of(t) + n0 + n, v);
        }
        if (bufs_of(NT) == 2) buf ^= 1;
        else products_sync();
    }
    if (!ok && lane == 0) {
        atomicOr(g.status, QMOE_DEV_WAIT_TIMEOUT);
        // time for the loads in flight to end (they take microseconds): none outlives the CTA
        for (const long long c = clock64(); clock64() - c < 4000000ll;) __nanosleep(1000);
    }
}

// Two E2M1 codes as fp16.
__device__ __forceinline__ uint32_t e2m1_pair(uint32_t byte) { return pair_of<__half, QMOE_W4_E2M1, 0>(byte); }

// W in 16 bits, [N, K], and {0, T} for the grouped product with one expert.  The
// tensor core takes no scale for each group of values beside 16-bit x, so the weights
// are multiplied with it here.  E2M1 values with their power of two are exact; an int4
// value has 14 bits with its scale's 11, so that W becomes two matrices whose sum is
// exact, the values rounded to x's type and what is left of them, and the product
// takes twice the steps.  (Rounded once: bf16 0.0024 of the result's norm off, of which
// 0.0017 is the output's own rounding, fp16 2.8e-4 and 2.1e-4.)
//
// Scales may lie anywhere in fp16 (int4) or from 2^-127 to 2^127 (E2M1), weights in
// fp16 may not.  So each row (the product), or each column (the gradient), is divided
// by a power of two, `by`, that its sums are multiplied with again.  In fp16 it moves
// the largest scale's values to at most 2^15: what is 2^-39 of the largest or more
// keeps its place.  In bf16 E2M1 values are divided by 4 (6 x 2^127 has no place there),
// which leaves the least of them 2^-130, above bf16's 2^-133.
struct Widen {
    int64_t N, K;
    int shift;
    const uint32_t* w;
    const void* s;
    uint4* to;
    float* by;
    int64_t lanes;  // of by
    int32_t* offsets;
    int tokens;
};
// A scale as a whole number that grows with it; 0 for one that is no finite number.
template <int FORMAT>
__device__ __forceinline__ int key_of(const void* s, int64_t i) {
    const int raw = static_cast<const typename Scale<FORMAT>::Raw*>(s)[i];
    if constexpr (FORMAT == QMOE_W4_INT4) return (raw & 0x7FFF) < 0x7C00 ? raw & 0x7FFF : 0;
    else return raw < 255 ? raw : 0;
}
// The exponent of `by` in bf16, and in fp16 from the largest key.
template <int FORMAT> constexpr int BF16_EXPONENT = FORMAT == QMOE_W4_INT4 ? 0 : 2;
template <int FORMAT>
__device__ __forceinline__ int exponent_of(int key) {
    if constexpr (FORMAT == QMOE_W4_INT4) return f16_row_exponent(8.f * __half2float(__ushort_as_half((unsigned short)key)));
    else return max(key - 127 + 2 - 14, -112);  // 6 x 2^(key - 127) becomes 6 x 2^12 (2^-112 leaves all below their places)
}

// `by` of each column in fp16.  A CTA takes 2 groups of columns, so that few rows fall to a thread (8 groups: 4096 x 4096 int4
// in groups of 128 has 4 CTAs, and the gradient of 17 tokens takes 30.5 us for 25.4).
template <int FORMAT>
__global__ void __launch_bounds__(1024) w4_columns_kernel(const Widen a) {
    constexpr int G = 2, EACH = 1024 / G;
    __shared__ int most[G];
    pdl_wait();
    pdl_trigger();
    const int groups = (int)(a.K >> a.shift), mine = threadIdx.x % G, g = blockIdx.x * G + mine;
    if (threadIdx.x < G) most[threadIdx.x] = 0;
    __syncthreads();
    int key = 0;
    if (g < groups) {
#pragma unroll 8
        for (int64_t n = threadIdx.x / G; n < a.N; n += EACH) key = max(key, key_of<FORMAT>(a.s, n * groups + g));
    }
#pragma unroll
    for (int o = 16; o >= G; o >>= 1) key = max(key, __shfl_xor_sync(0xFFFFFFFFu, key, o));
    if ((threadIdx.x & 31) < G) atomicMax(&most[mine], key);
    __syncthreads();
    const float f = exp2i(exponent_of<FORMAT>(most[mine]));
    for (int k = threadIdx.x / G; g < groups && k < 1 << a.shift; k += EACH) a.by[((int64_t)g << a.shift) + k] = f;
}

// ROW_WARPS warps take a row (each finds its largest scale for itself).  ROWS_BY: fp16's `by` is made for the row; else it is there,
// of each column.
template <typename T, int FORMAT, bool ROWS_BY, int ROW_WARPS>
__global__ void __launch_bounds__(256) w4_widen_kernel(const Widen a) {
    constexpr bool HALF = std::is_same<T, __half>::value;
    pdl_wait();
    pdl_trigger();
    const int64_t n = (int64_t)blockIdx.x * (8 / ROW_WARPS) + (threadIdx.x >> 5) / ROW_WARPS;
    const int lane = threadIdx.x % (32 * ROW_WARPS), words = (int)(a.K / 8), groups = (int)(a.K >> a.shift);
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        a.offsets[0] = 0;
        a.offsets[1] = a.tokens;
    }
    float down = 1.f;  // 1 / by
    if constexpr (!HALF) {
        down = exp2i(-BF16_EXPONENT<FORMAT>);
        for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < a.lanes; i += (int64_t)gridDim.x * 256)
            a.by[i] = exp2i(BF16_EXPONENT<FORMAT>);
    }
    if (n >= a.N) return;
    if constexpr (HALF && ROWS_BY) {
        int key = 0;
        for (int g = threadIdx.x & 31; g < groups; g += 32) key = max(key, key_of<FORMAT>(a.s, n * groups + g));
        key = __reduce_max_sync(0xFFFFFFFFu, key);
        const int e = exponent_of<FORMAT>(key);
        down = exp2i(-e);
        if (lane == 0) a.by[n] = exp2i(e);
    }
    const uint32_t* const from = a.w + n * words;
    uint4* const to = a.to + n * words;
    constexpr int U = 4, STEP = 32 * ROW_WARPS;
    for (int i0 = lane; i0 < words; i0 += STEP * U) {
        uint32_t v[U];
        float f[U];
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (i0 + j * STEP < words) {
                v[j] = from[i0 + j * STEP];
                const int k = (i0 + j * STEP) * 8;
                // powers of two first: a scale that fp32 holds times 6 need not be one
                f[j] = scale_at<FORMAT>(a.s, n * groups + (k >> a.shift)) * (HALF && !ROWS_BY ? 1.f / a.by[k] : down);
            }
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (i0 + j * STEP < words) {
                float d[8];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float2 c;
                    if constexpr (FORMAT == QMOE_W4_INT4) c = make_float2((int)(v[j] >> 8 * q & 15) - 8, (int)(v[j] >> (8 * q + 4) & 15) - 8);
                    else c = row::unpack2(e2m1_pair(v[j] >> 8 * q & 255), __half{});
                    d[2 * q] = f[j] * c.x;
                    d[2 * q + 1] = f[j] * c.y;
                }
                row::store<8>(reinterpret_cast<T*>(to + i0 + j * STEP), d);
                if constexpr (FORMAT == QMOE_W4_INT4) {
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        const float high = row::to_f32(row::from_f32<T>(d[q]));
                        d[q] = isfinite(high) ? d[q] - high : 0.f;
                    }
                    row::store<8>(reinterpret_cast<T*>(to + a.N * words + i0 + j * STEP), d);
                }
            }
    }
}

// ------------------------------------------------------------------ host side

constexpr int kMostSmem = 220 * 1024;

template <typename T, int FORMAT, int NT, int GC, bool IDS>
static int few_as(const CUtensorMap& map, Args& g, int64_t sets, cudaStream_t st) {
    const int tokens = g.pairs ? g.share : g.T, blocks = (g.K + BLOCK - 1) / BLOCK;
    g.chunk = blocks * BLOCK;
    constexpr int LEAST = WARPS * BLOCK;
    static_assert(1024 + RING + 8 * NT * pitch_of(LEAST) + LEAST / 32 * 8 * NT * 4 + bufs_of(NT) * WARPS * NT * 8 * ROWS * 4 +
                          LISTS <= kMostSmem, "the least chunk fits");
    while (smem_of(tokens, g.chunk, NT) > kMostSmem) g.chunk = (g.chunk / 2 + LEAST - 1) / LEAST * LEAST;
    const int smem = smem_of(tokens, g.chunk, NT);
    const int fit = 227 * 1024 / (smem + 1024);  // 1 KB a CTA is the system's
    const int64_t most = (fit > 2 ? 2 : fit) * row::kSMs;
    // As few warps share a reduction as keep the CTAs evenly busy: a tile's end costs a warp as much as a block.
    const int most_log = blocks >= 8 ? 3 : blocks >= 4 ? 2 : blocks >= 2 ? 1 : 0;
    int64_t units = 0;
    for (g.kw_log = 0;; ++g.kw_log) {
        const int rows = ROWS * (WARPS >> g.kw_log);
        g.tiles = (g.N + rows - 1) / rows;
        units = g.tiles * sets;
        const int64_t rounds = (units + most - 1) / most;
        if (g.kw_log == most_log || units * 8 >= rounds * most * 7) break;
    }
    if (units >= (1ll << 31)) return QMOE_ERR_UNSUPPORTED;
    g.units = (int)units;
    const int rc = row::allow_smem<w4_few_kernel<T, FORMAT, NT, GC, IDS>>(kMostSmem);
    if (rc != QMOE_OK) return rc;
    return launch_pdl(w4_few_kernel<T, FORMAT, NT, GC, IDS>, dim3((unsigned)(units < most ? units : most)), dim3(THREADS), (size_t)smem, st,
                      map, g);
}
template <typename T, int FORMAT, int NT, int GC>
static int few(const CUtensorMap& map, Args& g, int64_t sets, cudaStream_t st) {
    return g.pairs ? few_as<T, FORMAT, NT, GC, true>(map, g, sets, st) : few_as<T, FORMAT, NT, GC, false>(map, g, sets, st);
}

template <typename T, int FORMAT>
static int few_tokens(const CUtensorMap& map, Args& g, cudaStream_t st) {
    if (g.pairs > MOST_PAIRS) {
        g.share = 1;
        return few<T, FORMAT, 1, 4>(map, g, g.pairs, st);
    }
    // with ids as many tokens as the pairs of an expert are likely to be (84 pairs of 8 experts, 2816 -> 2048 int4: 90 us
    // pair by pair)
    const int each = g.pairs ? (g.pairs + g.E - 1) / g.E : g.T;
    g.share = each <= 1 ? 2 : each <= 2 ? 4 : each <= 6 ? 8 : 16;
    const int64_t sets = g.pairs ? (g.pairs < g.E ? g.pairs : g.E) : 1;  // about
    const int tokens = g.pairs ? g.share : g.T;
    if (tokens <= 2) return few<T, FORMAT, 1, 4>(map, g, sets, st);
    if (tokens <= 4) return few<T, FORMAT, 1, 2>(map, g, sets, st);
    if (tokens <= 8) return few<T, FORMAT, 1, 0>(map, g, sets, st);
    return few<T, FORMAT, 2, 0>(map, g, sets, st);
}

inline bool format_ok(int format, int group) {
    return (format == QMOE_W4_INT4 && (group == 32 || group == 64 || group == 128)) || (format == QMOE_W4_E2M1 && group == 32);
}
inline int log2_of(int group) { return group == 32 ? 5 : group == 64 ? 6 : 7; }
inline size_t up256(size_t n) { return (n + 255) / 256 * 256; }

template <typename T, int FORMAT, bool ROWS_BY>
static int widen_rows(const Widen& a, cudaStream_t st) {
    if (a.K >= 2048 || a.N < 8 * row::kSMs)  // a word at least for each thread of a CTA, or rows that would leave SMs idle
        return launch_pdl(w4_widen_kernel<T, FORMAT, ROWS_BY, 8>, dim3((unsigned)a.N), dim3(256), 0, st, a);
    return launch_pdl(w4_widen_kernel<T, FORMAT, ROWS_BY, 1>, dim3((unsigned)((a.N + 7) / 8)), dim3(256), 0, st, a);
}
template <typename T, int FORMAT>
static int widen(const Widen& a, int dx, cudaStream_t st) {
    if (!dx || std::is_same<T, __nv_bfloat16>::value) return widen_rows<T, FORMAT, true>(a, st);
    const int64_t groups = a.K >> a.shift;
    const int rc = launch_pdl(w4_columns_kernel<FORMAT>, dim3((unsigned)((groups + 1) / 2)), dim3(1024), 0, st, a);
    return rc != QMOE_OK ? rc : widen_rows<T, FORMAT, false>(a, st);
}
// Tokens up to which the codes are multiplied as they are, QMOE_W4_FEW of them by a
// launch.  us of two launches and widened, int4 bf16 in groups of 128, 17, 24 and 32
// tokens: 1024 x 1024 8.3 8.8 10.2 and 12.0 12.1 12.3; 2816 x 2048 13.1 14.8 17.5 and
// 17.2 17.2 17.4; 2816 x 4096 21.6 25.6 29.6 and 20.6 20.6 20.9; 4096 x 4096 21.9 25.8
// 29.8 and 26.9 27.0 27.3; 8192 x 4096 33 39 44 and 51 51 62; 8192 x 8192 99 110 161 and
// 98 99 117.  E2M1, which becomes one matrix, 4096 x 4096: 19.8 from 17 on, one launch
// of 16 tokens 16.1.
inline int unwidened(int format) { return format == QMOE_W4_INT4 ? 24 : QMOE_W4_FEW; }
inline int parts_of(int format) { return format == QMOE_W4_INT4 ? 2 : 1; }
inline size_t widened_bytes(int64_t T, int64_t N, int64_t K, int parts, int dx) {
    return up256((size_t)N * K * 2 * parts) + up256((size_t)(dx ? K : N) * 4) + 256 + eg::scaled_bytes(T, N, K, parts, dx);
}
// Widens W into the workspace: {W, by, offsets, what the product needs}.
static int widen_any(eg::Scaled& c, int format, int group, const uint8_t* w, const void* s, int dx, cudaStream_t st) {
    uint8_t* at = static_cast<uint8_t*>(c.ws);
    c.parts = parts_of(format);
    const size_t wide = up256((size_t)c.N * c.K * 2 * c.parts), lanes = up256((size_t)(dx ? c.K : c.N) * 4), before = wide + lanes + 256;
    const Widen a = {c.N, c.K, log2_of(group), reinterpret_cast<const uint32_t*>(w), s, reinterpret_cast<uint4*>(at),
                     reinterpret_cast<float*>(at + wide), dx ? c.K : c.N, reinterpret_cast<int32_t*>(at + wide + lanes), (int)c.T};
    c.w = at;
    c.by = a.by;
    c.offsets = a.offsets;
    c.ws = at + before;
    c.ws_bytes -= before;
    if (c.dtype == QMOE_BF16)
        return format == QMOE_W4_INT4 ? widen<__nv_bfloat16, QMOE_W4_INT4>(a, dx, st) : widen<__nv_bfloat16, QMOE_W4_E2M1>(a, dx, st);
    return format == QMOE_W4_INT4 ? widen<__half, QMOE_W4_INT4>(a, dx, st) : widen<__half, QMOE_W4_E2M1>(a, dx, st);
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
    // of either format
    return std::max(w4::widened_bytes(T, N, K, 1, dx), w4::widened_bytes(T, N, K, 2, dx));
}

extern "C" int qmoe_w4_linear(int64_t T, int k, int E, int64_t N, int64_t K, int format, int group, int dtype, const void* x,
                              int64_t ldx, const uint8_t* w, const void* s, const int32_t* ids, void* y, int y_dtype,
                              int64_t ldy, int32_t* dev_status, void* ws, size_t ws_bytes, qmoe_stream_t stream) {
    int rc = w4::check(T, N, K, format, group, dtype, y_dtype, ldy, N);
    if (rc != QMOE_OK) return rc;
    if (k <= 0 || E <= 0 || (!ids && (k != 1 || E != 1))) return QMOE_ERR_ARG;
    if (T == 0) return QMOE_OK;
    if (!w4::arrays_ok(x, ldx, K, w, s, format, y, y_dtype, dev_status) || (ids && !row::type_aligned(ids, 4))) return QMOE_ERR_ARG;
    if (ids && (T * k > 32768 || (int64_t)E * N > w4::kMost)) return QMOE_ERR_UNSUPPORTED;
    cudaStream_t st = (cudaStream_t)stream;
    if (!ids && T > QMOE_W4_FEW && (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < qmoe_w4_workspace_bytes(T, N, K, 0)))
        return QMOE_ERR_ARG;
    if (!ids && T > w4::unwidened(format)) {
        eg::Scaled c = {nullptr, 1, nullptr, T, N, K, dtype, nullptr, dev_status, ws, ws_bytes};
        rc = w4::widen_any(c, format, group, w, s, 0, st);
        return rc != QMOE_OK ? rc : eg::scaled_linear(c, x, ldx, y, y_dtype, ldy, st);
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
                  y_dtype, 0, 0, 0, 0,
                  group == 32 && K % 64 == 0 && row::type_aligned(s, format == QMOE_W4_INT4 ? 4 : 2), (int)(ids ? T * k : 0), 1,
                  dev_status};
    // With ids as many tokens a launch as have their pairs put in expert order (pair by pair, 33 tokens x 8 of 8 experts
    // 2816 -> 2048 int4 239 us, 32 tokens 54; 64 x 8 of 128, 2048 -> 1536, 264 us for 182 in two launches).
    const int size = row::dtype_size(y_dtype);
    const int64_t most = !ids ? QMOE_W4_FEW : k <= w4::MOST_PAIRS ? w4::MOST_PAIRS / k : T, each = ids ? k : 1;
    for (int64_t left = T; left > 0 && rc == QMOE_OK;) {
        g.T = (int)(left < most ? left : most);
        if (ids) g.pairs = g.T * k;
        if (dtype == QMOE_BF16)
            rc = format == QMOE_W4_INT4 ? w4::few_tokens<__nv_bfloat16, QMOE_W4_INT4>(map, g, st)
                                        : w4::few_tokens<__nv_bfloat16, QMOE_W4_E2M1>(map, g, st);
        else
            rc = format == QMOE_W4_INT4 ? w4::few_tokens<__half, QMOE_W4_INT4>(map, g, st)
                                        : w4::few_tokens<__half, QMOE_W4_E2M1>(map, g, st);
        left -= g.T;
        g.x = static_cast<const uint8_t*>(g.x) + g.T * ldx * 2;
        g.y = static_cast<uint8_t*>(g.y) + g.T * each * ldy * size;
        if (ids) g.ids += g.T * each;
    }
    return rc;
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
    eg::Scaled c = {nullptr, 1, nullptr, T, N, K, dtype, nullptr, dev_status, ws, ws_bytes};
    rc = w4::widen_any(c, format, group, w, s, 1, st);
    return rc != QMOE_OK ? rc : eg::scaled_linear_dx(c, dy, lddy, dx, dx_dtype, lddx, st);
}
