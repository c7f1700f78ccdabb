// Pieces shared by the kernels of the experts' products (expert_gemm.cu,
// expert_gemm_pair.cu): arguments, the walk over tiles, stores of sums.
#pragma once

#include <type_traits>

#include "row_ops.cuh"
#include "tc_ptx.cuh"
#include "tma_host.cuh"

namespace qmoe {
namespace eg {

enum { FWD = 0, DX = 1, DW = 2 };

constexpr int EPI_WARPS = 8;     // read sums and store them: two for each quadrant of lanes
constexpr int STEP = 64;         // reduction values of a stage: 128 bytes
constexpr int MAX_E = 1024;
constexpr int STAGE_OUT = 2048, STAGE_DW = 4096;  // bytes of a warp's output stage: 32 rows of 64, or 128
constexpr int Q_BOX = 32;        // rows of a box of the column side (y, dx)
// Most steps that the tensor core sums up by itself.  It cuts a sum off where fp32
// would round it, by up to 2^-23 for each 16 values and always towards zero: 8192
// values were 9.1e-6 of the result off, 65536 in two halves 3.8e-5.  Longer sums are
// made in pieces, each in an accumulator of its own, that are added with fp32's
// rounding: 2.1e-6 at any length.
constexpr int LONG = 32;

struct Args {
    int P, E;
    int lanes, cols, red;  // lanes of all tiles; columns (dw), reduction length (y, dx)
    const int32_t* offsets;
    const int32_t* pairs;  // NULL: the row of a slot is the slot
    int k, x_rows;
    void* out;
    int64_t ld, out_e;     // row stride, expert stride (dw)
    int ctype;
    int wide;              // rows of out start on 16-byte boundaries
    uint32_t idesc;        // without M and N
    int32_t* status;
    float* parts;          // sums of tiles in parts (few tiles), and where they belong
    int4* joins;
    const float* by;       // y, dx: a factor of each lane's sums (NULL: none)
    int per, steps;        // y, dx: steps of a matrix, and of all matrices whose products are summed up (one, or the two parts of w)
};
inline int steps_of(int64_t red) { return (int)((red + STEP - 1) / STEP); }

// Operand whose reduction axis is not the contiguous one: blocks of 64 lanes (or
// columns), 8192 bytes apart; in each, reduction rows of 128 bytes, swizzled in
// groups of 8 rows.
__device__ __forceinline__ uint64_t sdesc_across(uint32_t saddr) { return tc::smem_desc(saddr, 8192, 1024, 2); }

// Rows of x that are gathered come four at a time (TMA's gather; its map has boxes
// of one row).  A warp takes some 100 cycles to issue one, so four warps share a
// step's, and two sets of four take the steps in turn: 64 gathers by one warp took
// 2.4 us.
constexpr int GATHER_WARPS = 8, GATHER_SHARE = 4, GATHER_TURNS = GATHER_WARPS / GATHER_SHARE;

// The row of x of a slot; past its end, which reads as zeros, for none.
__device__ __forceinline__ int row_of(const Args& g, int pair) { return pair >= 0 ? min(pair / g.k, g.x_rows) : g.x_rows; }

// Four rows: of a tile's rows q0 .. q0 + n - 1 those of a group.
struct GatherRows {
    int at[4];
    __device__ __forceinline__ void read(const Args& g, int q0, int n, int group) {
#pragma unroll
        for (int i = 0; i < 4; ++i) at[i] = group * 4 + i < n ? g.pairs[q0 + group * 4 + i] : -1;
    }
    __device__ __forceinline__ void to_rows(const Args& g) {
#pragma unroll
        for (int i = 0; i < 4; ++i) at[i] = row_of(g, at[i]);
    }
    // from the rows of x of all slots
    __device__ __forceinline__ void take(const Args& g, const int* rows, int q0, int n, int group) {
#pragma unroll
        for (int i = 0; i < 4; ++i) at[i] = group * 4 + i < n ? rows[q0 + group * 4 + i] : g.x_rows;
    }
};
// So few slots that a CTA reads where all their rows lie while it waits for the
// offsets, and the first gather waits for no load of its own.
constexpr int FEW_SLOTS = 128;

__device__ __forceinline__ void tma_gather4(void* dst, const CUtensorMap* map, uint64_t* bar, int x, const GatherRows& r) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, "
        "%5, %6, %7}], [%2];" ::"r"(tc::smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(tc::smem_u32(bar)), "r"(x), "r"(r.at[0]), "r"(r.at[1]), "r"(r.at[2]), "r"(r.at[3])
        : "memory");
}

// One lane waits (a wait by all 32 takes four times as long even where the phase is
// over); __syncwarp passes on to the others what the barrier guards.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int32_t* status) {
    int ok = 1;
    if ((threadIdx.x & 31) == 0 && !tc::mbar_wait(bar, parity)) {
        *abort_flag = 1;
        atomicOr(status, QMOE_DEV_WAIT_TIMEOUT);
        ok = 0;
    }
    ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
    __syncwarp();
    return ok != 0;
}

// A bounded wait of one lane; false, and the flag set, where it ran out.
__device__ __forceinline__ bool lane_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int32_t* status) {
    if (tc::mbar_wait(bar, parity)) return true;
    *abort_flag = 1;
    atomicOr(status, QMOE_DEV_WAIT_TIMEOUT);
    return false;
}
// One lane waits for a warp that issues products; the answer by a vote, which the
// compiler knows to be the same for all lanes, so that what comes behind stays in
// uniform registers (by a shuffle each step took 130 cycles longer: 8 x 65 rows 1536 ->
// 768 12.8 us for 11.1).
__device__ __forceinline__ bool issue_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int32_t* status) {
    bool ok = true;
    if ((threadIdx.x & 31) == 0) ok = lane_wait(bar, parity, abort_flag, status);
    return __all_sync(0xFFFFFFFFu, ok);
}
// After a wait that ran out: time for the loads and products in flight to end (they
// take microseconds), so that none outlives the CTA.
__device__ __forceinline__ void wind_down(volatile int* abort_flag) {
    if (*abort_flag)
        for (const long long t0 = clock64(); clock64() - t0 < 4000000ll;) __nanosleep(1000);
}

// 32 columns of this warp's 32 lanes.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
        "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
        "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
        : "memory");
}

// A tile: its expert, first lane, first column (a row s, or a column of dw), the
// columns it has and its reduction steps.
struct Unit {
    int e, l0, q0, n, steps;
    int row0, end;  // dw: the expert's rows
};

// The units, in order.  For y and dx an expert has ceil(lanes / LT) tiles for
// each of its ceil(count / cap) parts of about the same number of rows (a multiple
// of ROUND); after the experts come the rows of none, whose outputs are zeros.
template <int LT, int ROUND>
struct Walk {
    const Args& g;
    const int* off;   // [E + 1], clamped to [0, P]
    const int* base;  // [E + 2]: units before expert e
    int cap;          // most columns of a tile
    int e = 0;
    __device__ Walk(const Args& g_, const int* off_, const int* base_, int cap_) : g(g_), off(off_), base(base_), cap(cap_) {}
    __device__ int total() const { return base[g.E + 1]; }
    __device__ Unit at(int u) {
        const int lt = (g.lanes + LT - 1) / LT;
        Unit t;
        if (u >= base[e + 1]) {  // the last expert that starts at u or before (empty ones start where the next does)
            int hi = g.E;
            ++e;
            while (e < hi) {
                const int mid = (e + hi + 1) >> 1;
                if (base[mid] <= u) e = mid;
                else hi = mid - 1;
            }
        }
        t.e = e;
        const int i = u - base[e], q = i / lt;
        const int r0 = off[e], count = (e < g.E ? off[e + 1] : g.P) - r0;
        const int qt = (count + cap - 1) / cap, per = ((count + qt - 1) / qt + ROUND - 1) & ~(ROUND - 1);
        t.l0 = (i - q * lt) * LT;
        t.q0 = r0 + q * per;
        t.n = min(per, r0 + count - t.q0);
        t.row0 = t.end = 0;
        t.steps = e < g.E ? g.steps : 0;
        return t;
    }
};

// The units of dw: the tiles of an expert, then the next one's.  The offsets are
// read where they are used, a unit ahead (shared memory has no room for them).
template <int LT, int NT>
struct WalkDw {
    const Args& g;
    int stride, lt, per;  // tiles of lanes, of an expert
    int e, i, a, b;       // the next unit's expert, place among its tiles, and offsets
    __device__ WalkDw(const Args& g_, int first, int stride_) : g(g_), stride(stride_) {
        lt = (g.lanes + LT - 1) / LT;
        per = lt * ((g.cols + NT - 1) / NT);
        e = first / per;
        i = first - e * per;
        read();
    }
    __device__ int total() const { return g.E * per; }
    __device__ void read() {
        const int32_t* from = g.offsets + min(e, g.E - 1);
        a = from[0];
        b = from[1];
    }
    __device__ Unit at(int) {
        Unit t;
        const int q = i / lt;
        t.e = e;
        t.l0 = (i - q * lt) * LT;
        t.q0 = q * NT;
        t.n = min(NT, g.cols - t.q0);
        t.row0 = min(max(a, 0), g.P);
        t.end = min(max(b, t.row0), g.P);
        t.steps = (t.end - t.row0 + STEP - 1) / STEP;
        i += stride;
        if (i >= per) {
            const int more = i / per;
            e += more;
            i -= more * per;
            read();
        }
        return t;
    }
};
// Offsets that fall, or lie outside [0, P].
__device__ __forceinline__ void check_offsets(const Args& g) {
    bool bad = false;
    for (int i = threadIdx.x; i <= g.E; i += blockDim.x) {
        const int o = g.offsets[i], next = i < g.E ? g.offsets[i + 1] : o;
        bad |= o < 0 || o > g.P || next < o || (i == 0 && o != 0);
    }
    if (bad) atomicOr(g.status, QMOE_DEV_BAD_OFFSETS);
}

// 32 columns of this warp's 32 lanes as 8 x 8 matrices: lane t holds of lanes
// 8 m + t / 4 the columns 8 i + 2 (t % 4) and the next, for m = 0, 1 in r[4 i ..],
// for m = 2, 3 in r[16 + 4 i ..].
__device__ __forceinline__ void tmem_ld_half_matrices(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_matrices(uint32_t taddr, uint32_t (&r)[32]) {
#pragma unroll
    for (int h = 0; h < 32; h += 16) tmem_ld_half_matrices(taddr + ((uint32_t)h << 16), r + h);
}
// A warp stores 32 columns of its 32 lanes in two steps: from registers to shared
// memory (stage_*), and on to HBM (send_*), so that a loop over columns, which lie in
// other registers each time, has the second one's code once.

// y or dx in 16 bits, from matrices: transposed on their way to shared memory, so that
// a column (a row of y) lies there as it is stored.  16-byte pieces of 64-byte rows,
// changed about so that 8 rows fall on all banks.
__device__ __forceinline__ int place_matrices(int row, int p) { return row * 64 + ((p ^ (row >> 1 & 3)) * 16); }
template <typename T>
__device__ __forceinline__ void stage_matrices(uint8_t* stage, int lane, const uint32_t (&r)[32]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t w[4];
#pragma unroll
        for (int m = 0; m < 4; ++m)
            w[m] = row::pack2(__uint_as_float(r[(m >> 1) * 16 + 4 * i + (m & 1) * 2]),
                              __uint_as_float(r[(m >> 1) * 16 + 4 * i + (m & 1) * 2 + 1]), T{});
        asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(
                         tc::smem_u32(stage + place_matrices(8 * i + (lane & 7), lane >> 3))),
                     "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                     : "memory");
    }
}
__device__ __forceinline__ void send_matrices(const Args& g, uint8_t* stage, int l0, int q0, int n, int lane) {
    __syncwarp();
    const int l = l0 + (lane & 3) * 8, row = lane >> 2;
    const uint8_t* const from = stage + place_matrices(row, lane & 3);  // and every 8th row
    uint16_t* to = static_cast<uint16_t*>(g.out) + (int64_t)(q0 + row) * g.ld + l;  // two types of two bytes
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const uint4*>(from + i * 8 * 64);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (row + i * 8 < n && l + 8 <= g.lanes) {
            *reinterpret_cast<uint4*>(to) = v[i];
        } else if (row + i * 8 < n) {
            for (int j = 0; j < 8 && l + j < g.lanes; ++j) to[j] = reinterpret_cast<const uint16_t*>(&v[i])[j];
        }
        to += 8 * g.ld;
    }
    __syncwarp();
}

// 32 columns of y or dx: lane l holds output l0 + l of rows q0 .. q0 + n - 1.
template <typename T>
__device__ __forceinline__ void put_rows(const Args& g, int l0, int q0, int n, int lane, const uint32_t (&r)[32]) {
    T* const out = static_cast<T*>(g.out);
    if (l0 + lane < g.lanes) {
        T* to = out + (int64_t)q0 * g.ld + l0 + lane;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            if (j < n) *to = row::from_f32<T>(__uint_as_float(r[j]));
            to += g.ld;
        }
    }
}

// 32 columns of dw: lane l holds columns q0 .. q0 + n - 1 of row l0 + l.  Through
// shared memory, so that rows of 128 bytes (64 in 16 bits) are written whole: by a TMA
// store (BULK), which runs while the warp goes on and leaves out what lies outside the
// expert's matrix, or by the warp's own stores, where TMA is to feed long sums at the
// same time.  us with the warp's stores and with TMA's, in fp32 and in bf16, rows an
// expert: 512 x 8 (1024 x 2048) 752 and 742, 557 and 464; 64 x 80 (2816 x 4096) 528
// and 559, 389 and 269; 128 x 256 (2048 x 768) 166 and 185, 119 and 108; 64 x 512
// (2816 x 2048) 339 and 351, 268 and 268.
//
// Where a row's piece of 16 bytes lies: rows that are read or written together fall on
// all banks, and the store's swizzle has it so.
template <typename T>
__device__ __forceinline__ int place_dw(int row, int p) {
    return row * 32 * (int)sizeof(T) + ((p ^ (sizeof(T) == 4 ? row & 7 : row >> 1 & 3)) * 16);
}
template <bool BULK, typename T>
__device__ __forceinline__ void stage_dw(uint8_t* stage, int lane, const uint32_t (&r)[32]) {
    constexpr int PER = 16 / sizeof(T), PIECES = 32 / PER;  // of 16 bytes
    static_assert(32 * 32 * sizeof(T) <= STAGE_DW, "");
    if constexpr (BULK) {
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        __syncwarp();
    }
    int at = place_dw<T>(lane, 0);
    asm volatile("" : "+r"(at));  // one address, not one for each piece that is kept over all tiles
#pragma unroll
    for (int p = 0; p < PIECES; ++p) {
        uint4 v;
        uint32_t* w = &v.x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 2)
                w[i] = row::pack2(__uint_as_float(r[p * 8 + 2 * i]), __uint_as_float(r[p * 8 + 2 * i + 1]), T{});
            else
                w[i] = r[p * 4 + i];
        }
        *reinterpret_cast<uint4*>(stage + (at ^ p * 16)) = v;
    }
}
template <bool BULK, typename T>
__device__ __forceinline__ void send_dw(const Args& g, const CUtensorMap* map, uint8_t* stage, int e, int l0, int q0, int n, int lane) {
    constexpr int PER = 16 / sizeof(T), PIECES = 32 / PER, ROWS = 32;
    T* const out = static_cast<T*>(g.out) + (int64_t)e * g.out_e;
    if constexpr (BULK) {
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && l0 < g.lanes && n > 0) {
            asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                             reinterpret_cast<uint64_t>(map)),
                         "r"(tc::smem_u32(stage)), "r"(q0), "r"(l0), "r"(e)
                         : "memory");
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        }
        __syncwarp();  // what follows reads TMEM, which all lanes do together
        return;
    }
    __syncwarp();
    if (g.wide) {
        constexpr int EACH = 32 / PIECES;  // rows of an instruction
        const int row = lane / PIECES, p = lane % PIECES, c = p * PER;
        int at = place_dw<T>(row, p);
        asm volatile("" : "+r"(at));
        T* to = out + (int64_t)(l0 + row) * g.ld + q0 + c;
#pragma unroll
        for (int i = 0; i < ROWS / EACH; ++i) {
            // in fp32 rows 4 apart have their pieces 4 apart
            const uint4 v = *reinterpret_cast<const uint4*>(stage + (sizeof(T) == 4 ? at ^ (i & 1) * 64 : at) + i * EACH * 32 * sizeof(T));
            if (l0 + row + i * EACH < g.lanes && c < n) {
                if (c + PER <= n) {
                    *reinterpret_cast<uint4*>(to) = v;
                } else {
                    for (int j = 0; j < PER && c + j < n; ++j) to[j] = reinterpret_cast<const T*>(&v)[j];
                }
            }
            to += EACH * g.ld;
        }
    } else {
        T* to = out + (int64_t)l0 * g.ld + q0 + lane;
        const int rows = lane < n ? min(ROWS, g.lanes - l0) : 0;
#pragma unroll
        for (int r0 = 0; r0 < ROWS; r0 += 16) {  // all reads of shared memory, then all stores
            T v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = reinterpret_cast<const T*>(stage + place_dw<T>(r0 + i, lane / PER))[lane % PER];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                if (r0 + i < rows) *to = v[i];
                to += g.ld;
            }
        }
    }
    __syncwarp();
}

// Whether a warp takes its sums from TMEM as matrices.
template <int MODE>
__device__ __forceinline__ bool by_matrices(const Args& g) { return MODE != DW && g.wide && g.ctype != QMOE_F32; }

template <int MODE>
__device__ __forceinline__ void take(bool matrices, uint32_t taddr, uint32_t (&r)[32]) {
    if (MODE != DW && matrices) tmem_ld_matrices(taddr, r);
    else tmem_ld32(taddr, r);
}
// Sums of weights that were divided by a power of two.
__device__ __forceinline__ void multiply(const Args& g, bool matrices, int l0, int lane, uint32_t (&r)[32]) {
    auto of = [&](int l) { return l < g.lanes ? g.by[l] : 0.f; };
    if (matrices) {
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const float f = of(l0 + 8 * m + (lane >> 2));
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                uint32_t& v = r[(m >> 1) * 16 + (i >> 1) * 4 + (m & 1) * 2 + (i & 1)];
                v = __float_as_uint(__uint_as_float(v) * f);
            }
        }
    } else {
        const float f = of(l0 + lane);
#pragma unroll
        for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * f);
    }
}
// BY: with the lanes' factors (in code of its own: 16 x 47 rows 128 -> 3157 8.5 us beside them, 7.8 without).
template <int MODE, bool BULK, bool BY>
__device__ __forceinline__ void stage_sums(const Args& g, bool matrices, uint8_t* stage, int l0, int q0, int n, int lane,
                                           uint32_t (&r)[32]) {
    if constexpr (BY) multiply(g, matrices, l0, lane, r);
    if constexpr (MODE == DW) {
        if (g.ctype == QMOE_F32) stage_dw<BULK, float>(stage, lane, r);
        else if (g.ctype == QMOE_BF16) stage_dw<BULK, __nv_bfloat16>(stage, lane, r);
        else stage_dw<BULK, __half>(stage, lane, r);
    } else if (matrices) {
        if (g.ctype == QMOE_BF16) stage_matrices<__nv_bfloat16>(stage, lane, r);
        else stage_matrices<__half>(stage, lane, r);
    } else {
        if (g.ctype == QMOE_F32) put_rows<float>(g, l0, q0, n, lane, r);
        else if (g.ctype == QMOE_BF16) put_rows<__nv_bfloat16>(g, l0, q0, n, lane, r);
        else put_rows<__half>(g, l0, q0, n, lane, r);
    }
}
template <int MODE, bool BULK>
__device__ __forceinline__ void send_sums(const Args& g, const CUtensorMap* map, bool matrices, uint8_t* stage, int e, int l0, int q0,
                                          int n, int lane) {
    if constexpr (MODE == DW) {
        if (g.ctype == QMOE_F32) send_dw<BULK, float>(g, map, stage, e, l0, q0, n, lane);
        else send_dw<BULK, uint16_t>(g, map, stage, e, l0, q0, n, lane);  // two types of two bytes
    } else if (matrices) {
        send_matrices(g, stage, l0, q0, n, lane);
    }
}
template <int MODE, bool BULK, bool BY>
__device__ __forceinline__ void put(const Args& g, const CUtensorMap* map, bool matrices, uint8_t* stage, int e, int l0, int q0, int n,
                                    int lane, uint32_t (&r)[32]) {
    stage_sums<MODE, BULK, BY>(g, matrices, stage, l0, q0, n, lane, r);
    send_sums<MODE, BULK>(g, map, matrices, stage, e, l0, q0, n, lane);
}

// The offsets, clamped to [0, P] and raised to the largest before them (no row
// has two experts, whatever they say), and the units before each expert, by all
// threads of the CTA; the caller's barrier makes them seen.  Chunks of 32 experts
// are scanned by a warp each, all at once (one warp after the other took 2 us of
// the 10 of a decoded token).
//
// Returns the most columns of a tile: CAP, or where `workers` then take their last
// tiles in a round of few, 7/8 or 6/8 of it if that makes for a shorter sum of rounds
// (2048 rows, 2816 outputs: 88 tiles of 256 are two rounds of 76, and so are 121 of
// 192).  Fewer columns do not make a step of the reduction shorter.
template <int LT, int CAP, bool CHOOSE>
__device__ __forceinline__ int read_offsets(const Args& g, int* off, int* base, int workers = 0) {
    constexpr int CHUNKS = (MAX_E + 32) / 32;
    __shared__ int sums[CHUNKS], parts[2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    if (CHOOSE && threadIdx.x < 2) parts[threadIdx.x] = 0;
    bool bad = false;
    for (int i = threadIdx.x; i <= g.E; i += blockDim.x) {
        const int o = g.offsets[i], next = i < g.E ? g.offsets[i + 1] : o;
        bad |= o < 0 || o > g.P || next < o || (i == 0 && o != 0);
        off[i] = min(max(o, 0), g.P);
    }
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) {
            atomicOr(g.status, QMOE_DEV_BAD_OFFSETS);
            for (int i = 1; i <= g.E; ++i) off[i] = max(off[i], off[i - 1]);
        }
        __syncthreads();
    }
    const int lt = (g.lanes + LT - 1) / LT;
    // parts of expert i for tiles of cap columns
    auto parts_of = [&](int i, int cap) {
        const int count = i < g.E ? off[i + 1] - off[i] : i == g.E ? g.P - off[i] : 0;
        return (count + cap - 1) / cap;
    };
    auto scan = [&](int cap) {
        for (int c = warp; c * 32 <= g.E; c += warps) {
            const int i = c * 32 + lane;
            int v = parts_of(i, cap) * lt;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int w = __shfl_up_sync(0xFFFFFFFFu, v, o);
                if (lane >= o) v += w;
            }
            if (i <= g.E) base[i + 1] = v;
            if (lane == 31) sums[c] = v;
        }
    };
    int cap = CAP;
    if (CHOOSE) {
        int a = 0, b = 0;
        for (int i = threadIdx.x; i < g.E; i += blockDim.x) {
            a += parts_of(i, CAP * 7 / 8);
            b += parts_of(i, CAP * 6 / 8);
        }
        if (a) atomicAdd(&parts[0], a);
        if (b) atomicAdd(&parts[1], b);
    }
    scan(cap);
    if (threadIdx.x == 0) base[0] = 0;
    if (!CHOOSE && g.E < 32) return cap;
    __syncthreads();
    if (CHOOSE) {
        int units = 0;
        for (int c = 0; c * 32 <= g.E; ++c) units += sums[c];
        if (units < 8 * workers) {
            auto cost = [&](int n, int columns) { return (n + workers - 1) / workers * columns; };
            const int whole = cost(units, 8), a = cost(parts[0] * lt, 7), b = cost(parts[1] * lt, 6);
            if (a < whole || b < whole) cap = a <= b ? CAP * 7 / 8 : CAP * 6 / 8;
        }
        if (cap != CAP) {
            __syncthreads();
            scan(cap);
            __syncthreads();
        }
    }
    if (g.E < 32) return cap;
    for (int c = warp; c * 32 <= g.E; c += warps) {
        int before = 0;
        for (int j = lane; j < c; j += 32) before += sums[j];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xFFFFFFFFu, before, o);
        const int i = c * 32 + lane;
        if (i <= g.E) base[i + 1] += before;
    }
    return cap;
}

__device__ __forceinline__ void put_value(void* y, int type, int64_t at, float v) {
    if (type == QMOE_F32) static_cast<float*>(y)[at] = v;
    else if (type == QMOE_BF16) static_cast<__nv_bfloat16*>(y)[at] = __float2bfloat16_rn(v);
    else static_cast<__half*>(y)[at] = __float2half_rn(v);
}

// A matrix of 16-bit values, or one for each expert.
struct Mat {
    const void* p;
    int64_t rows, cols, ld, experts, stride;
};
// Whether all its rows start on 16-byte boundaries.
inline bool fits(const Mat& m) {
    return aligned16(m.p) && (m.rows == 1 || m.ld % 8 == 0) && (m.experts == 1 || m.stride % 8 == 0);
}

// Products with one matrix, the sum of w [parts, N, K] (parts 1 or 2; contiguous rows of
// a multiple of 8 values), each of whose rows (y) or columns (dx) stands for `by` times
// what it holds.  ws: scaled_bytes (dx: 0 or 1).  offsets: {0, T} on the device.
struct Scaled {
    const void* w;
    int parts;
    const float* by;
    int64_t T, N, K;
    int dtype;
    const int32_t* offsets;
    int32_t* status;
    void* ws;
    size_t ws_bytes;
};
size_t scaled_bytes(int64_t T, int64_t N, int64_t K, int parts, int dx);
int scaled_linear(const Scaled& c, const void* x, int64_t ldx, void* y, int y_dtype, int64_t ldy, cudaStream_t st);
int scaled_linear_dx(const Scaled& c, const void* dy, int64_t lddy, void* dx, int dx_dtype, int64_t lddx, cudaStream_t st);

// y for few rows an expert, of any alignment.
int launch_few(const Mat& w, const Mat& x, const Args& g, int dtype, cudaStream_t st);

// What the kernels take: map_p of the lane side, map_q of the column side.
//
// Pairs of CTAs, 256 x 256 tiles: for many rows an expert, and for dw.
// BULK: dw goes out by TMA stores of 32 x 32 values, by way of mo.  BY: y and dx of a Scaled.
template <int MODE, bool BULK = false, bool BY = false>
int launch_pair(const CUtensorMap& mp, const CUtensorMap& mq, const CUtensorMap& mo, const Args& g, int64_t most, cudaStream_t st);

}  // namespace eg
}  // namespace qmoe
