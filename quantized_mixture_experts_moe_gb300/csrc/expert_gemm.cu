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
#include "row_ops.cuh"
#include "tc_ptx.cuh"
#include "tma_host.cuh"

namespace qmoe {
namespace eg {

enum { FWD = 0, DX = 1, DW = 2 };

// Warps: 8 read sums and store them (two for each quadrant of lanes), one loads
// tiles, one issues products.
constexpr int EPI_WARPS = 8, WARP_TMA = 8, WARP_MMA = 9, THREADS = 10 * 32;
constexpr int STEP = 64;         // reduction values of a stage: 128 bytes
constexpr int MAX_E = 1024;
constexpr int STAGE_OUT = 2048;  // bytes of a warp's output stage: 32 rows of 64
constexpr int Q_BOX = 32;        // rows of a box of the column side (y, dx)

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
    uint32_t idesc;        // without N
    int32_t* status;
};

template <int MODE, int NT>
struct Cfg {
    static constexpr int P_BYTES = 128 * STEP * 2, Q_BYTES = NT * STEP * 2, STAGE = P_BYTES + Q_BYTES;
    static constexpr int TMEM_COLS = 2 * NT < 32 ? 32 : 2 * NT;
    static constexpr int LIST = (MODE == DW ? MAX_E + 1 : 2 * (MAX_E + 2)) * 4;
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

// Operand whose reduction axis is not the contiguous one: blocks of 64 lanes (or
// columns), 8192 bytes apart; in each, reduction rows of 128 bytes, swizzled in
// groups of 8 rows.
__device__ __forceinline__ uint64_t sdesc_across(uint32_t saddr) { return tc::smem_desc(saddr, 8192, 1024, 2); }

// Four rows of a map with boxes of one row.
__device__ __forceinline__ void tma_gather4(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int r0, int r1, int r2,
                                            int r3) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, "
        "%5, %6, %7}], [%2];" ::"r"(tc::smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(tc::smem_u32(bar)), "r"(x), "r"(r0), "r"(r1), "r"(r2), "r"(r3)
        : "memory");
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

// A tile: its expert, first lane, first column (a row s, or a column of dw), the
// columns it has and its reduction steps.
struct Unit {
    int e, l0, q0, n, steps, row0;
};

// The units, in order.  For y and dx an expert has ceil(lanes / 128) tiles for
// each of its ceil(count / NT) parts of about the same number of rows; after the
// experts come the rows of none, whose outputs are zeros.
template <int MODE, int NT>
struct Walk {
    const Args& g;
    const int* off;   // [E + 1], clamped to [0, P]
    const int* base;  // [E + 2]: units before expert e (y, dx)
    int e = 0;
    __device__ Walk(const Args& g_, const int* off_, const int* base_) : g(g_), off(off_), base(base_) {}
    __device__ int total() const {
        if (MODE == DW) return g.E * ((g.lanes + 127) / 128) * ((g.cols + NT - 1) / NT);
        return base[g.E + 1];
    }
    __device__ Unit at(int u) {
        const int lt = (g.lanes + 127) / 128;
        Unit t;
        if (MODE == DW) {
            const int qt = (g.cols + NT - 1) / NT;
            t.e = u / (lt * qt);
            const int i = u - t.e * lt * qt;
            t.l0 = (i % lt) * 128;
            t.q0 = (i / lt) * NT;
            t.n = min(NT, g.cols - t.q0);
            t.row0 = off[t.e];
            t.steps = (off[t.e + 1] - t.row0 + STEP - 1) / STEP;
        } else {
            while (u >= base[e + 1]) ++e;
            t.e = e;
            const int i = u - base[e], q = i / lt;
            const int r0 = off[e], count = (e < g.E ? off[e + 1] : g.P) - r0;
            const int qt = (count + NT - 1) / NT, per = ((count + qt - 1) / qt + 15) & ~15;
            t.l0 = (i - q * lt) * 128;
            t.q0 = r0 + q * per;
            t.n = min(per, r0 + count - t.q0);
            t.row0 = 0;
            t.steps = e < g.E ? (g.red + STEP - 1) / STEP : 0;
        }
        return t;
    }
};

template <typename T> struct Bits;
template <> struct Bits<__nv_bfloat16> {
    static __device__ __forceinline__ uint16_t of(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }
};
template <> struct Bits<__half> {
    static __device__ __forceinline__ uint16_t of(float v) { return __half_as_ushort(__float2half_rn(v)); }
};

// 32 columns of y or dx: lane l holds output l0 + l of rows q0 .. q0 + n - 1.
template <typename T>
__device__ __forceinline__ void put_rows(const Args& g, uint8_t* stage, int l0, int q0, int n, int lane,
                                         const uint32_t (&r)[32]) {
    T* const out = static_cast<T*>(g.out);
    if constexpr (sizeof(T) == 2) {
        if (g.wide) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
                *reinterpret_cast<uint16_t*>(stage + j * 64 + lane * 2) = Bits<T>::of(__uint_as_float(r[j]));
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = i * 8 + (lane >> 2), l = l0 + (lane & 3) * 8;
                const uint4 v = *reinterpret_cast<const uint4*>(stage + row * 64 + (lane & 3) * 16);
                if (row < n && l < g.lanes) {
                    T* const to = out + (int64_t)(q0 + row) * g.ld + l;
                    if (l + 8 <= g.lanes) {
                        *reinterpret_cast<uint4*>(to) = v;
                    } else {
                        for (int j = 0; j < 8 && l + j < g.lanes; ++j) to[j] = reinterpret_cast<const T*>(&v)[j];
                    }
                }
            }
            __syncwarp();
            return;
        }
    }
    if (l0 + lane < g.lanes) {
        T* to = out + (int64_t)q0 * g.ld + l0 + lane;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            if (j < n) *to = row::from_f32<T>(__uint_as_float(r[j]));
            to += g.ld;
        }
    }
}

// 32 columns of dw: lane l holds columns q0 .. q0 + n - 1 of row l0 + l.
template <typename T>
__device__ __forceinline__ void put_dw(const Args& g, uint8_t* stage, int e, int l0, int q0, int n, int lane,
                                       const uint32_t (&r)[32]) {
    constexpr int PER = 16 / sizeof(T), COLS = 64 / sizeof(T);
    T* const out = static_cast<T*>(g.out) + (int64_t)e * g.out_e;
#pragma unroll
    for (int h = 0; h < 32 / COLS; ++h) {
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            uint4 v;
            uint32_t* w = &v.x;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (sizeof(T) == 2)
                    w[i] = row::pack2(__uint_as_float(r[p * 8 + 2 * i]), __uint_as_float(r[p * 8 + 2 * i + 1]), T{});
                else
                    w[i] = r[h * 16 + p * 4 + i];
            }
            *reinterpret_cast<uint4*>(stage + lane * 64 + ((p ^ (lane >> 1 & 3)) * 16)) = v;
        }
        __syncwarp();
        if (g.wide) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = i * 8 + (lane >> 2), p = lane & 3, c = h * COLS + p * PER;
                const uint4 v = *reinterpret_cast<const uint4*>(stage + row * 64 + ((p ^ (row >> 1 & 3)) * 16));
                if (l0 + row < g.lanes && c < n) {
                    T* const to = out + (int64_t)(l0 + row) * g.ld + q0 + c;
                    if (c + PER <= n) {
                        *reinterpret_cast<uint4*>(to) = v;
                    } else {
                        for (int j = 0; j < PER && c + j < n; ++j) to[j] = reinterpret_cast<const T*>(&v)[j];
                    }
                }
            }
        } else {
            const int col = lane % COLS, c = h * COLS + col;
#pragma unroll 4
            for (int row = lane / COLS; row < 32; row += 32 / COLS) {
                const T v = reinterpret_cast<const T*>(stage + row * 64 + (((col / PER) ^ (row >> 1 & 3)) * 16))[col % PER];
                if (l0 + row < g.lanes && c < n) out[(int64_t)(l0 + row) * g.ld + q0 + c] = v;
            }
        }
        __syncwarp();
    }
}

template <int MODE>
__device__ __forceinline__ void put(const Args& g, uint8_t* stage, int e, int l0, int q0, int n, int lane,
                                    const uint32_t (&r)[32]) {
    if constexpr (MODE == DW) {
        if (g.ctype == QMOE_F32) put_dw<float>(g, stage, e, l0, q0, n, lane, r);
        else if (g.ctype == QMOE_BF16) put_dw<__nv_bfloat16>(g, stage, e, l0, q0, n, lane, r);
        else put_dw<__half>(g, stage, e, l0, q0, n, lane, r);
    } else {
        if (g.ctype == QMOE_F32) put_rows<float>(g, stage, l0, q0, n, lane, r);
        else if (g.ctype == QMOE_BF16) put_rows<__nv_bfloat16>(g, stage, l0, q0, n, lane, r);
        else put_rows<__half>(g, stage, l0, q0, n, lane, r);
    }
}

template <int MODE, int NT, bool GATHER>
__global__ void __launch_bounds__(THREADS, 1)
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
    bool bad = false;
    for (int i = threadIdx.x; i <= g.E; i += THREADS) {
        const int o = g.offsets[i], next = i < g.E ? g.offsets[i + 1] : o;
        bad |= o < 0 || o > g.P || next < o || (i == 0 && o != 0);
        off[i] = min(max(o, 0), g.P);
    }
    if (bad) atomicOr(g.status, QMOE_DEV_BAD_OFFSETS);
    __syncthreads();
    if (warp == 0) {
        // offsets that fall are raised to the largest before them: no row has two experts, whatever they say
        int most = 0;
        for (int i0 = 0; i0 <= g.E; i0 += 32) {
            const int i = i0 + lane;
            int v = max(i <= g.E ? off[i] : 0, most);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) v = max(v, __shfl_up_sync(0xFFFFFFFFu, v, o));
            if (i <= g.E) off[i] = v;
            most = __shfl_sync(0xFFFFFFFFu, v, 31);
        }
        __syncwarp();
    }
    if (MODE != DW && warp == 0) {
        const int lt = (g.lanes + 127) / 128;
        int sum = 0;
        for (int i0 = 0; i0 <= g.E; i0 += 32) {
            const int i = i0 + lane;
            const int count = i < g.E ? off[i + 1] - off[i] : i == g.E ? g.P - off[i] : 0;
            int v = (count + NT - 1) / NT * lt;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int w = __shfl_up_sync(0xFFFFFFFFu, v, o);
                if (lane >= o) v += w;
            }
            if (i <= g.E) base[i + 1] = sum + v;
            sum += __shfl_sync(0xFFFFFFFFu, v, 31);
        }
        if (lane == 0) base[0] = 0;
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tm = *tmem_at;
    Walk<MODE, NT> walk(g, off, base);
    const int total = walk.total();

    if (warp == WARP_TMA) {
        int slot = 0, in_flight = 0;
        uint32_t phase = 0;
        for (int u = blockIdx.x; u < total && !*abort_flag; u += gridDim.x) {
            const Unit t = walk.at(u);
            // this lane's rows of x, where they are gathered: 4 rows of groups lane and lane + 32
            int rows[2][4];
            if (GATHER && MODE == FWD) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int i = (h * 32 + lane) * 4 + j;
                        const int p = i < t.n && t.steps ? g.pairs[t.q0 + i] : -1;
                        rows[h][j] = p >= 0 ? p / g.k : g.x_rows;  // past the end: zeros
                    }
            }
            for (int s = 0; s < t.steps; ++s) {
                int ok = 1;
                if (lane == 0) ok = tc::mbar_wait(&empty[slot], phase ^ 1);
                ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
                if (!ok) {
                    if (lane == 0) {
                        *abort_flag = 1;
                        atomicOr(g.status, QMOE_DEV_WAIT_TIMEOUT);
                    }
                    __syncwarp();
                    break;
                }
                uint8_t* st = smem + slot * C::STAGE;
                uint8_t* sq = st + C::P_BYTES;
                const int k0 = s * STEP;
                if constexpr (MODE == FWD || MODE == DX) {
                    const int boxes = GATHER ? 0 : (t.n + Q_BOX - 1) / Q_BOX, groups = GATHER ? (t.n + 3) / 4 : 0;
                    if (lane == 0)
                        tc::mbar_arrive_expect_tx(&full[slot], C::P_BYTES + boxes * Q_BOX * 128 + groups * 512);
                    __syncwarp();
                    if (lane == 0) {
                        if constexpr (MODE == FWD) {
                            tc::tma_load_3d(st, &map_p, &full[slot], k0, t.l0, t.e);
                        } else {
                            tc::tma_load_3d(st, &map_p, &full[slot], t.l0, k0, t.e);
                            tc::tma_load_3d(st + 8192, &map_p, &full[slot], t.l0 + 64, k0, t.e);
                        }
                    }
                    if constexpr (GATHER) {
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            if (h * 32 + lane < groups)
                                tma_gather4(sq + (h * 32 + lane) * 512, &map_q, &full[slot], k0, rows[h][0], rows[h][1],
                                            rows[h][2], rows[h][3]);
                    } else if (lane < boxes) {
                        tc::tma_load_2d(sq + lane * Q_BOX * 128, &map_q, &full[slot], k0, t.q0 + lane * Q_BOX);
                    }
                } else {
                    const int blocks = (t.n + 63) / 64, row = t.row0 + k0;
                    const int left = off[t.e + 1] - row, groups = (min(left, STEP) + 3) / 4;
                    if (lane == 0)
                        tc::mbar_arrive_expect_tx(&full[slot],
                                                  C::P_BYTES + blocks * (GATHER ? groups * 512 : 8192));
                    __syncwarp();
                    if (lane < 2) tc::tma_load_2d(st + lane * 8192, &map_p, &full[slot], t.l0 + lane * 64, row);
                    if constexpr (GATHER) {
                        // lane: group lane % 16, columns of blocks lane / 16, then + 2
                        const int gr = lane & 15;
                        int r[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int p = gr * 4 + j < left ? g.pairs[row + gr * 4 + j] : -1;
                            r[j] = p >= 0 ? p / g.k : g.x_rows;
                        }
                        for (int b = lane >> 4; b < blocks; b += 2)
                            if (gr < groups)
                                tma_gather4(sq + b * 8192 + gr * 512, &map_q, &full[slot], t.q0 + b * 64, r[0], r[1],
                                            r[2], r[3]);
                    } else if (lane < blocks) {
                        tc::tma_load_2d(sq + lane * 8192, &map_q, &full[slot], t.q0 + lane * 64, row);
                    }
                }
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
            const uint32_t idesc = g.idesc | (n16 >> 3) << 17;
            bool ok = true;
            if (lane == 0) ok = tc::mbar_wait(&acc_empty[buf], acc_phase ^ 1);
            for (int s = 0; s < t.steps; ++s) {
                if (lane == 0) ok = ok && tc::mbar_wait(&full[slot], phase);
                ok = __shfl_sync(0xFFFFFFFFu, (int)ok, 0) != 0;
                if (!ok) break;
                uint8_t* st = smem + slot * C::STAGE;
                int k16 = STEP / 16;
                if constexpr (MODE == DW) {
                    const int left = off[t.e + 1] - t.row0 - s * STEP;
                    if (left < STEP) {
                        // rows behind the expert's last, up to the 16 of a product, are another's: zeros in their place
                        k16 = (left + 15) / 16;
                        const int blocks = 2 + (t.n + 63) / 64, zero = k16 * 16 - left;
                        for (int i = lane; i < blocks * zero * 8; i += 32) {
                            const int b = i / (zero * 8), c = i - b * zero * 8;
                            *reinterpret_cast<uint4*>(st + b * 8192 + left * 128 + c * 16) = make_uint4(0, 0, 0, 0);
                        }
                        tc::fence_proxy_async_smem();
                        __syncwarp();
                    }
                }
                if (lane == 0) {
                    tc::tc_fence_after();
                    const uint32_t sa = tc::smem_u32(st), sb = sa + C::P_BYTES;
                    const uint64_t da = MODE == FWD ? tc::sdesc_kmajor_sw128(sa) : sdesc_across(sa);
                    const uint64_t db = MODE == DW ? sdesc_across(sb) : tc::sdesc_kmajor_sw128(sb);
                    constexpr int SA = MODE == FWD ? 2 : 128, SB = MODE == DW ? 128 : 2;  // of 16 values, in 16 bytes
                    for (int k = 0; k < k16; ++k)
                        tc::mma_f16(tm + buf * NT, da + SA * k, db + SB * k, idesc, s > 0 || k > 0);
                    tc::mma_commit(&empty[slot]);
                }
                __syncwarp();
                last = slot;
                last_phase = phase;
                if (++slot == C::STAGES) { slot = 0; phase ^= 1; }
            }
            if (!ok) {
                if (lane == 0) {
                    *abort_flag = 1;
                    atomicOr(g.status, QMOE_DEV_WAIT_TIMEOUT);
                }
                __syncwarp();
                break;
            }
            if (lane == 0) tc::mma_commit(&acc_full[buf]);
            __syncwarp();
            if (++buf == 2) { buf = 0; acc_phase ^= 1; }
        }
        if (*abort_flag && last >= 0 && lane == 0)  // no product outlives the accumulators
            tc::mbar_wait(&empty[last], last_phase);
        __syncwarp();
    } else {
        const int quad = warp & 3, half = warp >> 2;
        uint8_t* const stage = smem + C::OUT_OFF + warp * STAGE_OUT;
        int buf = 0;
        uint32_t acc_phase = 0;
        for (int u = blockIdx.x; u < total && !*abort_flag; u += gridDim.x) {
            const Unit t = walk.at(u);
            const int l0 = t.l0 + quad * 32;
            if (t.steps > 0) {
                int ok = 1;
                if (lane == 0 && !tc::mbar_wait_sleep(&acc_full[buf], acc_phase, 4000000000ll, 64)) {
                    *abort_flag = 1;
                    atomicOr(g.status, QMOE_DEV_WAIT_TIMEOUT);
                    ok = 0;
                }
                ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
                __syncwarp();
                if (!ok) break;
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

// Rows whose start TMA cannot address, copied to rows of whole 16-byte pieces.
__global__ void __launch_bounds__(256) pad_rows_kernel(const uint16_t* x, int64_t rows_inner, int64_t ld, int64_t outer,
                                                       int64_t cols, uint16_t* to, int64_t ldt, int64_t rows) {
    pdl_wait();
    pdl_trigger();
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const uint16_t* from = x + (r / rows_inner) * outer + (r % rows_inner) * ld;
        for (int64_t c = threadIdx.x; c < cols; c += 256) to[r * ldt + c] = from[c];
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

static int as_tma(Mat& m, uint8_t*& ws, size_t& left, cudaStream_t st) {
    if (fits(m)) {
        if (m.ld % 8) m.ld = (m.cols + 7) / 8 * 8;  // a single row: the stride is not used
        return QMOE_OK;
    }
    const int64_t rows = m.rows * m.experts, ld = (m.cols + 7) / 8 * 8;
    const size_t need = padded(rows, m.cols);
    if (need > left) return QMOE_ERR_ARG;
    const int64_t grid = rows < 8 * row::kSMs ? rows : 8 * row::kSMs;
    const int rc = launch_pdl(pad_rows_kernel, dim3((unsigned)grid), dim3(256), 0, st, static_cast<const uint16_t*>(m.p),
                              m.rows, m.ld, m.stride, m.cols, reinterpret_cast<uint16_t*>(ws), ld, rows);
    m.p = ws;
    m.ld = ld;
    m.stride = ld * m.rows;
    ws += need;
    left -= need;
    return rc;
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
    return launch_pdl(expert_gemm_kernel<MODE, NT, GATHER>, dim3((unsigned)grid), dim3(THREADS), (size_t)C::SMEM, st, mp, mq,
                      g);
}

// Few rows for each expert: narrow tiles, whose stages are almost all weight, so that more of them are in flight.
inline int tile_of(int64_t P, int E) {
    const int64_t touched = P < E ? P : E;
    return P <= 16 * touched ? 32 : P <= 96 * touched ? 128 : 256;
}

template <int MODE, bool GATHER>
static int run_rows(Mat w, Mat q, Args& g, int dtype, cudaStream_t st) {
    const int nt = tile_of(g.P, g.E);
    CUtensorMap mp, mq;
    int rc = MODE == FWD ? map_of(&mp, w, dtype, STEP, 128, true) : map_of(&mp, w, dtype, 64, STEP, true);
    if (rc != QMOE_OK) return rc;
    rc = map_of(&mq, q, dtype, STEP, GATHER ? 1 : Q_BOX, false);
    if (rc != QMOE_OK) return rc;
    // no more units than this, whatever the offsets
    const int64_t parts = (g.P < g.E ? g.P : g.E) + 1 + g.P / nt, most = parts * ((g.lanes + 127) / 128);
    if (most >= (1ll << 31)) return QMOE_ERR_UNSUPPORTED;
    switch (nt) {
        case 32: return launch<MODE, 32, GATHER>(mp, mq, g, most, st);
        case 128: return launch<MODE, 128, GATHER>(mp, mq, g, most, st);
        default: return launch<MODE, 256, GATHER>(mp, mq, g, most, st);
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
    if ((rc = eg::as_tma(mw, at, left, st)) != QMOE_OK || (rc = eg::as_tma(mx, at, left, st)) != QMOE_OK) return rc;
    const int size = row::dtype_size(y_dtype);
    eg::Args g = {(int)P, E, (int)N, 0, (int)K, offsets, pairs, k, (int)mx.rows, y, ldy, 0, y_dtype,
                  aligned16(y) && ldy * size % 16 == 0,
                  dtype == QMOE_BF16 ? tc::idesc_bf16_f32(128, 0) : tc::idesc_f16_f32(128, 0), dev_status};
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
                  (dtype == QMOE_BF16 ? tc::idesc_bf16_f32(128, 0) : tc::idesc_f16_f32(128, 0)) | 1u << 15, dev_status};
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
    const int64_t units = (int64_t)E * ((N + 127) / 128) * ((K + 255) / 256);
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
    if ((rc = eg::as_tma(my, at, left, st)) != QMOE_OK || (rc = eg::as_tma(mx, at, left, st)) != QMOE_OK) return rc;
    eg::Args g = {(int)P, E, (int)N, (int)K, 0, offsets, pairs, k, (int)mx.rows, dw, K, N * K, dw_dtype,
                  aligned16(dw) && K * size % 16 == 0,
                  (dtype == QMOE_BF16 ? tc::idesc_bf16_f32(128, 0) : tc::idesc_f16_f32(128, 0)) | 3u << 15, dev_status};
    CUtensorMap mp, mq;
    rc = eg::map_of(&mp, my, dtype, 64, eg::STEP, false);
    if (rc != QMOE_OK) return rc;
    rc = eg::map_of(&mq, mx, dtype, 64, pairs ? 1 : eg::STEP, false);
    if (rc != QMOE_OK) return rc;
    return pairs ? eg::launch<eg::DW, 256, true>(mp, mq, g, units, st) : eg::launch<eg::DW, 256, false>(mp, mq, g, units, st);
}
