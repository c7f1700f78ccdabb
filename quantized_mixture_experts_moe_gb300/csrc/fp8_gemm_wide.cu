// The FP8 product for many rows of a and a b whose rows share their scales by
// 128, as a weight's do (see fp8_gemm.cu for the arithmetic): 128 x 256 tiles of
// c, rows of a on the lanes.
//
// A thread's 128 columns then have one scale in a block, and adding a block is
// 64 paired fused multiply-adds a thread, with no scale read for each column
// (those reads are one wavefront a column and warp: 1024 cycles a block).  The
// two accumulators take the blocks in turn, and their halves are handed over
// separately: a block's products are 512 cycles, but issuing four of them and
// the way to the epilogue and back cost as much again, which the halves hide
// in part.  8192 x 2816 x 4096: 93 us, 2.02 PFLOP/s, with the tensor pipe 43% and
// the issue slots 42% busy: neither is the bound, the handing over is.
//
// Two-CTA products (256 x 256 a pair, half the rows of b loaded by each) were
// slower, 189 us at that size against 135 of the narrow kernel: loads that
// report to the other CTA's barrier took 0.8 us a block, and handing
// accumulators between the CTAs another 0.35 us.  So were 128 x 192 tiles with
// 12 epilogue warps (125 us) and 16 epilogue warps (120 us).
#include "fp8_gemm.cuh"

namespace qmoe {
namespace fp8 {

// Warps: 8 scale and sum, then one that loads, two that issue products (one for
// each accumulator) and one that brings scales.  Registers: launched with 168 a
// thread (64,512 in all); the epilogue's warpgroups take 232, the third keeps 40
// (64,512 in all).
constexpr int WIDE_TMA = 8, WIDE_MMA = 9, WIDE_SCALE = 11, WIDE_THREADS = 12 * 32;
constexpr int WIDE_EPI_REGS = 232, WIDE_OTHER_REGS = 40;
constexpr int WIDE_STAGE = (128 + 256) * 128, WIDE_STAGES = 4;
constexpr int OUT_PITCH = 80;  // bytes of a row (64 used) in a warp's output stage
struct WideCfg {
    static constexpr int SC_FLOATS = 128 + 4;  // 128 lane scales, then one for each half of the columns
    static constexpr int SC_OFF = WIDE_STAGES * WIDE_STAGE;
    static constexpr int OUT_OFF = SC_OFF + SC_SLOTS * SC_FLOATS * 4;
    static constexpr int BAR_OFF = OUT_OFF + EPI_WARPS * 32 * OUT_PITCH;
    static constexpr int MISC_OFF = BAR_OFF + (2 * WIDE_STAGES + 8 + 2 * SC_SLOTS) * 8;
    static constexpr int SMEM = MISC_OFF + 16 + 1024;
    static_assert(SMEM <= 232448, "shared memory per CTA");
};

// 4 bytes, or zero where there is nothing to copy.
__device__ __forceinline__ void cp_async_4_or_zero(void* dst, const void* src, bool real) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(tc::smem_u32(dst)), "l"(src), "r"(real ? 4 : 0)
                 : "memory");
}

__device__ __forceinline__ void tmem_load(uint32_t taddr, uint32_t (&r)[64]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,"
        "%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]),
          "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]),
          "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]),
          "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]),
          "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(taddr));
}

// A warp's 32 rows x 128 columns of c, through shared memory in pieces of 64
// bytes a row, so that a store instruction writes 8 rows of whole sectors.  Rows
// off the 16-byte boundaries go value by value, neighbouring lanes to
// neighbouring columns (8192 x 2815 x 4096: 107 us; a lane's 8 columns one by one
// took 180).
template <typename T>
__device__ __forceinline__ void put_rows(const GemmArgs& g, uint8_t* stage, int m0, int n0, int lane,
                                         const uint64_t (&acc)[64]) {
    constexpr int N = 64 / sizeof(T), PER = 16 / sizeof(T);  // columns of a piece, of 16 bytes
    T* const c = static_cast<T*>(g.c);
    const bool wide = (reinterpret_cast<uintptr_t>(c) & 15) == 0 && (g.ldc * sizeof(T)) % 16 == 0;
#pragma unroll
    for (int p = 0; p < 128 / N; ++p) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint4 v;
            uint32_t* w = &v.x;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (sizeof(T) == 2) {
                    const float2 f = halves_of(acc[p * 16 + j * 4 + i]);
                    w[i] = row::pack2(f.x, f.y, T{});
                } else {
                    const float2 f = halves_of(acc[p * 8 + j * 2 + i / 2]);
                    w[i] = __float_as_uint(i & 1 ? f.y : f.x);
                }
            }
            *reinterpret_cast<uint4*>(stage + lane * OUT_PITCH + j * 16) = v;
        }
        __syncwarp();
        if (wide) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = i * 8 + (lane >> 2), piece = lane & 3;
                const int m = m0 + r, n = n0 + p * N + piece * PER;
                const uint4 v = *reinterpret_cast<const uint4*>(stage + r * OUT_PITCH + piece * 16);
                if (m < g.M) {
                    T* const to = c + (int64_t)m * g.ldc + n;
                    if (n + PER <= g.N) {
                        *reinterpret_cast<uint4*>(to) = v;
                    } else {
#pragma unroll
                        for (int k = 0; k < PER; ++k)
                            if (n + k < g.N) to[k] = reinterpret_cast<const T*>(&v)[k];
                    }
                }
            }
        } else {
            const int col = lane % N, n = n0 + p * N + col;
#pragma unroll 8
            for (int r = lane / N; r < 32; r += 32 / N)
                if (m0 + r < g.M && n < g.N)
                    c[(int64_t)(m0 + r) * g.ldc + n] = reinterpret_cast<const T*>(stage + r * OUT_PITCH)[col];
        }
        __syncwarp();
    }
}

__global__ void __launch_bounds__(WIDE_THREADS, 1)
fp8_gemm_wide_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                     const GemmArgs g) {
    using C = WideCfg;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* sc = reinterpret_cast<float*>(smem + C::SC_OFF);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
    uint64_t* empty = full + WIDE_STAGES;
    uint64_t* acc_full = empty + WIDE_STAGES;
    uint64_t* acc_empty = acc_full + 4;  // [accumulator][half of the columns]
    uint64_t* sc_full = acc_empty + 4;
    uint64_t* sc_empty = sc_full + SC_SLOTS;
    uint32_t* tmem_at = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::MISC_OFF + 8);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int blocks = (g.K + 127) / 128;
    const int q_tiles = (g.N + 255) / 256, tiles = ((g.M + 127) / 128) * q_tiles;

    if (threadIdx.x == 0) {
        for (int i = 0; i < WIDE_STAGES; ++i) {
            tc::mbar_init(&full[i], 1);
            tc::mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 4; ++i) {
            tc::mbar_init(&acc_full[i], 1);
            tc::mbar_init(&acc_empty[i], EPI_WARPS / 2);
        }
        for (int i = 0; i < SC_SLOTS; ++i) {
            tc::mbar_init(&sc_full[i], 32);
            tc::mbar_init(&sc_empty[i], EPI_WARPS);
        }
        *abort_flag = 0;
        tc::fence_barrier_init();
    }
    if (warp == WIDE_MMA) {
        tc::tmem_alloc(tmem_at, 512);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tm = *tmem_at;
    pdl_wait();

    if (warp >= EPI_WARPS) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(WIDE_OTHER_REGS));
        if (warp == WIDE_TMA) {
            if (lane == 0) {
                int slot = 0, in_flight = 0;
                uint32_t phase = 0;
                for (int u = blockIdx.x; u < tiles && !*abort_flag; u += gridDim.x) {
                    const int m0 = (u / q_tiles) * 128, n0 = (u % q_tiles) * 256;
                    for (int kb = 0; kb < blocks; ++kb) {
                        if (!tc::mbar_wait(&empty[slot], phase ^ 1)) {
                            *abort_flag = 1;
                            atomicOr(g.status, QMOE_DEV_WAIT_TIMEOUT);
                            break;
                        }
                        uint8_t* st = smem + slot * WIDE_STAGE;
                        tc::mbar_arrive_expect_tx(&full[slot], WIDE_STAGE);
                        tc::tma_load_2d(st, &map_a, &full[slot], kb * 128, m0);
                        tc::tma_load_2d(st + 128 * 128, &map_b, &full[slot], kb * 128, n0);
                        if (in_flight < WIDE_STAGES) ++in_flight;
                        if (++slot == WIDE_STAGES) { slot = 0; phase ^= 1; }
                    }
                }
                if (*abort_flag)  // nobody may have waited for these: no load outlives the CTA
                    for (; in_flight > 0; --in_flight) {
                        if (slot == 0) { slot = WIDE_STAGES; phase ^= 1; }
                        --slot;
                        tc::mbar_wait(&full[slot], phase);
                    }
            }
            __syncwarp();
        } else if (warp < WIDE_SCALE) {
            if (lane == 0) {
                constexpr uint32_t idesc = idesc_f8(128, 128);
                const int turn = warp - WIDE_MMA;  // this warp's accumulator
                int it = 0, sent = 0;
                for (int u = blockIdx.x; u < tiles && !*abort_flag; u += gridDim.x) {
                    for (int kb = 0; kb < blocks; ++kb, ++it) {
                        if ((it & 1) != turn) continue;
                        const int slot = it % WIDE_STAGES;
                        bool ok = tc::mbar_wait(&full[slot], it / WIDE_STAGES & 1);
                        const uint32_t st = tc::smem_u32(smem + slot * WIDE_STAGE);
                        const uint64_t da = tc::sdesc_kmajor_sw128(st);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            ok = ok && tc::mbar_wait(&acc_empty[2 * turn + h], (it >> 1 & 1) ^ 1);
                            if (!ok) break;
                            tc::tc_fence_after();
                            const uint64_t db = tc::sdesc_kmajor_sw128(st + (1 + h) * 128 * 128);
#pragma unroll
                            for (int k = 0; k < 4; ++k)  // 32 codes a step: 2 descriptor units of 16 bytes
                                mma_f8(tm + turn * 256 + h * 128, da + 2 * k, db + 2 * k, idesc, k > 0);
                            tc::mma_commit(&acc_full[2 * turn + h]);
                        }
                        tc::mma_commit(&empty[slot]);
                        sent = it + 1;
                        if (!ok) {
                            *abort_flag = 1;
                            atomicOr(g.status, QMOE_DEV_WAIT_TIMEOUT);
                            break;
                        }
                    }
                }
                if (*abort_flag && sent)  // no product outlives the accumulators
                    tc::mbar_wait(&empty[(sent - 1) % WIDE_STAGES], (sent - 1) / WIDE_STAGES & 1);
            }
            __syncwarp();
        } else {
            int slot = 0;
            uint32_t phase = 0;
            for (int u = blockIdx.x; u < tiles && !*abort_flag; u += gridDim.x) {
                const int m0 = (u / q_tiles) * 128, n0 = (u % q_tiles) * 256;
                // this lane's rows of a (and lanes 0 and 1: a half's rows of b): where their scales in the block to
                // come lie, and whether there are such rows
                const float* at[5];
                uint32_t real = 0;
#pragma unroll
                for (int i = 0; i < 5; ++i) {
                    const Side& s = i < 4 ? g.a : g.b;
                    const int r = i < 4 ? m0 + i * 32 + lane : n0 + (lane & 1) * 128;
                    const bool there = r < (i < 4 ? g.M : g.N);
                    at[i] = s.s + (there ? (int64_t)(r >> s.shift) * s.s_row : 0);
                    real |= (uint32_t)there << i;
                }
                for (int kb = 0; kb < blocks; ++kb) {
                    if (!warp_wait(&sc_empty[slot], phase ^ 1, abort_flag, g.status)) break;
                    float* const to = sc + slot * C::SC_FLOATS + lane;
#pragma unroll
                    for (int i = 0; i < 5; ++i) {
                        if (i < 4 || lane < 2) cp_async_4_or_zero(to + i * 32, at[i], real >> i & 1);
                        at[i] += i < 4 ? g.a.s_blk : g.b.s_blk;
                    }
                    tc::cp_async_mbar_arrive_noinc(&sc_full[slot]);
                    if (++slot == SC_SLOTS) { slot = 0; phase ^= 1; }
                }
            }
            tc::cp_async_wait<0>();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(WIDE_EPI_REGS));
        const int quad = warp & 3, half = warp >> 2;
        const int p_lane = quad * 32 + lane;
        const uint32_t t_lane = tm + ((uint32_t)(quad * 32) << 16) + half * 128;
        uint8_t* const stage = smem + C::OUT_OFF + warp * 32 * OUT_PITCH;
        int slot = 0, buf = 0;
        uint32_t phase = 0, acc_phase = 0;
        uint64_t acc[64];
        for (int u = blockIdx.x; u < tiles && !*abort_flag; u += gridDim.x) {
            bool ok = true;
#pragma unroll
            for (int i = 0; i < 64; ++i) acc[i] = 0ull;
            for (int kb = 0; kb < blocks; ++kb) {
                ok = warp_wait(&sc_full[slot], phase, &acc_full[2 * buf + half], acc_phase, abort_flag, g.status);
                if (!ok) break;
                tc::tc_fence_after();
                const float* s = sc + slot * C::SC_FLOATS;
                const float own = s[p_lane] * s[128 + half];
                const uint64_t sp = pair_of(own, own);
#pragma unroll
                for (int i = 0; i < 128; i += 64) {
                    uint32_t d[64];
                    tmem_load(t_lane + buf * 256 + i, d);
                    tc::tmem_ld_wait();
                    if (i > 0) {
                        tc::tc_fence_before();
                        __syncwarp();
                        if (lane == 0) tc::mbar_arrive(&acc_empty[2 * buf + half]);
                    }
#pragma unroll
                    for (int j = 0; j < 64; j += 2)
                        acc[(i + j) / 2] = fma_pair(pair_of(d[j], d[j + 1]), sp, acc[(i + j) / 2]);
                }
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&sc_empty[slot]);
                if (++slot == SC_SLOTS) { slot = 0; phase ^= 1; }
                if (++buf == 2) { buf = 0; acc_phase ^= 1; }
            }
            if (!ok) break;
            const int m0 = (u / q_tiles) * 128 + quad * 32, n0 = (u % q_tiles) * 256 + half * 128;
            if (g.ctype == QMOE_F32) put_rows<float>(g, stage, m0, n0, lane, acc);
            else if (g.ctype == QMOE_BF16) put_rows<__nv_bfloat16>(g, stage, m0, n0, lane, acc);
            else put_rows<__half>(g, stage, m0, n0, lane, acc);
        }
    }
    __syncwarp();
    pdl_trigger();
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (warp == WIDE_MMA) tc::tmem_dealloc(tm, 512);
}

int gemm_wide(const CUtensorMap& ma, const CUtensorMap& mb, const GemmArgs& g, cudaStream_t st) {
    const int rc = row::allow_smem<fp8_gemm_wide_kernel>(WideCfg::SMEM);
    if (rc != QMOE_OK) return rc;
    const int64_t tiles = (int64_t)((g.M + 127) / 128) * ((g.N + WIDE_N - 1) / WIDE_N);
    return launch_pdl(fp8_gemm_wide_kernel, dim3((unsigned)(tiles < row::kSMs ? tiles : row::kSMs)), dim3(WIDE_THREADS),
                      (size_t)WideCfg::SMEM, st, ma, mb, g);
}

}  // namespace fp8
}  // namespace qmoe
