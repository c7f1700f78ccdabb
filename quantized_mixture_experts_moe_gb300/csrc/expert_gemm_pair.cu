// The experts' products in 256 x 256 tiles of two CTAs (see expert_gemm.cu for the
// three forms): each CTA has 128 of the lanes and loads its own part of them and
// half of the columns, so that a value of the column side comes to shared memory
// once for 256 lanes; one of the two issues the products of both.
//
// Both CTAs' loads report to the first one's barrier.  Where a thread has to touch
// a stage before its products (zeros in place of another expert's rows in the last
// step of dw), the second CTA's loads report to its own barrier, its product warp,
// which has no products to issue, waits for them, and arrives at a barrier of the
// first.  That arrival is of the CTA's scope, as the
// tile was written by the async proxy or is ordered by its fence: one that
// releases at the cluster's scope took 1100 cycles, twice what a step's products
// take.
//
// What bounds it: the tensor core under the power limit (64 x 1024 rows 4096 -> 2816:
// y 840 to 890 us by the card's clock, 1.7 to 1.8 PFLOP/s, dx 825 to 865, against 1.97 of
// a library's product of one matrix); for dw's 32-bit sums the stores too (64 x 512 rows,
// 2816 x 2048: 339 to 366 us, 1.1 PFLOP/s and 5.2 TB/s).  A lone CTA with 128 x 256 tiles
// reached 1.36 PFLOP/s: its loads, half as much again.
#include "expert_gemm.cuh"

namespace qmoe {
namespace eg {

// Warps: the epilogue's, two that load tiles, step by step in turn (a load takes a
// thread some 100 cycles to issue), one that issues products.
constexpr int PAIR_TMA = 8, TURNS = 2, PAIR_MMA = PAIR_TMA + TURNS;
constexpr int PAIR_THREADS = (PAIR_MMA + 1) * 32;

// Pieces of a sum: of steps / pieces_of(steps) steps each, rounded up.
__device__ __forceinline__ int pieces_of(int steps) { return (steps + LONG - 1) / LONG; }

template <int MODE>
struct PairCfg {
    static constexpr int P_BYTES = 128 * STEP * 2, STAGE = 2 * P_BYTES;
    static constexpr int LIST = MODE == DW ? 0 : 2 * (MAX_E + 2) * 4;
    static constexpr int OUT = MODE == DW ? STAGE_DW : STAGE_OUT;
    static constexpr int STAGES = 6;
    static constexpr int OUT_OFF = STAGES * STAGE;
    static constexpr int LIST_OFF = OUT_OFF + EPI_WARPS * OUT;
    static constexpr int BAR_OFF = LIST_OFF + (LIST + 15) / 16 * 16;
    static constexpr int MISC_OFF = BAR_OFF + (3 * STAGES + 4) * 8;
    static constexpr int SMEM = MISC_OFF + 64 + 1024;
    static_assert(SMEM <= 232448, "shared memory per CTA");
};

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// The address of this barrier in a CTA of the pair.
__device__ __forceinline__ uint32_t bar_in(uint64_t* bar, uint32_t rank) {
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(tc::smem_u32(bar)), "r"(rank));
    return at;
}
__device__ __forceinline__ void arrive_first(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar_in(bar, 0)) : "memory");
}
// Tiles into this CTA's shared memory that report to a barrier of either.
__device__ __forceinline__ void pair_load_2d(void* dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], "
        "[%2];" ::"r"(tc::smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
        : "memory");
}
__device__ __forceinline__ void pair_load_3d(void* dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, "
        "%5}], [%2];" ::"r"(tc::smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}
// All lanes of the warp call these with the same operands (which then stay in
// uniform registers) and one issues.
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrives at this barrier of both CTAs once the products issued so far are done.
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(
            tc::smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}
// The products of K16 times 16 values of a stage.
template <int MODE>
__device__ __forceinline__ void mma_stage(uint32_t d, uint32_t stage, uint32_t idesc, bool first, int k16 = STEP / 16) {
    const uint32_t sb = stage + 128 * STEP * 2;
    const uint64_t da = MODE == FWD ? tc::sdesc_kmajor_sw128(stage) : sdesc_across(stage);
    const uint64_t db = MODE == DW ? sdesc_across(sb) : tc::sdesc_kmajor_sw128(sb);
    constexpr int SA = MODE == FWD ? 2 : 128, SB = MODE == DW ? 128 : 2;  // of 16 values, in 16 bytes
#pragma unroll
    for (int k = 0; k < STEP / 16; ++k)
        if (k < k16) mma_pair(d, da + SA * k, db + SB * k, idesc, !first || k > 0);
}

template <int MODE, bool BULK, bool BY>
__global__ void __launch_bounds__(PAIR_THREADS, 1)
expert_pair_kernel(const __grid_constant__ CUtensorMap map_p, const __grid_constant__ CUtensorMap map_q,
                   const __grid_constant__ CUtensorMap map_o, const Args g) {
    using C = PairCfg<MODE>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    int* off = reinterpret_cast<int*>(smem + C::LIST_OFF);
    int* base = off + MAX_E + 1;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
    uint64_t* empty = full + C::STAGES;
    uint64_t* other = empty + C::STAGES;  // of the first CTA: the second one's stage is full
    uint64_t* acc_full = other + C::STAGES;
    uint64_t* acc_empty = acc_full + 2;  // of the first CTA: both have read the sums
    uint32_t* tmem_at = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::MISC_OFF + 8);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_rank();
    if (threadIdx.x == 32) {
        tc::prefetch_tensormap(&map_p);
        tc::prefetch_tensormap(&map_q);
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::STAGES; ++i) {
            tc::mbar_init(&full[i], 1);
            tc::mbar_init(&empty[i], 1);
            tc::mbar_init(&other[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&acc_full[i], 1);
            tc::mbar_init(&acc_empty[i], 2 * EPI_WARPS);
        }
        *abort_flag = 0;
        tc::fence_barrier_init();
    }
    if (warp == PAIR_MMA) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc::smem_u32(tmem_at)), "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    pdl_wait();
    int cap = 256;
    if constexpr (MODE == DW) {
        if (blockIdx.x == 0) check_offsets(g);
    } else {
        cap = read_offsets<256, 256, true>(g, off, base, gridDim.x >> 1);
    }
    tc::tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc::tc_fence_after();
    const uint32_t tm = *tmem_at;
    const int first = blockIdx.x >> 1, stride = gridDim.x >> 1;
    auto walk = [&] {
        if constexpr (MODE == DW) return WalkDw<256, 256>(g, first, stride);
        else return Walk<256, 32>(g, off, base, cap);
    }();
    const int total = walk.total();

    if (warp >= PAIR_TMA && warp < PAIR_MMA) {
        if (lane == 0) {
            const int turn = warp - PAIR_TMA;
            int it = 0;
            for (int u = first; u < total && !*abort_flag; u += stride) {
                const Unit t = walk.at(u);
                const int half = ((t.n + 31) & ~31) / 2, l0 = t.l0 + rank * 128, q0 = t.q0 + rank * half;
                const int boxes = MODE == DW ? (half + 63) / 64 : 1;
                const uint32_t bytes = C::P_BYTES + boxes * (MODE == DW ? 8192 : 128 * 128);
                for (int s = 0; s < t.steps; ++s, ++it) {
                    if (it % TURNS != turn) continue;
                    const int slot = it % C::STAGES;
                    if (!lane_wait(&empty[slot], (it / C::STAGES & 1) ^ 1, abort_flag, g.status)) break;
                    uint8_t* st = smem + slot * C::STAGE;
                    uint8_t* sq = st + C::P_BYTES;
                    const int second = MODE != DW && s >= g.per, k0 = (s - (second ? g.per : 0)) * STEP, z = t.e + second, row = t.row0 + k0;
                    const bool relay = MODE == DW && t.end - row < STEP;
                    const uint32_t bar = bar_in(&full[slot], relay ? rank : 0);
                    if (relay) tc::mbar_arrive_expect_tx(&full[slot], bytes);
                    else if (rank == 0) tc::mbar_arrive_expect_tx(&full[slot], 2 * bytes);
                    if constexpr (MODE == FWD) {
                        pair_load_3d(st, &map_p, bar, k0, l0, z);
                    } else if constexpr (MODE == DX) {
                        pair_load_3d(st, &map_p, bar, l0, k0, z);
                        pair_load_3d(st + 8192, &map_p, bar, l0 + 64, k0, z);
                    } else {
                        pair_load_2d(st, &map_p, bar, l0, row);
                        pair_load_2d(st + 8192, &map_p, bar, l0 + 64, row);
                    }
                    for (int b = 0; b < boxes; ++b) {
                        if constexpr (MODE == DW) pair_load_2d(sq + b * 8192, &map_q, bar, q0 + b * 64, row);
                        else pair_load_2d(sq, &map_q, bar, k0, q0);
                    }
                }
            }
        }
        __syncwarp();
    } else if (warp == PAIR_MMA) {
        int slot = 0, buf = 0;
        uint32_t phase = 0, acc_phase = 0, relayed = 0, here = 0;  // of each stage: the phases of other, and of full in the second CTA
        bool ok = true;  // after a wait that ran out no more products are issued and no more stages let go
        for (int u = first; u < total && ok; u += stride) {
            const Unit t = walk.at(u);
            if (t.steps == 0) continue;  // zeros: no sums to wait for
            const uint32_t n32 = (uint32_t)(t.n + 31) & ~31u;
            const uint32_t idesc = g.idesc | (n32 >> 3) << 17 | (256u >> 4) << 24;
            const int left = MODE == DW ? (t.end - t.row0) % STEP : 0, whole = t.steps - (left > 0);
            const int pieces = pieces_of(t.steps), per = pieces > 1 ? (t.steps + pieces - 1) / pieces : t.steps;
            for (int from = 0; from < t.steps; from += per) {  // the sum's pieces, each in an accumulator of its own
                if (rank == 0 && !(ok = issue_wait(&acc_empty[buf], acc_phase ^ 1, abort_flag, g.status))) break;
                const uint32_t d = tm + buf * 256;
                const int to = min(from + per, whole);
                if (rank == 0) {
#pragma unroll 1
                    for (int s = from; s < to; ++s) {
                        if (!(ok = issue_wait(&full[slot], phase, abort_flag, g.status))) break;
                        tc::tc_fence_after();
                        mma_stage<MODE>(d, tc::smem_u32(smem) + slot * C::STAGE, idesc, s == from);
                        commit_pair(&empty[slot]);
                        if (++slot == C::STAGES) { slot = 0; phase ^= 1; }
                    }
                } else {
                    slot += to - from;  // the first CTA's affair
                    phase ^= slot / C::STAGES & 1;
                    slot %= C::STAGES;
                }
                if (!ok) break;
                if (MODE == DW && left > 0 && from + per >= t.steps) {
                    const int k16 = (left + 15) / 16;
                    uint8_t* st = smem + slot * C::STAGE;
                    if (!(ok = issue_wait(&full[slot], rank == 0 ? phase : here >> slot & 1, abort_flag, g.status))) break;
                    here ^= 1u << slot;
                    // rows behind the expert's last, up to the 16 of a product, are another's: zeros in their place
                    const int zero = k16 * 16 - left;
                    for (int i = lane; i < 4 * zero * 8; i += 32) {
                        const int b = i / (zero * 8), c = i - b * zero * 8;
                        *reinterpret_cast<uint4*>(st + b * 8192 + left * 128 + c * 16) = make_uint4(0, 0, 0, 0);
                    }
                    tc::fence_proxy_async_smem();
                    __syncwarp();
                    if (rank == 0) {
                        if (!(ok = issue_wait(&other[slot], relayed >> slot & 1, abort_flag, g.status))) break;
                        relayed ^= 1u << slot;
                        tc::tc_fence_after();
                        mma_stage<MODE>(d, tc::smem_u32(st), idesc, whole == from, k16);
                        commit_pair(&empty[slot]);
                    } else if (lane == 0) {
                        arrive_first(&other[slot]);
                    }
                    __syncwarp();
                    if (++slot == C::STAGES) { slot = 0; phase ^= 1; }
                }
                if (rank == 0) commit_pair(&acc_full[buf]);
                if (++buf == 2) { buf = 0; acc_phase ^= 1; }
            }
        }
        __syncwarp();
    } else {
        const int quad = warp & 3, half = warp >> 2;
        uint8_t* const stage = smem + C::OUT_OFF + warp * C::OUT;
        const bool matrices = by_matrices<MODE>(g);
        int buf = 0;
        uint32_t acc_phase = 0;
        for (int u = first; u < total && !*abort_flag; u += stride) {
            const Unit t = walk.at(u);
            const int l0 = t.l0 + rank * 128 + quad * 32;
            uint32_t r[2][32];
            if (t.steps == 0) {
#pragma unroll
                for (int j = 0; j < 32; ++j) r[0][j] = 0;
                for (int c = half * 32; c < t.n; c += 64) put<MODE, BULK, BY>(g, &map_o, matrices, stage, t.e, l0, t.q0 + c, t.n - c, lane, r[0]);
                continue;
            }
            const uint32_t all = tm + ((uint32_t)(quad * 32) << 16);
            auto let_go = [&](int which) {
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_first(&acc_empty[which]);
            };
            if (!warp_wait(&acc_full[buf], acc_phase, abort_flag, g.status)) break;
            tc::tc_fence_after();
            bool ok = true;
#pragma unroll 1
            for (int p = pieces_of(t.steps); p > 1; --p) {
                // The sum so far is added to the next piece's, in TMEM, and its accumulator let go: products wait some 0.6 us
                // for it, as the other accumulator holds the sum (8192 rows 4096 -> 4096: 154 us, 152 in one piece).  128 sums a
                // thread in registers would leave both accumulators free, but spilled (155 there, but dw of 64 x 512 rows 2816 x
                // 2048 400 to 600 us for 360).
                const int before = buf;
                if (++buf == 2) { buf = 0; acc_phase ^= 1; }
                ok = warp_wait(&acc_full[buf], acc_phase, abort_flag, g.status);
                if (!ok) break;
                tc::tc_fence_after();
                for (int c = half * 32; c < t.n; c += 64) {
                    tmem_ld32(all + before * 256 + c, r[0]);
                    tmem_ld32(all + buf * 256 + c, r[1]);
                    tc::tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 32; ++j) r[0][j] = __float_as_uint(__uint_as_float(r[0][j]) + __uint_as_float(r[1][j]));
                    tmem_st32(all + buf * 256 + c, r[0]);
                }
                tc::tmem_st_wait();
                let_go(before);
            }
            if (!ok) break;
            // the next 32 columns are on their way while these are stored; the sums are let go when the last have come
            const uint32_t from = all + buf * 256;
            int at = half * 32;
            if (at < t.n) take<MODE>(matrices, from + at, r[0]);
            auto turn = [&](uint32_t (&now)[32], uint32_t (&next)[32]) {
                tc::tmem_ld_wait();
                if (at + 64 < t.n) take<MODE>(matrices, from + at + 64, next);
                else let_go(buf);
                put<MODE, BULK, BY>(g, &map_o, matrices, stage, t.e, l0, t.q0 + at, t.n - at, lane, now);
                at += 64;
            };
            if (at >= t.n) let_go(buf);  // no columns for this warp
            while (at < t.n) {
                turn(r[0], r[1]);
                if (at < t.n) turn(r[1], r[0]);
            }
            if (++buf == 2) { buf = 0; acc_phase ^= 1; }
        }
    }
    if (BULK && warp < EPI_WARPS && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
    pdl_trigger();
    tc::tc_fence_before();
    __syncthreads();
    wind_down(abort_flag);
    cluster_sync();  // neither CTA leaves while the other's products read its tiles or arrive at its barriers
    tc::tc_fence_after();
    if (warp == PAIR_MMA)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(512) : "memory");
}

template <int MODE, bool BULK, bool BY>
int launch_pair(const CUtensorMap& mp, const CUtensorMap& mq, const CUtensorMap& mo, const Args& g, int64_t most, cudaStream_t st) {
    using C = PairCfg<MODE>;
    const int rc = row::allow_smem<expert_pair_kernel<MODE, BULK, BY>>(C::SMEM);
    if (rc != QMOE_OK) return rc;
    const int64_t pairs = most < row::kSMs / 2 ? most : row::kSMs / 2;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * pairs));
    cfg.blockDim = dim3(PAIR_THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, expert_pair_kernel<MODE, BULK, BY>, mp, mq, mo, g) == cudaSuccess ? QMOE_OK : QMOE_ERR_LAUNCH;
}

template int launch_pair<FWD, false, false>(const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, const Args&, int64_t, cudaStream_t);
template int launch_pair<FWD, false, true>(const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, const Args&, int64_t, cudaStream_t);
template int launch_pair<DX, false, false>(const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, const Args&, int64_t, cudaStream_t);
template int launch_pair<DX, false, true>(const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, const Args&, int64_t, cudaStream_t);
template int launch_pair<DW, true, false>(const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, const Args&, int64_t, cudaStream_t);
template int launch_pair<DW, false, false>(const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, const Args&, int64_t, cudaStream_t);

}  // namespace eg
}  // namespace qmoe
