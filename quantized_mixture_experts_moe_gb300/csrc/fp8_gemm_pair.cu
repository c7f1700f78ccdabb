// The FP8 product for many rows (see fp8_gemm.cu for the arithmetic): a pair of
// CTAs works on a 256 x 256 tile of c with two-CTA tensor-core products.
//
// Each CTA holds 128 of the tile's rows of a and loads half of its rows of b,
// so 32 KB of codes arrive for 128 x 256 x 128 products instead of the 48 KB
// that a CTA alone needs: the loads, not the tensor core, are what a lone CTA
// waits for.  Here the lanes are rows of a.  Where 128 rows of b share a scale
// (weights), a thread's 128 columns have one scale in a block, and adding a
// block is 64 paired fused multiply-adds; otherwise (two activations, as in a
// weight's gradient) each column has its own, read from shared memory, and
// those reads (one wavefront a column and warp, 1024 cycles a block against
// 512 of products) are the bound.
//
// Of the pair the first CTA issues the products; barriers that it waits on
// (loads landed, accumulator drained) are its own and count both CTAs, those
// that both wait on (stage free, accumulator full) are signalled in both.
#include "fp8_gemm.cuh"

namespace qmoe {
namespace fp8 {

constexpr int PAIR_STAGE = 2 * 128 * 128, PAIR_STAGES = 6, PAIR_BUFS = 2;
constexpr int OUT_PITCH = 80;  // bytes of a row (64 used) in a warp's output stage
template <bool UNI>
struct PairCfg {
    // UNI: the product of both scales for each lane and half of the columns; else 256 column scales and 128 lane scales
    static constexpr int SC_FLOATS = UNI ? 256 : 384;
    static constexpr int SC_OFF = PAIR_STAGES * PAIR_STAGE;
    static constexpr int OUT_OFF = SC_OFF + SC_SLOTS * SC_FLOATS * 4;
    static constexpr int BAR_OFF = OUT_OFF + EPI_WARPS * 32 * OUT_PITCH;
    static constexpr int MISC_OFF = BAR_OFF + (2 * PAIR_STAGES + 2 * PAIR_BUFS + 2 * SC_SLOTS) * 8;
    static constexpr int SMEM = MISC_OFF + 16 + 1024;
    static_assert(SMEM <= 232448, "shared memory per CTA");
};

__device__ __forceinline__ uint32_t peer_addr(const void* p, uint32_t rank) {
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(tc::smem_u32(p)), "r"(rank));
    return at;
}
// A tile into this CTA's shared memory, its bytes counted by a barrier of the pair's first CTA.
__device__ __forceinline__ void tma_load_pair(void* dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], "
        "[%2];" ::"r"(tc::smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
        : "memory");
}
__device__ __forceinline__ void mma_f8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrives on the barrier at this offset in both CTAs once the products so far are done.
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            tc::smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}
__device__ __forceinline__ void arrive_at(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// A wait on a barrier that the other CTA arrives on.
__device__ __forceinline__ bool wait_cluster(uint64_t* bar, uint32_t parity) {
    const long long t0 = clock64();
    while (true) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(tc::smem_u32(bar)), "r"(parity)
            : "memory");
        if (ok) return true;
        if (clock64() - t0 > 4000000000ll) return false;
    }
}

// A warp's 32 rows x 128 columns of c, through shared memory in pieces of 64
// bytes a row, so that a store instruction writes 8 rows of whole sectors.
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
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = i * 8 + (lane >> 2), piece = lane & 3;
            const int m = m0 + r, n = n0 + p * N + piece * PER;
            const uint4 v = *reinterpret_cast<const uint4*>(stage + r * OUT_PITCH + piece * 16);
            if (m < g.M) {
                T* const to = c + (int64_t)m * g.ldc + n;
                if (wide && n + PER <= g.N) {
                    *reinterpret_cast<uint4*>(to) = v;
                } else {
#pragma unroll
                    for (int k = 0; k < PER; ++k)
                        if (n + k < g.N) to[k] = reinterpret_cast<const T*>(&v)[k];
                }
            }
        }
        __syncwarp();
    }
}

template <bool UNI>
__global__ void __launch_bounds__(THREADS, 1) __cluster_dims__(2, 1, 1)
fp8_gemm_pair_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                     const GemmArgs g) {
    using C = PairCfg<UNI>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* sc = reinterpret_cast<float*>(smem + C::SC_OFF);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
    uint64_t* empty = full + PAIR_STAGES;
    uint64_t* acc_full = empty + PAIR_STAGES;
    uint64_t* acc_empty = acc_full + PAIR_BUFS;
    uint64_t* sc_full = acc_empty + PAIR_BUFS;
    uint64_t* sc_empty = sc_full + SC_SLOTS;
    uint32_t* tmem_at = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::MISC_OFF + 8);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_rank();
    const int blocks = (g.K + 127) / 128;
    const int q_tiles = (g.N + 255) / 256, tiles = ((g.M + 255) / 256) * q_tiles;
    const int first = blockIdx.x / 2, stride = gridDim.x / 2;

    if (threadIdx.x == 0) {
        for (int i = 0; i < PAIR_STAGES; ++i) {
            tc::mbar_init(&full[i], 1);
            tc::mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < PAIR_BUFS; ++i) {
            tc::mbar_init(&acc_full[i], 1);
            tc::mbar_init(&acc_empty[i], 2 * EPI_WARPS);
        }
        for (int i = 0; i < SC_SLOTS; ++i) {
            tc::mbar_init(&sc_full[i], 1);
            tc::mbar_init(&sc_empty[i], EPI_WARPS);
        }
        *abort_flag = 0;
        tc::fence_barrier_init();
    }
    __syncthreads();
    cluster_sync();  // both CTAs' barriers stand before either signals the other's
    if (warp == WARP_MMA) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc::smem_u32(tmem_at)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tm = *tmem_at;
    cluster_sync();  // both have their accumulators
    pdl_wait();

    if (warp >= EPI_WARPS) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(OTHER_REGS));
        if (warp == WARP_TMA) {
            if (lane == 0) {
                int slot = 0, in_flight = 0;
                uint32_t phase = 0;
                for (int u = first; u < tiles && !*abort_flag; u += stride) {
                    const int m0 = (u / q_tiles) * 256 + rank * 128, n0 = (u % q_tiles) * 256 + rank * 128;
                    for (int kb = 0; kb < blocks; ++kb) {
                        if (!wait_cluster(&empty[slot], phase ^ 1)) {
                            *abort_flag = 1;
                            atomicOr(g.status, QMOE_DEV_WAIT_TIMEOUT);
                            break;
                        }
                        uint8_t* st = smem + slot * PAIR_STAGE;
                        const uint32_t bar = peer_addr(&full[slot], 0);
                        if (rank == 0) tc::mbar_arrive_expect_tx(&full[slot], 2 * PAIR_STAGE);
                        tma_load_pair(st, &map_a, bar, kb * 128, m0);
                        tma_load_pair(st + 128 * 128, &map_b, bar, kb * 128, n0);
                        if (in_flight < PAIR_STAGES) ++in_flight;
                        if (++slot == PAIR_STAGES) { slot = 0; phase ^= 1; }
                    }
                }
                if (rank == 0 && *abort_flag)  // no load outlives the pair (which leaves together)
                    for (; in_flight > 0; --in_flight) {
                        if (slot == 0) { slot = PAIR_STAGES; phase ^= 1; }
                        --slot;
                        tc::mbar_wait(&full[slot], phase);
                    }
            }
            __syncwarp();
        } else if (warp == WARP_MMA) {
            if (rank == 0 && lane == 0) {
                constexpr uint32_t idesc = idesc_f8(256, 256);
                int slot = 0, buf = 0;
                uint32_t phase = 0, acc_phase = 0;
                bool issued = false;
                for (int u = first; u < tiles && !*abort_flag; u += stride) {
                    for (int kb = 0; kb < blocks; ++kb) {
                        if (!wait_cluster(&acc_empty[buf], acc_phase ^ 1) || !wait_cluster(&full[slot], phase)) {
                            *abort_flag = 1;
                            atomicOr(g.status, QMOE_DEV_WAIT_TIMEOUT);
                            break;
                        }
                        tc::tc_fence_after();
                        const uint32_t st = tc::smem_u32(smem + slot * PAIR_STAGE);
                        const uint64_t da = tc::sdesc_kmajor_sw128(st), db = tc::sdesc_kmajor_sw128(st + 128 * 128);
#pragma unroll
                        for (int k = 0; k < 4; ++k)  // 32 codes a step: 2 descriptor units of 16 bytes
                            mma_f8_pair(tm + buf * 256, da + 2 * k, db + 2 * k, idesc, k > 0);
                        commit_pair(&empty[slot]);
                        commit_pair(&acc_full[buf]);
                        if (++slot == PAIR_STAGES) { slot = 0; phase ^= 1; }
                        if (++buf == PAIR_BUFS) { buf = 0; acc_phase ^= 1; }
                        issued = true;
                    }
                }
                if (*abort_flag && issued) {  // no product outlives the accumulators
                    if (buf == 0) { buf = PAIR_BUFS; acc_phase ^= 1; }
                    tc::mbar_wait(&acc_full[buf - 1], acc_phase);
                }
            }
            __syncwarp();
        } else {
            // the scale warps take the blocks in turn; a block's loads go out before the slot is waited for
            int it = 0;
            for (int u = first; u < tiles && !*abort_flag; u += stride) {
                const int m0 = (u / q_tiles) * 256 + rank * 128, n0 = (u % q_tiles) * 256;
                for (int kb = 0; kb < blocks; ++kb, ++it) {
                    if (it % SCALE_WARPS != warp - WARP_SCALE) continue;
                    const int slot = it % SC_SLOTS;
                    constexpr int BN = UNI ? 2 : 8;
                    float sa[4], sb[BN];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int m = m0 + i * 32 + lane;
                        sa[i] = m < g.M ? g.a.s[(m >> g.a.shift) * g.a.s_row + kb * g.a.s_blk] : 0.f;
                    }
#pragma unroll
                    for (int i = 0; i < BN; ++i) {
                        const int n = UNI ? n0 + i * 128 : n0 + i * 32 + lane;
                        sb[i] = n < g.N ? g.b.s[(n >> g.b.shift) * g.b.s_row + kb * g.b.s_blk] : 0.f;
                    }
                    if (!warp_wait(&sc_empty[slot], (it / SC_SLOTS & 1) ^ 1, abort_flag, g.status)) break;
                    float* to = sc + slot * C::SC_FLOATS;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (UNI) {
                            to[i * 32 + lane] = sa[i] * sb[0];
                            to[128 + i * 32 + lane] = sa[i] * sb[1];
                        } else {
                            to[256 + i * 32 + lane] = sa[i];
                        }
                    }
                    if (!UNI) {
#pragma unroll
                        for (int i = 0; i < BN; ++i) to[i * 32 + lane] = sb[i];
                    }
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&sc_full[slot]);
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(EPI_REGS));
        const int quad = warp & 3, half = warp >> 2;
        const int p_lane = quad * 32 + lane;
        const uint32_t t_lane = tm + ((uint32_t)(quad * 32) << 16) + half * 128;
        uint8_t* const stage = smem + C::OUT_OFF + warp * 32 * OUT_PITCH;
        int slot = 0, buf = 0;
        uint32_t phase = 0, acc_phase = 0;
        uint64_t acc[64];
        for (int u = first; u < tiles && !*abort_flag; u += stride) {
            bool ok = true;
#pragma unroll
            for (int i = 0; i < 64; ++i) acc[i] = 0ull;
            for (int kb = 0; kb < blocks; ++kb) {
                ok = warp_wait(&sc_full[slot], phase, abort_flag, g.status) &&
                     warp_wait(&acc_full[buf], acc_phase, abort_flag, g.status);
                if (!ok) break;
                tc::tc_fence_after();
                const float* s = sc + slot * C::SC_FLOATS;
                const float own = UNI ? s[half * 128 + p_lane] : s[256 + p_lane];
                const uint64_t sp = pair_of(own, own);
                uint32_t r[2][16];
                tmem_ld<16>(t_lane + buf * 256, r[0]);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    tc::tmem_ld_wait();
                    if (i < 7) {
                        tmem_ld<16>(t_lane + buf * 256 + (i + 1) * 16, r[(i + 1) & 1]);
                    } else {
                        tc::tc_fence_before();
                        __syncwarp();
                        if (lane == 0) arrive_at(peer_addr(&acc_empty[buf], 0));
                    }
                    const uint32_t* d = r[i & 1];
#pragma unroll
                    for (int j = 0; j < 16; j += 4) {
                        uint64_t s0 = sp, s1 = sp;
                        if (!UNI) {
                            const float4 v = *reinterpret_cast<const float4*>(s + half * 128 + i * 16 + j);
                            s0 = mul_pair(pair_of(v.x, v.y), sp);
                            s1 = mul_pair(pair_of(v.z, v.w), sp);
                        }
                        uint64_t* to = &acc[(i * 16 + j) / 2];
                        to[0] = fma_pair(pair_of(d[j], d[j + 1]), s0, to[0]);
                        to[1] = fma_pair(pair_of(d[j + 2], d[j + 3]), s1, to[1]);
                    }
                }
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&sc_empty[slot]);
                if (++slot == SC_SLOTS) { slot = 0; phase ^= 1; }
                if (++buf == PAIR_BUFS) { buf = 0; acc_phase ^= 1; }
            }
            if (!ok) break;
            const int m0 = (u / q_tiles) * 256 + rank * 128 + quad * 32, n0 = (u % q_tiles) * 256 + half * 128;
            if (g.ctype == QMOE_F32) put_rows<float>(g, stage, m0, n0, lane, acc);
            else if (g.ctype == QMOE_BF16) put_rows<__nv_bfloat16>(g, stage, m0, n0, lane, acc);
            else put_rows<__half>(g, stage, m0, n0, lane, acc);
        }
    }
    __syncwarp();
    pdl_trigger();
    tc::tc_fence_before();
    __syncthreads();
    cluster_sync();  // neither leaves while the other may still signal it or read its operands
    tc::tc_fence_after();
    if (warp == WARP_MMA)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(512) : "memory");
}

template <bool UNI>
static int pair_launch(const CUtensorMap& ma, const CUtensorMap& mb, const GemmArgs& g, cudaStream_t st) {
    auto kernel = fp8_gemm_pair_kernel<UNI>;
    const int smem = PairCfg<UNI>::SMEM;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return QMOE_ERR_CUDA;
    const int64_t tiles = (int64_t)((g.M + 255) / 256) * ((g.N + 255) / 256), pairs = row::kSMs / 2;
    return launch_pdl(kernel, dim3((unsigned)(2 * (tiles < pairs ? tiles : pairs))), dim3(THREADS), (size_t)smem, st, ma,
                      mb, g);
}

int gemm_pair(const CUtensorMap& ma, const CUtensorMap& mb, const GemmArgs& g, cudaStream_t st) {
    return g.b.shift ? pair_launch<true>(ma, mb, g, st) : pair_launch<false>(ma, mb, g, st);
}

}  // namespace fp8
}  // namespace qmoe
