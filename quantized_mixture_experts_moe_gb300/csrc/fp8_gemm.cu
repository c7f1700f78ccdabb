// FP8 (E4M3) matrix product with one scale for each 128 values of the
// reduction axis (qmoe_fp8_matmul, qmoe_fp8_linear):
//
//   C[m][n] = sum_kb sa(m, kb) sb(n, kb) sum_{k in block kb} a[m][k] b[n][k]
//
// The scales are fp32, not powers of two, so they cannot ride in the tensor
// core's scale inputs; each block of 128 is its own tensor-core product from
// zero, and the epilogue warps carry the scaled sum on in fp32 registers while
// the tensor core works on the next block in another accumulator.
//
// The 128 lanes of a tile are rows n of b (a weight's output rows), its NT
// columns rows m of a (tokens): few tokens then make narrow tiles, whose loads
// are almost all weight; and a store of one token's 128 outputs is contiguous
// across lanes.  Warps: 8 scale and sum (two for each quadrant of lanes, half
// the columns each); two load tiles by TMA, two issue the products and two
// bring the scales by plain loads, each pair taking the blocks in turn.
//
// Where the tiles are fewer than the SMs, the reduction axis is cut in S parts
// for a cluster of S CTAs, which add their parts through distributed shared
// memory in rank order: the same bits every time, one launch, no workspace.
//
// What bounds it: few tokens, the weight's bytes behind the start of the pipeline
// (1 x 2048 x 4096 5.6 us, 256 x 2816 x 4096 10.8 us); many, the sum in fp32
// registers, 64 paired fused multiply-adds a thread and block beside the reads
// of TMEM.  Operands that both have a scale for each row (a weight's gradient,
// 2048 x 4096 x 4096) run here at any size: 68 us, 1.0 PFLOP/s; every pair that
// is added needs its columns' scales read from shared memory and multiplied
// first.  A tile of two rows a thread, which read them half as often, was no
// faster (70 us): it issued 202 instructions a warp and block for the 128
// needed, with the FMA pipe 35% busy, so latency has a part in it that is not
// traced further.  Many rows of a and a b scaled by 128 rows go to the wide
// kernel.
#include "fp8_gemm.cuh"

namespace qmoe {
namespace fp8 {

int quant_rows_launch(int64_t rows, int64_t cols, int dtype, const void* x, int64_t ldx, uint8_t* q, int64_t ldq,
                      float* s, cudaStream_t st);

// UNI: the 128 rows of a tile's lane side share their scale, and the scale
// warps multiply it into the column scales; else each lane has its own.
template <int NT, bool UNI>
struct GemmCfg {
    static constexpr int BUFS = 4;  // accumulators in TMEM
    static constexpr int TMEM_COLS = BUFS * NT < 32 ? 32 : BUFS * NT;
    static constexpr int P_BYTES = 128 * 128, Q_BYTES = NT * 128, STAGE = P_BYTES + Q_BYTES;
    static constexpr int SC_FLOATS = NT + (UNI ? 0 : 128);
    static constexpr int FIXED = SC_SLOTS * SC_FLOATS * 4 + 1024 + 512;
    static constexpr int FIT = (232448 - FIXED) / STAGE;
    static constexpr int STAGES = FIT > 10 ? 10 : FIT;
    static constexpr int SC_OFF = STAGES * STAGE;
    static constexpr int BAR_OFF = SC_OFF + SC_SLOTS * SC_FLOATS * 4;
    static constexpr int BARS = 2 * STAGES + 2 * BUFS + 2 * SC_SLOTS;
    static constexpr int MISC_OFF = BAR_OFF + BARS * 8;
    static constexpr int SMEM = MISC_OFF + 16 + 1024;
    static constexpr int COLS = NT / 2;  // columns of an epilogue warp
    static_assert(SMEM <= 232448 && STAGES >= 4, "shared memory per CTA");
    static_assert(STAGES * STAGE >= 128 * NT * 4, "the ring holds a tile of sums");
};

__device__ __forceinline__ void put(void* c, int ctype, int64_t at, float v) {
    if (ctype == QMOE_F32) static_cast<float*>(c)[at] = v;
    else if (ctype == QMOE_BF16) static_cast<__nv_bfloat16*>(c)[at] = __float2bfloat16_rn(v);
    else static_cast<__half*>(c)[at] = __float2half_rn(v);
}

// One lane's outputs of a tile: COLS rows of c, as far as there are any.
template <int COLS, typename T>
__device__ __forceinline__ void put_cols(T* c, int64_t ldc, int rows, const uint64_t (&acc)[COLS / 2]) {
#pragma unroll
    for (int i = 0; i < COLS / 2; ++i) {
        const float2 v = halves_of(acc[i]);
        if (2 * i < rows) *c = row::from_f32<T>(v.x);
        c += ldc;
        if (2 * i + 1 < rows) *c = row::from_f32<T>(v.y);
        c += ldc;
    }
}

template <int NT, bool UNI>
__global__ void __launch_bounds__(THREADS, 1)
fp8_gemm_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                const GemmArgs g) {
    using C = GemmCfg<NT, UNI>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* sc = reinterpret_cast<float*>(smem + C::SC_OFF);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
    uint64_t* empty = full + C::STAGES;
    uint64_t* acc_full = empty + C::STAGES;
    uint64_t* acc_empty = acc_full + C::BUFS;
    uint64_t* sc_full = acc_empty + C::BUFS;
    uint64_t* sc_empty = sc_full + SC_SLOTS;
    uint32_t* tmem_at = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::MISC_OFF + 8);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int parts = (int)cluster_size(), part = (int)cluster_rank();
    const int blocks = (g.K + 127) / 128;
    const int kb0 = (int)((int64_t)blocks * part / parts), kb1 = (int)((int64_t)blocks * (part + 1) / parts);
    const int p_tiles = (g.N + 127) / 128, q_tiles = (g.M + NT - 1) / NT;
    const int tiles = p_tiles * q_tiles;
    const int first = blockIdx.x / parts, stride = gridDim.x / parts;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::STAGES; ++i) {
            tc::mbar_init(&full[i], 1);
            tc::mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < C::BUFS; ++i) {
            tc::mbar_init(&acc_full[i], 1);
            tc::mbar_init(&acc_empty[i], EPI_WARPS);
        }
        for (int i = 0; i < SC_SLOTS; ++i) {
            tc::mbar_init(&sc_full[i], 1);
            tc::mbar_init(&sc_empty[i], EPI_WARPS);
        }
        *abort_flag = 0;
        tc::fence_barrier_init();
    }
    if (warp == WARP_MMA) {
        tc::tmem_alloc(tmem_at, C::TMEM_COLS);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tm = *tmem_at;
    // what comes of a and its scales waits for the kernel before this one; b may not depend on it (weights_early)
    if (!g.weights_early) pdl_wait();

    if (warp >= EPI_WARPS) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(OTHER_REGS));
        if (warp < WARP_MMA) {
            if (lane == 0) {
                const int turn = warp - WARP_TMA;
                int it = 0, sent = 0, early = 0;
                if (g.weights_early) {
                    if (first < tiles) {
                        early = min(kb1 - kb0, C::STAGES);
                        for (int i = turn; i < early; i += TURNS) {
                            tc::mbar_arrive_expect_tx(&full[i], C::STAGE);
                            tc::tma_load_2d(smem + i * C::STAGE, &map_b, &full[i], (kb0 + i) * 128, (first % p_tiles) * 128);
                        }
                    }
                    pdl_wait();
                }
                for (int u = first; u < tiles && !*abort_flag; u += stride) {
                    const int p0 = (u % p_tiles) * 128, q0 = (u / p_tiles) * NT;
                    for (int kb = kb0; kb < kb1; ++kb, ++it) {
                        if ((it & 1) != turn) continue;
                        const int slot = it % C::STAGES;
                        uint8_t* st = smem + slot * C::STAGE;
                        if (it >= early) {
                            if (!tc::mbar_wait(&empty[slot], (it / C::STAGES & 1) ^ 1)) {
                                *abort_flag = 1;
                                atomicOr(g.status, QMOE_DEV_WAIT_TIMEOUT);
                                break;
                            }
                            tc::mbar_arrive_expect_tx(&full[slot], C::STAGE);
                            tc::tma_load_2d(st, &map_b, &full[slot], kb * 128, p0);
                        }
                        tc::tma_load_2d(st + C::P_BYTES, &map_a, &full[slot], kb * 128, q0);
                        sent = it + 1;
                    }
                }
                if (*abort_flag)  // nobody may have waited for these: no load outlives the CTA
                    for (int i = sent - 1; i >= 0 && i > sent - 1 - C::STAGES; i -= TURNS)
                        tc::mbar_wait(&full[i % C::STAGES], i / C::STAGES & 1);
            }
            __syncwarp();
        } else if (warp < WARP_SCALE) {
            if (lane == 0) {
                constexpr uint32_t idesc = idesc_f8(128, NT);
                const int turn = warp - WARP_MMA;
                int it = 0, sent = 0;
                for (int u = first; u < tiles && !*abort_flag; u += stride) {
                    for (int kb = kb0; kb < kb1; ++kb, ++it) {
                        if ((it & 1) != turn) continue;
                        const int slot = it % C::STAGES, buf = it % C::BUFS;
                        if (!tc::mbar_wait(&acc_empty[buf], (it / C::BUFS & 1) ^ 1) ||
                            !tc::mbar_wait(&full[slot], it / C::STAGES & 1)) {
                            *abort_flag = 1;
                            atomicOr(g.status, QMOE_DEV_WAIT_TIMEOUT);
                            break;
                        }
                        tc::tc_fence_after();
                        const uint32_t st = tc::smem_u32(smem + slot * C::STAGE);
                        const uint64_t dp = tc::sdesc_kmajor_sw128(st), dq = tc::sdesc_kmajor_sw128(st + C::P_BYTES);
#pragma unroll
                        for (int k = 0; k < 4; ++k)  // 32 codes a step: 2 descriptor units of 16 bytes
                            mma_f8(tm + buf * NT, dp + 2 * k, dq + 2 * k, idesc, k > 0);
                        tc::mma_commit(&empty[slot]);
                        tc::mma_commit(&acc_full[buf]);
                        sent = it + 1;
                    }
                }
                if (*abort_flag && sent)  // no product outlives the accumulators
                    tc::mbar_wait(&acc_full[(sent - 1) % C::BUFS], (sent - 1) / C::BUFS & 1);
            }
            __syncwarp();
        } else if (warp < WARP_SCALE + TURNS) {
        // the scale warps take the blocks in turn; a block's loads go out before the slot is waited for
        if (g.weights_early) pdl_wait();
        int it = 0;
        for (int u = first; u < tiles && !*abort_flag; u += stride) {
            const int p0 = (u % p_tiles) * 128, q0 = (u / p_tiles) * NT;
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                if ((it & 1) != warp - WARP_SCALE) continue;
                const int slot = it % SC_SLOTS;
                constexpr int QN = (NT + 31) / 32;
                float sq[QN], sp[4];
                const float uni = UNI ? g.b.s[(p0 >> 7) * g.b.s_row + kb * g.b.s_blk] : 1.f;
#pragma unroll
                for (int i = 0; i < QN; ++i) {
                    const int m = q0 + i * 32 + lane;
                    sq[i] = m < g.M && i * 32 + lane < NT ? g.a.s[(m >> g.a.shift) * g.a.s_row + kb * g.a.s_blk] : 0.f;
                }
                if (!UNI) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int n = p0 + i * 32 + lane;
                        sp[i] = n < g.N ? g.b.s[(n >> g.b.shift) * g.b.s_row + kb * g.b.s_blk] : 0.f;
                    }
                }
                if (!warp_wait(&sc_empty[slot], (it / SC_SLOTS & 1) ^ 1, abort_flag, g.status)) break;
                float* to = sc + slot * C::SC_FLOATS;
#pragma unroll
                for (int i = 0; i < QN; ++i)
                    if (i * 32 + lane < NT) to[i * 32 + lane] = sq[i] * uni;
                if (!UNI) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) to[NT + i * 32 + lane] = sp[i];
                }
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&sc_full[slot]);
            }
        }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(EPI_REGS));
        constexpr int STEP = C::COLS < 16 ? C::COLS : 16, STEPS = C::COLS / STEP;
        const int quad = warp & 3, half = warp >> 2;
        const int p_lane = quad * 32 + lane;
        const uint32_t t_lane = tm + ((uint32_t)(quad * 32) << 16) + half * C::COLS;
        int slot = 0, buf = 0;
        uint32_t phase = 0, acc_phase = 0;
        uint64_t acc[C::COLS / 2];
        for (int u = first; u < tiles && !*abort_flag; u += stride) {
            const int p0 = (u % p_tiles) * 128, q0 = (u / p_tiles) * NT;
            bool ok = true;
#pragma unroll
            for (int i = 0; i < C::COLS / 2; ++i) acc[i] = 0ull;
            for (int kb = kb0; kb < kb1; ++kb) {
                ok = warp_wait(&sc_full[slot], phase, &acc_full[buf], acc_phase, abort_flag, g.status);
                if (!ok) break;
                tc::tc_fence_after();
                const float* s = sc + slot * C::SC_FLOATS + half * C::COLS;
                const float own = UNI ? 1.f : sc[slot * C::SC_FLOATS + NT + p_lane];
                const uint64_t sp = pair_of(own, own);
                uint32_t r[2][STEP];
                tmem_ld<STEP>(t_lane + buf * NT, r[0]);
#pragma unroll
                for (int i = 0; i < STEPS; ++i) {
                    tc::tmem_ld_wait();
                    if (i + 1 < STEPS) {
                        tmem_ld<STEP>(t_lane + buf * NT + (i + 1) * STEP, r[(i + 1) & 1]);
                    } else {
                        tc::tc_fence_before();
                        __syncwarp();
                        if (lane == 0) tc::mbar_arrive(&acc_empty[buf]);
                    }
#pragma unroll
                    for (int j = 0; j < STEP; j += 4) {
                        // volatile: read when they are used, not all ahead (512 x 2816 x 4096: 16.9 us against 19.0)
                        float4 v;
                        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                                     : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                                     : "r"(tc::smem_u32(s + i * STEP + j)));
                        uint64_t s0 = pair_of(v.x, v.y), s1 = pair_of(v.z, v.w);
                        if (!UNI) {
                            s0 = mul_pair(s0, sp);
                            s1 = mul_pair(s1, sp);
                        }
                        uint64_t* to = &acc[(i * STEP + j) / 2];
                        const uint32_t* d = &r[i & 1][j];
                        to[0] = fma_pair(pair_of(d[0], d[1]), s0, to[0]);
                        to[1] = fma_pair(pair_of(d[2], d[3]), s1, to[1]);
                    }
                }
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&sc_empty[slot]);
                if (++slot == SC_SLOTS) { slot = 0; phase ^= 1; }
                if (++buf == C::BUFS) { buf = 0; acc_phase ^= 1; }
            }
            if (!ok) break;
            if (parts == 1) {
                const int n = p0 + p_lane, m0 = q0 + half * C::COLS;
                const int64_t at = (int64_t)m0 * g.ldc + n;
                if (n < g.N) {
                    if (g.ctype == QMOE_F32) put_cols<C::COLS>(static_cast<float*>(g.c) + at, g.ldc, g.M - m0, acc);
                    else if (g.ctype == QMOE_BF16)
                        put_cols<C::COLS>(static_cast<__nv_bfloat16*>(g.c) + at, g.ldc, g.M - m0, acc);
                    else put_cols<C::COLS>(static_cast<__half*>(g.c) + at, g.ldc, g.M - m0, acc);
                }
            } else {
                // every load of this CTA's only tile has been consumed: the ring is free
                float* sums = reinterpret_cast<float*>(smem);
#pragma unroll
                for (int i = 0; i < C::COLS / 2; ++i) {
                    const float2 v = halves_of(acc[i]);
                    sums[(half * C::COLS + 2 * i) * 128 + p_lane] = v.x;
                    sums[(half * C::COLS + 2 * i + 1) * 128 + p_lane] = v.y;
                }
            }
        }
    }
    __syncwarp();
    if (parts > 1) {
        cluster_sync();
        const float* sums = reinterpret_cast<const float*>(smem);
        const int p0 = (first % p_tiles) * 128, q0 = (first / p_tiles) * NT;
        const int cols = min(NT, g.M - q0);
        // four rows of b at a time, the loads of up to four CTAs on their way at once (one value after the other cost
        // 2.5 us more at 128 columns); added in rank order
        for (int i = part * THREADS + threadIdx.x; i < cols * 32; i += parts * THREADS) {
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int r0 = 0; r0 < parts; r0 += 4) {
                float4 x[4];
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (r0 + r < parts) x[r] = peer_load(sums + i * 4, r0 + r);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (r0 + r < parts) {
                        v.x += x[r].x;
                        v.y += x[r].y;
                        v.z += x[r].z;
                        v.w += x[r].w;
                    }
            }
            const int n = p0 + (i & 31) * 4, m = q0 + (i >> 5);
            const int64_t at = (int64_t)m * g.ldc + n;
            const float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (n + j < g.N) put(g.c, g.ctype, at + j, e[j]);
        }
        cluster_sync();
    }
    // a kernel is let go only after the wait: a CTA counts as having done so by its first warp, and the warps without
    // work have not waited for weights_early's predecessor
    if (g.weights_early) pdl_wait();
    pdl_trigger();
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (warp == WARP_MMA) tc::tmem_dealloc(tm, C::TMEM_COLS);
}

// ------------------------------------------------------------------ host side

static int code_map(CUtensorMap* map, const uint8_t* q, int64_t ld, int rows, int K, int box_rows) {
    EncodeTiledFn enc = encode_tiled_fn();
    if (!enc) return QMOE_ERR_CUDA;
    const cuuint64_t dim[2] = {(cuuint64_t)K, (cuuint64_t)rows};
    const cuuint64_t stride[1] = {(cuuint64_t)ld};
    const cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
    const cuuint32_t one[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(q), dim, stride, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? QMOE_OK
               : QMOE_ERR_UNSUPPORTED;
}

struct Plan {
    int nt, parts;  // parts 0: the wide kernel
};

// Tile and split by a model of the time in us, fitted to sweeps of both on
// GB300 (K 64 to 8192, M 1 to 2048, N 1024 to 4096; within 15% of every
// measured time):
//   start + rounds * blocks * per_block + (split: 1.5 + nt / 80)
// rounds: tiles an SM takes in turn; blocks: of 128 along the reduction, in one
// part.  A split gives every cluster one tile; clusters of 8 fill no more than
// some 96 SMs, smaller ones 132.  A block costs a narrow tile little more than
// its handshakes (0.24 us at 16 columns, 0.29 at 64), so few tokens take the
// narrowest tile and split far: 5.6 us at M 1, N 2048, K 4096, 10.8 unsplit; at
// M 256, N 2816 three parts of 128 columns take 10.8, 64 columns unsplit 12.0.
// The wide kernel does twice the columns of nt = 128 in 0.55 us against 0.43,
// and only where a row block of b shares its scales: with column scales it took
// 0.92.
inline Plan plan_of(int M, int N, int K, bool uniform) {
    struct Tile {
        int nt;
        float start, per_block;
    };
    const Tile shared[4] = {{16, 2.6f, 0.24f}, {32, 2.6f, 0.25f}, {64, 2.9f, 0.29f}, {128, 3.1f, 0.43f}};
    const Tile own[4] = {{16, 2.6f, 0.28f}, {32, 2.6f, 0.30f}, {64, 2.9f, 0.37f}, {128, 3.1f, 0.51f}};  // a scale a row of b
    const Tile(&tile)[4] = uniform ? shared : own;
    const int splits[6] = {1, 2, 3, 4, 6, 8};
    const int blocks = (K + 127) / 128;
    Plan best = {128, 1};
    float least = 1e30f;
    for (const Tile& c : tile) {
        const int64_t tiles = (int64_t)((N + 127) / 128) * ((M + c.nt - 1) / c.nt);
        for (const int parts : splits) {
            if (parts > 1 && (parts > blocks || tiles * parts > (parts == 8 ? 96 : 132))) continue;
            const int64_t rounds = parts > 1 ? 1 : (tiles + row::kSMs - 1) / row::kSMs;
            const float us = c.start + (float)rounds * (float)((blocks + parts - 1) / parts) * c.per_block +
                             (parts > 1 ? 1.5f + (float)c.nt / 80.f : 0.f);
            if (us < least) {
                least = us;
                best = {c.nt, parts};
            }
        }
    }
    if (uniform) {
        const int64_t tiles = (int64_t)((M + 127) / 128) * ((N + WIDE_N - 1) / WIDE_N);
        const float us = 4.2f + (float)((tiles + row::kSMs - 1) / row::kSMs) * (float)blocks * 0.55f;
        if (us < least) best = {WIDE_N, 0};
    }
    return best;
}

template <int NT, bool UNI>
static int gemm_launch(const CUtensorMap& ma, const CUtensorMap& mb, const GemmArgs& g, int parts, cudaStream_t st) {
    using C = GemmCfg<NT, UNI>;
    const int rc = row::allow_smem<fp8_gemm_kernel<NT, UNI>>(C::SMEM);
    if (rc != QMOE_OK) return rc;
    const int64_t tiles = (int64_t)((g.N + 127) / 128) * ((g.M + NT - 1) / NT);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)parts;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    // a split reduction gives each cluster exactly one tile
    cfg.gridDim = dim3((unsigned)(parts > 1 ? tiles * parts : tiles < row::kSMs ? tiles : row::kSMs));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, fp8_gemm_kernel<NT, UNI>, ma, mb, g) == cudaSuccess ? QMOE_OK : QMOE_ERR_LAUNCH;
}

template <int NT>
static int gemm_kind(const CUtensorMap& ma, const CUtensorMap& mb, const GemmArgs& g, int parts, cudaStream_t st) {
    return g.b.shift ? gemm_launch<NT, true>(ma, mb, g, parts, st) : gemm_launch<NT, false>(ma, mb, g, parts, st);
}

static int gemm_run(const qmoe_fp8_mat* a, const qmoe_fp8_mat* b, GemmArgs& g, cudaStream_t st) {
    const Plan p = plan_of(g.M, g.N, g.K, g.b.shift != 0);
    CUtensorMap ma, mb;
    int rc = code_map(&ma, a->q, a->ld, g.M, g.K, p.parts ? p.nt : 128);
    if (rc != QMOE_OK) return rc;
    rc = code_map(&mb, b->q, b->ld, g.N, g.K, p.parts ? 128 : 256);
    if (rc != QMOE_OK) return rc;
    if (!p.parts) return gemm_wide(ma, mb, g, st);
    switch (p.nt) {
        case 16: return gemm_kind<16>(ma, mb, g, p.parts, st);
        case 32: return gemm_kind<32>(ma, mb, g, p.parts, st);
        case 64: return gemm_kind<64>(ma, mb, g, p.parts, st);
        case 128: return gemm_kind<128>(ma, mb, g, p.parts, st);
        default: return QMOE_ERR_UNSUPPORTED;  // the maps' boxes go with the kernels' tiles: no other kernel may take them
    }
}

inline bool mat_ok(const qmoe_fp8_mat* m, int64_t K) {
    return m && m->q && m->s && aligned16(m->q) && m->ld >= K && m->ld % 16 == 0 && row::type_aligned(m->s, 4) &&
           (m->s_rows == 1 || m->s_rows == 128);
}
inline Side side_of(const qmoe_fp8_mat* m) { return {m->s, m->s_row, m->s_blk, m->s_rows == 128 ? 7 : 0}; }

static int check_sizes(int64_t M, int64_t N, int64_t K, int ctype, int64_t ldc) {
    if (M < 0 || N <= 0 || K <= 0 || !row::dtype_ok(ctype) || ldc < N) return QMOE_ERR_ARG;
    const int64_t most = 1ll << 30;
    if (M > most || N > most || K > most || ((M + 15) / 16) * ((N + 127) / 128) >= most) return QMOE_ERR_UNSUPPORTED;
    return QMOE_OK;
}

}  // namespace fp8
}  // namespace qmoe

using namespace qmoe;

extern "C" int qmoe_fp8_matmul(int64_t M, int64_t N, int64_t K, const qmoe_fp8_mat* a, const qmoe_fp8_mat* b, void* c,
                               int c_dtype, int64_t ldc, int32_t* dev_status, qmoe_stream_t stream) {
    const int rc = fp8::check_sizes(M, N, K, c_dtype, ldc);
    if (rc != QMOE_OK) return rc;
    if (M == 0) return QMOE_OK;
    if (!fp8::mat_ok(a, K) || !fp8::mat_ok(b, K) || !c || !row::type_aligned(c, row::dtype_size(c_dtype)) ||
        !dev_status || !row::type_aligned(dev_status, 4))
        return QMOE_ERR_ARG;
    fp8::GemmArgs g = {(int)M, (int)N, (int)K, fp8::side_of(a), fp8::side_of(b), c, ldc, c_dtype,
                       dev_status, 0};
    return fp8::gemm_run(a, b, g, (cudaStream_t)stream);
}

static int64_t linear_ld(int64_t K) { return (K + 15) / 16 * 16; }
static size_t linear_codes(int64_t M, int64_t K) { return ((size_t)M * linear_ld(K) + 255) / 256 * 256; }

extern "C" size_t qmoe_fp8_linear_workspace_bytes(int64_t M, int64_t K) {
    if (M <= 0 || K <= 0) return 0;
    return linear_codes(M, K) + ((size_t)M * ((K + 127) / 128) * 4 + 255) / 256 * 256;
}

extern "C" int qmoe_fp8_linear(int64_t M, int64_t N, int64_t K, int x_dtype, const void* x, int64_t ldx,
                               const qmoe_fp8_mat* w, void* y, int y_dtype, int64_t ldy, int32_t* dev_status, void* ws,
                               size_t ws_bytes, qmoe_stream_t stream) {
    int rc = fp8::check_sizes(M, N, K, y_dtype, ldy);
    if (rc != QMOE_OK) return rc;
    if (!row::dtype_ok(x_dtype)) return QMOE_ERR_ARG;
    if (M == 0) return QMOE_OK;
    if (!x || ldx < K || !row::type_aligned(x, row::dtype_size(x_dtype)) || !fp8::mat_ok(w, K) || !y ||
        !row::type_aligned(y, row::dtype_size(y_dtype)) || !dev_status || !row::type_aligned(dev_status, 4) || !ws ||
        (reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < qmoe_fp8_linear_workspace_bytes(M, K))
        return QMOE_ERR_ARG;
    uint8_t* q = static_cast<uint8_t*>(ws);
    float* s = reinterpret_cast<float*>(q + linear_codes(M, K));
    rc = fp8::quant_rows_launch(M, K, x_dtype, x, ldx, q, linear_ld(K), s, (cudaStream_t)stream);
    if (rc != QMOE_OK) return rc;
    const qmoe_fp8_mat a = {q, linear_ld(K), s, 1, M, 1, 0};
    fp8::GemmArgs g = {(int)M, (int)N, (int)K, fp8::side_of(&a), fp8::side_of(w), y, ldy, y_dtype,
                       dev_status, 1};
    return fp8::gemm_run(&a, w, g, (cudaStream_t)stream);
}
