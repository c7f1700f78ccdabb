// Pieces shared by the FP8 product kernels (fp8_gemm.cu, fp8_gemm_wide.cu):
// arguments, fp32 pairs, waits, cluster addressing.
#pragma once

#include "row_ops.cuh"
#include "tc_ptx.cuh"
#include "tma_host.cuh"

namespace qmoe {
namespace fp8 {

// Warps: 8 scale and sum; then two each that load tiles, issue products and
// bring scales, and two without work (registers are split by warpgroups).  The
// two of a kind take the reduction's blocks in turn: a thread needs about 400
// cycles to wait for a stage and issue its loads, and about 700 to issue a
// block's products, against 512 cycles that the products of a block take.
constexpr int EPI_WARPS = 8, WARP_TMA = 8, WARP_MMA = 10, WARP_SCALE = 12, THREADS = 16 * 32;
constexpr int TURNS = 2;
constexpr int SC_SLOTS = 8;  // scale ring
// Registers: launched with 128 a thread (65,536 in all); the epilogue's two
// warpgroups take 200, the others keep 56 (65,536 in all).
constexpr int EPI_REGS = 200, OTHER_REGS = 56;

struct Side {
    const float* s;
    int64_t s_row, s_blk;
    int shift;  // log2 of the rows that share a scale (0 or 7)
};

struct GemmArgs {
    int M, N, K;  // rows of a, rows of b, reduction
    Side a, b;
    void* c;
    int64_t ldc;
    int ctype;
    int32_t* status;
    int weights_early;  // b does not depend on the kernel before this one (narrow kernel)
};

__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Instruction descriptor: E4M3 operands (format 0), fp32 sums, both K-major.
__host__ __device__ constexpr uint32_t idesc_f8(int M, int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Two fp32 values in a 64-bit register pair.
__device__ __forceinline__ uint64_t pair_of(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ uint64_t pair_of(uint32_t a, uint32_t b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ float2 halves_of(uint64_t p) {
    float2 v;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(p));
    return v;
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t mul_pair(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[N]) {
    static_assert(N == 8 || N == 16, "");
    if constexpr (N == 16) {
        tc::tmem_ld_32x32b_x16(taddr, r);
    } else {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "r"(taddr));
    }
}

// One lane waits for both barriers (a wait by all 32 lanes takes some 200
// cycles even where the phase is over, by one lane 50); __syncwarp passes on
// to the others what the barriers guard.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, uint64_t* bar2, uint32_t parity2,
                                          volatile int* abort_flag, int32_t* status) {
    int ok = 1;
    if ((threadIdx.x & 31) == 0 && !(tc::mbar_wait(bar, parity) && (!bar2 || tc::mbar_wait(bar2, parity2)))) {
        *abort_flag = 1;
        atomicOr(status, QMOE_DEV_WAIT_TIMEOUT);
        ok = 0;
    }
    ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
    __syncwarp();
    return ok != 0;
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int32_t* status) {
    return warp_wait(bar, parity, nullptr, 0, abort_flag, status);
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// 16 bytes of the shared memory of the cluster's CTA `rank`, at this CTA's address `p`.
__device__ __forceinline__ float4 peer_load(const float* p, uint32_t rank) {
    uint32_t at;
    float4 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(tc::smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(at)
                 : "memory");
    return v;
}

// The product of both maps (boxes of 128 rows of a, 256 of b) in 128 x 256
// tiles, for b whose rows share their scales by 128.
constexpr int WIDE_N = 256;
int gemm_wide(const CUtensorMap& ma, const CUtensorMap& mb, const GemmArgs& g, cudaStream_t st);

}  // namespace fp8
}  // namespace qmoe
