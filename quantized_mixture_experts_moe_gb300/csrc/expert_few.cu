// y[s] = w[e] x[s] for few rows an expert and weights whose rows lie off the 16-byte
// boundaries, where TMA cannot read them and a copy would take the experts' bytes
// twice more: they go from HBM into the registers of mma.sync m16n8k16, 16 rows of w and
// 8 rows of x, by aligned loads and shifts.  The order of the
// reduction is free, so a lane's operand is 16 contiguous bytes of its row of w
// and of its row of x.  A CTA takes 16 rows of one expert; its 8 warps share the
// reduction and add their parts in order.
//
// The CTA of slot s works for the expert whose first row s is, the others of the
// expert end: no expert without rows costs anything, and every CTA finds its
// expert in one parallel look at the offsets.  One token x 8 of 128 experts, 2047 ->
// 1536: 22 us, 2.3 TB/s, bounded by the latency of a CTA's few rounds of loads; 41
// with a copy of the eight experts' weights.
#include "expert_gemm.cuh"

namespace qmoe {
namespace eg {

constexpr int FEW_WARPS = 8, FEW_THREADS = FEW_WARPS * 32, FEW_ROWS = 16, FEW_COLS = 8;
constexpr int FEW_DEPTH = 4;  // pieces of 32 reduction values on their way

struct FewArgs {
    const uint16_t *x, *w;
    int64_t ldx, ldw, w_expert;
    int P, E, N, K;
    const int32_t *offsets, *pairs;
    int k, x_rows;
    void* y;
    int64_t ldy;
    int ytype;
    int32_t* status;
};

// Values k .. k + 7 of a row of n, as they lie in memory: loaded first, put in
// place when all loads of a round are on their way.  WIDE: rows on 16-byte
// boundaries; else two aligned pieces, each read only where it holds values of the
// row.
template <bool WIDE>
struct Piece {
    uint4 v, w;
    __device__ __forceinline__ void load(const uint16_t* row, int k, int n) {
        const bool there = row != nullptr && k < n;
        v = w = make_uint4(0, 0, 0, 0);
        if constexpr (WIDE) {
            if (there) v = *reinterpret_cast<const uint4*>(row + k);
        } else {
            const uintptr_t a = reinterpret_cast<uintptr_t>(row + k), p = a & ~uintptr_t(15);
            if (there) v = *reinterpret_cast<const uint4*>(p);
            if (there && p != a && p + 16 < reinterpret_cast<uintptr_t>(row + n)) w = *reinterpret_cast<const uint4*>(p + 16);
        }
    }
    // zeros from n on
    __device__ __forceinline__ uint4 get(const uint16_t* row, int k, int n) const {
        uint4 o = v;
        if constexpr (!WIDE) {
            const uint32_t shift = (uint32_t)reinterpret_cast<uintptr_t>(row + k) & 15;
            const bool two = shift & 8, one = shift & 4;
            const uint32_t b[6] = {two ? v.z : v.x, two ? v.w : v.y, two ? w.x : v.z, two ? w.y : v.w, two ? w.z : w.x, two ? w.w : w.y};
            const uint32_t by = shift & 2 ? 0x5432 : 0x3210;
            uint32_t c[5];
#pragma unroll
            for (int i = 0; i < 5; ++i) c[i] = one ? b[i + 1] : b[i];
            o = make_uint4(__byte_perm(c[0], c[1], by), __byte_perm(c[1], c[2], by), __byte_perm(c[2], c[3], by), __byte_perm(c[3], c[4], by));
        }
        if (k + 8 > n) {
            uint32_t* u = &o.x;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (k + 2 * i >= n) u[i] = 0;
                else if (k + 2 * i + 1 >= n) u[i] &= 0xFFFFu;
            }
        }
        return o;
    }
};

template <typename T, bool WIDE_X>
__global__ void __launch_bounds__(FEW_THREADS) expert_few_kernel(const FewArgs g) {
    __shared__ float part[FEW_WARPS][FEW_COLS][FEW_ROWS];
    __shared__ int span[2];  // the expert and the end of its rows
    constexpr bool BF16 = std::is_same<T, __nv_bfloat16>::value;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = lane >> 2, quad = lane & 3;
    const int s0 = blockIdx.y, n0 = blockIdx.x * FEW_ROWS;
    if (threadIdx.x == 0) span[0] = -1;
    __syncthreads();
    pdl_wait();
    bool bad = false;
    for (int e = threadIdx.x; e <= g.E; e += FEW_THREADS) {
        const int a = g.offsets[e], b = e < g.E ? g.offsets[e + 1] : a;
        bad |= a < 0 || a > g.P || b < a || (e == 0 && a != 0);
        if (e < g.E && a == s0 && b > s0) {
            span[0] = e;
            span[1] = min(b, g.P);
        }
        if (e == g.E && a <= s0) {  // a row of no expert
            span[0] = g.E;
            span[1] = s0;
        }
    }
    if (bad && blockIdx.x == 0 && blockIdx.y == 0) atomicOr(g.status, QMOE_DEV_BAD_OFFSETS);
    __syncthreads();
    pdl_trigger();
    const int e = span[0];
    if (e < 0) return;
    if (e == g.E) {
        if (threadIdx.x < FEW_ROWS && n0 + threadIdx.x < g.N) put_value(g.y, g.ytype, s0 * g.ldy + n0 + threadIdx.x, 0.f);
        return;
    }
    const int end = span[1];
    const uint16_t* const w = g.w + e * g.w_expert + (int64_t)(n0 + row) * g.ldw;
    const uint16_t *const w0 = n0 + row < g.N ? w : nullptr, *const w1 = n0 + row + 8 < g.N ? w + 8 * g.ldw : nullptr;
    const int pieces = (g.K + 31) / 32;  // of 32 values, 8 a lane of a quad
    for (int s = s0; s < end; s += FEW_COLS) {
        const uint16_t* x = nullptr;
        if (s + row < end) {
            int r = s + row;
            if (g.pairs) {
                const int p = g.pairs[r];
                r = p >= 0 ? min(p / g.k, g.x_rows) : g.x_rows;
            }
            if (r < g.x_rows) x = g.x + r * g.ldx;
        }
        float acc[4] = {0.f, 0.f, 0.f, 0.f};  // sums of a round's products, which the tensor core cuts off, added by fp32's rounding
        for (int i0 = warp; i0 < pieces; i0 += FEW_WARPS * FEW_DEPTH) {
            Piece<false> a[FEW_DEPTH], b[FEW_DEPTH];
            Piece<WIDE_X> v[FEW_DEPTH];
            float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < FEW_DEPTH; ++j) {
                const int k = (i0 + j * FEW_WARPS) * 32 + quad * 8;
                a[j].load(w0, k, g.K);
                b[j].load(w1, k, g.K);
                v[j].load(x, k, g.K);
            }
#pragma unroll
            for (int j = 0; j < FEW_DEPTH; ++j) {
                const int k = (i0 + j * FEW_WARPS) * 32 + quad * 8;
                const uint4 p = a[j].get(w0, k, g.K), q = b[j].get(w1, k, g.K), r = v[j].get(x, k, g.K);
                tc::mma_sync<BF16>(d, p.x, q.x, p.y, q.y, r.x, r.y);
                tc::mma_sync<BF16>(d, p.z, q.z, p.w, q.w, r.z, r.w);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[j] += d[j];
        }
        if (s > s0) __syncthreads();
        part[warp][quad * 2][row] = acc[0];
        part[warp][quad * 2 + 1][row] = acc[1];
        part[warp][quad * 2][row + 8] = acc[2];
        part[warp][quad * 2 + 1][row + 8] = acc[3];
        __syncthreads();
        if (threadIdx.x < FEW_COLS * FEW_ROWS) {
            const int c = threadIdx.x / FEW_ROWS, n = threadIdx.x % FEW_ROWS;
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < FEW_WARPS; ++i) sum += part[i][c][n];
            if (s + c < end && n0 + n < g.N) put_value(g.y, g.ytype, (s + c) * g.ldy + n0 + n, sum);
        }
    }
}

template <typename T>
static int few_launch(const FewArgs& g, bool wide_x, cudaStream_t st) {
    return launch_pdl(wide_x ? expert_few_kernel<T, true> : expert_few_kernel<T, false>,
                      dim3((unsigned)((g.N + FEW_ROWS - 1) / FEW_ROWS), (unsigned)g.P), dim3(FEW_THREADS), 0, st, g);
}

int launch_few(const Mat& w, const Mat& x, const Args& a, int dtype, cudaStream_t st) {
    const FewArgs g = {static_cast<const uint16_t*>(x.p), static_cast<const uint16_t*>(w.p), x.ld, w.ld, w.stride, a.P, a.E, a.lanes, a.red,
                       a.offsets, a.pairs, a.k, a.x_rows, a.out, a.ld, a.ctype, a.status};
    return dtype == QMOE_BF16 ? few_launch<__nv_bfloat16>(g, fits(x), st) : few_launch<__half>(g, fits(x), st);
}

}  // namespace eg
}  // namespace qmoe
