// Top-k routing with the balance loss and the per-expert counts
// (qmoe_route_topk), and its gradient (qmoe_route_topk_backward).
//
//   p = softmax(logit),  ids = the k experts of largest logit + bias,
//   counts_e = pairs of expert e,  P_e = mean_t p_te,
//   loss = coef E sum_e counts_e / (k n) P_e   (n routed tokens)
//   dlogit = p (a - sum p a - s) + [selected] w_j (dw_j - r),
//   a_e = dloss coef E counts_e / (k n^2)
//
// A warp takes a token at a time, its logits spread over the lanes' registers
// (by 16-byte loads where rows allow it), so a row is read once for the
// softmax, the selection and the statistics.  Selection goes by
// order-preserving integer keys from the largest down: the next key is the
// largest below the last one, a warp-wide maximum of key - last, which wraps
// so that what has been taken falls to the bottom (one fused add-and-maximum
// for each register, nothing to clear).  A 16-bit logit's key leaves room for
// the expert's number, so one redux gives both and equal logits come lowest
// expert first.  32-bit scores (fp32 logits, a bias) give their lowest bits, up
// to 10, to the number; where the k + 1 largest differ above them, that order is the
// scores' own, and the rare token where two do not is selected anew by whole
// scores.  Instruction issue, not the 2 E bytes of a row, is the bound.
// Probabilities are summed per lane over a warp's tokens, then over a CTA's
// warps, then over CTAs, in a fixed order, so the loss has the same bits every
// time.  Exponentials are __expf's: a relative error of about |logit - maximum|
// roundings, which is most for the experts of least weight.
//
// T=8192, E=512, k=8, bf16: 9.7 us without statistics (0.9 TB/s), 17.5 with
// them, which takes a second launch (up to 16 tokens one CTA does both: T=1
// 4.6 us, 8.2 with two launches); with a bias 16 and 23 us, fp32 logits 14.5 and
// 22; the gradient 8.8 us.
#include "row_ops.cuh"

namespace qmoe {
namespace route {

constexpr int MAX_E = 1024, MAX_K = 32, WARPS = 16;

struct Args {
    int64_t T;
    int E, k;
    const void* logits;
    int64_t ld;
    const float* bias;
    const uint8_t* mask;
    int renorm;
    float scale;
    int32_t* ids;
    float* w;
    float* lse;
    // statistics (part_p null: none): per CTA, probabilities and counts by expert, then the routed tokens
    float* part_p;
    int32_t* part_c;
    int32_t* arrived;
    float coef;
    // where one CTA has all tokens, what route_stats_kernel writes otherwise
    int32_t* counts_out;
    float *probs, *loss;
    // gradient
    const float* dw;
    const int32_t* counts;
    const float* dloss;
    void* dlogits;
    int64_t ldd;
};

// NaN counts as -inf (an invalid logit selects nothing), +inf as the largest
// finite value.
constexpr float LARGEST = 3.402823466e38f;
__device__ __forceinline__ float clean(float v) { return v > -INFINITY ? fminf(v, LARGEST) : -INFINITY; }

// Larger floats have larger keys; -0 and +0 have the same.  Keys below
// AVAILABLE are -inf's.
constexpr uint32_t AVAILABLE = 0x00800000u;
__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t u = __float_as_uint(v + 0.f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
// A bf16 or fp16 value is told by the upper 19 bits of its fp32 form (8 of
// exponent, at most 10 of mantissa): below them goes the expert, reversed.
// Only what +inf became has bits below them; it is above every 16-bit value.
constexpr uint32_t VALUE_BITS = 0xFFFFE000u;
constexpr float LARGEST_16 = 3.38953139e38f;  // bf16's
__device__ __forceinline__ uint32_t packed_key(float v, int e) {
    return (key_of(v) & VALUE_BITS) | (0x1FFFu - (uint32_t)e);
}
__device__ __forceinline__ int packed_expert(uint32_t key) { return (int)(0x1FFFu - (key & 0x1FFFu)); }
__device__ __forceinline__ float packed_value(uint32_t key) {
    return __uint_as_float(((key & 0x80000000u) ? (key & 0x7FFFFFFFu) : ~key) & VALUE_BITS);
}

// A 32-bit score's key with the expert, reversed, in the bits that number the NE * 32 experts.
template <int NE>
constexpr uint32_t NUMBER_BITS = NE * 32 - 1;
template <int NE>
__device__ __forceinline__ uint32_t rough_key(float v, int e) {
    return (key_of(v) & ~NUMBER_BITS<NE>) | (NUMBER_BITS<NE> - (uint32_t)e);
}
template <int NE>
__device__ __forceinline__ int rough_expert(uint32_t key) {
    return (int)(NUMBER_BITS<NE> - (key & NUMBER_BITS<NE>));
}

using row::warp_sum;
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}

// Which experts a lane holds: value i is expert (i / V) 32 V + lane V + i % V.
template <int V>
__device__ __forceinline__ int expert_of(int i, int lane) {
    return (i / V) * (32 * V) + lane * V + i % V;
}

// A row's logits, cleaned; -inf past the last expert.
template <typename T, int NE, int V>
__device__ __forceinline__ void load_logits(const T* row, int E, int lane, float (&v)[NE]) {
    bool fine = true;
#pragma unroll
    for (int i = 0; i < NE; i += V) {
        const int e = expert_of<V>(i, lane);
        if (V == 1) {
            v[i] = e < E ? row::to_f32(row[e]) : -INFINITY;
        } else if (e < E) {
            struct alignas(sizeof(T) * V) Pack { T x[V]; };
            const Pack p = *reinterpret_cast<const Pack*>(row + e);
#pragma unroll
            for (int j = 0; j < V; ++j) v[i + j] = row::to_f32(p.x[j]);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) v[i + j] = -INFINITY;
        }
    }
#pragma unroll
    for (int i = 0; i < NE; ++i) fine = fine && v[i] <= LARGEST;
    if (!fine) {
#pragma unroll
        for (int i = 0; i < NE; ++i) v[i] = clean(v[i]);
    }
}

// Keys of a lane's scores; past the last expert, where a logit is -inf, not
// available.  The bias comes 16 bytes at a time where logits do.
template <int NE, int V>
__device__ __forceinline__ void rough_keys(const float* bias, int E, int lane, const float (&v)[NE], uint32_t (&key)[NE]) {
    constexpr int W = V < 4 ? V : 4;
    struct alignas(4 * W) Pack { float x[W]; };
#pragma unroll
    for (int i = 0; i < NE; i += W) {
        const int e = expert_of<V>(i, lane);
        Pack p = {};
        if (bias && e < E) p = *reinterpret_cast<const Pack*>(bias + e);
        bool fine = true;
#pragma unroll
        for (int j = 0; j < W; ++j) {
            p.x[j] += v[i + j];
            fine = fine && p.x[j] <= LARGEST;
        }
        if (!fine) {
#pragma unroll
            for (int j = 0; j < W; ++j) p.x[j] = clean(p.x[j]);
        }
#pragma unroll
        for (int j = 0; j < W; ++j) key[i + j] = rough_key<NE>(p.x[j], e + j);
    }
}

// The largest key below `last` of all lanes' (last = 0: of all); false: there is none that is available.
template <int NE>
__device__ __forceinline__ bool next_key(const uint32_t (&key)[NE], uint32_t& last) {
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < NE; ++i) best = __viaddmax_u32(key[i], 0u - last, best);
    const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, best) + last;
    if (top < AVAILABLE || (last != 0 && top >= last)) return false;
    last = top;
    return true;
}

// Selection by whole 32-bit scores: all experts of one score leave in ascending order.  Lane j gets the j-th.
template <typename T, int NE, int V>
__device__ __noinline__ int select_by_score(const T* row, const float* bias, int E, int k, int lane) {
    float v[NE];
    uint32_t key[NE], last = 0;
    load_logits<T, NE, V>(row, E, lane, v);
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        const int e = expert_of<V>(i, lane);
        key[i] = e < E ? key_of(bias ? clean(v[i] + bias[e]) : v[i]) : 0u;
    }
    int mine = -1;
    for (int j = 0; j < k && next_key(key, last);) {
        uint32_t here = 0;  // which of this lane's experts have this score
#pragma unroll
        for (int i = 0; i < NE; ++i) here |= key[i] == last ? 1u << i : 0u;
        while (j < k) {
            const int i = __ffs(here) - 1;
            const unsigned e = here ? (unsigned)expert_of<V>(i, lane) : 0x7FFFFFFFu;
            const unsigned win = __reduce_min_sync(0xFFFFFFFFu, e);
            if (win == 0x7FFFFFFFu) break;
            if (e == win) here &= here - 1;
            if (lane == j) mine = (int)win;
            ++j;
        }
    }
    return mine;
}

template <typename T, int NE, int V, bool PACK>
__global__ void __launch_bounds__(WARPS * 32, NE > 16 ? 1 : 2)
route_kernel(const Args a) {
    extern __shared__ float smem[];  // statistics: [WARPS][E] sums of p, then [E + 1] counts
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = a.E;
    int* const count = reinterpret_cast<int*>(smem + WARPS * E);
    const bool stats = a.part_p != nullptr;
    pdl_sync();
    if (stats) {
        for (int i = threadIdx.x; i <= E; i += blockDim.x) count[i] = 0;
        if (blockIdx.x == 0 && threadIdx.x == 0) *a.arrived = 0;  // for route_stats_kernel
        __syncthreads();
    }
    float psum[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) psum[i] = 0.f;
    for (int64_t t = (int64_t)blockIdx.x * WARPS + warp; t < a.T; t += (int64_t)gridDim.x * WARPS) {
        const T* row = static_cast<const T*>(a.logits) + t * a.ld;
        float v[NE], m = -INFINITY;
        load_logits<T, NE, V>(row, E, lane, v);
#pragma unroll
        for (int i = 0; i < NE; ++i) m = fmaxf(m, v[i]);
        m = warp_max(m);
        const bool routed = m > -INFINITY && (!a.mask || a.mask[t]);
        if (!routed) {
            if (lane < a.k) {
                a.ids[t * a.k + lane] = -1;
                a.w[t * a.k + lane] = 0.f;
            }
            if (lane == 0 && a.lse) a.lse[t] = -INFINITY;
            continue;
        }
        uint32_t key[NE];
        if constexpr (PACK) {
#pragma unroll
            for (int i = 0; i < NE; ++i) key[i] = packed_key(v[i], expert_of<V>(i, lane));
        } else {
            rough_keys<NE, V>(a.bias, E, lane, v, key);
        }
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            v[i] = __expf(v[i] - m);
            sum += v[i];
        }
        sum = warp_sum(sum);
        const float inv = 1.f / sum;
        if (stats) {
#pragma unroll
            for (int i = 0; i < NE; ++i) psum[i] = fmaf(v[i], inv, psum[i]);
        }
        // lane j: the expert of rank j and its logit
        int mine = -1;
        float l = -INFINITY;
        uint32_t last = 0;  // key - 0: at first all keys are below
        if constexpr (PACK) {
            for (int j = 0; j < a.k && next_key(key, last); ++j)
                if (lane == j) {
                    mine = packed_expert(last);
                    l = packed_value(last);
                }
            if (l > LARGEST_16) l = LARGEST;  // +inf's key without its low bits
        } else {
            bool sure = true;
            for (int j = 0; j <= a.k; ++j) {
                const uint32_t before = last;
                if (!next_key(key, last)) break;
                sure = j == 0 || (before ^ last) > NUMBER_BITS<NE>;
                if (!sure) break;
                if (lane == j && j < a.k) mine = rough_expert<NE>(last);
            }
            if (!sure) mine = select_by_score<T, NE, V>(row, a.bias, E, a.k, lane);
            if (mine >= 0) l = clean(row::to_f32(row[mine]));
        }
        float w;
        if (a.renorm) {
            const float best = warp_max(l);
            w = __expf(l - best);
            w *= a.scale / warp_sum(w);
        } else {
            w = a.scale * (__expf(l - m) * inv);
        }
        if (lane < a.k) {
            a.ids[t * a.k + lane] = mine;
            a.w[t * a.k + lane] = mine >= 0 ? w : 0.f;
            if (stats && mine >= 0) atomicAdd(&count[mine], 1);
        }
        if (lane == 0) {
            if (a.lse) a.lse[t] = m + logf(sum);
            if (stats) atomicAdd(&count[E], 1);
        }
    }
    if (!stats) return;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        const int e = expert_of<V>(i, lane);
        if (e < E) smem[warp * E + e] = psum[i];
    }
    __syncthreads();
    if (gridDim.x == 1) {  // a launch less: T=16, E=512, k=8 5.4 us against 9.0
        const int n = count[E];
        const float total = (float)max(n, 1);
        float part = 0.f;
        for (int e = threadIdx.x; e < E; e += blockDim.x) {
            float p = 0.f;
#pragma unroll
            for (int i = 0; i < WARPS; ++i) p += smem[i * E + e];
            p /= total;
            a.counts_out[e] = count[e];
            a.probs[e] = p;
            part = fmaf((float)count[e] / (total * (float)a.k), p, part);
        }
        if (threadIdx.x == 0) a.counts_out[E] = n;
        part = warp_sum(part);
        __syncthreads();
        if (lane == 0) smem[warp] = part;
        __syncthreads();
        if (warp == 0) {
            part = warp_sum(lane < WARPS ? smem[lane] : 0.f);
            if (lane == 0) a.loss[0] = a.coef * (float)E * part;
        }
        return;
    }
    for (int e = threadIdx.x; e <= E; e += blockDim.x) {
        a.part_c[(int64_t)blockIdx.x * (E + 1) + e] = count[e];
        if (e == E) break;
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < WARPS; ++i) s += smem[i * E + e];
        a.part_p[(int64_t)blockIdx.x * E + e] = s;
    }
}

// Sums the CTAs' statistics: counts[E + 1], probs[E] and the loss.  A CTA takes
// 32 experts, 32 threads each; the CTA that is last to arrive adds the CTAs'
// parts of the loss, in their order.
struct StatArgs {
    int parts, E, k;
    const float* part_p;
    const int32_t* part_c;
    float* part_loss;
    int32_t* arrived;
    float coef;
    int32_t* counts;
    float* probs;
    float* loss;
};
__global__ void __launch_bounds__(1024) route_stats_kernel(const StatArgs a) {
    __shared__ float sp[32][33];
    __shared__ int sc[32][33];
    __shared__ int last, routed;
    pdl_sync();
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, E = a.E, e = blockIdx.x * 32 + tx;
    int n = 0;
    for (int i = threadIdx.x; i < a.parts; i += 1024) n += a.part_c[(int64_t)i * (E + 1) + E];
    int c = 0;
    float p = 0.f;
    if (e < E) {
#pragma unroll 4
        for (int i = ty; i < a.parts; i += 32) {
            c += a.part_c[(int64_t)i * (E + 1) + e];
            p += a.part_p[(int64_t)i * E + e];
        }
    }
    if (threadIdx.x == 0) routed = 0;
    sp[ty][tx] = p;
    sc[ty][tx] = c;
    __syncthreads();
    n = __reduce_add_sync(0xFFFFFFFFu, n);
    if (tx == 0 && n) atomicAdd(&routed, n);
    // warp ty sums expert ty
    p = warp_sum(sp[tx][ty]);
    c = __reduce_add_sync(0xFFFFFFFFu, sc[tx][ty]);
    __syncthreads();
    const float total = (float)(routed > 0 ? routed : 1);
    const int mine = blockIdx.x * 32 + ty;
    p /= total;
    if (tx == 0) {
        if (mine < E) {
            a.counts[mine] = c;
            a.probs[mine] = p;
        }
        sp[0][ty] = mine < E ? (float)c / (total * (float)a.k) * p : 0.f;
    }
    __syncthreads();
    if (ty != 0) return;
    const float part = warp_sum(sp[0][tx]);
    if (tx == 0) {
        if (blockIdx.x == 0) a.counts[E] = routed;
        a.part_loss[blockIdx.x] = part;
        __threadfence();
        last = atomicAdd(a.arrived, 1) == (int)gridDim.x - 1;
    }
    __syncwarp();
    if (!last) return;
    __threadfence();
    const float loss = warp_sum(tx < (int)gridDim.x ? __ldcg(a.part_loss + tx) : 0.f);  // E <= 1024: 32 CTAs at most
    if (tx == 0) a.loss[0] = a.coef * (float)E * loss;
}

template <typename T, int NE, int V>
__global__ void __launch_bounds__(WARPS * 32, NE > 16 ? 1 : 2)
route_bwd_kernel(const Args a) {
    extern __shared__ float smem[];  // [WARPS][NE * 32]: what the selected experts get besides
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = a.E;
    float* const extra = smem + warp * NE * 32;
    pdl_sync();
    for (int e = lane; e < NE * 32; e += 32) extra[e] = 0.f;
    __syncwarp();
    float ga[NE];
    float c = 0.f;
    if (a.dloss) {
        const float n = (float)max(a.counts[E], 1);
        c = a.dloss[0] * a.coef * (float)E / (n * (float)a.k) / n;
    }
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        const int e = expert_of<V>(i, lane);
        ga[i] = a.dloss && e < E ? c * (float)a.counts[e] : 0.f;
    }
    for (int64_t t = (int64_t)blockIdx.x * WARPS + warp; t < a.T; t += (int64_t)gridDim.x * WARPS) {
        const T* row = static_cast<const T*>(a.logits) + t * a.ld;
        T* out = static_cast<T*>(a.dlogits) + t * a.ldd;
        // the softmax again from the row's maximum: exp(logit - lse) would lose what lse has lost beside a large logit
        float p[NE], m = -INFINITY, sum = 0.f, u = 0.f;
        load_logits<T, NE, V>(row, E, lane, p);
        const bool routed = a.lse[t] > -INFINITY;
        int id = -1;
        float w = 0.f, wdw = 0.f;
        if (a.dw && lane < a.k) {
            id = a.ids[t * a.k + lane];
            w = a.w[t * a.k + lane];
            wdw = w * a.dw[t * a.k + lane];
            if (id < 0 || id >= E || !routed) {
                id = -1;
                w = wdw = 0.f;
            }
        }
#pragma unroll
        for (int i = 0; i < NE; ++i) m = fmaxf(m, p[i]);
        m = warp_max(m);
        if (!routed) m = 0.f;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            p[i] = __expf(p[i] - m);
            sum += p[i];
        }
        const float inv = routed ? 1.f / warp_sum(sum) : 0.f;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            p[i] = routed ? p[i] * inv : 0.f;
            u = fmaf(p[i], ga[i], u);
        }
        const float s = a.dw ? warp_sum(wdw) : 0.f;
        u = warp_sum(u);
        if (a.renorm) wdw -= w * (s / a.scale);
        else u += s;
        if (id >= 0) extra[id] = wdw;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < NE; i += V) {
            const int e = expert_of<V>(i, lane);
            struct alignas(sizeof(T) * V) Pack { T x[V]; } o;
#pragma unroll
            for (int j = 0; j < V; ++j) o.x[j] = row::from_f32<T>(fmaf(p[i + j], ga[i + j] - u, extra[e + j]));
            if (e < E) *reinterpret_cast<Pack*>(out + e) = o;
        }
        __syncwarp();
        if (id >= 0) extra[id] = 0.f;
        __syncwarp();
    }
}

// At most this many CTAs: 32 warps an SM.
inline int ctas(int64_t T) {
    const int64_t n = (T + WARPS - 1) / WARPS, most = row::kSMs * 2;
    return (int)(n < most ? n : most);
}

template <auto Kernel>
inline int launch(const Args& a, size_t smem, cudaStream_t st) {
    if (smem > 48 * 1024) {
        const int rc = row::allow_smem<Kernel>(((WARPS + 1) * MAX_E + 1) * 4);
        if (rc != QMOE_OK) return rc;
    }
    return launch_pdl(Kernel, ctas(a.T), WARPS * 32, smem, st, a);
}
template <bool BWD, typename T, int NE, int V>
inline int start(const Args& a, cudaStream_t st) {
    if constexpr (BWD) {
        return launch<route_bwd_kernel<T, NE, V>>(a, (size_t)WARPS * NE * 32 * 4, st);
    } else {
        const size_t smem = a.part_p ? ((size_t)WARPS * a.E + a.E + 1) * 4 : 0;
        if constexpr (sizeof(T) == 2)
            if (!a.bias) return launch<route_kernel<T, NE, V, true>>(a, smem, st);
        return launch<route_kernel<T, NE, V, false>>(a, smem, st);
    }
}
// The widest loads, up to 16 bytes, that the rows allow: else one value at a time.
template <bool BWD, typename T, int NE>
inline int by_rows(const Args& a, cudaStream_t st) {
    constexpr int most = 16 / sizeof(T), V = NE < most ? NE : most;
    const uintptr_t bytes = V * sizeof(T);
    const bool fits = a.E % V == 0 && reinterpret_cast<uintptr_t>(a.logits) % bytes == 0 && a.ld % V == 0 &&
                      (BWD || !a.bias || reinterpret_cast<uintptr_t>(a.bias) % (V < 4 ? V * 4 : 16) == 0) &&
                      (!BWD || (reinterpret_cast<uintptr_t>(a.dlogits) % bytes == 0 && a.ldd % V == 0));
    return fits ? start<BWD, T, NE, V>(a, st) : start<BWD, T, NE, 1>(a, st);
}
template <bool BWD, typename T>
inline int by_experts(const Args& a, cudaStream_t st) {
    if (a.E <= 32) return by_rows<BWD, T, 1>(a, st);
    if (a.E <= 64) return by_rows<BWD, T, 2>(a, st);
    if (a.E <= 128) return by_rows<BWD, T, 4>(a, st);
    if (a.E <= 256) return by_rows<BWD, T, 8>(a, st);
    if (a.E <= 512) return by_rows<BWD, T, 16>(a, st);
    return by_rows<BWD, T, 32>(a, st);
}
template <bool BWD>
inline int run(int dtype, const Args& a, cudaStream_t st) {
    if (dtype == QMOE_F32) return by_experts<BWD, float>(a, st);
    if (dtype == QMOE_BF16) return by_experts<BWD, __nv_bfloat16>(a, st);
    return by_experts<BWD, __half>(a, st);
}

// The workspace: the CTAs' sums of p, their counts, the parts of the loss, and the arrivals.
inline size_t ws_words(int64_t T, int E) { return (size_t)ctas(T) * (2 * (size_t)E + 1) + 32 + 1; }

inline int check(int64_t T, int E, int k, int dtype, int64_t ld, float scale) {
    if (T < 0 || E <= 0 || k <= 0 || k > E || !row::dtype_ok(dtype) || ld < E || !(scale > 0.f && scale < INFINITY))
        return QMOE_ERR_ARG;
    if (E > MAX_E || k > MAX_K || T * k >= (1ll << 31)) return QMOE_ERR_UNSUPPORTED;
    return QMOE_OK;
}

}  // namespace route
}  // namespace qmoe

using namespace qmoe;

extern "C" size_t qmoe_route_workspace_bytes(int64_t T, int E) {
    if (T < 0 || E <= 0 || E > route::MAX_E) return 0;
    return (route::ws_words(T, E) * 4 + 255) / 256 * 256;
}

extern "C" int qmoe_route_topk(int64_t T, int E, int k, int dtype, const void* logits, int64_t ld, const float* bias,
                               const uint8_t* mask, int renorm, float scale, int32_t* ids, float* w, float* lse,
                               float coef, int32_t* counts, float* probs, float* loss, void* ws, size_t ws_bytes,
                               qmoe_stream_t stream) {
    const int rc = route::check(T, E, k, dtype, ld, scale);
    if (rc != QMOE_OK) return rc;
    const bool stats = counts || probs || loss;
    if (stats && (!counts || !probs || !loss || !ws || (reinterpret_cast<uintptr_t>(ws) & 255u) ||
                  ws_bytes < qmoe_route_workspace_bytes(T, E) || !row::type_aligned(counts, 4) ||
                  !row::type_aligned(probs, 4) || !row::type_aligned(loss, 4)))
        return QMOE_ERR_ARG;
    if (T > 0 && (!logits || !ids || !w || !row::type_aligned(logits, row::dtype_size(dtype)) ||
                  !row::type_aligned(ids, 4) || !row::type_aligned(w, 4) || !row::type_aligned(lse, 4) ||
                  !row::type_aligned(bias, 4)))
        return QMOE_ERR_ARG;
    route::Args a = {};
    a.T = T;
    a.E = E;
    a.k = k;
    a.logits = logits;
    a.ld = ld;
    a.bias = bias;
    a.mask = mask;
    a.renorm = renorm;
    a.scale = scale;
    a.ids = ids;
    a.w = w;
    a.lse = lse;
    const int parts = route::ctas(T);
    route::StatArgs s = {};
    if (stats) {
        a.part_p = static_cast<float*>(ws);
        a.part_c = reinterpret_cast<int32_t*>(a.part_p + (size_t)parts * E);
        float* const part_loss = reinterpret_cast<float*>(a.part_c + (size_t)parts * (E + 1));
        a.arrived = reinterpret_cast<int32_t*>(part_loss + 32);
        a.coef = coef;
        a.counts_out = counts;
        a.probs = probs;
        a.loss = loss;
        s = {parts, E, k, a.part_p, a.part_c, part_loss, a.arrived, coef, counts, probs, loss};
        if (T == 0 && cudaMemsetAsync(a.arrived, 0, 4, (cudaStream_t)stream) != cudaSuccess) return QMOE_ERR_CUDA;
    }
    if (T > 0) {
        const int started = route::run<false>(dtype, a, (cudaStream_t)stream);
        if (started != QMOE_OK) return started;
    }
    if (!stats || parts == 1) return QMOE_OK;
    return launch_pdl(route::route_stats_kernel, ceil_div(E, 32), 1024, 0, (cudaStream_t)stream, s);
}

extern "C" int qmoe_route_topk_backward(int64_t T, int E, int k, int dtype, const void* logits, int64_t ld,
                                        const int32_t* ids, const float* w, const float* lse, int renorm, float scale,
                                        const float* dw, float coef, const int32_t* counts, const float* dloss,
                                        void* dlogits, int64_t ldd, qmoe_stream_t stream) {
    const int rc = route::check(T, E, k, dtype, ld, scale);
    if (rc != QMOE_OK) return rc;
    if (ldd < E || (!dw && !dloss)) return QMOE_ERR_ARG;
    if (T == 0) return QMOE_OK;
    const int size = row::dtype_size(dtype);
    if (!logits || !lse || !dlogits || (dw && (!ids || !w)) || (dloss && !counts)) return QMOE_ERR_ARG;
    if (!row::type_aligned(logits, size) || !row::type_aligned(dlogits, size) || !row::type_aligned(ids, 4) ||
        !row::type_aligned(w, 4) || !row::type_aligned(lse, 4) || !row::type_aligned(dw, 4) ||
        !row::type_aligned(counts, 4) || !row::type_aligned(dloss, 4))
        return QMOE_ERR_ARG;
    route::Args a = {};
    a.T = T;
    a.E = E;
    a.k = k;
    a.logits = logits;
    a.ld = ld;
    a.renorm = renorm;
    a.scale = scale;
    a.ids = const_cast<int32_t*>(ids);
    a.w = const_cast<float*>(w);
    a.lse = const_cast<float*>(lse);
    a.dw = dw;
    a.coef = coef;
    a.counts = counts;
    a.dloss = dloss;
    a.dlogits = dlogits;
    a.ldd = ldd;
    return route::run<true>(dtype, a, (cudaStream_t)stream);
}
