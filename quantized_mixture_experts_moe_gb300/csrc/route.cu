// Top-k routing with the balance loss and the per-expert counts
// (qmoe_route_topk), and its gradient (qmoe_route_topk_backward).
//
//   p = softmax(logit),  ids = the k experts of largest logit + bias,
//   counts_e = pairs of expert e,  P_e = mean_t p_te,
//   loss = coef E sum_e counts_e / (k n) P_e   (n routed tokens)
//   dlogit = p (a - sum p a - s) + [selected] w_j (dw_j - r),
//   a_e = dloss coef E counts_e / (k n^2)
//
// A warp takes a token at a time, its logits spread over the lanes' registers,
// so a row is read once for the softmax, the selection and the statistics.
// Selection is k rounds of a warp-wide maximum over order-preserving integer
// keys, the lowest expert first among equal keys.  That, not the 2 E bytes of a
// row, is the bound: the rounds are instruction issue and the latency of
// redux.  Probabilities are summed per lane over a warp's tokens, then over a
// CTA's warps, then over CTAs, in a fixed order.
#include "row_ops.cuh"

namespace qmoe {
namespace route {

constexpr int MAX_E = 1024, MAX_K = 32, WARPS = 8;
constexpr uint32_t KEY_NONE = 0x007FFFFFu;  // key of -inf: that expert is not available

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
    // gradient
    const float* dw;
    float coef;
    const int32_t* counts;
    const float* dloss;
    void* dlogits;
    int64_t ldd;
};

// NaN counts as -inf (an invalid logit selects nothing), +inf as the largest
// finite value.
__device__ __forceinline__ float clean(float v) { return v > -INFINITY ? fminf(v, 3.402823466e38f) : -INFINITY; }

// Larger floats have larger keys; -0 and +0 have the same.
__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t u = __float_as_uint(v == 0.f ? 0.f : v);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}

template <typename T, int NE>
__global__ void __launch_bounds__(WARPS * 32)
route_kernel(const Args a) {
    extern __shared__ float smem[];  // statistics: [WARPS][E] sums of p, then [E + 1] counts
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = a.E;
    int* const count = reinterpret_cast<int*>(smem + WARPS * E);
    const bool stats = a.part_p != nullptr;
    pdl_sync();
    if (stats) {
        for (int i = threadIdx.x; i <= E; i += blockDim.x) count[i] = 0;
        __syncthreads();
    }
    float psum[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) psum[i] = 0.f;
    for (int64_t t = (int64_t)blockIdx.x * WARPS + warp; t < a.T; t += (int64_t)gridDim.x * WARPS) {
        const T* row = static_cast<const T*>(a.logits) + t * a.ld;
        float v[NE], m = -INFINITY;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const int e = i * 32 + lane;
            v[i] = e < E ? clean(row::to_f32(row[e])) : -INFINITY;
            m = fmaxf(m, v[i]);
        }
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
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const int e = i * 32 + lane;
            key[i] = e < E ? key_of(a.bias ? clean(v[i] + a.bias[e]) : v[i]) : 0u;
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
        int mine = -1;  // lane j: the expert of rank j
        for (int j = 0; j < a.k; ++j) {
            uint32_t best = key[0];
            int at = 0;
#pragma unroll
            for (int i = 1; i < NE; ++i)
                if (key[i] > best) {
                    best = key[i];
                    at = i;
                }
            const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, best);
            if (top <= KEY_NONE) break;
            const int e = at * 32 + lane;
            const int win = (int)__reduce_min_sync(0xFFFFFFFFu, best == top ? (unsigned)e : 0x7FFFFFFFu);
            if (lane == j) mine = win;
            if (win == e) {
#pragma unroll
                for (int i = 0; i < NE; ++i)
                    if (i == at) key[i] = 0u;
            }
        }
        // the chosen logits again (they are in L1), so that no register is indexed by a variable
        const float l = mine >= 0 ? clean(row::to_f32(row[mine])) : -INFINITY;
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
    for (int i = 0; i < NE; ++i)
        if (i * 32 + lane < E) smem[warp * E + i * 32 + lane] = psum[i];
    __syncthreads();
    for (int e = threadIdx.x; e <= E; e += blockDim.x) {
        a.part_c[(int64_t)blockIdx.x * (E + 1) + e] = count[e];
        if (e == E) break;
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < WARPS; ++i) s += smem[i * E + e];
        a.part_p[(int64_t)blockIdx.x * E + e] = s;
    }
}

// Sums the CTAs' statistics: counts[E + 1], probs[E] and the loss.  One CTA.
struct StatArgs {
    int parts, E, k;
    const float* part_p;
    const int32_t* part_c;
    float coef;
    int32_t* counts;
    float* probs;
    float* loss;
};
__global__ void __launch_bounds__(1024) route_stats_kernel(const StatArgs a) {
    __shared__ float warp_part[32];
    __shared__ int routed;
    pdl_sync();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = a.E;
    if (warp == 0) {
        int n = 0;
        for (int i = lane; i < a.parts; i += 32) n += a.part_c[(int64_t)i * (E + 1) + E];
        n = __reduce_add_sync(0xFFFFFFFFu, n);
        if (lane == 0) {
            routed = n;
            a.counts[E] = n;
        }
    }
    __syncthreads();
    const float n = (float)(routed > 0 ? routed : 1);
    float loss = 0.f;
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        int c = 0;
        float p = 0.f;
#pragma unroll 8
        for (int i = 0; i < a.parts; ++i) {
            c += a.part_c[(int64_t)i * (E + 1) + e];
            p += a.part_p[(int64_t)i * E + e];
        }
        p /= n;
        a.counts[e] = c;
        a.probs[e] = p;
        loss = fmaf((float)c / (n * (float)a.k), p, loss);
    }
    loss = warp_sum(loss);
    if (lane == 0) warp_part[warp] = loss;
    __syncthreads();
    if (warp == 0) {
        loss = warp_sum(warp_part[lane]);
        if (lane == 0) a.loss[0] = a.coef * (float)E * loss;
    }
}

template <typename T, int NE>
__global__ void __launch_bounds__(WARPS * 32)
route_bwd_kernel(const Args a) {
    extern __shared__ float smem[];  // [WARPS][E]: what the selected experts get besides
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = a.E;
    float* const extra = smem + warp * E;
    pdl_sync();
    for (int e = lane; e < E; e += 32) extra[e] = 0.f;
    __syncwarp();
    float ga[NE];
    float c = 0.f;
    if (a.dloss) {
        const float n = (float)max(a.counts[E], 1);
        c = a.dloss[0] * a.coef * (float)E / (n * (float)a.k) / n;
    }
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        const int e = i * 32 + lane;
        ga[i] = a.dloss && e < E ? c * (float)a.counts[e] : 0.f;
    }
    for (int64_t t = (int64_t)blockIdx.x * WARPS + warp; t < a.T; t += (int64_t)gridDim.x * WARPS) {
        const T* row = static_cast<const T*>(a.logits) + t * a.ld;
        T* out = static_cast<T*>(a.dlogits) + t * a.ldd;
        if (!(a.lse[t] > -INFINITY)) {  // routed nowhere
            for (int e = lane; e < E; e += 32) out[e] = row::from_f32<T>(0.f);
            continue;
        }
        // the softmax again from the row's maximum: exp(logit - lse) would lose what lse has lost beside a large logit
        float p[NE], m = -INFINITY, sum = 0.f, u = 0.f;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const int e = i * 32 + lane;
            p[i] = e < E ? clean(row::to_f32(row[e])) : -INFINITY;
            m = fmaxf(m, p[i]);
        }
        m = warp_max(m);
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            p[i] = __expf(p[i] - m);
            sum += p[i];
        }
        const float inv = 1.f / warp_sum(sum);
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            p[i] *= inv;
            u = fmaf(p[i], ga[i], u);
        }
        int id = -1;
        float w = 0.f, wdw = 0.f;
        if (a.dw && lane < a.k) {
            id = a.ids[t * a.k + lane];
            if (id >= E) id = -1;
            if (id >= 0) {
                w = a.w[t * a.k + lane];
                wdw = w * a.dw[t * a.k + lane];
            }
        }
        const float s = a.dw ? warp_sum(wdw) : 0.f;
        u = warp_sum(u);
        if (a.renorm) wdw -= w * (s / a.scale);
        else u += s;
        if (id >= 0) extra[id] = wdw;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const int e = i * 32 + lane;
            if (e < E) out[e] = row::from_f32<T>(fmaf(p[i], ga[i] - u, extra[e]));
        }
        __syncwarp();
        if (id >= 0) extra[id] = 0.f;
        __syncwarp();
    }
}

// At most this many CTAs: 32 warps an SM.
inline int ctas(int64_t T) {
    const int64_t n = (T + WARPS - 1) / WARPS, most = row::kSMs * 4;
    return (int)(n < most ? n : most);
}

template <bool BWD, typename T, int NE>
inline int start(const Args& a, cudaStream_t st) {
    const size_t smem = BWD ? (size_t)WARPS * a.E * 4 : a.part_p ? ((size_t)WARPS * a.E + a.E + 1) * 4 : 0;
    if constexpr (BWD) return launch_pdl(route_bwd_kernel<T, NE>, ctas(a.T), WARPS * 32, smem, st, a);
    else return launch_pdl(route_kernel<T, NE>, ctas(a.T), WARPS * 32, smem, st, a);
}
template <bool BWD, typename T>
inline int by_experts(const Args& a, cudaStream_t st) {
    if (a.E <= 32) return start<BWD, T, 1>(a, st);
    if (a.E <= 64) return start<BWD, T, 2>(a, st);
    if (a.E <= 128) return start<BWD, T, 4>(a, st);
    if (a.E <= 256) return start<BWD, T, 8>(a, st);
    if (a.E <= 512) return start<BWD, T, 16>(a, st);
    return start<BWD, T, 32>(a, st);
}
template <bool BWD>
inline int run(int dtype, const Args& a, cudaStream_t st) {
    if (dtype == QMOE_F32) return by_experts<BWD, float>(a, st);
    if (dtype == QMOE_BF16) return by_experts<BWD, __nv_bfloat16>(a, st);
    return by_experts<BWD, __half>(a, st);
}

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
    const size_t n = (size_t)route::ctas(T > 0 ? T : 1);
    return (n * (2 * (size_t)E + 1) * 4 + 255) / 256 * 256;
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
    if (stats) {
        a.part_p = static_cast<float*>(ws);
        a.part_c = reinterpret_cast<int32_t*>(a.part_p + (size_t)parts * E);
    }
    if (T > 0) {
        const int started = route::run<false>(dtype, a, (cudaStream_t)stream);
        if (started != QMOE_OK) return started;
    }
    if (!stats) return QMOE_OK;
    const route::StatArgs s = {parts, E, k, a.part_p, a.part_c, coef, counts, probs, loss};
    return launch_pdl(route::route_stats_kernel, 1, 1024, 0, (cudaStream_t)stream, s);
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
