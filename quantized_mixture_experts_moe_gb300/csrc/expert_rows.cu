// What stands between and behind the experts' products when they are trained:
// SwiGLU and its gradient (qmoe_swiglu, qmoe_swiglu_backward), the weighted sum
// over a token's experts and its gradient (qmoe_weighted_sum,
// qmoe_weighted_sum_backward).  Every value is read once and written once; all
// of them are bound by HBM (SwiGLU's gradient with h, 65536 x 1408 bf16: 156 us, 7.1
// TB/s; the weighted sum's, 8192 x 10 rows of 4096: 200 us, 6.9 TB/s), or by the
// launch where there are few rows (1.3 and 2.8 us on the device).
#include "row_ops.cuh"

namespace qmoe {
namespace er {

// s(v) = 1 / (1 + exp(-v)), as e / (1 + e) with e = exp(v) for v < 0: a divisor is
// never above 2 (the fast division gives 0 for divisors above 2^126, which is v below
// -87.3).  For 16-bit values the fast exponential: its error is up to 2 + 1.2 |v| ulp,
// 2^-16 relative where s is least, against 2^-12 of the rounding that follows.
template <typename T>
__device__ __forceinline__ float sigmoid(float v) {
    if constexpr (sizeof(T) == 4) {
        const float e = expf(-fabsf(v));
        return (v >= 0.f ? 1.0f : e) / (1.0f + e);
    } else {
        const float e = __expf(-fabsf(v));
        return __fdividef(v >= 0.f ? 1.0f : e, 1.0f + e);
    }
}
template <typename T>
__device__ __forceinline__ float swiglu_of(float g, float u) { return g * sigmoid<T>(g) * u; }
// The gradients in place of g and u, and h.  The factors that are at most 1.1 come
// before dh: dh u alone may leave fp32 where dg does not.
template <typename T>
__device__ __forceinline__ float swiglu_grad(float dh, float& g, float& u) {
    const float s = sigmoid<T>(g), gs = g * s, h = gs * u, dg = u * (s * (1.0f + g * (1.0f - s))) * dh;
    u = dh * gs;
    g = dg;
    return h;
}

// One value, or two that lie in one aligned word (16-bit types).
template <typename T, int VEC> struct Pair {
    T v;
    __device__ __forceinline__ void load(const T* p) { v = *p; }
    __device__ __forceinline__ void widen(float* f) const { f[0] = row::to_f32(v); }
    static __device__ __forceinline__ void store(T* p, const float* f) { *p = row::from_f32<T>(f[0]); }
};
template <typename T> struct Pair<T, 2> {
    uint32_t v;
    __device__ __forceinline__ void load(const T* p) { v = *reinterpret_cast<const uint32_t*>(p); }
    __device__ __forceinline__ void widen(float* f) const {
        const float2 x = row::unpack2(v, T{});
        f[0] = x.x;
        f[1] = x.y;
    }
    static __device__ __forceinline__ void store(T* p, const float* f) { *reinterpret_cast<uint32_t*>(p) = row::pack2(f[0], f[1], T{}); }
};

// A thread takes VEC columns of a row.
template <typename T, int VEC>
__global__ void __launch_bounds__(256)
swiglu_kernel(int64_t total, uint32_t per_row, int64_t I, const T* gu, int64_t ldgu, T* h, int64_t ldh) {
    pdl_wait();
    pdl_trigger();
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t r = total < (1ll << 32) ? (uint32_t)i / per_row : i / per_row;
        const int64_t c = (i - r * per_row) * VEC;
        float g[VEC], u[VEC];
        row::Raw<T, VEC> a, b;
        row::load_raw<VEC>(a, gu + r * ldgu + c);
        row::load_raw<VEC>(b, gu + r * ldgu + I + c);
        row::widen<VEC>(a, g);
        row::widen<VEC>(b, u);
#pragma unroll
        for (int j = 0; j < VEC; ++j) g[j] = swiglu_of<T>(g[j], u[j]);
        row::store<VEC>(h + r * ldh + c, g);
    }
}

template <typename T, int VEC>
__global__ void __launch_bounds__(256)
swiglu_backward_kernel(int64_t total, uint32_t per_row, int64_t I, const T* dh, int64_t lddh, const T* gu, int64_t ldgu,
                       T* dgu, int64_t lddgu, T* h, int64_t ldh) {
    pdl_wait();
    pdl_trigger();
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t r = total < (1ll << 32) ? (uint32_t)i / per_row : i / per_row;
        const int64_t c = (i - r * per_row) * VEC;
        float g[VEC], u[VEC], d[VEC];
        row::Raw<T, VEC> a, b, e;
        row::load_raw<VEC>(a, gu + r * ldgu + c);
        row::load_raw<VEC>(b, gu + r * ldgu + I + c);
        row::load_raw<VEC>(e, dh + r * lddh + c);
        row::widen<VEC>(a, g);
        row::widen<VEC>(b, u);
        row::widen<VEC>(e, d);
        float o[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) o[j] = swiglu_grad<T>(d[j], g[j], u[j]);
        row::store<VEC>(dgu + r * lddgu + c, g);
        row::store<VEC>(dgu + r * lddgu + I + c, u);
        if (h) row::store<VEC>(h + r * ldh + c, o);
    }
}

// Rows off the 16-byte boundaries: a warp takes a row, a lane VEC neighbouring
// columns (2 where all rows and halves start on whole pairs), U times: 10829 x 966
// bf16 44 us with a thread a value.
template <typename T, int VEC>
__global__ void __launch_bounds__(256) swiglu_odd_kernel(int64_t rows, int64_t I, const T* gu, int64_t ldgu, T* h, int64_t ldh) {
    pdl_wait();
    pdl_trigger();
    constexpr int U = 4;
    for (int64_t r = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); r < rows; r += (int64_t)gridDim.x * 8)
        for (int64_t c = (threadIdx.x & 31) * VEC; c < I; c += 32 * VEC * U) {
            Pair<T, VEC> a[U], b[U];
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (c + i * 32 * VEC < I) {
                    a[i].load(gu + r * ldgu + c + i * 32 * VEC);
                    b[i].load(gu + r * ldgu + I + c + i * 32 * VEC);
                }
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (c + i * 32 * VEC < I) {
                    float g[VEC], u[VEC];
                    a[i].widen(g);
                    b[i].widen(u);
#pragma unroll
                    for (int j = 0; j < VEC; ++j) g[j] = swiglu_of<T>(g[j], u[j]);
                    Pair<T, VEC>::store(h + r * ldh + c + i * 32 * VEC, g);
                }
        }
}
template <typename T, int VEC>
__global__ void __launch_bounds__(256)
swiglu_backward_odd_kernel(int64_t rows, int64_t I, const T* dh, int64_t lddh, const T* gu, int64_t ldgu, T* dgu, int64_t lddgu, T* h,
                           int64_t ldh) {
    pdl_wait();
    pdl_trigger();
    constexpr int U = 4;
    for (int64_t r = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); r < rows; r += (int64_t)gridDim.x * 8)
        for (int64_t c = (threadIdx.x & 31) * VEC; c < I; c += 32 * VEC * U) {
            Pair<T, VEC> a[U], b[U], e[U];
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (c + i * 32 * VEC < I) {
                    a[i].load(gu + r * ldgu + c + i * 32 * VEC);
                    b[i].load(gu + r * ldgu + I + c + i * 32 * VEC);
                    e[i].load(dh + r * lddh + c + i * 32 * VEC);
                }
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (c + i * 32 * VEC < I) {
                    float g[VEC], u[VEC], d[VEC], o[VEC];
                    a[i].widen(g);
                    b[i].widen(u);
                    e[i].widen(d);
#pragma unroll
                    for (int j = 0; j < VEC; ++j) o[j] = swiglu_grad<T>(d[j], g[j], u[j]);
                    Pair<T, VEC>::store(dgu + r * lddgu + c + i * 32 * VEC, g);
                    Pair<T, VEC>::store(dgu + r * lddgu + I + c + i * 32 * VEC, u);
                    if (h) Pair<T, VEC>::store(h + r * ldh + c + i * 32 * VEC, o);
                }
        }
}

// A thread takes VEC columns of a token and its k rows in turn.
template <typename T, int VEC>
__global__ void __launch_bounds__(256)
weighted_sum_kernel(int64_t total, uint32_t per_row, int k, int64_t P, const T* y, int64_t ldy, const float* w,
                    const int32_t* slot, T* out, int64_t ldo) {
    pdl_wait();
    pdl_trigger();
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t t = total < (1ll << 32) ? (uint32_t)i / per_row : i / per_row;
        const int64_t c = (i - t * per_row) * VEC;
        float sum[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) sum[j] = 0.f;
        for (int j0 = 0; j0 < k; j0 += 4) {
            row::Raw<T, VEC> raw[4];
            float f[4];
            bool on[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t s = j0 + j < k ? slot[t * k + j0 + j] : -1;
                on[j] = s >= 0 && s < P;
                if (on[j]) {
                    f[j] = w ? w[t * k + j0 + j] : 1.f;
                    row::load_raw<VEC>(raw[j], y + s * ldy + c);
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (on[j]) {
                    float v[VEC];
                    row::widen<VEC>(raw[j], v);
#pragma unroll
                    for (int x = 0; x < VEC; ++x) sum[x] = fmaf(f[j], v[x], sum[x]);
                }
        }
        row::store<VEC>(out + t * ldo + c, sum);
    }
}

// A warp takes a pair: its row of y and of dy, and its token's row of dout, which
// the warps of the token's other pairs, next to it, read too.
template <typename T, int VEC>
__global__ void __launch_bounds__(256)
weighted_sum_backward_kernel(int64_t pairs, int k, int64_t P, int64_t H, const T* dout, int64_t lddout, const T* y,
                             int64_t ldy, const float* w, const int32_t* slot, const int32_t* routed, T* dy,
                             int64_t lddy, float* dw) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int64_t p = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (p >= pairs) return;
    const float zero[VEC] = {};
    int64_t first = *routed;
    if (first < 0) first = 0;
    for (int64_t r = first + p; r < P; r += pairs)
        for (int64_t c = lane * VEC; c < H; c += 32 * VEC) row::store<VEC>(dy + r * lddy + c, zero);
    const int64_t s = slot[p];
    if (s < 0 || s >= P) {
        if (dw && lane == 0) dw[p] = 0.f;
        return;
    }
    const float f = w ? w[p] : 1.f;
    const T* d = dout + p / k * lddout;
    const T* a = y + s * ldy;
    T* o = dy + s * lddy;
    float dot = 0.f;
    constexpr int U = 4;
    for (int64_t c0 = lane * VEC; c0 < H; c0 += 32 * VEC * U) {
        row::Raw<T, VEC> rd[U], ra[U];
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (c0 + i * 32 * VEC < H) {
                row::load_raw<VEC>(rd[i], d + c0 + i * 32 * VEC);
                if (dw) row::load_raw<VEC>(ra[i], a + c0 + i * 32 * VEC);
            }
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (c0 + i * 32 * VEC < H) {
                float v[VEC], q[VEC];
                row::widen<VEC>(rd[i], v);
                if (dw) {
                    row::widen<VEC>(ra[i], q);
#pragma unroll
                    for (int j = 0; j < VEC; ++j) dot = fmaf(v[j], q[j], dot);
                }
#pragma unroll
                for (int j = 0; j < VEC; ++j) v[j] *= f;
                row::store<VEC>(o + c0 + i * 32 * VEC, v);
            }
    }
    if (dw) {
        dot = row::warp_sum(dot);
        if (lane == 0) dw[p] = dot;
    }
}

// ------------------------------------------------------------------ host side

// Rows of 16-byte pieces: 8 values of 16 bits, 4 of 32 (which the loads of 8 take as two pieces).
inline bool wide(const void* p, int64_t ld, int size) { return !p || (aligned16(p) && ld * size % 16 == 0); }
inline bool mat_ok(const void* p, int64_t ld, int64_t cols, int size) {
    return p && ld >= cols && row::type_aligned(p, size);
}
// Rows whose pairs of 16-bit values lie in whole words.
inline bool paired(const void* p, int64_t ld) { return !p || ((reinterpret_cast<uintptr_t>(p) & 3) == 0 && ld % 2 == 0); }
inline unsigned rows_grid(int64_t rows) { return (unsigned)((rows + 7) / 8 < 32 * row::kSMs ? (rows + 7) / 8 : 32 * row::kSMs); }
inline unsigned grid_of(int64_t total) {
    const int64_t g = (total + 255) / 256;
    return (unsigned)(g < (1 << 30) ? g : 1 << 30);
}

template <typename F>
static int by_type(int dtype, F f) {
    if (dtype == QMOE_F32) return f(float{});
    if (dtype == QMOE_BF16) return f(__nv_bfloat16{});
    return f(__half{});
}

constexpr int64_t kMost = 1ll << 31;

}  // namespace er
}  // namespace qmoe

using namespace qmoe;

extern "C" int qmoe_swiglu(int64_t rows, int64_t I, int dtype, const void* gu, int64_t ldgu, void* h, int64_t ldh,
                           qmoe_stream_t stream) {
    if (rows < 0 || I <= 0 || !row::dtype_ok(dtype)) return QMOE_ERR_ARG;
    if (rows >= er::kMost || I >= er::kMost / 4) return QMOE_ERR_UNSUPPORTED;
    if (rows == 0) return QMOE_OK;
    const int size = row::dtype_size(dtype);
    if (!er::mat_ok(gu, ldgu, 2 * I, size) || !er::mat_ok(h, ldh, I, size)) return QMOE_ERR_ARG;
    return er::by_type(dtype, [&](auto z) {
        using T = decltype(z);
        const bool wide = I % 8 == 0 && er::wide(gu, ldgu, size) && er::wide(h, ldh, size);
        const T* const gt = static_cast<const T*>(gu);
        T* const ht = static_cast<T*>(h);
        cudaStream_t st = (cudaStream_t)stream;
        if (wide)
            return launch_pdl(er::swiglu_kernel<T, 8>, dim3(er::grid_of(rows * (I / 8))), dim3(256), 0, st, rows * (I / 8),
                              (uint32_t)(I / 8), I, gt, ldgu, ht, ldh);
        if constexpr (sizeof(T) == 2)
            if (I % 2 == 0 && er::paired(gu, ldgu) && er::paired(h, ldh))
                return launch_pdl(er::swiglu_odd_kernel<T, 2>, dim3(er::rows_grid(rows)), dim3(256), 0, st, rows, I, gt, ldgu, ht, ldh);
        return launch_pdl(er::swiglu_odd_kernel<T, 1>, dim3(er::rows_grid(rows)), dim3(256), 0, st, rows, I, gt, ldgu, ht, ldh);
    });
}

extern "C" int qmoe_swiglu_backward(int64_t rows, int64_t I, int dtype, const void* dh, int64_t lddh, const void* gu,
                                    int64_t ldgu, void* dgu, int64_t lddgu, void* h, int64_t ldh, qmoe_stream_t stream) {
    if (rows < 0 || I <= 0 || !row::dtype_ok(dtype)) return QMOE_ERR_ARG;
    if (rows >= er::kMost || I >= er::kMost / 4) return QMOE_ERR_UNSUPPORTED;
    if (rows == 0) return QMOE_OK;
    const int size = row::dtype_size(dtype);
    if (!er::mat_ok(dh, lddh, I, size) || !er::mat_ok(gu, ldgu, 2 * I, size) || !er::mat_ok(dgu, lddgu, 2 * I, size) ||
        (h && !er::mat_ok(h, ldh, I, size)))
        return QMOE_ERR_ARG;
    return er::by_type(dtype, [&](auto z) {
        using T = decltype(z);
        const bool wide = I % 8 == 0 && er::wide(dh, lddh, size) && er::wide(gu, ldgu, size) && er::wide(dgu, lddgu, size) &&
                          er::wide(h, ldh, size);
        const T *const dt = static_cast<const T*>(dh), *const gt = static_cast<const T*>(gu);
        T *const ot = static_cast<T*>(dgu), *const ht = static_cast<T*>(h);
        cudaStream_t st = (cudaStream_t)stream;
        if (wide)
            return launch_pdl(er::swiglu_backward_kernel<T, 8>, dim3(er::grid_of(rows * (I / 8))), dim3(256), 0, st, rows * (I / 8),
                              (uint32_t)(I / 8), I, dt, lddh, gt, ldgu, ot, lddgu, ht, ldh);
        if constexpr (sizeof(T) == 2)
            if (I % 2 == 0 && er::paired(dh, lddh) && er::paired(gu, ldgu) && er::paired(dgu, lddgu) && er::paired(h, ldh))
                return launch_pdl(er::swiglu_backward_odd_kernel<T, 2>, dim3(er::rows_grid(rows)), dim3(256), 0, st, rows, I, dt, lddh, gt,
                                  ldgu, ot, lddgu, ht, ldh);
        return launch_pdl(er::swiglu_backward_odd_kernel<T, 1>, dim3(er::rows_grid(rows)), dim3(256), 0, st, rows, I, dt, lddh, gt, ldgu,
                          ot, lddgu, ht, ldh);
    });
}

static int sum_sizes(int64_t T, int k, int64_t P, int64_t H, int dtype) {
    if (T < 0 || k <= 0 || P < 0 || H <= 0 || !row::dtype_ok(dtype)) return QMOE_ERR_ARG;
    if (H > (1 << 30) || P >= er::kMost || T >= er::kMost || T * k >= er::kMost) return QMOE_ERR_UNSUPPORTED;
    return QMOE_OK;
}

extern "C" int qmoe_weighted_sum(int64_t T, int k, int64_t P, int64_t H, int dtype, const void* y, int64_t ldy,
                                 const float* w, const int32_t* pair_slot, void* out, int64_t ldo, qmoe_stream_t stream) {
    const int rc = sum_sizes(T, k, P, H, dtype);
    if (rc != QMOE_OK) return rc;
    if (T == 0) return QMOE_OK;
    const int size = row::dtype_size(dtype);
    if ((P > 0 && !er::mat_ok(y, ldy, H, size)) || !er::mat_ok(out, ldo, H, size) || !pair_slot ||
        !row::type_aligned(pair_slot, 4) || !row::type_aligned(w, 4))
        return QMOE_ERR_ARG;
    return er::by_type(dtype, [&](auto z) {
        using T_ = decltype(z);
        const bool wide = H % 8 == 0 && er::wide(y, ldy, size) && er::wide(out, ldo, size);
        const int64_t per = wide ? H / 8 : H;
        return launch_pdl(wide ? er::weighted_sum_kernel<T_, 8> : er::weighted_sum_kernel<T_, 1>, dim3(er::grid_of(T * per)),
                          dim3(256), 0, (cudaStream_t)stream, T * per, (uint32_t)per, k, P, static_cast<const T_*>(y), ldy,
                          w, pair_slot, static_cast<T_*>(out), ldo);
    });
}

extern "C" int qmoe_weighted_sum_backward(int64_t T, int k, int64_t P, int64_t H, int dtype, const void* dout,
                                          int64_t lddout, const void* y, int64_t ldy, const float* w,
                                          const int32_t* pair_slot, const int32_t* routed, void* dy, int64_t lddy,
                                          float* dw, qmoe_stream_t stream) {
    const int rc = sum_sizes(T, k, P, H, dtype);
    if (rc != QMOE_OK) return rc;
    const int size = row::dtype_size(dtype);
    if (T == 0) {
        if (P == 0) return QMOE_OK;
        if (!er::mat_ok(dy, lddy, H, size)) return QMOE_ERR_ARG;
        return cudaMemset2DAsync(dy, (size_t)lddy * size, 0, (size_t)H * size, (size_t)P, (cudaStream_t)stream) == cudaSuccess
                   ? QMOE_OK
                   : QMOE_ERR_LAUNCH;
    }
    if (!er::mat_ok(dout, lddout, H, size) || (P > 0 && !er::mat_ok(dy, lddy, H, size)) || !pair_slot ||
        !row::type_aligned(pair_slot, 4) || !row::type_aligned(w, 4) || !routed || !row::type_aligned(routed, 4) ||
        (P > 0 && !y != !dw) || (y && !er::mat_ok(y, ldy, H, size)) || !row::type_aligned(dw, 4))
        return QMOE_ERR_ARG;
    return er::by_type(dtype, [&](auto z) {
        using T_ = decltype(z);
        const bool wide = H % 8 == 0 && er::wide(dout, lddout, size) && er::wide(y, ldy, size) && er::wide(dy, lddy, size);
        const int64_t pairs = T * k;
        return launch_pdl(wide ? er::weighted_sum_backward_kernel<T_, 8> : er::weighted_sum_backward_kernel<T_, 1>,
                          dim3((unsigned)((pairs + 7) / 8)), dim3(256), 0, (cudaStream_t)stream, pairs, k, P, H,
                          static_cast<const T_*>(dout), lddout, static_cast<const T_*>(y), ldy, w, pair_slot, routed,
                          static_cast<T_*>(dy), lddy, dw);
    });
}
