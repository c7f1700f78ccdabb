// Shared pieces of the row-wise operators (norms, FP8 quantisation): element
// types, 8-element vector loads and stores, and the sum over the threads that
// share a row.
#pragma once

#include <atomic>

#include "qmoe_common.cuh"

namespace qmoe {
namespace row {

constexpr int kSMs = 152;  // GB300

// Lets a kernel use `bytes` of dynamic shared memory; asked of the runtime once
// for each kernel and device.
template <auto Kernel>
inline int allow_smem(int bytes) {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return QMOE_ERR_CUDA;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_acquire) & bit) return QMOE_OK;
    if (cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
        return QMOE_ERR_CUDA;
    done.fetch_or(bit, std::memory_order_release);
    return QMOE_OK;
}

inline bool dtype_ok(int t) { return t == QMOE_F32 || t == QMOE_BF16 || t == QMOE_F16; }
inline int dtype_size(int t) { return t == QMOE_F32 ? 4 : 2; }
inline bool type_aligned(const void* p, int size) { return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(size - 1)) == 0; }

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// Two values in one 32-bit word, the first in the low half.
__device__ __forceinline__ float2 unpack2(uint32_t u, __nv_bfloat16) {
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
}
__device__ __forceinline__ float2 unpack2(uint32_t u, __half) {
    return __half22float2(*reinterpret_cast<const __half2*>(&u));
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// VEC consecutive values as they lie in memory: loaded early, widened when
// they are used.  VEC = 4 and 8 need an address aligned to their bytes, up to 16.
template <typename T, int VEC> struct Raw { T v; };
template <typename T> struct Raw<T, 8> { uint4 v; };
template <typename T> struct Raw<T, 4> { uint2 v; };
template <> struct Raw<float, 8> { float4 a, b; };
template <> struct Raw<float, 4> { float4 a; };

template <int VEC>
__device__ __forceinline__ void load_raw(Raw<float, VEC>& r, const float* p) {
    if constexpr (VEC == 8) {
        r.a = reinterpret_cast<const float4*>(p)[0];
        r.b = reinterpret_cast<const float4*>(p)[1];
    } else if constexpr (VEC == 4) {
        r.a = reinterpret_cast<const float4*>(p)[0];
    } else {
        r.v = p[0];
    }
}
template <int VEC, typename T>
__device__ __forceinline__ void load_raw(Raw<T, VEC>& r, const T* p) {
    if constexpr (VEC == 8) r.v = *reinterpret_cast<const uint4*>(p);
    else if constexpr (VEC == 4) r.v = *reinterpret_cast<const uint2*>(p);
    else r.v = p[0];
}
template <int VEC>
__device__ __forceinline__ void widen(const Raw<float, VEC>& r, float* v) {
    if constexpr (VEC == 8) {
        v[0] = r.a.x; v[1] = r.a.y; v[2] = r.a.z; v[3] = r.a.w;
        v[4] = r.b.x; v[5] = r.b.y; v[6] = r.b.z; v[7] = r.b.w;
    } else if constexpr (VEC == 4) {
        v[0] = r.a.x; v[1] = r.a.y; v[2] = r.a.z; v[3] = r.a.w;
    } else {
        v[0] = r.v;
    }
}
template <int VEC, typename T>
__device__ __forceinline__ void widen(const Raw<T, VEC>& r, float* v) {
    if constexpr (VEC == 8) {
        const uint32_t u[4] = {r.v.x, r.v.y, r.v.z, r.v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = unpack2(u[i], T{});
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    } else if constexpr (VEC == 4) {
        const float2 f = unpack2(r.v.x, T{}), g = unpack2(r.v.y, T{});
        v[0] = f.x; v[1] = f.y; v[2] = g.x; v[3] = g.y;
    } else {
        v[0] = to_f32(r.v);
    }
}
template <int VEC, typename T>
__device__ __forceinline__ void load(const T* p, float* v) {
    Raw<T, VEC> r;
    load_raw<VEC>(r, p);
    widen<VEC>(r, v);
}
template <int VEC>
__device__ __forceinline__ void store(float* p, const float* v) {
    if constexpr (VEC == 8) {
        reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else if constexpr (VEC == 4) {
        reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    } else {
        p[0] = v[0];
    }
}
template <int VEC, typename T>
__device__ __forceinline__ void store(T* p, const float* v) {
    if constexpr (VEC == 8) {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack2(v[0], v[1], T{}), pack2(v[2], v[3], T{}),
                                                  pack2(v[4], v[5], T{}), pack2(v[6], v[7], T{}));
    } else if constexpr (VEC == 4) {
        *reinterpret_cast<uint2*>(p) = make_uint2(pack2(v[0], v[1], T{}), pack2(v[2], v[3], T{}));
    } else {
        p[0] = from_f32<T>(v[0]);
    }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}
// Sums of a (and of b where TWO) over the threads of a row: the lanes of a warp
// where the row has 32 threads, else the whole CTA (blockDim.x <= 512 threads).
// `buf` is one of the two halves of a 2 x 2 x 16 float array, zeroed before the
// first sum and alternated by the caller, so that one barrier is enough.  The
// order is fixed.
template <bool TWO>
__device__ __forceinline__ float2 row_sums(float a, float b, float (&buf)[2][16]) {
    a = warp_sum(a);
    if (TWO) b = warp_sum(b);
    if (blockDim.x == 32) return make_float2(a, b);
    if ((threadIdx.x & 31) == 0) {
        buf[0][threadIdx.x >> 5] = a;
        if (TWO) buf[1][threadIdx.x >> 5] = b;
    }
    __syncthreads();
    float sum[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < (TWO ? 2 : 1); ++i) {
        const float4* part = reinterpret_cast<const float4*>(buf[i]);
        const float4 p = part[0], q = part[1];
        sum[i] = ((p.x + p.y) + (p.z + p.w)) + ((q.x + q.y) + (q.z + q.w));
        if (blockDim.x > 256) {
            const float4 r = part[2], s = part[3];
            sum[i] += ((r.x + r.y) + (r.z + r.w)) + ((s.x + s.y) + (s.z + s.w));
        }
    }
    return make_float2(sum[0], sum[1]);
}
__device__ __forceinline__ float row_sum(float a, float (&buf)[2][16]) { return row_sums<false>(a, 0.f, buf).x; }

}  // namespace row
}  // namespace qmoe
