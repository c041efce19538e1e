// values.cuh -- bf16, fp16 and fp32 values to and from fp32 registers, eight at
// a time: what the router's and the rows' kernels share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <type_traits>

namespace tcg {

template <typename T>
__device__ __forceinline__ float to_float(T v);
template <>
__device__ __forceinline__ float to_float(float v) { return v; }
template <>
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }

// Rounded once, to nearest even.
template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_float(float v) { return __float2half_rn(v); }

template <typename T>
__device__ __forceinline__ uint32_t pack_pair(float lo, float hi) {
    static_assert(sizeof(T) == 2, "16-bit types");
    if constexpr (std::is_same<T, __half>::value) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&b);
    }
}

template <typename T>
__device__ __forceinline__ void unpack_pair(uint32_t w, float& lo, float& hi) {
    static_assert(sizeof(T) == 2, "16-bit types");
    if constexpr (std::is_same<T, __half>::value) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
        lo = f.x;
        hi = f.y;
    } else {
        lo = __uint_as_float(w << 16);
        hi = __uint_as_float(w & 0xFFFF0000u);
    }
}

// Eight values of a row as they lie in memory: one 16-byte word, or two of fp32.
template <typename T>
struct Raw8 {
    uint4 w[sizeof(T) / 2];
};

// From a 16-byte aligned address; kOnce: a row that is read once passes the caches by.
template <typename T, bool kOnce = false>
__device__ __forceinline__ Raw8<T> load_raw8(const T* src) {
    Raw8<T> r;
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i)
        r.w[i] = kOnce ? __ldcs(reinterpret_cast<const uint4*>(src) + i) : *(reinterpret_cast<const uint4*>(src) + i);
    return r;
}

// The first n of eight values, one by one (zeros after them).
template <typename T>
__device__ __forceinline__ Raw8<T> load_some8(const T* src, int n) {
    Raw8<T> r;
    T v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? src[i] : from_float<T>(0.0f);
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            r.w[i] = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]), __float_as_uint(v[4 * i + 2]),
                                __float_as_uint(v[4 * i + 3]));
    } else {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            u[i] = static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(&v[2 * i])) |
                   (static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(&v[2 * i + 1])) << 16);
        r.w[0] = make_uint4(u[0], u[1], u[2], u[3]);
    }
    return r;
}

template <typename T>
__device__ __forceinline__ void values_of(const Raw8<T>& r, float (&x)[8]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            x[4 * i] = __uint_as_float(r.w[i].x);
            x[4 * i + 1] = __uint_as_float(r.w[i].y);
            x[4 * i + 2] = __uint_as_float(r.w[i].z);
            x[4 * i + 3] = __uint_as_float(r.w[i].w);
        }
    } else {
        unpack_pair<T>(r.w[0].x, x[0], x[1]);
        unpack_pair<T>(r.w[0].y, x[2], x[3]);
        unpack_pair<T>(r.w[0].z, x[4], x[5]);
        unpack_pair<T>(r.w[0].w, x[6], x[7]);
    }
}

template <typename T>
__device__ __forceinline__ Raw8<T> raw_of(const float (&x)[8]) {
    Raw8<T> r;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            r.w[i] = make_uint4(__float_as_uint(x[4 * i]), __float_as_uint(x[4 * i + 1]), __float_as_uint(x[4 * i + 2]),
                                __float_as_uint(x[4 * i + 3]));
    } else {
        r.w[0] = make_uint4(pack_pair<T>(x[0], x[1]), pack_pair<T>(x[2], x[3]), pack_pair<T>(x[4], x[5]), pack_pair<T>(x[6], x[7]));
    }
    return r;
}

template <typename T>
__device__ __forceinline__ void store_raw8(T* dst, const Raw8<T>& r) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) __stcs(reinterpret_cast<uint4*>(dst) + i, r.w[i]);
}

template <typename T>
__device__ __forceinline__ void store_some8(T* dst, const Raw8<T>& r, int n) {
    if constexpr (sizeof(T) == 4) {
        float x[8];
        values_of<T>(r, x);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) dst[i] = x[i];
    } else {
        const uint32_t u[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) reinterpret_cast<uint16_t*>(dst)[i] = static_cast<uint16_t>(u[i / 2] >> (16 * (i & 1)));
    }
}

}  // namespace tcg
