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

// Eight values of a row that starts anywhere, from element e0 on (which may lie
// before the row, or so that some lie past its end: zeros there).  Whole 16-byte
// words are loaded, each of them holding a value that is asked for, and shifted
// into place.
template <typename T>
__device__ __forceinline__ Raw8<T> load_any8(const T* row, int e0, int cols) {
    constexpr int kWords = 2 * static_cast<int>(sizeof(T));          // of four bytes
    const uintptr_t at = reinterpret_cast<uintptr_t>(row) + static_cast<long long>(e0) * static_cast<int>(sizeof(T));
    const uintptr_t first = reinterpret_cast<uintptr_t>(row + max(e0, 0)), last = reinterpret_cast<uintptr_t>(row + min(e0 + 8, cols));
    const uintptr_t base = at & ~static_cast<uintptr_t>(15);
    const uint32_t off = static_cast<uint32_t>(at & 15);
    uint32_t w[kWords + 4];
#pragma unroll
    for (int i = 0; i <= kWords / 4; ++i) {
        const uintptr_t b = base + 16 * i;
        uint4 q = make_uint4(0u, 0u, 0u, 0u);
        if ((i < kWords / 4 || off) && b + 16 > first && b < last) q = *reinterpret_cast<const uint4*>(b);
        w[4 * i] = q.x, w[4 * i + 1] = q.y, w[4 * i + 2] = q.z, w[4 * i + 3] = q.w;
    }
    uint32_t o[kWords];
    if (off) {
        uint32_t u[kWords + 2], t[kWords + 1];
#pragma unroll
        for (int i = 0; i < kWords + 2; ++i) u[i] = off & 8u ? w[i + 2] : w[i];
#pragma unroll
        for (int i = 0; i < kWords + 1; ++i) t[i] = off & 4u ? u[i + 1] : u[i];
#pragma unroll
        for (int i = 0; i < kWords; ++i) o[i] = sizeof(T) == 4 ? t[i] : __funnelshift_r(t[i], t[i + 1], (off & 2u) * 8u);
    } else {
#pragma unroll
        for (int i = 0; i < kWords; ++i) o[i] = w[i];
    }
    if (e0 < 0 || e0 + 8 > cols) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (e0 + i >= 0 && e0 + i < cols) continue;
            if constexpr (sizeof(T) == 4) o[i] = 0u;
            else o[i / 2] &= i & 1 ? 0x0000FFFFu : 0xFFFF0000u;
        }
    }
    Raw8<T> r;
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i) r.w[i] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
    return r;
}

// Elements that a row's first value lies past a 16-byte boundary.
template <typename T>
__device__ __forceinline__ int past16(const T* row) {
    return static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
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

// To elements e0 on of a row, those that lie in it; row + e0 starts on 16 bytes.
template <typename T>
__device__ __forceinline__ void store_any8(T* row, int e0, int cols, const Raw8<T>& r) {
    if (e0 >= 0 && e0 + 8 <= cols) {
        store_raw8<T>(row + e0, r);
        return;
    }
    uint32_t u[2 * sizeof(T)];
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) u[4 * i] = r.w[i].x, u[4 * i + 1] = r.w[i].y, u[4 * i + 2] = r.w[i].z, u[4 * i + 3] = r.w[i].w;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (e0 + i < 0 || e0 + i >= cols) continue;
        if constexpr (sizeof(T) == 4) reinterpret_cast<uint32_t*>(row)[e0 + i] = u[i];
        else reinterpret_cast<uint16_t*>(row)[e0 + i] = static_cast<uint16_t>(u[i / 2] >> (16 * (i & 1)));
    }
}

}  // namespace tcg
