// moe_route.cu -- a router's choice of experts, their weights, and the logits'
// gradient.
//
//   top_k: the k largest logits of a token, in falling order, ties to the lower
//     expert; -inf never
//   w_j = exp(x_{e_j} - max) / sum of exp over all experts, or over the chosen
//   all:    dx_e = p_e (sum_{j: e_j = e} g_j - sum_j g_j p_{e_j})
//   chosen: dx_{e_j} = w_j (g_j - sum_i g_i w_i)
//
// A warp holds a row, kN neighbouring experts a lane.  Logits become integers
// that sort alike, and each round takes the warp's largest in one reduction;
// then the lane that held it alone looks for its next.  16-bit logits share a
// 32-bit key with the expert's number, so keys differ and "removed" is "not
// below the last one taken"; fp32 keys need the lowest lane and place of equal
// ones.  Statistics are fp32.
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "host.h"
#include "values.cuh"

namespace {

using tcg::from_float;
using tcg::to_float;

constexpr int kMaxExperts = 1024;
constexpr int kMaxK = 32;       // a lane each
constexpr int kWarps = 8;
constexpr uint32_t kAll = 0xFFFFFFFFu;

struct Route {
    const void* logits;
    long long ld;
    const uint8_t* mask;
    int tokens, experts, k;
    int chosen_only;
    int* topk;
    long long ld_topk;
    float* weights;
    long long ld_weights;
    int vec;          // a lane's logits may be read as whole words
    // backward
    const float* grad;
    long long ld_grad;
    int accumulate;
    void* dlogits;
    long long ldd;
    tcg_dtype d_dtype;
};

// kN values of a lane from an address aligned to their size, at most 16 bytes.
template <typename T, int kN>
__device__ __forceinline__ void load_lane(const T* src, T (&x)[kN]) {
    constexpr int kBytes = kN * static_cast<int>(sizeof(T));
    if constexpr (kBytes >= 16) {
#pragma unroll
        for (int i = 0; i < kBytes / 16; ++i) reinterpret_cast<uint4*>(x)[i] = *(reinterpret_cast<const uint4*>(src) + i);
    } else if constexpr (kBytes == 8) {
        *reinterpret_cast<uint2*>(x) = *reinterpret_cast<const uint2*>(src);
    } else if constexpr (kBytes == 4) {
        *reinterpret_cast<uint32_t*>(x) = *reinterpret_cast<const uint32_t*>(src);
    } else {
        x[0] = src[0];
    }
}

template <typename T>
__device__ __forceinline__ T lowest();
template <>
__device__ __forceinline__ float lowest<float>() { return __uint_as_float(0xFF800000u); }
template <>
__device__ __forceinline__ __nv_bfloat16 lowest<__nv_bfloat16>() { return __ushort_as_bfloat16(0xFF80u); }
template <>
__device__ __forceinline__ __half lowest<__half>() { return __ushort_as_half(0xFC00u); }

// A lane's kN experts of row t, -inf past the last expert.
template <typename T, int kN>
__device__ __forceinline__ void load_row(const Route& p, long long t, int lane, T (&x)[kN]) {
    const T* row = static_cast<const T*>(p.logits) + t * p.ld;
    const int e0 = lane * kN;
    if (p.vec && e0 + kN <= p.experts) {
        load_lane<T, kN>(row + e0, x);
    } else {
#pragma unroll
        for (int i = 0; i < kN; ++i) x[i] = e0 + i < p.experts ? row[e0 + i] : lowest<T>();
    }
}

// Integers that sort as the values do: -inf is 0, both zeros are one, NaN is
// the largest.  16-bit values share the word with the expert's number turned
// over, so that of equal ones the lower expert is the larger key.
__device__ __forceinline__ uint32_t key_of(float v, int) {
    if (v != v) return 0xFFFFFFFFu;
    if (v == -INFINITY) return 0u;
    const uint32_t b = __float_as_uint(v + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
template <uint32_t kInf>
__device__ __forceinline__ uint32_t key16(uint32_t b, int e) {
    if (b == (0x8000u | kInf)) return 0u;
    if (b == 0x8000u) b = 0u;
    const uint32_t o = (b & 0x7FFFu) > kInf ? 0xFFFFu : (b & 0x8000u ? b ^ 0xFFFFu : b | 0x8000u);
    return (o << 16) | static_cast<uint32_t>(0xFFFF - e);
}
__device__ __forceinline__ uint32_t key_of(__nv_bfloat16 v, int e) { return key16<0x7F80u>(__bfloat16_as_ushort(v), e); }
__device__ __forceinline__ uint32_t key_of(__half v, int e) { return key16<0x7C00u>(__half_as_ushort(v), e); }

// The value a key stands for.
template <typename T>
__device__ __forceinline__ float value_of(uint32_t key) {
    if constexpr (sizeof(T) == 4) {
        if (key == 0xFFFFFFFFu) return __uint_as_float(0x7FC00000u);
        return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
    } else {
        const uint32_t o = key >> 16;
        if (o == 0xFFFFu) return __uint_as_float(0x7FC00000u);
        const uint32_t b = o & 0x8000u ? o & 0x7FFFu : o ^ 0xFFFFu;
        if constexpr (std::is_same<T, __half>::value) return __half2float(__ushort_as_half(static_cast<unsigned short>(b)));
        else return __uint_as_float(b << 16);
    }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, d));
    return v;
}

template <typename T, int kN>
__global__ void __launch_bounds__(32 * kWarps) route_kernel(const __grid_constant__ Route p) {
    tcg::host::wait_for_kernel_ahead();
    const int lane = threadIdx.x & 31;
    const long long t = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (t >= p.tokens) return;
    int* topk = p.topk + t * p.ld_topk;
    float* weights = p.weights + t * p.ld_weights;
    if (p.mask && !p.mask[t]) {
        if (lane < p.k) {
            topk[lane] = -1;
            weights[lane] = 0.0f;
        }
        return;
    }
    alignas(16) T x[kN];
    load_row<T, kN>(p, t, lane, x);
    uint32_t key[kN], mine = 0u;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
        key[i] = key_of(x[i], lane * kN + i);
        mine = max(mine, key[i]);
    }
    int my_e = -1;
    uint32_t my_key = 0u, top = 0u;
    for (int j = 0; j < p.k; ++j) {
        const uint32_t best = __reduce_max_sync(kAll, mine);
        if (best == 0u) break;
        if (j == 0) top = best;
        int e;
        if constexpr (sizeof(T) == 2) {
            e = 0xFFFF - static_cast<int>(best & 0xFFFFu);
            if (mine == best) {
                mine = 0u;
#pragma unroll
                for (int i = 0; i < kN; ++i) mine = max(mine, key[i] < best ? key[i] : 0u);
            }
        } else {
            const int holder = __ffs(__ballot_sync(kAll, mine == best)) - 1;
            int at = 0;
            if (lane == holder) {
                bool found = false;
                mine = 0u;
#pragma unroll
                for (int i = 0; i < kN; ++i) {
                    if (!found && key[i] == best) {
                        found = true;
                        at = i;
                        key[i] = 0u;
                    }
                    mine = max(mine, key[i]);
                }
                at += lane * kN;
            }
            e = __shfl_sync(kAll, at, holder);
        }
        if (lane == j) {
            my_e = e;
            my_key = best;
        }
    }
    // (a token without experts has top = 0, and no lane a choice)
    const float m = value_of<T>(top);
    const float z = my_e >= 0 ? expf(value_of<T>(my_key) - m) : 0.0f;
    float s = z;
    if (!p.chosen_only) {
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < kN; ++i) s += expf(to_float(x[i]) - m);
    }
    s = warp_sum(s);
    if (lane < p.k) {
        topk[lane] = my_e;
        weights[lane] = my_e >= 0 ? z / s : 0.0f;
    }
}

// kN gradients of a lane, added to what is there or not, rounded once.
template <typename D, int kN>
__device__ __forceinline__ void store_lane(const Route& p, long long t, int lane, const float (&d)[kN]) {
    D* row = static_cast<D*>(p.dlogits) + t * p.ldd;
    const int e0 = lane * kN;
    constexpr int kBytes = kN * static_cast<int>(sizeof(D));
    const bool whole = e0 + kN <= p.experts && (reinterpret_cast<uintptr_t>(row + e0) & (kBytes < 16 ? kBytes - 1 : 15)) == 0;
    alignas(16) D v[kN];
    if (whole) {
        if (p.accumulate) load_lane<D, kN>(row + e0, v);
#pragma unroll
        for (int i = 0; i < kN; ++i) v[i] = from_float<D>(p.accumulate ? to_float(v[i]) + d[i] : d[i]);
        if constexpr (kBytes >= 16) {
#pragma unroll
            for (int i = 0; i < kBytes / 16; ++i) reinterpret_cast<uint4*>(row + e0)[i] = reinterpret_cast<const uint4*>(v)[i];
        } else if constexpr (kBytes == 8) {
            *reinterpret_cast<uint2*>(row + e0) = *reinterpret_cast<const uint2*>(v);
        } else if constexpr (kBytes == 4) {
            *reinterpret_cast<uint32_t*>(row + e0) = *reinterpret_cast<const uint32_t*>(v);
        } else {
            row[e0] = v[0];
        }
    } else {
#pragma unroll
        for (int i = 0; i < kN; ++i)
            if (e0 + i < p.experts) row[e0 + i] = from_float<D>(p.accumulate ? to_float(row[e0 + i]) + d[i] : d[i]);
    }
}

template <typename T, int kN>
__global__ void __launch_bounds__(32 * kWarps) route_grad_kernel(const __grid_constant__ Route p) {
    tcg::host::wait_for_kernel_ahead();
    const int lane = threadIdx.x & 31;
    const long long t = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (t >= p.tokens) return;
    int e = lane < p.k ? p.topk[t * p.ld_topk + lane] : -1;
    if (e >= p.experts) e = -1;
    float g = e >= 0 ? p.grad[t * p.ld_grad + lane] : 0.0f;
    uint32_t live = __ballot_sync(kAll, e >= 0);
    float d[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) d[i] = 0.0f;
    if (live == 0u && p.accumulate) return;   // a token of nobody adds nothing, whatever its logits hold
    if (live != 0u) {
        if (p.chosen_only) {
            const float x = e >= 0 ? to_float(static_cast<const T*>(p.logits)[t * p.ld + e]) : -INFINITY;
            float m = warp_max(x);
            if (m == -INFINITY) m = 0.0f;
            const float z = expf(x - m);
            const float s = warp_sum(z);
            const float w = s == 0.0f ? 0.0f : z / s;
            g = w * (g - warp_sum(e >= 0 ? w * g : 0.0f));
        }
        // what the lane's experts get of the chosen ones, in their order
        while (live) {
            const int j = __ffs(live) - 1;
            live &= live - 1;
            const int at = __shfl_sync(kAll, e, j) - lane * kN;
            const float gj = __shfl_sync(kAll, g, j);
#pragma unroll
            for (int i = 0; i < kN; ++i) d[i] += i == at ? gj : 0.0f;
        }
        if (!p.chosen_only) {
            alignas(16) T x[kN];
            load_row<T, kN>(p, t, lane, x);
            float m = -INFINITY;
#pragma unroll
            for (int i = 0; i < kN; ++i) m = fmaxf(m, to_float(x[i]));
            m = warp_max(m);
            if (m == -INFINITY) m = 0.0f;
            float z[kN], s = 0.0f, inner = 0.0f;
#pragma unroll
            for (int i = 0; i < kN; ++i) {
                z[i] = expf(to_float(x[i]) - m);
                s += z[i];
                inner += z[i] * d[i];
            }
            s = warp_sum(s);
            const float inv = s == 0.0f ? 0.0f : 1.0f / s;
            inner = warp_sum(inner) * inv;
#pragma unroll
            for (int i = 0; i < kN; ++i) d[i] = z[i] * inv * (d[i] - inner);
        }
    }
    if (p.d_dtype == TCG_F32) store_lane<float, kN>(p, t, lane, d);
    else if (p.d_dtype == TCG_F16) store_lane<__half, kN>(p, t, lane, d);
    else store_lane<__nv_bfloat16, kN>(p, t, lane, d);
}

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
int size_of(tcg_dtype t) { return t == TCG_F32 ? 4 : 2; }
bool known(tcg_dtype t) { return t == TCG_BF16 || t == TCG_F16 || t == TCG_F32; }

// neighbouring experts a lane holds
int lane_experts(int experts) {
    int n = 1;
    while (32 * n < experts) n *= 2;
    return n;
}

template <typename T, typename F>
void with_experts(int experts, F f) {
    using std::integral_constant;
    switch (lane_experts(experts)) {
        case 1: return f(T{}, integral_constant<int, 1>{});
        case 2: return f(T{}, integral_constant<int, 2>{});
        case 4: return f(T{}, integral_constant<int, 4>{});
        case 8: return f(T{}, integral_constant<int, 8>{});
        case 16: return f(T{}, integral_constant<int, 16>{});
        default: return f(T{}, integral_constant<int, 32>{});
    }
}
template <typename F>
void with_types(tcg_dtype dtype, int experts, F f) {
    if (dtype == TCG_BF16) with_experts<__nv_bfloat16>(experts, f);
    else if (dtype == TCG_F16) with_experts<__half>(experts, f);
    else with_experts<float>(experts, f);
}

tcg_status start(Route& p, int tokens, int experts, int k, tcg_dtype dtype, const void* logits, int ld, const int* topk,
                 int ld_topk, int chosen_only) {
    if (tokens < 0 || experts < 1 || k < 1 || k > experts || !known(dtype)) return TCG_ERR_INVALID_ARG;
    if (experts > kMaxExperts || k > kMaxK || tokens > tcg::host::kMaxExtent) return TCG_ERR_UNSUPPORTED;
    if (tokens == 0) return TCG_OK;
    if (!logits || ld < experts || !topk || ld_topk < k) return TCG_ERR_INVALID_ARG;
    if (!aligned(logits, size_of(dtype)) || !aligned(topk, 4)) return TCG_ERR_MISALIGNED;
    p.logits = logits;
    p.ld = ld;
    p.tokens = tokens;
    p.experts = experts;
    p.k = k;
    p.chosen_only = chosen_only != 0;
    p.topk = const_cast<int*>(topk);
    p.ld_topk = ld_topk;
    const long long word = std::min(16, lane_experts(experts) * size_of(dtype));
    p.vec = aligned(logits, word) && static_cast<long long>(ld) * size_of(dtype) % word == 0;
    return TCG_OK;
}

tcg_status launched(cudaError_t e, const char* what) { return e == cudaSuccess ? TCG_OK : tcg::host::fail_launch(what, e); }
dim3 grid_of(int tokens) { return dim3((static_cast<unsigned>(tokens) + kWarps - 1) / kWarps); }

}  // namespace

extern "C" {

tcg_status tcg_moe_route(int tokens, int experts, int k, tcg_dtype dtype, const void* logits, int ld, const uint8_t* mask,
                         int renormalize, int* topk, int ld_topk, float* weights, int ld_weights, void* stream) {
    Route p = {};
    tcg_status st = start(p, tokens, experts, k, dtype, logits, ld, topk, ld_topk, renormalize);
    if (st != TCG_OK || tokens == 0) return st;
    if (!weights || ld_weights < k) return TCG_ERR_INVALID_ARG;
    if (!aligned(weights, 4)) return TCG_ERR_MISALIGNED;
    tcg::host::Device dev;
    if ((st = tcg::host::device(dev)) != TCG_OK) return st;
    p.mask = mask;
    p.weights = weights;
    p.ld_weights = ld_weights;
    cudaError_t err = cudaSuccess;
    with_types(dtype, experts, [&](auto x, auto n) {
        err = tcg::host::launch_early(route_kernel<decltype(x), decltype(n)::value>, grid_of(tokens), 32 * kWarps,
                                      static_cast<cudaStream_t>(stream), p);
    });
    return launched(err, "tcg_moe_route");
}

tcg_status tcg_moe_route_backward(int tokens, int experts, int k, tcg_dtype dtype, const void* logits, int ld, const int* topk,
                                  int ld_topk, int renormalize, const float* grad_weights, int ld_grad, int accumulate,
                                  void* dlogits, int ldd, tcg_dtype d_dtype, void* stream) {
    Route p = {};
    if (!known(d_dtype)) return TCG_ERR_INVALID_ARG;
    tcg_status st = start(p, tokens, experts, k, dtype, logits, ld, topk, ld_topk, renormalize);
    if (st != TCG_OK || tokens == 0) return st;
    if (!grad_weights || ld_grad < k || !dlogits || ldd < experts) return TCG_ERR_INVALID_ARG;
    if (!aligned(grad_weights, 4) || !aligned(dlogits, size_of(d_dtype))) return TCG_ERR_MISALIGNED;
    tcg::host::Device dev;
    if ((st = tcg::host::device(dev)) != TCG_OK) return st;
    p.grad = grad_weights;
    p.ld_grad = ld_grad;
    p.accumulate = accumulate != 0;
    p.dlogits = dlogits;
    p.ldd = ldd;
    p.d_dtype = d_dtype;
    cudaError_t err = cudaSuccess;
    with_types(dtype, experts, [&](auto x, auto n) {
        err = tcg::host::launch_early(route_grad_kernel<decltype(x), decltype(n)::value>, grid_of(tokens), 32 * kWarps,
                                      static_cast<cudaStream_t>(stream), p);
    });
    return launched(err, "tcg_moe_route_backward");
}

}  // extern "C"
