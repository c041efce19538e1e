// moe_balance.cu -- a router's balance loss, its assignments per expert and
// the loss's gradient with respect to the logits.
//
//   p_te = softmax of token t's logits over the E experts
//   n    = tokens that count (mask != 0),  c_e = assignments to e of those
//   f_e  = E c_e / (k n),  P_e = 1/n sum_t p_te      (all 0 when n = 0)
//   loss = coef sum_e f_e P_e
//   dlogits_te = g coef / n  p_te (f_e - sum_j f_j p_tj)
//
// The assignments are constants of the gradient.  A token whose logits are
// all -inf has p = 0 (and gradient 0).  Statistics and sums are fp32.
//
// Bound by memory (logits once forward; once more, and their gradient,
// backward) and, for few tokens, by the launch.  A row is held by the fewest
// lanes that take eight elements each, so a warp reads whole lines whatever
// E is, and P_e sums stay in the registers of the lane that owns the columns.
// Partial sums go to the workspace CTA by CTA; the last CTA adds them in CTA
// order, so the loss does not depend on the order of arrival.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <climits>
#include <cstdint>

#include "host.h"
#include "ptx.cuh"

namespace {

constexpr int kMaxExperts = 1024;
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCtas = 152;
constexpr size_t kPartialBytes = static_cast<size_t>(kMaxCtas) * (2 * kMaxExperts + 1) * 4;

struct Balance {
    const void* logits;
    long long ld;
    const int* topk;
    long long ld_topk;
    const uint8_t* mask;
    int tokens, experts, k;
    float coef;
    int* counts;
    int* offsets;
    int* valid;
    float* loss;
    float* part_p;      // [cta][experts]
    int* part_c;        // [cta][experts]
    int* part_n;        // [cta]
    int* arrivals;
    const float* grad;
    void* dlogits;
    long long ldd;
    int lanes;          // lanes per row (a power of two)
    int vec;            // rows may be read 16 bytes at a time
    int d_vec;          // and the gradient's rows written so
    tcg_dtype d_dtype;
};

template <typename T>
__device__ __forceinline__ float to_float(T v);
template <>
__device__ __forceinline__ float to_float(float v) { return v; }
template <>
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }

__device__ __forceinline__ uint32_t pair16(float lo, float hi, tcg_dtype t) {
    if (t == TCG_F16) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
}

// Columns [e0, e0 + 8) of one row of the gradient, rounded once to its type.
__device__ __forceinline__ void store_grad(const Balance& p, long long t, int e0, const float (&v)[8]) {
    const long long at = t * p.ldd + e0;
    const bool f32 = p.d_dtype == TCG_F32;
    if (p.d_vec && e0 + 8 <= p.experts) {
        if (f32) {
            float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.dlogits) + at);
            dst[0] = make_float4(v[0], v[1], v[2], v[3]);
            dst[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.dlogits) + at) =
                make_uint4(pair16(v[0], v[1], p.d_dtype), pair16(v[2], v[3], p.d_dtype), pair16(v[4], v[5], p.d_dtype),
                           pair16(v[6], v[7], p.d_dtype));
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (e0 + i >= p.experts) continue;
        if (f32) static_cast<float*>(p.dlogits)[at + i] = v[i];
        else static_cast<uint16_t*>(p.dlogits)[at + i] = static_cast<uint16_t>(pair16(v[i], 0.0f, p.d_dtype));
    }
}

template <typename T>
struct alignas(16) Pack {
    T v[16 / sizeof(T)];
};

// kC chunks of eight columns per lane: column (chunk * lanes + l) * 8 + i.
template <typename T, int kC>
__device__ __forceinline__ void load_row(const Balance& p, int t, int l, float (&x)[kC][8]) {
    const T* row = static_cast<const T*>(p.logits) + t * p.ld;
    constexpr int kPer = 16 / sizeof(T);
#pragma unroll
    for (int c = 0; c < kC; ++c) {
        const int e0 = (c * p.lanes + l) * 8;
        if (p.vec && e0 + 8 <= p.experts) {
#pragma unroll
            for (int h = 0; h < 8 / kPer; ++h) {
                const Pack<T> q = *reinterpret_cast<const Pack<T>*>(row + e0 + h * kPer);
#pragma unroll
                for (int i = 0; i < kPer; ++i) x[c][h * kPer + i] = to_float<T>(q.v[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[c][i] = e0 + i < p.experts ? to_float<T>(row[e0 + i]) : -INFINITY;
        }
    }
}

// x becomes the row's softmax; columns past the experts become 0.
template <int kC>
__device__ __forceinline__ void softmax_row(const Balance& p, float (&x)[kC][8]) {
    float m = -INFINITY;
#pragma unroll
    for (int c = 0; c < kC; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, x[c][i]);
    for (int d = 1; d < p.lanes; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    if (m == -INFINITY) m = 0.0f;   // nothing but -inf: every exp is 0
    float s = 0.0f;
#pragma unroll
    for (int c = 0; c < kC; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[c][i] = expf(x[c][i] - m);
            s += x[c][i];
        }
    for (int d = 1; d < p.lanes; d <<= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    const float r = s == 0.0f ? 0.0f : 1.0f / s;
#pragma unroll
    for (int c = 0; c < kC; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) x[c][i] *= r;
}

template <typename T, int kC>
__global__ void __launch_bounds__(kThreads) balance_kernel(const __grid_constant__ Balance p) {
    __shared__ float sum_p[kMaxExperts];
    __shared__ int hist[kMaxExperts];
    __shared__ float red[kThreads];
    __shared__ int n_valid, last;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int l = lane & (p.lanes - 1), slot = lane / p.lanes, per_warp = 32 / p.lanes;
    for (int e = threadIdx.x; e < p.experts; e += kThreads) hist[e] = 0;
    if (threadIdx.x == 0) n_valid = 0;
    __syncthreads();
    // this CTA's tokens
    const int t0 = static_cast<int>(static_cast<long long>(blockIdx.x) * p.tokens / gridDim.x);
    const int t1 = static_cast<int>(static_cast<long long>(blockIdx.x + 1) * p.tokens / gridDim.x);

    for (long long i = threadIdx.x; i < static_cast<long long>(t1 - t0) * p.k; i += kThreads) {
        const int t = t0 + static_cast<int>(i / p.k), j = static_cast<int>(i % p.k);
        if (p.mask && !p.mask[t]) continue;
        const int e = __ldg(p.topk + t * p.ld_topk + j);
        if (e >= 0 && e < p.experts) atomicAdd(&hist[e], 1);
    }
    float acc[kC][8];
#pragma unroll
    for (int c = 0; c < kC; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[c][i] = 0.0f;
    int n = 0;
    for (int tb = t0 + warp * per_warp; tb < t1; tb += kWarps * per_warp) {
        const int t = tb + slot;
        const bool in = t < t1 && (!p.mask || p.mask[t]);
        float x[kC][8];
        if (in) {
            load_row<T, kC>(p, t, l, x);
        } else {
#pragma unroll
            for (int c = 0; c < kC; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) x[c][i] = -INFINITY;
        }
        softmax_row<kC>(p, x);
        if (in && l == 0) ++n;
#pragma unroll
        for (int c = 0; c < kC; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[c][i] += x[c][i];
    }
    if (n) atomicAdd(&n_valid, n);
    // rows of one warp, then of the CTA's warps, in a fixed order
#pragma unroll
    for (int c = 0; c < kC; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            for (int d = p.lanes; d < 32; d <<= 1) acc[c][i] += __shfl_xor_sync(0xffffffffu, acc[c][i], d);
    for (int w = 0; w < kWarps; ++w) {
        if (warp == w && slot == 0) {
#pragma unroll
            for (int c = 0; c < kC; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int e = (c * p.lanes + l) * 8 + i;
                    if (e < p.experts) sum_p[e] = w == 0 ? acc[c][i] : sum_p[e] + acc[c][i];
                }
        }
        __syncthreads();
    }
    for (int e = threadIdx.x; e < p.experts; e += kThreads) {
        p.part_p[static_cast<long long>(blockIdx.x) * p.experts + e] = sum_p[e];
        p.part_c[static_cast<long long>(blockIdx.x) * p.experts + e] = hist[e];
    }
    if (threadIdx.x == 0) p.part_n[blockIdx.x] = n_valid;
    __syncthreads();
    if (threadIdx.x == 0) {
        const int old = tcg::ptx::atomic_add_acq_rel_gpu(p.arrivals, 1);
        last = old == static_cast<int>(gridDim.x) - 1;
        if (last) atomicExch(p.arrivals, 0);   // ready for the next call
    }
    __syncthreads();
    if (!last) return;

    // The last CTA: sums over the CTAs in their order.
    if (threadIdx.x == 0) {
        int total = 0;
        for (int b = 0; b < static_cast<int>(gridDim.x); ++b) total += __ldcg(p.part_n + b);
        n_valid = total;
    }
    for (int e = threadIdx.x; e < p.experts; e += kThreads) {
        float s = 0.0f;
        int c = 0;
#pragma unroll 8
        for (int b = 0; b < static_cast<int>(gridDim.x); ++b) {
            s += __ldcg(p.part_p + static_cast<long long>(b) * p.experts + e);
            c += __ldcg(p.part_c + static_cast<long long>(b) * p.experts + e);
        }
        sum_p[e] = s;
        hist[e] = c;
        p.counts[e] = c;
    }
    __syncthreads();
    const float inv_n = n_valid > 0 ? 1.0f / static_cast<float>(n_valid) : 0.0f;
    float mine = 0.0f;
    for (int e = threadIdx.x; e < p.experts; e += kThreads)
        mine += (static_cast<float>(hist[e]) * inv_n) * (sum_p[e] * inv_n);
    red[threadIdx.x] = mine;
    __syncthreads();
    for (int d = kThreads / 2; d > 0; d >>= 1) {
        if (threadIdx.x < d) red[threadIdx.x] += red[threadIdx.x + d];
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        *p.loss = p.coef * (static_cast<float>(p.experts) / static_cast<float>(p.k)) * red[0];
        *p.valid = n_valid;
    }
    if (p.offsets && warp == 0) {
        int base = 0;
        for (int e0 = 0; e0 < p.experts; e0 += 32) {
            const int e = e0 + lane;
            const int c = e < p.experts ? hist[e] : 0;
            int incl = c;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, incl, d);
                if (lane >= d) incl += o;
            }
            if (e < p.experts) p.offsets[e] = base + incl - c;
            base += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) p.offsets[p.experts] = base;
    }
}

template <typename T, int kC>
__global__ void __launch_bounds__(256) balance_grad_kernel(const __grid_constant__ Balance p) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int l = lane & (p.lanes - 1), slot = lane / p.lanes, per_warp = 32 / p.lanes;
    const int n = __ldg(p.valid);
    const float inv_n = n > 0 ? 1.0f / static_cast<float>(n) : 0.0f;
    const float to_f = static_cast<float>(p.experts) / static_cast<float>(p.k) * inv_n;
    const float g = __ldg(p.grad) * p.coef * inv_n;
    float f[kC][8];
#pragma unroll
    for (int c = 0; c < kC; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int e = (c * p.lanes + l) * 8 + i;
            f[c][i] = e < p.experts ? static_cast<float>(__ldg(p.counts + e)) * to_f : 0.0f;
        }
    const long long step = static_cast<long long>(gridDim.x) * 8 * per_warp;
    for (long long tb = (static_cast<long long>(blockIdx.x) * 8 + warp) * per_warp; tb < p.tokens; tb += step) {
        const long long t = tb + slot;
        const bool real = t < p.tokens;
        const bool in = real && (!p.mask || p.mask[t]);
        float x[kC][8];
        if (in) {
            load_row<T, kC>(p, static_cast<int>(t), l, x);
        } else {
#pragma unroll
            for (int c = 0; c < kC; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) x[c][i] = -INFINITY;
        }
        softmax_row<kC>(p, x);
        float dot = 0.0f;
#pragma unroll
        for (int c = 0; c < kC; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) dot = fmaf(f[c][i], x[c][i], dot);
        for (int d = 1; d < p.lanes; d <<= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
        if (!real) continue;
#pragma unroll
        for (int c = 0; c < kC; ++c) {
            float d[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] = g * (x[c][i] * (f[c][i] - dot));
            store_grad(p, t, (c * p.lanes + l) * 8, d);
        }
    }
}

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
int size_of(tcg_dtype t) { return t == TCG_F32 ? 4 : 2; }

tcg_status start(Balance& p, int tokens, int experts, int k, tcg_dtype dtype, const void* logits, int ld,
                 const uint8_t* mask, float coef) {
    if (tokens < 0 || experts < 1 || k < 1) return TCG_ERR_INVALID_ARG;
    if (dtype != TCG_BF16 && dtype != TCG_F16 && dtype != TCG_F32) return TCG_ERR_INVALID_ARG;
    if (experts > kMaxExperts) return TCG_ERR_UNSUPPORTED;
    if (tokens > 0 && (!logits || ld < experts)) return TCG_ERR_INVALID_ARG;
    if (!aligned(logits, size_of(dtype))) return TCG_ERR_MISALIGNED;
    p.logits = logits;
    p.ld = ld;
    p.mask = mask;
    p.tokens = tokens;
    p.experts = experts;
    p.k = k;
    p.coef = coef;
    p.lanes = 1;
    while (p.lanes < 32 && p.lanes * 8 < experts) p.lanes *= 2;
    p.vec = aligned(logits, 16) && (static_cast<long long>(ld) * size_of(dtype)) % 16 == 0;
    return TCG_OK;
}

template <typename T>
void launch_forward(const Balance& p, int ctas, cudaStream_t s) {
    const int chunks = (p.experts + p.lanes * 8 - 1) / (p.lanes * 8);
    if (chunks == 1) balance_kernel<T, 1><<<ctas, kThreads, 0, s>>>(p);
    else if (chunks == 2) balance_kernel<T, 2><<<ctas, kThreads, 0, s>>>(p);
    else balance_kernel<T, 4><<<ctas, kThreads, 0, s>>>(p);
}

template <typename T>
void launch_backward(const Balance& p, int ctas, cudaStream_t s) {
    const int chunks = (p.experts + p.lanes * 8 - 1) / (p.lanes * 8);
    if (chunks == 1) balance_grad_kernel<T, 1><<<ctas, 256, 0, s>>>(p);
    else if (chunks == 2) balance_grad_kernel<T, 2><<<ctas, 256, 0, s>>>(p);
    else balance_grad_kernel<T, 4><<<ctas, 256, 0, s>>>(p);
}

tcg_status launched(const char* what) {
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? TCG_OK : tcg::host::fail_launch(what, e);
}

}  // namespace

extern "C" {

size_t tcg_moe_balance_workspace_size(void) { return tcg::host::kWorkspaceHeader + kPartialBytes; }

tcg_status tcg_moe_balance(int tokens, int experts, int k, tcg_dtype dtype, const void* logits, int ld,
                           const int* topk, int ld_topk, const uint8_t* mask, float coef, int* counts, int* offsets,
                           int* num_valid, float* loss, void* workspace, size_t workspace_bytes, void* stream) {
    Balance p = {};
    tcg_status st = start(p, tokens, experts, k, dtype, logits, ld, mask, coef);
    if (st != TCG_OK) return st;
    if (!counts || !num_valid || !loss || (tokens > 0 && (!topk || ld_topk < k))) return TCG_ERR_INVALID_ARG;
    if (!aligned(topk, 4) || !aligned(counts, 4) || !aligned(offsets, 4) || !aligned(num_valid, 4) || !aligned(loss, 4))
        return TCG_ERR_MISALIGNED;
    tcg::host::Device dev;
    if ((st = tcg::host::device(dev)) != TCG_OK) return st;
    if (!workspace || !aligned(workspace, 16) || workspace_bytes < tcg_moe_balance_workspace_size())
        return tcg::host::fail(TCG_ERR_WORKSPACE, "workspace NULL, not 16-byte aligned or smaller than tcg_moe_balance_workspace_size");
    p.topk = topk;
    p.ld_topk = ld_topk;
    p.counts = counts;
    p.offsets = offsets;
    p.valid = num_valid;
    p.loss = loss;
    char* ws = static_cast<char*>(workspace);
    p.arrivals = reinterpret_cast<int*>(ws + 128);
    p.part_p = reinterpret_cast<float*>(ws + tcg::host::kWorkspaceHeader);
    p.part_c = reinterpret_cast<int*>(p.part_p + static_cast<size_t>(kMaxCtas) * kMaxExperts);
    p.part_n = p.part_c + static_cast<size_t>(kMaxCtas) * kMaxExperts;
    const int per_cta = kWarps * (32 / p.lanes);
    const int ctas = std::max(1, std::min({kMaxCtas, dev.num_sms, (tokens + per_cta - 1) / per_cta}));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == TCG_BF16) launch_forward<__nv_bfloat16>(p, ctas, s);
    else if (dtype == TCG_F16) launch_forward<__half>(p, ctas, s);
    else launch_forward<float>(p, ctas, s);
    return launched("tcg_moe_balance");
}

tcg_status tcg_moe_balance_backward(int tokens, int experts, int k, tcg_dtype dtype, const void* logits, int ld,
                                    const uint8_t* mask, float coef, const int* counts, const int* num_valid,
                                    const float* grad_loss, void* dlogits, int ldd, tcg_dtype d_dtype, void* stream) {
    if (d_dtype != TCG_BF16 && d_dtype != TCG_F16 && d_dtype != TCG_F32) return TCG_ERR_INVALID_ARG;
    Balance p = {};
    tcg_status st = start(p, tokens, experts, k, dtype, logits, ld, mask, coef);
    if (st != TCG_OK) return st;
    if (tokens == 0) return TCG_OK;
    if (!counts || !num_valid || !grad_loss || !dlogits || ldd < experts) return TCG_ERR_INVALID_ARG;
    if (!aligned(counts, 4) || !aligned(num_valid, 4) || !aligned(grad_loss, 4) || !aligned(dlogits, size_of(d_dtype)))
        return TCG_ERR_MISALIGNED;
    tcg::host::Device dev;
    if ((st = tcg::host::device(dev)) != TCG_OK) return st;
    p.counts = const_cast<int*>(counts);
    p.valid = const_cast<int*>(num_valid);
    p.grad = grad_loss;
    p.dlogits = dlogits;
    p.ldd = ldd;
    p.d_dtype = d_dtype;
    p.d_vec = aligned(dlogits, 16) && (static_cast<long long>(ldd) * size_of(d_dtype)) % 16 == 0;
    const long long per_cta = 8LL * (32 / p.lanes);
    const int ctas = static_cast<int>(std::max(1LL, std::min<long long>(8LL * dev.num_sms, (tokens + per_cta - 1) / per_cta)));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == TCG_BF16) launch_backward<__nv_bfloat16>(p, ctas, s);
    else if (dtype == TCG_F16) launch_backward<__half>(p, ctas, s);
    else launch_backward<float>(p, ctas, s);
    return launched("tcg_moe_balance_backward");
}

}  // extern "C"
