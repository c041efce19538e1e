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
// all -inf has p = 0, and gradient 0 as masked ones have, whatever g is.  Statistics and sums are fp32.
//
// Bound by memory on paper (logits once forward; once more, and their
// gradient, backward: 5 us for 32768 x 256), in fact by latencies at that size
// (forward 16.7, backward 17.0, one after the other 29.8 us): both issue in
// 42-44 % of the cycles, the forward's largest stall is its barriers (eight
// in the tree over the warps' column sums; then the totals, and one CTA that
// finishes alone), the backward's the wait for a row's loads.  Few tokens are
// bound by the launch.  P_e sums stay in the registers
// of the lane that owns the columns.  A CTA's sums are added to fixed-point
// totals in the workspace, three 64-bit words an expert (integer sums do not
// depend on the order of arrival, and 2^-136 steps lose nothing of an fp32 sum
// above 2^-113), which the last CTA reads in one go and leaves at zero; sums of
// every CTA read back one after the other took 10 us more.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <climits>
#include <cstdint>
#include <type_traits>

#include "host.h"
#include "ptx.cuh"

namespace {

constexpr int kMaxExperts = tcg::host::kMaxBalanceExperts;
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
// Words of a total, in units of 2^-32, 2^-84 and 2^-136: the lower ones hold 52
// bits of each CTA's sum, so that 2^11 CTAs' fit.
constexpr int kWords = 3, kWordBits = 52;
static_assert(kMaxExperts * (8 * kWords + 4) + 8 <= tcg::host::kBalanceBytes, "the totals fit their range of the workspace");
// rows that a warp has on their way at once, by chunks of eight values a lane
__host__ __device__ constexpr int rows_in_flight(int chunks) { return chunks == 2 ? 2 : 1; }

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
    unsigned long long* total_p;   // [kWords][kMaxExperts]
    int* total_c;                  // [experts]
    int* total_n;
    int* arrivals;
    const float* grad;
    void* dlogits;
    long long ldd;
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

// Eight values from a 16-byte aligned address.
template <typename T>
__device__ __forceinline__ void load8(const T* src, float (&x)[8]) {
    const uint4 q = *reinterpret_cast<const uint4*>(src);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    if constexpr (sizeof(T) == 4) {
        const uint4 q2 = *(reinterpret_cast<const uint4*>(src) + 1);
        const uint32_t w2[4] = {q2.x, q2.y, q2.z, q2.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = __uint_as_float(w[i]);
            x[4 + i] = __uint_as_float(w2[i]);
        }
    } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
}

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

// kL lanes hold a row, kC chunks of eight columns each: column (chunk * kL + l)
// * 8 + i; -inf
// past the experts and in a row that does not count.
template <typename T, int kL, int kC>
__device__ __forceinline__ void load_row(const Balance& p, long long t, int l, bool in, float (&x)[kC][8]) {
    const T* row = static_cast<const T*>(p.logits) + t * p.ld;
#pragma unroll
    for (int c = 0; c < kC; ++c) {
        const int e0 = (c * kL + l) * 8;
        if (in && p.vec && e0 + 8 <= p.experts) {
            load8<T>(row + e0, x[c]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[c][i] = in && e0 + i < p.experts ? to_float<T>(row[e0 + i]) : -INFINITY;
        }
    }
}

// x becomes exp(x - max), 0 past the experts; returns 1 / their sum (0 for a row
// of nothing but -inf).
template <int kL, int kC>
__device__ __forceinline__ float exp_row(float (&x)[kC][8]) {
    float m = -INFINITY;
#pragma unroll
    for (int c = 0; c < kC; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, x[c][i]);
#pragma unroll
    for (int d = 1; d < kL; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    if (m == -INFINITY) m = 0.0f;
    float s = 0.0f;
#pragma unroll
    for (int c = 0; c < kC; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[c][i] = expf(x[c][i] - m);
            s += x[c][i];
        }
#pragma unroll
    for (int d = 1; d < kL; d <<= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    return s == 0.0f ? 0.0f : 1.0f / s;
}

// Adds s >= 0 to a total, exactly down to the last word's unit: s is 24 bits
// from bit b of the fixed-point number on, which reach into two words at most
// (sums of 2^-8 and more, the ordinary ones, into the first alone).  A sum that
// is not a number sets the first word's top bit, which totals of at most 2^31
// tokens never reach.
__device__ __forceinline__ void add_total(unsigned long long* total, float s) {
    if (!(s <= 2147483648.0f)) {
        atomicOr(total, 1ull << 63);
        return;
    }
    const uint32_t bits = __float_as_uint(s) & 0x7FFFFFFFu, e = bits >> 23;
    unsigned long long m = (bits & 0x7FFFFFu) | (e ? 0x800000u : 0u);
    int b = static_cast<int>(e ? e : 1u) - 150 + (32 + (kWords - 1) * kWordBits);
    if (b < 0) {
        m = (m + (1ull << (-b - 1))) >> -b;
        b = 0;
    }
    const int word = max(kWords - 1 - b / kWordBits, 0), off = b - (kWords - 1 - word) * kWordBits;
    unsigned long long here = m << off, above = 0ull;
    if (word > 0) {
        above = m >> (kWordBits - off);
        here &= (1ull << kWordBits) - 1;
    }
    if (here) atomicAdd(total + word * kMaxExperts, here);
    if (above) atomicAdd(total + (word - 1) * kMaxExperts, above);
}

// The total as a float (its words' sum in 64 bits, rounded once), left at zero.
__device__ __forceinline__ float take_total(unsigned long long* total) {
    unsigned long long w[kWords];
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = __ldcg(total + i * kMaxExperts);
    double v = 0.0;
#pragma unroll
    for (int i = kWords - 1; i >= 0; --i) {
        if (w[i] == 0ull) continue;
        constexpr double kUnit[kWords] = {0x1p-32, 0x1p-84, 0x1p-136};
        v += static_cast<double>(w[i]) * kUnit[i];
        total[i * kMaxExperts] = 0ull;
    }
    return w[0] >> 63 ? __int_as_float(0x7FC00000) : static_cast<float>(v);
}

template <typename T, int kL, int kC>
__global__ void __launch_bounds__(kThreads) balance_kernel(const __grid_constant__ Balance p) {
    tcg::host::wait_for_kernel_ahead();
    constexpr int kR = rows_in_flight(kC);
    __shared__ float sums[kWarps / 2 * kMaxExperts];
    __shared__ int hist[kMaxExperts];
    __shared__ int n_valid, last;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int l = lane & (kL - 1), slot = lane / kL, per_warp = 32 / kL;
    for (int e = threadIdx.x; e < p.experts; e += kThreads) hist[e] = 0;
    if (threadIdx.x == 0) n_valid = 0;
    __syncthreads();
    // this CTA's tokens
    const int t0 = static_cast<int>(static_cast<long long>(blockIdx.x) * p.tokens / gridDim.x);
    const int t1 = static_cast<int>(static_cast<long long>(blockIdx.x + 1) * p.tokens / gridDim.x);

    for (int t = t0 + static_cast<int>(threadIdx.x); t < t1; t += kThreads) {
        if (p.mask && !p.mask[t]) continue;
        const int* row = p.topk + t * p.ld_topk;
#pragma unroll 4
        for (int j = 0; j < p.k; ++j) {
            const int e = __ldg(row + j);
            if (e >= 0 && e < p.experts) atomicAdd(&hist[e], 1);
        }
    }
    float acc[kC][8];
#pragma unroll
    for (int c = 0; c < kC; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[c][i] = 0.0f;
    int n = 0;
    const int step = kWarps * per_warp;
    for (int tb = t0 + warp * per_warp; tb < t1; tb += kR * step) {
        float x[kR][kC][8];
#pragma unroll
        for (int r = 0; r < kR; ++r) {
            const int t = tb + r * step + slot;
            const bool in = t < t1 && (!p.mask || p.mask[t]);
            load_row<T, kL, kC>(p, t, l, in, x[r]);
            if (in && l == 0) ++n;
        }
#pragma unroll
        for (int r = 0; r < kR; ++r) {
            const float inv = exp_row<kL, kC>(x[r]);
#pragma unroll
            for (int c = 0; c < kC; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[c][i] = fmaf(x[r][c][i], inv, acc[c][i]);
        }
    }
    if (n) atomicAdd(&n_valid, n);
    // rows of one warp, then of the CTA's warps, in a fixed order
#pragma unroll
    for (int c = 0; c < kC; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int d = kL; d < 32; d <<= 1) acc[c][i] += __shfl_xor_sync(0xffffffffu, acc[c][i], d);
    for (int half = kWarps / 2; half > 0; half >>= 1) {
        __syncthreads();
        if (warp >= half && warp < 2 * half && slot == 0) {
#pragma unroll
            for (int c = 0; c < kC; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int e = (c * kL + l) * 8 + i;
                    if (e < p.experts) sums[(warp - half) * p.experts + e] = acc[c][i];
                }
        }
        __syncthreads();
        if (warp < half && slot == 0) {
#pragma unroll
            for (int c = 0; c < kC; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int e = (c * kL + l) * 8 + i;
                    if (e < p.experts) acc[c][i] += sums[warp * p.experts + e];
                }
        }
    }
    __syncthreads();
    if (warp == 0 && slot == 0) {
#pragma unroll
        for (int c = 0; c < kC; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int e = (c * kL + l) * 8 + i;
                if (e < p.experts) sums[e] = acc[c][i];
            }
    }
    __syncthreads();
    const bool alone = gridDim.x == 1;
    if (!alone) {
        for (int e = threadIdx.x; e < p.experts; e += kThreads) {
            add_total(p.total_p + e, sums[e]);
            if (hist[e]) atomicAdd(p.total_c + e, hist[e]);
        }
        if (threadIdx.x == 0 && n_valid) atomicAdd(p.total_n, n_valid);
        __syncthreads();
        if (threadIdx.x == 0) {
            __threadfence();
            const int old = tcg::ptx::atomic_add_acq_rel_gpu(p.arrivals, 1);
            last = old == static_cast<int>(gridDim.x) - 1;
        }
        __syncthreads();
        if (!last) return;
        // The last CTA: the totals, left at zero for the next call.
        for (int e = threadIdx.x; e < p.experts; e += kThreads) {
            sums[e] = take_total(p.total_p + e);
            hist[e] = __ldcg(p.total_c + e);
            p.total_c[e] = 0;
        }
        if (threadIdx.x == 0) {
            n_valid = __ldcg(p.total_n);
            *p.total_n = 0;
            *p.arrivals = 0;
        }
        __syncthreads();
    }
    const float inv_n = n_valid > 0 ? 1.0f / static_cast<float>(n_valid) : 0.0f;
    float mine = 0.0f;
    for (int e = threadIdx.x; e < p.experts; e += kThreads) {
        p.counts[e] = hist[e];
        mine += (static_cast<float>(hist[e]) * inv_n) * (sums[e] * inv_n);
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) mine += __shfl_xor_sync(0xffffffffu, mine, d);
    float* red = sums + kMaxExperts;
    if (lane == 0) red[warp] = mine;
    __syncthreads();
    if (threadIdx.x == 0) {
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) sum += red[w];
        *p.loss = p.coef * (static_cast<float>(p.experts) / static_cast<float>(p.k)) * sum;
        *p.valid = n_valid;
    }
    if (p.offsets && warp == kWarps - 1) {
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

template <typename T, int kL, int kC>
__global__ void __launch_bounds__(256) balance_grad_kernel(const __grid_constant__ Balance p) {
    tcg::host::wait_for_kernel_ahead();
    constexpr int kR = rows_in_flight(kC);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int l = lane & (kL - 1), slot = lane / kL, per_warp = 32 / kL;
    const long long step = static_cast<long long>(gridDim.x) * 8 * per_warp;
    const int n = __ldg(p.valid);
    const float inv_n = n > 0 ? 1.0f / static_cast<float>(n) : 0.0f;
    const float to_f = static_cast<float>(p.experts) / static_cast<float>(p.k) * inv_n;
    const float g = __ldg(p.grad) * p.coef * inv_n;
    float f[kC][8];
#pragma unroll
    for (int c = 0; c < kC; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int e = (c * kL + l) * 8 + i;
            f[c][i] = e < p.experts ? static_cast<float>(__ldg(p.counts + e)) * to_f : 0.0f;
        }
    for (long long tb = (static_cast<long long>(blockIdx.x) * 8 + warp) * per_warp; tb < p.tokens; tb += kR * step) {
        float x[kR][kC][8];
#pragma unroll
        for (int r = 0; r < kR; ++r) {
            const long long t = tb + r * step + slot;
            load_row<T, kL, kC>(p, t, l, t < p.tokens && (!p.mask || p.mask[t]), x[r]);
        }
#pragma unroll
        for (int r = 0; r < kR; ++r) {
            const long long t = tb + r * step + slot;
            const float inv = exp_row<kL, kC>(x[r]);
            float dot = 0.0f;
#pragma unroll
            for (int c = 0; c < kC; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) dot = fmaf(f[c][i], x[r][c][i], dot);
#pragma unroll
            for (int d = 1; d < kL; d <<= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
            dot *= inv;
            // (a row of nothing, masked or all -inf, has gradient 0 whatever g is)
            const float gi = inv == 0.0f ? 0.0f : g * inv;
            if (t < p.tokens) {
#pragma unroll
                for (int c = 0; c < kC; ++c) {
                    float d[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) d[i] = (x[r][c][i] * gi) * (f[c][i] - dot);
                    store_grad(p, t, (c * kL + l) * 8, d);
                }
            }
        }
    }
}

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
int size_of(tcg_dtype t) { return t == TCG_F32 ? 4 : 2; }

tcg_status start(Balance& p, int tokens, int experts, int k, tcg_dtype dtype, const void* logits, int ld,
                 const uint8_t* mask, float coef) {
    if (tokens < 0 || experts < 1 || k < 1) return TCG_ERR_INVALID_ARG;
    if (dtype != TCG_BF16 && dtype != TCG_F16 && dtype != TCG_F32) return TCG_ERR_INVALID_ARG;
    if (experts > kMaxExperts || tokens > tcg::host::kMaxExtent) return TCG_ERR_UNSUPPORTED;
    if (tokens > 0 && (!logits || ld < experts)) return TCG_ERR_INVALID_ARG;
    if (!aligned(logits, size_of(dtype))) return TCG_ERR_MISALIGNED;
    p.logits = logits;
    p.ld = ld;
    p.mask = mask;
    p.tokens = tokens;
    p.experts = experts;
    p.k = k;
    p.coef = coef;
    p.vec = aligned(logits, 16) && (static_cast<long long>(ld) * size_of(dtype)) % 16 == 0;
    return TCG_OK;
}

// Lanes that hold a row and chunks of eight values a lane.  Few lanes with many
// values: the steps across lanes, the row's address and its reciprocal are then
// shared by more rows of the warp (32768 x 256, forward and backward: 20.9 +
// 22.3 us with 32 lanes of 8 values).
int chunks_of(int experts) { return experts <= 64 ? 2 : 4; }
int lanes_of(int experts) {
    const int per = 8 * chunks_of(experts);
    int lanes = 1;
    while (lanes * per < experts) lanes *= 2;
    return lanes;
}

template <typename T, typename F>
void with_shape(int experts, F f) {
    using std::integral_constant;
    if (chunks_of(experts) == 2) {
        switch (lanes_of(experts)) {
            case 1: return f(T{}, integral_constant<int, 1>{}, integral_constant<int, 2>{});
            case 2: return f(T{}, integral_constant<int, 2>{}, integral_constant<int, 2>{});
            default: return f(T{}, integral_constant<int, 4>{}, integral_constant<int, 2>{});
        }
    }
    switch (lanes_of(experts)) {
        case 4: return f(T{}, integral_constant<int, 4>{}, integral_constant<int, 4>{});
        case 8: return f(T{}, integral_constant<int, 8>{}, integral_constant<int, 4>{});
        case 16: return f(T{}, integral_constant<int, 16>{}, integral_constant<int, 4>{});
        default: return f(T{}, integral_constant<int, 32>{}, integral_constant<int, 4>{});
    }
}
template <typename F>
void with_types(tcg_dtype dtype, int experts, F f) {
    if (dtype == TCG_BF16) with_shape<__nv_bfloat16>(experts, f);
    else if (dtype == TCG_F16) with_shape<__half>(experts, f);
    else with_shape<float>(experts, f);
}

tcg_status launched(cudaError_t e, const char* what) { return e == cudaSuccess ? TCG_OK : tcg::host::fail_launch(what, e); }

}  // namespace

extern "C" {

size_t tcg_moe_balance_workspace_size(void) { return tcg::host::kScratchAt; }

tcg_status tcg_moe_balance(int tokens, int experts, int k, tcg_dtype dtype, const void* logits, int ld,
                           const int* topk, int ld_topk, const uint8_t* mask, float coef, int* counts, int* offsets,
                           int* num_valid, float* loss, void* workspace, size_t workspace_bytes, void* stream) {
    Balance p = {};
    tcg_status st = start(p, tokens, experts, k, dtype, logits, ld, mask, coef);
    if (st != TCG_OK) return st;
    // (counts and offsets are ints)
    if (static_cast<long long>(tokens) * k > INT_MAX) return TCG_ERR_UNSUPPORTED;
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
    p.total_p = reinterpret_cast<unsigned long long*>(ws + tcg::host::kBalanceAt);
    p.total_c = reinterpret_cast<int*>(p.total_p + kWords * kMaxExperts);
    p.total_n = p.total_c + kMaxExperts;
    p.arrivals = p.total_n + 1;
    const int chunks = chunks_of(experts);
    const int per_cta = kWarps * (32 / lanes_of(experts)) * rows_in_flight(chunks);
    const int ctas = std::max(1, std::min(dev.num_sms, (tokens + per_cta - 1) / per_cta));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t err = cudaSuccess;
    with_types(dtype, experts, [&](auto x, auto l, auto c) {
        err = tcg::host::launch_early(balance_kernel<decltype(x), decltype(l)::value, decltype(c)::value>, dim3(ctas), kThreads, s, p);
    });
    return launched(err, "tcg_moe_balance");
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
    const long long per_cta = 8LL * (32 / lanes_of(experts)) * rows_in_flight(chunks_of(experts));
    const int ctas = static_cast<int>(std::max(1LL, std::min<long long>(4LL * dev.num_sms, (tokens + per_cta - 1) / per_cta)));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t err = cudaSuccess;
    with_types(dtype, experts, [&](auto x, auto l, auto c) {
        err = tcg::host::launch_early(balance_grad_kernel<decltype(x), decltype(l)::value, decltype(c)::value>, dim3(ctas), 256, s, p);
    });
    return launched(err, "tcg_moe_balance_backward");
}

}  // extern "C"
