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
// that sort alike; a lane sorts its own in runs of eight and leaves them in
// shared memory, and each round takes the warp's largest head in one reduction,
// after which the lane that had it reads its next.  16-bit logits share a
// 32-bit key with the expert's number, so keys differ; an fp32 logit takes all 32
// bits, of equal ones the lowest lane has the lower expert, and the expert's
// number is found at the end, for all of a row's choices at once.  Weights, their
// gradients and the chosen logits are worked on k lanes a row, for as many rows
// as fit a warp.  Statistics are fp32.
//
// Most of the time goes to instructions (a row of 256 bf16 logits, eight chosen:
// about 310, most of them integer compares and selects, which issue every other
// cycle: 59 % of the issue slots, 62 % of the ALU pipe), the rest to waiting for
// the row, of which a warp has one under way (all keys are made and sorted before
// the next is asked for); memory's part is 2.5 us each way.  32768 x 256, one call after the
// other in a graph: forward 13.1 us, backward 7.4 (over all experts 16.1 and
// 12.1; fp32 logits 19.8 and 11.6).  Steps that helped, both ways and calls
// included: one reduction a round on keys that hold the expert's number, in place
// of value, then place (37 us); runs sorted once in place of a search after each
// round (29); a row's k weights on k lanes, so that exponentials and divisions
// serve several rows (27); heads replaced under a predicate, without a branch
// (24); zeros first and then the few chosen, where the gradient has no others (22).
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
constexpr int kWarps = 4;
// CTAs an SM is to hold, forward and backward
constexpr int resident(int n, bool grad) { return n > 8 ? 4 : grad ? 8 : 10; }
constexpr uint32_t kAll = 0xFFFFFFFFu;

struct Route {
    const void* logits;
    long long ld;
    const uint8_t* mask;
    int tokens, experts, k;
    int width;        // lanes of k places: a power of two
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

// A lane's kN experts of a row: fp32 values, or words of two 16-bit ones.
template <typename T, int kN>
struct Row {
    static constexpr int kBytes = kN * static_cast<int>(sizeof(T)), kWords = (kBytes + 3) / 4;
    uint32_t w[kWords];

    __device__ __forceinline__ float value(int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else if constexpr (std::is_same<T, __half>::value)
            return __half2float(__ushort_as_half(static_cast<unsigned short>(w[i / 2] >> (16 * (i & 1)))));
        else return __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
    }

    // From an address aligned to kBytes, at most 16.
    __device__ __forceinline__ void load(const T* src) {
        if constexpr (kBytes >= 16) {
#pragma unroll
            for (int i = 0; i < kBytes / 16; ++i) {
                const uint4 q = reinterpret_cast<const uint4*>(src)[i];
                w[4 * i] = q.x, w[4 * i + 1] = q.y, w[4 * i + 2] = q.z, w[4 * i + 3] = q.w;
            }
        } else if constexpr (kBytes == 8) {
            const uint2 q = *reinterpret_cast<const uint2*>(src);
            w[0] = q.x, w[1] = q.y;
        } else if constexpr (kBytes == 4) {
            w[0] = *reinterpret_cast<const uint32_t*>(src);
        } else {
            w[0] = *reinterpret_cast<const uint16_t*>(src);
        }
    }

    // The first n of them, -inf for the others.
    __device__ __forceinline__ void load_some(const T* src, int n) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < kN; ++i) w[i] = i < n ? __float_as_uint(src[i]) : 0xFF800000u;
        } else {
            constexpr uint32_t kLow = std::is_same<T, __half>::value ? 0xFC00u : 0xFF80u;
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                const uint32_t lo = 2 * i < n ? reinterpret_cast<const uint16_t*>(src)[2 * i] : kLow;
                const uint32_t hi = 2 * i + 1 < n ? reinterpret_cast<const uint16_t*>(src)[2 * i + 1] : kLow;
                w[i] = lo | hi << 16;
            }
        }
    }
};

template <typename T, int kN>
__device__ __forceinline__ void load_row(const Route& p, long long t, int lane, Row<T, kN>& x) {
    const T* src = static_cast<const T*>(p.logits) + t * p.ld + lane * kN;
    const int left = p.experts - lane * kN;
    if (p.vec && left >= kN) x.load(src);
    else x.load_some(src, left);
}

// Integers that sort as the values do.  NaN is the largest, both zeros are one,
// and what stands for -inf is below kFloor.  A 16-bit value's key ends in the
// expert's number turned over, so that of equal values the lower expert has the
// larger key; an fp32 value has all 32 bits.
template <typename T>
struct Keys {   // 16-bit values
    static constexpr uint32_t kFloor = std::is_same<T, __half>::value ? 0x04000000u : 0x00800000u;

    // Experts i and i + 1 of a row, `turned` the first one's number turned over.
    template <int kN>
    static __device__ __forceinline__ void make2(const Row<T, kN>& x, int i, uint32_t turned, uint32_t& k0, uint32_t& k1) {
        // (adding zero makes -0 into +0, and every NaN into the positive one)
        uint32_t w = x.w[i / 2];
        if constexpr (std::is_same<T, __half>::value) {
            const __half2 v = __hadd2(*reinterpret_cast<const __half2*>(&w), __float2half2_rn(0.0f));
            w = *reinterpret_cast<const uint32_t*>(&v);
        } else {
            const __nv_bfloat162 v = __hadd2(*reinterpret_cast<const __nv_bfloat162*>(&w), __float2bfloat162_rn(0.0f));
            w = *reinterpret_cast<const uint32_t*>(&v);
        }
        k0 = make(w << 16, turned);
        k1 = make(w, turned - 1u);
    }
    static __device__ __forceinline__ uint32_t make(uint32_t x, uint32_t turned) {
        const uint32_t o = x ^ (static_cast<uint32_t>(static_cast<int>(x) >> 31) | 0x80000000u);
        return __byte_perm(o, turned, 0x3254);   // o's upper half over the number
    }
    static __device__ __forceinline__ float value(uint32_t key) {
        const uint32_t x = (key & 0x80000000u ? key ^ 0x80000000u : ~key) & 0xFFFF0000u;
        if constexpr (std::is_same<T, __half>::value) return __half2float(__ushort_as_half(static_cast<unsigned short>(x >> 16)));
        else return __uint_as_float(x);
    }
};
template <>
struct Keys<float> {
    static constexpr uint32_t kFloor = 0x00800000u;

    static __device__ __forceinline__ uint32_t make(float v) {
        const uint32_t x = __float_as_uint(v + 0.0f);
        return v != v ? 0xFFFFFFFFu : x ^ (static_cast<uint32_t>(static_cast<int>(x) >> 31) | 0x80000000u);
    }
    template <int kN>
    static __device__ __forceinline__ void make2(const Row<float, kN>& x, int i, uint32_t, uint32_t& k0, uint32_t& k1) {
        k0 = make(x.value(i));
        k1 = make(x.value(i + 1 < kN ? i + 1 : i));
    }
    static __device__ __forceinline__ float value(uint32_t key) {
        return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
    }
};

// Where the head was taken, the run's next key takes its place (no branch: one
// lane of 32 does it).
__device__ __forceinline__ void advance(uint32_t& head, uint32_t& next, bool taken) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %2, 0;\n\t"
        "@p ld.shared.u32 %0, [%1];\n\t"
        "@p add.u32 %1, %1, 4;\n\t}"
        : "+r"(head), "+r"(next)
        : "r"(static_cast<uint32_t>(taken))
        : "memory");
}

// Falling order, for one, two, four or eight keys (odd-even merges).
template <int kL>
__device__ __forceinline__ void sort_run(uint32_t (&k)[kL]) {
    auto order = [&](int i, int j) {
        const uint32_t a = k[i], b = k[j];
        k[i] = max(a, b);
        k[j] = min(a, b);
    };
    if constexpr (kL >= 2) {
#pragma unroll
        for (int i = 0; i < kL; i += 2) order(i, i + 1);
    }
    if constexpr (kL >= 4) {
#pragma unroll
        for (int i = 0; i < kL; i += 4) {
            order(i, i + 2);
            order(i + 1, i + 3);
            order(i + 1, i + 2);
        }
    }
    if constexpr (kL >= 8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) order(i, i + 4);
        order(2, 4);
        order(3, 5);
        order(1, 2);
        order(3, 4);
        order(5, 6);
    }
}

// Sums and maxima over neighbouring lanes, width of them (a power of two).
__device__ __forceinline__ float lanes_sum(float v, int width = 32) {
    for (int d = width >> 1; d > 0; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
    return v;
}
__device__ __forceinline__ float lanes_max(float v, int width = 32) {
    for (int d = width >> 1; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, d));
    return v;
}

// This warp's tokens: a run of neighbours.
struct Run {
    long long t0, t1;
};
__device__ __forceinline__ Run run_of(const Route& p) {
    const long long w = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5), n = static_cast<long long>(gridDim.x) * kWarps;
    return {p.tokens * w / n, p.tokens * (w + 1) / n};
}

// The largest logit of a row, kN a lane (0 where all are -inf).
template <typename T, int kN>
__device__ __forceinline__ float row_max(const Row<T, kN>& x) {
    float m = x.value(0);
#pragma unroll
    for (int i = 1; i < kN; ++i) m = fmaxf(m, x.value(i));
    m = lanes_max(m);
    return m == -INFINITY ? 0.0f : m;
}

template <typename T, int kN>
__global__ void __launch_bounds__(32 * kWarps, resident(kN, false)) route_kernel(const __grid_constant__ Route p) {
    tcg::host::wait_for_kernel_ahead();
    using K = Keys<T>;
    constexpr bool kWide = sizeof(T) == 4;   // equal keys are possible
    constexpr int kL = kN < 8 ? kN : 8, kRuns = kN / kL;
    // each run ends in a key that is below any
    __shared__ uint32_t sorted[kWarps][32 * kRuns * (kL + 1)];
    const int lane = threadIdx.x & 31;
    uint32_t* mine = sorted[threadIdx.x >> 5] + lane * kRuns * (kL + 1);
    const uint32_t mine_at = static_cast<uint32_t>(__cvta_generic_to_shared(mine));
#pragma unroll
    for (int g = 0; g < kRuns; ++g) mine[g * (kL + 1) + kL] = 0u;
    const int slot = lane / p.width, place = lane - slot * p.width, fit = 32 / p.width;
    const Run tokens = run_of(p);
    for (long long tb = tokens.t0; tb < tokens.t1; tb += fit) {
        const int rows = static_cast<int>(min(static_cast<long long>(fit), tokens.t1 - tb));
        // lane (slot, place): the place's choice of row tb + slot
        uint32_t my_key = 0u;
        int my_e = -1;
        float my_sum = 0.0f;
        for (int r = 0; r < rows; ++r) {
            const long long t = tb + r;
            if (p.mask && !p.mask[t]) continue;
            Row<T, kN> x;
            load_row<T, kN>(p, t, lane, x);
            uint32_t head[kRuns], next[kRuns];   // next: shared addresses
            uint32_t keys[kWide ? kN : 1];
#pragma unroll
            for (int g = 0; g < kRuns; ++g) {
                uint32_t run[kL];
                const uint32_t turned = 0xFFFFu - static_cast<uint32_t>(lane * kN + g * kL);
                if constexpr (kL == 1) {
                    uint32_t other;
                    K::make2(x, 0, turned, run[0], other);
                } else {
#pragma unroll
                    for (int i = 0; i < kL; i += 2) K::make2(x, g * kL + i, turned - i, run[i], run[i + 1]);
                }
                if constexpr (kWide) {
#pragma unroll
                    for (int i = 0; i < kL; ++i) keys[g * kL + i] = run[i];
                }
                sort_run<kL>(run);
                // (only this lane reads them)
#pragma unroll
                for (int i = 1; i < kL; ++i) mine[g * (kL + 1) + i] = run[i];
                head[g] = run[0];
                next[g] = mine_at + (g * (kL + 1) + 1) * 4u;
            }
            const int from = r * p.width, last = from + p.k;
            if constexpr (kWide) {
                // A choice is its key, the lowest lane that holds it, and how many equal ones that lane gave before.
                uint32_t before = 0u;
                int holder = -1, nth = 0, my_holder = 0, my_nth = 0;
                for (int to = from; to < last; ++to) {
                    uint32_t most = head[0];
#pragma unroll
                    for (int g = 1; g < kRuns; ++g) most = max(most, head[g]);
                    const uint32_t best = __reduce_max_sync(kAll, most);
                    const int owner = __ffs(__ballot_sync(kAll, most == best)) - 1;
                    nth = best == before && owner == holder ? nth + 1 : 0;
                    before = best;
                    holder = owner;
                    if (lane == to) my_key = best, my_holder = owner, my_nth = nth;
                    bool open = lane == owner && best >= K::kFloor;   // nothing below the floor is ever taken
#pragma unroll
                    for (int g = 0; g < kRuns; ++g) {
                        const bool here = open && head[g] == best;
                        advance(head[g], next[g], here);
                        open = open && !here;
                    }
                }
                // ... and so its expert is the nth of the lane's that have that key.
                const bool of_row = lane >= from && lane < last && my_key >= K::kFloor;
#pragma unroll
                for (int i = 0; i < kN; ++i) {
                    const uint32_t key = __shfl_sync(kAll, keys[i], my_holder);
                    if (of_row && key == my_key && my_nth-- == 0) my_e = my_holder * kN + i;
                }
            } else {
                for (int to = from; to < last; ++to) {
                    uint32_t most = head[0];
#pragma unroll
                    for (int g = 1; g < kRuns; ++g) most = max(most, head[g]);
                    const uint32_t best = __reduce_max_sync(kAll, most);
                    if (lane == to) my_key = best;
#pragma unroll
                    for (int g = 0; g < kRuns; ++g) advance(head[g], next[g], head[g] == best && best >= K::kFloor);
                }
            }
            if (!p.chosen_only) {
                const float m = K::value(__shfl_sync(kAll, my_key, from));
                float s = 0.0f;
#pragma unroll
                for (int i = 0; i < kN; ++i) s += expf(x.value(i) - m);
                s = lanes_sum(s);
                if (slot == r) my_sum = s;
            }
        }
        // (a row's first choice has its largest logit; rows without one have no choice at all)
        if (!kWide && my_key >= K::kFloor) my_e = 0xFFFF - static_cast<int>(my_key & 0xFFFFu);
        const float v = K::value(my_key), m = __shfl_sync(kAll, v, slot * p.width);
        const float z = my_e >= 0 ? expf(v - m) : 0.0f;
        const float s = lanes_sum(z, p.width);
        if (slot < rows && place < p.k) {
            p.topk[(tb + slot) * p.ld_topk + place] = my_e;
            p.weights[(tb + slot) * p.ld_weights + place] = my_e >= 0 ? z / (p.chosen_only ? s : my_sum) : 0.0f;
        }
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
        if (p.accumulate) {
            Row<D, kN> old;
            old.load(row + e0);
#pragma unroll
            for (int i = 0; i < kN; ++i) v[i] = from_float<D>(old.value(i) + d[i]);
        } else {
#pragma unroll
            for (int i = 0; i < kN; ++i) v[i] = from_float<D>(d[i]);
        }
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

template <int kN>
__device__ __forceinline__ void store_typed(const Route& p, long long t, int lane, const float (&d)[kN]) {
    if (p.d_dtype == TCG_F32) store_lane<float, kN>(p, t, lane, d);
    else if (p.d_dtype == TCG_F16) store_lane<__half, kN>(p, t, lane, d);
    else store_lane<__nv_bfloat16, kN>(p, t, lane, d);
}

template <typename T, int kN>
__global__ void __launch_bounds__(32 * kWarps, resident(kN, true)) route_grad_kernel(const __grid_constant__ Route p) {
    tcg::host::wait_for_kernel_ahead();
    // Per warp a row of what the chosen experts get, zeros elsewhere and between rows.
    __shared__ alignas(16) float given[kWarps][32 * kN];
    const int lane = threadIdx.x & 31;
    float* row = given[threadIdx.x >> 5];
    float* mine = row + lane * kN;
#pragma unroll
    for (int i = 0; i < kN; ++i) mine[i] = 0.0f;
    __syncwarp();
    const int slot = lane / p.width, place = lane - slot * p.width, fit = 32 / p.width;
    const uint32_t of_slot = (p.width == 32 ? kAll : (1u << p.width) - 1u) << (slot * p.width);
    const Run tokens = run_of(p);
    for (long long tb = tokens.t0; tb < tokens.t1; tb += fit) {
        const int rows = static_cast<int>(min(static_cast<long long>(fit), tokens.t1 - tb));
        // lane (slot, place): the place's expert in row tb + slot, and what it gets
        const long long my_t = tb + slot;
        int e = slot < rows && place < p.k ? p.topk[my_t * p.ld_topk + place] : -1;
        if (e >= p.experts) e = -1;
        float g = e >= 0 ? p.grad[my_t * p.ld_grad + place] : 0.0f;
        if (p.chosen_only) {
            const float x = e >= 0 ? to_float(static_cast<const T*>(p.logits)[my_t * p.ld + e]) : -INFINITY;
            float m = lanes_max(x, p.width);
            if (m == -INFINITY) m = 0.0f;
            const float z = expf(x - m);
            const float s = lanes_sum(z, p.width);
            const float w = s == 0.0f ? 0.0f : z / s;
            g = w * (g - lanes_sum(e >= 0 ? w * g : 0.0f, p.width));
        }
        const uint32_t live = __ballot_sync(kAll, e >= 0);
        // an expert named twice gets both, in their order, through the first
        const uint32_t same = __match_any_sync(kAll, e >= 0 ? slot << 16 | e : -1 - lane);
        const bool first = e >= 0 && (same & ((1u << lane) - 1u)) == 0u;
        if (__any_sync(kAll, e >= 0 && !first)) {
            float sum = 0.0f;
            for (int j = 0; j < 32; ++j) {
                const float gj = __shfl_sync(kAll, g, j);
                if (same >> j & 1u) sum += gj;
            }
            g = sum;
        }
        if (p.chosen_only && !p.accumulate) {
            // zeros, then the few that are not
            const float zero[kN] = {};
            for (int r = 0; r < rows; ++r) store_typed<kN>(p, tb + r, lane, zero);
            __syncwarp();
            if (first) {
                const long long at = my_t * p.ldd + e;
                if (p.d_dtype == TCG_F32) static_cast<float*>(p.dlogits)[at] = g;
                else if (p.d_dtype == TCG_F16) static_cast<__half*>(p.dlogits)[at] = __float2half_rn(g);
                else static_cast<__nv_bfloat16*>(p.dlogits)[at] = __float2bfloat16_rn(g);
            }
            continue;
        }
        for (int r = 0; r < rows; ++r) {
            const bool any = (__shfl_sync(kAll, live & of_slot, r * p.width)) != 0u;
            if (!any && p.accumulate) continue;   // a token of nobody adds nothing, whatever its logits hold
            const bool here = first && slot == r;
            if (here) row[e] = g;
            __syncwarp();
            float d[kN];
#pragma unroll
            for (int i = 0; i < kN; ++i) d[i] = mine[i];
            __syncwarp();
            if (here) row[e] = 0.0f;
            __syncwarp();
            if (any && !p.chosen_only) {
                Row<T, kN> x;
                load_row<T, kN>(p, tb + r, lane, x);
                const float m = row_max<T, kN>(x);
                float z[kN], s = 0.0f, inner = 0.0f;
#pragma unroll
                for (int i = 0; i < kN; ++i) {
                    z[i] = expf(x.value(i) - m);
                    s += z[i];
                    inner += z[i] * d[i];
                }
                s = lanes_sum(s);
                const float inv = s == 0.0f ? 0.0f : 1.0f / s;
                inner = lanes_sum(inner) * inv;
#pragma unroll
                for (int i = 0; i < kN; ++i) d[i] = z[i] * inv * (d[i] - inner);
            }
            store_typed<kN>(p, tb + r, lane, d);
        }
    }
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
    for (p.width = 1; p.width < k;) p.width *= 2;
    p.topk = const_cast<int*>(topk);
    p.ld_topk = ld_topk;
    const long long word = std::min(16, lane_experts(experts) * size_of(dtype));
    p.vec = aligned(logits, word) && static_cast<long long>(ld) * size_of(dtype) % word == 0;
    return TCG_OK;
}

tcg_status launched(cudaError_t e, const char* what) { return e == cudaSuccess ? TCG_OK : tcg::host::fail_launch(what, e); }
// A warp a token, up to what the SMs hold at once.
dim3 grid_of(const Route& p, int sms, bool grad) {
    const long long ctas = (static_cast<long long>(p.tokens) + kWarps - 1) / kWarps;
    return dim3(static_cast<unsigned>(std::min<long long>(ctas, static_cast<long long>(sms) * resident(lane_experts(p.experts), grad))));
}

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
        err = tcg::host::launch_early(route_kernel<decltype(x), decltype(n)::value>, grid_of(p, dev.num_sms, false), 32 * kWarps,
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
        err = tcg::host::launch_early(route_grad_kernel<decltype(x), decltype(n)::value>, grid_of(p, dev.num_sms, true), 32 * kWarps,
                                      static_cast<cudaStream_t>(stream), p);
    });
    return launched(err, "tcg_moe_route_backward");
}

}  // extern "C"
