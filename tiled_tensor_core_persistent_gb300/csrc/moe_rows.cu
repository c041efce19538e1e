// moe_rows.cu -- the way of tokens to their experts and back.
//
//   sort      the assignments (t, j) in the order of (expert, t, j): where each
//             expert's rows start, the token of a row, the row of an assignment
//   dispatch  x[row_of[t, j]] = y[t]
//   combine   y[t] = sum_j w_tj x[row_of[t, j]]
//   gradient  dx[row_of[t, j]] = w_tj dy[t],  dw_tj = sum_c dy[t, c] x[row_of[t, j], c]
//
// The sort counts: CTAs own runs of neighbouring assignments and their warps
// runs of those, so a row is the expert's start, plus the expert's assignments
// in the CTAs and warps before, plus its place among equal ones of the warp.
// Two launches (counts per CTA; places), one where a single CTA holds all; the
// second starts while the first runs and counts its own run meanwhile.  Bound by
// latencies: two launches, a load of the assignments in each, the sums over the
// CTAs' counts.  262144 assignments to 256 experts 8.9 us in a graph, 128 to 16
// 2.7.  What helped: a thread's loads four at a time (2.7 us off), four experts'
// counts a load and the starts by all warps (0.7), the first batch kept (0.4).
//
// The other three go by tokens, so that a token's row is read or written once
// however many experts it has, and each expert's row once.  Bound by memory:
// 16384 tokens x 2 rows of 4096 bf16 values, dispatch and its gradient 124 us
// (800 MB, 6.4 TB/s, 0.95 of the copy rate), combine and both gradients 166 us
// (1070 MB in the two calls, 6.4 TB/s, 0.96).  Rows that start anywhere take half to
// four fifths longer (4095 columns: dispatch 91, combine 120 us, its gradient
// 152; whole words 61, 67 and 102): each is read in words that are shifted into place.
#include <algorithm>
#include <climits>
#include <cstdint>

#include "host.h"
#include "split.cuh"
#include "values.cuh"

namespace {

using namespace tcg;

constexpr int kMaxExperts = 1024;
constexpr uint32_t kAll = 0xFFFFFFFFu;

// ------------------------------------------------------------------- sort

constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
// Assignments a CTA takes at least (262144 to 256 experts 8.9 us, 9.3 with 2048;
// 32768 6.2 and 6.6, 6.5 with 512).
constexpr int kSortRun = 1024;
// As many as this are one CTA's, in one launch: 2048 to 16 experts 3.5 us and 4.3
// in two launches, 4096 5.4 and 4.5.
constexpr int kSortAlone = 2048;
// Assignments whose loads a thread has on their way at once.
constexpr int kSortBatch = 4;

struct Sort {
    const int* topk;
    long long ld_topk;
    const uint8_t* mask;
    int total, k, experts;       // total: tokens * k
    uint32_t div_mul;            // a / k = (a + high half of a * div_mul) >> div_shift for 0 <= a < 2^31
    int div_shift;
    int* offsets;
    int* row_token;
    int* row_of;
    long long ld_row_of;
    int* counts;                 // [CTA][pitch_of(experts)], nullptr where one CTA holds all
};

// A CTA's counts start on 16 bytes (what lies past the experts is never used).
__host__ __device__ __forceinline__ int pitch_of(int experts) { return (experts + 3) & ~3; }

struct Assignment {
    int t, j, e;   // e: -1 where it has no expert
};
// Assignments a, a + step, ...: those below end (the others have no expert).
// Both loads of all of them are on their way before one is used.
template <int kStep>
__device__ __forceinline__ void load_batch(const Sort& p, int a, int end, Assignment (&v)[kSortBatch]) {
    uint8_t counts[kSortBatch];
#pragma unroll
    for (int i = 0; i < kSortBatch; ++i) {
        const int at = min(a + i * kStep, p.total - 1);
        v[i].t = static_cast<int>((static_cast<uint32_t>(at) + __umulhi(static_cast<uint32_t>(at), p.div_mul)) >> p.div_shift);
        v[i].j = at - v[i].t * p.k;
        counts[i] = p.mask ? __ldcg(p.mask + v[i].t) : 1;
        v[i].e = __ldcg(p.topk + v[i].t * p.ld_topk + v[i].j);
    }
#pragma unroll
    for (int i = 0; i < kSortBatch; ++i)
        if (!counts[i] || v[i].e < 0 || v[i].e >= p.experts || a + i * kStep >= end) v[i].e = -1;
}

__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(const __grid_constant__ Sort p) {
    __shared__ int hist[kMaxExperts];
    // (the second launch may read the assignments from here on: they were there before this one)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (int e = threadIdx.x; e < p.experts; e += kSortThreads) hist[e] = 0;
    __syncthreads();
    const int a1 = run_start(p.total, blockIdx.x + 1, gridDim.x);
    for (int a = run_start(p.total, blockIdx.x, gridDim.x) + static_cast<int>(threadIdx.x); a < a1; a += kSortBatch * kSortThreads) {
        Assignment v[kSortBatch];
        load_batch<kSortThreads>(p, a, a1, v);
#pragma unroll
        for (int i = 0; i < kSortBatch; ++i)
            if (v[i].e >= 0) atomicAdd(&hist[v[i].e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.experts; e += kSortThreads) p.counts[static_cast<size_t>(blockIdx.x) * pitch_of(p.experts) + e] = hist[e];
}

__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(const __grid_constant__ Sort p) {
    extern __shared__ int smem[];
    int* total = smem;                       // [experts]: all assignments
    int* before = smem + p.experts;          // [experts]: those of the CTAs before
    int* place = smem + 2 * p.experts;       // [warp][experts]: counts, then the warp's next row
    __shared__ int of_warp[kSortWarps];      // those of its threads' experts
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool alone = p.counts == nullptr;
    if (alone) asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int i = threadIdx.x; i < (kSortWarps + 2) * p.experts; i += kSortThreads) smem[i] = 0;
    __syncthreads();
    const int c0 = run_start(p.total, blockIdx.x, gridDim.x), c1 = run_start(p.total, blockIdx.x + 1, gridDim.x);
    const int a0 = c0 + run_start(c1 - c0, warp, kSortWarps), a1 = c0 + run_start(c1 - c0, warp + 1, kSortWarps);
    int* mine = place + warp * p.experts;
    // (the first batch stays in registers until the rows are known)
    Assignment v[kSortBatch], first[kSortBatch];
    if (a0 < a1) load_batch<32>(p, a0 + lane, a1, first);
    for (int b = a0; b < a1; b += kSortBatch * 32) {
        if (b != a0) load_batch<32>(p, b + lane, a1, v);
#pragma unroll
        for (int i = 0; i < kSortBatch; ++i) {
            const int e = b == a0 ? first[i].e : v[i].e;
            if (e >= 0) atomicAdd(&mine[e], 1);
        }
    }
    if (!alone) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        // four experts a thread, each CTA's four in one load; parts threads share the CTAs
        const int quads = pitch_of(p.experts) / 4, per = max(quads, 16), parts = kSortThreads / per;
        const int part = threadIdx.x / per, e = 4 * (static_cast<int>(threadIdx.x) - part * per);
        if (part < parts && e < p.experts) {
            int4 all = make_int4(0, 0, 0, 0), ahead = all;
#pragma unroll 16
            for (int b = part; b < static_cast<int>(gridDim.x); b += parts) {
                const int4 n = *reinterpret_cast<const int4*>(p.counts + static_cast<size_t>(b) * pitch_of(p.experts) + e);
                const int is = b < static_cast<int>(blockIdx.x) ? -1 : 0;
                all.x += n.x, all.y += n.y, all.z += n.z, all.w += n.w;
                ahead.x += n.x & is, ahead.y += n.y & is, ahead.z += n.z & is, ahead.w += n.w & is;
            }
            const int sums[2][4] = {{all.x, all.y, all.z, all.w}, {ahead.x, ahead.y, ahead.z, ahead.w}};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (e + i >= p.experts) continue;
                atomicAdd(&total[e + i], sums[0][i]);
                atomicAdd(&before[e + i], sums[1][i]);
            }
        }
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __syncthreads();
    // a thread's experts: one, or two neighbours
    const int own = p.experts > kSortThreads ? 2 : 1, e0 = own * static_cast<int>(threadIdx.x), e1 = min(e0 + own, p.experts);
    int n = 0;
    for (int e = e0; e < e1; ++e) {
        if (alone) {
            int sum = 0;
#pragma unroll
            for (int w = 0; w < kSortWarps; ++w) sum += place[w * p.experts + e];
            total[e] = sum;
        }
        n += total[e];
    }
    int start = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(kAll, start, d);
        if (lane >= d) start += o;
    }
    if (lane == 31) of_warp[warp] = start;
    __syncthreads();
    start -= n;
    int rows = 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
        const int m = of_warp[w];
        start += w < warp ? m : 0;
        rows += m;
    }
    for (int e = e0; e < e1; ++e) {
        int of[kSortWarps], next = start + before[e];
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) of[w] = place[w * p.experts + e];
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) {
            place[w * p.experts + e] = next;
            next += of[w];
        }
        if (p.offsets && blockIdx.x == 0) p.offsets[e] = start;
        start += total[e];
    }
    if (p.offsets && blockIdx.x == 0 && threadIdx.x == 0) p.offsets[p.experts] = rows;
    __syncthreads();
    for (int b = a0; b < a1; b += kSortBatch * 32) {
        if (b != a0) load_batch<32>(p, b + lane, a1, v);
#pragma unroll
        for (int i = 0; i < kSortBatch; ++i) {
            const Assignment at = b == a0 ? first[i] : v[i];
            const int e = at.e;
            const uint32_t same = __match_any_sync(kAll, e);
            int row = -1;
            if (e >= 0) row = mine[e] + __popc(same & ((1u << lane) - 1u));
            __syncwarp();
            if (e >= 0 && (same >> lane) == 1u) mine[e] = row + 1;   // the last of its equals
            __syncwarp();
            if (row >= 0) p.row_token[row] = at.t;
            if (b + i * 32 + lane < a1) p.row_of[at.t * p.ld_row_of + at.j] = row;
        }
    }
    for (int r = rows + static_cast<int>(blockIdx.x * kSortThreads + threadIdx.x); r < p.total; r += static_cast<int>(gridDim.x) * kSortThreads)
        p.row_token[r] = -1;
}

// --------------------------------------------- rows to their experts and back

constexpr int kMoveThreads = 256;
// Groups of eight columns that a thread has on its way: two, but one in combine
// where rows start anywhere (9761 x 8 rows of 1268 87 us, 102 with two).
constexpr int kSteps = 2;
__host__ __device__ constexpr int combine_steps(bool whole) { return whole ? kSteps : 1; }
// CTAs an SM is to hold, which bounds their registers.  Where rows start anywhere and
// hold 16 bits, eight (9761 x 8 rows of 1268: combine 70 us, 79 without a bound; its
// gradient 139, 149 with five).  Where they do not and at most two assignments are on
// their way, four of combine (16384 x 2 rows of 4096: 67 us, 77 with the registers of
// three, 82 with five, which spills; three of fp32 rows, which take more) and five of
// the gradient (102; 106 with four).
template <bool kWhole, bool kGrad, typename TX, typename TY, int kJ>
constexpr int resident() {
    constexpr bool kHalf = sizeof(TX) == 2 && sizeof(TY) == 2;
    if (kJ > 2) return 2;
    if (!kWhole) return kHalf ? 8 : 2;
    if (kGrad) return kHalf ? 5 : 2;
    return sizeof(TX) == 2 ? 4 : 3;
}
constexpr int kMaxCols = 65535 * kMoveThreads * 8 - 8;   // a grid's second extent

struct Rows {
    const void* y;      // tokens' side: read by dispatch and the gradient, written by combine
    long long ldy;
    const void* x;      // experts' side
    long long ldx;
    void* out;          // what is written
    long long ldo;
    int tokens, k, cols, rows;
    const int* row_of;
    long long ld_row_of;
    const float* weights;
    long long ld_weights;
    float* dweights;
    long long ld_dweights;
    int lanes;          // threads a token
};

// Eight neighbouring columns are a thread's at a time.  kWhole: all rows start on
// 16 bytes.  Otherwise a thread's eight lie between the 16-byte boundaries of the
// row that is written, and what is read is shifted into place.  Those at a row's
// ends go one by one.

// Where this thread works: its token and its first group of eight columns.
struct Place {
    long long t;
    int g0;
};
__device__ __forceinline__ Place place_of(const Rows& p, int steps) {
    const int slot = threadIdx.x / p.lanes;
    return {static_cast<long long>(blockIdx.x) * (kMoveThreads / p.lanes) + slot,
            static_cast<int>(blockIdx.y) * p.lanes * steps + static_cast<int>(threadIdx.x) - slot * p.lanes};
}

// The first column of group g of a row that is written: at or before it.
template <bool kWhole, typename T>
__device__ __forceinline__ int column_of(const T* row, int g) { return kWhole ? 8 * g : 8 * g - past16(row); }

template <bool kWhole, typename T>
__device__ __forceinline__ Raw8<T> fetch(const T* row, int c, int cols) {
    if constexpr (kWhole)
        if (c + 8 <= cols) return load_raw8<T, true>(row + c);
    return load_any8<T>(row, c, cols);
}

// The row of an assignment, -1 where it has none.
__device__ __forceinline__ int row_at(const Rows& p, long long t, int j) {
    const int r = p.row_of[t * p.ld_row_of + j];
    return r >= 0 && r < p.rows ? r : -1;
}

template <typename TX, typename TY>
__device__ __forceinline__ Raw8<TX> as_type(const Raw8<TY>& r) {
    if constexpr (std::is_same<TX, TY>::value) {
        return r;
    } else {
        float f[8];
        values_of<TY>(r, f);
        return raw_of<TX>(f);
    }
}

template <bool kWhole, typename TY, typename TX>
__global__ void __launch_bounds__(kMoveThreads) dispatch_kernel(const __grid_constant__ Rows p) {
    tcg::host::wait_for_kernel_ahead();
    const Place w = place_of(p, kSteps);
    if (w.t >= p.tokens) return;
    const TY* src = static_cast<const TY*>(p.y) + w.t * p.ldy;
    Raw8<TX> v[kSteps];
    if constexpr (kWhole) {
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const int c = 8 * (w.g0 + s * p.lanes);
            if (c < p.cols) v[s] = as_type<TX, TY>(fetch<true, TY>(src, c, p.cols));
        }
    }
    for (int j = 0; j < p.k; ++j) {
        const int r = row_at(p, w.t, j);
        if (r < 0) continue;
        TX* dst = static_cast<TX*>(p.out) + r * p.ldo;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const int c = column_of<kWhole>(dst, w.g0 + s * p.lanes);
            if (c >= p.cols) continue;
            if constexpr (!kWhole) v[s] = as_type<TX, TY>(fetch<false, TY>(src, c, p.cols));   // (from the L1 after the first)
            store_any8<TX>(dst, c, p.cols, v[s]);
        }
    }
}

// kJ assignments' rows are on their way at once; sums in the order of j.  (Rows that
// start anywhere: one, whose shifting takes the registers; 9761 x 8 rows of 1268 83
// us and 108 with two, the gradient 203 and 255.)
template <bool kWhole, typename TX, typename TY, int kJ>
__global__ void __launch_bounds__(kMoveThreads, resident<kWhole, false, TX, TY, kJ>()) combine_kernel(const __grid_constant__ Rows p) {
    tcg::host::wait_for_kernel_ahead();
    constexpr int kS = combine_steps(kWhole);
    const Place w = place_of(p, kS);
    if (w.t >= p.tokens) return;
    TY* dst = static_cast<TY*>(p.out) + w.t * p.ldo;
    int col[kS];
#pragma unroll
    for (int s = 0; s < kS; ++s) col[s] = column_of<kWhole>(dst, w.g0 + s * p.lanes);
    float acc[kS][8];
#pragma unroll
    for (int s = 0; s < kS; ++s)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[s][i] = 0.0f;
    for (int j0 = 0; j0 < p.k; j0 += kJ) {
        Raw8<TX> v[kJ][kS];
        int row[kJ];
        float wt[kJ];
#pragma unroll
        for (int q = 0; q < kJ; ++q) {
            row[q] = j0 + q < p.k ? row_at(p, w.t, j0 + q) : -1;
            wt[q] = row[q] < 0 ? 0.0f : (p.weights ? p.weights[w.t * p.ld_weights + j0 + q] : 1.0f);
        }
#pragma unroll
        for (int q = 0; q < kJ; ++q)
#pragma unroll
            for (int s = 0; s < kS; ++s) {
                if (row[q] >= 0 && col[s] < p.cols) v[q][s] = fetch<kWhole, TX>(static_cast<const TX*>(p.x) + row[q] * p.ldx, col[s], p.cols);
            }
#pragma unroll
        for (int q = 0; q < kJ; ++q)
#pragma unroll
            for (int s = 0; s < kS; ++s) {
                if (row[q] < 0 || col[s] >= p.cols) continue;
                float f[8];
                values_of<TX>(v[q][s], f);
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[s][i] = fmaf(wt[q], f[i], acc[s][i]);
            }
    }
#pragma unroll
    for (int s = 0; s < kS; ++s)
        if (col[s] < p.cols) store_any8<TY>(dst, col[s], p.cols, raw_of<TY>(acc[s]));
}

// p.lanes threads a token (a power of two from 32 on), over all its columns;
// kJ assignments at a time, whose weights' gradients are summed in a fixed order.
template <bool kWhole, typename TX, typename TY, int kJ>
__global__ void __launch_bounds__(kMoveThreads, resident<kWhole, true, TX, TY, kJ>()) combine_grad_kernel(const __grid_constant__ Rows p) {
    tcg::host::wait_for_kernel_ahead();
    __shared__ float part[kJ][kMoveThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int slot = threadIdx.x / p.lanes, per_cta = kMoveThreads / p.lanes, warps = p.lanes / 32;
    const long long t = static_cast<long long>(blockIdx.x) * per_cta + slot;
    const bool in = t < p.tokens;
    const int thread = static_cast<int>(threadIdx.x) - slot * p.lanes;
    const TY* dy = static_cast<const TY*>(p.y) + (in ? t : 0) * p.ldy;
    for (int j0 = 0; j0 < p.k; j0 += kJ) {
        int row[kJ];
        float wt[kJ], dot[kJ];
#pragma unroll
        for (int q = 0; q < kJ; ++q) {
            row[q] = in && j0 + q < p.k ? row_at(p, t, j0 + q) : -1;
            wt[q] = row[q] < 0 ? 0.0f : (p.weights ? p.weights[t * p.ld_weights + j0 + q] : 1.0f);
            dot[q] = 0.0f;
        }
        if (in) {
            // (rows that start anywhere: a group more, each row's columns its own, dy from the L1 after the first)
            const int groups = (p.cols + (kWhole ? 7 : 14)) / 8;
            for (int g = thread; g < groups; g += p.lanes) {
                Raw8<TX> v[kJ];
                Raw8<TY> r[kWhole ? 1 : kJ];
                int col[kJ];
#pragma unroll
                for (int q = 0; q < kJ; ++q) col[q] = column_of<kWhole>(static_cast<TX*>(p.out) + row[q] * p.ldo, g);
                if constexpr (kWhole) r[0] = fetch<true, TY>(dy, 8 * g, p.cols);
#pragma unroll
                for (int q = 0; q < kJ; ++q) {
                    if (row[q] < 0 || col[q] >= p.cols) continue;
                    if constexpr (!kWhole) r[q] = fetch<false, TY>(dy, col[q], p.cols);
                    if (p.dweights) v[q] = fetch<kWhole, TX>(static_cast<const TX*>(p.x) + row[q] * p.ldx, col[q], p.cols);
                }
#pragma unroll
                for (int q = 0; q < kJ; ++q) {
                    if (row[q] < 0 || col[q] >= p.cols) continue;
                    float d[8], f[8];
                    values_of<TY>(r[kWhole ? 0 : q], d);
                    if (p.dweights) {
                        values_of<TX>(v[q], f);
#pragma unroll
                        for (int i = 0; i < 8; ++i) dot[q] = fmaf(f[i], d[i], dot[q]);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[i] = wt[q] * d[i];
                    store_any8<TX>(static_cast<TX*>(p.out) + row[q] * p.ldo, col[q], p.cols, raw_of<TX>(f));
                }
            }
        }
        if (!p.dweights) continue;
#pragma unroll
        for (int q = 0; q < kJ; ++q) {
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) dot[q] += __shfl_xor_sync(kAll, dot[q], d);
            if (lane == 0) part[q][warp] = dot[q];
        }
        __syncthreads();
        if (in && thread == 0) {
#pragma unroll
            for (int q = 0; q < kJ; ++q) {
                if (j0 + q >= p.k) continue;
                float sum = 0.0f;
                for (int i = 0; i < warps; ++i) sum += part[q][warp + i];
                p.dweights[t * p.ld_dweights + j0 + q] = row[q] < 0 ? 0.0f : sum;
            }
        }
        __syncthreads();
    }
}

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
int size_of(tcg_dtype t) { return t == TCG_F32 ? 4 : 2; }
bool known(tcg_dtype t) { return t == TCG_BF16 || t == TCG_F16 || t == TCG_F32; }
bool whole_words(const void* p, int ld, tcg_dtype t) { return aligned(p, 16) && static_cast<long long>(ld) * size_of(t) % 16 == 0; }

tcg_status start(Rows& p, int tokens, int k, int cols, int rows, const int* row_of, int ld_row_of) {
    if (tokens < 0 || k < 1 || cols < 0 || rows < 0) return TCG_ERR_INVALID_ARG;
    if (std::max(tokens, rows) > tcg::host::kMaxExtent || cols > kMaxCols) return TCG_ERR_UNSUPPORTED;
    if (tokens == 0) return TCG_OK;
    if (!row_of || ld_row_of < k) return TCG_ERR_INVALID_ARG;
    if (!aligned(row_of, 4)) return TCG_ERR_MISALIGNED;
    p.tokens = tokens;
    p.k = k;
    p.cols = cols;
    p.rows = rows;
    p.row_of = row_of;
    p.ld_row_of = ld_row_of;
    return TCG_OK;
}

// A matrix of `cols` columns that has to be there (where it has rows).
tcg_status check_matrix(const void* m, int ld, int cols, tcg_dtype t, bool needed = true) {
    if (!known(t)) return TCG_ERR_INVALID_ARG;
    if (needed && (!m || ld < cols)) return TCG_ERR_INVALID_ARG;
    return aligned(m, size_of(t)) ? TCG_OK : TCG_ERR_MISALIGNED;
}

template <typename F>
void with_type(tcg_dtype t, F f) {
    if (t == TCG_BF16) f(__nv_bfloat16{});
    else if (t == TCG_F16) f(__half{});
    else f(float{});
}

// Threads a token: as many as its columns occupy at `steps` of eight each.
int lanes_for(int cols, int steps) {
    const int want = (cols + 8 * steps - 1) / (8 * steps);
    int lanes = 32;
    while (lanes < want && lanes < kMoveThreads) lanes *= 2;
    return lanes;
}
dim3 move_grid(const Rows& p, bool whole, int steps) {
    // (a row that starts anywhere may take a group more)
    const int per_cta = kMoveThreads / p.lanes, span = p.lanes * 8 * steps;
    return dim3(static_cast<unsigned>((static_cast<long long>(p.tokens) + per_cta - 1) / per_cta),
                static_cast<unsigned>((static_cast<long long>(p.cols) + (whole ? 0 : 7) + span - 1) / span));
}

// Whether all CTAs run at once with four assignments' rows on their way, whose
// registers let two be on an SM: then four, where there are as many, else two
// (4096 columns, 8 rows a token: combine of 256 tokens 5.8 us with four and 6.6
// with two, of 512 10.1 and 7.8; its gradient of 512 17 and 23, of 1024 32 and 30).
bool few(dim3 grid, int sms) { return static_cast<long long>(grid.x) * grid.y <= 2LL * sms; }

tcg_status launched(cudaError_t e, const char* what) { return e == cudaSuccess ? TCG_OK : tcg::host::fail_launch(what, e); }

int sort_ctas(long long total, int sms) {
    return total <= kSortAlone ? 1 : static_cast<int>(std::min<long long>(sms, (total + kSortRun - 1) / kSortRun));
}

}  // namespace

extern "C" {

size_t tcg_moe_sort_workspace_size(int tokens, int experts, int k) {
    if (tokens < 0 || experts < 1 || k < 1 || experts > kMaxExperts) return 0;
    tcg::host::Device dev;
    if (tcg::host::device(dev) != TCG_OK) dev.num_sms = 1024;
    const int ctas = sort_ctas(static_cast<long long>(tokens) * k, dev.num_sms);
    return tcg::host::kScratchAt + (ctas > 1 ? static_cast<size_t>(ctas) * pitch_of(experts) * sizeof(int) : 0);
}

tcg_status tcg_moe_sort(int tokens, int experts, int k, const int* topk, int ld_topk, const uint8_t* mask, int* offsets,
                        int* row_token, int* row_of, int ld_row_of, void* workspace, size_t workspace_bytes, void* stream) {
    if (tokens < 0 || experts < 1 || k < 1) return TCG_ERR_INVALID_ARG;
    // (rows are ints, and a run's end plus a step still is one)
    if (experts > kMaxExperts || static_cast<long long>(tokens) * k > tcg::host::kMaxExtent - (1 << 20)) return TCG_ERR_UNSUPPORTED;
    if (tokens > 0 && (!topk || ld_topk < k || !row_token || !row_of || ld_row_of < k)) return TCG_ERR_INVALID_ARG;
    if (!aligned(topk, 4) || !aligned(offsets, 4) || !aligned(row_token, 4) || !aligned(row_of, 4)) return TCG_ERR_MISALIGNED;
    tcg::host::Device dev;
    tcg_status st = tcg::host::device(dev);
    if (st != TCG_OK) return st;
    if (!workspace || !aligned(workspace, 16) || workspace_bytes < tcg_moe_sort_workspace_size(tokens, experts, k))
        return tcg::host::fail(TCG_ERR_WORKSPACE, "workspace NULL, not 16-byte aligned or smaller than tcg_moe_sort_workspace_size");
    static tcg::host::OncePerDevice once;
    cudaError_t err = once([] {
        return cudaFuncSetAttribute(sort_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (kSortWarps + 2) * kMaxExperts * static_cast<int>(sizeof(int)));
    });
    if (err != cudaSuccess) return launched(err, "tcg_moe_sort kernel attributes");
    Sort p = {};
    p.topk = topk;
    p.ld_topk = ld_topk;
    p.mask = mask;
    p.total = tokens * k;
    p.k = k;
    p.experts = experts;
    while ((1ll << p.div_shift) < k) ++p.div_shift;
    p.div_mul = static_cast<uint32_t>((((1ull << p.div_shift) - k) << 32) / k + 1);
    p.offsets = offsets;
    p.row_token = row_token;
    p.row_of = row_of;
    p.ld_row_of = ld_row_of;
    const int ctas = sort_ctas(p.total, dev.num_sms);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (ctas > 1) {
        p.counts = reinterpret_cast<int*>(static_cast<char*>(workspace) + tcg::host::kScratchAt);
        err = tcg::host::launch_early(sort_count_kernel, dim3(ctas), kSortThreads, s, p);
        if (err != cudaSuccess) return launched(err, "tcg_moe_sort");
    }
    return launched(tcg::host::launch_early(sort_place_kernel, dim3(ctas), kSortThreads, s, p,
                                            (kSortWarps + 2) * static_cast<size_t>(experts) * sizeof(int)), "tcg_moe_sort");
}

tcg_status tcg_moe_dispatch(int tokens, int k, int cols, int rows, const void* x, int ldx, tcg_dtype x_dtype, const int* row_of,
                            int ld_row_of, void* out, int ldo, tcg_dtype out_dtype, void* stream) {
    Rows p = {};
    tcg_status st = start(p, tokens, k, cols, rows, row_of, ld_row_of);
    if (st == TCG_OK) st = check_matrix(x, ldx, cols, x_dtype, tokens > 0);
    if (st == TCG_OK) st = check_matrix(out, ldo, cols, out_dtype, rows > 0 && tokens > 0);
    if (st != TCG_OK || tokens == 0 || cols == 0 || rows == 0) return st;
    tcg::host::Device dev;
    if ((st = tcg::host::device(dev)) != TCG_OK) return st;
    p.y = x;
    p.ldy = ldx;
    p.out = out;
    p.ldo = ldo;
    const bool whole = whole_words(x, ldx, x_dtype) && whole_words(out, ldo, out_dtype);
    p.lanes = lanes_for(cols, kSteps);
    cudaError_t err = cudaSuccess;
    with_type(x_dtype, [&](auto y) {
        with_type(out_dtype, [&](auto o) {
            const auto kernel = whole ? dispatch_kernel<true, decltype(y), decltype(o)> : dispatch_kernel<false, decltype(y), decltype(o)>;
            err = tcg::host::launch_early(kernel, move_grid(p, whole, kSteps), kMoveThreads, static_cast<cudaStream_t>(stream), p);
        });
    });
    return launched(err, "tcg_moe_dispatch");
}

tcg_status tcg_moe_combine(int tokens, int k, int cols, int rows, const void* x, int ldx, tcg_dtype x_dtype, const int* row_of,
                           int ld_row_of, const float* weights, int ld_weights, void* y, int ldy, tcg_dtype y_dtype,
                           void* stream) {
    Rows p = {};
    tcg_status st = start(p, tokens, k, cols, rows, row_of, ld_row_of);
    if (st == TCG_OK) st = check_matrix(x, ldx, cols, x_dtype, rows > 0 && tokens > 0);
    if (st == TCG_OK) st = check_matrix(y, ldy, cols, y_dtype, tokens > 0);
    if (st != TCG_OK || tokens == 0 || cols == 0) return st;
    if (weights && ld_weights < k) return TCG_ERR_INVALID_ARG;
    if (!aligned(weights, 4)) return TCG_ERR_MISALIGNED;
    tcg::host::Device dev;
    if ((st = tcg::host::device(dev)) != TCG_OK) return st;
    p.x = x;
    p.ldx = ldx;
    p.weights = weights;
    p.ld_weights = ld_weights;
    p.out = y;
    p.ldo = ldy;
    const bool whole = whole_words(x, ldx, x_dtype) && whole_words(y, ldy, y_dtype);
    p.lanes = lanes_for(cols, combine_steps(whole));
    const dim3 grid = move_grid(p, whole, combine_steps(whole));
    cudaError_t err = cudaSuccess;
    with_type(x_dtype, [&](auto a) {
        with_type(y_dtype, [&](auto b) {
            const auto run = [&](auto* kernel) {
                err = tcg::host::launch_early(kernel, grid, kMoveThreads, static_cast<cudaStream_t>(stream), p);
            };
            if (!whole) run(combine_kernel<false, decltype(a), decltype(b), 1>);
            else if (k == 1) run(combine_kernel<true, decltype(a), decltype(b), 1>);
            else if (k == 2 || !few(grid, dev.num_sms)) run(combine_kernel<true, decltype(a), decltype(b), 2>);
            else run(combine_kernel<true, decltype(a), decltype(b), 4>);
        });
    });
    return launched(err, "tcg_moe_combine");
}

tcg_status tcg_moe_combine_backward(int tokens, int k, int cols, int rows, const void* x, int ldx, tcg_dtype x_dtype,
                                    const int* row_of, int ld_row_of, const float* weights, int ld_weights, const void* dy,
                                    int lddy, tcg_dtype dy_dtype, void* dx, int lddx, float* dweights, int ld_dweights,
                                    void* stream) {
    Rows p = {};
    tcg_status st = start(p, tokens, k, cols, rows, row_of, ld_row_of);
    if (tokens > 0 && st == TCG_OK && dweights && ld_dweights < k) return TCG_ERR_INVALID_ARG;
    if (st == TCG_OK) st = check_matrix(x, ldx, cols, x_dtype, rows > 0 && tokens > 0 && dweights);
    if (st == TCG_OK) st = check_matrix(dy, lddy, cols, dy_dtype, tokens > 0);
    if (st == TCG_OK) st = check_matrix(dx, lddx, cols, x_dtype, rows > 0 && tokens > 0);
    if (st != TCG_OK || tokens == 0) return st;
    if (weights && ld_weights < k) return TCG_ERR_INVALID_ARG;
    if (!aligned(weights, 4) || !aligned(dweights, 4)) return TCG_ERR_MISALIGNED;
    tcg::host::Device dev;
    if ((st = tcg::host::device(dev)) != TCG_OK) return st;
    p.tokens = tokens;
    p.k = k;
    p.x = x;
    p.ldx = ldx;
    p.y = dy;
    p.ldy = lddy;
    p.weights = weights;
    p.ld_weights = ld_weights;
    p.out = dx;
    p.ldo = lddx;
    p.dweights = dweights;
    p.ld_dweights = ld_dweights;
    // (without a column there is no word that may be read; the weights' gradients are written all the same)
    const bool whole = cols == 0 || ((!dweights || whole_words(x, ldx, x_dtype)) && whole_words(dy, lddy, dy_dtype) && whole_words(dx, lddx, x_dtype));
    p.lanes = lanes_for(cols, 4);
    const int per_cta = kMoveThreads / p.lanes;
    const dim3 grid(static_cast<unsigned>((static_cast<long long>(tokens) + per_cta - 1) / per_cta));
    cudaError_t err = cudaSuccess;
    with_type(x_dtype, [&](auto a) {
        with_type(dy_dtype, [&](auto b) {
            const auto run = [&](auto* kernel) {
                err = tcg::host::launch_early(kernel, grid, kMoveThreads, static_cast<cudaStream_t>(stream), p);
            };
            if (!whole) run(combine_grad_kernel<false, decltype(a), decltype(b), 1>);
            else if (k == 1) run(combine_grad_kernel<true, decltype(a), decltype(b), 1>);
            else if (k == 2 || !few(grid, dev.num_sms)) run(combine_grad_kernel<true, decltype(a), decltype(b), 2>);
            else run(combine_grad_kernel<true, decltype(a), decltype(b), 4>);
        });
    });
    return launched(err, "tcg_moe_combine_backward");
}

}  // extern "C"
