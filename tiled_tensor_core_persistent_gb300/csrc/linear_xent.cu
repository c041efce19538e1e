// linear_xent.cu -- softmax cross entropy of a linear layer over a vocabulary:
// checks, the pieces of the vocabulary, launches.  The tiles: xent_kernel.cuh,
// xent_product_kernel.cuh.
//
//   z = X W^T,  lse_t = log sum_v exp z_tv,  loss_t = lse_t - z_{t, y_t}
//   mean = sum of loss_t / n over the n tokens whose target names a word
//   dz_tv = r_t (exp(z_tv - lse_t) - [v = y_t]),  r_t = grad_mean / n + grad_loss_t
//   dX = dz W,  dW = dz^T X
//
// Forward, the tiles leave (M, s) of every row and column tile, which one small
// kernel joins.  Backward, the logits of a piece of the vocabulary are computed
// again and leave dz of that piece in the workspace, in the operands' type; one
// launch (xent_product_kernel.cuh) takes it to dX (summed over the pieces in
// fp32) and dW.  One rounding of dz to 16 bits stands between the logits and the
// gradients, of the same size as that of a 16-bit gradient: the other products
// would need fp32 operands.  What is rounded is dz over the largest finite |r_t|, which
// the products multiply by: where all tokens weigh alike, dz of an unlikely
// target is then a number just above -1, which 16 bits hold to 2^-9 of itself or
// exactly, where r_t times it would be off by the same part of a step for every
// token (dX and dW of 849 x 30575 x 2285: 2.8e-3 off, now 1.9e-3; 1.7e-3 is
// their own rounding).  fp16, whose small numbers end at 2^-24, has 2^14 times
// that.
#include <algorithm>
#include <climits>
#include <cstring>

#include "xent_product_kernel.cuh"

namespace {

using tcg::xent::Params;

// What dz of a piece may take of the workspace (more only where 256 words, a piece's
// least, do: from 2^20 tokens on): the fewer pieces, the fewer last waves and sums of
// dX, and a dz of the whole vocabulary that fits is one piece (backward of 8192 x 100000 x 512 1.80 ms; 2.27 with 64 MB, 1.92
// with 256, 1.70 with 1 GB; of 4096 x 65536 x 4096 3.74, 3.91, 3.74 and 3.75).
constexpr size_t kPieceBytes = size_t(512) << 20;
constexpr int kMinTileN = 128;
constexpr int kPartK = 1024;           // k of the logits' products that the tensor cores sum in one go, about
// Row tiles that are walked before the next column tile (by themselves: 4096 x 65536 x
// 4096 forward 1036 us and backward 3270; 1123 and 3561 with 4, 1059 and 3295 with 8,
// 1037 and 3260 with 32; 8192 x 100000 x 512 534 and 1915, 530 and 1883 with 8, 537 and
// 1911 with 32; no difference at 1000 and fewer tokens).
constexpr int kRasterM = 16;
constexpr int kFinishRows = 32, kFinishSlices = 32, kFinishThreads = kFinishRows * kFinishSlices;
constexpr int kFinishBatch = 8;
constexpr float kHalfTop = 16384.0f;   // fp16: what the largest |r_t| becomes

// ------------------------------------------------------- joining the tiles

struct Finish {
    const float2* part;
    int num_n, tokens, vocab;   // num_n: half column tiles
    const float* picked;
    const int* target;
    float* lse;
    float* loss;          // may be nullptr
    float* mean;
    int* valid;
    double* sums;         // [CTA]
    int* counts;          // [CTA]
    int* arrivals;
};

// 32 threads a row, each some of the column tiles, eight of them on their way at
// once: first a warp's lanes are 32 rows (whose tiles lie side by side), then, the
// 32 x 32 results turned in shared memory, the threads of one row.  What is in
// 64 bits is one warp's (64-bit operations are slow, and as slow for one lane as
// for 32).  Sums in a fixed order.
__global__ void __launch_bounds__(kFinishThreads) finish_kernel(const __grid_constant__ Finish p) {
    tcg::host::wait_for_kernel_ahead();
    __shared__ float2 slot[kFinishSlices][kFinishRows + 1];
    __shared__ float2 joined[kFinishRows];
    __shared__ int last;
    static_assert(kFinishRows == 32 && kFinishSlices == 32, "a warp a row, a lane a slice");
    const int r = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const long long row = static_cast<long long>(blockIdx.x) * kFinishRows + r;
    const bool in = row < p.tokens;
    float2 v = make_float2(-INFINITY, 0.0f);
    for (int n0 = slice; in && n0 < p.num_n; n0 += kFinishSlices * kFinishBatch) {
        float2 w[kFinishBatch];
        float m = v.x;
#pragma unroll
        for (int i = 0; i < kFinishBatch; ++i) {
            const int n = n0 + i * kFinishSlices;
            w[i] = n < p.num_n ? p.part[static_cast<size_t>(n) * p.tokens + row] : make_float2(-INFINITY, 0.0f);
        }
#pragma unroll
        for (int i = 0; i < kFinishBatch; ++i) m = fmaxf(m, w[i].x);
        const float base = m == -INFINITY ? 0.0f : m;
        float s = v.y * exp2f(v.x - base);
#pragma unroll
        for (int i = 0; i < kFinishBatch; ++i) s += w[i].y * exp2f(w[i].x - base);
        v = make_float2(m, s);
    }
    slot[slice][r] = v;
    __syncthreads();
    // row `slice` of the CTA's
    v = slot[r][slice];
    float m = v.x;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    float s = v.y * exp2f(v.x - (m == -INFINITY ? 0.0f : m));
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    if (r == 0) joined[slice] = make_float2(m, s);
    __syncthreads();
    double sum = 0.0;
    int count = 0;
    if (slice == 0) {
        if (in) {
            // (logits were multiplied by kLog2e as it is held, so that is what divides here)
            const double lse = (static_cast<double>(joined[r].x) + static_cast<double>(log2f(joined[r].y))) *
                               (1.0 / static_cast<double>(tcg::xent::kLog2e));
            p.lse[row] = static_cast<float>(lse);
            const int y = p.target[row];
            const bool counts = y >= 0 && y < p.vocab;
            const float loss = counts ? static_cast<float>(lse - static_cast<double>(p.picked[row])) : 0.0f;
            if (p.loss) p.loss[row] = loss;
            sum = static_cast<double>(loss);
            count = counts;
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            sum += __shfl_xor_sync(0xffffffffu, sum, d);
            count += __shfl_xor_sync(0xffffffffu, count, d);
        }
    }
    if (gridDim.x > 1) {
        if (threadIdx.x == 0) {
            p.sums[blockIdx.x] = sum;
            p.counts[blockIdx.x] = count;
            __threadfence();
            last = tcg::ptx::atomic_add_acq_rel_gpu(p.arrivals, 1) == static_cast<int>(gridDim.x) - 1;
        }
        __syncthreads();
        if (!last) return;
        // the last CTA: every CTA's sum, in the same order whichever is last
        if (threadIdx.x >= 32) return;
        sum = 0.0;
        count = 0;
        for (int i = r; i < static_cast<int>(gridDim.x); i += 32) {
            sum += __ldcg(p.sums + i);
            count += __ldcg(p.counts + i);
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            sum += __shfl_xor_sync(0xffffffffu, sum, d);
            count += __shfl_xor_sync(0xffffffffu, count, d);
        }
        if (threadIdx.x == 0) *p.arrivals = 0;
    }
    if (threadIdx.x == 0) {
        *p.mean = count > 0 ? static_cast<float>(sum) / static_cast<float>(count) : 0.0f;
        *p.valid = count;
    }
}

// ----------------------------------------------------------------- plans

long long blocks(long long n, long long b) { return (n + b - 1) / b; }
size_t padded(size_t n) { return (n + 255) / 256 * 256; }

struct Plan {
    bool pair = false;
    int parts = 1;     // accumulations that share a tile's K
    int tile_n = 256, num_m = 1, num_n = 1, workers = 1;
};

// A pair of CTAs a tile where one CTA's rows do not hold all tokens (128 x 32768 x
// 4096 51.6 us, 56.7 with pairs; 129 56.0, 63.4 without).  The width whose waves of
// tiles take the least: a tile's time goes with its columns, plus what a tile costs
// by itself (about sixteen columns' worth).
Plan make_plan(int tokens, long long cols, int hidden, int sms) {
    Plan pl;
    pl.pair = tokens > tcg::xent::kBM;
    pl.parts = std::max(1, (hidden + kPartK / 2) / kPartK);
    pl.num_m = static_cast<int>(blocks(tokens, pl.pair ? 256 : 128));
    const int workers = std::max(1, pl.pair ? sms / 2 : sms);
    long long best = LLONG_MAX;
    for (int w = tcg::xent::kMaxN; w >= kMinTileN; w -= 32) {
        const long long cost = blocks(pl.num_m * blocks(cols, w), workers) * (w + 16);
        if (cost < best) {
            best = cost;
            pl.tile_n = w;
        }
    }
    pl.num_n = static_cast<int>(blocks(cols, pl.tile_n));
    pl.workers = static_cast<int>(std::min<long long>(static_cast<long long>(pl.num_m) * pl.num_n, workers));
    return pl;
}

// Words a piece of the vocabulary has (the last one may have fewer).
int piece_words(int tokens, int vocab) {
    const long long fit = std::max<long long>(256, static_cast<long long>(kPieceBytes / 2) / std::max(1, tokens) / 256 * 256);
    const long long pieces = blocks(vocab, fit);
    return static_cast<int>(std::min<long long>(vocab, blocks(blocks(vocab, pieces), 256) * 256));
}

// a counter for each warp of both CTAs of a split tile
constexpr long long kMaxSplitTiles = tcg::host::kCounterBytes / sizeof(int) / (2 * tcg::xent::kRowWarps);

// Columns of the products' tiles.  128 where hidden has no more, and where dX has
// so few tiles that their long sums and the joining of their pieces are the time,
// of which half as wide ones take half (256 x 32768 x 1024, four tiles: backward 68
// us, 79 with 256; 512 x 32768 x 512 63 and 72).  Elsewhere a stage or a tile's way
// to memory takes three quarters as long at half the width (1000 x 50021 x 512,
// eight: 147 and 125; 1000 x 50021 x 1280 311 and 235).
int product_columns(int tokens, int hidden, bool want_dx) {
    const long long tiles = blocks(tokens, 2 * tcg::xent::kBM) * blocks(hidden, 256);
    return hidden <= 128 || (want_dx && tiles <= 4) ? 128 : 256;
}

// How dX's and dW's tiles go to the workers (pairs of CTAs).
struct ProductPlan {
    int tile_n = 256, splits = 1, early = 0, workers = 1;
};

// first, second: dX's and dW's tiles (0 where it is not wanted), kb: their
// stages of K.  A stage is 1024 cycles of the tensor cores on a tile of 256
// columns; a tile's way to memory takes about three stages' time and hides
// behind the next tile's longer sums.  A piece of a split tile costs three more,
// and the last one two for each piece that it adds.  Splits by the shortest time
// of the fullest worker.
ProductPlan plan_products(long long first, int first_kb, long long second, int second_kb, int workers) {
    ProductPlan best;
    long long least = LLONG_MAX;
    const long long c2 = std::max(second_kb, 3);
    for (int s = 1; s <= 16; ++s) {
        if (s > 1 && (first * s > 2 * workers || first > kMaxSplitTiles || first_kb < 4 * s)) break;
        const long long units = first * s, c1 = std::max(blocks(first_kb, s), 3LL) + (s > 1 ? 3 + 2 * s : 0);
        const long long rest = units % workers, early = rest > 0 ? c1 / c2 : 0;
        const long long taken = std::min(second, early * (workers - rest));
        const long long time = blocks(units, workers) * c1 + blocks(second - taken, workers) * c2;
        if (time < least) {
            least = time;
            best.splits = s;
            best.early = static_cast<int>(std::min(early, 1LL << 20));
        }
    }
    best.workers = static_cast<int>(std::max(1LL, std::min<long long>(workers, std::max(first * best.splits, second))));
    if (best.workers < workers) {   // fewer tiles than workers: round they go as they are
        const long long rest = first * best.splits % best.workers;
        best.early = rest > 0 ? static_cast<int>(std::min((blocks(first_kb, best.splits) + 3) / c2, 1LL << 20)) : 0;
    }
    return best;
}

// Where things lie in the workspace, behind the ranges that are kept zero.
struct Layout {
    size_t part = 0, picked = 0, sums = 0, counts = 0;                      // forward
    size_t back = 0, dz = 0, dx = 0, partials = 0;                          // backward
    size_t bytes = tcg::host::kScratchAt;
    size_t take(size_t n) {
        const size_t at = bytes;
        bytes += padded(n);
        return at;
    }
};

Layout forward_layout(int tokens, int vocab) {
    Layout l;
    l.part = l.take(2 * static_cast<size_t>(blocks(vocab, kMinTileN)) * tokens * sizeof(float2));
    l.picked = l.take(static_cast<size_t>(tokens) * sizeof(float));
    l.sums = l.take(static_cast<size_t>(blocks(tokens, kFinishRows)) * sizeof(double));
    l.counts = l.take(static_cast<size_t>(blocks(tokens, kFinishRows)) * sizeof(int));
    return l;
}

// Rows of any type start on 32 bytes, as dz is stored in such words: its first
// one past a workspace that starts on 16.
constexpr size_t kWord = 32;
int pitch_of(int n) { return static_cast<int>(blocks(n, kWord) * kWord); }

Layout backward_layout(int tokens, int vocab, int hidden, int sms) {
    Layout l;
    const int words = piece_words(tokens, vocab);
    l.back = l.take(sizeof(float));
    l.dz = l.take(static_cast<size_t>(tokens) * pitch_of(words) * 2 + kWord);
    l.dx = l.take(words < vocab ? static_cast<size_t>(tokens) * pitch_of(hidden) * sizeof(float) : 0);
    // (tiles are split while their pieces are at most two for each pair of SMs)
    l.partials = l.take(static_cast<size_t>(sms / 2 * 2) * tcg::xent::kPartialFloats * sizeof(float));
    return l;
}

// ---------------------------------------------------------------- launches

template <auto* kKernel, int kSmem>
cudaError_t set_attributes() {
    static tcg::host::OncePerDevice once;
    return once([] {
        cudaError_t e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        cudaFuncAttributes a;
        if (e == cudaSuccess) e = cudaFuncGetAttributes(&a, kKernel);
        // the register hand-over draws on what the block is launched with
        if (e == cudaSuccess && a.numRegs < tcg::xent::kLaunchRegs) e = cudaErrorInvalidConfiguration;
        return e;
    });
}

template <typename P>
tcg_status launch_ctas(void (*kernel)(P), const P& p, bool pair, int workers, int smem, cudaStream_t stream) {
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof cfg);
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3((pair ? 2 : 1) * workers);
    cfg.blockDim = dim3(tcg::xent::kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pair ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
    return e == cudaSuccess ? TCG_OK : tcg::host::fail_launch("tcg_linear_xent", e);
}

template <typename T, bool kPair, bool kGrad>
tcg_status launch(const Params& p, const Plan& pl, cudaStream_t stream) {
    constexpr auto* kKernel = &tcg::xent::xent_kernel<T, kPair, kGrad>;
    constexpr int kSmem = tcg::xent::Shape<kPair>::kSmemBytes;
    const cudaError_t e = set_attributes<kKernel, kSmem>();
    if (e != cudaSuccess) return tcg::host::fail_launch("tcg_linear_xent kernel attributes", e);
    return launch_ctas(kKernel, p, kPair, pl.workers, kSmem, stream);
}

template <typename T, bool kGrad>
tcg_status launch_plan(const Params& p, const Plan& pl, cudaStream_t stream) {
    return pl.pair ? launch<T, true, kGrad>(p, pl, stream) : launch<T, false, kGrad>(p, pl, stream);
}

// The tiles of words [first, first + cols) on X's rows.
template <bool kGrad>
tcg_status launch_tiles(Params& p, tcg_dtype dtype, const void* X, int ldx, const void* W, int ldw, int tokens, int hidden,
                        int first, int cols, const tcg::host::Device& dev, cudaStream_t stream) {
    const Plan pl = make_plan(tokens, cols, hidden, dev.num_sms);
    const int atoms = pl.pair ? tcg::xent::Shape<true>::kAtoms : tcg::xent::Shape<false>::kAtoms;
    p.tokens = tokens;
    p.cols = cols;
    p.first = first;
    p.num_m = pl.num_m;
    p.num_n = pl.num_n;
    p.num_kb = static_cast<int>(blocks(2LL * hidden, tcg::xent::kRowBytes * atoms));
    p.parts = std::min(pl.parts, p.num_kb);
    p.tile_n = pl.tile_n;
    p.raster_m = kRasterM;
    p.fmt = dtype == TCG_F16 ? 0u : 1u;
    p.timeout_ns = tcg::host::wait_timeout_ns();
    p.fault_inject = tcg::host::fault_inject();
    const char* w = static_cast<const char*>(W) + static_cast<size_t>(first) * ldw * 2;
    tcg_status st = tcg::host::map_bytes(&p.tmX, X, 2ull * hidden, tokens, 2ull * ldx, tcg::xent::kRowBytes, tcg::xent::kBM);
    if (st == TCG_OK)
        st = tcg::host::map_bytes(&p.tmW, w, 2ull * hidden, cols, 2ull * ldw, tcg::xent::kRowBytes, pl.pair ? pl.tile_n / 2 : pl.tile_n);
    if (st != TCG_OK) return st;
    return dtype == TCG_F16 ? launch_plan<__half, kGrad>(p, pl, stream) : launch_plan<__nv_bfloat16, kGrad>(p, pl, stream);
}

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
int size_of(tcg_dtype t) { return t == TCG_F32 ? 4 : 2; }

int out_type(tcg_dtype t) { return t == TCG_F32 ? tcg::xent::kOutF32 : t == TCG_F16 ? tcg::xent::kOutF16 : tcg::xent::kOutBf16; }

void set_output(tcg::xent::Product& q, void* out, long long ld, tcg_dtype t, float beta) {
    q.out = out;
    q.ldo = ld;
    q.type = out_type(t);
    q.beta = beta;
    const long long pitch = ld * size_of(t);
    q.vec = aligned(out, 32) && pitch % 32 == 0 ? 32 : aligned(out, 16) && pitch % 16 == 0 ? 16 : 0;
}

tcg_status launch_products(tcg::xent::Products& p, const ProductPlan& pl, cudaStream_t stream) {
    constexpr auto* kKernel = &tcg::xent::xent_product_kernel;
    const cudaError_t e = set_attributes<kKernel, tcg::xent::kProductSmem>();
    if (e != cudaSuccess) return tcg::host::fail_launch("tcg_linear_xent_backward kernel attributes", e);
    p.timeout_ns = tcg::host::wait_timeout_ns();
    p.fault_inject = tcg::host::fault_inject();
    return launch_ctas(kKernel, p, true, pl.workers, tcg::xent::kProductSmem, stream);
}

tcg_status check(int tokens, int vocab, int hidden, tcg_dtype dtype, const void* X, int ldx, const void* W, int ldw,
                 const int* target) {
    if (tokens < 0 || vocab < 1 || hidden < 1) return TCG_ERR_INVALID_ARG;
    if (dtype != TCG_BF16 && dtype != TCG_F16) return TCG_ERR_INVALID_ARG;
    // (extents in bytes, and the number of tiles, are ints)
    if (tokens > tcg::host::kMaxExtent / 2 || vocab > tcg::host::kMaxExtent / 2 || hidden > tcg::host::kMaxExtent / 4 ||
        blocks(tokens, 128) * blocks(vocab, kMinTileN) > tcg::host::kMaxExtent / 2)
        return TCG_ERR_UNSUPPORTED;
    if (!W || ldw < hidden || (tokens > 0 && (!X || ldx < hidden || !target))) return TCG_ERR_INVALID_ARG;
    if (!aligned(X, 2) || !aligned(W, 2) || !aligned(target, 4)) return TCG_ERR_MISALIGNED;
    // what the TMA can address
    if (!aligned(W, 16) || ldw % 8 || (tokens > 0 && (!aligned(X, 16) || ldx % 8))) return TCG_ERR_UNSUPPORTED;
    return TCG_OK;
}

tcg_status check_gradient(const void* d, int ld, int hidden, tcg_dtype t) {
    if (!d) return TCG_OK;
    if (t != TCG_BF16 && t != TCG_F16 && t != TCG_F32) return TCG_ERR_INVALID_ARG;
    if (ld < hidden) return TCG_ERR_INVALID_ARG;
    return aligned(d, size_of(t)) ? TCG_OK : TCG_ERR_MISALIGNED;
}

}  // namespace

extern "C" {

size_t tcg_linear_xent_workspace_size(int tokens, int vocab, int hidden, int backward) {
    if (tokens < 0 || vocab < 1 || hidden < 1) return 0;
    tcg::host::Device dev;
    if (tcg::host::device(dev) != TCG_OK) dev.num_sms = 1024;
    const size_t forward = forward_layout(tokens, vocab).bytes;
    return backward ? std::max(forward, backward_layout(tokens, vocab, hidden, dev.num_sms).bytes) : forward;
}

tcg_status tcg_linear_xent(int tokens, int vocab, int hidden, tcg_dtype dtype, const void* X, int ldx, const void* W, int ldw,
                           const int* target, float* lse, float* loss, float* mean, int* num_valid, void* workspace,
                           size_t workspace_bytes, void* stream) {
    tcg_status st = check(tokens, vocab, hidden, dtype, X, ldx, W, ldw, target);
    if (st != TCG_OK) return st;
    if (!mean || !num_valid || (tokens > 0 && !lse)) return TCG_ERR_INVALID_ARG;
    if (!aligned(lse, 4) || !aligned(loss, 4) || !aligned(mean, 4) || !aligned(num_valid, 4)) return TCG_ERR_MISALIGNED;
    tcg::host::Device dev;
    if ((st = tcg::host::device(dev)) != TCG_OK) return st;
    const Layout l = forward_layout(tokens, vocab);
    if (!workspace || !aligned(workspace, 16) || workspace_bytes < l.bytes)
        return tcg::host::fail(TCG_ERR_WORKSPACE, "workspace NULL, not 16-byte aligned or smaller than tcg_linear_xent_workspace_size");
    char* ws = static_cast<char*>(workspace);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    Params p;
    memset(&p, 0, sizeof p);
    p.target = target;
    p.part = reinterpret_cast<float2*>(ws + l.part);
    p.picked = reinterpret_cast<float*>(ws + l.picked);
    p.status = reinterpret_cast<int*>(ws);
    if (tokens > 0 && (st = launch_tiles<false>(p, dtype, X, ldx, W, ldw, tokens, hidden, 0, vocab, dev, s)) != TCG_OK) return st;
    Finish f = {};
    f.part = p.part;
    f.num_n = 2 * p.num_n;
    f.tokens = tokens;
    f.vocab = vocab;
    f.picked = p.picked;
    f.target = target;
    f.lse = lse;
    f.loss = loss;
    f.mean = mean;
    f.valid = num_valid;
    f.sums = reinterpret_cast<double*>(ws + l.sums);
    f.counts = reinterpret_cast<int*>(ws + l.counts);
    f.arrivals = reinterpret_cast<int*>(ws + tcg::host::kWorkspaceHeader);
    const dim3 grid(static_cast<unsigned>(std::max(1LL, blocks(tokens, kFinishRows))));
    const cudaError_t e = tcg::host::launch_early(finish_kernel, grid, kFinishThreads, s, f);
    return e == cudaSuccess ? TCG_OK : tcg::host::fail_launch("tcg_linear_xent", e);
}

tcg_status tcg_linear_xent_backward(int tokens, int vocab, int hidden, tcg_dtype dtype, const void* X, int ldx, const void* W,
                                    int ldw, const int* target, const float* lse, const int* num_valid, const float* grad_mean,
                                    const float* grad_loss, void* dX, int lddx, tcg_dtype dx_dtype, float dw_beta, void* dW,
                                    int lddw, tcg_dtype dw_dtype, void* workspace, size_t workspace_bytes, void* stream) {
    tcg_status st = check(tokens, vocab, hidden, dtype, X, ldx, W, ldw, target);
    if (st == TCG_OK) st = check_gradient(dX, lddx, hidden, dx_dtype);
    if (st == TCG_OK) st = check_gradient(dW, lddw, hidden, dw_dtype);
    if (st != TCG_OK) return st;
    if (!num_valid || (tokens > 0 && !lse)) return TCG_ERR_INVALID_ARG;
    if (!aligned(lse, 4) || !aligned(num_valid, 4) || !aligned(grad_mean, 4) || !aligned(grad_loss, 4)) return TCG_ERR_MISALIGNED;
    tcg::host::Device dev;
    if ((st = tcg::host::device(dev)) != TCG_OK) return st;
    const Layout l = backward_layout(tokens, vocab, hidden, dev.num_sms);
    if (!workspace || !aligned(workspace, 16) || workspace_bytes < l.bytes)
        return tcg::host::fail(TCG_ERR_WORKSPACE, "workspace NULL, not 16-byte aligned or smaller than tcg_linear_xent_workspace_size");
    if (!dX && !dW) return TCG_OK;
    // (no tokens: dW is dw_beta times itself, which a product over no tokens at all gives as well)
    char* ws = static_cast<char*>(workspace);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int words = piece_words(tokens, vocab), pitch = pitch_of(words), ld = pitch_of(hidden);
    float* back = reinterpret_cast<float*>(ws + l.back);
    float* dx32 = reinterpret_cast<float*>(ws + l.dx);
    char* dz = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(ws + l.dz) + kWord - 1) & ~uintptr_t(kWord - 1));
    for (int v0 = 0; v0 < vocab; v0 += words) {
        const int n = std::min(words, vocab - v0);
        const bool last = v0 + n == vocab;
        const char* w = static_cast<const char*>(W) + static_cast<size_t>(v0) * ldw * 2;
        tcg::xent::Products q;
        memset(&q, 0, sizeof q);
        if (tokens > 0) {
            Params p;
            memset(&p, 0, sizeof p);
            p.target = target;
            p.lse = lse;
            p.valid = num_valid;
            p.grad_mean = grad_mean;
            p.grad_loss = grad_loss;
            p.vocab = vocab;
            p.top = dtype == TCG_F16 ? kHalfTop : 1.0f;
            p.back = back;
            p.d = dz;
            p.ldd = pitch;
            p.status = reinterpret_cast<int*>(ws);
            if ((st = launch_tiles<true>(p, dtype, X, ldx, W, ldw, tokens, hidden, v0, n, dev, s)) != TCG_OK) return st;
            // dz as the rows operand of both, its words or its tokens being K
            CUtensorMap map_dz;
            st = tcg::host::map_bytes(&map_dz, dz, 2ull * n, tokens, 2ull * pitch, tcg::xent::kRowBytes, tcg::xent::kStageK);
            q.q[0].a = q.q[1].a = map_dz;
            if (st == TCG_OK) st = tcg::host::map_bytes(&q.q[0].b, w, 2ull * hidden, n, 2ull * ldw, tcg::xent::kRowBytes, tcg::xent::kStageK);
            if (st == TCG_OK) st = tcg::host::map_bytes(&q.q[1].b, X, 2ull * hidden, tokens, 2ull * ldx, tcg::xent::kRowBytes, tcg::xent::kStageK);
            if (st != TCG_OK) return st;
        }
        q.tile_n = product_columns(tokens, hidden, dX != nullptr);
        q.fmt = dtype == TCG_F16 ? 0u : 1u;
        q.back = tokens > 0 ? back : nullptr;
        q.partials = reinterpret_cast<float*>(ws + l.partials);
        q.counters = reinterpret_cast<int*>(ws + tcg::host::kWorkspaceHeader);
        q.status = reinterpret_cast<int*>(ws);
        q.q[1].a_along_m = 1;
        for (int i = 0; i < 2; ++i) {
            tcg::xent::Product& one = q.q[i];
            one.M = i == 0 ? tokens : n;
            one.N = hidden;
            one.num_kb = static_cast<int>(blocks(i == 0 ? n : tokens, tcg::xent::kStageK));
            one.num_n = static_cast<int>(blocks(hidden, q.tile_n));
            one.num_m = (i == 0 ? dX : dW) ? static_cast<int>(blocks(one.M, 2 * tcg::xent::kBM)) : 0;
            one.splits = 1;
        }
        // dX: fp32 sums of the pieces so far, in dX itself where it is fp32
        if (dX && tokens > 0) {
            if (dx_dtype == TCG_F32) set_output(q.q[0], dX, lddx, TCG_F32, v0 > 0 ? 1.0f : 0.0f);
            else if (!last) set_output(q.q[0], dx32, ld, TCG_F32, v0 > 0 ? 1.0f : 0.0f);
            else set_output(q.q[0], dX, lddx, dx_dtype, 0.0f);
            if (dx_dtype != TCG_F32 && last && v0 > 0) {
                q.q[0].sum = dx32;
                q.q[0].ld_sum = ld;
            }
        }
        if (dW)
            set_output(q.q[1], static_cast<char*>(dW) + static_cast<size_t>(v0) * lddw * size_of(dw_dtype), lddw, dw_dtype, dw_beta);
        const long long first = static_cast<long long>(q.q[0].num_m) * q.q[0].num_n, second = static_cast<long long>(q.q[1].num_m) * q.q[1].num_n;
        const ProductPlan pl = plan_products(first, q.q[0].num_kb, second, q.q[1].num_kb, std::max(1, dev.num_sms / 2));
        q.q[0].splits = pl.splits;
        q.early = pl.early;
        if (first + second > 0 && (st = launch_products(q, pl, s)) != TCG_OK) return st;
    }
    return TCG_OK;
}

}  // extern "C"
