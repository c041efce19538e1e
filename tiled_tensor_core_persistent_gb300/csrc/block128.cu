// block128.cu -- C ABI of the 8-bit products with one fp32 scale per 128 K:
// argument checks, the choice of tile, the launch.  Kernels: block128_kernel.cuh.
#include <algorithm>
#include <climits>
#include <cstring>

#include "block128_kernel.cuh"
#include "host.h"

namespace {

using tcg::b128::Params;

enum Tile { kPairTile, kOneTile, kFew16, kFew32 };

struct Plan {
    Tile tile = kOneTile;
    bool stream = false;
    int workers = 1;   // CTAs, or CTA pairs
};

int tile_cols(Tile t) { return t == kPairTile ? 256 : t == kOneTile ? 128 : t == kFew16 ? 16 : 32; }
bool few(Tile t) { return t == kFew16 || t == kFew32; }

size_t workspace_bytes(const Plan& pl) {
    if (!pl.stream) return tcg::host::kWorkspaceHeader;
    return tcg::host::kScratchAt + static_cast<size_t>(2) * pl.workers * 128 * tile_cols(pl.tile) * sizeof(float);
}

long long blocks(long long n, int b) { return (n + b - 1) / b; }

// Pair tiles run in whole waves, a k-block of a wave in 0.57 us; single tiles
// deal their k-blocks out evenly, a quarter of a pair tile's work in 0.46 us.
// (512 x 8192 x 8192, 64 pair tiles: 57.7 us in single tiles, 41.6 in one wave of
// pairs; 1024 rows: 100 and 77 us.)
bool pair_pays(long long tiles, int sms) { return 5 * blocks(tiles, sms / 2) * sms <= 16 * tiles; }

// rows: rows of A a group has (dense: M).  groups: 1 for a dense product.
Plan make_plan(int mode, long long rows, int groups, int M, int N, int num_kb, int sms) {
    Plan pl;
    const long long per = groups > 0 ? (rows + groups - 1) / groups : rows;
    const long long pair_tiles = blocks(per, 256) * groups * blocks(N, 256);
    if (mode == tcg::b128::kGroupedK) {
        pl.tile = (M > 128 && N > 128 && blocks(M, 256) * blocks(N, 256) * groups * 2 >= sms) ? kPairTile : kOneTile;
        const long long tiles = static_cast<long long>(groups) *
                                (pl.tile == kPairTile ? blocks(M, 256) * blocks(N, 256) : blocks(M, 128) * blocks(N, 128));
        pl.workers = static_cast<int>(std::max(1LL, std::min<long long>(tiles, pl.tile == kPairTile ? sms / 2 : sms)));
        return pl;
    }
    // Few rows take the MMA's columns.  A grouped call does not know its longest
    // group: room for twice the mean.  Past 32 rows the 128-row tile is ahead
    // (64 x 4096 x 4096: 21 us; with 64 columns 28 us).
    const long long want = mode == tcg::b128::kGroupedRows ? 2 * per : per;
    if (want <= 32) {
        pl.tile = want <= 16 ? kFew16 : kFew32;
    } else if (per > 128 && N > 128 && pair_pays(pair_tiles, sms)) {
        pl.tile = kPairTile;
    }
    pl.stream = pl.tile != kPairTile && num_kb > 0;
    const int tm = few(pl.tile) ? tile_cols(pl.tile) : (pl.tile == kPairTile ? 256 : 128);
    const int tn = few(pl.tile) ? 128 : tile_cols(pl.tile);
    // (grouped: at most one partly filled tile row per group)
    const long long tile_rows = mode == tcg::b128::kGroupedRows ? rows / tm + std::min<long long>(groups, rows) : blocks(rows, tm);
    long long units = tile_rows * blocks(N, tn);
    if (pl.stream) units *= std::max(1, num_kb / 4);   // a run of fewer k-blocks than a pipeline holds gains nothing
    pl.workers = static_cast<int>(std::max(1LL, std::min<long long>(units, pl.tile == kPairTile ? sms / 2 : sms)));
    // (a counter each)
    if (pl.stream) pl.workers = std::min(pl.workers, static_cast<int>(tcg::host::kCounterBytes / sizeof(int)));
    return pl;
}

template <int TN, bool kPair, bool kSwap, bool kCol>
tcg_status launch(Params& p, const Plan& pl, const tcg::host::Device& dev, cudaStream_t stream) {
    using S = tcg::b128::Shape<TN, kPair, kSwap, kCol>;
    auto* kernel = tcg::b128::block128_kernel<TN, kPair, kSwap, kCol>;
    static tcg::host::OncePerDevice once;
    const cudaError_t err = once([&] {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, tcg::b128::kSmemBytes);
        cudaFuncAttributes a;
        if (e == cudaSuccess) e = cudaFuncGetAttributes(&a, kernel);
        // the register hand-over draws on what the block is launched with
        if (e == cudaSuccess && S::kSplitRegs && a.numRegs < S::kLaunchRegs) e = cudaErrorInvalidConfiguration;
        return e;
    });
    if (err != cudaSuccess) return tcg::host::fail_launch("tcg_gemm_block128 kernel attributes", err);
    const int tables = p.mode == tcg::b128::kDense ? 0 : p.mode == tcg::b128::kGroupedK ? 1 : 2;
    p.stages = std::min(S::kMaxStages, (dev.max_smem_optin - S::smem_bytes(0, tables, p.num_groups)) / S::kStageBytes);
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof cfg);
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3((kPair ? 2 : 1) * pl.workers);
    cfg.blockDim = dim3(S::kThreads);
    cfg.dynamicSmemBytes = S::smem_bytes(p.stages, tables, p.num_groups);
    cfg.stream = stream;
    // the blocks may be launched while the kernel ahead ends (they wait for it
    // before they read anything)
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (kPair) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = 2;
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
    return e == cudaSuccess ? TCG_OK : tcg::host::fail_launch("cudaLaunchKernelEx", e);
}

tcg_status launch_plan(Params& p, const Plan& pl, bool col, const tcg::host::Device& dev, cudaStream_t s) {
    switch (pl.tile) {
        case kPairTile: return col ? launch<256, true, false, true>(p, pl, dev, s) : launch<256, true, false, false>(p, pl, dev, s);
        case kOneTile: return col ? launch<128, false, false, true>(p, pl, dev, s) : launch<128, false, false, false>(p, pl, dev, s);
        case kFew16: return launch<16, false, true, false>(p, pl, dev, s);
        case kFew32: return launch<32, false, true, false>(p, pl, dev, s);
    }
    return TCG_ERR_INVALID_ARG;
}

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
int out_bytes(tcg_dtype t) { return t == TCG_F32 ? 4 : 2; }

tcg_status check_operand(const tcg_block_operand& o, int K, bool must_be_rows) {
    if (o.scale_rows != 1 && o.scale_rows != 128) return TCG_ERR_INVALID_ARG;
    if (must_be_rows && o.scale_rows != 1) return TCG_ERR_UNSUPPORTED;
    if (K == 0) return TCG_OK;
    if (!o.data || !o.scales || o.ld < K) return TCG_ERR_INVALID_ARG;
    if (!aligned(o.scales, 4)) return TCG_ERR_MISALIGNED;
    if (!aligned(o.data, 16) || o.ld % 16) return TCG_ERR_UNSUPPORTED;   // what the TMA can address
    if (o.row_stride < 0 || o.k_stride < 0 || o.group_stride < 0) return TCG_ERR_INVALID_ARG;
    return TCG_OK;
}

tcg_status check_output(int N, float beta, const void* C, int ldc, tcg_dtype c_dtype, const void* D, int ldd,
                        tcg_dtype d_dtype) {
    if (d_dtype != TCG_BF16 && d_dtype != TCG_F32) return TCG_ERR_INVALID_ARG;
    if (!D || ldd < N) return TCG_ERR_INVALID_ARG;
    if (!aligned(D, out_bytes(d_dtype))) return TCG_ERR_MISALIGNED;
    if (beta != 0.0f) {
        if (c_dtype != TCG_BF16 && c_dtype != TCG_F32) return TCG_ERR_INVALID_ARG;
        if (!C || ldc < N) return TCG_ERR_INVALID_ARG;
        if (!aligned(C, out_bytes(c_dtype))) return TCG_ERR_MISALIGNED;
    }
    return TCG_OK;
}

tcg::b128::ScaleRef scale_ref(const tcg_block_operand& o) {
    tcg::b128::ScaleRef s;
    s.ptr = o.scales;
    s.rs = o.row_stride;
    s.ks = o.k_stride;
    s.gs = o.group_stride;
    s.shift = o.scale_rows == 128 ? 7 : 0;
    return s;
}

void set_output(Params& p, float beta, const void* C, int ldc, tcg_dtype c_dtype, void* D, int ldd, tcg_dtype d_dtype) {
    p.beta = beta;
    p.C = beta != 0.0f ? C : nullptr;
    p.ldc = ldc;
    p.c_f32 = c_dtype == TCG_F32;
    p.c_vec = beta != 0.0f && aligned(C, 16) && (static_cast<long long>(ldc) * out_bytes(c_dtype)) % 16 == 0;
    p.D = D;
    p.ldd = ldd;
    p.d_f32 = d_dtype == TCG_F32;
    const long long pitch = static_cast<long long>(ldd) * out_bytes(d_dtype);
    p.d_vec = aligned(D, 32) && pitch % 32 == 0 ? 32 : (aligned(D, 16) && pitch % 16 == 0 ? 16 : 0);
}

// a_rows / b_rows: rows of the operands in memory
tcg_status run(Params& p, const Plan& pl, const tcg_block_operand& A, const tcg_block_operand& B, long long a_rows,
               long long b_rows, int K, const tcg::host::Device& dev, void* workspace, size_t ws_bytes, void* stream) {
    if (!workspace || !aligned(workspace, 16) || ws_bytes < workspace_bytes(pl))
        return tcg::host::fail(TCG_ERR_WORKSPACE, "workspace NULL, not 16-byte aligned or smaller than tcg_block128_workspace_size");
    char* ws = static_cast<char*>(workspace);
    p.status = reinterpret_cast<int*>(ws);
    p.counters = reinterpret_cast<int*>(ws + tcg::host::kWorkspaceHeader);
    p.partials = reinterpret_cast<float*>(ws + tcg::host::kScratchAt);
    p.stream = pl.stream;
    p.timeout_ns = tcg::host::wait_timeout_ns();
    p.fault_inject = tcg::host::fault_inject();
    const int tn = tile_cols(pl.tile);
    if (p.num_kb > 0) {
        const int box_a = few(pl.tile) ? tn : 128;
        const int box_b = pl.tile == kPairTile ? tn / 2 : 128;
        tcg_status st = tcg::host::map_bytes(&p.tmA, A.data, K, a_rows, A.ld, 128, box_a);
        if (st == TCG_OK) st = tcg::host::map_bytes(&p.tmB, B.data, K, b_rows, B.ld, 128, box_b);
        if (st != TCG_OK) return st;
    }
    const int tm = few(pl.tile) ? tn : (pl.tile == kPairTile ? 256 : 128);
    p.num_m = static_cast<int>(blocks(p.M, tm));
    p.num_n = static_cast<int>(blocks(p.N, few(pl.tile) ? 128 : tn));
    p.raster_m = 16;
    return launch_plan(p, pl, B.scale_rows == 1, dev, static_cast<cudaStream_t>(stream));
}

uint32_t format_of(tcg_dtype t) { return t == TCG_E5M2 ? 1u : 0u; }

}  // namespace

extern "C" {

size_t tcg_block128_workspace_size(int num_groups, int M, int N, int K) {
    if (num_groups < 0 || M < 0 || N < 0 || K < 0) return 0;
    tcg::host::Device dev;
    if (tcg::host::device(dev) != TCG_OK) dev.num_sms = 1024;
    if (M == 0 || N == 0) return tcg::host::kWorkspaceHeader;
    const int mode = num_groups > 0 ? tcg::b128::kGroupedRows : tcg::b128::kDense;
    return workspace_bytes(make_plan(mode, M, std::max(1, num_groups), M, N, static_cast<int>(blocks(K, 128)), dev.num_sms));
}

tcg_status tcg_gemm_block128(int M, int N, int K, tcg_dtype ab_dtype, tcg_block_operand A, tcg_block_operand B,
                             float beta, const void* C, int ldc, tcg_dtype c_dtype, void* D, int ldd,
                             tcg_dtype d_dtype, tcg_epilogue epi, void* workspace, size_t workspace_bytes,
                             void* stream) {
    if (M < 0 || N < 0 || K < 0) return TCG_ERR_INVALID_ARG;
    if (ab_dtype != TCG_E4M3 && ab_dtype != TCG_E5M2) return TCG_ERR_INVALID_ARG;
    if (epi.act != TCG_ACT_NONE && epi.act != TCG_ACT_RELU && epi.act != TCG_ACT_GELU) return TCG_ERR_INVALID_ARG;
    if (epi.bias && epi.bias_dtype != TCG_BF16 && epi.bias_dtype != TCG_F32) return TCG_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return TCG_OK;
    if (std::max({M, N, K}) > tcg::host::kMaxExtent) return TCG_ERR_UNSUPPORTED;
    tcg_status st = check_operand(A, K, true);
    if (st == TCG_OK) st = check_operand(B, K, false);
    if (st == TCG_OK) st = check_output(N, beta, C, ldc, c_dtype, D, ldd, d_dtype);
    if (st != TCG_OK) return st;
    if (epi.bias && !aligned(epi.bias, out_bytes(epi.bias_dtype))) return TCG_ERR_MISALIGNED;
    tcg::host::Device dev;
    if ((st = tcg::host::device(dev)) != TCG_OK) return st;
    Params p;
    memset(&p, 0, sizeof p);
    p.mode = tcg::b128::kDense;
    p.M = M;
    p.N = N;
    p.num_kb = static_cast<int>(blocks(K, 128));
    p.sa = scale_ref(A);
    p.sb = scale_ref(B);
    p.ab_fmt = format_of(ab_dtype);
    p.bias = epi.bias;
    p.bias_f32 = epi.bias_dtype == TCG_F32;
    p.act = static_cast<int>(epi.act);
    set_output(p, beta, C, ldc, c_dtype, D, ldd, d_dtype);
    const Plan pl = make_plan(p.mode, M, 1, M, N, p.num_kb, dev.num_sms);
    return run(p, pl, A, B, M, N, K, dev, workspace, workspace_bytes, stream);
}

tcg_status tcg_gemm_block128_grouped(int num_groups, const int* offsets, int rows, int N, int K, tcg_dtype ab_dtype,
                                     tcg_block_operand A, tcg_block_operand B, void* D, int ldd, tcg_dtype d_dtype,
                                     void* workspace, size_t workspace_bytes, void* stream) {
    if (num_groups < 0 || rows < 0 || N < 0 || K < 0) return TCG_ERR_INVALID_ARG;
    if (ab_dtype != TCG_E4M3 && ab_dtype != TCG_E5M2) return TCG_ERR_INVALID_ARG;
    if (num_groups == 0 || rows == 0 || N == 0) return TCG_OK;
    if (num_groups > tcg::b128::kMaxGroups || std::max(rows, K) > tcg::host::kMaxExtent ||
        static_cast<long long>(num_groups) * N > tcg::host::kMaxExtent)
        return TCG_ERR_UNSUPPORTED;
    if (!offsets) return TCG_ERR_INVALID_ARG;
    if (!aligned(offsets, 4)) return TCG_ERR_MISALIGNED;
    tcg_status st = check_operand(A, K, true);
    if (st == TCG_OK) st = check_operand(B, K, false);
    if (st == TCG_OK) st = check_output(N, 0.0f, nullptr, 0, TCG_F32, D, ldd, d_dtype);
    if (st != TCG_OK) return st;
    tcg::host::Device dev;
    if ((st = tcg::host::device(dev)) != TCG_OK) return st;
    Params p;
    memset(&p, 0, sizeof p);
    p.mode = tcg::b128::kGroupedRows;
    p.M = rows;
    p.N = N;
    p.num_kb = static_cast<int>(blocks(K, 128));
    p.num_groups = num_groups;
    p.offsets = offsets;
    p.sa = scale_ref(A);
    p.sb = scale_ref(B);
    p.ab_fmt = format_of(ab_dtype);
    set_output(p, 0.0f, nullptr, 0, TCG_F32, D, ldd, d_dtype);
    const Plan pl = make_plan(p.mode, rows, num_groups, rows, N, p.num_kb, dev.num_sms);
    return run(p, pl, A, B, rows, static_cast<long long>(num_groups) * N, K, dev, workspace, workspace_bytes, stream);
}

tcg_status tcg_gemm_block128_grouped_k(int num_groups, const int* offsets, int M, int N, int padded_rows,
                                       tcg_dtype ab_dtype, tcg_block_operand A, tcg_block_operand B, float beta,
                                       const void* C, int ldc, tcg_dtype c_dtype, void* D, int ldd,
                                       tcg_dtype d_dtype, void* workspace, size_t workspace_bytes, void* stream) {
    if (num_groups < 0 || M < 0 || N < 0 || padded_rows < 0) return TCG_ERR_INVALID_ARG;
    if (ab_dtype != TCG_E4M3 && ab_dtype != TCG_E5M2) return TCG_ERR_INVALID_ARG;
    if (num_groups == 0 || M == 0 || N == 0) return TCG_OK;
    if (num_groups > tcg::b128::kMaxGroups || std::max(N, padded_rows) > tcg::host::kMaxExtent ||
        static_cast<long long>(num_groups) * M > tcg::host::kMaxExtent ||
        static_cast<long long>(num_groups) * blocks(M, 128) * blocks(N, 128) > INT_MAX)
        return TCG_ERR_UNSUPPORTED;
    if (padded_rows % 128) return TCG_ERR_INVALID_ARG;
    if (!offsets) return TCG_ERR_INVALID_ARG;
    if (!aligned(offsets, 4)) return TCG_ERR_MISALIGNED;
    tcg_status st = check_operand(A, padded_rows, true);
    if (st == TCG_OK) st = check_operand(B, padded_rows, true);
    if (st == TCG_OK) st = check_output(N, beta, C, ldc, c_dtype, D, ldd, d_dtype);
    if (st != TCG_OK) return st;
    tcg::host::Device dev;
    if ((st = tcg::host::device(dev)) != TCG_OK) return st;
    Params p;
    memset(&p, 0, sizeof p);
    p.mode = tcg::b128::kGroupedK;
    p.M = M;
    p.N = N;
    p.num_kb = padded_rows / 128;
    p.num_groups = num_groups;
    p.offsets = offsets;
    p.sa = scale_ref(A);
    p.sb = scale_ref(B);
    p.ab_fmt = format_of(ab_dtype);
    set_output(p, beta, C, ldc, c_dtype, D, ldd, d_dtype);
    const Plan pl = make_plan(p.mode, 0, num_groups, M, N, p.num_kb, dev.num_sms);
    return run(p, pl, A, B, M, N, padded_rows, dev, workspace, workspace_bytes, stream);
}

}  // extern "C"
