// xent_kernel.cuh -- the product X @ W^T of hidden states and a vocabulary's
// weights whose tiles never reach memory: a forward kernel that keeps each
// row's softmax statistics, and a backward one that turns a tile into the
// loss's gradient with respect to its logits.
//
//   z_tv = sum_h X_th W_vh                                   (fp32, in TMEM)
//   forward:  for each tile and row  M = max_v z_tv log2(e),  s = sum_v 2^(z_tv log2(e) - M),
//             and z_ty where the row's target y lies in the tile
//   backward: d_tv = r_t (2^((z_tv - lse_t) log2(e)) - [v = y_t]), rounded to the
//             operands' type
//
// Tiles of 256 rows (a pair of CTAs; 128, one CTA, where there are no more rows
// than that) and up to 256 columns; the width is the one whose waves fit
// (the launcher's rule).  Roles: warp 0 TMA producer, warp 1 MMA issuer and TMEM
// owner, warps 2-5 read the accumulator, a row a thread, one of two so that a
// tile's exponentials run beside the next tile's products.  A tile of 128 rows
// of a CTA is 8 H cycles of the tensor cores (H = hidden) and 2048 of its
// exponentials, so H >= 512 hides them.  All waits are bounded; on expiry the
// status word gets TCG_ERR_TIMEOUT, the roles drain their copies and MMAs, free
// the TMEM and return.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "host.h"
#include "ptx.cuh"
#include "values.cuh"

namespace tcg {
namespace xent {

constexpr float kLog2e = 1.44269504088896341f;
constexpr int kThreads = 192;
constexpr int kRowBytes = 128;          // one K atom: a 128-byte swizzle row, 64 elements
constexpr int kBM = 128;                // rows of a CTA's tile = TMEM lanes
constexpr int kMaxN = 256;
constexpr int kAccCols = 256;           // columns between the two accumulators

struct Params {
    CUtensorMap tmX, tmW;               // as bytes
    int tokens, cols;                   // rows of X, and of W in this launch
    int num_m, num_n, num_kb;           // tiles; pipeline stages of K
    int tile_n, raster_m;
    uint32_t fmt;                       // operand format of the instruction descriptor: 0 fp16, 1 bf16
    const int* target;                  // [tokens]
    int first;                          // the word of W's first row
    // forward
    float2* part;                       // [column tile][tokens]: (M, s)
    float* picked;                      // [tokens]: z of the target
    // backward
    const float* lse;                   // [tokens]
    const float* scale;                 // [tokens]: r_t
    void* d;
    long long ldd;                      // a multiple of 32
    int* status;
    long long timeout_ns;
    int fault_inject;
};

template <bool kPair>
struct Shape {
    static constexpr int kAtoms = kPair ? 2 : 1;                 // K atoms a stage
    static constexpr int kTileM = kPair ? 2 * kBM : kBM;
    static constexpr int kBRows = kPair ? kMaxN / 2 : kMaxN;     // rows of W a CTA has room for
    static constexpr int kABytes = kAtoms * kBM * kRowBytes;
    static constexpr int kBBytes = kAtoms * kBRows * kRowBytes;
    static constexpr int kStageBytes = kABytes + kBBytes;
    static constexpr int kStages = kPair ? 3 : 4;
    static constexpr int kSmemBytes = kStages * kStageBytes + 1024 + 512;   // alignment, barriers
};

struct alignas(16) Ctl {
    uint64_t full[4], empty[4];
    uint64_t tmem_full[2], tmem_empty[2];
    uint64_t drain;
    uint32_t tmem_base;
    int abort_flag;
};
static_assert(sizeof(Ctl) <= 512, "the barriers fit");

static __device__ __noinline__ bool spin(uint64_t* bar, uint32_t parity, int* status, long long limit_ns, Ctl* ctl, int where,
                                         bool honor_abort) {
    const uint32_t a = ptx::smem_u32(bar);
    const uint64_t t0 = ptx::globaltimer_ns();
    for (uint32_t n = 1;; ++n) {
        if (ptx::mbar_try_wait(a, parity)) return true;
        if (n & 31u) continue;
        if (honor_abort && *reinterpret_cast<volatile int*>(&ctl->abort_flag)) return false;
        if (static_cast<long long>(ptx::globaltimer_ns() - t0) > limit_ns) {
            *reinterpret_cast<volatile int*>(&ctl->abort_flag) = 1;
            if (atomicCAS(status, 0, static_cast<int>(TCG_ERR_TIMEOUT)) == 0) {
                status[1] = where;
                status[2] = static_cast<int>(blockIdx.x);
            }
            return false;
        }
    }
}

// The whole warp waits on one barrier and agrees on the outcome.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, const Params& p, Ctl* ctl, int where, bool honor_abort = true) {
    bool ok = ptx::mbar_try_wait(ptx::smem_u32(bar), parity);
    if (!ok) ok = spin(bar, parity, p.status, p.timeout_ns, ctl, where, honor_abort);
    return __all_sync(0xffffffffu, ok);
}

// Tile -> (row tile, column tile): raster_m row tiles are walked before the next
// column tile, so the CTAs at work share the columns' weights in L2.
__host__ __device__ __forceinline__ void tile_of(const Params& p, int tile, int& m, int& n) {
    const int span = p.raster_m * p.num_n, group = tile / span, first = group * p.raster_m;
    const int size = p.num_m - first < p.raster_m ? p.num_m - first : p.raster_m, local = tile - group * span;
    m = first + local % size;
    n = local / size;
}

// 32 columns of a warp's 32 TMEM lanes; the values are there after landed().
__device__ __forceinline__ void fetch32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void landed(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                   "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                   "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                   "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}

// One row's running maximum (times log2 e) and sum.
struct RowStats {
    float m = -INFINITY, m2 = -INFINITY, s = 0.0f;

    __device__ __forceinline__ void add(const float (&z)[32]) {
        float c = z[0];
#pragma unroll
        for (int i = 1; i < 32; ++i) c = fmaxf(c, z[i]);
        if (c > m) {
            const float next = c * kLog2e;
            s = m == -INFINITY ? s : s * ptx::ex2_approx(m2 - next);   // (s holds NaN, if any, from here on)
            m = c;
            m2 = next;
        }
        const float base = m == -INFINITY ? 0.0f : m2;
        float q[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < 32; ++i) q[i & 3] += ptx::ex2_approx(fmaf(z[i], kLog2e, -base));
        s += (q[0] + q[1]) + (q[2] + q[3]);
    }
};

// kGrad: false the statistics, true the logits' gradient.  T: the operands' type
// (the gradient's, that is).
template <typename T, bool kPair, bool kGrad>
__global__ void __launch_bounds__(kThreads, 1) xent_kernel(const __grid_constant__ Params p) {
    using S = Shape<kPair>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Ctl* ctl = reinterpret_cast<Ctl*>(smem + S::kStages * S::kStageBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = kPair ? ptx::cluster_ctarank() : 0u;
    const bool leader = rank == 0;
    const int worker = kPair ? static_cast<int>(blockIdx.x >> 1) : static_cast<int>(blockIdx.x);
    const int workers = kPair ? static_cast<int>(gridDim.x >> 1) : static_cast<int>(gridDim.x);
    const int tiles = p.num_m * p.num_n;
    constexpr uint32_t kTmemCols = 512;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            ptx::mbar_init(&ctl->full[s], 1);
            ptx::mbar_init(&ctl->empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            ptx::mbar_init(&ctl->tmem_full[a], 1);
            ptx::mbar_init(&ctl->tmem_empty[a], kPair ? 8 : 4);
        }
        ptx::mbar_init(&ctl->drain, 1);
        ctl->abort_flag = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 1) {
        if constexpr (kPair) {
            ptx::tmem_alloc_pair(&ctl->tmem_base, kTmemCols);
            ptx::tmem_relinquish_alloc_permit_pair();
        } else {
            ptx::tmem_alloc(&ctl->tmem_base, kTmemCols);
            ptx::tmem_relinquish_alloc_permit();
        }
    }
    ptx::tc_fence_before_sync();
    if constexpr (kPair) ptx::cluster_sync();   // the peer's barriers exist before anyone signals them
    else __syncthreads();
    ptx::tc_fence_after_sync();
    const uint32_t tmem_base = ctl->tmem_base;
    tcg::host::wait_for_kernel_ahead();

    if (warp == 0) {
        // ------------------------------------------------------ TMA producer
        const bool issuer = lane == 0;
        const int b_rows = kPair ? p.tile_n / 2 : p.tile_n;
        const uint32_t tx = static_cast<uint32_t>((kPair ? 2 : 1) * S::kAtoms * (kBM + b_rows) * kRowBytes);
        if (issuer) {
            ptx::prefetch_tensormap(&p.tmX);
            ptx::prefetch_tensormap(&p.tmW);
        }
        int stage = 0;
        uint32_t phase = 0, armed = 0, armed_parity = 0;
        bool ok = true, first = true;
        for (int tile = worker; ok && tile < tiles; tile += workers) {
            int m, n;
            tile_of(p, tile, m, n);
            const int a_row = m * S::kTileM + static_cast<int>(rank) * kBM;
            const int b_row = n * p.tile_n + static_cast<int>(rank) * b_rows;
            for (int kb = 0; kb < p.num_kb; ++kb) {
                if (!wait(&ctl->empty[stage], phase ^ 1u, p, ctl, 1)) { ok = false; break; }
                const bool skip = first && p.fault_inject == 1 && blockIdx.x == 0;
                first = false;
                if (!skip && issuer) {
                    uint8_t* sA = smem + stage * S::kStageBytes;
                    uint8_t* sB = sA + S::kABytes;
                    uint64_t* fb = &ctl->full[stage];
                    if (leader) ptx::mbar_arrive_expect_tx(fb, tx);
                    const uint32_t fbc = kPair ? ptx::map_to_cta(ptx::smem_u32(fb), 0) : 0u;
#pragma unroll
                    for (int at = 0; at < S::kAtoms; ++at) {
                        const int x = (kb * S::kAtoms + at) * kRowBytes;
                        if constexpr (kPair) {
                            ptx::tma_load_2d_pair(sA + at * kBM * kRowBytes, &p.tmX, fbc, x, a_row);
                            ptx::tma_load_2d_pair(sB + at * S::kBRows * kRowBytes, &p.tmW, fbc, x, b_row);
                        } else {
                            ptx::tma_load_2d(sA + at * kBM * kRowBytes, &p.tmX, fb, x, a_row);
                            ptx::tma_load_2d(sB + at * S::kBRows * kRowBytes, &p.tmW, fb, x, b_row);
                        }
                    }
                }
                if (!skip) {
                    armed |= 1u << stage;
                    armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
                }
                __syncwarp();
                if (++stage == S::kStages) { stage = 0; phase ^= 1u; }
            }
        }
        // Every stage filled has landed before the CTA may leave (the leader sees
        // its own and the peer's copies on its full barriers; the peer sees its
        // stages consumed).
        for (int s = 0; s < S::kStages; ++s) {
            if (!(armed & (1u << s))) continue;
            const uint32_t par = (armed_parity >> s) & 1u;
            if (leader) wait(&ctl->full[s], par, p, ctl, 11, false);
            else wait(&ctl->empty[s], par, p, ctl, 13, false);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------- MMA issuer
        if (leader) {
            const bool issuer = lane == 0;
            const uint32_t idesc = (1u << 4) | (p.fmt << 7) | (p.fmt << 10) | (static_cast<uint32_t>(p.tile_n >> 3) << 17) |
                                   (static_cast<uint32_t>(S::kTileM >> 4) << 24);
            int stage = 0, t = 0;
            uint32_t phase = 0;
            bool ok = true, issued = false;
            for (int tile = worker; ok && tile < tiles; tile += workers, ++t) {
                const int acc = t & 1;
                if (!wait(&ctl->tmem_empty[acc], ((t >> 1) & 1) ^ 1u, p, ctl, 2)) break;
                ptx::tc_fence_after_sync();
                const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * kAccCols);
                for (int kb = 0; kb < p.num_kb; ++kb) {
                    if (!wait(&ctl->full[stage], phase, p, ctl, 3)) { ok = false; break; }
                    ptx::tc_fence_after_sync();
                    if (issuer) {
                        const uint32_t sA = ptx::smem_u32(smem + stage * S::kStageBytes);
                        const uint64_t a_desc = ptx::smem_desc_sw128(sA, 16, 1024);
                        const uint64_t b_desc = ptx::smem_desc_sw128(sA + S::kABytes, 16, 1024);
#pragma unroll
                        for (int k = 0; k < S::kAtoms * 4; ++k) {
                            // four MMAs of 32 bytes of K an atom; descriptors count 16-byte units
                            const uint64_t ad = a_desc + static_cast<uint64_t>(((k / 4) * kBM * kRowBytes + (k % 4) * 32) >> 4);
                            const uint64_t bd = b_desc + static_cast<uint64_t>(((k / 4) * S::kBRows * kRowBytes + (k % 4) * 32) >> 4);
                            const uint32_t accum = (kb > 0 || k > 0) ? 1u : 0u;
                            if constexpr (kPair) ptx::mma_f16_pair(d_tmem, ad, bd, idesc, accum);
                            else ptx::mma_f16(d_tmem, ad, bd, idesc, accum);
                        }
                        if constexpr (kPair) ptx::mma_commit_pair(&ctl->empty[stage], 0x3);
                        else ptx::mma_commit(&ctl->empty[stage]);
                    }
                    __syncwarp();
                    issued = true;
                    if (++stage == S::kStages) { stage = 0; phase ^= 1u; }
                }
                if (ok && issuer) {
                    if constexpr (kPair) ptx::mma_commit_pair(&ctl->tmem_full[acc], 0x3);
                    else ptx::mma_commit(&ctl->tmem_full[acc]);
                }
                __syncwarp();
            }
            // Every MMA is done before the TMEM is freed.
            if (issued) {
                if (issuer) {
                    if constexpr (kPair) ptx::mma_commit_pair(&ctl->drain, 0x1);
                    else ptx::mma_commit(&ctl->drain);
                }
                __syncwarp();
                wait(&ctl->drain, 0, p, ctl, 12, false);
            }
        }
    } else {
        // ------------------------------------- statistics, or the gradient
        const int g = warp & 3;                 // the TMEM lanes this warp may read
        int t = 0;
        for (int tile = worker; tile < tiles; tile += workers, ++t) {
            int m, n;
            tile_of(p, tile, m, n);
            const int row = m * S::kTileM + static_cast<int>(rank) * kBM + g * 32 + lane;
            const bool live = row < p.tokens;
            const int n0 = n * p.tile_n, width = min(p.tile_n, p.cols - n0);
            const int y = live ? p.target[row] : -1;
            // the target's place in this tile, negative or past it where it is elsewhere
            const long long at_tile = static_cast<long long>(y) - p.first - n0;
            const int at = y >= 0 && at_tile >= 0 && at_tile < width ? static_cast<int>(at_tile) : -1;
            float scale = 0.0f, lse2 = 0.0f;
            if constexpr (kGrad) {
                if (live) {
                    scale = p.scale[row];
                    lse2 = p.lse[row] * kLog2e;
                }
            }
            const int acc = t & 1;
            if (!wait(&ctl->tmem_full[acc], (t >> 1) & 1, p, ctl, 4)) break;
            ptx::tc_fence_after_sync();
            const uint32_t taddr = tmem_base + (static_cast<uint32_t>(g * 32) << 16) + static_cast<uint32_t>(acc * kAccCols);
            const int chunks = (width + 31) / 32;
            RowStats stats;
            uint32_t r[2][32];
            auto use = [&](uint32_t (&raw)[32], int c) {
                float z[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) z[i] = __uint_as_float(raw[i]);
                const int here = at - 32 * c;
                const bool any = __any_sync(0xffffffffu, static_cast<unsigned>(here) < 32u);
                if constexpr (kGrad) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) z[i] = ptx::ex2_approx(fmaf(z[i], kLog2e, -lse2));
                    if (any) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) z[i] -= i == here ? 1.0f : 0.0f;
                    }
                    // (a token that does not count has gradient 0, whatever its logits are)
#pragma unroll
                    for (int i = 0; i < 32; ++i) z[i] = scale == 0.0f ? 0.0f : scale * z[i];
                    if (live) {
                        T* dst = static_cast<T*>(p.d) + row * p.ldd + n0 + 32 * c;
                        uint32_t w[8];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) w[i] = pack_pair<T>(z[16 * h + 2 * i], z[16 * h + 2 * i + 1]);
                            ptx::st_global_v8(dst + 16 * h, w);
                        }
                    }
                } else {
                    if (any) {
                        float picked = 0.0f;
#pragma unroll
                        for (int i = 0; i < 32; ++i) picked = i == here ? z[i] : picked;
                        if (static_cast<unsigned>(here) < 32u) p.picked[row] = picked;
                    }
                    if (32 * c + 32 > width) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) z[i] = 32 * c + i < width ? z[i] : -INFINITY;
                    }
                    stats.add(z);
                }
            };
            // The next 32 columns are on their way while these are used; once the
            // last have left the TMEM the accumulator goes back.
            auto hand_back = [&] {
                ptx::tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    if (kPair && !leader) ptx::mbar_arrive_cluster(ptx::map_to_cta(ptx::smem_u32(&ctl->tmem_empty[acc]), 0));
                    else ptx::mbar_arrive(&ctl->tmem_empty[acc]);
                }
            };
            fetch32(taddr, r[0]);
            for (int c = 0; c < chunks; c += 2) {
                landed(r[0]);
                if (c + 1 < chunks) fetch32(taddr + static_cast<uint32_t>(32 * c + 32), r[1]);
                else hand_back();
                use(r[0], c);
                if (c + 1 < chunks) {
                    landed(r[1]);
                    if (c + 2 < chunks) fetch32(taddr + static_cast<uint32_t>(32 * c + 64), r[0]);
                    else hand_back();
                    use(r[1], c + 1);
                }
            }
            if constexpr (!kGrad) {
                if (live) p.part[static_cast<size_t>(n) * p.tokens + row] = make_float2(stats.m2, stats.s);
            }
        }
    }

    ptx::tc_fence_before_sync();
    if constexpr (kPair) ptx::cluster_sync();   // the leader's MMAs into the peer's TMEM are done
    else __syncthreads();
    if (warp == 1) {
        __syncwarp();
        ptx::tc_fence_after_sync();
        if constexpr (kPair) ptx::tmem_dealloc_pair(tmem_base, kTmemCols);
        else ptx::tmem_dealloc(tmem_base, kTmemCols);
    }
}

}  // namespace xent
}  // namespace tcg
