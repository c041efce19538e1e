// xent_kernel.cuh -- the product X @ W^T of hidden states and a vocabulary's
// weights whose tiles never reach memory: a forward kernel that keeps each
// row's softmax statistics, and a backward one that turns a tile into the
// loss's gradient with respect to its logits.
//
//   z_tv = sum_h X_th W_vh                                   (fp32, in TMEM)
//   forward:  for each tile and row  M = max_v z_tv log2(e),  s = sum_v 2^(z_tv log2(e) - M),
//             and z_ty where the row's target y lies in the tile
//   backward: r_t = grad_mean / n + grad_loss_t (0 where y is no word), and
//             d_tv = top r_t / max |r| (2^((z_tv - lse_t) log2(e)) - [v = y_t]), rounded to
//             the operands' type
//
// Tiles of 256 rows (a pair of CTAs; 128, one CTA, where there are no more rows
// than that) and up to 256 columns; the width is the one whose waves fit
// (the launcher's rule).  Roles: warp 0 TMA producer, warp 1 MMA issuer and TMEM
// owner, warps 2 and 3 idle (they fill the control warps' group of four, which
// give up registers together), warps 4-11 take the accumulators into registers, half of a row a thread,
// and work on them while the next products go to the other accumulator.  A tile
// of 128 rows of a CTA and 256 columns is 8 H cycles of the tensor cores (H =
// hidden) and 2048 of its exponentials, so H >= 512 hides them.
//
// The tensor cores' fp32 sums are cut, not rounded, after every 16 k, so a long
// sum is a little too near zero: with H = 4096 lse came out 1.2e-6 of itself
// off, 30 times what fp32 arithmetic gives.  The logits' sums are therefore
// taken in parts of K that are added, rounded, in the registers: in the same ones
// forward and backward (the split goes by K and by whether a pair of CTAs has the
// tile, that is by the tokens), so that the gradient's z_tv is the forward's bit for
// bit and a target that is all but certain has exp(z - lse) - 1 of what the other
// words have, where sums in one go, 3e-5 too low at z = 30 and H = 4096, would add
// that to each such token (backward of 4096 x 65536 x 4096 3.27 ms either way).
//
// What it takes: 4096 x 131072 x 2048 forward 1.08 ms by itself (2.03 PFLOP/s,
// above the library's 1.93 in bf16) and 1.19 in a loop that draws the power limit
// (1.85, the library's 1.74); 64 x 32768 x 4096 51 us, 5.3 TB/s of weights (0.79 of
// the copy rate; the rest is a launch's start, the last tile and the joining).
// Sums in one go instead of in parts take the same time.  Measured and slower:
// two accumulators of a tile side by side (1.20 ms against 1.07 at 4096 x 65536 x
// 4096: nothing is left for the next tile), tiles of 160 columns with three (1.30),
// of 128 with four (1.55).
//
// All waits are bounded; on expiry the status word gets TCG_ERR_TIMEOUT, the
// roles drain their copies and MMAs, free the TMEM and return.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "host.h"
#include "ptx.cuh"
#include "split.cuh"
#include "values.cuh"

namespace tcg {
namespace xent {

constexpr float kLog2e = 1.44269504088896341f;
constexpr int kControlWarps = 4, kRowWarps = 8;
constexpr int kThreads = 32 * (kControlWarps + kRowWarps);
// Registers a thread: at the launch, and once they are handed over.
constexpr int kLaunchRegs = 168, kControlRegs = 56, kRowRegs = 224;
static_assert(kControlWarps * kControlRegs + kRowWarps * kRowRegs <= (kControlWarps + kRowWarps) * kLaunchRegs,
              "the shares add up to the launch's registers");
constexpr int kRowBytes = 128;          // one K atom: a 128-byte swizzle row, 64 elements
constexpr int kBM = 128;                // rows of a CTA's tile = TMEM lanes
constexpr int kMaxN = 256;
constexpr int kTmemCols = 512;
constexpr int kAccs = 2, kAccCols = kTmemCols / kAccs;
constexpr int kHalf = kMaxN / 2;        // columns a thread has room for
constexpr int kChunk = 16;

struct Params {
    CUtensorMap tmX, tmW;               // as bytes
    int tokens, cols;                   // rows of X, and of W in this launch
    int num_m, num_n, num_kb;           // tiles; pipeline stages of K
    int parts;                          // accumulations that share a tile's K
    int tile_n, raster_m;
    uint32_t fmt;                       // operand format of the instruction descriptor: 0 fp16, 1 bf16
    const int* target;                  // [tokens]
    int first;                          // the word of W's first row
    // forward
    float2* part;                       // [half column tile][tokens]: (M, s)
    float* picked;                      // [tokens]: z of the target
    // backward
    const float* lse;                   // [tokens]
    const int* valid;                   // n
    const float* grad_mean;             // may be nullptr
    const float* grad_loss;             // [tokens], may be nullptr
    int vocab;                          // targets in [0, vocab) count
    float top;                          // what the largest finite |r_t| becomes in d
    float* back;                        // what undoes that
    void* d;
    long long ldd;                      // a multiple of 32
    int* status;
    long long timeout_ns;
    int fault_inject;
};

constexpr int kCtlBytes = 512;

template <bool kPair>
struct Shape {
    static constexpr int kAtoms = kPair ? 2 : 1;                 // K atoms a stage
    static constexpr int kTileM = kPair ? 2 * kBM : kBM;
    static constexpr int kBRows = kPair ? kMaxN / 2 : kMaxN;     // rows of W a CTA has room for
    static constexpr int kABytes = kAtoms * kBM * kRowBytes;
    static constexpr int kBBytes = kAtoms * kBRows * kRowBytes;
    static constexpr int kStageBytes = kABytes + kBBytes;
    static constexpr int kStages = kPair ? 3 : 4;
    static constexpr int kSmemBytes = kStages * kStageBytes + 1024 + kCtlBytes;   // 1024: alignment
};

struct alignas(16) Ctl {
    uint64_t full[4], empty[4];
    uint64_t tmem_full[kAccs], tmem_empty[kAccs];
    uint64_t drain;
    uint32_t tmem_base;
    int abort_flag;
    float most[kRowWarps];
};
static_assert(sizeof(Ctl) <= kCtlBytes, "the barriers fit");

// (inlined: a call's registers do not fit between the two shares)
__device__ __forceinline__ bool spin(uint64_t* bar, uint32_t parity, int* status, long long limit_ns, Ctl* ctl, int where,
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
                status[3] = 1;   // arrival counters may be left counting
            }
            return false;
        }
    }
}

// The whole warp waits on one barrier and agrees on the outcome.
template <typename P>
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, const P& p, Ctl* ctl, int where, bool honor_abort = true) {
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

// 16 columns of a warp's 32 TMEM lanes; the values are there after landed().
__device__ __forceinline__ void fetch(uint32_t taddr, float (&r)[kChunk]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
          "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void landed(float (&r)[kChunk]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7]), "+f"(r[8]),
                   "+f"(r[9]), "+f"(r[10]), "+f"(r[11]), "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15])
                 :
                 : "memory");
}

// A warp's 32 rows of an accumulator, hw columns from taddr on, into z or added to it.
__device__ __forceinline__ void take_rows(uint32_t taddr, int hw, bool first, float (&z)[kHalf / kChunk][kChunk]) {
    ptx::tc_fence_after_sync();
    if (first) {
#pragma unroll
        for (int c = 0; c < kHalf / kChunk; ++c)
            if (c * kChunk < hw) fetch(taddr + static_cast<uint32_t>(c * kChunk), z[c]);
#pragma unroll
        for (int c = 0; c < kHalf / kChunk; ++c) landed(z[c]);
        return;
    }
#pragma unroll
    for (int c = 0; c < kHalf / kChunk; c += 2) {
        if (c * kChunk >= hw) continue;
        float more[2][kChunk];
        fetch(taddr + static_cast<uint32_t>(c * kChunk), more[0]);
        if ((c + 1) * kChunk < hw) fetch(taddr + static_cast<uint32_t>((c + 1) * kChunk), more[1]);
        landed(more[0]);
        landed(more[1]);
#pragma unroll
        for (int i = 0; i < kChunk; ++i) {
            z[c][i] += more[0][i];
            z[c + 1][i] += more[1][i];
        }
    }
}

// The accumulator goes back as soon as it is in registers.  It hands over columns
// that this warp has read, no memory, so the arrival on the pair leader's barrier
// needs no release at cluster scope: with one, the fence in front of it waited
// for the warp's stores (2000 cycles a tile in the peer CTA).
template <bool kPair>
__device__ __forceinline__ void hand_back(uint64_t* bar, bool leader, int lane) {
    ptx::tc_fence_before_sync();
    __syncwarp();
    if (lane == 0) {
        if (kPair && !leader)
            asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(ptx::map_to_cta(ptx::smem_u32(bar), 0)) : "memory");
        else ptx::mbar_arrive(bar);
    }
}

// The two accumulators in turn, and how often both were walked.
struct Ring {
    int at = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next() {
        phase ^= static_cast<uint32_t>(at);
        at ^= 1;
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

    if (threadIdx.x == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            ptx::mbar_init(&ctl->full[s], 1);
            ptx::mbar_init(&ctl->empty[s], 1);
        }
        for (int a = 0; a < kAccs; ++a) {
            ptx::mbar_init(&ctl->tmem_full[a], 1);
            ptx::mbar_init(&ctl->tmem_empty[a], kPair ? 16 : 8);
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

    if (warp < kControlWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kControlRegs));
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
        } else if (warp == 1 && leader) {
        // ------------------------------------------------------- MMA issuer
            const bool issuer = lane == 0;
            const uint32_t idesc = (1u << 4) | (p.fmt << 7) | (p.fmt << 10) | (static_cast<uint32_t>(p.tile_n >> 3) << 17) |
                                   (static_cast<uint32_t>(S::kTileM >> 4) << 24);
            const long long mine = static_cast<long long>((tiles - worker + workers - 1) / workers) * p.parts;   // accumulations
            int stage = 0;
            uint32_t phase = 0;
            Ring acc;
            Pieces of(p.num_kb, p.parts);
            bool ok = true, issued = false;
            for (long long u = 0; ok && u < mine; ++u) {
                of.next();
                if (!wait(&ctl->tmem_empty[acc.at], acc.phase ^ 1u, p, ctl, 2)) break;
                ptx::tc_fence_after_sync();
                const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc.at * kAccCols);
                for (int kb = of.begin; kb < of.end; ++kb) {
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
                            const uint32_t accum = (kb > of.begin || k > 0) ? 1u : 0u;
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
                    if constexpr (kPair) ptx::mma_commit_pair(&ctl->tmem_full[acc.at], 0x3);
                    else ptx::mma_commit(&ctl->tmem_full[acc.at]);
                }
                __syncwarp();
                acc.next();
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
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRowRegs));
        const int g = warp & 3;                 // the TMEM lanes this warp may read
        const int half = (warp - kControlWarps) >> 2, hw = p.tile_n / 2;   // the columns [half * hw, half * hw + hw) of a tile
        float each = 0.0f, to_top = 1.0f;
        if constexpr (kGrad) {
            // the largest |r_t| that is finite, by every CTA for itself while its first products run
            const int count = *p.valid;
            each = p.grad_mean && count > 0 ? *p.grad_mean / static_cast<float>(count) : 0.0f;
            float most = fabsf(each);
            if (p.grad_loss) {
                most = 0.0f;   // (a token whose weight is not finite leaves the others' scale alone)
                for (int t = static_cast<int>(threadIdx.x) - 32 * kControlWarps; t < p.tokens; t += 32 * kRowWarps) {
                    const int y = p.target[t];
                    const float r = fabsf(each + p.grad_loss[t]);
                    if (y >= 0 && y < p.vocab && r < INFINITY) most = fmaxf(most, r);
                }
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
                if (lane == 0) ctl->most[warp - kControlWarps] = most;
                ptx::named_barrier_sync(1, 32 * kRowWarps);
#pragma unroll
                for (int i = 0; i < kRowWarps; ++i) most = fmaxf(most, ctl->most[i]);
            }
            if (!(most > 0.0f && most < INFINITY)) most = 1.0f;
            to_top = most;
            if (blockIdx.x == 0 && warp == kControlWarps && lane == 0) *p.back = most / p.top;
        }
        Ring acc;
        bool ok = true;
        for (int tile = worker; ok && tile < tiles; tile += workers) {
            int m, n;
            tile_of(p, tile, m, n);
            const int row = m * S::kTileM + static_cast<int>(rank) * kBM + g * 32 + lane;
            const bool live = row < p.tokens;
            const int n0 = n * p.tile_n + half * hw, width = max(0, min(hw, p.cols - n0));
            const int y = live ? p.target[row] : -1;
            // the target's place in these columns, -1 where it is elsewhere
            const long long at_tile = static_cast<long long>(y) - p.first - n0;
            const int at = y >= 0 && at_tile >= 0 && at_tile < width ? static_cast<int>(at_tile) : -1;
            float scale = 0.0f, lse2 = 0.0f;
            if constexpr (kGrad) {
                if (live) {
                    if (y >= 0 && y < p.vocab) scale = (each + (p.grad_loss ? p.grad_loss[row] : 0.0f)) / to_top * p.top;
                    lse2 = p.lse[row] * kLog2e;
                }
            }
            float z[kHalf / kChunk][kChunk];
            for (int part = 0; part < p.parts; ++part) {
                ok = wait(&ctl->tmem_full[acc.at], acc.phase, p, ctl, 4);
                if (!ok) break;
                take_rows(tmem_base + (static_cast<uint32_t>(g * 32) << 16) + static_cast<uint32_t>(acc.at * kAccCols + half * hw), hw, part == 0, z);
                hand_back<kPair>(&ctl->tmem_empty[acc.at], leader, lane);
                acc.next();
            }
            if (!ok) break;
            const bool any = __any_sync(0xffffffffu, at >= 0);
            if constexpr (kGrad) {
                T* dst = static_cast<T*>(p.d) + row * p.ldd + n0;
#pragma unroll
                for (int c = 0; c < kHalf / kChunk; ++c) {
                    if (c * kChunk >= width) continue;
#pragma unroll
                    for (int i = 0; i < kChunk; ++i) z[c][i] = ptx::ex2_approx_ftz(fmaf(z[c][i], kLog2e, -lse2));
                    if (any) {
#pragma unroll
                        for (int i = 0; i < kChunk; ++i) z[c][i] -= c * kChunk + i == at ? 1.0f : 0.0f;
                    }
                    uint32_t w[8];
                    // (a token that does not count has gradient 0, whatever its logits are)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        w[i] = scale == 0.0f ? 0u : pack_pair<T>(scale * z[c][2 * i], scale * z[c][2 * i + 1]);
                    if (live) ptx::st_global_v8(dst + c * kChunk, w);
                }
            } else {
                if (width < hw) {
#pragma unroll
                    for (int c = 0; c < kHalf / kChunk; ++c)
#pragma unroll
                        for (int i = 0; i < kChunk; ++i) z[c][i] = c * kChunk + i < width ? z[c][i] : -INFINITY;
                }
                if (any) {
                    float picked = 0.0f;
#pragma unroll
                    for (int c = 0; c < kHalf / kChunk; ++c)
#pragma unroll
                        for (int i = 0; i < kChunk; ++i) picked = c * kChunk + i == at ? z[c][i] : picked;
                    if (at >= 0) p.picked[row] = picked;
                }
                float most[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY}, sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int c = 0; c < kHalf / kChunk; ++c) {
                    if (c * kChunk >= hw) continue;
#pragma unroll
                    for (int i = 0; i < kChunk; i += 2) most[i / 2 & 3] = fmaxf(most[i / 2 & 3], fmaxf(z[c][i], z[c][i + 1]));
                }
                const float m2 = fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3])) * kLog2e;
                const float base = m2 == -INFINITY ? 0.0f : m2;   // (nothing but -inf, or no column: s = 0)
#pragma unroll
                for (int c = 0; c < kHalf / kChunk; ++c) {
                    if (c * kChunk >= hw) continue;
#pragma unroll
                    for (int i = 0; i < kChunk; ++i) sum[i & 3] += ptx::ex2_approx_ftz(fmaf(z[c][i], kLog2e, -base));
                }
                if (live) p.part[static_cast<size_t>(2 * n + half) * p.tokens + row] = make_float2(m2, (sum[0] + sum[1]) + (sum[2] + sum[3]));
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
