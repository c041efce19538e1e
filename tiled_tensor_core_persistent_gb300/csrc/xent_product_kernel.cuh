// xent_product_kernel.cuh -- the two products that take the loss's gradient with
// respect to its logits, dz (tokens x words, 16 bits), to those of X and W, in
// one launch:
//
//   dX = b dz W      (tokens x hidden, K = words:  few tiles, long sums)
//   dW = b dz^T X    (words x hidden,  K = tokens: many tiles, short sums)
//
// b, one number, undoes the scale of dz.  dz, W and X are read as they lie: as
// the rows operand with K contiguous (dz for dX) or with M contiguous (dz for
// dW), as the columns operand with N contiguous (W and X); no copy is turned.
//
// One launch, because the two fill the SMs together where neither does alone:
// dX's tiles (their K in `splits` pieces where there are few) go round the
// workers first, and those that have one less begin dW's tiles meanwhile.  A
// split tile's pieces go to the workspace, each warp's 32 rows by themselves,
// and the warp that arrives last adds them in the order of their place, so the
// result does not depend on which that is.
//
// Roles, registers, accumulators and bounded waits as in xent_kernel.cuh: pairs
// of CTAs on tiles of 256 rows, 256 or 128 columns.  Sums longer than 8192 k are
// added up in registers in pieces of that length.
#pragma once

#include "xent_kernel.cuh"

namespace tcg {
namespace xent {

enum : int { kOutBf16 = 0, kOutF16 = 1, kOutF32 = 2 };

// out = b A B^T + beta out + sum; A is M x K, B (as it lies) K x N.
struct Product {
    CUtensorMap a, b;
    int a_along_m;            // A's M is contiguous (else its K)
    int M, N, num_kb;         // num_kb: pipeline stages of K
    int num_m, num_n, splits;
    void* out;
    long long ldo;
    int type;
    int vec;                  // rows of out start on 32 bytes
    float beta;
    const float* sum;         // fp32 sums of the pieces before, or nullptr (rows start on 32 bytes)
    long long ld_sum;
};

struct Products {
    Product q[2];             // dX, dW; no tiles where one is not wanted
    int tile_n;
    uint32_t fmt;
    int early;                // tiles of the second that a worker takes while others have a unit of the first more
    const float* back;        // b
    float* partials;          // [unit of the first][rank][warp][column][lane]
    int* counters;            // [tile of the first][rank][warp]
    int* status;
    long long timeout_ns;
    int fault_inject;
};

constexpr int kStageK = 128;                       // k a stage: two atoms of 64
constexpr int kPartStages = 64;                    // 8192 k
constexpr int kStagePad = kChunk + 1;
constexpr int kTurnBytes = kRowWarps * 32 * kStagePad * static_cast<int>(sizeof(float));
constexpr int kProductSmem = Shape<true>::kStages * Shape<true>::kStageBytes + 1024 + 512 + kTurnBytes;
constexpr int kPartialFloats = 2 * kRowWarps * kHalf * 32;   // a unit's

struct Unit {
    int which, tile, split, u;
};

// A worker's units, in order.
struct Walk {
    int w, workers, first_units, rest, second_tiles, early;
    int j = 0, stage = 0;

    __device__ __forceinline__ Walk(const Products& p, int worker, int count) : w(worker), workers(count) {
        first_units = p.q[0].num_m * p.q[0].num_n * p.q[0].splits;
        second_tiles = p.q[1].num_m * p.q[1].num_n;
        rest = first_units % workers;
        early = rest > 0 ? p.early : 0;
    }
    __device__ __forceinline__ bool next(const Products& p, Unit& v) {
        if (stage == 0) {
            const int u = w + j * workers;
            if (u < first_units) {
                const int tiles = p.q[0].num_m * p.q[0].num_n;
                v = {0, u % tiles, u / tiles, u};   // the pieces of one part of K at a time: they share its operands
                ++j;
                return true;
            }
            stage = 1;
            j = 0;
        }
        if (stage == 1) {
            const int t = j * (workers - rest) + w - rest;
            if (w >= rest && j < early && t < second_tiles) {
                v = {1, t, 0, 0};
                ++j;
                return true;
            }
            stage = 2;
            j = 0;
        }
        const int t = early * (workers - rest) + j * workers + w;
        if (t >= second_tiles) return false;
        v = {1, t, 0, 0};
        ++j;
        return true;
    }
};

__device__ __forceinline__ int first_stage(const Product& q, int split) {
    return static_cast<int>(static_cast<long long>(q.num_kb) * split / q.splits);
}

template <typename T>
__device__ __forceinline__ float old_value(const void* out, long long at) { return to_float(static_cast<const T*>(out)[at]); }

// 16 neighbouring values of a row that starts on 32 bytes.
__device__ __forceinline__ void add_old(const Product& q, long long at, float (&v)[kChunk]) {
    if (q.type == kOutF32) {
#pragma unroll
        for (int i = 0; i < kChunk; i += 4) {
            const float4 o = *reinterpret_cast<const float4*>(static_cast<const float*>(q.out) + at + i);
            v[i] = fmaf(q.beta, o.x, v[i]), v[i + 1] = fmaf(q.beta, o.y, v[i + 1]);
            v[i + 2] = fmaf(q.beta, o.z, v[i + 2]), v[i + 3] = fmaf(q.beta, o.w, v[i + 3]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kChunk; i += 8) {
            float o[8];
            if (q.type == kOutF16) values_of<__half>(load_raw8(static_cast<const __half*>(q.out) + at + i), o);
            else values_of<__nv_bfloat16>(load_raw8(static_cast<const __nv_bfloat16*>(q.out) + at + i), o);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[i + k] = fmaf(q.beta, o[k], v[i + k]);
        }
    }
}
__device__ __forceinline__ void store16(const Product& q, long long at, const float (&v)[kChunk]) {
    uint32_t w[8];
    if (q.type == kOutF32) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(v[8 * h + i]);
            ptx::st_global_v8(static_cast<float*>(q.out) + at + 8 * h, w);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w[i] = q.type == kOutF16 ? pack_pair<__half>(v[2 * i], v[2 * i + 1]) : pack_pair<__nv_bfloat16>(v[2 * i], v[2 * i + 1]);
        ptx::st_global_v8(static_cast<uint16_t*>(q.out) + at, w);
    }
}
__device__ __forceinline__ void store1(const Product& q, long long at, float v) {
    if (q.type == kOutF32) static_cast<float*>(q.out)[at] = v;
    else if (q.type == kOutF16) static_cast<__half*>(q.out)[at] = __float2half_rn(v);
    else static_cast<__nv_bfloat16*>(q.out)[at] = __float2bfloat16_rn(v);
}
__device__ __forceinline__ float load1(const Product& q, long long at) {
    return q.type == kOutF32 ? old_value<float>(q.out, at) : q.type == kOutF16 ? old_value<__half>(q.out, at) : old_value<__nv_bfloat16>(q.out, at);
}

__global__ void __launch_bounds__(kThreads, 1) xent_product_kernel(const __grid_constant__ Products p) {
    using S = Shape<true>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Ctl* ctl = reinterpret_cast<Ctl*>(smem + S::kStages * S::kStageBytes);
    float* turn = reinterpret_cast<float*>(smem + S::kStages * S::kStageBytes + 512);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = ptx::cluster_ctarank();
    const bool leader = rank == 0;
    const int worker = static_cast<int>(blockIdx.x >> 1), workers = static_cast<int>(gridDim.x >> 1);

    if (threadIdx.x == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            ptx::mbar_init(&ctl->full[s], 1);
            ptx::mbar_init(&ctl->empty[s], 1);
        }
        for (int a = 0; a < kAccs; ++a) {
            ptx::mbar_init(&ctl->tmem_full[a], 1);
            ptx::mbar_init(&ctl->tmem_empty[a], 2 * kRowWarps);
        }
        ptx::mbar_init(&ctl->drain, 1);
        ctl->abort_flag = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 1) {
        ptx::tmem_alloc_pair(&ctl->tmem_base, kTmemCols);
        ptx::tmem_relinquish_alloc_permit_pair();
    }
    ptx::tc_fence_before_sync();
    ptx::cluster_sync();   // the peer's barriers exist before anyone signals them
    ptx::tc_fence_after_sync();
    const uint32_t tmem_base = ctl->tmem_base;
    tcg::host::wait_for_kernel_ahead();

    Walk walk(p, worker, workers);
    Unit v;
    if (warp < kControlWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kControlRegs));
        if (warp == 0) {
        // ------------------------------------------------------ TMA producer
        const bool issuer = lane == 0;
        const int b_cols = p.tile_n / 2;           // columns this CTA loads: one or two runs of 64
        const uint32_t tx = 2u * static_cast<uint32_t>(S::kABytes + b_cols * 2 * kStageK);
        int stage = 0;
        uint32_t phase = 0, armed = 0, armed_parity = 0;
        bool ok = true, first = true;
        while (ok && walk.next(p, v)) {
            const Product& q = p.q[v.which];
            const int m0 = v.tile / q.num_n * S::kTileM + static_cast<int>(rank) * kBM;
            const int n0 = v.tile % q.num_n * p.tile_n + static_cast<int>(rank) * b_cols;
            const int kb1 = first_stage(q, v.split + 1);
            for (int kb = first_stage(q, v.split); kb < kb1; ++kb) {
                if (!wait(&ctl->empty[stage], phase ^ 1u, p, ctl, 21)) { ok = false; break; }
                const bool skip = first && p.fault_inject == 1 && blockIdx.x == 0;
                first = false;
                if (!skip && issuer) {
                    uint8_t* sA = smem + stage * S::kStageBytes;
                    uint8_t* sB = sA + S::kABytes;
                    uint64_t* fb = &ctl->full[stage];
                    if (leader) ptx::mbar_arrive_expect_tx(fb, tx);
                    const uint32_t fbc = ptx::map_to_cta(ptx::smem_u32(fb), 0);
                    const int k0 = kb * kStageK;
                    // boxes of 64 elements (128 bytes; x counts bytes) by 128 rows
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int along = q.a_along_m ? m0 + 64 * i : k0 + 64 * i;
                        ptx::tma_load_2d_pair(sA + i * kStageK * kRowBytes, &q.a, fbc, 2 * along, q.a_along_m ? k0 : m0);
                        if (64 * i < b_cols) ptx::tma_load_2d_pair(sB + i * kStageK * kRowBytes, &q.b, fbc, 2 * (n0 + 64 * i), k0);
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
        for (int s = 0; s < S::kStages; ++s) {
            if (!(armed & (1u << s))) continue;
            const uint32_t par = (armed_parity >> s) & 1u;
            if (leader) wait(&ctl->full[s], par, p, ctl, 31, false);
            else wait(&ctl->empty[s], par, p, ctl, 33, false);
        }
        } else if (warp == 1 && leader) {
        // ------------------------------------------------------- MMA issuer
            const bool issuer = lane == 0;
            int stage = 0;
            uint32_t phase = 0;
            Ring acc;
            bool ok = true, issued = false;
            while (ok && walk.next(p, v)) {
                const Product& q = p.q[v.which];
                // bits 15 and 16: M and N contiguous in shared memory
                const uint32_t idesc = (1u << 4) | (p.fmt << 7) | (p.fmt << 10) | (static_cast<uint32_t>(q.a_along_m) << 15) | (1u << 16) |
                                       (static_cast<uint32_t>(p.tile_n >> 3) << 17) | (static_cast<uint32_t>(S::kTileM >> 4) << 24);
                const int kb1 = first_stage(q, v.split + 1);
                for (int kb0 = first_stage(q, v.split); ok && kb0 < kb1; kb0 += kPartStages) {
                    if (!wait(&ctl->tmem_empty[acc.at], acc.phase ^ 1u, p, ctl, 22)) { ok = false; break; }
                    ptx::tc_fence_after_sync();
                    const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc.at * kAccCols);
                    const int end = min(kb1, kb0 + kPartStages);
                    for (int kb = kb0; kb < end; ++kb) {
                        if (!wait(&ctl->full[stage], phase, p, ctl, 23)) { ok = false; break; }
                        ptx::tc_fence_after_sync();
                        if (issuer) {
                            const uint32_t sA = ptx::smem_u32(smem + stage * S::kStageBytes);
                            // K contiguous: 8-row groups 1024 bytes apart, 16 k are 32 bytes on; else runs of 64
                            // elements 16 KiB apart, 8-row groups of K 1024 bytes apart, 16 k are 2 KiB on
                            const uint64_t a_desc = ptx::smem_desc_sw128(sA, q.a_along_m ? kStageK * kRowBytes : 16, 1024);
                            const uint64_t b_desc = ptx::smem_desc_sw128(sA + S::kABytes, kStageK * kRowBytes, 1024);
#pragma unroll
                            for (int k = 0; k < kStageK / 16; ++k) {
                                const uint32_t a_off = q.a_along_m ? k * 16 * kRowBytes : (k / 4) * kBM * kRowBytes + (k % 4) * 32;
                                ptx::mma_f16_pair(d_tmem, a_desc + (a_off >> 4), b_desc + static_cast<uint32_t>((k * 16 * kRowBytes) >> 4), idesc,
                                                  (kb > kb0 || k > 0) ? 1u : 0u);
                            }
                            ptx::mma_commit_pair(&ctl->empty[stage], 0x3);
                        }
                        __syncwarp();
                        issued = true;
                        if (++stage == S::kStages) { stage = 0; phase ^= 1u; }
                    }
                    if (ok && issuer) ptx::mma_commit_pair(&ctl->tmem_full[acc.at], 0x3);
                    __syncwarp();
                    acc.next();
                }
            }
            if (issued) {
                if (issuer) ptx::mma_commit_pair(&ctl->drain, 0x1);
                __syncwarp();
                wait(&ctl->drain, 0, p, ctl, 32, false);
            }
        }
    } else {
        // ------------------------------------------------------ rows to memory
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRowRegs));
        const int g = warp & 3, rw = warp - kControlWarps, half = rw >> 2, hw = p.tile_n / 2;
        turn += rw * 32 * kStagePad;
        const float back = *p.back;
        Ring acc;
        bool ok = true;
        while (ok && walk.next(p, v)) {
            const Product& q = p.q[v.which];
            const int row0 = v.tile / q.num_n * S::kTileM + static_cast<int>(rank) * kBM + g * 32, row = row0 + lane;
            const int n0 = v.tile % q.num_n * p.tile_n + half * hw, width = max(0, min(hw, q.N - n0));
            const int kb0 = first_stage(q, v.split), kb1 = first_stage(q, v.split + 1);
            float z[kHalf / kChunk][kChunk];
            if (kb0 == kb1) {   // a sum over no tokens
#pragma unroll
                for (int c = 0; c < kHalf / kChunk; ++c)
#pragma unroll
                    for (int i = 0; i < kChunk; ++i) z[c][i] = 0.0f;
            }
            for (int kb = kb0; kb < kb1; kb += kPartStages) {
                ok = wait(&ctl->tmem_full[acc.at], acc.phase, p, ctl, 24);
                if (!ok) break;
                take_rows(tmem_base + (static_cast<uint32_t>(g * 32) << 16) + static_cast<uint32_t>(acc.at * kAccCols + half * hw), hw, kb == kb0, z);
                hand_back<true>(&ctl->tmem_empty[acc.at], leader, lane);
                acc.next();
            }
            if (!ok) break;
            if (q.splits > 1) {
                // this warp's place among the unit's partial sums
                const int mine = static_cast<int>(rank) * kRowWarps + rw;
                auto place = [&](int split) {
                    const size_t unit = static_cast<size_t>(split) * (q.num_m * q.num_n) + v.tile;
                    return p.partials + unit * kPartialFloats + static_cast<size_t>(mine) * (kHalf * 32) + lane;
                };
                float* dst = place(v.split);
#pragma unroll
                for (int c = 0; c < kHalf / kChunk; ++c) {
                    if (c * kChunk >= hw) continue;
#pragma unroll
                    for (int i = 0; i < kChunk; ++i) __stcg(dst + (c * kChunk + i) * 32, z[c][i]);
                }
                __threadfence();
                __syncwarp();
                int* counter = p.counters + v.tile * 2 * kRowWarps + mine;
                int before = 0;
                if (lane == 0) before = ptx::atomic_add_acq_rel_gpu(counter, 1);
                before = __shfl_sync(0xffffffffu, before, 0);
                if (before != q.splits - 1) continue;
                __threadfence();
                if (lane == 0) *counter = 0;
                for (int s = 0; s < q.splits; ++s) {
                    const float* src = place(s);
#pragma unroll
                    for (int c = 0; c < kHalf / kChunk; ++c) {
                        if (c * kChunk >= hw) continue;
#pragma unroll
                        for (int i = 0; i < kChunk; ++i) {
                            const float more = __ldcg(src + (c * kChunk + i) * 32);
                            z[c][i] = s == 0 ? more : z[c][i] + more;
                        }
                    }
                }
            }
            if (row0 >= q.M) continue;
#pragma unroll
            for (int c = 0; c < kHalf / kChunk; ++c) {
                if (c * kChunk >= width) continue;
                float (&x)[kChunk] = z[c];
#pragma unroll
                for (int i = 0; i < kChunk; ++i) x[i] *= back;
                const int col = n0 + c * kChunk;
                if (q.vec && col + kChunk <= q.N) {
                    if (row < q.M) {
                        if (q.sum) {
#pragma unroll
                            for (int i = 0; i < kChunk; i += 4) {
                                const float4 o = *reinterpret_cast<const float4*>(q.sum + row * q.ld_sum + col + i);
                                x[i] += o.x, x[i + 1] += o.y, x[i + 2] += o.z, x[i + 3] += o.w;
                            }
                        }
                        const long long at = row * q.ldo + col;
                        if (q.beta != 0.0f) add_old(q, at, x);
                        store16(q, at, x);
                    }
                } else {
                    // turned in shared memory: 16 lanes have a row's 16 columns
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < kChunk; ++i) turn[lane * kStagePad + i] = x[i];
                    __syncwarp();
                    const int own = col + (lane & 15);
                    for (int r = lane >> 4; r < 32; r += 2) {
                        if (row0 + r >= q.M || own >= q.N) continue;
                        float y = turn[r * kStagePad + (lane & 15)];
                        const long long at = (row0 + r) * q.ldo + own;
                        if (q.sum) y += q.sum[(row0 + r) * q.ld_sum + own];
                        if (q.beta != 0.0f) y = fmaf(q.beta, load1(q, at), y);
                        store1(q, at, y);
                    }
                }
            }
        }
    }

    ptx::tc_fence_before_sync();
    ptx::cluster_sync();   // the leader's MMAs into the peer's TMEM are done
    if (warp == 1) {
        __syncwarp();
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc_pair(tmem_base, kTmemCols);
    }
}

}  // namespace xent
}  // namespace tcg
