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
// added up in registers in pieces of that length.  (Of 1024 k, as the logits' are,
// dX of 64 x 32768 x 4096 is 7e-6 of itself less near zero, where dz's rounding is
// 6.7e-4 in the 2-norm, and backward takes 1 % longer at 4096 x 65536 x 4096 and
// 2 % at 8192 x 100000 x 512.)
//
// Bound by the tensor cores where the sums are long (1000 x 50021 x 1280: both
// products 151 us, tensor pipe 79 %; as two calls of tcg_gemm 245), by the way of
// dW's tiles to memory where there are few tokens (64 x 32768 x 4096: a tile of 64
// KB a CTA in 2.1 us, of which the stores 1.5: 32 rows of 32 bytes at a time).
// What helped there: an accumulator's hand-back without a release at cluster scope
// (265 -> 195 us for all of the backward pass), one output type's code at a time
// (fewer instructions fetched), stores straight from registers (186; 177 as it stands).
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
    int vec;                  // bytes that rows of out start on: 32, 16, or fewer (0)
    float beta;
    const float* sum;         // fp32 sums of the pieces before, or nullptr
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
constexpr int kTurnPad = kChunk + 1;
constexpr int kTurnFloats = 32 * kTurnPad;         // a row warp's
constexpr int kProductSmem = Shape<true>::kSmemBytes + kRowWarps * kTurnFloats * static_cast<int>(sizeof(float));
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

// A field of the unit's product, both products' read at places known to the
// compiler (an index into the parameters would make each a load with a latency).
#define TCG_OF(p, v, field) ((v).which == 0 ? (p).q[0].field : (p).q[1].field)

// Stages [kb0, kb1) of a unit, and where its tile starts in units of tiles.
struct Span {
    int kb0, kb1, m, n;
};
__device__ __forceinline__ Span span_of(const Products& p, const Unit& v) {
    const int num_kb = TCG_OF(p, v, num_kb), splits = TCG_OF(p, v, splits), num_n = TCG_OF(p, v, num_n);
    Span s;
    s.kb0 = splits == 1 ? 0 : run_start(num_kb, v.split, splits);
    s.kb1 = splits == 1 ? num_kb : run_start(num_kb, v.split + 1, splits);
    s.m = v.tile / num_n;
    s.n = v.tile - s.m * num_n;
    return s;
}

// Where a warp's rows go: row0 + lane, columns [n0, n0 + width).
struct Target {
    int row0, rows, n0, width, N;   // rows: M - row0
    long long ldo, ld_sum;
    float beta, back;
    const float* sum;
    int vec;                        // bytes that rows of out start on: 32, 16, or fewer (0)
};

// The whole chunks of 16 columns as type O, times back: a lane its row, in words
// of 32 or 16 bytes.  kMore: plus what was there and the sums of the pieces
// before.  (Through shared memory and TMA, a box of 128 bytes a row at a time, it
// took longer: each box waits for the one before to be read, 1400 cycles.  dW of
// 64 x 32768 x 4096: 145 us with dz, 133 this way.)
template <typename O, bool kMore>
__device__ __forceinline__ void store_rows(const Target& o, O* out, int lane, float (&z)[kHalf / kChunk][kChunk]) {
    constexpr int kWords = kChunk * static_cast<int>(sizeof(O)) / 4;
    if (lane >= o.rows) return;
    O* row = out + (o.row0 + lane) * o.ldo + o.n0;
    const float* sum = kMore && o.sum ? o.sum + (o.row0 + lane) * o.ld_sum + o.n0 : nullptr;
#pragma unroll
    for (int c = 0; c < kHalf / kChunk; ++c) {
        if ((c + 1) * kChunk > o.width) continue;
        float x[kChunk];
#pragma unroll
        for (int i = 0; i < kChunk; ++i) x[i] = z[c][i] * o.back;
        if constexpr (kMore) {
            if (sum) {
#pragma unroll
                for (int i = 0; i < kChunk; i += 4) {
                    const float4 f = *reinterpret_cast<const float4*>(sum + c * kChunk + i);
                    x[i] += f.x, x[i + 1] += f.y, x[i + 2] += f.z, x[i + 3] += f.w;
                }
            }
            if (o.beta != 0.0f) {
#pragma unroll
                for (int i = 0; i < kChunk; i += 8) {
                    float f[8];
                    values_of<O>(load_raw8(row + c * kChunk + i), f);
#pragma unroll
                    for (int k = 0; k < 8; ++k) x[i + k] = fmaf(o.beta, f[k], x[i + k]);
                }
            }
        }
        uint32_t w[kWords];
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            if constexpr (sizeof(O) == 4) w[i] = __float_as_uint(x[i]);
            else w[i] = pack_pair<O>(x[2 * i], x[2 * i + 1]);
        }
        uint8_t* dst = reinterpret_cast<uint8_t*>(row + c * kChunk);
        if (o.vec == 32) {
#pragma unroll
            for (int h = 0; h < kWords; h += 8) {
                const uint32_t q[8] = {w[h], w[h + 1], w[h + 2], w[h + 3], w[h + 4], w[h + 5], w[h + 6], w[h + 7]};
                ptx::st_global_v8(dst + 4 * h, q);
            }
        } else {
#pragma unroll
            for (int h = 0; h < kWords; h += 4) *reinterpret_cast<uint4*>(dst + 4 * h) = make_uint4(w[h], w[h + 1], w[h + 2], w[h + 3]);
        }
    }
}

// Chunks from `first` on to rows that start anywhere, or that end inside one:
// turned in shared memory, so that 16 lanes have a row's 16 columns.  (One copy of
// the code: z moves up instead.)
template <typename O>
__device__ __forceinline__ void turn_rows(const Target& o, O* out, float* turn, int lane, int first, float (&z)[kHalf / kChunk][kChunk]) {
#pragma unroll 1
    for (int c = 0; c * kChunk < o.width; ++c) {
        if (c >= first) {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < kChunk; ++i) turn[lane * kTurnPad + i] = z[0][i] * o.back;
            __syncwarp();
            const int col = o.n0 + c * kChunk + (lane & 15), r0 = lane >> 4;
            if (col < o.N) {
                O* dst = out + (o.row0 + r0) * o.ldo + col;
                const float* sum = o.sum ? o.sum + (o.row0 + r0) * o.ld_sum + col : nullptr;
#pragma unroll 4
                for (int r = r0; r < 32; r += 2) {
                    if (r >= o.rows) break;
                    float y = turn[r * kTurnPad + (lane & 15)];
                    const long long step = r - r0;
                    if (sum) y += sum[step * o.ld_sum];
                    if (o.beta != 0.0f) y = fmaf(o.beta, to_float(dst[step * o.ldo]), y);
                    dst[step * o.ldo] = from_float<O>(y);
                }
            }
        }
#pragma unroll
        for (int k = 0; k + 1 < kHalf / kChunk; ++k)
#pragma unroll
            for (int i = 0; i < kChunk; ++i) z[k][i] = z[k + 1][i];
    }
}

template <typename O>
__device__ __forceinline__ void write_rows(const Target& o, void* out, float* turn, int lane, float (&z)[kHalf / kChunk][kChunk]) {
    int first = 0;
    if (o.vec >= 16) {
        if (o.sum || o.beta != 0.0f) store_rows<O, true>(o, static_cast<O*>(out), lane, z);
        else store_rows<O, false>(o, static_cast<O*>(out), lane, z);
        first = o.width / kChunk;
        if (first * kChunk == o.width) return;
    }
    turn_rows<O>(o, static_cast<O*>(out), turn, lane, first, z);
}

__global__ void __launch_bounds__(kThreads, 1) xent_product_kernel(const __grid_constant__ Products p) {
    using S = Shape<true>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Ctl* ctl = reinterpret_cast<Ctl*>(smem + S::kStages * S::kStageBytes);
    float* turn = reinterpret_cast<float*>(smem + S::kStages * S::kStageBytes + kCtlBytes);
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
            const Span at = span_of(p, v);
            const bool along_m = TCG_OF(p, v, a_along_m) != 0;
            const CUtensorMap *ma = v.which == 0 ? &p.q[0].a : &p.q[1].a, *mb = v.which == 0 ? &p.q[0].b : &p.q[1].b;
            const int m0 = at.m * S::kTileM + static_cast<int>(rank) * kBM, n0 = at.n * p.tile_n + static_cast<int>(rank) * b_cols;
            for (int kb = at.kb0; kb < at.kb1; ++kb) {
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
                        const int along = along_m ? m0 + 64 * i : k0 + 64 * i;
                        ptx::tma_load_2d_pair(sA + i * kStageK * kRowBytes, ma, fbc, 2 * along, along_m ? k0 : m0);
                        if (64 * i < b_cols) ptx::tma_load_2d_pair(sB + i * kStageK * kRowBytes, mb, fbc, 2 * (n0 + 64 * i), k0);
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
                const Span of = span_of(p, v);
                const uint32_t along_m = static_cast<uint32_t>(TCG_OF(p, v, a_along_m));
                // bits 15 and 16: M and N contiguous in shared memory
                const uint32_t idesc = (1u << 4) | (p.fmt << 7) | (p.fmt << 10) | (along_m << 15) | (1u << 16) |
                                       (static_cast<uint32_t>(p.tile_n >> 3) << 17) | (static_cast<uint32_t>(S::kTileM >> 4) << 24);
                for (int kb0 = of.kb0; ok && kb0 < of.kb1; kb0 += kPartStages) {
                    if (!wait(&ctl->tmem_empty[acc.at], acc.phase ^ 1u, p, ctl, 22)) { ok = false; break; }
                    ptx::tc_fence_after_sync();
                    const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc.at * kAccCols);
                    const int end = min(of.kb1, kb0 + kPartStages);
                    for (int kb = kb0; kb < end; ++kb) {
                        if (!wait(&ctl->full[stage], phase, p, ctl, 23)) { ok = false; break; }
                        ptx::tc_fence_after_sync();
                        if (issuer) {
                            const uint32_t sA = ptx::smem_u32(smem + stage * S::kStageBytes);
                            // K contiguous: 8-row groups 1024 bytes apart, 16 k are 32 bytes on; else runs of 64
                            // elements 16 KiB apart, 8-row groups of K 1024 bytes apart, 16 k are 2 KiB on
                            const uint64_t a_desc = ptx::smem_desc_sw128(sA, along_m ? kStageK * kRowBytes : 16, 1024);
                            const uint64_t b_desc = ptx::smem_desc_sw128(sA + S::kABytes, kStageK * kRowBytes, 1024);
#pragma unroll
                            for (int k = 0; k < kStageK / 16; ++k) {
                                const uint32_t a_off = along_m ? k * 16 * kRowBytes : (k / 4) * kBM * kRowBytes + (k % 4) * 32;
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
        turn += rw * kTurnFloats;
        const float back = p.back ? *p.back : 1.0f;
        Ring acc;
        bool ok = true;
        while (ok && walk.next(p, v)) {
            const Span of = span_of(p, v);
            const int kb0 = of.kb0, kb1 = of.kb1, row0 = of.m * S::kTileM + static_cast<int>(rank) * kBM + g * 32;
            const int n0 = of.n * p.tile_n + half * hw, N = TCG_OF(p, v, N), width = max(0, min(hw, N - n0));
            const int splits = TCG_OF(p, v, splits);
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
            const int M = TCG_OF(p, v, M), type = TCG_OF(p, v, type);
            if (row0 >= M) continue;
            if (splits > 1) {
                // this warp's place among the unit's partial sums
                const int mine = static_cast<int>(rank) * kRowWarps + rw;
                auto place = [&](int split) {
                    const size_t unit = static_cast<size_t>(split) * (p.q[0].num_m * p.q[0].num_n) + v.tile;   // (only dX's are split)
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
                if (before != splits - 1) continue;
                __threadfence();
                if (lane == 0) *counter = 0;
                for (int s = 0; s < splits; ++s) {
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
            const Target o = {row0, M - row0, n0, width, N, TCG_OF(p, v, ldo), TCG_OF(p, v, ld_sum), TCG_OF(p, v, beta), back,
                              TCG_OF(p, v, sum), TCG_OF(p, v, vec)};
            void* out = TCG_OF(p, v, out);
            if (type == kOutF32) write_rows<float>(o, out, turn, lane, z);
            else if (type == kOutF16) write_rows<__half>(o, out, turn, lane, z);
            else write_rows<__nv_bfloat16>(o, out, turn, lane, z);
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

#undef TCG_OF

}  // namespace xent
}  // namespace tcg
