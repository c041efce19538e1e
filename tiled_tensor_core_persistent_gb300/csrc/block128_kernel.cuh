// block128_kernel.cuh -- the 8-bit matrix product whose operands carry one
// fp32 scale per 128 consecutive K (per row of A; per row or per 128 rows of
// B), for sm_103a:
//
//   D[m, n] = act( sum_kb sA[m, kb] sB[n, kb] T_kb[m, n] + beta C[m, n] + bias[n] )
//   T_kb[m, n] = sum over the 128 k of block kb of A[m, k] B[n, k]
//
// T_kb is what the tensor cores sum exactly as fp32 in TMEM; the scales are
// arbitrary fp32 numbers, which the MMA's own block scaling (powers of two or
// 8-bit scales per 16 or 32) cannot hold.  So every k-block is one fresh TMEM
// accumulation of four K = 32 MMAs, and the promote warps fold it into fp32
// registers: acc += (sA sB) * T_kb.
//
// What bounds it.  A k-block of a 256 x 256 pair tile keeps each SM's tensor
// core busy for 128 * 256 * 128 / 8192 = 512 cycles; its fold is 128 x 256 words
// from TMEM (256 cycles at 16 bytes per lane and clock) and as many FMAs (256
// issue cycles of each scheduler, next to the waits and the hand-overs).  Two
// accumulators of 256 columns fill the TMEM, so the chain MMAs -> commit ->
// fold -> hand-back closes over two k-blocks, and one takes about 950 cycles:
// 8192^3 in 506-526 us, 2.09-2.17 PFLOP/s, 1.1 times the bf16 rate of the
// library on this GPU.  Measured at 8192^3 and slower: FMAs of two sums an
// instruction (the pairs cost a move each), 128-column accumulators with an
// issuer each or one issuer for both (513-565 us beside 498-520), the next
// k-block's first chunk read ahead of the fold's end (574-589), 256 x 192
// tiles under twelve promote warps (613-640), 128 x 256 tiles on one CTA (557).
// A per-column scale (both operands scaled per row, the weight gradients) adds
// one multiply per element, and fp32 C and D their traffic: 4096 x 4096 over
// 16384 rows of K in 16 groups, 870-892 us, 2.6 TB/s.  Few rows are bound by B's
// bytes and a launch's start and end (1 x 8192 x 8192: 19.6 us, 3.4 TB/s; 32
// rows over 16 experts of 4096 x 4096: 45.7 us, 5.1 TB/s).
//
// Roles (one CTA or a CTA pair, persistent): warp 0 TMA producer, warp 1 MMA
// issuer and TMEM owner, warp 2 copies the scales ahead, warp 3 idle (it fills
// the control warps' group of four, which give up registers together), the
// others promote and store.  All waits are
// bounded; on expiry the status word gets TCG_ERR_TIMEOUT, the roles drain
// their copies and MMAs, free the TMEM and return.
#pragma once

#include "gemm_kernel.cuh"
#include "groups.cuh"
#include "host.h"

namespace tcg {
namespace b128 {

constexpr int kBlock = 128;                 // K elements per scale = bytes per swizzle row
constexpr int kMaxGroups = 1024;
constexpr int kScaleSlots = 8;              // k-blocks of scales in flight
constexpr int kMaxPromoteWarps = 8;

enum Mode : int { kDense = 0, kGroupedRows = 1, kGroupedK = 2 };

// How the scales of one operand are addressed: row r, k-block kb, group g at
// ptr[(r >> shift) * rs + kb * ks + g * gs].
struct ScaleRef {
    const float* ptr;
    long long rs, ks, gs;
    int shift;   // 0: one scale per row, 7: one per 128 rows
};

struct Params {
    CUtensorMap tmA, tmB;
    ScaleRef sa, sb;
    int mode;
    int M, N, num_kb;          // grouped rows: M = all rows; grouped K: num_kb = all k-blocks
    int num_m, num_n;          // tile grid of one problem (grouped rows: num_m unused)
    int num_groups;
    const int* offsets;        // device, num_groups + 1 (grouped modes)
    int stream;                // k-block iterations dealt evenly to the workers (dense, grouped rows)
    int raster_m;              // tile rows walked before the next tile column
    int stages;
    uint32_t ab_fmt;
    float beta;
    const void* C;
    long long ldc;
    int c_f32, c_vec;
    const void* bias;
    int bias_f32;
    int act;
    void* D;
    long long ldd;
    int d_f32;
    int d_vec;                 // bytes of one vector store of D: 32, 16, or 0 (staged, element-wise)
    float* partials;           // [2 * worker + which][column][128]
    int* counters;             // [worker]
    int* status;
    long long timeout_ns;
    int fault_inject;
};

// One piece of work: the output tile's place, its k-blocks, and its share of
// the tile.  Row and k-block numbers are those of the operands in memory.
struct Piece {
    int g, m0, m_end, n0;      // rows [m0, m_end) may be stored
    int b_row;                 // row of B's map where the tile starts
    int d_row;                 // added to a row number for D and C (grouped K: g * M)
    int kb0, kb1;              // k-blocks of this piece
    int nsplit, split, first;  // pieces of the tile, this one's place, the first piece's worker
    int tile;
};

struct alignas(16) Ctl {
    uint64_t full[16];
    uint64_t empty[16];
    uint64_t tmem_full[4];
    uint64_t tmem_empty[4];
    uint64_t scale_full[kScaleSlots];
    uint64_t scale_empty[kScaleSlots];
    uint64_t drain;
    uint32_t tmem_base;
    int abort_flag;
    int last;
    Piece piece[kMaxPromoteWarps];
};

// (the clock is read once every 64 tries: reading it takes longer than most waits)
__device__ __forceinline__ bool spin(uint64_t* bar, uint32_t parity, const Params& p, Ctl* ctl, int where,
                                     bool honor_abort) {
    const uint32_t a = ptx::smem_u32(bar);
    uint64_t t0 = 0;
    uint32_t n = 0;
    while (true) {
        if (ptx::mbar_try_wait(a, parity)) return true;
        if ((++n & 63u) == 0) {
            if (honor_abort && *reinterpret_cast<volatile int*>(&ctl->abort_flag)) return false;
            const uint64_t now = ptx::globaltimer_ns();
            if (t0 == 0) t0 = now;
            if (static_cast<long long>(now - t0) > p.timeout_ns) {
                *reinterpret_cast<volatile int*>(&ctl->abort_flag) = 1;
                if (p.stream) p.status[3] = 1;   // shared tiles' counters may be left counting
                if (atomicCAS(p.status, 0, kStatusTimeout) == 0) {
                    p.status[1] = where;
                    p.status[2] = static_cast<int>(blockIdx.x);
                }
                return false;
            }
        }
    }
}

// Two barriers in one question: the even lanes ask about the first, the odd
// ones about the second.  A vote passes on that both have completed, not what
// either lane's wait made visible to it; the warp barrier does, so that every
// lane may use what both barriers guard.  (It stands between the wait and the
// vote: 8192^3 506 us, 514 with the vote first; every lane asking both barriers
// needs none, 520.)
__device__ __forceinline__ bool wait_pair(uint64_t* bar0, uint32_t parity0, uint64_t* bar1, uint32_t parity1, int lane,
                                          const Params& p, Ctl* ctl, int where) {
    const bool odd = lane & 1;
    const uint32_t a = ptx::smem_u32(odd ? bar1 : bar0), parity = odd ? parity1 : parity0;
    bool ok = ptx::mbar_try_wait(a, parity);
    __syncwarp();
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) {
        ok = __all_sync(0xffffffffu, spin(odd ? bar1 : bar0, parity, p, ctl, where, true));
        __syncwarp();
    }
    return ok;
}

// One lane of the converged warp, chosen by the hardware: the compiler knows
// that a single thread runs what follows and keeps the MMA's operands in
// uniform registers (issuing a k-block takes 200 cycles; 390 with `lane == 0`).
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred P;\n\t"
        "elect.sync _|P, 0xffffffff;\n\t"
        "selp.b32 %0, 1, 0, P;\n\t}"
        : "=r"(r));
    return r != 0;
}

// The whole warp waits, then agrees on the outcome.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, const Params& p, Ctl* ctl, int where,
                                          bool honor_abort = true) {
    bool ok = ptx::mbar_try_wait(ptx::smem_u32(bar), parity);
    if (!ok) ok = spin(bar, parity, p, ctl, where, honor_abort);
    return __all_sync(0xffffffffu, ok);
}

// 32 lanes x 16 or 32 consecutive TMEM columns.  The registers are valid
// after tmem_wait; what uses them is volatile too (fold), so that none moves
// ahead of it.
__device__ __forceinline__ void tmem_load(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_load(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// (volatile, so that none moves ahead of the wait for its operand)
__device__ __forceinline__ void fold(float& acc, uint32_t t, float s) {
    asm volatile("fma.rn.f32 %0, %1, %2, %0;" : "+f"(acc) : "r"(t), "f"(s));
}

// The four K = 32 MMAs of one k-block into fresh accumulator columns, and the
// arrival on `full` (of both CTAs of a pair) when they have ended.  One block
// of instructions, operand descriptors as 32-bit halves: what the issuing
// thread spends here (elect_one) and on everything else of a k-block has to
// fit into the 512 cycles that the MMAs of a pair tile take.
template <bool kPair>
__device__ __forceinline__ void mma_kblock(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc,
                                           uint64_t* full) {
    if constexpr (kPair) {
        asm volatile(
            "{\n\t.reg .pred z, o;\n\t.reg .b64 a, b;\n\t.reg .b32 x, y;\n\t.reg .b16 m;\n\t"
            "setp.ne.b32 z, 0, 0;\n\tsetp.eq.b32 o, 0, 0;\n\tmov.b16 m, 3;\n\t"
            "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a, b, %4, z;\n\t"
            "add.u32 x, %1, 2;\n\tadd.u32 y, %2, 2;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a, b, %4, o;\n\t"
            "add.u32 x, %1, 4;\n\tadd.u32 y, %2, 4;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a, b, %4, o;\n\t"
            "add.u32 x, %1, 6;\n\tadd.u32 y, %2, 6;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a, b, %4, o;\n\t"
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%5], m;\n\t}" ::"r"(d_tmem),
            "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(ptx::smem_u32(full))
            : "memory");
    } else {
        asm volatile(
            "{\n\t.reg .pred z, o;\n\t.reg .b64 a, b;\n\t.reg .b32 x, y;\n\t"
            "setp.ne.b32 z, 0, 0;\n\tsetp.eq.b32 o, 0, 0;\n\t"
            "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %4, z;\n\t"
            "add.u32 x, %1, 2;\n\tadd.u32 y, %2, 2;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %4, o;\n\t"
            "add.u32 x, %1, 4;\n\tadd.u32 y, %2, 4;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %4, o;\n\t"
            "add.u32 x, %1, 6;\n\tadd.u32 y, %2, 6;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %4, o;\n\t"
            "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%5];\n\t}" ::"r"(d_tmem),
            "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(ptx::smem_u32(full))
            : "memory");
    }
}

// 4-byte asynchronous copy global -> shared, and the arrival (one of the
// barrier's expected ones) once this thread's copies so far have landed.
__device__ __forceinline__ void copy4_async(uint32_t smem_addr, const float* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr), "l"(reinterpret_cast<uint64_t>(src)) : "memory");
}
__device__ __forceinline__ void copies_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(ptx::smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void copies_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Arrival on the pair leader's barrier.  It hands over TMEM columns that this
// warp has read (tcgen05.wait::ld returned the values to registers), no
// memory, so it needs no release at cluster scope: with one, the fence in
// front of it held each k-block up for over a thousand cycles (8192^3: 1064 us).
__device__ __forceinline__ void arrive_cluster(uint32_t addr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

// ------------------------------------------------------------------ schedule

__device__ __forceinline__ Piece load_piece(const volatile Piece* s) {
    Piece w;
    w.g = s->g;
    w.m0 = s->m0;
    w.m_end = s->m_end;
    w.n0 = s->n0;
    w.b_row = s->b_row;
    w.d_row = s->d_row;
    w.kb0 = s->kb0;
    w.kb1 = s->kb1;
    w.nsplit = s->nsplit;
    w.split = s->split;
    w.first = s->first;
    w.tile = s->tile;
    return w;
}

// Group tables in shared memory, built once per CTA: first tile (grouped
// rows) or first k-block (grouped K) of each group, and, for grouped rows, its
// first row.  The groups lie one after the other, so each ends where the next
// begins.
struct Groups {
    const int* start;   // num_groups + 1
    const int* row;     // num_groups + 1 (grouped rows alone)
};

// (group_rows: whatever the offsets hold, the groups share the operand's rows
// out, so every sum here is bounded by the operand's own tiles or k-blocks
// and one more a group.)
template <int kTileM>
__device__ __forceinline__ void build_groups(const Params& p, int* start, int* row, int lane) {
    const int cap = p.mode == kGroupedRows ? p.M : p.num_kb * kBlock;
    int base = 0, last = 0;
    for (int g0 = 0; g0 < p.num_groups; g0 += 32) {
        const int g = g0 + lane;
        int n, r;
        group_rows(p.offsets, p.num_groups, cap, g0, lane, last, r, n);
        if (g < p.num_groups && p.mode == kGroupedRows) {
            if (g == 0) row[0] = r;
            row[g + 1] = r + n;
        }
        int c = p.mode == kGroupedRows ? (n + kTileM - 1) / kTileM * p.num_n : (n + kBlock - 1) / kBlock;
        int incl = c;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += o;
        }
        if (g < p.num_groups) start[g] = base + incl - c;
        base += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) start[p.num_groups] = base;
}

__device__ __forceinline__ int find_group(const Groups& gr, int n, int t) {
    int lo = 0, hi = n - 1;   // the last group that starts at or before t
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (gr.start[mid] <= t) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ int total_tiles(const Params& p, const Groups& gr) {
    if (p.mode == kGroupedRows) return gr.start[p.num_groups];
    return p.num_m * p.num_n * (p.mode == kGroupedK ? p.num_groups : 1);
}

template <int kTileM, int kTileN>
__device__ __forceinline__ void decode_tile(const Params& p, const Groups& gr, int t, Piece& w) {
    int local = t, nm = p.num_m;
    w.tile = t;
    w.g = 0;
    w.d_row = 0;
    int row0 = 0;
    w.m_end = p.M;
    w.kb0 = 0;
    w.kb1 = p.num_kb;
    int brow = 0;
    if (p.mode == kGroupedRows) {
        w.g = find_group(gr, p.num_groups, t);
        local = t - gr.start[w.g];
        row0 = gr.row[w.g];
        w.m_end = gr.row[w.g + 1];
        nm = (w.m_end - row0 + kTileM - 1) / kTileM;
        brow = w.g * p.N;
    } else if (p.mode == kGroupedK) {
        const int per = p.num_m * p.num_n;
        w.g = t / per;
        local = t - w.g * per;
        w.kb0 = min(gr.start[w.g], p.num_kb);
        w.kb1 = min(gr.start[w.g + 1], p.num_kb);
        w.d_row = w.g * p.M;
    }
    // raster_m tile rows at a time, column by column ("CUTLASS", Part IV
    // Stage 2: the tile order that lets co-resident tiles share operands in L2)
    const int span = p.raster_m * p.num_n;
    const int band = local / span;
    const int rows = min(nm - band * p.raster_m, p.raster_m);
    const int in = local - band * span;
    const int mb = band * p.raster_m + in % rows;
    const int nb = in / rows;
    w.m0 = row0 + mb * kTileM;
    w.n0 = nb * kTileN;
    w.b_row = brow + w.n0;
    w.nsplit = 1;
    w.split = 0;
    w.first = 0;
}

// The pieces of one worker.  Whole tiles: every workers-th one.  stream: the
// k-block iterations of all tiles in one line, an equal run of them per
// worker; a tile whose iterations fall to several workers is finished by the
// last of them (one such tile at most begins in any worker's run, so the
// first worker's number also names its arrival counter).
template <bool kMayStream>
struct Walk {
    int it, end, step;   // tiles
    __device__ __forceinline__ Walk(const Params& p, const Groups& gr, int wid, int workers)
        : it(wid), end(total_tiles(p, gr)), step(workers) {}
    template <int kTileM, int kTileN>
    __device__ __forceinline__ bool next(const Params& p, const Groups& gr, Piece& w) {
        if (it >= end) return false;
        decode_tile<kTileM, kTileN>(p, gr, it, w);
        it += step;
        return true;
    }
};
template <>
struct Walk<true> {
    long long it, end;   // stream: iterations; otherwise tiles
    long long total;
    int wid, workers;
    __device__ __forceinline__ Walk(const Params& p, const Groups& gr, int wid_, int workers_) : wid(wid_), workers(workers_) {
        const int tiles = total_tiles(p, gr);
        if (p.stream) {
            total = static_cast<long long>(tiles) * p.num_kb;
            // never more workers than iterations, so that every worker of a tile holds a piece of it
            if (total < workers) workers = static_cast<int>(total);
            it = wid < workers ? wid * total / workers : 0;
            end = wid < workers ? (wid + 1) * total / workers : 0;
        } else {
            total = tiles;
            it = wid;
            end = tiles;
        }
    }
    __device__ __forceinline__ int worker_of(long long i) const { return static_cast<int>(((i + 1) * workers - 1) / total); }
    template <int kTileM, int kTileN>
    __device__ __forceinline__ bool next(const Params& p, const Groups& gr, Piece& w) {
        if (it >= end) return false;
        if (!p.stream) {
            decode_tile<kTileM, kTileN>(p, gr, static_cast<int>(it), w);
            it += workers;
            return true;
        }
        const int t = static_cast<int>(it / p.num_kb);
        const long long t0 = static_cast<long long>(t) * p.num_kb;
        decode_tile<kTileM, kTileN>(p, gr, t, w);
        w.kb0 = static_cast<int>(it - t0);
        const long long left = end - t0;
        w.kb1 = left < p.num_kb ? static_cast<int>(left) : p.num_kb;
        w.first = worker_of(t0);
        w.nsplit = worker_of(t0 + p.num_kb - 1) - w.first + 1;
        w.split = wid - w.first;
        it = t0 + w.kb1;
        return true;
    }
};

// Partial slot of piece q of a shared tile.  A worker's run can share the tile
// it starts in (slot 0: the run starts at or after the tile's first k-block)
// and the one it ends in (slot 1: the run starts before the tile).
__device__ __forceinline__ int slot_of(const Params& p, const Walk<true>& s, const Piece& w, int q) {
    const int c = w.first + q;
    const bool begins = c * s.total / s.workers >= static_cast<long long>(w.tile) * p.num_kb;
    return 2 * c + (begins ? 0 : 1);
}

// Where the scales of a row of group g start (rows past the group's last one
// take that one's: nobody stores what they scale).
__device__ __forceinline__ const float* scale_row(const ScaleRef& s, int row, int last, int g) {
    return s.ptr + static_cast<long long>(min(row, last) >> s.shift) * s.rs + g * s.gs;
}

// ------------------------------------------------------------------ epilogue

__device__ __forceinline__ float load_elem(const void* base, int is_f32, long long i) {
    return is_f32 ? static_cast<const float*>(base)[i] : bf16_bits_to_float(static_cast<const uint16_t*>(base)[i]);
}

// beta C + bias (the columns' values in shared memory), activation, on CN (16
// or 32) consecutive columns of one row
template <int CN>
__device__ __forceinline__ void finish_values(const Params& p, float (&v)[CN], long long row, int col0, int rows_ok, int lane,
                                              const float* bias, uint32_t* stage) {
    if (p.beta != 0.0f) {
        const long long at = row * p.ldc + col0;
        if (p.c_vec && col0 + CN <= p.N) {
            if (lane < rows_ok) {
                if (p.c_f32) {
                    const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(p.C) + at);
#pragma unroll
                    for (int i = 0; i < CN / 4; ++i) {
                        const float4 c = __ldcs(src + i);
                        v[4 * i] = fmaf(p.beta, c.x, v[4 * i]);
                        v[4 * i + 1] = fmaf(p.beta, c.y, v[4 * i + 1]);
                        v[4 * i + 2] = fmaf(p.beta, c.z, v[4 * i + 2]);
                        v[4 * i + 3] = fmaf(p.beta, c.w, v[4 * i + 3]);
                    }
                } else {
                    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.C) + at);
#pragma unroll
                    for (int i = 0; i < CN / 8; ++i) {
                        const uint4 c = __ldcs(src + i);
                        const uint32_t u[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
                            v[8 * i + 2 * h] = fmaf(p.beta, bf16_bits_to_float(u[h] & 0xFFFFu), v[8 * i + 2 * h]);
                            v[8 * i + 2 * h + 1] = fmaf(p.beta, bf16_bits_to_float(u[h] >> 16), v[8 * i + 2 * h + 1]);
                        }
                    }
                }
            }
        } else {
            // Rows that do not start on 16 bytes turn through shared memory: 16
            // lanes read consecutive elements of one row (a thread reading its own
            // row element by element fetches a sector for each: 16 x 1280 x 522
            // f32, 210 us).
            const long long base = (row - lane) * p.ldc + col0 + (lane & 15);
            float* st = reinterpret_cast<float*>(stage);
#pragma unroll
            for (int h = 0; h < CN / 16; ++h) {
                const bool in = col0 + 16 * h + (lane & 15) < p.N;
                float got[16];   // (every load first: the compiler moves none past a store)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int r = 2 * i + (lane >> 4);
                    got[i] = in && r < rows_ok ? load_elem(p.C, p.c_f32, base + r * p.ldc + 16 * h) : 0.0f;
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 16; ++i) st[(2 * i + (lane >> 4)) * 17 + (lane & 15)] = got[i];
                __syncwarp();
                if (lane < rows_ok) {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (col0 + 16 * h + i < p.N) v[16 * h + i] = fmaf(p.beta, st[lane * 17 + i], v[16 * h + i]);
                }
            }
        }
    }
    if (p.bias) {
#pragma unroll
        for (int i = 0; i < CN / 4; ++i) {
            const float4 b = reinterpret_cast<const float4*>(bias)[i];
            v[4 * i] += b.x;
            v[4 * i + 1] += b.y;
            v[4 * i + 2] += b.z;
            v[4 * i + 3] += b.w;
        }
    }
    if (p.act == 2) {
#pragma unroll
        for (int i = 0; i < CN / 2; ++i)
            ptx::unpack2(gelu_erf2(ptx::pack2(v[2 * i], v[2 * i + 1])), v[2 * i], v[2 * i + 1]);
    } else if (p.act == 1) {
#pragma unroll
        for (int i = 0; i < CN; ++i) v[i] = apply_act(1, v[i]);
    }
}

constexpr int kStageWords = 32 * 17;   // per promote warp: 32 rows of 16 words, one word apart from the next row

// Store CN columns of the warp's 32 rows.  Rows whose addresses allow it go
// out from registers, 32 or 16 bytes at a time; otherwise (an odd pitch, a
// ragged last chunk) the chunk turns through shared memory so that each store
// instruction covers consecutive elements of one row.
template <int CN>
__device__ __forceinline__ void store_values(const Params& p, const float (&v)[CN], long long row, int col0,
                                             int rows_ok, int lane, uint32_t* stage) {
    if (p.d_vec && col0 + CN <= p.N) {
        if (lane < rows_ok) {
            char* dst = static_cast<char*>(p.D) + (row * p.ldd + col0) * (p.d_f32 ? 4 : 2);
            uint32_t w[CN];
            if (p.d_f32) {
#pragma unroll
                for (int i = 0; i < CN; ++i) w[i] = __float_as_uint(v[i]);
            } else {
#pragma unroll
                for (int i = 0; i < CN / 2; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
            }
            const int words = p.d_f32 ? CN : CN / 2;
            if (p.d_vec == 32) {
#pragma unroll
                for (int i = 0; i < CN / 8; ++i) {
                    if (8 * i < words) {
                        const uint32_t q[8] = {w[8 * i], w[8 * i + 1], w[8 * i + 2], w[8 * i + 3],
                                               w[8 * i + 4], w[8 * i + 5], w[8 * i + 6], w[8 * i + 7]};
                        ptx::st_global_v8(dst + 32 * i, q);
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < CN / 4; ++i)
                    if (4 * i < words)
                        *reinterpret_cast<uint4*>(dst + 16 * i) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
            }
        }
        return;
    }
    const long long row_base = row - lane;
    if (p.d_f32) {
#pragma unroll
        for (int h = 0; h < CN / 16; ++h) {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 16; ++i) stage[lane * 17 + i] = __float_as_uint(v[16 * h + i]);
            __syncwarp();
            const int c = col0 + 16 * h + (lane & 15);
#pragma unroll 4
            for (int r = lane >> 4; r < rows_ok; r += 2)
                if (c < p.N) static_cast<float*>(p.D)[(row_base + r) * p.ldd + c] = __uint_as_float(stage[r * 17 + (lane & 15)]);
        }
    } else {
#pragma unroll
        for (int h = 0; h < (CN + 31) / 32; ++h) {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < (CN < 32 ? CN : 32) / 2; ++i)
                stage[lane * 17 + i] = pack_bf16x2(v[32 * h + 2 * i], v[32 * h + 2 * i + 1]);
            __syncwarp();
            const int c = col0 + 32 * h + lane;
            const uint16_t* s16 = reinterpret_cast<const uint16_t*>(stage);
            if (lane < CN && c < p.N)
#pragma unroll 4
                for (int r = 0; r < rows_ok; ++r)
                    static_cast<uint16_t*>(p.D)[(row_base + r) * p.ldd + c] = s16[r * 34 + lane];
        }
    }
}

// ------------------------------------------------------------------ kernels

// kPair: 256 x 256 tiles on CTA pairs; otherwise kTileN columns per CTA.
// kSwap: few rows of A.  B's rows take the 128 TMEM lanes and A's rows the
// kTileN MMA columns, so that no lane computes padding; the tile is
// D[m0 .. m0 + kTileN, n0 .. n0 + 128].
// kColScale: one scale per B row (per MMA column), else one per 128.
template <int kTileN, bool kPair, bool kSwap, bool kColScale>
struct Shape {
    static constexpr int kPromoteWarps = kSwap ? 4 : kMaxPromoteWarps;
    // The eight promote warps of a wide tile hold 128 (a pair) or 64 sums a
    // thread; they take over registers that the four control warps give back
    // (128 * 56 + 256 * 224 = 384 * 168, what the block is launched with; 40 and
    // 232 or 72 and 216: 8192^3 the same, weight gradients 1 and 4 % slower).
    static constexpr int kControlWarps = 4;
    static constexpr bool kSplitRegs = !kSwap;
    static constexpr int kControlRegs = 56, kPromoteRegs = 224, kLaunchRegs = 168;
    static constexpr int kThreads = 32 * (kControlWarps + kPromoteWarps);
    static_assert(!kSplitRegs || 32 * (kControlWarps * kControlRegs + kPromoteWarps * kPromoteRegs) <= kThreads * kLaunchRegs,
                  "the shares add up to the launch's registers");
    static constexpr int kLaneRows = 128;                          // rows of the lane operand per CTA
    static constexpr int kColRows = kPair ? kTileN / 2 : kTileN;   // rows of the column operand per CTA
    static constexpr int kAtomBytes = (kLaneRows + kColRows) * kBlock;
    static constexpr int kAtoms = kSwap ? 1 : 2;                   // k-blocks per pipeline stage
    static constexpr int kStageBytes = kAtoms * kAtomBytes;
    static constexpr int kBufs = kPair ? 2 : 4;
    static constexpr int kTmemCols = kBufs * kTileN < 32 ? 32 : kBufs * kTileN;
    static constexpr int kWarpCols = kSwap ? kTileN : kTileN / 2;  // MMA columns of one promote warp
    // store stage and bias of one promote warp
    static constexpr int kWarpWords = kSwap ? 0 : kStageWords + kWarpCols;
    // scales of one k-block: a word per lane row, then one per MMA column (or
    // per 128 columns)
    static constexpr bool kCols = kColScale || kSwap;
    static constexpr int kColWords = kCols ? kTileN : 4;
    static constexpr int kSlotWords = 128 + kColWords;
    // Stages at most.  Few rows: five of one k-block, so that two blocks fit on
    // an SM and the next call's set up beside this one's (1 x 8192 x 8192 back to
    // back: 24.6 us with the SM's memory full of stages, 22.3 with five, 19.6 with
    // the early launch).  Pairs: two, although three fit where there are few
    // groups; the L1 that the third would take holds what the promote warps spill
    // (8192^3 521 us with three, 514 with two; a scale per row of B 742 and 707;
    // weight gradients of 4096 x 4096 over 16384 rows in 7 groups 618 and 587).
    // Single tiles: three (256 x 8192 x 8192 35 us, 38 with two), two where the
    // tables of 780 groups and more and a scale per row of B leave no room.
    static constexpr int kMaxStages = kSwap ? 5 : kPair ? 2 : 3;
    static constexpr int kMinStages = kSwap ? 5 : 2;   // fit whatever the groups (asserted below)
    static constexpr int kTileM = kSwap ? kTileN : (kPair ? 256 : 128);   // rows of D per tile
    static constexpr int kTileNOut = kSwap ? 128 : kTileN;                // columns of D per tile
    static_assert((kTmemCols & (kTmemCols - 1)) == 0 && kTmemCols <= 512, "TMEM columns are a power of two");
    static_assert(kAtomBytes % 1024 == 0, "atoms stay 1024-byte aligned");
    // tables: 0 (dense), 1 (grouped K) or 2 (grouped rows) of groups + 1 words
    static constexpr int smem_bytes(int stages, int tables, int groups) {
        return 1024 + stages * kStageBytes + (kPromoteWarps * kWarpWords + kScaleSlots * kSlotWords) * 4 + static_cast<int>(sizeof(Ctl)) +
               tables * (groups + 1) * 4;
    }
};

constexpr int kSmemBytes = 232448;   // 227 KiB, the most a block may have
template <typename S>
constexpr bool fits_any_groups() { return S::smem_bytes(S::kMinStages, 2, kMaxGroups) <= kSmemBytes; }
static_assert(fits_any_groups<Shape<256, true, false, true>>() && fits_any_groups<Shape<256, true, false, false>>() &&
                  fits_any_groups<Shape<128, false, false, true>>() && fits_any_groups<Shape<128, false, false, false>>() &&
                  fits_any_groups<Shape<16, false, true, false>>() && fits_any_groups<Shape<32, false, true, false>>(),
              "group tables take no stage below kMinStages");

template <int kTileN, bool kPair, bool kSwap, bool kColScale>
__global__ void __launch_bounds__(Shape<kTileN, kPair, kSwap, kColScale>::kThreads, 1)
    block128_kernel(const __grid_constant__ Params p) {
    using S = Shape<kTileN, kPair, kSwap, kColScale>;
    constexpr int kAtoms = S::kAtoms;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int stages = p.stages;
    uint32_t* warp_words = reinterpret_cast<uint32_t*>(smem + stages * S::kStageBytes);
    float* scale_words = reinterpret_cast<float*>(warp_words + S::kPromoteWarps * S::kWarpWords);
    Ctl* ctl = reinterpret_cast<Ctl*>(scale_words + kScaleSlots * S::kSlotWords);
    int* tables = reinterpret_cast<int*>(ctl + 1);
    const Groups gr{tables, tables + p.num_groups + 1};

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = kPair ? ptx::cluster_ctarank() : 0u;
    const bool leader = rank == 0;
    using WalkT = Walk<!kPair>;
    const int wid = kPair ? static_cast<int>(blockIdx.x >> 1) : static_cast<int>(blockIdx.x);
    const int workers = kPair ? static_cast<int>(gridDim.x >> 1) : static_cast<int>(gridDim.x);

    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            ptx::mbar_init(&ctl->full[s], 1);
            ptx::mbar_init(&ctl->empty[s], 1);
        }
        for (int b = 0; b < S::kBufs; ++b) {
            ptx::mbar_init(&ctl->tmem_full[b], 1);
            ptx::mbar_init(&ctl->tmem_empty[b], S::kPromoteWarps * (kPair ? 2 : 1));
        }
        for (int s = 0; s < kScaleSlots; ++s) {
            ptx::mbar_init(&ctl->scale_full[s], 32);
            ptx::mbar_init(&ctl->scale_empty[s], S::kPromoteWarps);
        }
        ptx::mbar_init(&ctl->drain, 1);
        ctl->abort_flag = 0;
        ctl->last = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 1) {
        if constexpr (kPair) {
            ptx::tmem_alloc_pair(&ctl->tmem_base, S::kTmemCols);
            ptx::tmem_relinquish_alloc_permit_pair();
        } else {
            ptx::tmem_alloc(&ctl->tmem_base, S::kTmemCols);
            ptx::tmem_relinquish_alloc_permit();
        }
    }
    // Blocks of the next call may start as this one's end, and set up so far;
    // what the call before has written is read only from here on.
    host::wait_for_kernel_ahead();
    if (warp == 0 && p.mode != kDense)
        build_groups<S::kTileM>(p, tables, tables + p.num_groups + 1, lane);
    ptx::tc_fence_before_sync();
    if constexpr (kPair) ptx::cluster_sync();   // the peer's barriers exist before anyone signals them
    __syncthreads();
    ptx::tc_fence_after_sync();
    const uint32_t tmem_base = ctl->tmem_base;

    if (warp < S::kControlWarps) {
        if constexpr (S::kSplitRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kControlRegs));
        if (warp == 0) {
        // ------------------------------------------------------ TMA producer
        WalkT walk(p, gr, wid, workers);
        Piece w;
        const bool issuer = lane == 0;
        if (issuer && p.num_kb > 0) {
            ptx::prefetch_tensormap(&p.tmA);
            ptx::prefetch_tensormap(&p.tmB);
        }
        int stage = 0;
        uint32_t phase = 0, armed = 0, armed_parity = 0;
        bool first = true, ok = true;
        while (ok && walk.template next<S::kTileM, S::kTileNOut>(p, gr, w)) {
            const int a_row = w.m0 + (kPair ? static_cast<int>(rank) * 128 : 0);
            const int b_row = w.b_row + (kPair ? static_cast<int>(rank) * S::kColRows : 0);
            for (int kb = w.kb0; kb < w.kb1; kb += kAtoms) {
                if (!wait_warp(&ctl->empty[stage], phase ^ 1u, p, ctl, 1)) { ok = false; break; }
                const int atoms = min(kAtoms, w.kb1 - kb);
                const bool skip = first && p.fault_inject == 1 && blockIdx.x == 0;
                first = false;
                if (!skip) {
                    if (issuer) {
                        uint64_t* fb = &ctl->full[stage];
                        if (leader) ptx::mbar_arrive_expect_tx(fb, static_cast<uint32_t>((kPair ? 2 : 1) * atoms * S::kAtomBytes));
                        const uint32_t fbc = kPair ? ptx::map_to_cta(ptx::smem_u32(fb), 0) : 0u;
                        for (int at = 0; at < atoms; ++at) {
                            uint8_t* sl = smem + stage * S::kStageBytes + at * S::kAtomBytes;
                            uint8_t* sc = sl + S::kLaneRows * kBlock;
                            const int x = (kb + at) * kBlock;
                            const CUtensorMap* tl = kSwap ? &p.tmB : &p.tmA;
                            const CUtensorMap* tc = kSwap ? &p.tmA : &p.tmB;
                            const int yl = kSwap ? b_row : a_row, yc = kSwap ? a_row : b_row;
                            if constexpr (kPair) {
                                ptx::tma_load_2d_pair(sl, tl, fbc, x, yl);
                                ptx::tma_load_2d_pair(sc, tc, fbc, x, yc);
                            } else {
                                ptx::tma_load_2d(sl, tl, fb, x, yl);
                                ptx::tma_load_2d(sc, tc, fb, x, yc);
                            }
                        }
                    }
                    armed |= 1u << stage;
                    armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
                }
                __syncwarp();
                if (++stage == stages) { stage = 0; phase ^= 1u; }
            }
        }
        // Every copy of this thread has landed before the CTA may leave: the
        // leader sees it on its full barriers, the peer (whose copies count on
        // the leader's) by their consumption.
        for (int s = 0; s < stages; ++s) {
            if (!(armed & (1u << s))) continue;
            const uint32_t par = (armed_parity >> s) & 1u;
            if (leader) wait_warp(&ctl->full[s], par, p, ctl, 11, false);
            else wait_warp(&ctl->empty[s], par, p, ctl, 13, false);
        }
        } else if (warp == 1 && leader) {
        // ------------------------------------------------------- MMA issuer
        {
        WalkT walk(p, gr, wid, workers);
        Piece w;
            const uint32_t idesc = (1u << 4) | (p.ab_fmt << 7) | (p.ab_fmt << 10) |
                                   (static_cast<uint32_t>(kTileN >> 3) << 17) |
                                   (static_cast<uint32_t>((kPair ? 256 : 128) >> 4) << 24);
            // descriptor halves: 128-byte swizzle, 8-row groups 1024 bytes apart
            constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
            const uint32_t desc0 = (ptx::smem_u32(smem) >> 4) | (1u << 16);
            int stage = 0, buf = 0;
            uint32_t phase = 0, bphase = 0;
            bool ok = true, issued = false;
            while (ok && walk.template next<S::kTileM, S::kTileNOut>(p, gr, w)) {
                for (int kb = w.kb0; kb < w.kb1; kb += kAtoms) {
#pragma unroll
                    for (int at = 0; at < kAtoms; ++at) {
                        if (kb + at >= w.kb1) break;
                        ok = at == 0 ? wait_pair(&ctl->full[stage], phase, &ctl->tmem_empty[buf], bphase ^ 1u, lane, p, ctl, 3)
                                     : wait_warp(&ctl->tmem_empty[buf], bphase ^ 1u, p, ctl, 2);
                        if (!ok) break;
                        ptx::tc_fence_after_sync();
                        if (elect_one()) {
                            const uint32_t a_lo = desc0 + static_cast<uint32_t>(stage * S::kStageBytes + at * S::kAtomBytes) / 16;
                            mma_kblock<kPair>(tmem_base + static_cast<uint32_t>(buf * kTileN), a_lo,
                                              a_lo + S::kLaneRows * kBlock / 16, kDescHi, idesc, &ctl->tmem_full[buf]);
                            if (at == kAtoms - 1 || kb + at + 1 == w.kb1) {   // the stage's last k-block
                                if constexpr (kPair) ptx::mma_commit_pair(&ctl->empty[stage], 0x3);
                                else ptx::mma_commit(&ctl->empty[stage]);
                            }
                        }
                        issued = true;
                        if (++buf == S::kBufs) { buf = 0; bphase ^= 1u; }
                    }
                    if (!ok) break;
                    if (++stage == stages) { stage = 0; phase ^= 1u; }
                }
            }
            __syncwarp();
            if (issued) {   // every MMA has ended before the TMEM is freed
                if (elect_one()) {
                    if constexpr (kPair) ptx::mma_commit_pair(&ctl->drain, 0x1);
                    else ptx::mma_commit(&ctl->drain);
                }
                __syncwarp();
                wait_warp(&ctl->drain, 0, p, ctl, 12, false);
            }
        }
        } else if (warp == 2) {
        // ---------------------------------------------------- scales, ahead
        WalkT walk(p, gr, wid, workers);
        Piece w;
        const ScaleRef& sl = kSwap ? p.sb : p.sa;
        const ScaleRef& sc = kSwap ? p.sa : p.sb;
        constexpr int kColLoads = S::kCols ? (kTileN + 31) / 32 : 1;
        const bool col_lane = S::kCols ? lane < kTileN : lane < kTileN / 128;
        int slot = 0;
        uint32_t phase = 0;
        bool ok = true;
        while (ok && walk.template next<S::kTileM, S::kTileNOut>(p, gr, w)) {
            const int l0 = kSwap ? w.n0 : w.m0 + static_cast<int>(rank) * 128;
            const int c0 = kSwap ? w.m0 : w.n0;
            const int l_last = (kSwap ? p.N : w.m_end) - 1, c_last = (kSwap ? w.m_end : p.N) - 1;
            const float* lp[4];
            const float* cp[kColLoads];
#pragma unroll
            for (int i = 0; i < 4; ++i) lp[i] = scale_row(sl, l0 + lane + 32 * i, l_last, w.g) + w.kb0 * sl.ks;
#pragma unroll
            for (int i = 0; i < kColLoads; ++i)
                cp[i] = scale_row(sc, c0 + (S::kCols ? lane + 32 * i : 128 * lane), c_last, w.g) + w.kb0 * sc.ks;
            for (int kb = w.kb0; kb < w.kb1; ++kb) {
                if (!wait_warp(&ctl->scale_empty[slot], phase ^ 1u, p, ctl, 6)) { ok = false; break; }
                const uint32_t dst = ptx::smem_u32(scale_words + slot * S::kSlotWords + lane);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    copy4_async(dst + 128 * i, lp[i]);
                    lp[i] += sl.ks;
                }
#pragma unroll
                for (int i = 0; i < kColLoads; ++i) {
                    if (col_lane) copy4_async(dst + 512 + 128 * i, cp[i]);
                    cp[i] += sc.ks;
                }
                copies_arrive(&ctl->scale_full[slot]);
                if (++slot == kScaleSlots) { slot = 0; phase ^= 1u; }
            }
        }
        copies_wait_all();
        }
    } else {
        // ------------------------------------------------ promote and store
        if constexpr (S::kSplitRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::kPromoteRegs));
        WalkT walk(p, gr, wid, workers);
        Piece w;
        const int pw = warp - S::kControlWarps;
        const int quad = warp & 3;               // the TMEM lanes this warp may read
        const int col_base = kSwap ? 0 : (pw >> 2) * S::kWarpCols;
        constexpr int WC = S::kWarpCols;
        // (16 on a pair tile: with two chunks of 32 next to 128 sums the compiler
        // spills in the loop, and with next to no L1 left a reload comes from L2)
        constexpr int kChunk = WC < 32 ? WC : (kPair ? 16 : 32);
        constexpr int kChunks = WC / kChunk;
        constexpr int kOut = WC < 32 ? WC : 32;   // columns stored at a time
        uint32_t* my_words = warp_words + pw * S::kWarpWords;
        Piece* my_piece = &ctl->piece[pw];
        float* bias_cols = reinterpret_cast<float*>(my_words + kStageWords);
        int buf = 0, slot = 0;
        uint32_t bphase = 0, sphase = 0;
        bool ok = true;
        const int bar_threads = 32 * S::kPromoteWarps;
        // the barriers this warp arrives on: the leader's TMEM buffers, its own CTA's scale slots
        const uint32_t empty_addr = kPair ? ptx::map_to_cta(ptx::smem_u32(&ctl->tmem_empty[0]), 0) : ptx::smem_u32(&ctl->tmem_empty[0]);
        const uint32_t scale_addr = kPair ? ptx::map_to_cta(ptx::smem_u32(&ctl->scale_empty[0]), rank) : ptx::smem_u32(&ctl->scale_empty[0]);
        const int lane_row = quad * 32 + lane;   // this thread's row of the lane operand's tile
        while (ok && walk.template next<S::kTileM, S::kTileNOut>(p, gr, w)) {
            if constexpr (!kSwap) {
                // The epilogue's operands set out while the tile is computed: the
                // bias of this warp's columns to shared memory, this thread's row
                // of C to L2.
                if (p.bias) {
                    __syncwarp();   // (the last tile's readers are done)
#pragma unroll
                    for (int i = 0; i < WC / 32; ++i) {
                        const int n = w.n0 + col_base + lane + 32 * i;
                        bias_cols[lane + 32 * i] = n < p.N ? load_elem(p.bias, p.bias_f32, n) : 0.0f;
                    }
                }
                const int row = w.m0 + static_cast<int>(rank) * 128 + lane_row;
                if (p.beta != 0.0f && row < w.m_end) {
                    const long long at = (static_cast<long long>(w.d_row) + row) * p.ldc + w.n0 + col_base;
                    const int size = p.c_f32 ? 4 : 2;
                    const char* c = static_cast<const char*>(p.C) + at * size;
                    const char* end = c + min(WC, p.N - w.n0 - col_base) * size;
                    for (; c < end; c += 128) ptx::prefetch_l2(c);
                }
            }
            // (the piece waits in shared memory: the loop needs the registers; weight
            // gradients of 4096 x 4096 over 16384 rows: 904 -> 878 us)
            const int kb0 = w.kb0, kb1 = w.kb1;
            __syncwarp();   // (no lane still reads the piece before)
            if (lane == 0) *my_piece = w;
            float acc[WC];
#pragma unroll
            for (int i = 0; i < WC; ++i) acc[i] = 0.0f;
            float l_next = 0.0f, c_next = 0.0f;
            auto read_scale = [&](int sl) {
                const float* sw = scale_words + sl * S::kSlotWords;
                l_next = sw[lane_row];
                if constexpr (!S::kCols) c_next = sw[128 + col_base / 128];
            };
            if (kb0 < kb1) {
                ok = wait_warp(&ctl->scale_full[slot], sphase, p, ctl, 5);
                if (ok) read_scale(slot);
            }
            for (int kb = kb0; ok && kb < kb1; ++kb) {
                // The k-block's sums, and with them the next one's scales: those are
                // there long before, and read a whole k-block ahead of their use.
                const int nslot = slot + 1 == kScaleSlots ? 0 : slot + 1;
                const uint32_t nphase = sphase ^ (nslot == 0 ? 1u : 0u);
                const bool more = kb + 1 < kb1;
                if (!wait_pair(&ctl->tmem_full[buf], bphase, more ? &ctl->scale_full[nslot] : &ctl->tmem_full[buf],
                               more ? nphase : bphase, lane, p, ctl, 4)) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after_sync();
                const uint32_t t0 = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) +
                                    static_cast<uint32_t>(buf * kTileN + col_base);
                // one chunk is on its way from TMEM while the one before is folded in
                uint32_t r[2][kChunk];
                tmem_load(t0, r[0]);
                const float* sw = scale_words + slot * S::kSlotWords;
                const float s = S::kCols ? l_next : l_next * c_next;
                if (more) read_scale(nslot);
#pragma unroll
                for (int j = 0; j < kChunks; ++j) {
                    tmem_wait();
                    if (j + 1 < kChunks) {
                        tmem_load(t0 + (j + 1) * kChunk, r[(j + 1) & 1]);
                    } else {
                        // the buffer is free for the next k-block's MMAs (and the
                        // scales, which this thread holds unless every column has one)
                        ptx::tc_fence_before_sync();
                        __syncwarp();
                        if (lane < (S::kCols ? 1 : 2))
                            arrive_cluster(lane == 0 ? empty_addr + 8 * buf : scale_addr + 8 * slot);
                    }
#pragma unroll
                    for (int i = 0; i < kChunk / 4; ++i) {
                        const uint32_t(&q)[kChunk] = r[j & 1];
                        float* a = acc + j * kChunk + 4 * i;
                        if constexpr (S::kCols) {
                            const float4 c4 = *reinterpret_cast<const float4*>(sw + 128 + col_base + j * kChunk + 4 * i);
                            float s0, s1, s2, s3;   // (two products an instruction)
                            ptx::unpack2(ptx::mul2(ptx::pack2(s, s), ptx::pack2(c4.x, c4.y)), s0, s1);
                            ptx::unpack2(ptx::mul2(ptx::pack2(s, s), ptx::pack2(c4.z, c4.w)), s2, s3);
                            fold(a[0], q[4 * i], s0);
                            fold(a[1], q[4 * i + 1], s1);
                            fold(a[2], q[4 * i + 2], s2);
                            fold(a[3], q[4 * i + 3], s3);
                        } else {
#pragma unroll
                            for (int k = 0; k < 4; ++k) fold(a[k], q[4 * i + k], s);
                        }
                    }
                }
                if constexpr (S::kCols) {
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(&ctl->scale_empty[slot]);
                }
                if (++buf == S::kBufs) { buf = 0; bphase ^= 1u; }
                slot = nslot;
                sphase = nphase;
            }
            __syncwarp();
            w = load_piece(my_piece);
            if constexpr (!kPair) {
                // all promote warps leave together: the barriers below need every thread
                if (p.stream) ok = ptx::named_barrier_and(1, bar_threads, ok);
            }
            if (!ok) break;

            bool finish = true;
            if constexpr (!kPair) {
                if (w.nsplit > 1) {
                    // This piece's raw sums, column by column, 32 lanes on one line.
                    // The barrier orders the CTA's stores before one thread's
                    // acquire-release add; for the last arrival that add makes the
                    // others' sums visible, and the second barrier passes it on.
                    float* mine = p.partials + static_cast<size_t>(slot_of(p, walk, w, w.split)) * (128 * kTileN) +
                                  static_cast<size_t>(col_base) * 128 + lane_row;
                    // (kSwap: the columns of rows that exist; one token has one)
                    const int used_cols = kSwap ? min(WC, w.m_end - w.m0) : WC;
#pragma unroll
                    for (int i = 0; i < WC; ++i)
                        if (i < used_cols) mine[i * 128] = acc[i];
                    ptx::named_barrier_sync(1, bar_threads);
                    if (threadIdx.x == 32 * S::kControlWarps) {
                        const int old = ptx::atomic_add_acq_rel_gpu(p.counters + w.first, 1);
                        ctl->last = old == w.nsplit - 1;
                        if (ctl->last) atomicExch(p.counters + w.first, 0);   // ready for the next launch
                    }
                    ptx::named_barrier_sync(1, bar_threads);
                    finish = ctl->last != 0;
                    if (finish) {
                        // in the order of the pieces, whoever finishes: the sum is the same every time
#pragma unroll
                        for (int i = 0; i < WC; ++i) acc[i] = 0.0f;
                        // (kQ pieces' values are on their way at once)
                        constexpr int kQ = WC <= 16 ? 4 : WC <= 32 ? 2 : 1;
                        for (int q = 0; q < w.nsplit; q += kQ) {
                            float got[kQ][WC];
#pragma unroll
                            for (int h = 0; h < kQ; ++h) {
                                const float* src = p.partials + static_cast<size_t>(slot_of(p, walk, w, min(q + h, w.nsplit - 1))) * (128 * kTileN) +
                                                   static_cast<size_t>(col_base) * 128 + lane_row;
#pragma unroll
                                for (int i = 0; i < WC; ++i) got[h][i] = i < used_cols && q + h < w.nsplit ? __ldcg(src + i * 128) : 0.0f;
                            }
#pragma unroll
                            for (int h = 0; h < kQ; ++h)
#pragma unroll
                                for (int i = 0; i < WC; ++i) acc[i] += got[h][i];
                        }
                    }
                    // (ctl->last is not written again before every thread has passed this piece's
                    // barriers and reached the next piece's first one)
                }
            }
            if (!finish) continue;

            if constexpr (kSwap) {
                // lane_row is D's column n, the MMA columns are D's rows: 32 lanes store
                // consecutive columns of one row
                const int n = w.n0 + lane_row;
                if (n < p.N) {
                    const float bv = p.bias ? load_elem(p.bias, p.bias_f32, n) : 0.0f;
#pragma unroll
                    for (int i = 0; i < WC; ++i) {
                        float v = acc[i];
                        const int m = w.m0 + i;
                        if (m < w.m_end) {
                            const long long row = static_cast<long long>(w.d_row) + m;
                            if (p.beta != 0.0f) v = fmaf(p.beta, load_elem(p.C, p.c_f32, row * p.ldc + n), v);
                            v = apply_act(p.act, v + bv);
                            if (p.d_f32) static_cast<float*>(p.D)[row * p.ldd + n] = v;
                            else static_cast<__nv_bfloat16*>(p.D)[row * p.ldd + n] = __float2bfloat16_rn(v);
                        }
                    }
                }
            } else {
                const int warp_row = w.m0 + static_cast<int>(rank) * 128 + quad * 32;
                const int rows_ok = min(32, w.m_end - warp_row);
                if (rows_ok > 0) {
                    const long long row = static_cast<long long>(w.d_row) + warp_row + lane;
#pragma unroll
                    for (int j = 0; j < WC / kOut; ++j) {
                        const int col0 = w.n0 + col_base + j * kOut;
                        if (col0 < p.N) {
                            float v[kOut];
#pragma unroll
                            for (int i = 0; i < kOut; ++i) v[i] = acc[j * kOut + i];
                            finish_values<kOut>(p, v, row, col0, rows_ok, lane, bias_cols + j * kOut, my_words);
                            store_values<kOut>(p, v, row, col0, rows_ok, lane, my_words);
                        }
                    }
                }
            }
        }
    }

    ptx::tc_fence_before_sync();
    if constexpr (kPair) ptx::cluster_sync();   // the leader's MMAs into the peer's TMEM are done
    else __syncthreads();
    if (warp == 1) {
        __syncwarp();
        ptx::tc_fence_after_sync();
        if constexpr (kPair) ptx::tmem_dealloc_pair(tmem_base, S::kTmemCols);
        else ptx::tmem_dealloc(tmem_base, S::kTmemCols);
    }
}

}  // namespace b128
}  // namespace tcg
