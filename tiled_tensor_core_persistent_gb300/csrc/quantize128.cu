// quantize128.cu -- 8-bit codes and fp32 scales per block of 128, in the three
// forms the block-scaled products read:
//
//   s = max(amax, 2^-96) / top        (times fl(1 / top); top = 448 or 57344;
//                                      optionally rounded up to a power of two)
//   q = rn8(clamp(x * fl(1 / s)))
//
// rows: a block is 128 consecutive elements of a row; cols: 128 rows of one
// column, written transposed; tiles: 128 x 128, with an optional transposed
// copy.  The arithmetic is fp32 with one rounding to 8 bits at the end, so
// the codes are the same whatever the variant or the launch shape.
//
// All three are bound by memory: x is read once, the codes written once, and
// the amax needs only the registers (rows), or one pass through shared memory
// (cols and tiles, whose transposed codes turn there too).  32768 x 4096 bf16
// rows gathered from 16384: 53 us, 5.1 TB/s of what must move; 20011 x 4104 by
// columns: 51 us, 5.1 TB/s; 16 x 4096 x 4096 in tiles with the transposed copy:
// 169 us, 6.4 TB/s, 94 % of the copy rate.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <climits>
#include <cstdint>
#include <type_traits>

#include "groups.cuh"
#include "host.h"

namespace {

constexpr float kTiny = 0x1p-96f;   // keeps the scale and its reciprocal finite on a block of zeros
constexpr int kMaxGroups = 1024;

struct Quant {
    const void* x;
    long long ldx;
    int rows, cols;
    const int* index;      // rows of x to take, or NULL
    int source;            // rows of x that index may name
    uint8_t* q;
    long long ldq;
    uint8_t* qt;           // tiles: transposed copy, or NULL
    long long ldqt;
    float* scales;
    long long lds;
    float inv_top;
    int pow2;
    int e5m2;
    int vec;               // x may be read, q written, in whole vectors
    const int* offsets;
    int groups;
};

__device__ __forceinline__ float scale_of(const Quant& p, float amax) {
    const float s = fmaxf(amax, kTiny) * p.inv_top;
    if (!p.pow2) return s;
    return __uint_as_float((__float_as_uint(s) + 0x7FFFFFu) & 0x7F800000u);
}

// Two values to two 8-bit codes, round to nearest even, saturating; NaN stays NaN.
template <bool kE5m2>
__device__ __forceinline__ uint32_t code2(float lo, float hi) {
    uint16_t r;
    if constexpr (kE5m2) asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
template <bool kE5m2>
__device__ __forceinline__ uint32_t code4(float a, float b, float c, float d) {
    return code2<kE5m2>(a, b) | (code2<kE5m2>(c, d) << 16);
}

// N elements as they are stored: 16-bit types stay packed in pairs, which
// halves the registers of a load in flight and the steps of an amax.
template <typename T, int N>
struct Raw {
    static constexpr int kPer = 4 / static_cast<int>(sizeof(T));   // elements per word
    static constexpr int kWords = N / kPer;
    uint32_t w[kWords];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0u;
    }
    __device__ __forceinline__ float at(int i) const;
};
template <typename T>
__device__ __forceinline__ float widen(uint32_t word, int i);   // element i of a word
template <>
__device__ __forceinline__ float widen<__nv_bfloat16>(uint32_t word, int i) {
    return __uint_as_float(i ? word & 0xFFFF0000u : word << 16);
}
template <>
__device__ __forceinline__ float widen<__half>(uint32_t word, int i) {
    return __half2float(__ushort_as_half(static_cast<unsigned short>(i ? word >> 16 : word & 0xFFFFu)));
}
template <>
__device__ __forceinline__ float widen<float>(uint32_t word, int) { return __uint_as_float(word); }
template <typename T, int N>
__device__ __forceinline__ float Raw<T, N>::at(int i) const { return widen<T>(w[i / kPer], i % kPer); }

// Element-wise largest magnitude of two words; NaN is ignored.
template <typename T>
__device__ __forceinline__ uint32_t amax_word(uint32_t a, uint32_t b);
template <>
__device__ __forceinline__ uint32_t amax_word<__nv_bfloat16>(uint32_t a, uint32_t b) {
    b &= 0x7FFF7FFFu;
    const __nv_bfloat162 m = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&m);
}
template <>
__device__ __forceinline__ uint32_t amax_word<__half>(uint32_t a, uint32_t b) {
    b &= 0x7FFF7FFFu;
    const __half2 m = __hmax2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&m);
}
template <>
__device__ __forceinline__ uint32_t amax_word<float>(uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), fabsf(__uint_as_float(b))));
}
template <typename T>
__device__ __forceinline__ float amax_of(uint32_t word) {   // the larger element of a word
    return sizeof(T) == 4 ? widen<T>(word, 0) : fmaxf(widen<T>(word, 0), widen<T>(word, 1));
}

// Elements [i, i + N) of a row of x, zeros past its end.
template <typename T, int N>
__device__ __forceinline__ void load_some(const Quant& p, long long row_at, int i, Raw<T, N>& v) {
    using R = Raw<T, N>;
    const T* src = static_cast<const T*>(p.x) + row_at + i;
    if (p.vec && i + N <= p.cols) {
#pragma unroll
        for (int k = 0; k < R::kWords / 4; ++k) {
            const uint4 q = __ldg(reinterpret_cast<const uint4*>(src) + k);
            v.w[4 * k] = q.x;
            v.w[4 * k + 1] = q.y;
            v.w[4 * k + 2] = q.z;
            v.w[4 * k + 3] = q.w;
        }
    } else {
#pragma unroll
        for (int k = 0; k < R::kWords; ++k) {
            uint32_t word = 0u;
            if constexpr (sizeof(T) == 4) {
                if (i + k < p.cols) word = __ldg(reinterpret_cast<const uint32_t*>(src) + k);
            } else {
                const unsigned short* s16 = reinterpret_cast<const unsigned short*>(src);
                if (i + 2 * k < p.cols) word = __ldg(s16 + 2 * k);
                if (i + 2 * k + 1 < p.cols) word |= static_cast<uint32_t>(__ldg(s16 + 2 * k + 1)) << 16;
            }
            v.w[k] = word;
        }
    }
}

// The row of x that output row r takes, or -1 (a row of zeros).
__device__ __forceinline__ int source_row(const Quant& p, int r) {
    if (!p.index) return r;
    const int s = __ldg(p.index + r);
    return s >= 0 && s < p.source ? s : -1;
}

// ------------------------------------------------------------------------ rows
//
// Eight lanes hold a block (16 elements each), a warp four rows of one block
// column, a CTA 32 rows: the scales of a CTA are one 128-byte line.  kU blocks
// along the row per warp keep that many loads in flight.  The codes are stored
// to leave the L2 first: rows gathered twice then find more of x there (32768 x
// 4096 from 16384 rows: 61.4 -> 55.3 us with kU = 2, 61.3 with kU = 4; without
// the hint 61.4 either way).
template <typename T, int kU, bool kE5m2>
__global__ void __launch_bounds__(256) rows_kernel(const __grid_constant__ Quant p) {
    tcg::host::wait_for_kernel_ahead();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r = blockIdx.y * 32 + warp * 4 + (lane >> 3);
    const int kb0 = blockIdx.x * kU;
    if (r >= p.rows) return;
    const unsigned peers = 0xFFu << (lane & 24);
    const int src = source_row(p, r);
    const long long at = src * p.ldx;
    const int blocks = (p.cols + 127) >> 7;
    Raw<T, 16> v[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        if (src >= 0 && kb0 + u < blocks) load_some<T, 16>(p, at, (kb0 + u) * 128 + (lane & 7) * 16, v[u]);
        else v[u].zero();
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        if (kb0 + u >= blocks) break;
        uint32_t m = 0u;
#pragma unroll
        for (int k = 0; k < Raw<T, 16>::kWords; ++k) m = amax_word<T>(m, v[u].w[k]);
        float a = amax_of<T>(m);
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) a = fmaxf(a, __shfl_xor_sync(peers, a, d));
        const float s = scale_of(p, a);
        const float inv = 1.0f / s;
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            w[k] = code4<kE5m2>(v[u].at(4 * k) * inv, v[u].at(4 * k + 1) * inv, v[u].at(4 * k + 2) * inv, v[u].at(4 * k + 3) * inv);
        const int c = (kb0 + u) * 128 + (lane & 7) * 16;
        uint8_t* dst = p.q + r * p.ldq + c;
        if (p.vec && c + 16 <= p.cols) {
            __stcs(reinterpret_cast<uint4*>(dst), make_uint4(w[0], w[1], w[2], w[3]));
        } else {
#pragma unroll
            for (int k = 0; k < 16; ++k)
                if (c + k < p.cols) dst[k] = static_cast<uint8_t>(w[k / 4] >> (8 * (k % 4)));
        }
        if ((lane & 7) == 0) p.scales[(kb0 + u) * p.lds + r] = s;
    }
}

// A 128 x 128 tile of codes turning in shared memory, as words of four rows of
// one column.  Thread (cg, rg) of 16 x 16 holds columns 8 cg .. 8 cg + 7 of rows
// 8 rg .. 8 rg + 7; the words of a column are rotated by turn(cg), which puts
// the 32 words that a warp writes at once into 32 banks (and a column's words,
// read together, stay in 32 banks too).
__device__ __forceinline__ int turn(int cg) { return ((cg >> 1) << 2) | (cg & 1); }

template <bool kE5m2>
__device__ __forceinline__ void put_words(uint32_t* words, int cg, int rg, int k, const float (&v)[8]) {
    uint32_t* col = words + (cg * 8 + k) * 32;
    col[(2 * rg + turn(cg)) & 31] = code4<kE5m2>(v[0], v[1], v[2], v[3]);
    col[(2 * rg + 1 + turn(cg)) & 31] = code4<kE5m2>(v[4], v[5], v[6], v[7]);
}

// Rows [r, r + n) of the transposed tile (n of its 128 columns) to 128-byte lines.
__device__ __forceinline__ void write_columns(const uint32_t* words, uint8_t* dst, long long ld, int cols, int rows, int warp,
                                              int lane) {
    const bool whole = ld % 4 == 0 && reinterpret_cast<uintptr_t>(dst) % 4 == 0 && 4 * lane + 4 <= rows;
#pragma unroll 4
    for (int c = warp; c < cols; c += 8) {
        const uint32_t w = words[c * 32 + ((lane + turn(c >> 3)) & 31)];
        uint8_t* at = dst + c * ld + 4 * lane;
        if (whole) {
            *reinterpret_cast<uint32_t*>(at) = w;
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (4 * lane + k < rows) at[k] = static_cast<uint8_t>(w >> (8 * k));
        }
    }
}

// ------------------------------------------------------------------------ cols
//
// One CTA: the 128 rows of one block row, 128 columns.  The amax of a column
// goes over a thread's eight rows, two lanes and eight warps.

// The first row and the rows of padded block b: the groups' blocks one after
// the other, each group's last block partly empty.  One warp; the same for
// all its lanes.
__device__ __forceinline__ void find_block(const Quant& p, int b, int lane, int& row, int& n) {
    if (!p.offsets) {
        row = b * 128;
        n = min(128, p.rows - row);
        return;
    }
    int base = 0, last = 0;
    row = 0;
    n = 0;
    for (int g0 = 0; g0 < p.groups; g0 += 32) {
        int r, len;
        tcg::group_rows(p.offsets, p.groups, p.rows, g0, lane, last, r, len);
        const int blocks = (len + 127) >> 7;
        int incl = blocks;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += o;
        }
        const int first = base + incl - blocks;
        const unsigned hit = __ballot_sync(0xffffffffu, b >= first && b < first + blocks);
        if (hit) {
            const int who = __ffs(hit) - 1;
            const int in = (b - __shfl_sync(0xffffffffu, first, who)) * 128;
            row = __shfl_sync(0xffffffffu, r, who) + in;
            n = min(128, __shfl_sync(0xffffffffu, len, who) - in);
            return;
        }
        base += __shfl_sync(0xffffffffu, incl, 31);
    }
}

template <typename T, bool kE5m2>
__global__ void __launch_bounds__(256) cols_kernel(const __grid_constant__ Quant p) {
    using R = Raw<T, 8>;
    __shared__ float part[8][128];
    __shared__ float inv_s[128];
    __shared__ uint32_t words[128 * 32];
    tcg::host::wait_for_kernel_ahead();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int block = blockIdx.y, c0 = blockIdx.x * 128;
    int row, n;
    find_block(p, block, lane, row, n);
    const int cg = threadIdx.x & 15, rg = threadIdx.x >> 4;
    R v[8];
    uint32_t m[R::kWords];
#pragma unroll
    for (int k = 0; k < R::kWords; ++k) m[k] = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = rg * 8 + i;
        const int src = r < n ? source_row(p, row + r) : -1;
        if (src >= 0) load_some<T, 8>(p, src * p.ldx, c0 + cg * 8, v[i]);
        else v[i].zero();
    }
#pragma unroll
    for (int k = 0; k < R::kWords; ++k) {
#pragma unroll
        for (int i = 0; i < 8; ++i) m[k] = amax_word<T>(m[k], v[i].w[k]);
        m[k] = amax_word<T>(m[k], __shfl_xor_sync(0xffffffffu, m[k], 16));
        if (lane < 16) {
#pragma unroll
            for (int e = 0; e < R::kPer; ++e) part[warp][cg * 8 + k * R::kPer + e] = widen<T>(m[k], e);
        }
    }
    __syncthreads();
    if (threadIdx.x < 128) {
        float a = part[0][threadIdx.x];
#pragma unroll
        for (int i = 1; i < 8; ++i) a = fmaxf(a, part[i][threadIdx.x]);
        const float s = scale_of(p, a);
        inv_s[threadIdx.x] = 1.0f / s;
        const int c = c0 + threadIdx.x;
        if (c < p.cols) p.scales[block * p.lds + c] = s;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float inv = inv_s[cg * 8 + k];
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = v[i].at(k) * inv;
        put_words<kE5m2>(words, cg, rg, k, x);
    }
    __syncthreads();
    write_columns(words, p.q + c0 * p.ldq + block * 128LL, p.ldq, min(128, p.cols - c0), 128, warp, lane);
}

// ----------------------------------------------------------------------- tiles
//
// One CTA: one 128 x 128 tile of one matrix of the batch (matrix b is rows
// [b rows, (b + 1) rows) of x).  The row-major codes leave from registers,
// eight bytes a row and 128 a half warp, the transposed ones through shared
// memory.
template <typename T, bool kE5m2>
__global__ void __launch_bounds__(256) tiles_kernel(const __grid_constant__ Quant p) {
    using R = Raw<T, 8>;
    __shared__ float part[8];
    __shared__ uint32_t words[128 * 32];
    tcg::host::wait_for_kernel_ahead();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int b = blockIdx.z, r0 = blockIdx.y * 128, c0 = blockIdx.x * 128;
    const int cg = threadIdx.x & 15, rg = threadIdx.x >> 4;
    R v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = r0 + rg * 8 + i;
        if (r < p.rows) load_some<T, 8>(p, (static_cast<long long>(b) * p.rows + r) * p.ldx, c0 + cg * 8, v[i]);
        else v[i].zero();
    }
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int k = 0; k < R::kWords; ++k) m = amax_word<T>(m, v[i].w[k]);
    float a = amax_of<T>(m);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, d));
    if (lane == 0) part[warp] = a;
    __syncthreads();
    a = part[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) a = fmaxf(a, part[i]);
    const float s = scale_of(p, a);
    const float inv = 1.0f / s;
    if (threadIdx.x == 0)
        p.scales[(static_cast<long long>(b) * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x] = s;
    if (p.q) {
        const int c = c0 + cg * 8;
        const bool whole = p.ldq % 8 == 0 && reinterpret_cast<uintptr_t>(p.q) % 8 == 0 && c + 8 <= p.cols;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = r0 + rg * 8 + i;
            if (r >= p.rows) continue;
            uint8_t* dst = p.q + (static_cast<long long>(b) * p.rows + r) * p.ldq + c;
            const uint2 w = make_uint2(code4<kE5m2>(v[i].at(0) * inv, v[i].at(1) * inv, v[i].at(2) * inv, v[i].at(3) * inv),
                                       code4<kE5m2>(v[i].at(4) * inv, v[i].at(5) * inv, v[i].at(6) * inv, v[i].at(7) * inv));
            if (whole) {
                *reinterpret_cast<uint2*>(dst) = w;
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (c + k < p.cols) dst[k] = static_cast<uint8_t>((k < 4 ? w.x : w.y) >> (8 * (k & 3)));
            }
        }
    }
    if (!p.qt) return;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = v[i].at(k) * inv;
        put_words<kE5m2>(words, cg, rg, k, x);
    }
    __syncthreads();
    write_columns(words, p.qt + (static_cast<long long>(b) * p.cols + c0) * p.ldqt + r0, p.ldqt, min(128, p.cols - c0),
                  min(128, p.rows - r0), warp, lane);
}

// ------------------------------------------------------------------------ host

int x_bytes(tcg_dtype t) { return t == TCG_F32 ? 4 : 2; }
bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// The rules the three forms share; fills everything but the outputs' shapes.
tcg_status start(Quant& p, int rows, int cols, tcg_dtype x_dtype, const void* x, int ldx, tcg_dtype q_dtype,
                 float* scales, int pow2, const int* index, int source) {
    if (rows < 0 || cols < 0 || source < 0) return TCG_ERR_INVALID_ARG;
    if (x_dtype != TCG_BF16 && x_dtype != TCG_F16 && x_dtype != TCG_F32) return TCG_ERR_INVALID_ARG;
    if (q_dtype != TCG_E4M3 && q_dtype != TCG_E5M2) return TCG_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return TCG_OK;
    if (std::max(rows, cols) > tcg::host::kMaxExtent) return TCG_ERR_UNSUPPORTED;
    if ((!x && !(index && source == 0)) || !scales || ldx < cols) return TCG_ERR_INVALID_ARG;
    if (!aligned(x, x_bytes(x_dtype)) || !aligned(scales, 4) || !aligned(index, 4)) return TCG_ERR_MISALIGNED;
    p.x = x;
    p.ldx = ldx;
    p.rows = rows;
    p.cols = cols;
    p.index = index;
    p.source = source;
    p.scales = scales;
    p.inv_top = 1.0f / (q_dtype == TCG_E5M2 ? 57344.0f : 448.0f);
    p.pow2 = pow2 != 0;
    p.e5m2 = q_dtype == TCG_E5M2;
    p.vec = aligned(x, 16) && (static_cast<long long>(ldx) * x_bytes(x_dtype)) % 16 == 0;
    return TCG_OK;
}

tcg_status launched(cudaError_t e, const char* what) { return e == cudaSuccess ? TCG_OK : tcg::host::fail_launch(what, e); }

// f(element type, whether the codes are e5m2) for the types of a call
template <typename F>
void with_types(tcg_dtype x, bool e5m2, F f) {
    auto go = [&](auto element) {
        if (e5m2) f(element, std::true_type{});
        else f(element, std::false_type{});
    };
    if (x == TCG_BF16) go(__nv_bfloat16{});
    else if (x == TCG_F16) go(__half{});
    else go(float{});
}

}  // namespace

extern "C" {

tcg_status tcg_quantize_rows128(int rows, int cols, tcg_dtype x_dtype, const void* x, int ldx, const int* row_index,
                                int source_rows, void* q, int ldq, tcg_dtype q_dtype, float* scales, int ld_scales,
                                int pow2, void* stream) {
    Quant p = {};
    tcg_status st = start(p, rows, cols, x_dtype, x, ldx, q_dtype, scales, pow2, row_index, source_rows);
    if (st != TCG_OK || rows == 0 || cols == 0) return st;
    if (!q || ldq < cols || ld_scales < rows) return TCG_ERR_INVALID_ARG;
    tcg::host::Device dev;
    if ((st = tcg::host::device(dev)) != TCG_OK) return st;
    p.q = static_cast<uint8_t*>(q);
    p.ldq = ldq;
    p.lds = ld_scales;
    p.vec = p.vec && aligned(q, 16) && ldq % 16 == 0;
    const int blocks = (cols + 127) / 128, row_ctas = (rows + 31) / 32;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t err = cudaSuccess;
    for (int done = 0; done < row_ctas && err == cudaSuccess; done += 65535) {   // gridDim.y's limit
        const int n = std::min(row_ctas - done, 65535);
        Quant part = p;
        const long long first = static_cast<long long>(done) * 32;
        part.rows = static_cast<int>(std::min<long long>(rows - first, static_cast<long long>(n) * 32));
        if (p.index) part.index = p.index + first;
        else part.x = static_cast<const char*>(p.x) + first * ldx * x_bytes(x_dtype);
        part.q = p.q + first * ldq;
        part.scales = p.scales + first;
        // two blocks per warp once that still gives every SM several CTAs
        if (static_cast<long long>(n) * ((blocks + 1) / 2) >= 4LL * dev.num_sms)
            with_types(x_dtype, p.e5m2, [&](auto x0, auto e) {
                err = tcg::host::launch_early(rows_kernel<decltype(x0), 2, decltype(e)::value>, dim3((blocks + 1) / 2, n), 256, s, part);
            });
        else
            with_types(x_dtype, p.e5m2, [&](auto x0, auto e) {
                err = tcg::host::launch_early(rows_kernel<decltype(x0), 1, decltype(e)::value>, dim3(blocks, n), 256, s, part);
            });
    }
    return launched(err, "tcg_quantize_rows128");
}

tcg_status tcg_quantize_cols128(int rows, int cols, tcg_dtype x_dtype, const void* x, int ldx, const int* row_index,
                                int source_rows, int num_groups, const int* offsets, int padded_rows, void* q,
                                int ldq, tcg_dtype q_dtype, float* scales, int ld_scales, int pow2, void* stream) {
    Quant p = {};
    if (padded_rows < 0 || padded_rows % 128 || num_groups < 0) return TCG_ERR_INVALID_ARG;
    if (num_groups > kMaxGroups || padded_rows / 128 > 65535) return TCG_ERR_UNSUPPORTED;
    if (padded_rows == 0 || cols == 0) return rows < 0 || cols < 0 ? TCG_ERR_INVALID_ARG : TCG_OK;
    // (no rows at all still writes the padding)
    tcg_status st = start(p, rows > 0 ? rows : rows == 0 ? 1 : -1, cols, x_dtype, rows == 0 ? scales : x, rows == 0 ? INT_MAX : ldx,
                          q_dtype, scales, pow2, row_index, source_rows);
    if (st != TCG_OK) return st;
    p.rows = rows;
    if (!q || ldq < padded_rows || ld_scales < cols) return TCG_ERR_INVALID_ARG;
    if (offsets ? num_groups == 0 : num_groups > 1) return TCG_ERR_INVALID_ARG;
    if (!offsets && padded_rows < rows) return TCG_ERR_INVALID_ARG;
    if (!aligned(offsets, 4)) return TCG_ERR_MISALIGNED;
    tcg::host::Device dev;
    if ((st = tcg::host::device(dev)) != TCG_OK) return st;
    p.q = static_cast<uint8_t*>(q);
    p.ldq = ldq;
    p.lds = ld_scales;
    p.offsets = offsets;
    p.groups = num_groups;
    const int row_blocks = padded_rows / 128;
    const dim3 grid((cols + 127) / 128, row_blocks);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t err = cudaSuccess;
    with_types(x_dtype, p.e5m2, [&](auto x0, auto e) { err = tcg::host::launch_early(cols_kernel<decltype(x0), decltype(e)::value>, grid, 256, s, p); });
    return launched(err, "tcg_quantize_cols128");
}

tcg_status tcg_quantize_tiles128(int batch, int rows, int cols, tcg_dtype x_dtype, const void* x, int ldx, void* q,
                                 int ldq, void* qt, int ldqt, tcg_dtype q_dtype, float* scales, int pow2,
                                 void* stream) {
    Quant p = {};
    if (batch < 0) return TCG_ERR_INVALID_ARG;
    tcg_status st = start(p, rows, cols, x_dtype, x, ldx, q_dtype, scales, pow2, nullptr, 0);
    if (st != TCG_OK || rows == 0 || cols == 0 || batch == 0) return st;
    if ((!q && !qt) || (q && ldq < cols) || (qt && ldqt < rows)) return TCG_ERR_INVALID_ARG;
    if (batch > 65535 || (rows + 127) / 128 > 65535) return TCG_ERR_UNSUPPORTED;
    tcg::host::Device dev;
    if ((st = tcg::host::device(dev)) != TCG_OK) return st;
    p.q = static_cast<uint8_t*>(q);
    p.ldq = ldq;
    p.qt = static_cast<uint8_t*>(qt);
    p.ldqt = ldqt;
    const dim3 grid((cols + 127) / 128, (rows + 127) / 128, batch);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t err = cudaSuccess;
    with_types(x_dtype, p.e5m2, [&](auto x0, auto e) { err = tcg::host::launch_early(tiles_kernel<decltype(x0), decltype(e)::value>, grid, 256, s, p); });
    return launched(err, "tcg_quantize_tiles128");
}

}  // extern "C"
