// split.cuh -- where the pieces of a run start: of a sort's assignments among CTAs
// and warps, of a sum's K among accumulations and workers.
#pragma once

#include <cuda_runtime.h>

namespace tcg {

// Piece `part` of `parts` is [run_start(part), run_start(part + 1)); the product of
// two ints needs 64 bits.
__host__ __device__ __forceinline__ int run_start(int total, int part, int parts) {
    return static_cast<int>(static_cast<long long>(total) * part / parts);
}

// The same pieces in their order, over and over, without a division each (64-bit
// ones stand in an MMA issuer's way: forward of 8192 x 100000 x 512 473 us, 448
// this way).  floor(total p / parts) goes up by total / parts, and by one more
// where the remainders add up to parts.
struct Pieces {
    int total, parts, each, rest;
    int begin = 0, end = 0, owed = 0;

    __host__ __device__ __forceinline__ Pieces(int n, int count) : total(n), parts(count), each(n / count), rest(n % count) {}
    __host__ __device__ __forceinline__ void next() {
        if (end == total) end = owed = 0;
        begin = end;
        end += each;
        owed += rest;
        if (owed >= parts) {
            owed -= parts;
            ++end;
        }
    }
};

}  // namespace tcg
