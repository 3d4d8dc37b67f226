// even_cut.cuh -- a line of work in equal contiguous parts.
#pragma once

#include <stdint.h>

namespace pkv {

// a / b for a >= 0: a 64-bit division takes hundreds of cycles, and lines are
// short of 2^32 nearly always.
__device__ __forceinline__ long long quotient(long long a, int b) {
    return a >> 32 ? a / b : (long long)((uint32_t)a / (uint32_t)b);
}

// A line of cost `total` in equal parts, the first ones longer by one.
struct EvenCut {
    long long q;
    int r;
    __device__ __forceinline__ EvenCut(long long total, int parts) : q(quotient(total, parts)), r((int)(total - q * parts)) {}
    __device__ __forceinline__ long long begin(int i) const { return q * i + min(i, r); }
    __device__ __forceinline__ int part_of(long long y) const {
        const long long y1 = (q + 1) * r;
        return y < y1 ? (int)quotient(y, (int)(q + 1)) : r + (int)quotient(y - y1, (int)q);
    }
};

}  // namespace pkv
