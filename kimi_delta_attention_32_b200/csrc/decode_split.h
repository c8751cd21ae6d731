// decode_split.h -- how paged_decode.cu divides its work: W equal tiles, in order, over C blocks.
// Plain C++ (host and device), so that the arithmetic can be checked away from a GPU.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define KDA_HD __host__ __device__ __forceinline__
#else
#define KDA_HD inline
#endif

namespace kda {

// Blocks that get work: never more than tiles, so that each has at least one.
KDA_HD int split_blocks(int64_t W, int most) { return W < most ? (int)W : most; }

// a / b for a >= 0, b > 0: in 32 bits where they hold a, as they nearly always do (a 64-bit division
// takes some hundred cycles on the device).
KDA_HD int64_t split_div(int64_t a, int64_t b) {
    return (a >> 31) == 0 && (b >> 31) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// Block c takes the tiles [split_begin(c), split_begin(c + 1)): contiguous, sizes differ by one
// at most. floor(W c / C), from W = q C + r. C is a few hundred.
KDA_HD int64_t split_begin(int64_t W, int C, int c) {
    const int64_t q = split_div(W, C);
    const int r = (int)(W - q * C);
    return q * c + (int)((uint32_t)(r * c) / (uint32_t)C);
}

// The block whose range holds tile t: the largest c with W c / C < t + 1.
KDA_HD int split_block_of(int64_t W, int C, int64_t t) { return (int)split_div((t + 1) * C - 1, W); }

}  // namespace kda
