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

// Block c takes the tiles [split_begin(c), split_begin(c + 1)): contiguous, sizes differ by one
// at most. W * C stays below 2^63: C is a few hundred.
KDA_HD int64_t split_begin(int64_t W, int C, int c) { return W * c / C; }

// The block whose range holds tile t: the largest c with W c / C < t + 1.
KDA_HD int split_block_of(int64_t W, int C, int64_t t) { return (int)(((t + 1) * C - 1) / W); }

}  // namespace kda
