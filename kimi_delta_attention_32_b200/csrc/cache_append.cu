// cache_append.cu -- new tokens' keys and values into the paged cache of the softmax-attention
// layers (m.lqnn.cn/news/205170, section "KDA 与 Gated Attention：每 4 层只留 1 层全注意力").
//
// Token i of sequence n goes to slot seqlens[n] + i of its block table; the entry's gathered
// weight becomes 0 and its position positions[n] + i. A copy, bound by HBM: each row is read and
// written once. The place of a token takes a chain of dependent loads (its sequence, the length,
// the page number), so a block first finds the places of all its tokens, a thread each, and then
// copies them, a warp a token with eight 16-byte loads a lane in flight.
#include "paged.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256, kMostTokens = 16;

template <int kPieces>      // 16-byte pieces of a row
__global__ void __launch_bounds__(kThreads) cache_append_kernel(const AppendArgs a, int tokens, int esz) {
    __shared__ int64_t s_off[kMostTokens], s_side[kMostTokens];    // -1: not written
    __shared__ int s_pos[kMostTokens];
    const int64_t t0 = (int64_t)blockIdx.x * tokens;
    const int count = (int)min((int64_t)tokens, a.T_tot - t0);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool side = a.acc != nullptr || a.pos != nullptr;
    if (tid < count) {
        const int64_t t = t0 + tid;
        int64_t n, i;
        if (a.cu != nullptr) {
            n = find_seq(a.cu, a.N, t);
            i = t - __ldg(a.cu + n);
        } else {
            n = t / a.T_pad;
            i = t - n * a.T_pad;
        }
        const int len = __ldg(a.seqlens + n);
        const int64_t slot = len + i;
        const int seen = __ldg(a.positions + n);
        int64_t off = -1;
        if (len < 0 || slot >= (int64_t)a.c.max_pages * a.c.page_size || (side && slot >= a.slots))
            atomicOr(a.c.err, kErrIndex);
        else
            off = slot_offset(a.c, n, (int)slot);
        s_off[tid] = off < 0 ? -1 : off * esz;
        s_side[tid] = n * a.H * a.slots + slot;
        s_pos[tid] = seen + (int)i;
    }
    __syncthreads();
    const int row_pieces = a.H * kPieces;
    const int64_t head_bytes = a.c.head_stride * esz;
    for (int u = warp; u < count; u += kThreads / 32) {
        if (s_off[u] < 0) continue;
        const uint4* k = static_cast<const uint4*>(a.k) + (t0 + u) * row_pieces;
        const uint4* v = static_cast<const uint4*>(a.v) + (t0 + u) * row_pieces;
        char* kc = static_cast<char*>(a.c.k) + s_off[u];
        char* vc = static_cast<char*>(a.c.v) + s_off[u];
        for (int e0 = lane; e0 < row_pieces; e0 += 128) {
            uint4 x[4], y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (e0 + 32 * j < row_pieces) {
                    x[j] = __ldcs(k + e0 + 32 * j);
                    y[j] = __ldcs(v + e0 + 32 * j);
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int e = e0 + 32 * j;
                if (e < row_pieces) {
                    const int64_t to = e / kPieces * head_bytes + e % kPieces * 16;
                    *reinterpret_cast<uint4*>(kc + to) = x[j];
                    *reinterpret_cast<uint4*>(vc + to) = y[j];
                }
            }
        }
    }
    if (!side) return;
    // consecutive threads take consecutive tokens, whose entries lie side by side
    for (int e = tid; e < count * a.H; e += kThreads) {
        const int u = e % count, h = e / count;
        if (s_off[u] < 0) continue;
        const int64_t at = s_side[u] + (int64_t)h * a.slots;
        if (a.acc != nullptr) a.acc[at] = 0.f;
        if (a.pos != nullptr) a.pos[at] = s_pos[u];
    }
}

}  // namespace

cudaError_t launch_cache_append(const AppendArgs& a, cudaStream_t stream) {
    if (a.T_tot == 0) return cudaSuccess;
    const int sms = sm_count();
    if (sms == 0) return cudaErrorInvalidDevice;
    // few tokens (a decode step) are spread over the GPU, many share a block's chain of lookups
    int64_t tokens = a.T_tot / (4 * sms);
    tokens = tokens < 1 ? 1 : tokens > kMostTokens ? kMostTokens : tokens;
    const unsigned grid = (unsigned)((a.T_tot + tokens - 1) / tokens);
    const int esz = a.io == Io::BF16 ? 2 : 4;
    switch (a.d * esz / 16) {
        case 8: cache_append_kernel<8><<<grid, kThreads, 0, stream>>>(a, (int)tokens, esz); break;
        case 16: cache_append_kernel<16><<<grid, kThreads, 0, stream>>>(a, (int)tokens, esz); break;
        case 32: cache_append_kernel<32><<<grid, kThreads, 0, stream>>>(a, (int)tokens, esz); break;
        default: return cudaErrorInvalidValue;
    }
    return cudaGetLastError();
}

}  // namespace kda
