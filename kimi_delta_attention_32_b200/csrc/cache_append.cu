// cache_append.cu -- new tokens' keys and values into the paged cache of the softmax-attention
// layers (m.lqnn.cn/news/205170, section "KDA 与 Gated Attention：每 4 层只留 1 层全注意力").
//
// Token i of sequence n goes to slot seqlens[n] + i of its block table; the entry's gathered
// weight becomes 0 and its position positions[n] + i. A copy: each row is read and written once.
#include "paged.cuh"

namespace kda {
namespace {

// One CTA per token.
__global__ void cache_append_kernel(const AppendArgs a, int row16) {
    const int64_t t = blockIdx.x;
    int64_t n, i;
    if (a.cu != nullptr) {
        n = find_seq(a.cu, a.N, t);
        i = t - a.cu[n];
    } else {
        n = t / a.T_pad;
        i = t % a.T_pad;
    }
    const int64_t room = (int64_t)a.c.max_pages * a.c.page_size;
    const int64_t slot = a.seqlens[n] + i;
    const bool side = a.acc != nullptr || a.pos != nullptr;
    if (a.seqlens[n] < 0 || slot >= room || (side && slot >= a.slots)) {
        if (threadIdx.x == 0) atomicOr(a.c.err, kErrIndex);
        return;
    }
    const int64_t off = slot_offset(a.c, n, (int)slot);
    if (off < 0) return;
    const int64_t esz = a.io == Io::BF16 ? 2 : 4;
    for (int e = threadIdx.x; e < a.H * row16; e += blockDim.x) {
        const int h = e / row16, c = e % row16;
        const int64_t to = (off + h * a.c.head_stride) * esz + c * 16;
        const int64_t from = (t * a.H + h) * row16 + c;
        *reinterpret_cast<uint4*>(static_cast<char*>(a.c.k) + to) = static_cast<const uint4*>(a.k)[from];
        *reinterpret_cast<uint4*>(static_cast<char*>(a.c.v) + to) = static_cast<const uint4*>(a.v)[from];
        if (c == 0) {
            const int64_t at = (n * a.H + h) * a.slots + slot;
            if (a.acc != nullptr) a.acc[at] = 0.f;
            if (a.pos != nullptr) a.pos[at] = a.positions[n] + (int)i;
        }
    }
}

}  // namespace

cudaError_t launch_cache_append(const AppendArgs& a, cudaStream_t stream) {
    if (a.T_tot == 0) return cudaSuccess;
    const int row16 = a.d * (a.io == Io::BF16 ? 2 : 4) / 16;
    cache_append_kernel<<<(unsigned)a.T_tot, 128, 0, stream>>>(a, row16);
    return cudaGetLastError();
}

}  // namespace kda
