// cache_evict.cu -- cuts every (sequence, key-value head) of the paged cache to a budget of
// entries, by the attention weight that they have gathered. (The softmax-attention layers are the
// only ones whose cache grows with the context: m.lqnn.cn/news/205170, section "KDA 与 Gated
// Attention：每 4 层只留 1 层全注意力". The pages have no eviction.)
//
// Entries rank by a 32-bit key: guarded ones first, then larger acc; equal keys by slot. The keep
// best stay. Those behind slot keep move into the free slots before it, both in slot order: the
// number of rows that move is the number that are evicted below keep, however long the cache.
#include "paged.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;

// Rank key of an entry: order-preserving bits of the fp32 weight (NaN lowest, -0 equal to 0).
__device__ __forceinline__ uint32_t rank_key(float acc, int64_t pos, int n_first, int64_t recent_from) {
    if (pos < n_first || pos >= recent_from) return 0xffffffffu;
    if (acc != acc) return 0u;
    const uint32_t b = __float_as_uint(acc + 0.f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// Exclusive prefix sum of x over the CTA; *total receives the sum.
__device__ __forceinline__ int block_scan(int x, int* buf, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int y = x;
    for (int o = 1; o < 32; o <<= 1) {
        const int z = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) y += z;
    }
    __syncthreads();
    if (lane == 31) buf[warp] = y;
    __syncthreads();
    int before = 0, sum = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += buf[w];
        sum += buf[w];
    }
    *total = sum;
    return before + y - x;
}

// One CTA per (sequence, head): the keep-th key by bisection over its bits, then the lists of
// holes and of the entries that fill them. lists: [N * H][2][most] and counts [N * H].
__global__ void __launch_bounds__(kThreads) select_kernel(const EvictArgs a, int* counts, int* lists, int most) {
    __shared__ int s_buf[kThreads / 32];
    const int64_t nh = blockIdx.x, n = nh / a.H;
    const int len = checked_len(a.seqlens[n], a.max_len, a.c.err);
    const int64_t recent_from = (int64_t)a.positions[n] - a.n_recent, at = nh * a.slots;
    auto key = [&](int j) { return rank_key(a.acc[at + j], a.pos[at + j], a.n_first, recent_from); };
    if (len <= a.keep) {
        for (int j = threadIdx.x; j < len; j += kThreads) {
            a.acc_out[at + j] = a.acc[at + j];
            a.pos_out[at + j] = a.pos[at + j];
        }
        if (threadIdx.x == 0) counts[nh] = 0;
        return;
    }
    // the largest T with at least keep keys >= T
    uint32_t T = 0;
    for (int bit = 31; bit >= 0; --bit) {
        const uint32_t t = T | (1u << bit);
        int c = 0, total;
        for (int j = threadIdx.x; j < len; j += kThreads) c += key(j) >= t;
        block_scan(c, s_buf, &total);
        if (total >= a.keep) T = t;
    }
    int above = 0;
    {
        int c = 0;
        for (int j = threadIdx.x; j < len; j += kThreads) c += key(j) > T;
        block_scan(c, s_buf, &above);
    }
    const int ties = a.keep - above;          // of the entries with key T, so many lowest slots stay
    int seen = 0, holes = 0, tails = 0;
    int* hole = lists + nh * 2 * most;
    int* tail = hole + most;
    for (int j0 = 0; j0 < len; j0 += kThreads) {
        const int j = j0 + threadIdx.x;
        const uint32_t k = j < len ? key(j) : 0;
        const bool tie = j < len && k == T;
        int n_tie, n_hole, n_tail;
        const int r = block_scan(tie, s_buf, &n_tie);
        const bool kept = j < len && (k > T || (tie && seen + r < ties));
        const bool is_hole = j < len && j < a.keep && !kept, is_tail = kept && j >= a.keep;
        const int rh = block_scan(is_hole, s_buf, &n_hole), rt = block_scan(is_tail, s_buf, &n_tail);
        if (is_hole) hole[holes + rh] = j;
        if (is_tail) tail[tails + rt] = j;
        seen += n_tie; holes += n_hole; tails += n_tail;
        if (kept && j < a.keep) {
            a.acc_out[at + j] = a.acc[at + j];
            a.pos_out[at + j] = a.pos[at + j];
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < holes; i += kThreads) {
        a.acc_out[at + hole[i]] = a.acc[at + tail[i]];
        a.pos_out[at + hole[i]] = a.pos[at + tail[i]];
    }
    if (threadIdx.x == 0) counts[nh] = holes;
}

__global__ void __launch_bounds__(kThreads) move_kernel(const EvictArgs a, const int* counts, const int* lists, int most, int row16) {
    const int64_t nh = blockIdx.x, n = nh / a.H, h = nh % a.H;
    if (h == 0 && threadIdx.x == 0)        // after every head's select has read seqlens
        a.seqlens_out[n] = min(checked_len(a.seqlens[n], a.max_len, a.c.err), a.keep);
    const int* hole = lists + nh * 2 * most;
    const int* tail = hole + most;
    const int64_t esz = a.io == Io::BF16 ? 2 : 4;
    const int count = counts[nh];
    for (int i = threadIdx.x / row16; i < count; i += kThreads / row16) {
        const int64_t to = slot_offset(a.c, n, hole[i]), from = slot_offset(a.c, n, tail[i]);
        if (to < 0 || from < 0) continue;
        const int64_t dst = (to + h * a.c.head_stride) * esz + (threadIdx.x % row16) * 16;
        const int64_t src = (from + h * a.c.head_stride) * esz + (threadIdx.x % row16) * 16;
        *reinterpret_cast<uint4*>(static_cast<char*>(a.c.k) + dst) =
            *reinterpret_cast<const uint4*>(static_cast<const char*>(a.c.k) + src);
        *reinterpret_cast<uint4*>(static_cast<char*>(a.c.v) + dst) =
            *reinterpret_cast<const uint4*>(static_cast<const char*>(a.c.v) + src);
    }
}

// Moves of one (sequence, head): at most the slots below keep, or those behind it.
int64_t most_moves(int64_t max_len, int64_t keep) {
    const int64_t behind = max_len > keep ? max_len - keep : 0;
    return behind < keep ? behind : keep;
}

}  // namespace

bool cache_evict_workspace(int64_t N, int64_t H, int64_t max_len, int64_t keep, size_t* bytes) {
    const int64_t most = most_moves(max_len, keep);
    if ((double)N * H * (2.0 * most + 1) * 4 > 9e18) return false;
    *bytes = (size_t)(N * H) * (size_t)(2 * most + 1) * 4;
    return true;
}

cudaError_t launch_cache_evict(const EvictArgs& a, cudaStream_t stream) {
    if (a.N == 0) return cudaSuccess;
    const int row16 = a.d * (a.io == Io::BF16 ? 2 : 4) / 16;
    const int most = (int)most_moves(a.max_len, a.keep);
    int* counts = static_cast<int*>(a.workspace);
    int* lists = counts + (int64_t)a.N * a.H;
    const unsigned grid = (unsigned)(a.N * a.H);
    select_kernel<<<grid, kThreads, 0, stream>>>(a, counts, lists, most);
    move_kernel<<<grid, kThreads, 0, stream>>>(a, counts, lists, most, row16);
    return cudaGetLastError();
}

}  // namespace kda
