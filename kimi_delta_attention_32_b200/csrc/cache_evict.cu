// cache_evict.cu -- cuts every (sequence, key-value head) of the paged cache to a budget of
// entries, by the attention weight that they have gathered. (The softmax-attention layers are the
// only ones whose cache grows with the context: m.lqnn.cn/news/205170, section "KDA 与 Gated
// Attention：每 4 层只留 1 层全注意力". The pages have no eviction.)
//
// Entries rank by a 32-bit key: guarded ones first, then larger acc; equal keys by slot. The keep
// best stay. Those behind slot keep move into the free slots before it ("holes"), both in slot
// order, so the rows that move are only as many as were evicted below keep, however long the
// cache; keeping the slots in order instead would move nearly every row behind the first hole.
//
// Select: one thread-block cluster per (sequence, head), of 1 to 8 blocks by the cache's length.
// Each block reads its part of acc and pos once, into 32-bit keys in shared memory (up to 49152 a
// block; with a bound max_len above 393216 none are held, and acc and pos are read again in every
// pass), and all passes run on those: three of a
// radix select (11, 11 and 10 bits from the top; the blocks' histograms are summed through
// distributed shared memory), one that counts what lies before each warp's slots, and one that
// writes the lists of holes and of the entries that fill them. Integers only: no order of
// atomics can show. The traffic is one read of acc and pos. One sequence of 262144 slots and 8 heads
// on 64 SMs, in thousands of cycles: 17 that read and count, 5 more counting passes, 13 barriers
// and searches between them, 6 counting before each warp, 9 listing, 4 the last barrier. The moves
// then take 94 us.
// Move: the whole GPU copies the listed rows, 64 entries a block, bound by HBM (each moved row is
// read and written once).
#include <cooperative_groups.h>

#include <type_traits>

#include "paged.cuh"

namespace kda {
namespace {

namespace cg = cooperative_groups;

constexpr int kMaxKeys = 49152;           // keys of one block in shared memory: 192 KB
constexpr int kBins = 2048;               // histogram of one pass (three of them: 24 KB)
constexpr int kMaxCluster = 8;
constexpr int kRun = 128;                 // slots that a warp walks at a time

// Rank key of an entry: order-preserving bits of the fp32 weight (NaN lowest, -0 equal to 0).
__device__ __forceinline__ uint32_t rank_key(float acc, int pos, int n_first, int recent_from) {
    if (pos < n_first || pos >= recent_from) return 0xffffffffu;
    if (acc != acc) return 0u;
    const uint32_t b = __float_as_uint(acc + 0.f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

struct SelectArgs {
    EvictArgs e;
    int* counts;              // [N * H] moves
    int* lists;               // [N * H][2][most]: holes, then the entries that fill them
    int most;
    int keys;                 // keys a block holds in shared memory, 0: none
};

// kMany: the cluster has more than one block.
template <int kThreads, bool kMany>
__global__ void __launch_bounds__(kThreads, kThreads == 1024 ? 1 : 1536 / kThreads) evict_select_kernel(const SelectArgs s) {
    extern __shared__ __align__(16) uint32_t s_keys[];
    constexpr int kWarps = kThreads / 32, kStep = 4 * kThreads;
    constexpr int kAhead = 2;                            // steps of four slots that a thread loads ahead
    __shared__ int s_hist[3][kBins], s_coarse[3][kBins / 32];
    __shared__ int s_pick[2];
    __shared__ int s_warp[kWarps][4], s_share[4];        // counts of the warps, and of the block
    const EvictArgs& a = s.e;
    int CS = 1, rank = 0;
    if constexpr (kMany) {
        CS = (int)cg::this_cluster().num_blocks();
        rank = (int)cg::this_cluster().block_rank();
    }
    auto sync_all = [&]() {
        if constexpr (kMany) cg::this_cluster().sync();
        else __syncthreads();
    };
    const int64_t nh = blockIdx.x / CS, n = nh / a.H;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int len = checked_len(a.seqlens[n], a.max_len, a.c.err);
    const int64_t at = nh * a.slots;
    const int recent_from = (int)max((int64_t)INT32_MIN, (int64_t)a.positions[n] - a.n_recent);
    const bool copy_acc = a.acc_out != a.acc, copy_pos = a.pos_out != a.pos;

    if (len <= a.keep || a.keep == 0) {                  // nothing moves (the whole cluster agrees)
        const int m = len <= a.keep ? len : 0;
        for (int j = rank * kThreads + tid; j < m; j += CS * kThreads) {
            if (copy_acc) a.acc_out[at + j] = a.acc[at + j];
            if (copy_pos) a.pos_out[at + j] = a.pos[at + j];
        }
        if (rank == 0 && tid == 0) s.counts[nh] = 0;
        return;
    }
    // the block's slots [lo, hi), a warp's a contiguous run of whole kRun of them; hi_run: whole kRun
    const int per_warp = (len + CS * kWarps * kRun - 1) / (CS * kWarps * kRun) * kRun;
    const int lo = min(len, rank * kWarps * per_warp);
    const int hi = min(len, lo + kWarps * per_warp);
    const int hi_run = lo + (hi - lo + kRun - 1) / kRun * kRun;
    const bool held = hi - lo <= s.keys;
    const float* acc = a.acc + at;
    const int* pos = a.pos + at;
    auto key = [&](int j) { return rank_key(acc[j], pos[j], a.n_first, recent_from); };
    // The keys of four slots from j on, j a multiple of 4 below hi_run. Slots of len and behind have
    // key 0, the lowest: as they also come last, none of the counts below can reach them before
    // entries to be kept or moved.
    auto keys4 = [&](int j, uint32_t (&k)[4]) {
        if (held) {
            const uint4 v = *reinterpret_cast<const uint4*>(s_keys + (j - lo));
            k[0] = v.x; k[1] = v.y; k[2] = v.z; k[3] = v.w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) k[i] = j + i < hi ? key(j + i) : 0;
        }
    };

    const int keep_here = min(hi, a.keep);               // the block's slots in front end here
    const bool wide = ((reinterpret_cast<uintptr_t>(acc) | reinterpret_cast<uintptr_t>(pos) |
                        reinterpret_cast<uintptr_t>(a.acc_out + at) |
                        reinterpret_cast<uintptr_t>(a.pos_out + at)) & 15) == 0;
    for (int i = tid; i < 3 * kBins; i += kThreads) (&s_hist[0][0])[i] = 0;
    __syncthreads();

    // ---- the keep-th largest key T, 11 + 11 + 10 bits from the top; `left` of those equal to the
    // bits found so far are still to be kept
    uint32_t T = 0;
    int left = a.keep;
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
        const uint32_t above = pass == 0 ? 0u : 0xffffffffu << (shift + bits);   // bits found already
        // (the atomics need no help where a warp's keys agree: gathering such first cost a quarter more)
        auto count = [&](uint32_t k) {
            if (((k ^ T) & above) == 0) atomicAdd(&s_hist[pass][(k >> shift) & ((1u << bits) - 1)], 1);
        };
        if (pass == 0) {                                 // the one read of acc and pos
            float w[kAhead][4];
            int q[kAhead][4];
            auto load = [&](int j, int u) {
                if (wide && j + 4 <= hi) {
                    const float4 x = *reinterpret_cast<const float4*>(acc + j);
                    const int4 y = *reinterpret_cast<const int4*>(pos + j);
                    w[u][0] = x.x; w[u][1] = x.y; w[u][2] = x.z; w[u][3] = x.w;
                    q[u][0] = y.x; q[u][1] = y.y; q[u][2] = y.z; q[u][3] = y.w;
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        w[u][i] = j + i < hi ? acc[j + i] : 0.f;
                        q[u][i] = j + i < hi ? pos[j + i] : 0;
                    }
                }
            };
            const int first = lo + 4 * tid;
#pragma unroll
            for (int u = 0; u < kAhead; ++u) load(first + u * kStep, u);
            for (int j0 = first; j0 < hi_run; j0 += kAhead * kStep) {
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const int j = j0 + u * kStep;
                    if (j >= hi_run) break;
                    uint32_t k[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        k[i] = j + i < hi ? rank_key(w[u][i], q[u][i], a.n_first, recent_from) : 0;
                    if (held) *reinterpret_cast<uint4*>(s_keys + (j - lo)) = make_uint4(k[0], k[1], k[2], k[3]);
                    if (wide && j + 4 <= keep_here) {    // a hole's are overwritten by the move
                        if (copy_acc)
                            *reinterpret_cast<float4*>(a.acc_out + at + j) =
                                make_float4(w[u][0], w[u][1], w[u][2], w[u][3]);
                        if (copy_pos)
                            *reinterpret_cast<int4*>(a.pos_out + at + j) =
                                make_int4(q[u][0], q[u][1], q[u][2], q[u][3]);
                    } else if (j < keep_here) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (j + i >= keep_here) break;
                            if (copy_acc) a.acc_out[at + j + i] = w[u][i];
                            if (copy_pos) a.pos_out[at + j + i] = q[u][i];
                        }
                    }
                    load(j + kAhead * kStep, u);
#pragma unroll
                    for (int i = 0; i < 4; ++i) count(k[i]);
                }
            }
        } else {
            for (int j = lo + 4 * tid; j < hi_run; j += kStep) {
                uint32_t k[4];
                keys4(j, k);
#pragma unroll
                for (int i = 0; i < 4; ++i) count(k[i]);
            }
        }
        __syncthreads();
        // sums of 32 bins; one warp then finds the 32 and the bin, from all blocks' histograms
        for (int g = warp; g < kBins / 32; g += kWarps) {
            const int sum = __reduce_add_sync(0xffffffffu, s_hist[pass][g * 32 + lane]);
            if (lane == 0) s_coarse[pass][g] = sum;
        }
        sync_all();
        if (warp == 0) {
            // the value of bin i, summed over the cluster
            auto sum_over = [&](int* bins, int i) {
                if constexpr (!kMany) return bins[i];
                int v = 0;
#pragma unroll
                for (int r = 0; r < kMaxCluster; ++r)
                    if (r < CS) v += cg::this_cluster().map_shared_rank(bins, r)[i];
                return v;
            };
            // of 32 counts, lane l's the l-th from the top: the lane at which `left` is reached
            auto reach = [&](int c, int& over) {
                int upto = c;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int u = __shfl_up_sync(0xffffffffu, upto, o);
                    if (lane >= o) upto += u;
                }
                const unsigned hit = __ballot_sync(0xffffffffu, upto >= left);
                const int at_lane = __ffs(hit) - 1;      // -1: not among these
                over = __shfl_sync(0xffffffffu, at_lane < 0 ? upto : upto - c, at_lane < 0 ? 31 : at_lane);
                return at_lane;
            };
            const int upper = sum_over(s_coarse[pass], kBins / 32 - 1 - lane);
            const int lower = sum_over(s_coarse[pass], kBins / 64 - 1 - lane);
            int over, group = reach(upper, over);
            if (group >= 0) {
                group = kBins / 32 - 1 - group;
                left -= over;
            } else {
                left -= over;
                group = kBins / 64 - 1 - reach(lower, over);
                left -= over;
            }
            const int bin = 31 - reach(sum_over(s_hist[pass] + group * 32, 31 - lane), over);
            if (lane == 0) {
                s_pick[0] = group * 32 + bin;
                s_pick[1] = left - over;
            }
        }
        __syncthreads();
        T |= (uint32_t)s_pick[0] << shift;
        left = s_pick[1];
    }

    // ---- Of the entries with key T the `left` lowest slots stay, so what is kept before a slot
    // follows from four counts before it: keys above T and keys equal to T, in front (slots < keep)
    // and behind. Front slots come first, so the kept ties in front are min(left, ties in front).
    // A lane takes four slots at a time.
    const int w0 = min(hi, lo + warp * per_warp), w1 = min(hi, w0 + per_warp);
    int cnt[4] = {0, 0, 0, 0};                           // above in front, behind; ties in front, behind
    for (int j0 = w0; j0 < w1; j0 += kRun) {
        uint32_t k[4];
        keys4(j0 + 4 * lane, k);
        if (j0 < a.keep && j0 + kRun > a.keep) {         // keep lies within
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bool front = j0 + 4 * lane + i < a.keep;
                cnt[0] += front && k[i] > T;
                cnt[1] += !front && k[i] > T;
                cnt[2] += front && k[i] == T;
                cnt[3] += !front && k[i] == T;
            }
        } else {
            int up = 0, ties = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                up += k[i] > T;
                ties += k[i] == T;
            }
            if (j0 < a.keep) {
                cnt[0] += up;
                cnt[2] += ties;
            } else {
                cnt[1] += up;
                cnt[3] += ties;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        cnt[i] = __reduce_add_sync(0xffffffffu, cnt[i]);
        if (lane == 0) s_warp[warp][i] = cnt[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {                        // before this warp, and of the whole block
        const int v = lane < kWarps ? s_warp[lane][i] : 0;
        cnt[i] = __reduce_add_sync(0xffffffffu, lane < warp ? v : 0);
        if constexpr (kMany) {
            const int all = __reduce_add_sync(0xffffffffu, v);
            if (tid == 0) s_share[i] = all;
        }
    }
    if constexpr (kMany) {
        cg::this_cluster().sync();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int v = lane < rank ? cg::this_cluster().map_shared_rank(&s_share[0], lane)[i] : 0;
            cnt[i] += __reduce_add_sync(0xffffffffu, v);
        }
    }
    int* hole = s.lists + nh * 2 * s.most;
    int* tail = hole + s.most;
    // the slots [from, to) of one side: a front slot that goes is a hole, a slot behind that stays
    // fills one
    auto list = [&](auto is_front, int from, int to) {
        constexpr bool kFront = decltype(is_front)::value;
        int up = kFront ? cnt[0] : cnt[1], ties = cnt[2] + (kFront ? 0 : cnt[3]);
        const int stay_f = min(left, cnt[2]);            // (for the slots behind: all front ties kept)
        if (from >= to) return;                          // (a block behind the end has no keys to read)
        for (int j0 = from & ~(kRun - 1); j0 < to; j0 += kRun) {
            const int j = j0 + 4 * lane;
            uint32_t k[4];
            keys4(j, k);
            const bool tie = k[0] == T || k[1] == T || k[2] == T || k[3] == T;
            if (j0 >= from && j0 + kRun <= to && !__any_sync(0xffffffffu, tie)) {
                // nearly always: all of it is asked for, and it has no ties
                const int kept = up + min(left, ties) - (kFront ? 0 : stay_f);   // before j0
                int in_run = 0, at_list = kFront ? j0 - kept : kept;
                bool put[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    put[i] = (k[i] > T) != kFront;
                    const unsigned who = __ballot_sync(0xffffffffu, put[i]);
                    at_list += __popc(who & ((1u << lane) - 1));
                    in_run += __popc(who);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (put[i]) (kFront ? hole : tail)[at_list++] = j + i;
                up += kFront ? kRun - in_run : in_run;
                continue;
            }
            uint32_t one[4], mine = 0;                   // counts: above in the low half, ties in the high
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                one[i] = j + i < from || j + i >= to || k[i] < T ? 0u : k[i] > T ? 1u : 0x10000u;
                mine += one[i];
            }
            uint32_t upto = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t u = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += u;
            }
            const uint32_t all = __shfl_sync(0xffffffffu, upto, 31);
            upto -= mine;                                // before this lane's first slot
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int tied = ties + (int)(upto >> 16), above = up + (int)(upto & 0xffffu);
                const bool kept = one[i] == 1u || (one[i] != 0 && tied < left);
                const int before = above + min(left, tied) - (kFront ? 0 : stay_f);   // kept before j + i
                if constexpr (kFront) {
                    if (!kept && j + i >= from && j + i < to) hole[j + i - before] = j + i;
                } else {
                    if (kept) tail[before] = j + i;
                }
                upto += one[i];
            }
            up += (int)(all & 0xffffu);
            ties += (int)(all >> 16);
        }
        cnt[kFront ? 0 : 1] = up;
        if constexpr (kFront) cnt[2] = ties;
        else cnt[3] = ties - cnt[2];
    };
    list(std::true_type{}, w0, min(w1, a.keep));
    list(std::false_type{}, max(w0, a.keep), w1);
    // after the last warp's slots: all that is kept behind keep
    if (rank == CS - 1 && tid == kThreads - 1)
        s.counts[nh] = cnt[1] + min(left, cnt[2] + cnt[3]) - min(left, cnt[2]);
    if constexpr (kMany) cg::this_cluster().sync();      // shared memory stays until all have read it
}

constexpr int kMoveThreads = 256, kMoveRows = 64;
template <int kPieces>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const SelectArgs s, int chunks, int esz) {
    __shared__ int64_t s_to[kMoveRows], s_from[kMoveRows];
    const EvictArgs& a = s.e;
    grid_wait();
    const int64_t nh = blockIdx.x / chunks, n = nh / a.H, at = nh * a.slots;
    const int h = (int)(nh % a.H), first = (int)(blockIdx.x % chunks) * kMoveRows, tid = threadIdx.x;
    if (h == 0 && first == 0 && tid == 0)      // after every head's select has read seqlens
        a.seqlens_out[n] = min(checked_len(a.seqlens[n], a.max_len, a.c.err), a.keep);
    const int rows = min(kMoveRows, s.counts[nh] - first);
    if (rows <= 0) return;
    if (tid < 2 * kMoveRows) {
        const int i = tid % kMoveRows;
        int64_t off = -1;
        if (i < rows) {
            const int* list = s.lists + nh * 2 * s.most + first + i;
            const int slot = list[tid < kMoveRows ? 0 : s.most];
            off = slot_offset(a.c, n, slot);
            if (off >= 0) off = (off + h * a.c.head_stride) * esz;
            if (tid < kMoveRows) {
                const int from = list[s.most];
                a.acc_out[at + slot] = a.acc[at + from];
                a.pos_out[at + slot] = a.pos[at + from];
            }
        }
        (tid < kMoveRows ? s_to : s_from)[i] = off;
    }
    __syncthreads();
    // K and V rows, 16 bytes a thread; a batch of loads, then its stores
    constexpr int kStep = kMoveThreads / kPieces;        // rows a pass covers
    constexpr int kBatch = kMoveRows / kStep < 4 ? kMoveRows / kStep : 4;
    const int piece = (tid % kPieces) * 16;
    char* kc = static_cast<char*>(a.c.k) + piece;
    char* vc = static_cast<char*>(a.c.v) + piece;
    for (int r0 = tid / kPieces; r0 < rows; r0 += kStep * kBatch) {
        uint4 x[kBatch], y[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int r = r0 + i * kStep;
            x[i] = y[i] = make_uint4(0, 0, 0, 0);        // (what a row on a bad page reads as)
            if (r < rows && s_from[r] >= 0) {
                x[i] = *reinterpret_cast<const uint4*>(kc + s_from[r]);
                y[i] = *reinterpret_cast<const uint4*>(vc + s_from[r]);
            }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int r = r0 + i * kStep;
            if (r < rows && s_to[r] >= 0) {
                *reinterpret_cast<uint4*>(kc + s_to[r]) = x[i];
                *reinterpret_cast<uint4*>(vc + s_to[r]) = y[i];
            }
        }
    }
}

// Moves of one (sequence, head): at most the slots below keep, or those behind it.
int64_t most_moves(int64_t max_len, int64_t keep) {
    const int64_t behind = max_len > keep ? max_len - keep : 0;
    return behind < keep ? behind : keep;
}

template <int kThreads, bool kMany>
cudaError_t launch_select(const SelectArgs& s, int cluster, size_t smem, cudaStream_t stream) {
    auto kernel = evict_select_kernel<kThreads, kMany>;
    cudaError_t e = allow_smem(kernel, sizeof(uint32_t) * kMaxKeys);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(s.e.N * s.e.H * cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = kMany ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, s);
}

// Blocks of the two launches count in 31 bits.
bool grids_fit(int64_t N, int64_t H, int64_t most) {
    const int64_t chunks = (most + kMoveRows - 1) / kMoveRows;
    return N * H * kMaxCluster <= INT32_MAX && (double)N * H * (chunks > 0 ? chunks : 1) <= INT32_MAX;
}

}  // namespace

bool cache_evict_workspace(int64_t N, int64_t H, int64_t max_len, int64_t keep, size_t* bytes) {
    const int64_t most = most_moves(max_len, keep);
    if (!grids_fit(N, H, most)) return false;
    *bytes = (size_t)(N * H) * (size_t)(2 * most + 1) * 4;
    return true;
}

cudaError_t launch_cache_evict(const EvictArgs& a, cudaStream_t stream) {
    if (a.N == 0) return cudaSuccess;
    SelectArgs s;
    s.e = a;
    s.most = (int)most_moves(a.max_len, a.keep);
    s.counts = static_cast<int*>(a.workspace);
    s.lists = s.counts + (int64_t)a.N * a.H;
    // A block for up to 8192 slots, or 16384 once more blocks would outnumber the SMs (32 sequences of
    // 32768, 8 heads: 423 us with 2 blocks a head, 433 with 4; 4 sequences of 65536: 114 with 4, 116
    // with 8; but one of 16384: 27.6 with 2, 31.6 with 1). 8 at most: of clusters of 16 only 7 fit the
    // GPU at once (of 8, 15), so that the 8 heads of one long sequence took two waves of them. Shorter
    // caches take fewer threads: fewer meet at the barriers, and more blocks share an SM (64 sequences
    // of 2000, 8 heads: 66.6 us with 256, 69.6 with 512).
    const int64_t heads = (int64_t)a.N * a.H;
    int cluster = 1;
    while (cluster < kMaxCluster && (int64_t)cluster * (heads * cluster * 2 > sm_count() ? 16384 : 8192) < a.max_len)
        cluster *= 2;
    // A long cache alone takes all the threads that a block can have; where more blocks than SMs are
    // to run, blocks of 512 share an SM, and one's barriers overlap another's work (32 sequences of
    // 32768, 4 blocks a head: 480 us with 1024 threads, 433 with 512).
    const bool crowd = heads * cluster > sm_count();
    const int threads = a.max_len <= 2048 ? 256 : cluster == 1 || crowd ? 512 : 1024;
    const int block = threads / 32 * kRun;               // a block's slots come in whole runs of its warps
    const int64_t need = ((int64_t)a.max_len + cluster * block - 1) / (cluster * block) * block;
    s.keys = need <= kMaxKeys ? (int)need : 0;
    const size_t smem = (size_t)s.keys * 4;
    const cudaError_t e = threads == 256   ? launch_select<256, false>(s, 1, smem, stream)
                          : cluster == 1   ? launch_select<512, false>(s, 1, smem, stream)
                          : threads == 512 ? launch_select<512, true>(s, cluster, smem, stream)
                                           : launch_select<1024, true>(s, cluster, smem, stream);
    if (e != cudaSuccess) return e;
    const int esz = a.io == Io::BF16 ? 2 : 4;
    const int chunks = s.most > 0 ? (s.most + kMoveRows - 1) / kMoveRows : 1;
    const unsigned grid = (unsigned)((int64_t)a.N * a.H * chunks);
    switch (a.d * esz / 16) {
        case 8: return launch_after(evict_move_kernel<8>, grid, kMoveThreads, stream, s, chunks, esz);
        case 16: return launch_after(evict_move_kernel<16>, grid, kMoveThreads, stream, s, chunks, esz);
        case 32: return launch_after(evict_move_kernel<32>, grid, kMoveThreads, stream, s, chunks, esz);
    }
    return cudaErrorInvalidValue;
}

}  // namespace kda
