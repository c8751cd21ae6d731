// paged_decode.cu -- attention of one new token per sequence over its paged cache
// (m.lqnn.cn/news/205170, section "KDA 与 Gated Attention：每 4 层只留 1 层全注意力": the
// softmax-attention layer with its sigmoid output gate).
//
// Per (sequence, query head), over the slots j < len:  s_j = scale q . K_j,  w = softmax(s),
// o = sum_j w_j V_j, o *= sigmoid(z); the weights are added to acc per key-value head.
//
// What bounds it: every key and value is read once and meets only the G = Hq / Hkv queries of its
// head, G flops a byte in bf16, so HBM does. The design is a stream of K and V rows through shared
// memory that never waits for the arithmetic.
//
// Division. A segment is (sequence, key-value head, tile of at most 8 NT query heads). Its slots
// are cut into tiles of 16 W slots (W warps); all tiles of all segments, in order, are divided
// evenly over a grid that just fills the GPU (decode_split.h), whatever the mix of lengths. A
// segment inside one block is finished by it; the parts of a segment that spans blocks are joined
// by a second kernel. Lengths are read on the device: the grid does not depend on them.
//
// One pass, online softmax. Each warp takes 16 slots of a tile and keeps its own running maximum,
// sum and output in registers, so warps meet only at a segment's end. The slots are the M side of
// the products and the queries the N side (padded to 8, not 16): S^T = K Q^T and O^T = V^T P^T.
// With M >= 64 rows an instruction, the tcgen05 path would be at least 7/8 padding for such G and
// its operands would pass through tensor memory; the warp-level MMA feeds from ldmatrix directly,
// and with 4 queries a head its pipe is busy 14% of the time (32 sequences of 4000 slots).
//  - bf16: m16n8k16, P as the sum of two bf16 (one would add an error as large as the rounding of
//    the output, 1.35 times it together; the second product costs about 1% of the time for G <= 8
//    and a tenth for G >= 16).
//  - fp32: m16n8k8 TF32, each operand split in two (x = hi + lo, both TF32) and three products,
//    which leaves about 2^-20 of a product at most, and 2^-22 of it on average.
//  - The tensor cores cut their sums instead of rounding them: running sums kept in them drift
//    downwards with the cache's length (8e-5 of the output in 4096 steps). Each step's outputs
//    therefore start at zero and are added to the running ones in fp32. Of the outputs of 64 sequences
//    of 128 to 16384 tokens 4.5e-4 are then not the nearest bf16, 1.5e-3 otherwise; it takes no
//    measurable time for G <= 16, 3 to 8% for G = 32.
//
// Memory. Every warp owns a ring of U units (16 K rows or 16 V rows, in turn), filled by 16-byte
// cp.async and waited for by its own lanes only: no warp waits for another between a segment's
// first tile and its end. 16-byte piece c of row r lies at piece c ^ (r % 8): ldmatrix reads eight
// rows without a bank conflict. Page numbers are read two tiles before their rows are.
// Rows behind the end or with a bad page number are filled with zeros and masked.
//
// Measured on one B200, whole calls: 64 sequences of 128 to 16384 tokens, 32 query and 8 key-value
// heads of 128, bf16, with the gate, 353 to 363 us, 97 to 99% of the 6459 GB/s of a copy and as fast as
// a kernel that only reads them (362 us); 262144 tokens, 8 and 2 heads, 54 us, of which 9 are the join;
// fp32, 32 sequences of 4096, 32 and 8 heads of 128, 165 to 167 us.
#include "decode_split.h"
#include "paged.cuh"

namespace kda {
namespace {

constexpr int kMaxBlocks = 480;          // blocks of one launch: 3 an SM, for up to 160 SMs
constexpr float kSlack = 8.f;            // log2: a weight may reach 2^8 before the running maximum moves

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// 16 bytes, or zeros when !live (src is then not read).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                 ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int n>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory"); }

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t* r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t* r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ void mma_bf16(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, "
                 "{%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, "
                 "{%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// x = hi + lo up to 2^-21 x, both TF32 values (fp32 with 10 bits of fraction): hi is rounded to
// the nearest, so |lo| <= 2^-11 x, and lo is cut. Values from (2 - 2^-11) 2^127 on would round to
// infinity: hi then is the largest TF32, and an infinite x is lo's. (Rounded by two integer operations
// instead, without that limit, 32 sequences of 4096, 32/8 heads of 128, took 171 us, 167 this way.)
__device__ __forceinline__ void split_tf32(uint32_t x, uint32_t& hi, uint32_t& lo) {
    asm("cvt.rn.satfinite.tf32.f32 %0, %1;" : "=r"(hi) : "f"(__uint_as_float(x)));
    lo = __float_as_uint(__uint_as_float(x) - __uint_as_float(hi)) & 0xffffe000u;
}
// d += a b to fp32's accuracy: the two small cross products, then the large one, summed from zero
// and added to d in fp32 (1.8e-6 of the output was measured with the tensor cores' running sums over a
// long cache, 2.4e-7 this way).
__device__ __forceinline__ void mma_f32(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
    uint32_t ah[4], al[4], bh0, bh1, bl0, bl1;
#pragma unroll
    for (int i = 0; i < 4; ++i) split_tf32(a[i], ah[i], al[i]);
    split_tf32(b0, bh0, bl0);
    split_tf32(b1, bh1, bl1);
    float t[4] = {0.f, 0.f, 0.f, 0.f};
    mma_tf32(t, al, bh0, bh1);
    mma_tf32(t, ah, bl0, bl1);
    mma_tf32(t, ah, bh0, bh1);
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] += t[i];
}
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float sigmoid(float z) { return 1.f / (1.f + expf(-z)); }

// Sizes of one instantiation. NT: tiles of 8 query heads that a block works on at once.
//  - two blocks of 4 warps an SM, three where a row is 128 bytes and the registers allow: a block's
//    join of its warps then overlaps the others' streams. fp32 rows of 512 bytes leave room for one
//    block, of 8 warps with three units each;
//  - 128 to 168 KB of rows an SM are in flight beside what is being read;
//  - every tile in flight, and the current one, may begin a segment: room for NQ segments' queries.
template <typename T, int D, int NT>
struct Shape {
    static constexpr bool kBf16 = sizeof(T) == 2;
    static constexpr int kRowBytes = D * (int)sizeof(T);
    static constexpr int kPieces = kRowBytes / 16;               // 16-byte pieces of a row
    static constexpr int W = kRowBytes == 512 ? 8 : 4;
    static constexpr int kPerSm = kRowBytes == 512 ? 1 : kRowBytes == 128 && NT < 4 ? 3 : 2;
    static constexpr int U = kRowBytes == 512 ? 3 : kRowBytes == 128 ? (NT < 4 ? 8 : 10) : NT < 4 ? 6 : 5;
    static constexpr int NQ = U / 2 + 1;
    static constexpr int kTile = 16 * W;                         // slots of a tile
    static constexpr int kUnit = 16 * kRowBytes;                 // a warp's K or V rows of a tile
    static constexpr int kQ = 8 * NT * kRowBytes;                // a segment's queries
    static constexpr int kRegs = D / 4 * NT;                     // output registers a lane (D/16 x 4 x NT)
    static constexpr int kPart = kRegs * 32 + 16 * NT;           // floats of a part: O, m, l
    static constexpr size_t kSmem = (size_t)U * W * kUnit + NQ * kQ + (2 * W * 8 * NT + W * NQ) * 4;
    static_assert(kSmem <= 227 * 1024 && kPerSm * (kSmem + 1024) <= 228 * 1024, "shared memory");
    static_assert(D / 4 * 32 * 4 <= kUnit, "a unit holds a head tile's outputs");
};

struct Params {
    PagedCache c;
    uint32_t page16, slot16, head16; // strides in 16 bytes: their products take one instruction
    int step_pages, step_rows;       // a tile's slots, in whole pages and the rest
    const void *q, *z;
    const int32_t* seqlens;
    float scale_log2;
    void* o;
    int N, Hq, H, G, GT;             // GT: head tiles of a group
    int max_len;
    int most_blocks;
    int whole;                       // > 0: a block a segment, of at most so many tiles; no joins
    int* meta;                       // [blocks][4]: n, head * GT + gt, last block of a segment to join
    float* parts;                    // [2 blocks][kPart]: a block's first and last segments' parts
    // for acc: scores (log2 units) [tile][GS][kTile]; {max, 1 / sum} [N, Hq] of the segments inside
    // one block; and the tiles of the sequences before n, of one head [N + 1]
    float* scores;
    float2* stats;
    int* tiles_before;
    int GS;                          // heads of a tile's scores: min(G, 8 NT)
    float* acc;
    int slots;
};

// Which head, output channel a lane's register r of a part stands for (r = ((nt, mt), c); c & 1 is
// the column, c >> 1 the row). The rows of the products are channels in an order of their own: for
// bf16 ldmatrix's, for fp32 D / 8 in a row for each of 8 groups of lanes.
template <typename T, int D>
__device__ __forceinline__ void part_coord(int r, int lane, int& head, int& ch) {
    const int c = r & 3, mt = (r >> 2) % (D / 16), nt = (r >> 2) / (D / 16);
    head = nt * 8 + 2 * (lane & 3) + (c & 1);
    ch = sizeof(T) == 2 ? mt * 16 + (lane >> 2) + 8 * (c >> 1) : (lane >> 2) * (D / 8) + 2 * mt + (c >> 1);
}

// kCount of the outputs of a segment (its first query head's row is row0, of live_heads): registers
// r0 on, of heads 2 (lane % 4) + {0, 1}. load_gate reads their z, store_out stores them, times inv
// of their head and sigmoid(z).
template <typename T, int D, int kCount>
__device__ __forceinline__ void load_gate(const Params& p, int64_t row0, int live_heads, int r0, int lane,
                                          float (&z)[kCount]) {
    if (p.z == nullptr) return;
#pragma unroll
    for (int u = 0; u < kCount; ++u) {
        int h, ch;
        part_coord<T, D>(r0 + u, lane, h, ch);
        z[u] = h < live_heads ? to_f32(static_cast<const T*>(p.z)[(row0 + h) * D + ch]) : 0.f;
    }
}
template <typename T, int D, int kCount>
__device__ __forceinline__ void store_out(const Params& p, int64_t row0, int live_heads, int r0, int lane,
                                          const float (&y)[kCount], const float (&z)[kCount],
                                          const float (&inv)[2]) {
#pragma unroll
    for (int u = 0; u < kCount; ++u) {
        int h, ch;
        part_coord<T, D>(r0 + u, lane, h, ch);
        float v = y[u] * inv[u & 1];
        if (p.z != nullptr) v *= sigmoid(z[u]);
        if (h < live_heads) static_cast<T*>(p.o)[(row0 + h) * D + ch] = from_f32<T>(v);
    }
}

// kRuns: a page holds a multiple of 16 slots, so a warp's 16 lie in one page.
template <typename T, int D, int NT, bool kRuns>
__global__ void __launch_bounds__(Shape<T, D, NT>::W * 32, Shape<T, D, NT>::kPerSm)
paged_decode_kernel(const Params p) {
    using X = Shape<T, D, NT>;
    constexpr int W = X::W, U = X::U, NQ = X::NQ, kThreads = W * 32, kTile = X::kTile;
    constexpr bool kBf16 = X::kBf16;
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t* s_ring = smem;                                        // [W][U][16 rows]
    uint8_t* s_q = s_ring + (size_t)U * W * X::kUnit;              // [NQ][8 NT rows]
    float* s_m = reinterpret_cast<float*>(s_q + (size_t)NQ * X::kQ);    // [W][8 NT]
    float* s_l = s_m + W * 8 * NT;
    uint32_t* s_live = reinterpret_cast<uint32_t*>(s_l + W * 8 * NT);   // [W][NQ] slots to attend to

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int heads = p.H * p.GT;                                  // segments of a sequence
    const T* q = static_cast<const T*>(p.q);

    // ---- the block's tiles: `count` of them from tile t0 of all on, the first at `cur`
    auto len_of = [&](int n) { return checked_len(__ldg(p.seqlens + n), p.max_len, p.c.err); };
    auto tiles_of = [&](int len) { return (len + kTile - 1) / kTile; };
    struct Cursor { int n, hkv, gt, tile, len, tiles; };
    Cursor cur;
    const int b = blockIdx.x;
    int64_t t0, all_tiles = 0;
    int count, C = 0;
    if (p.whole > 0) {
        cur.n = b / heads;
        cur.hkv = (b - cur.n * heads) / p.GT;
        cur.gt = b - cur.n * heads - cur.hkv * p.GT;
        cur.tile = 0;
        cur.len = len_of(cur.n);
        cur.tiles = count = tiles_of(cur.len);
        t0 = (int64_t)b * p.whole;
        if (count == 0) {
            const int g0 = cur.gt * 8 * NT, end = min(8 * NT, p.G - g0) * D;
            T* o = static_cast<T*>(p.o) + ((int64_t)cur.n * p.Hq + cur.hkv * p.G + g0) * D;
            for (int e = tid; e < end; e += kThreads) o[e] = from_f32<T>(0.f);
            return;
        }
    } else {
    // Up to 32 sequences every warp scans their tiles on its own; more are summed by groups first,
    // the warps sharing them, in the ring that is still empty.
    auto tiles_at = [&](int n, int end) { return n < end ? tiles_of(len_of(n)) : 0; };
    auto warp_scan = [&](int x) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += u;
        }
        return x;
    };
    // a group is 32 sequences, or as many more as keep the groups' sums within 4096
    const bool grouped = p.N > 32;
    const int group = 32 * ((p.N + 32 * 4096 - 1) / (32 * 4096)), groups = (p.N + group - 1) / group;
    int* s_sum = reinterpret_cast<int*>(smem);
    int mine = 0, own0 = 0, own1 = 0;                  // lane l's sequences, or its groups
    if (grouped) {
#pragma unroll 8
        for (int g = warp; g < groups; g += W) {
            int x = 0;
            for (int n = g * group + lane; n < (g + 1) * group; n += 32) x += tiles_at(n, p.N);
            x = __reduce_add_sync(0xffffffffu, x);
            if (lane == 0) s_sum[g] = x;
        }
        __syncthreads();
        const int per = (groups + 31) / 32;
        own0 = min(groups, lane * per);
        own1 = min(groups, own0 + per);
        for (int g = own0; g < own1; ++g) mine += s_sum[g];
    } else {
        mine = tiles_at(lane, p.N);
    }
    const int incl = warp_scan(mine);
    const int64_t work = all_tiles = (int64_t)__shfl_sync(0xffffffffu, incl, 31) * heads;
    C = split_blocks(work, p.most_blocks);
    if (tid == 0) p.meta[4 * b + 2] = -1;
    // sequences of length 0 have no tiles: their outputs are written here
    for (int n = b; n < p.N; n += gridDim.x)
        if (len_of(n) == 0)
            for (int e = tid; e < p.Hq * D; e += kThreads)
                static_cast<T*>(p.o)[(int64_t)n * p.Hq * D + e] = from_f32<T>(0.f);
    if (b >= C) return;
    if (p.tiles_before != nullptr && warp == 0) {
        if (b == 0 && lane == 31) p.tiles_before[p.N] = incl;
        if (!grouped) {
            if (b == 0 && lane < p.N) p.tiles_before[lane] = incl - mine;
        } else {
            for (int g = b; g < groups; g += C) {
                int run = 0;
                for (int i = lane; i < g; i += 32) run += s_sum[i];
                run = __reduce_add_sync(0xffffffffu, run);
                for (int n = g * group + lane; n - lane < min(p.N, (g + 1) * group); n += 32) {
                    const int x = tiles_at(n, p.N), upto = warp_scan(x);
                    if (n < p.N) p.tiles_before[n] = run + upto - x;
                    run += __shfl_sync(0xffffffffu, upto, 31);
                }
            }
        }
    }
    t0 = split_begin(work, C, b);
    count = (int)(split_begin(work, C, b + 1) - t0);
    const int target = (int)split_div(t0, heads);      // tiles of earlier sequences <= target
    const int owner = __ffs(__ballot_sync(0xffffffffu, mine > 0 && target < incl)) - 1;
    int first_n = owner, first_before = __shfl_sync(0xffffffffu, incl - mine, owner);
    if (grouped) {
        int g = __shfl_sync(0xffffffffu, own0, owner);
        while (target >= first_before + s_sum[g]) first_before += s_sum[g++];
        first_n = g * group;
        while (true) {
            const int x = tiles_at(first_n + lane, p.N), upto = first_before + warp_scan(x);
            const unsigned here = __ballot_sync(0xffffffffu, x > 0 && target < upto);
            if (here != 0) {
                first_n += __ffs(here) - 1;
                first_before = __shfl_sync(0xffffffffu, upto - x, __ffs(here) - 1);
                break;
            }
            first_before = __shfl_sync(0xffffffffu, upto, 31);
            first_n += 32;
        }
        __syncthreads();                               // the sums have been read: the ring may fill
    }

    cur.n = first_n;
    cur.len = len_of(cur.n);
    cur.tiles = tiles_of(cur.len);
    const int64_t in_seq = t0 - (int64_t)first_before * heads;
    const int head = (int)split_div(in_seq, cur.tiles);
    cur.tile = (int)(in_seq - (int64_t)head * cur.tiles);
    cur.hkv = head / p.GT;
    cur.gt = head % p.GT;
    }

    // on to the next segment: head tile, key-value head, sequence
    auto next_segment = [&](Cursor& u) {
        u.tile = 0;
        if (++u.gt < p.GT) return;
        u.gt = 0;
        if (++u.hkv < p.H) return;
        u.hkv = 0;
        do {
            ++u.n;
            u.len = u.n < p.N ? len_of(u.n) : 1;
        } while (u.len == 0);
        u.tiles = tiles_of(u.len);
    };

    // ---- page numbers: with kRuns one for the warp's 16 slots of a tile, else lanes l and l + 16
    // hold slot l's. That of the tile behind the next is on its way while the next one's is used; the
    // heads of a sequence walk the same table, so only a new sequence starts without one.
    Cursor ahead = cur;                                            // the tile to be loaded next
    const int own = warp * 16 + (kRuns ? 0 : lane & 15);           // the lane's slot of a tile
    const int own_page = own / p.c.page_size, own_row = own - own_page * p.c.page_size;
    int at_page = (ahead.tile * kTile + own) / p.c.page_size;
    int row = ahead.tile * kTile + own - at_page * p.c.page_size;
    int left = ahead.len - ahead.tile * kTile - own;               // slots from the lane's on
    const int32_t* table = p.c.block_table + (int64_t)ahead.n * p.c.max_pages;
    int page = left > 0 ? __ldg(table + at_page) : -1, page_behind = -1;
    int loaded = 0, seg_loaded = -1, at_unit = 0, live_slot = 0;
    bool begins = true;                                            // the tile brings its queries
    // the first touch of a sequence's table would stall a tile for its trip to memory
    auto warm_table = [&]() {
        if (warp == 0) {
            const int e = at_page + lane * 32;
            if (e * (int64_t)p.c.page_size < ahead.len)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(table + e));
            if (lane == 0 && ahead.n + 1 < p.N)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(table + p.c.max_pages));
        }
    };
    auto fetch_behind = [&]() {
        if (ahead.tile + 1 < ahead.tiles) {
            if (left > kTile)
                page_behind = __ldg(table + at_page + p.step_pages + (row + p.step_rows >= p.c.page_size));
        } else if ((ahead.gt + 1 < p.GT || ahead.hkv + 1 < p.H) && own < ahead.len) {
            page_behind = __ldg(table + own_page);
        }
    };
    uint8_t* ring = s_ring + (size_t)warp * U * X::kUnit;
    // row a of those that a warp instruction covers, 16-byte piece `piece`; rows r0 + a lie r0 rows
    // on, with the piece's place exchanged by r0's low bits
    constexpr int kRows = 32 / X::kPieces;
    const int la = lane / X::kPieces, piece = lane % X::kPieces;
    const uint32_t lane_dst = smem_u32(ring) + la * X::kRowBytes + ((piece ^ la) << 4);
    const int64_t lane_src = ((kRuns ? (int64_t)la * p.slot16 : 0) + piece) * 16;
    const int64_t rows_bytes = (int64_t)kRows * p.slot16 * 16;
    const uint8_t* kbase = static_cast<const uint8_t*>(p.c.k) + lane_src;
    const uint8_t* vbase = static_cast<const uint8_t*>(p.c.v) + lane_src;
    int64_t off = 0;                                   // of the tile being loaded: its rows,
    uint32_t mask = 0;                                 // and of the 16 slots those to attend to
    auto load_rows = [&](const uint8_t* from_base) {
        const uint32_t dst = lane_dst + at_unit * X::kUnit;
        if (kRuns && mask == 0xffffu) {
            // (each load has an address register of its own: one that is reused waits for the load
            // before it to have read it)
            const uint8_t* src[16 / kRows];
#pragma unroll
            for (int i = 0; i < 16 / kRows; ++i) src[i] = from_base + off + i * rows_bytes;
#pragma unroll
            for (int r0 = 0; r0 < 16; r0 += kRows)
                cp_async16((dst + r0 * X::kRowBytes) ^ ((r0 & 7) << 4), src[r0 / kRows]);
        } else {
#pragma unroll
            for (int r0 = 0; r0 < 16; r0 += kRows) {
                const bool ok = mask >> (r0 + la) & 1;
                int64_t from = off;
                if constexpr (kRuns) from = ok ? off + r0 / kRows * rows_bytes : 0;
                else from = __shfl_sync(0xffffffffu, off, r0 + la);
                cp_async16((dst + r0 * X::kRowBytes) ^ ((r0 & 7) << 4), from_base + from, ok);
            }
        }
        if (++at_unit == U) at_unit = 0;
    };
    auto load_k = [&]() {        // K rows of tile `loaded`, and its queries if it begins a segment
        if (loaded < count) {
            bool live = left > 0;
            if (live && (unsigned)page >= (unsigned)p.c.num_pages) {
                atomicOr(p.c.err, kErrIndex);
                live = false;
            }
            mask = kRuns ? (live ? 0xffffu >> (16 - min(16, left)) : 0u)
                         : __ballot_sync(0xffffffffu, live) & 0xffffu;
            if (lane == 0) s_live[warp * NQ + live_slot] = mask;
            if (++live_slot == NQ) live_slot = 0;
            off = live ? ((uint64_t)(uint32_t)page * p.page16 + (uint64_t)(uint32_t)row * p.slot16 +
                          (uint64_t)(uint32_t)ahead.hkv * p.head16) * 16 : 0;
            load_rows(kbase);
            if (begins) {
                if (++seg_loaded == NQ) seg_loaded = 0;
                const uint32_t qd = smem_u32(s_q) + seg_loaded * X::kQ;
                const int g0 = ahead.gt * 8 * NT;
                const T* src = q + ((int64_t)ahead.n * p.Hq + ahead.hkv * p.G + g0) * D;
                for (int e = tid; e < 8 * NT * X::kPieces; e += kThreads) {
                    const int g = e / X::kPieces, pc = e % X::kPieces;
                    const bool ok = g0 + g < p.G;
                    cp_async16(qd + g * X::kRowBytes + ((pc ^ (g & 7)) << 4),
                               reinterpret_cast<const uint8_t*>(src) + (ok ? e * 16 : 0), ok);
                }
            }
        }
        cp_commit();
    };
    auto load_v = [&]() {        // its V rows; then on to the next tile
        if (loaded < count) {
            load_rows(vbase);
            if (++loaded < count) {
                page = page_behind;
                if (++ahead.tile < ahead.tiles) {
                    begins = false;
                    row += p.step_rows;
                    at_page += p.step_pages;
                    if (row >= p.c.page_size) {
                        row -= p.c.page_size;
                        ++at_page;
                    }
                    left -= kTile;
                } else {
                    const int n = ahead.n;
                    next_segment(ahead);
                    begins = true;
                    row = own_row;
                    at_page = own_page;
                    left = ahead.len - own;
                    if (ahead.n != n) {
                        table = p.c.block_table + (int64_t)ahead.n * p.c.max_pages;
                        if (left > 0) page = __ldg(table + own_page);
                        warm_table();
                    }
                }
                fetch_behind();
            }
        }
        cp_commit();
    };
    // the unit loaded while unit u is read is u + U - 1: of the other kind if U is even
    auto load_at_k = [&]() { if constexpr (U % 2) load_k(); else load_v(); };
    auto load_at_v = [&]() { if constexpr (U % 2) load_v(); else load_k(); };
    fetch_behind();
    warm_table();
#pragma unroll
    for (int u = 0; u < U - 1; ++u) {
        if (u % 2 == 0) load_k();
        else load_v();
    }

    // ---- the tiles
    float out[NT][D / 16][4], m[NT][2], base[NT][2], l[NT][2];     // base: m, or 0 while m is -inf
    auto reset = [&]() {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt][0] = m[nt][1] = -INFINITY;
            base[nt][0] = base[nt][1] = 0.f;
            l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
            for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
                for (int c = 0; c < 4; ++c) out[nt][mt][c] = 0.f;
        }
    };
    reset();
    int k_unit = 0, at_q = 0, tile_slot = 0;
    // bf16 queries of up to 16 heads stay in registers through their segment
    constexpr bool kHoldQ = kBf16 && NT <= 2;
    uint32_t held_q[kHoldQ ? NT : 1][kHoldQ ? X::kPieces / 4 : 1][4];
    bool from_start = cur.tile == 0;               // the segment begins in this block
    bool first = true;                             // its first tile here
    // this lane's scores of the tile: of head h at h * kTile
    float* scores = p.scores == nullptr ? nullptr
                    : p.scores + t0 * p.GS * kTile + 2 * (lane & 3) * kTile + warp * 16 + (lane >> 2);
#pragma unroll 1
    for (int i = 0; i < count; ++i) {
        const int ar = lane & 15, ax = ar & 7, bx = lane & 7;
        cp_wait<U - 2>();
        // the segment's queries are there, and its predecessor's outputs have been read from the
        // ring; otherwise the warp's own rows are all it needs
        if (first) __syncthreads();
        else __syncwarp();
        load_at_k();                               // into the unit read last: the tile before's V rows
        const uint32_t kd = smem_u32(ring) + k_unit * X::kUnit;
        const uint32_t qd = smem_u32(s_q) + at_q * X::kQ;
        const uint32_t attend = s_live[warp * NQ + tile_slot];
        if (++tile_slot == NQ) tile_slot = 0;
        if constexpr (kHoldQ) {
            if (first) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int ks = 0; ks < X::kPieces / 4; ++ks)
                        ldsm4(qd + (nt * 8 + bx) * X::kRowBytes + (((4 * ks + (lane >> 3)) ^ bx) << 4),
                              held_q[nt][ks]);
            }
        }

        // S^T = K Q^T: rows slots, columns heads. Two accumulators halve the chain; four tiles of
        // heads are chains enough, and need the registers.
        constexpr bool kTwo = NT < 4;
        float s[NT][4], s2[kTwo ? NT : 1][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c) s[nt][c] = s2[kTwo ? nt : 0][c] = 0.f;
        // (fp32's 16 or 8 steps of three products and their splits are kept a loop: unrolled, the
        // tile's code no longer fits the instruction cache)
#pragma unroll (kBf16 ? X::kPieces / 4 : 1)
        for (int ks = 0; ks < X::kPieces / 2; ks += 2) {
            uint32_t a0[4], a1[4];
            ldsm4(kd + ar * X::kRowBytes + (((2 * ks + (lane >> 4)) ^ ax) << 4), a0);
            ldsm4(kd + ar * X::kRowBytes + (((2 * ks + 2 + (lane >> 4)) ^ ax) << 4), a1);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                uint32_t bq[4];
                if constexpr (kHoldQ) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) bq[c] = held_q[nt][ks / 2][c];
                } else {
                    ldsm4(qd + (nt * 8 + bx) * X::kRowBytes + (((2 * ks + (lane >> 3)) ^ bx) << 4), bq);
                }
                if constexpr (kBf16) {
                    mma_bf16(s[nt], a0, bq[0], bq[1]);
                    mma_bf16(kTwo ? s2[kTwo ? nt : 0] : s[nt], a1, bq[2], bq[3]);
                } else {
                    mma_f32(s[nt], a0, bq[0], bq[1]);
                    mma_f32(kTwo ? s2[kTwo ? nt : 0] : s[nt], a1, bq[2], bq[3]);
                }
            }
        }
        const bool ok0 = attend >> (lane >> 2) & 1, ok1 = attend >> ((lane >> 2) + 8) & 1;
        bool above = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                s[nt][c] = (c < 2 ? ok0 : ok1) ? (s[nt][c] + s2[kTwo ? nt : 0][c]) * p.scale_log2 : -INFINITY;
                above |= s[nt][c] > m[nt][c & 1] + kSlack;
            }
            if (scores != nullptr) {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (nt * 8 + 2 * (lane & 3) + (c & 1) < p.GS)
                        scores[(nt * 8 + (c & 1)) * kTile + 8 * (c >> 1)] = s[nt][c];
            }
        }
        if (scores != nullptr) scores += p.GS * kTile;
        // The running maximum moves only when a score passes it by kSlack: until then the weights
        // stay below 2^kSlack, as exact as below 1, and no lane has to ask the others.
        if (__any_sync(0xffffffffu, above)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float corr[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float mx = fmaxf(s[nt][e], s[nt][e + 2]);
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                    const float mn = fmaxf(m[nt][e], mx);
                    base[nt][e] = mn == -INFINITY ? 0.f : mn;
                    corr[e] = exp2_fast(m[nt][e] - base[nt][e]);
                    m[nt][e] = mn;
                    l[nt][e] *= corr[e];
                }
#pragma unroll
                for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
                    for (int c = 0; c < 4; ++c) out[nt][mt][c] *= corr[c & 1];
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                s[nt][c] = exp2_fast(s[nt][c] - base[nt][c & 1]);
                l[nt][c & 1] += s[nt][c];
            }
        // O^T += V^T P^T: rows channels, columns heads
        cp_wait<U - 2>();
        __syncwarp();
        load_at_v();                               // into the tile's K rows
        if (++k_unit == U) k_unit = 0;
        const int v_unit = k_unit;
        if (++k_unit == U) k_unit = 0;
        const uint32_t vd = smem_u32(ring) + v_unit * X::kUnit;
        if constexpr (kBf16) {
            uint32_t ph[NT][2], pl[NT][2];                         // P = hi + lo, both bf16
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float x = s[nt][2 * e], y = s[nt][2 * e + 1];
                    const __nv_bfloat162 hi = __floats2bfloat162_rn(x, y);
                    const float2 f = __bfloat1622float2(hi);
                    const __nv_bfloat162 lo = __floats2bfloat162_rn(x - f.x, y - f.y);
                    ph[nt][e] = transpose8x8(*reinterpret_cast<const uint32_t*>(&hi));
                    pl[nt][e] = transpose8x8(*reinterpret_cast<const uint32_t*>(&lo));
                }
            const int vr = (lane & 7) + 8 * (lane >> 4);
#pragma unroll
            for (int mt = 0; mt < D / 16; ++mt) {
                uint32_t a[4];
                ldsm4_t(vd + vr * X::kRowBytes + (((2 * mt + ((lane >> 3) & 1)) ^ (vr & 7)) << 4), a);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float t[4] = {0.f, 0.f, 0.f, 0.f};             // the step's own sum
                    mma_bf16(t, a, pl[nt][0], pl[nt][1]);
                    mma_bf16(t, a, ph[nt][0], ph[nt][1]);
#pragma unroll
                    for (int c = 0; c < 4; ++c) out[nt][mt][c] += t[c];
                }
            }
        } else {
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {                 // 8 slots each
                uint32_t pb[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {                  // slot lane % 4 + 4 e, head lane / 4
                        const int from = ((lane & 3) + 4 * e) * 4 + (lane >> 3);
                        const float u = __shfl_sync(0xffffffffu, half ? s[nt][2] : s[nt][0], from);
                        const float v = __shfl_sync(0xffffffffu, half ? s[nt][3] : s[nt][1], from);
                        pb[nt][e] = __float_as_uint((lane >> 2) & 1 ? v : u);
                    }
                // a lane's D / 8 channels in a row, of slots lane % 4 and 4 on: two pieces each at a
                // time make the rows of two of the products
                const int r = 8 * half + (lane & 3);
                const uint8_t* v0 = ring + v_unit * X::kUnit + r * X::kRowBytes;
#pragma unroll
                for (int pc = 0; pc < D / 32; ++pc) {
                    const int at = (lane >> 2) * (D / 32) + pc;
                    const uint4 x = *reinterpret_cast<const uint4*>(v0 + ((at ^ (r & 7)) << 4));
                    const uint4 y = *reinterpret_cast<const uint4*>(
                        v0 + 4 * X::kRowBytes + ((at ^ ((r + 4) & 7)) << 4));
                    const uint32_t a0[4] = {x.x, x.y, y.x, y.y}, a1[4] = {x.z, x.w, y.z, y.w};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma_f32(out[nt][2 * pc], a0, pb[nt][0], pb[nt][1]);
                        mma_f32(out[nt][2 * pc + 1], a1, pb[nt][0], pb[nt][1]);
                    }
                }
            }
        }

        // ---- the segment's end, or the block's
        const bool to_end = cur.tile + 1 == cur.tiles;
        if (to_end || i + 1 == count) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], o);
                    if (lane < 4) {
                        s_m[warp * 8 * NT + nt * 8 + 2 * lane + e] = m[nt][e];
                        s_l[warp * 8 * NT + nt * 8 + 2 * lane + e] = l[nt][e];
                    }
                }
            const bool whole = from_start && to_end;
            // a part that began earlier, or spans the block, is its first; one that goes on its last
            float* part = p.parts + (int64_t)(2 * b + (from_start ? 1 : 0)) * X::kPart;
            const int64_t row0 = (int64_t)cur.n * p.Hq + cur.hkv * p.G + cur.gt * 8 * NT;   // of q, z, o
            const int live_heads = p.G - cur.gt * 8 * NT;
            // One tile of 8 heads after the other: the warps put their outputs where their V rows
            // were, and each sums an eighth or a quarter of the registers, weighted by its own
            // maximum and the block's.
            constexpr int kRound = D / 4, kShare = kRound / W;
            float* mine = reinterpret_cast<float*>(ring + v_unit * X::kUnit) + lane;
            const float* theirs = reinterpret_cast<const float*>(s_ring + v_unit * X::kUnit) + lane;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                if (nt == 0) __syncwarp();         // every lane has read its V rows
                else __syncthreads();
#pragma unroll
                for (int r = 0; r < kRound; ++r) mine[r * 32] = out[nt][r >> 2][r & 3];
                float z[kShare];
                if (whole) load_gate<T, D, kShare>(p, row0, live_heads, nt * kRound + warp * kShare, lane, z);
                __syncthreads();
                float f[W][2], sum[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int h = nt * 8 + 2 * (lane & 3) + e;
                    float mx = -INFINITY, sm = 0.f;
#pragma unroll
                    for (int w = 0; w < W; ++w) mx = fmaxf(mx, s_m[w * 8 * NT + h]);
                    const float top = mx == -INFINITY ? 0.f : mx;
#pragma unroll
                    for (int w = 0; w < W; ++w) {
                        f[w][e] = exp2_fast(s_m[w * 8 * NT + h] - top);
                        sm += s_l[w * 8 * NT + h] * f[w][e];
                    }
                    sum[e] = sm > 0.f ? 1.f / sm : 0.f;
                    if (warp == 0 && lane < 4) {
                        if (!whole) {
                            part[X::kRegs * 32 + h] = mx;
                            part[X::kRegs * 32 + 8 * NT + h] = sm;
                        } else if (p.stats != nullptr && h < live_heads) {
                            p.stats[row0 + h] = make_float2(top, sum[e]);
                        }
                    }
                }
                float y[kShare];
#pragma unroll
                for (int u = 0; u < kShare; ++u) {
                    const int r = warp * kShare + u;
                    y[u] = 0.f;
#pragma unroll
                    for (int w = 0; w < W; ++w) y[u] += theirs[w * (U * X::kUnit / 4) + r * 32] * f[w][u & 1];
                }
                if (!whole) {
#pragma unroll
                    for (int u = 0; u < kShare; ++u) part[(nt * kRound + warp * kShare + u) * 32 + lane] = y[u];
                } else {
                    store_out<T, D, kShare>(p, row0, live_heads, nt * kRound + warp * kShare, lane, y, z, sum);
                }
            }
            if (!whole && from_start && tid == 0) {            // this block's last: join it with the next ones'
                const int64_t last = t0 + i + (cur.tiles - 1 - cur.tile);
                p.meta[4 * b] = cur.n;
                p.meta[4 * b + 1] = cur.hkv * p.GT + cur.gt;
                p.meta[4 * b + 2] = split_block_of(all_tiles, C, last);
            }
            reset();
            if (++at_q == NQ) at_q = 0;
            from_start = true;
        }
        first = to_end;
        if (!to_end) ++cur.tile;
        else if (i + 1 < count) next_segment(cur);
    }
    cp_wait<0>();
    grid_release();
}

constexpr int kJoinWarps = 8, kJoinPerSm = 3, kFew = 8;

// acc[n, h, j] += sum over the group's heads of exp2(score - max) / sum: 1024 slots of one head a
// block, four a thread. The maximum and sum of a segment that spans blocks come from its parts, so
// this does not wait for the join of the outputs and shares its launch.
constexpr int kWeightSlots = 4 * kJoinWarps * 32;
template <typename T, int D, int NT>
__device__ __forceinline__ void gather_weights(const Params& p, int block, int blocks, float2* s_stat) {
    using X = Shape<T, D, NT>;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int chunks = (p.max_len + kWeightSlots - 1) / kWeightSlots;
    const int64_t all = (int64_t)p.N * p.H * chunks;
    for (int64_t w = block; w < all; w += blocks) {
        const int64_t nh = split_div(w, chunks), n = (uint32_t)nh / (uint32_t)p.H;     // nh < 2^31
        const int chunk = (int)(w - nh * chunks), h = (int)(nh - n * p.H);
        const int j = chunk * kWeightSlots + tid * 4;
        const int len = checked_len(__ldg(p.seqlens + n), p.max_len, p.c.err);
        const int64_t before = p.whole > 0 ? 0 : p.tiles_before[n];
        const int64_t work = p.whole > 0 ? 1 : (int64_t)p.tiles_before[p.N] * p.H * p.GT;
        if (chunk * kWeightSlots >= len) continue;                 // the whole block agrees
        float* acc = p.acc + nh * p.slots + j;
        float old[4], sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int u = 0; u < 4; ++u) old[u] = j + u < len ? acc[u] : 0.f;
        const int tiles = p.whole > 0 ? p.whole : (len + X::kTile - 1) / X::kTile;
        const int C = split_blocks(work, p.most_blocks);
        // the head's first tile
        const int64_t seg = (p.whole > 0 ? nh * tiles : before * p.H + (int64_t)h * tiles) * p.GT;
        for (int gt = 0; gt < p.GT; ++gt) {
            const int64_t t0 = seg + (int64_t)gt * tiles;
            const int b0 = p.whole > 0 ? 0 : split_block_of(work, C, t0);
            const int k = p.whole > 0 ? 1 : split_block_of(work, C, t0 + tiles - 1) - b0 + 1;
            const int heads = min(8 * NT, p.G - gt * 8 * NT);
            // four heads' scores are on their way while the statistics are formed
            const float* s = p.scores + (t0 + j / X::kTile) * p.GS * X::kTile + j % X::kTile;
            float4 x[4];
            if (j < len) {
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    if (g < heads) x[g] = *reinterpret_cast<const float4*>(s + g * X::kTile);
            }
            __syncthreads();                                       // the stats before have been read
            for (int g = warp; g < heads; g += kJoinWarps) {       // a warp a head
                if (k == 1) {
                    if (lane == 0) s_stat[g] = p.stats[n * p.Hq + h * p.G + gt * 8 * NT + g];
                    continue;
                }
                float m = -INFINITY, l = 0.f;                      // over the lane's parts
                for (int i = lane; i < k; i += 32) {
                    const float* ml = p.parts + (int64_t)(i == 0 ? 2 * b0 + 1 : 2 * (b0 + i)) * X::kPart +
                                      X::kRegs * 32 + g;
                    const float mi = ml[0], mn = fmaxf(m, mi), base = mn == -INFINITY ? 0.f : mn;
                    l = l * exp2_fast(m - base) + ml[8 * NT] * exp2_fast(mi - base);
                    m = mn;
                }
                float top = m;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                const float base = top == -INFINITY ? 0.f : top;
                l = warp_sum(l * exp2_fast(m - base));
                if (lane == 0) s_stat[g] = make_float2(base, l > 0.f ? 1.f / l : 0.f);
            }
            __syncthreads();
            if (j >= len) continue;
            for (int g0 = 0; g0 < heads; g0 += 4) {
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    if (g0 + g >= heads) break;
                    const float2 t = s_stat[g0 + g];
                    sum[0] = fmaf(exp2_fast(x[g].x - t.x), t.y, sum[0]);
                    sum[1] = fmaf(exp2_fast(x[g].y - t.x), t.y, sum[1]);
                    sum[2] = fmaf(exp2_fast(x[g].z - t.x), t.y, sum[2]);
                    sum[3] = fmaf(exp2_fast(x[g].w - t.x), t.y, sum[3]);
                    if (g0 + 4 + g < heads) x[g] = *reinterpret_cast<const float4*>(s + (g0 + 4 + g) * X::kTile);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (j + u < len) acc[u] = old[u] + sum[u];
    }
}

// Joins the parts of every segment that spans blocks, by two kinds of work items:
//  - up to kFew parts (many segments then): a tile of 8 heads of a segment; each of eight warps
//    takes an eighth of its output registers, of all parts at once;
//  - more parts (one long sequence leaves a hundred to each of its heads): two registers of a
//    segment; the warps take every eighth part. 148 parts of 2 heads: 18.6 us with items of eight
//    registers, 9.8 us with these.
// The blocks from join_blocks on gather the weights instead.
template <int NT>
struct JoinShared {
    float2 stat[8 * NT];
    float f[kMaxBlocks][8], l[kMaxBlocks][8];
    float few[kFew][8];
    float sum[8];
    float o[kJoinWarps][2][32];
    int4 list[kMaxBlocks];                     // n, head, last block, first block
    int count[(kMaxBlocks + kJoinWarps * 32 - 1) / (kJoinWarps * 32)][2][kJoinWarps];
};

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kJoinWarps * 32, kJoinPerSm) paged_join_kernel(const Params p, int join_blocks) {
    using X = Shape<T, D, NT>;
    constexpr int kThreads = kJoinWarps * 32, kShare = D / 4 / kJoinWarps, kPairs = X::kRegs / 2;
    __shared__ JoinShared<NT> sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    grid_wait();
    if ((int)blockIdx.x >= join_blocks) {
        gather_weights<T, D, NT>(p, blockIdx.x - join_blocks, gridDim.x - join_blocks, sh.stat);
        return;
    }
    // the blocks whose last segment goes on: those of few parts from the list's start, of many
    // from its end
    constexpr int kEach = (kMaxBlocks + kThreads - 1) / kThreads;
    int4 meta[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int b = i * kThreads + tid;
        meta[i] = make_int4(0, 0, -1, 0);
        if (b < p.most_blocks) meta[i] = *reinterpret_cast<const int4*>(p.meta + 4 * b);
        meta[i].w = b;
    }
    int few = 0, many = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const bool open = meta[i].z >= 0, is_few = open && meta[i].z - meta[i].w < kFew;
        const unsigned mf = __ballot_sync(0xffffffffu, is_few), mm = __ballot_sync(0xffffffffu, open && !is_few);
        if (lane == 0) {
            sh.count[i][0][warp] = __popc(mf);
            sh.count[i][1][warp] = __popc(mm);
        }
        __syncthreads();
        int at_few = few + __popc(mf & ((1u << lane) - 1)), at_many = many + __popc(mm & ((1u << lane) - 1));
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) {
            if (w < warp) {
                at_few += sh.count[i][0][w];
                at_many += sh.count[i][1][w];
            }
            few += sh.count[i][0][w];
            many += sh.count[i][1][w];
        }
        if (open) sh.list[is_few ? at_few : kMaxBlocks - 1 - at_many] = meta[i];
    }
    __syncthreads();
    auto part = [&](int b, int j) { return p.parts + (int64_t)(j == 0 ? 2 * b + 1 : 2 * (b + j)) * X::kPart; };

    for (int w = blockIdx.x; w < few * NT + many * kPairs; w += join_blocks) {
        const bool pair = w < many * kPairs;
        const int4 open = pair ? sh.list[kMaxBlocks - 1 - w / kPairs] : sh.list[(w - many * kPairs) / NT];
        const int n = open.x, hkv = open.y / p.GT, gt = open.y % p.GT, b = open.w, k = open.z - b + 1;
        const int64_t row0 = (int64_t)n * p.Hq + hkv * p.G + gt * 8 * NT;
        const int live_heads = p.G - gt * 8 * NT;
        const float ones[2] = {1.f, 1.f};
        __syncthreads();                       // the item before has been read
        if (!pair) {
            const int nt = (w - many * kPairs) % NT, r0 = nt * (D / 4) + warp * kShare;
            if (nt * 8 >= live_heads) continue;
            float x[kFew][kShare], y[kShare], z[kShare];           // all parts on their way at once
            load_gate<T, D, kShare>(p, row0, live_heads, r0, lane, z);
#pragma unroll
            for (int j = 0; j < kFew; ++j)
#pragma unroll
                for (int r = 0; r < kShare; ++r) x[j][r] = j < k ? part(b, j)[(r0 + r) * 32 + lane] : 0.f;
            if (tid < 8) {                     // factors exp2(m - max) / sum of each part
                float m[kFew], l[kFew], mx = -INFINITY, sm = 0.f;
#pragma unroll
                for (int j = 0; j < kFew; ++j) {
                    m[j] = j < k ? part(b, j)[X::kRegs * 32 + nt * 8 + tid] : -INFINITY;
                    l[j] = j < k ? part(b, j)[X::kRegs * 32 + 8 * NT + nt * 8 + tid] : 0.f;
                    mx = fmaxf(mx, m[j]);
                }
                const float base = mx == -INFINITY ? 0.f : mx;
#pragma unroll
                for (int j = 0; j < kFew; ++j) {
                    m[j] = exp2_fast(m[j] - base);
                    sm += m[j] * l[j];
                }
                const float inv = sm > 0.f ? 1.f / sm : 0.f;
#pragma unroll
                for (int j = 0; j < kFew; ++j) sh.few[j][tid] = m[j] * inv;
            }
            __syncthreads();
#pragma unroll
            for (int r = 0; r < kShare; ++r) {
                y[r] = 0.f;
#pragma unroll
                for (int j = 0; j < kFew; ++j) y[r] += x[j][r] * sh.few[j][2 * (lane & 3) + (r & 1)];
            }
            store_out<T, D, kShare>(p, row0, live_heads, r0, lane, y, z, ones);
            continue;
        }
        const int r0 = w % kPairs * 2, nt = r0 / (D / 4);
        float z[1];
        if (warp < 2) load_gate<T, D, 1>(p, row0, live_heads, r0 + warp, lane, z);
        for (int e = tid; e < k * 8; e += kThreads) {
            const float* ml = part(b, e >> 3) + X::kRegs * 32 + nt * 8 + (e & 7);
            sh.f[e >> 3][e & 7] = ml[0];
            sh.l[e >> 3][e & 7] = ml[8 * NT];
        }
        __syncthreads();
        {                                      // a warp a head: the maximum, then factors and sum
            float mx = -INFINITY, sm = 0.f;
            for (int j = lane; j < k; j += 32) mx = fmaxf(mx, sh.f[j][warp]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const float base = mx == -INFINITY ? 0.f : mx;
            for (int j = lane; j < k; j += 32) {
                const float f = exp2_fast(sh.f[j][warp] - base);
                sh.f[j][warp] = f;
                sm += f * sh.l[j][warp];
            }
            sm = warp_sum(sm);
            if (lane == 0) sh.sum[warp] = sm > 0.f ? 1.f / sm : 0.f;
        }
        __syncthreads();
        float y0 = 0.f, y1 = 0.f;
#pragma unroll 16
        for (int j = warp; j < k; j += kJoinWarps) {
            const float* src = part(b, j) + r0 * 32 + lane;
            y0 += src[0] * sh.f[j][2 * (lane & 3)];
            y1 += src[32] * sh.f[j][2 * (lane & 3) + 1];
        }
        sh.o[warp][0][lane] = y0;
        sh.o[warp][1][lane] = y1;
        __syncthreads();
        if (warp < 2) {
            float v = 0.f;
#pragma unroll
            for (int u = 0; u < kJoinWarps; ++u) v += sh.o[u][warp][lane];
            int h, ch;
            part_coord<T, D>(r0 + warp, lane, h, ch);
            const float one[1] = {v * sh.sum[h & 7]};
            store_out<T, D, 1>(p, row0, live_heads, r0 + warp, lane, one, z, ones);
        }
    }
}

// NT for a group of G heads: one tile of 8, two, or four (fp32: two at most, for its ring).
int head_tiles(int64_t G, bool bf16) { return G <= 8 ? 1 : (G <= 16 || !bf16) ? 2 : 4; }

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

struct Layout {
    size_t meta, parts, tiles_before, stats, scores, total;
};
Layout layout(int64_t N, int64_t Hq, int64_t H, int64_t max_len, bool with_acc, int NT, size_t part_floats) {
    const int64_t G = Hq / H, GT = (G + 8 * NT - 1) / (8 * NT), GS = G < 8 * NT ? G : 8 * NT;
    Layout l;
    l.meta = 0;
    l.parts = up256(kMaxBlocks * 4 * sizeof(int));
    l.tiles_before = l.parts + up256(2 * kMaxBlocks * part_floats * sizeof(float));
    l.stats = l.tiles_before + (with_acc ? up256((N + 1) * sizeof(int)) : 0);
    l.scores = l.stats + (with_acc ? up256(N * Hq * sizeof(float2)) : 0);
    const int64_t padded = (max_len + 127) / 128 * 128;          // whole tiles of 64 or 128 slots
    l.total = l.scores + (with_acc ? (size_t)(N * H * GT) * padded * GS * sizeof(float) : 0);
    return l;
}

template <typename T, int D, int NT>
cudaError_t launch_t(const DecodeArgs& a, cudaStream_t stream) {
    using X = Shape<T, D, NT>;
    const int sms = sm_count();
    if (sms == 0) return cudaErrorInvalidDevice;
    const Layout l = layout(a.N, a.Hq, a.H, a.max_len, a.acc != nullptr, NT, X::kPart);
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    Params p;
    p.c = a.c;
    p.page16 = (uint32_t)(a.c.page_stride * (int64_t)sizeof(T) / 16);
    p.slot16 = (uint32_t)(a.c.slot_stride * (int64_t)sizeof(T) / 16);
    p.head16 = (uint32_t)(a.c.head_stride * (int64_t)sizeof(T) / 16);
    p.step_pages = X::kTile / a.c.page_size;
    p.step_rows = X::kTile % a.c.page_size;
    p.q = a.q; p.z = a.z;
    p.seqlens = a.seqlens;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.o = a.o;
    p.N = a.N; p.Hq = a.Hq; p.H = a.H;
    p.G = a.Hq / a.H;
    p.GT = (p.G + 8 * NT - 1) / (8 * NT);
    p.max_len = a.max_len;
    p.most_blocks = sms * X::kPerSm < kMaxBlocks ? sms * X::kPerSm : kMaxBlocks;
    p.meta = reinterpret_cast<int*>(ws + l.meta);
    p.parts = reinterpret_cast<float*>(ws + l.parts);
    p.tiles_before = a.acc ? reinterpret_cast<int*>(ws + l.tiles_before) : nullptr;
    p.stats = a.acc ? reinterpret_cast<float2*>(ws + l.stats) : nullptr;
    p.scores = a.acc ? reinterpret_cast<float*>(ws + l.scores) : nullptr;
    p.GS = p.G < 8 * NT ? p.G : 8 * NT;
    p.acc = a.acc;
    p.slots = a.slots;
    // pages of a multiple of 16 slots, the common ones, need one page number a warp and no exchange
    // of row addresses between lanes
    const bool runs = a.c.page_size % 16 == 0;
    auto kernel = runs ? paged_decode_kernel<T, D, NT, true> : paged_decode_kernel<T, D, NT, false>;
    cudaError_t e = allow_smem(kernel, X::kSmem);
    if (e != cudaSuccess) return e;
    // Short segments, no more than blocks, are a block each: the scan of the lengths and the joins
    // cost as much as some tiles, more than dividing gains while t tiles in sequence are no more
    // than that above the t S / C of a divided block. Of bf16's tiles it is five, of fp32's, which take
    // longer, three and a half with rows of 256 bytes and two and a half with 512. Whole and divided,
    // us, 8 segments: bf16, 128 channels, 4 tiles 11.4 and 13.6, 8 tiles 15.4 and 13.6; fp32, 64
    // channels, 3 tiles 11.3 and 13.1, 5 tiles 14.8 and 13.1; fp32, 128 channels, 2 tiles 13.5 and 14.8,
    // 4 tiles 19.3 and 15.0 (16 heads: 24.4 and 18.9). 128 segments of 8 tiles: 15.5 and 21.0, 18.9 and
    // 22.9, 34.8 and 41.6. With weights gathered the whole form gains 2 to 4 us less; the rule does not
    // go by that, so that the outputs are the same with them and without. max_len may be far above
    // the lengths, whose balance the division keeps: 16 at most.
    const int64_t segments = (int64_t)a.N * a.H * p.GT, blocks = p.most_blocks;
    const int64_t t = (a.max_len + X::kTile - 1) / X::kTile;
    const int half_tiles = X::kBf16 ? 10 : X::kRowBytes == 256 ? 7 : 5;
    p.whole = segments <= blocks && t <= 16 && 2 * t * (blocks - segments) <= half_tiles * blocks ? (int)t : 0;
    kernel<<<p.whole > 0 ? (unsigned)segments : p.most_blocks, X::W * 32, X::kSmem, stream>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if (p.whole > 0 && a.acc == nullptr) return cudaSuccess;
    int join_blocks = sms * kJoinPerSm;
    int64_t weight_blocks = 0;
    if (a.acc != nullptr) {
        weight_blocks = (int64_t)a.N * a.H * ((a.max_len + kWeightSlots - 1) / kWeightSlots);
        if (weight_blocks > sms * kJoinPerSm) weight_blocks = sms * kJoinPerSm;
        join_blocks = p.whole > 0 ? 0 : join_blocks / 2;
    }
    return launch_after(paged_join_kernel<T, D, NT>, dim3(join_blocks + (unsigned)weight_blocks),
                        kJoinWarps * 32, stream, p, join_blocks);
}

template <typename T, int D>
cudaError_t launch_d(const DecodeArgs& a, cudaStream_t stream) {
    switch (head_tiles(a.Hq / a.H, sizeof(T) == 2)) {
        case 1: return launch_t<T, D, 1>(a, stream);
        case 2: return launch_t<T, D, 2>(a, stream);
    }
    if constexpr (sizeof(T) == 2) return launch_t<T, D, 4>(a, stream);
    return cudaErrorInvalidValue;
}

}  // namespace

bool paged_decode_workspace(int64_t N, int64_t Hq, int64_t H, int d, int64_t max_len, bool with_acc,
                            size_t* bytes) {
    const double scores = (double)N * H * (Hq / H + 32) * (max_len + 128) * 4;
    // tiles of all sequences count in 31 bits
    if (N * Hq > INT32_MAX || N * (max_len / 64 + 1) > INT32_MAX || scores > 4e18) return false;
    size_t most = 0;                     // whichever io: bf16 and fp32 differ in their head tiles
    for (bool bf16 : {false, true}) {
        const int NT = head_tiles(Hq / H, bf16);
        const size_t t = layout(N, Hq, H, max_len, with_acc, NT, (size_t)(d / 4 * 32 + 16) * NT).total;
        if (t > most) most = t;
    }
    *bytes = most;
    return true;
}

cudaError_t launch_paged_decode(const DecodeArgs& a, cudaStream_t stream) {
    if (a.N == 0) return cudaSuccess;
    if (a.io == Io::BF16)
        return a.d == 128 ? launch_d<__nv_bfloat16, 128>(a, stream) : launch_d<__nv_bfloat16, 64>(a, stream);
    return a.d == 128 ? launch_d<float, 128>(a, stream) : launch_d<float, 64>(a, stream);
}

}  // namespace kda
