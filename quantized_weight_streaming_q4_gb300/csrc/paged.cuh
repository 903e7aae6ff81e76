// paged.cuh -- what the kernels of attention over a paged cache share: the
// call's arguments, the split of the work, and the joining of partial results.
//
// The lengths of the sequences are known on the device only.  An item is one
// token row, one K/V head and up to 16 of its query heads; its work are the
// tiles of TILE positions that hold rows it sees.  Every block finds the same
// split for itself, in one of two ways:
//  - few tiles a block: each item is cut into pieces of up to `chunk` tiles, one
//    a block.  Joining the results of an item's blocks costs about as much as
//    four tiles, so where no item has more than four, all are left whole; else
//    all are cut, with the smallest chunk for which there are blocks.
//  - else all items' tiles in a row are cut into as many equal runs as there are
//    blocks, so that a run may end inside an item.  An item counts as some tiles
//    more than it has, for what a block spends on its start and its end: two
//    up to 8 query rows, four for 16 (16 sequences of 500 to 40,000 rows, 16
//    query rows: 43.5 us with two, 39.8 with four; 48 sequences of 30 to 1,500
//    rows, four query rows: 25.7 and 26.7).
// The blocks of an item leave partial results, and the last of them to finish
// joins these in the items' order (of more than 16, in groups first).  No
// block waits for another.
#pragma once

#include "attn_parts.cuh"
#include "pages.cuh"

namespace muser {

constexpr int kPagedMaxBlocks = 160;   // blocks of a launch: one an SM
constexpr size_t kPagedTicketBytes = 2048;
static_assert(kPagedTicketBytes >= 3 * kPagedMaxBlocks * sizeof(unsigned), "a ticket for each block's item and two for its parts");
constexpr int kPagedRows = 16;         // query rows of an item, at most

struct PagedArgs {
    uint16_t *key, *value;
    int64_t page_stride, row_stride, head_stride;  // in elements
    int32_t pages, page_rows, page_shift;          // page_shift: log2(page_rows), where it is one
    const int32_t* table;
    int64_t stride;
    int32_t n_tables, rows_end;  // rows_end: positions that the table has entries for
    const int32_t *position, *sequence;
    const float *q, *k, *v, *gate;
    float* out;
    int n, H, G, D, group, blocks_per_head;
    int32_t window, n_sink;  // window 0: all rows
    float scale_log2;
    unsigned* ticket;  // [2 * blocks] of eight parts, at the first one's place; [blocks] of an item, at its first block's
    float2* part_ml;   // [2 * blocks][16]: maximum (base 2) and sum
    float* part_o;     // [2 * blocks][16][D]
    unsigned* status;
};

// paged_tc.cu
bool paged_tc_supported(const PagedArgs& a);
int launch_paged_tc(const PagedArgs& a, int blocks, cudaStream_t s);

namespace {

// The rows that the token at position t sees, by TILE positions: [0, sink) and
// [low, end), and itself.  Tile i of the `tiles` covers positions from
// first(i) * TILE on.
template <int TILE>
struct Sight {
    int t, end, low, sink, lead, tail0, tiles;
    __device__ __forceinline__ Sight(const PagedArgs& a, int pos) : t(pos) {
        end = a.k ? min(pos, a.rows_end) : min(pos, a.rows_end - 1) + 1;  // pos may be the largest int32
        low = a.window > 0 ? min(max(0, pos - a.window + 1), end) : 0;
        sink = min(a.n_sink, low);
        lead = (sink + TILE - 1) / TILE;
        tail0 = max(low / TILE, lead);
        tiles = max(1, lead + max(0, (end + TILE - 1) / TILE - tail0));
    }
    __device__ __forceinline__ int first(int i) const { return i < lead ? i : tail0 + i - lead; }
    __device__ __forceinline__ bool sees(int p) const { return p < end && (p < sink || p >= low); }
    // rows of the tile from position p0 on, up to the last one that is seen
    __device__ __forceinline__ int real(int p0) const {
        const int last = p0 + TILE <= low ? sink : end;
        return min(TILE, max(0, last - p0));
    }
};

// The split: positions (-1: no work) and the units before each token row,
// tiles (chunk 0) or pieces of up to `chunk` tiles, in shared memory; the rest
// in every warp's registers.
struct PagedPlan {
    int32_t t[kMaxSequences];
    uint32_t before[kMaxSequences + 1];
};
constexpr int kMostChunk = 8, kWholeTiles = 4;
__device__ __forceinline__ uint32_t over(const PagedArgs& a) { return a.group > 8 ? 4u : 2u; }

__device__ __forceinline__ uint32_t ceil_div(uint32_t x, uint32_t y) { return (x + y - 1) / y; }

// x / y for x < 2^24 and a quotient below 2^20, by way of binary32.
__device__ __forceinline__ uint32_t quotient(uint32_t x, uint32_t y) {
    uint32_t q = __float2uint_rz(__fdividef(static_cast<float>(x), static_cast<float>(y)));
    const int r = static_cast<int>(x - q * y);  // the quotient is one off at most
    return r < 0 ? q - 1 : r >= static_cast<int>(y) ? q + 1 : q;
}

// A block's share [at, end) of `total` < 2^24 units; blocks behind the units'
// number have none.
struct PagedShare {
    uint32_t total, blocks, at, end;
    PagedShare() = default;
    __device__ __forceinline__ explicit PagedShare(uint32_t units) : total(units), at(0), end(0) {
        blocks = min(total, gridDim.x);
        if (blockIdx.x >= blocks) return;
        if (total == blocks) {
            at = blockIdx.x;
            end = at + 1;
        } else {
            at = total * blockIdx.x / blocks;
            end = total * (blockIdx.x + 1) / blocks;
        }
    }
};

struct PagedSplit {
    PagedShare share;
    uint32_t chunk, shift;  // shift: a unit is 2^shift tiles (0 unless a call has more than 2^23)
    int first_row;          // that the block's first unit is of
};

// The position of token row i, -1 where it has no work.
__device__ __forceinline__ int position_of(const PagedArgs& a, int i) {
    if (i >= a.n) return -1;
    const int t = __ldcg(a.position + i), s = a.sequence ? __ldcg(a.sequence + i) : i;
    return s >= 0 && s < a.n_tables ? t : -1;
}

// The chunk for sums of pieces, lane c's those of chunk c (lane 0: the longest
// row's tiles), or 0, and what makes 2^23 units at most.
__device__ __forceinline__ void choose_units(const PagedArgs& a, uint32_t sum, PagedSplit& split) {
    const int lane = threadIdx.x & 31;
    const uint64_t all = static_cast<uint64_t>(sum) * static_cast<uint32_t>(a.G * a.blocks_per_head);
    const uint32_t fit = __ballot_sync(0xffffffffu, lane > 0 && lane <= kMostChunk && all <= gridDim.x);
    split.chunk = fit == 0 ? 0 : __ffs(fit) - 1;
    if (split.chunk > 0 && __shfl_sync(0xffffffffu, sum, 0) <= kWholeTiles) split.chunk = kWholeTiles;
    const uint32_t high = __shfl_sync(0xffffffffu, static_cast<uint32_t>(all >> 23), 1);
    split.shift = high == 0 ? 0 : 32 - __clz(high);
}

// Fills the plan; all of the block's threads (256) call it.  Up to 32 token
// rows every warp does it for itself, without a barrier; `warp_sums`: 80 words
// of shared memory for more.
template <int TILE>
__device__ __forceinline__ PagedSplit make_plan(const PagedArgs& a, PagedPlan& plan, uint32_t* warp_sums) {
    static_assert(kMaxSequences == 256, "a thread a token row");
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const bool one = a.n <= 32;
    const int i = one ? lane : tid;
    const int t = position_of(a, i);
    const uint32_t mine = t >= 0 ? static_cast<uint32_t>(Sight<TILE>(a, t).tiles) : 0;
    uint32_t sum = __reduce_max_sync(0xffffffffu, mine);  // lane 0; lane c: pieces of chunk c
#pragma unroll
    for (uint32_t c = 1; c <= kMostChunk; ++c) {
        const uint32_t x = __reduce_add_sync(0xffffffffu, ceil_div(mine, c));
        if (lane == static_cast<int>(c)) sum = x;
    }
    if (!one) {
        if (lane <= kMostChunk) warp_sums[w * 10 + lane] = sum;
        __syncthreads();
        sum = 0;
        if (lane <= kMostChunk)
            for (int j = 0; j < 8; ++j) sum = lane == 0 ? max(sum, warp_sums[j * 10]) : sum + warp_sums[j * 10 + lane];
        __syncthreads();
    }
    PagedSplit split;
    choose_units(a, sum, split);
    const uint32_t units = mine == 0          ? 0
                           : split.chunk == 0 ? ((mine + (1u << split.shift) - 1) >> split.shift) + over(a)
                                              : quotient(mine + split.chunk - 1, split.chunk);
    uint32_t v = units;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += x;
    }
    uint32_t all = __shfl_sync(0xffffffffu, v, 31);
    if (!one) {
        if (lane == 31) warp_sums[w] = v;
        __syncthreads();
        all = 0;
        for (int j = 0; j < 8; ++j) {
            if (j == w) v += all;
            all += warp_sums[j];
        }
    }
    // every warp writes the same where `one`
    plan.t[i] = t;
    plan.before[i] = v - units;
    if (one ? lane == 31 : tid == 255) plan.before[i + 1] = v;
    const uint32_t per = static_cast<uint32_t>(a.G * a.blocks_per_head);
    split.share = PagedShare(all * per);
    const bool here = (v - units) * per <= split.share.at && split.share.at < v * per;
    if (one) {
        split.first_row = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
        __syncwarp();
    } else {
        if (here) warp_sums[16] = i;
        __syncthreads();
        split.first_row = static_cast<int>(warp_sums[16]);
    }
    return split;
}

// A run of one item's tiles.
struct PagedRun {
    int row, head, r0;    // token row, K/V head, first of its query heads
    int a, b, tiles;      // tiles [a, b) of `tiles`
    uint32_t u0, units;   // the item's first unit, and their number
    __device__ __forceinline__ bool whole() const { return a == 0 && b == tiles; }
};

// The block's runs, one after another.
template <int TILE>
struct PagedWalk {
    PagedShare share;
    uint32_t per, chunk, shift, extra;  // per: items of a token row; extra: units of an item before its first tile
    int m;
    __device__ __forceinline__ PagedWalk(const PagedArgs& a, const PagedSplit& split)
        : share(split.share),
          per(static_cast<uint32_t>(a.G * a.blocks_per_head)),
          chunk(split.chunk),
          shift(split.shift),
          extra(split.chunk == 0 ? over(a) : 0),
          m(split.first_row) {}
    // no further run: what is left of the share ends before the next item's first tile
    // (a share is more units than that: more pieces of 8 tiles than blocks make as
    // many units as pieces times one more, at least)
    __device__ __forceinline__ bool last() const { return share.at + extra >= share.end; }
    __device__ __forceinline__ bool next(const PagedArgs& a, const PagedPlan& plan, PagedRun& run) {
        if (last()) return false;
        while (plan.before[m + 1] * per <= share.at) ++m;
        const uint32_t units = plan.before[m + 1] - plan.before[m];  // of an item
        uint32_t sub = share.at - plan.before[m] * per, x = 0;
        if (units > 1) {
            const uint32_t off = sub;
            sub = quotient(off, units);
            x = off - sub * units;
        }
        run.row = m;
        run.units = units;
        run.u0 = share.at - x;
        run.head = static_cast<int>(sub);
        run.r0 = 0;
        if (a.blocks_per_head > 1) {
            run.head = static_cast<int>(sub) / a.blocks_per_head;
            run.r0 = (static_cast<int>(sub) - run.head * a.blocks_per_head) * kPagedRows;
        }
        run.tiles = Sight<TILE>(a, plan.t[m]).tiles;
        if (chunk == 0) {
            const uint32_t x1 = min(units, x + (share.end - share.at));
            run.a = static_cast<int>((max(x, extra) - extra) << shift);
            run.b = min(run.tiles, static_cast<int>((max(x1, extra) - extra) << shift));
            share.at += x1 - x;
            return true;
        }
        run.a = 0;
        run.b = run.tiles;
        if (units > 1) {  // pieces of equal size, the first ones of a tile more
            const int each = static_cast<int>(quotient(run.tiles, units)), rest = run.tiles - each * static_cast<int>(units), i = static_cast<int>(x);
            run.a = i * each + min(i, rest);
            run.b = run.a + each + (i < rest ? 1 : 0);
        }
        ++share.at;
        return true;
    }
    // the first and the last block that have tiles of the run's item
    __device__ __forceinline__ int owner(uint32_t unit) const {
        if (share.total == share.blocks) return static_cast<int>(unit);
        return static_cast<int>(((unit + 1) * share.blocks - 1) / share.total);
    }
    __device__ __forceinline__ int first_block(const PagedRun& run) const { return owner(run.u0 + extra); }
    __device__ __forceinline__ int last_block(const PagedRun& run) const { return owner(run.u0 + run.units - 1); }
};

// The partial result of block `b` of an item's blocks first..last: the block
// where the item begins keeps it in its second place, the others in their first.
__device__ __forceinline__ int part_of(int b, int first) { return 2 * b + (b == first ? 1 : 0); }

__device__ __forceinline__ float gated(float y, float z) { return __fdividef(y, 1.f + __expf(-z)); }

// What the kernels do once a run, or once an item, is written as short loops:
// instructions that an SM does not have at hand cost more than what they do
// (unrolled for sixteen rows, the end of a run took 2.8 us, a join 15).

// A row's float4s, a lane one or (D > 128) two.
template <typename F>
__device__ __forceinline__ void each_piece(int D, int lane, F&& f) {
    for (int d = 4 * lane; d < D; d += 128) f(d);
}
__device__ __forceinline__ float4 scaled(float4 v, float f) { return make_float4(v.x * f, v.y * f, v.z * f, v.w * f); }
__device__ __forceinline__ float4 gated4(float4 v, float4 z) { return make_float4(gated(v.x, z.x), gated(v.y, z.y), gated(v.z, z.z), gated(v.w, z.w)); }

// Parts that are joined at once; more of them in groups first.
constexpr int kJoinMost = 16;
static_assert(kPagedMaxBlocks <= kJoinMost * kJoinMost, "two levels");
// What a join needs, by value: through a reference to the kernel's parameters
// every access went to memory, and a join took 15 us.
struct JoinWork {
    float2* part_ml;
    float* part_o;
    const float* gate;  // of the item's first row, or null
    float* out;
    unsigned* ticket;
    int D, live, first, last;  // first, last: the item's blocks
};
// Whether this was the last of `count` arrivals at a ticket; called by one
// thread, when all threads that wrote what it announces have passed a barrier
// with it (the atomic releases what is ordered before it).
__device__ __forceinline__ bool last_of(unsigned* ticket, int count) {
    const bool last = atom_add_acq_rel_gpu(ticket, 1u) == static_cast<unsigned>(count - 1);
    if (last) *ticket = 0;
    return last;
}

template <int TILE>
__device__ __forceinline__ JoinWork join_work(const PagedArgs& a, const PagedWalk<TILE>& walk, const PagedRun& run) {
    const int64_t at = (static_cast<int64_t>(run.row) * a.H + run.head * a.group + run.r0) * a.D;
    return JoinWork{a.part_ml, a.part_o, a.gate ? a.gate + at : nullptr, a.out + at, a.ticket, a.D, min(kPagedRows, a.group - run.r0),
                    walk.first_block(run), walk.last_block(run)};
}

}  // namespace
}  // namespace muser
