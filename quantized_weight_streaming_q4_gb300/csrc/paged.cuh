// paged.cuh -- what the kernels of attention over a paged cache share: the
// call's arguments, the split of the work, and the joining of partial results.
//
// The lengths of the sequences are known on the device only.  An item is one
// token row, one K/V head and up to 16 of its query heads; its work are the
// tiles of TILE positions that hold rows it sees.  Every block finds the same
// split for itself, in one of two ways:
//  - few tiles a block: each item is cut into pieces of up to `chunk` tiles, one
//    a block.  Joining the results of an item's blocks costs about as much as
//    four tiles, so items of up to four are left whole; longer ones are cut as
//    far as there are blocks.
//  - else all items' tiles in a row are cut into as many equal runs as there are
//    blocks, so that a run may end inside an item.
// The blocks of an item leave partial results, and the last of them to finish
// joins these in the items' order (of more than 16, eight at a time first).  No
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
    int32_t window, n_sink;
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
        end = min(a.k ? pos : pos + 1, a.rows_end);
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
    // whether every row of the tile's first `n` is seen
    __device__ __forceinline__ bool whole(int p0, int n) const { return n == TILE && (p0 >= low || p0 + TILE <= sink); }
};

// The split, in shared memory: positions (-1: no work) and the units before
// each token row, tiles (chunk 0) or pieces of up to `chunk` tiles.
struct PagedPlan {
    int32_t t[kMaxSequences];
    uint32_t before[kMaxSequences + 1];
    uint32_t chunk, first_row;  // first_row: that the block's first unit is of
};
constexpr int kMostChunk = 8, kWholeTiles = 4;

__device__ __forceinline__ uint32_t ceil_div(uint32_t x, uint32_t y) { return (x + y - 1) / y; }

// x / y; most calls' numbers fit 32 bits, whose division is a third of the work.
__device__ __forceinline__ uint64_t divide(uint64_t x, uint64_t y) {
    if ((x | y) >> 32) return x / y;
    return static_cast<uint32_t>(x) / static_cast<uint32_t>(y);
}

// A block's share [at, end) of `total` units; blocks behind the units' number
// have none.
struct PagedShare {
    uint64_t total, at, end;
    uint32_t blocks;
    __device__ __forceinline__ PagedShare(const PagedArgs& a, uint32_t units) : at(0), end(0) {
        total = static_cast<uint64_t>(units) * static_cast<uint32_t>(a.G * a.blocks_per_head);
        blocks = total < gridDim.x ? static_cast<uint32_t>(total) : gridDim.x;
        if (blockIdx.x >= blocks) return;
        if (total == blocks) {
            at = blockIdx.x;
            end = at + 1;
        } else {
            at = divide(total * blockIdx.x, blocks);
            end = divide(total * (blockIdx.x + 1), blocks);
        }
    }
};

// Fills the plan; all of the block's threads (256) call it.  `warp_sums`: 80
// words of shared memory.
template <int TILE>
__device__ __forceinline__ void make_plan(const PagedArgs& a, PagedPlan& plan, uint32_t* warp_sums) {
    static_assert(kMaxSequences == 256, "a thread a token row");
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int warps = (a.n + 31) / 32;  // that have rows
    uint32_t mine = 0;
    int t = -1;
    if (tid < a.n) {
        t = __ldcg(a.position + tid);
        if (a.sequence) {
            const int s = __ldcg(a.sequence + tid);
            if (s < 0 || s >= a.n_tables) t = -1;
        } else if (tid >= a.n_tables) {
            t = -1;
        }
        t = min(t, 0x3fffffff);
    }
    plan.t[tid] = t;
    if (t >= 0) mine = static_cast<uint32_t>(Sight<TILE>(a, t).tiles);
    // sums over the rows: tiles, the longest, and pieces for each chunk
    if (w < warps) {
        const uint32_t most = __reduce_max_sync(0xffffffffu, mine);
        if (lane == 0) warp_sums[w * 10] = most;
#pragma unroll
        for (uint32_t c = 1; c <= kMostChunk; ++c) {
            const uint32_t sum = __reduce_add_sync(0xffffffffu, ceil_div(mine, c));
            if (lane == 0) warp_sums[w * 10 + c] = sum;
        }
    }
    __syncthreads();
    // lane c of every warp: the pieces of chunk c; lane 0: the longest
    uint32_t sum = 0;
    if (lane <= kMostChunk)
        for (int j = 0; j < warps; ++j) sum = lane == 0 ? max(sum, warp_sums[j * 10]) : sum + warp_sums[j * 10 + lane];
    const bool fits = lane > 0 && lane <= kMostChunk && static_cast<uint64_t>(sum) * static_cast<uint32_t>(a.G * a.blocks_per_head) <= gridDim.x;
    const uint32_t fit = __ballot_sync(0xffffffffu, fits);
    uint32_t chunk = fit == 0 ? 0 : __ffs(fit) - 1;
    if (chunk > 0 && __shfl_sync(0xffffffffu, sum, 0) <= kWholeTiles) chunk = kWholeTiles;
    const uint32_t all = __shfl_sync(0xffffffffu, sum, chunk == 0 ? 1 : chunk);
    const uint32_t units = chunk <= 1 ? mine : divide(mine + chunk - 1, chunk);
    uint32_t v = units;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += x;
    }
    if (warps > 1) {
        __syncthreads();
        if (lane == 31) warp_sums[w] = v;
        __syncthreads();
        for (int j = 0; j < w; ++j) v += warp_sums[j];
    }
    if (w >= warps) v = all;  // rows behind the last one
    plan.before[tid] = v - units;
    if (tid == 0) plan.before[kMaxSequences] = all;
    const PagedShare share(a, all);
    const uint64_t per = static_cast<uint32_t>(a.G * a.blocks_per_head);
    if ((v - units) * per <= share.at && share.at < v * per) {
        plan.first_row = tid;
        plan.chunk = chunk;
    }
    __syncthreads();
}

// A run of one item's tiles.
struct PagedRun {
    int row, head, r0;    // token row, K/V head, first of its query heads
    int a, b, tiles;      // tiles [a, b) of `tiles`
    uint64_t u0;          // the item's first unit, and their number
    uint32_t units;
    __device__ __forceinline__ bool whole() const { return a == 0 && b == tiles; }
};

// The block's runs, one after another.
template <int TILE>
struct PagedWalk {
    PagedShare share;
    uint32_t chunk;
    int m;
    __device__ __forceinline__ PagedWalk(const PagedArgs& a, const PagedPlan& plan)
        : share(a, plan.before[kMaxSequences]), chunk(plan.chunk), m(static_cast<int>(plan.first_row)) {}
    __device__ __forceinline__ bool next(const PagedArgs& a, const PagedPlan& plan, PagedRun& run) {
        if (share.at >= share.end) return false;
        const uint64_t per = static_cast<uint32_t>(a.G * a.blocks_per_head);
        while (plan.before[m + 1] * per <= share.at) ++m;
        const uint64_t base = plan.before[m] * per;
        const uint32_t units = plan.before[m + 1] - plan.before[m];  // of an item
        const uint64_t off = share.at - base;
        uint32_t sub = static_cast<uint32_t>(off), x = 0;
        if (units > 1) {
            sub = static_cast<uint32_t>(divide(off, units));
            x = static_cast<uint32_t>(off - static_cast<uint64_t>(sub) * units);
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
        if (chunk == 0) {
            run.tiles = static_cast<int>(units);
            run.a = static_cast<int>(x);
            run.b = static_cast<int>(min(static_cast<uint64_t>(units), x + (share.end - share.at)));
            share.at += run.b - run.a;
            return true;
        }
        run.tiles = Sight<TILE>(a, plan.t[m]).tiles;
        run.a = 0;
        run.b = run.tiles;
        if (units > 1) {  // pieces of equal size, the first ones of a tile more
            const int each = run.tiles / static_cast<int>(units), rest = run.tiles - each * static_cast<int>(units), i = static_cast<int>(x);
            run.a = i * each + min(i, rest);
            run.b = run.a + each + (i < rest ? 1 : 0);
        }
        ++share.at;
        return true;
    }
    // the first and the last block that share the run's item
    __device__ __forceinline__ int owner(uint64_t unit) const {
        if (share.total == share.blocks) return static_cast<int>(unit);
        return static_cast<int>(divide((unit + 1) * share.blocks - 1, share.total));
    }
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
__device__ __forceinline__ float4 load4(const float* p, bool vec, int left) {
    if (vec) return __ldcg(reinterpret_cast<const float4*>(p));
    return make_float4(__ldcg(p), left > 1 ? __ldcg(p + 1) : 0.f, left > 2 ? __ldcg(p + 2) : 0.f, left > 3 ? __ldcg(p + 3) : 0.f);
}
__device__ __forceinline__ void store4(float* p, float4 v, bool vec, int left) {
    if (vec) {
        *reinterpret_cast<float4*>(p) = v;
        return;
    }
    p[0] = v.x;
    if (left > 1) p[1] = v.y;
    if (left > 2) p[2] = v.z;
    if (left > 3) p[3] = v.w;
}
__device__ __forceinline__ float4 scaled(float4 v, float f) { return make_float4(v.x * f, v.y * f, v.z * f, v.w * f); }
__device__ __forceinline__ float4 gated4(float4 v, float4 z) { return make_float4(gated(v.x, z.x), gated(v.y, z.y), gated(v.z, z.z), gated(v.w, z.w)); }

// `count` parts, the first that of block `from` and each of a block `step`
// further, are joined, into the item's result or (!final) into the first part.
// A warp (w of W) takes every W-th row: its lanes hold the parts' shares.
constexpr int kJoinMost = 16;
__device__ __noinline__ void join_parts(const PagedArgs& a, const PagedRun& run, int first, int from, int step, int count, int w,
                                        int W, bool final) {
    constexpr int B = 8;  // loads in flight
    const int lane = threadIdx.x & 31, live = min(kPagedRows, a.group - run.r0);
    const bool vec = a.D % 4 == 0;
    const int64_t row0 = static_cast<int64_t>(run.row) * a.H + run.head * a.group + run.r0;
    for (int j = w; j < live; j += W) {
        float2 ml = make_float2(kNegInf, 0.f);
        const int64_t mine = (static_cast<int64_t>(part_of(from + lane * step, first)) * kPagedRows) + j;  // of lane i: part i
        if (lane < count) ml = __ldcg(a.part_ml + mine);
        for (int d = 4 * lane; d - 4 * lane < a.D; d += 128) {
            const bool real = d < a.D;
            const float* p = a.part_o + (static_cast<int64_t>(part_of(from, first)) * kPagedRows + j) * a.D + d;
            float4 z = make_float4(0.f, 0.f, 0.f, 0.f), o = z;
            if (final && a.gate && real) z = load4(a.gate + (row0 + j) * a.D + d, vec, a.D - d);
            float m = 0.f, l = 0.f, f = 0.f;
            for (int i0 = 0; i0 < count; i0 += B) {
                float4 v[B];
#pragma unroll
                for (int i = 0; i < B; ++i) {
                    v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (real && i0 + i < count)
                        v[i] = load4(a.part_o + (static_cast<int64_t>(part_of(from + (i0 + i) * step, first)) * kPagedRows + j) * a.D + d, vec, a.D - d);
                }
                if (i0 == 0) {  // the shares, while the sums are on the way
                    m = ml.x;
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                    const bool empty = ml.x == kNegInf && ml.y == 0.f;  // no rows there: its sums are not looked at
                    f = empty ? kNegInf : share(ml.x, m);
                    l = warp_sum(empty ? 0.f : f * ml.y);
                }
#pragma unroll
                for (int i = 0; i < B; ++i) {
                    const float fi = __shfl_sync(0xffffffffu, f, min(i0 + i, 31));
                    if (i0 + i < count && fi != kNegInf)
                        o = make_float4(fmaf(fi, v[i].x, o.x), fmaf(fi, v[i].y, o.y), fmaf(fi, v[i].z, o.z), fmaf(fi, v[i].w, o.w));
                }
            }
            if (!real) continue;
            if (final) {
                o = scaled(o, l == 0.f ? 0.f : __fdividef(1.f, l));
                store4(a.out + (row0 + j) * a.D + d, a.gate ? gated4(o, z) : o, vec, a.D - d);
            } else {
                store4(const_cast<float*>(p), o, vec, a.D - d);
                if (d == 0) a.part_ml[mine] = make_float2(m, l);
            }
        }
    }
}

// Whether this was the last of `count` arrivals at a ticket; called by one
// thread, when all threads that wrote what it announces have passed a barrier.
__device__ __forceinline__ bool last_of(unsigned* ticket, int count) {
    __threadfence();
    const bool last = atom_add_acq_rel_gpu(ticket, 1u) == static_cast<unsigned>(count - 1);
    if (last) *ticket = 0;
    return last;
}

// After the block's part of an item is written, by `threads` threads (whole
// warps) that share barrier 1 and have passed it since: what is left to join,
// if this is the last block to get there.  `flag` is in shared memory.
template <int TILE>
__device__ __forceinline__ void finish_item(const PagedArgs& a, const PagedWalk<TILE>& walk, const PagedRun& run, int first, int tid,
                                            int threads, volatile uint32_t& flag) {
    const int last = walk.owner(run.u0 + run.units - 1), count = last - first + 1, w = tid >> 5, W = threads >> 5;
    static_assert(kPagedMaxBlocks <= kJoinMost * kJoinMost, "two levels");
    int step = 1, parts = count;
    if (count > kJoinMost) {
        while (step * step < count) ++step;  // as many groups as parts in each
        const int from = first + (static_cast<int>(blockIdx.x) - first) / step * step, size = min(step, last - from + 1);
        if (tid == 0) flag = last_of(a.ticket + part_of(from, first), size);
        named_barrier_sync(1, threads);
        if (!flag) return;
        join_parts(a, run, first, from, 1, size, w, W, false);
        parts = (count + step - 1) / step;
        named_barrier_sync(1, threads);
    }
    if (tid == 0) flag = last_of(a.ticket + 2 * kPagedMaxBlocks + first, parts);
    named_barrier_sync(1, threads);
    if (flag) join_parts(a, run, first, first, step, parts, w, W, true);
}

}  // namespace
}  // namespace muser
