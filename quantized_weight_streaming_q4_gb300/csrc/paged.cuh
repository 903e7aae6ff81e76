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
};
constexpr int kMostChunk = 8, kWholeTiles = 4;

__device__ __forceinline__ uint32_t ceil_div(uint32_t x, uint32_t y) { return (x + y - 1) / y; }

// Fills the plan; all of the block's threads (256) call it.  Returns the chunk.
// `warp_sums`: 80 words of shared memory.
template <int TILE>
__device__ __forceinline__ uint32_t make_plan(const PagedArgs& a, PagedPlan& plan, uint32_t* warp_sums) {
    static_assert(kMaxSequences == 256, "a thread a token row");
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int warps = (a.n + 31) / 32;  // that have rows
    uint32_t mine = 0;
    int t = -1;
    if (tid < a.n) {
        t = __ldcg(a.position + tid);
        const int s = a.sequence ? __ldcg(a.sequence + tid) : tid;
        if (s < 0 || s >= a.n_tables) t = -1;
        t = min(t, 0x3fffffff);
    }
    plan.t[tid] = t;
    if (t >= 0) mine = static_cast<uint32_t>(Sight<TILE>(a, t).tiles);
    // sums over the rows: tiles, the longest, and pieces for each chunk
    if (w < warps) {
        const uint32_t most = __reduce_max_sync(0xffffffffu, mine);
        uint32_t sums[kMostChunk];
#pragma unroll
        for (uint32_t c = 1; c <= kMostChunk; ++c) sums[c - 1] = __reduce_add_sync(0xffffffffu, ceil_div(mine, c));
        if (lane == 0) {
            warp_sums[w * 10] = most;
#pragma unroll
            for (int c = 0; c < kMostChunk; ++c) warp_sums[w * 10 + 1 + c] = sums[c];
        }
    }
    __syncthreads();
    uint32_t most = 0, sums[kMostChunk] = {};
    for (int j = 0; j < warps; ++j) {
        most = max(most, warp_sums[j * 10]);
#pragma unroll
        for (int c = 0; c < kMostChunk; ++c) sums[c] += warp_sums[j * 10 + 1 + c];
    }
    const uint64_t per = static_cast<uint64_t>(a.G) * a.blocks_per_head;
    uint32_t chunk = 0;
#pragma unroll
    for (int c = kMostChunk; c >= 1; --c)
        if (sums[c - 1] * per <= gridDim.x) chunk = c;
    if (chunk > 0 && most <= kWholeTiles) chunk = kWholeTiles;
    uint32_t units = chunk == 0 ? mine : ceil_div(mine, chunk), v = units;
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
    } else if (w > 0) {
        v = chunk == 0 ? sums[0] : 0;
        if (chunk != 0) {
#pragma unroll
            for (int c = 1; c <= kMostChunk; ++c) v = static_cast<uint32_t>(c) == chunk ? sums[c - 1] : v;
        }
        units = 0;
    }
    plan.before[tid] = v - units;
    if (tid == kMaxSequences - 1) plan.before[kMaxSequences] = v;
    __syncthreads();
    return chunk;
}

// A run of one item's tiles.
struct PagedRun {
    int row, head, r0;      // token row, K/V head, first of its query heads
    int a, b, tiles;        // tiles [a, b) of `tiles`
    int first, last;        // blocks that share the item
    __device__ __forceinline__ bool whole() const { return a == 0 && b == tiles; }
};

// x * y / z, in 32 bits where that is enough.
__device__ __forceinline__ uint64_t mul_div(uint64_t x, uint32_t y, uint64_t z) {
    if (((x * y) | z) >> 32) return x * y / z;
    return static_cast<uint32_t>(x * y) / static_cast<uint32_t>(z);
}

// The block's runs, one after another.
template <int TILE>
struct PagedWalk {
    uint64_t at, end, total;
    uint32_t per;     // items of a token row
    uint32_t blocks;  // that have work: each has a unit at least
    uint32_t chunk;
    int m;
    __device__ __forceinline__ PagedWalk(const PagedArgs& a, const PagedPlan& plan, uint32_t chunk) : chunk(chunk) {
        per = static_cast<uint32_t>(a.G * a.blocks_per_head);
        total = static_cast<uint64_t>(plan.before[kMaxSequences]) * per;
        blocks = static_cast<uint32_t>(min(total, static_cast<uint64_t>(gridDim.x)));
        at = end = 0;
        m = 0;
        if (blockIdx.x >= blocks) return;
        if (total == blocks) {
            at = blockIdx.x;
            end = at + 1;
        } else {
            at = mul_div(total, blockIdx.x, blocks);
            end = mul_div(total, blockIdx.x + 1, blocks);
        }
        int lo = 0, hi = a.n - 1;
        while (lo < hi) {  // the row that holds unit `at`
            const int mid = (lo + hi) >> 1;
            if (static_cast<uint64_t>(plan.before[mid + 1]) * per > at) hi = mid;
            else lo = mid + 1;
        }
        m = lo;
    }
    __device__ __forceinline__ int owner(uint64_t unit) const { return static_cast<int>(((unit + 1) * blocks - 1) / total); }
    __device__ __forceinline__ bool next(const PagedArgs& a, const PagedPlan& plan, PagedRun& run) {
        if (at >= end) return false;
        while (static_cast<uint64_t>(plan.before[m + 1]) * per <= at) ++m;
        const uint64_t base = static_cast<uint64_t>(plan.before[m]) * per;
        const uint32_t units = plan.before[m + 1] - plan.before[m];  // of an item
        const uint64_t off = at - base;
        const uint32_t sub = static_cast<uint32_t>(mul_div(off, 1, units)), x = static_cast<uint32_t>(off - static_cast<uint64_t>(sub) * units);
        run.row = m;
        run.head = static_cast<int>(sub) / a.blocks_per_head;
        run.r0 = (static_cast<int>(sub) - run.head * a.blocks_per_head) * kPagedRows;
        if (chunk != 0) {
            run.tiles = Sight<TILE>(a, plan.t[m]).tiles;
            run.a = run.tiles * x / units;
            run.b = run.tiles * (x + 1) / units;
            run.first = static_cast<int>(blockIdx.x - x);
            run.last = run.first + static_cast<int>(units) - 1;
            ++at;
            return true;
        }
        run.tiles = static_cast<int>(units);
        run.a = static_cast<int>(x);
        run.b = static_cast<int>(min(static_cast<uint64_t>(units), x + (end - at)));
        const uint64_t u0 = base + static_cast<uint64_t>(sub) * units;
        run.first = run.a == 0 ? static_cast<int>(blockIdx.x) : owner(u0);
        run.last = run.b == run.tiles ? static_cast<int>(blockIdx.x) : owner(u0 + units - 1);
        at += run.b - run.a;
        return true;
    }
};

// The partial result of block `b` of an item's blocks first..last: the block
// where the item begins keeps it in its second place, the others in their first.
__device__ __forceinline__ int part_of(int b, int first) { return 2 * b + (b == first ? 1 : 0); }

__device__ __forceinline__ float gated(float y, float z) { return __fdividef(y, 1.f + __expf(-z)); }

// Parts of the blocks from..from + (count - 1) * step are joined, into the
// item's result or (!FINAL) into the first one's part: THREADS threads that
// share barrier 1; `sm` has room for 18 * count floats.  The parts' shares are
// found while their first sums are on the way.
constexpr int kJoinMost = 24, kJoinBytes = 18 * kJoinMost * 4;
template <int THREADS, bool FINAL>
__device__ __forceinline__ void join_parts(const PagedArgs& a, const PagedRun& run, int from, int step, int count, int tid, float* sm) {
    constexpr int U = 4, B = 8;  // pieces of a thread, parts in flight
    const int live = min(kPagedRows, a.group - run.r0);
    const bool vec = a.D % 4 == 0;
    const int per = vec ? a.D / 4 : a.D, units = live * per;
    const int64_t row0 = static_cast<int64_t>(run.row) * a.H + run.head * a.group + run.r0;
    float* const inv = sm + 16 * count;
    float* const most = inv + 16;
    bool shares = false;
    for (int x0 = tid; x0 - tid < units; x0 += U * THREADS) {
        float4 o[U], z[U], v[U][B];
        int r[U], d[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int x = x0 + u * THREADS;
            r[u] = x < units ? x / per : -1;
            d[u] = (x - r[u] * per) * (vec ? 4 : 1);
            o[u] = z[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (FINAL && a.gate && r[u] >= 0) {
                const float* p = a.gate + (row0 + r[u]) * a.D + d[u];
                if (vec) z[u] = __ldcg(reinterpret_cast<const float4*>(p));
                else z[u].x = __ldcg(p);
            }
        }
        for (int i0 = 0; i0 < count; i0 += B) {
#pragma unroll
            for (int i = 0; i < B; ++i)
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    v[u][i] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (i0 + i < count && r[u] >= 0) {
                        const float* p = a.part_o + (static_cast<int64_t>(part_of(from + (i0 + i) * step, run.first)) * kPagedRows + r[u]) * a.D + d[u];
                        if (vec) v[u][i] = __ldcg(reinterpret_cast<const float4*>(p));
                        else v[u][i].x = __ldcg(p);
                    }
                }
            if (!shares) {
                shares = true;
                // sixteen rows' maxima and sums of a part, by sixteen threads; then a row a thread
                float2 w[(kJoinMost * 16 + THREADS - 1) / THREADS];
#pragma unroll
                for (int k = 0; k < (kJoinMost * 16 + THREADS - 1) / THREADS; ++k) {
                    const int y = tid + k * THREADS, row = y & 15;
                    w[k] = make_float2(kNegInf, 0.f);
                    if (y < 16 * count && row < live)
                        w[k] = __ldcg(a.part_ml + static_cast<int64_t>(part_of(from + (y >> 4) * step, run.first)) * kPagedRows + row);
                    if (y < 16 * count) sm[y] = w[k].x;
                }
                named_barrier_sync(1, THREADS);
                if (tid < 16) {
                    float m = kNegInf;
                    for (int i = 0; i < count; ++i) m = fmaxf(m, sm[16 * i + tid]);
                    most[tid] = m;
                }
                named_barrier_sync(1, THREADS);
#pragma unroll
                for (int k = 0; k < (kJoinMost * 16 + THREADS - 1) / THREADS; ++k) {
                    const int y = tid + k * THREADS;
                    const bool empty = w[k].x == kNegInf && w[k].y == 0.f;  // no rows there
                    const float f = empty ? 0.f : share(w[k].x, most[y & 15]);
                    if (y < 16 * count) sm[y] = empty ? kNegInf : f;  // -infinity: its sums are not looked at
                    w[k].y = empty ? 0.f : f * w[k].y;
                }
                // the rows' sums: each thread's over its parts, then over a row's threads
                float l = 0.f;
#pragma unroll
                for (int k = 0; k < (kJoinMost * 16 + THREADS - 1) / THREADS; ++k) l += w[k].y;
                l += __shfl_xor_sync(0xffffffffu, l, 16);
                if (tid < 16) inv[tid] = 0.f;
                named_barrier_sync(1, THREADS);
                for (int q = 0; q < THREADS / 32; ++q) {  // one warp after another: always the same order
                    if (tid >> 5 == q && (tid & 31) < 16) inv[tid & 15] += l;
                    named_barrier_sync(1, THREADS);
                }
                if (!FINAL && tid < live)
                    a.part_ml[static_cast<int64_t>(part_of(from, run.first)) * kPagedRows + tid] = make_float2(most[tid], inv[tid]);
            }
#pragma unroll
            for (int i = 0; i < B; ++i)
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (i0 + i < count && r[u] >= 0) {
                        const float f = sm[16 * (i0 + i) + r[u]];
                        if (f == kNegInf) continue;
                        o[u] = make_float4(fmaf(f, v[u][i].x, o[u].x), fmaf(f, v[u][i].y, o[u].y), fmaf(f, v[u][i].z, o[u].z), fmaf(f, v[u][i].w, o[u].w));
                    }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (r[u] < 0) continue;
            float* p;
            if (FINAL) {
                const float l = inv[r[u]], y = l == 0.f ? 0.f : __fdividef(1.f, l);
                o[u] = make_float4(o[u].x * y, o[u].y * y, o[u].z * y, o[u].w * y);
                if (a.gate) o[u] = make_float4(gated(o[u].x, z[u].x), gated(o[u].y, z[u].y), gated(o[u].z, z[u].z), gated(o[u].w, z[u].w));
                p = a.out + (row0 + r[u]) * a.D + d[u];
            } else {
                p = a.part_o + (static_cast<int64_t>(part_of(from, run.first)) * kPagedRows + r[u]) * a.D + d[u];
            }
            if (vec) *reinterpret_cast<float4*>(p) = o[u];
            else *p = o[u].x;
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

// After the block's part of an item is written: what is left to join, if this
// is the last block to get there.  `flag` is in shared memory.
template <int THREADS>
__device__ __forceinline__ void finish_item(const PagedArgs& a, const PagedRun& run, int tid, float* sm, volatile uint32_t& flag) {
    const int count = run.last - run.first + 1;
    constexpr int kGroup = 8, kOnce = 16;
    static_assert(kOnce <= kJoinMost && (kPagedMaxBlocks + kGroup - 1) / kGroup <= kJoinMost, "the shares fit");
    int step = 1, parts = count;
    if (count > kOnce) {
        const int i = (static_cast<int>(blockIdx.x) - run.first) / kGroup, from = run.first + i * kGroup, size = min(kGroup, run.last - from + 1);
        if (tid == 0) flag = last_of(a.ticket + part_of(from, run.first), size);
        named_barrier_sync(1, THREADS);
        if (!flag) return;
        join_parts<THREADS, false>(a, run, from, 1, size, tid, sm);
        step = kGroup;
        parts = (count + kGroup - 1) / kGroup;
        named_barrier_sync(1, THREADS);
    }
    if (tid == 0) flag = last_of(a.ticket + 2 * kPagedMaxBlocks + run.first, parts);
    named_barrier_sync(1, THREADS);
    if (flag) join_parts<THREADS, true>(a, run, run.first, step, parts, tid, sm);
}

}  // namespace
}  // namespace muser
