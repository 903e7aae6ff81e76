// paged.cuh -- what the kernels of attention over a paged cache share: the
// call's arguments, the split of the work, and the joining of partial results.
//
// The lengths of the sequences are known on the device only.  An item is one
// token row, one K/V head and up to ROWS of its query heads; its work are the
// tiles of TILE positions that hold rows it sees.  All items' tiles in a row
// are cut into as many equal runs as there are blocks, so a run may end inside
// an item: its blocks leave partial results, and the last of them to finish
// joins these in the items' order.  No block waits for another.
#pragma once

#include "attn_parts.cuh"
#include "pages.cuh"

namespace muser {

constexpr int kPagedMaxBlocks = 160;   // blocks of a launch: one an SM
constexpr size_t kPagedTicketBytes = 1024;
static_assert(kPagedTicketBytes >= kPagedMaxBlocks * sizeof(unsigned), "a ticket a block");
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
    unsigned* ticket;  // of the block where an item that is split begins
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

// The split, in shared memory: positions (-1: no work) and tiles before each row.
struct PagedPlan {
    int32_t t[kMaxSequences];
    uint32_t before[kMaxSequences + 1];
    uint32_t warp[8];
};

// Fills the plan; the block's first 256 threads take part, all wait.
template <int TILE>
__device__ __forceinline__ void make_plan(const PagedArgs& a, PagedPlan& plan) {
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    uint32_t mine = 0;
    uint32_t v = 0;
    if (tid < kMaxSequences) {
        int t = -1;
        if (tid < a.n) {
            t = __ldcg(a.position + tid);
            const int s = a.sequence ? __ldcg(a.sequence + tid) : tid;
            if (s < 0 || s >= a.n_tables) t = -1;
            t = min(t, 0x3fffffff);
        }
        plan.t[tid] = t;
        if (t >= 0) mine = static_cast<uint32_t>(Sight<TILE>(a, t).tiles);
        v = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t x = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += x;
        }
        if (lane == 31) plan.warp[w] = v;
    }
    __syncthreads();
    if (tid < kMaxSequences) {
        uint32_t base = 0;
        for (int j = 0; j < w; ++j) base += plan.warp[j];
        plan.before[tid] = base + v - mine;
        if (tid == kMaxSequences - 1) plan.before[kMaxSequences] = base + v;
    }
    __syncthreads();
}

// A run of one item's tiles.
struct PagedRun {
    int row, head, r0;      // token row, K/V head, first of its query heads
    int a, b, tiles;        // tiles [a, b) of `tiles`
    int first, last;        // blocks that share the item
    __device__ __forceinline__ bool whole() const { return a == 0 && b == tiles; }
};

// The block's runs, one after another.
struct PagedWalk {
    uint64_t at, end, total;
    uint32_t per;     // items of a token row
    uint32_t blocks;  // that have work: each has a tile at least
    int m;
    __device__ __forceinline__ PagedWalk(const PagedArgs& a, const PagedPlan& plan) {
        per = static_cast<uint32_t>(a.G * a.blocks_per_head);
        total = static_cast<uint64_t>(plan.before[kMaxSequences]) * per;
        blocks = static_cast<uint32_t>(min(total, static_cast<uint64_t>(gridDim.x)));
        if (blockIdx.x >= blocks) {
            at = end = 0;
            m = 0;
            return;
        }
        at = total * blockIdx.x / blocks;
        end = total * (blockIdx.x + 1) / blocks;
        int lo = 0, hi = kMaxSequences - 1;
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
        const uint32_t tiles = plan.before[m + 1] - plan.before[m];
        const uint64_t off = at - base;
        const uint32_t sub = static_cast<uint32_t>(off / tiles);
        run.row = m;
        run.head = static_cast<int>(sub) / a.blocks_per_head;
        run.r0 = (static_cast<int>(sub) % a.blocks_per_head) * kPagedRows;
        run.tiles = static_cast<int>(tiles);
        run.a = static_cast<int>(off - static_cast<uint64_t>(sub) * tiles);
        run.b = static_cast<int>(min(static_cast<uint64_t>(tiles), run.a + (end - at)));
        const uint64_t u0 = base + static_cast<uint64_t>(sub) * tiles;
        run.first = run.a == 0 ? static_cast<int>(blockIdx.x) : owner(u0);
        run.last = run.b == run.tiles ? static_cast<int>(blockIdx.x) : owner(u0 + tiles - 1);
        at += run.b - run.a;
        return true;
    }
};

// The partial result of block `b` of an item's blocks first..last: the block
// where the item begins keeps it in its second place, the others in their first.
__device__ __forceinline__ int part_of(int b, int first) { return 2 * b + (b == first ? 1 : 0); }

__device__ __forceinline__ float gated(float y, float z) { return __fdividef(y, 1.f + __expf(-z)); }

// Joins an item's parts and writes its rows out: THREADS threads, tid counts them.
template <int THREADS>
__device__ __forceinline__ void join_parts(const PagedArgs& a, const PagedRun& run, int tid) {
    const int live = min(kPagedRows, a.group - run.r0);
    const bool vec = a.D % 4 == 0;
    const int per = vec ? a.D / 4 : a.D, units = live * per;
    const int64_t row0 = static_cast<int64_t>(run.row) * a.H + run.head * a.group + run.r0;
    for (int x = tid; x < units; x += THREADS) {
        const int r = x / per, d = (x - r * per) * (vec ? 4 : 1);
        float m = kNegInf, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f), z = o;
        if (a.gate) {
            const float* p = a.gate + (row0 + r) * a.D + d;
            if (vec) z = __ldcg(reinterpret_cast<const float4*>(p));
            else z.x = __ldcg(p);
        }
        for (int b0 = run.first; b0 <= run.last; b0 += 8) {
            float2 w[8];
            float4 v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                w[u] = make_float2(kNegInf, 0.f);
                v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (b0 + u <= run.last) {
                    const int64_t at = static_cast<int64_t>(part_of(b0 + u, run.first)) * kPagedRows + r;
                    w[u] = __ldcg(a.part_ml + at);
                    const float* p = a.part_o + at * a.D + d;
                    if (vec) v[u] = __ldcg(reinterpret_cast<const float4*>(p));
                    else v[u].x = __ldcg(p);
                }
            }
            float mn = m;
#pragma unroll
            for (int u = 0; u < 8; ++u) mn = fmaxf(mn, w[u].x);
            const float f0 = share(m, mn);
            m = mn;
            l *= f0;
            o = make_float4(o.x * f0, o.y * f0, o.z * f0, o.w * f0);
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                if (w[u].x == kNegInf && w[u].y == 0.f) continue;  // no rows there
                const float f = share(w[u].x, m);
                l = fmaf(f, w[u].y, l);
                o = make_float4(fmaf(f, v[u].x, o.x), fmaf(f, v[u].y, o.y), fmaf(f, v[u].z, o.z), fmaf(f, v[u].w, o.w));
            }
        }
        const float inv = l == 0.f ? 0.f : __fdividef(1.f, l);
        o = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
        if (a.gate) o = make_float4(gated(o.x, z.x), gated(o.y, z.y), gated(o.z, z.z), gated(o.w, z.w));
        float* p = a.out + (row0 + r) * a.D + d;
        if (vec) *reinterpret_cast<float4*>(p) = o;
        else *p = o.x;
    }
}

// One of an item's blocks has written its part (all its threads have passed a
// barrier): whether it was the last.  Called by one thread.
__device__ __forceinline__ bool last_part(const PagedArgs& a, const PagedRun& run) {
    __threadfence();
    unsigned* ticket = a.ticket + run.first;
    const bool last = atom_add_acq_rel_gpu(ticket, 1u) == static_cast<unsigned>(run.last - run.first);
    if (last) *ticket = 0;
    return last;
}

}  // namespace
}  // namespace muser
