// paged_tc.cu -- attention of one token row each of several sequences over a
// paged K/V cache on the fifth-generation tensor cores: head sizes that are
// multiples of 8 up to 256, pages of a power of two of at least 8 rows, 16-byte
// aligned buffers.
//
// The mathematics of a tile is that of the tree attention of few rows: the keys
// take the tile's 128 lanes and the R query rows (8 or 16 of one K/V head) its
// columns, twice: the binary16 high parts of the scaled q beside the low ones.
//   S^T = K Q^T   A = K [keys][d], B = Q [2 R][d]
//   O^T = V^T P^T A = V as it lies in the cache (M along its rows), B = P
//         [keys][2 R], high and low parts of p again
// p = 2^(s - m + 11) with a reference m per row that moves only when some s
// exceeds it by more than 4.  O tiles are fresh accumulators added in registers.
//
// A block goes through its runs of items (see paged.cuh) without emptying its
// pipeline: K and V tiles come through one ring of stages, each tile as a TMA
// box per page, and one warp lays out the next run's q while the present one's
// tiles are worked on.
//
// Rows of a tile that are not seen (behind the sequence's end, before a window,
// pages that are not there) may hold anything: their scores are replaced, and
// their V rows in shared memory are zeroed before the product reads them.
//
// Bound: the bytes of the rows that are seen for long sequences (one of 130,815
// rows, 134 MB: the loop takes 19 us, 7 TB/s; 36 us with the start and the joins
// of 76 parts a head), latency for short ones (16 of 9 to 190 rows: 7.8 us).
#include <cuda.h>

#include <algorithm>

#include "kernels.cuh"
#include "paged.cuh"
#include "tc.cuh"

namespace muser {
namespace {

constexpr int kTile = 128;               // keys of a tile
constexpr uint32_t kHalf = kTile * 128;  // 64 elements of each of a tile's rows
constexpr int kThreads = 256;            // warps: products, loads, q (two), softmax (four)
constexpr int kQThreads = 64;
constexpr float kOff = 11.f, kMost = 15.f;

template <int R, int DB>  // query rows; blocks of 64 elements: D <= 64 * DB
struct Layout {
    static constexpr uint32_t kItem = DB * kHalf;
    static constexpr int kNS = 196608 / static_cast<int>(kItem);  // stages of the ring: 12, 6 or 3
    // the barriers: the stages' full and empty ones first
    static constexpr int kFull = 0, kEmpty = kNS, kSFull = 2 * kNS, kPFull = kSFull + 2, kOFull = kPFull + 2,
                         kQFull = kOFull + 2, kQFree = kQFull + 2, kJoin = kQFree + 2, kBars = kJoin + 1;
    static constexpr uint32_t kN = 2 * R;                         // columns
    static constexpr uint32_t kKeyRow = kN / 8 * 128;             // P: bytes from 8 keys to the next 8
    static constexpr uint32_t kPBytes = kTile / 8 * kKeyRow;
    static constexpr uint32_t kQBytes = DB * kN * 128;            // [d / 64][2 R][128 bytes]
    static constexpr int kQBufs = DB == 4 ? 1 : 2;                // q of this run and the next one
    static constexpr uint32_t kQOff = kNS * kItem, kPOff = kQOff + kQBufs * kQBytes;
    static constexpr uint32_t kScaleOff = kPOff + 2 * kPBytes;    // float[2][16]: the rows' scales
    static constexpr uint32_t kSelfOff = kScaleOff + 2 * 64;      // float[2][16]: scores against themselves
    static constexpr uint32_t kRedOff = kSelfOff + 2 * 64;        // float[4][16]
    static constexpr uint32_t kSumsOff = kRedOff + 256;           // float[2][16]: the rows' sums and references
    static constexpr uint32_t kBarOff = kSumsOff + 128;
    static constexpr uint32_t kPlanOff = kBarOff + (kBars * 8 + 15) / 16 * 16;
    static constexpr uint32_t kUsed = kPlanOff + sizeof(PagedPlan) + 16;
    // with 64 elements a row the product's upper 64 lanes read the next stage, which is nobody's output
    static constexpr uint32_t kBytes = DB == 1 && kUsed < (kNS + 1) * kItem ? (kNS + 1) * kItem : kUsed;
    static constexpr int kHalves = DB == 4 ? 2 : 1;               // output tiles of 128 elements
    static constexpr uint32_t kOCols = kHalves * kN;              // columns of an output buffer
    static constexpr uint32_t kCols = 2 * kN + 2 * kOCols;
    static constexpr uint32_t kTmemCols = kCols <= 64 ? 64 : kCols <= 128 ? 128 : 256;
    static_assert(kBytes <= 227 * 1024, "a block's shared memory");
    static_assert(R * 128 * kHalves * 4 <= 2 * kPBytes, "a run's output fits where P was");
};

// Whether `mine` holds for any of the 128 threads that share barrier `id`.
__device__ __forceinline__ bool group_any(int id, bool mine) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\tbarrier.cta.red.or.pred q, %1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(id), "r"(mine ? 1 : 0)
        : "memory");
    return r != 0;
}

// v[j] joined over the warp's lanes, j < R: afterwards v[0] of lane l holds
// that of j = l / (32 / R) (each step halves what a lane keeps).
template <int R, typename F>
__device__ __forceinline__ void fold(float (&v)[R], F&& f) {
    const int lane = threadIdx.x & 31;
    int o = 16;
#pragma unroll
    for (int h = R / 2; h >= 1; h >>= 1, o >>= 1) {
        const bool up = (lane & o) != 0;
#pragma unroll
        for (int j = 0; j < h; ++j) {
            const float give = up ? v[j] : v[j + h], keep = up ? v[j + h] : v[j];
            v[j] = f(keep, __shfl_xor_sync(0xffffffffu, give, o));
        }
    }
#pragma unroll
    for (; o >= 1; o >>= 1) v[0] = f(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float (&v)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                 : "r"(taddr));
}
__device__ __forceinline__ void tc_wait_ld(float (&v)[8]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7])
                 :
                 : "memory");
}
__device__ __forceinline__ void load_rows(uint32_t taddr, float (&v)[8]) { tmem_ld8(taddr, v); }
__device__ __forceinline__ void load_rows(uint32_t taddr, float (&v)[16]) { tmem_ld16(taddr, v); }

// A box of a page's rows into shared memory: elements [64 x, 64 x + 64), rows
// from `row` on, of head g of a page.
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* map, int x, int row, int g, int page, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::
            "r"(dst),
        "l"(map), "r"(x * 64), "r"(row), "r"(g), "r"(page), "r"(smem_u32(bar))
        : "memory");
}

template <int R, int DB>
__global__ void __launch_bounds__(kThreads, 1)
    paged_tc_kernel(const __grid_constant__ PagedArgs a, const __grid_constant__ CUtensorMap kmap,
                    const __grid_constant__ CUtensorMap vmap) {
    using L = Layout<R, DB>;
    constexpr int kNS = L::kNS, NH = L::kHalves;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t base = smem_u32(smem);
    PagedPlan& plan = *reinterpret_cast<PagedPlan*>(smem + L::kPlanOff);
    uint32_t& tmem_slot = *reinterpret_cast<uint32_t*>(smem + L::kPlanOff + sizeof(PagedPlan));
    volatile uint32_t& lost = (&tmem_slot)[1];  // a wait ran out
    volatile uint32_t* joining = &tmem_slot + 2;  // whether this block joins the parts of its first and of its last item
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint64_t* bar = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
    pdl_launch_dependents();
    if (tid == 0) {
        for (int i = 0; i < kNS; ++i) {
            mbar_init(&bar[L::kFull + i], 1);
            mbar_init(&bar[L::kEmpty + i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar[L::kSFull + i], 1);
            mbar_init(&bar[L::kPFull + i], 128);
            mbar_init(&bar[L::kOFull + i], 1);
            mbar_init(&bar[L::kQFull + i], kQThreads);
            mbar_init(&bar[L::kQFree + i], 128);
        }
        mbar_init(&bar[L::kJoin], 1);
        lost = 0;
        fence_mbar_init();
    }
    if (warp == 0) tmem_alloc(&tmem_slot, L::kTmemCols);
    if (tid == 32) prefetch_map(&kmap);
    if (tid == 64) prefetch_map(&vmap);
    tc_fence_before();
    __syncthreads();  // the barriers and tensor memory
    tc_fence_after();
    pdl_wait();  // no global access before this
    const PagedSplit split = make_plan<kTile>(a, plan, reinterpret_cast<uint32_t*>(smem + L::kPOff));
    const uint32_t tmem = tmem_slot;
    // A thread whose wait has run out waits no more and goes on with what is
    // there, so that warps and warpgroups stay together; what it would write
    // becomes NaN, and a joined result is not written.
    bool ok = true;
    auto wait = [&](int b, int phase) {
        if (ok) ok = mbar_wait_bounded(&bar[b], static_cast<uint32_t>(phase & 1), a.status, kDevStatusWaitTimeout);
    };
    PagedWalk<kTile> walk(a, split);
    PagedRun run;
    const int D = a.D;

    if (warp == 0) {
        // --------------------------------------------- matrix products
        const bool leader = elect_one();
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint32_t ids = idesc(L::kN, false, false), ido = idesc(L::kN, true, true);
        const int ksteps = (D + 15) / 16;
        // the scores are one tile ahead of the outputs, across runs
        int item = 0, done = 0, runs = 0, left = 0, at = 0;
        int steps[2];
        bool more = true;
        int t0 = 0;
        auto scores = [&]() -> bool {
            if (left == 0) {
                if (more) more = walk.next(a, plan, run);
                if (!more) return false;
                wait(L::kQFull + runs % L::kQBufs, runs / L::kQBufs);
                ++runs;
                left = run.b - run.a;
                t0 = run.a;
            }
            const Sight<kTile> sight(a, plan.t[run.row]);
            const int s = at & 1, st = item % kNS;
            steps[s] = (sight.real(sight.first(t0) * kTile) + 15) / 16;
            wait(L::kFull + st, item / kNS);
            tc_fence_after();
            const uint64_t kd = desc_swizzle128(base + st * L::kItem, 16, 1024);
            const uint64_t qd = desc_swizzle128(base + L::kQOff + (runs - 1) % L::kQBufs * L::kQBytes, 16, 1024);
            const uint32_t d = tm + s * L::kN;
            if (leader && ok) {
#pragma unroll
                for (int ks = 0; ks < 4 * DB; ++ks)
                    if (ks < ksteps) {
                        const uint64_t ka = kd + ((ks >> 2) * kHalf + (ks & 3) * 32 >> 4), qb = qd + ((ks >> 2) * (L::kN * 128) + (ks & 3) * 32 >> 4);
                        if (ks == 0) mma_ss<false>(d, ka, qb, ids);
                        else mma_ss<true>(d, ka, qb, ids);
                    }
                mma_commit(&bar[L::kSFull + s]);
                mma_commit(&bar[L::kEmpty + st]);
            }
            __syncwarp();
            item += 2;  // V's stage is the next one
            ++at;
            ++t0;
            --left;
            return true;
        };
        bool next = scores();
        while (next) {
            next = scores();
            const int s = done & 1, vi = 2 * done + 1, st = vi % kNS;
            wait(L::kPFull + s, done >> 1);
            wait(L::kFull + st, vi / kNS);
            tc_fence_after();
            const uint64_t vd = desc_swizzle128(base + st * L::kItem, kHalf, 1024);
            const uint64_t pd = desc_bits(base + L::kPOff + s * L::kPBytes, L::kKeyRow, 128);
            if (leader && ok) {
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    const uint32_t d = tm + 2 * L::kN + s * L::kOCols + h * L::kN;
                    const uint64_t vh = vd + (h * 2 * kHalf >> 4);
                    mma_ss<false>(d, vh, pd, ido);
#pragma unroll
                    for (int ks = 1; ks < kTile / 16; ++ks)
                        if (ks < steps[s]) mma_ss<true>(d, vh + (ks * 2048 >> 4), pd + (ks * 2 * L::kKeyRow >> 4), ido);
                }
                mma_commit(&bar[L::kOFull + s]);
                mma_commit(&bar[L::kEmpty + st]);
            }
            __syncwarp();
            ++done;
        }
    } else if (warp == 1) {
        // ------------------------------------------------- K, V loads
        // lane b brings box b of each tile: the rows of one page, or 128 of them
        const int box = min(a.page_rows, kTile), boxes = kTile / box, blocks = (D + 63) / 64;
        const uint32_t bytes = static_cast<uint32_t>(box) * 128u * blocks;
        int item = 0;
        while (ok && walk.next(a, plan, run)) {
            const Sight<kTile> sight(a, plan.t[run.row]);
            const int seq = a.sequence ? __ldcg(a.sequence + run.row) : run.row;
            const int32_t* table = a.table + seq * a.stride;
            // the page of this lane's box of tile t, -1 where no row of it is seen;
            // looked at a tile later, so that nothing waits for the load
            auto entry = [&](int t) {
                if (t >= run.b || lane >= boxes) return -1;
                const int p0 = sight.first(t) * kTile, p = p0 + lane * box;
                if (lane * box >= sight.real(p0) || (p + box <= sight.low && p >= sight.sink)) return -1;
                return __ldcg(table + (p >> a.page_shift));
            };
            int next_page = entry(run.a);
            for (int t = run.a; t < run.b && ok; ++t) {
                const int page = static_cast<uint32_t>(next_page) < static_cast<uint32_t>(a.pages) ? next_page : -1;
                next_page = entry(t + 1);
                const int p = sight.first(t) * kTile + lane * box, row = p & (a.page_rows - 1);
                const uint32_t have = __ballot_sync(0xffffffffu, page >= 0);
#pragma unroll
                for (int v = 0; v < 2; ++v, ++item) {
                    const int st = item % kNS;
                    uint64_t* full = &bar[L::kFull + st];
                    if (item >= kNS) wait(L::kEmpty + st, item / kNS - 1);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    if (lane == 0) {
                        if (have) mbar_arrive_expect_tx(full, bytes * __popc(have));
                        else mbar_arrive(full);
                    }
                    __syncwarp();
                    if (page >= 0) {
                        const uint32_t dst = base + st * L::kItem + lane * box * 128;
                        for (int x = 0; x < blocks; ++x) load_box(dst + x * kHalf, v ? &vmap : &kmap, x, row, run.head, page, full);
                    }
                }
            }
        }
        if (!ok) {  // copies under way still write into this block's memory
            if (lane == 0)
                for (int u = max(0, item - kNS); u < item; ++u)
                    mbar_wait_bounded(&bar[L::kFull + u % kNS], static_cast<uint32_t>(u / kNS) & 1u, a.status, kDevStatusTxTimeout);
        }
        __syncwarp();
    } else if (warp < 4) {
        // ------------- a run's q, its rows' scores against themselves, the new row
        // thread: row r, a quarter of its elements
        const int u0 = tid - 64, r = u0 >> 2, quarter = u0 & 3;
        int runs = 0;
        while (walk.next(a, plan, run)) {
            const int buf = runs % L::kQBufs, t = plan.t[run.row];
            const bool self = a.k && run.b == run.tiles;
            const int live = min(R, a.group - run.r0);
            const int64_t row0 = static_cast<int64_t>(run.row) * a.H + run.head * a.group + run.r0;
            const float* q = a.q + (row0 + r) * D;
            const float* kt = a.k + static_cast<int64_t>(run.row) * a.G * D + run.head * D;
            constexpr int kVec = 4 * DB;  // float4s of a quarter; 8 consecutive elements are a piece
            float4 x[kVec];
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                const int d = ((i >> 1) * 4 + quarter) * 8 + (i & 1) * 4;
                x[i] = r < live && d < D ? __ldcg(reinterpret_cast<const float4*>(q + d)) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            float dot = 0.f, mx = 0.f;
            auto scale_row = [&](float4& y) {
                y = make_float4(y.x * a.scale_log2, y.y * a.scale_log2, y.z * a.scale_log2, y.w * a.scale_log2);
                mx = fmaxf(fmaxf(mx, fmaxf(fabsf(y.x), fabsf(y.y))), fmaxf(fabsf(y.z), fabsf(y.w)));
            };
#pragma unroll
            for (int i = 0; i < kVec; ++i) scale_row(x[i]);
            if (self) {  // K rounded as the cache will hold it
                auto f16 = [](float k) { return __half2float(__float2half_rn(k)); };
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    const int d = ((i >> 1) * 4 + quarter) * 8 + (i & 1) * 4;
                    if (d < D) {
                        const float4 k = __ldcg(reinterpret_cast<const float4*>(kt + d));
                        dot = fmaf(x[i].x, f16(k.x), dot);
                        dot = fmaf(x[i].y, f16(k.y), dot);
                        dot = fmaf(x[i].z, f16(k.z), dot);
                        dot = fmaf(x[i].w, f16(k.w), dot);
                    }
                }
            }
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                dot += __shfl_xor_sync(0xffffffffu, dot, o);
            }
            if (runs >= L::kQBufs) wait(L::kQFree + buf, runs / L::kQBufs - 1);
            const int e = min(127, max(-119, ((__float_as_int(mx) >> 23) & 0xff) - 127)) - 7;
            const float up = __int_as_float((127 - e) << 23);
            if (quarter == 0) {
                reinterpret_cast<float*>(smem + L::kScaleOff)[buf * 16 + r] = __int_as_float((127 + e) << 23);
                reinterpret_cast<float*>(smem + L::kSelfOff)[buf * 16 + r] = dot;
            }
            if (r < R) {
                uint8_t* qs = smem + L::kQOff + buf * L::kQBytes;
#pragma unroll
                for (int i = 0; i < kVec / 2; ++i) {
                    uint4 hi, lo;
                    split2(x[2 * i].x * up, x[2 * i].y * up, hi.x, lo.x);
                    split2(x[2 * i].z * up, x[2 * i].w * up, hi.y, lo.y);
                    split2(x[2 * i + 1].x * up, x[2 * i + 1].y * up, hi.z, lo.z);
                    split2(x[2 * i + 1].z * up, x[2 * i + 1].w * up, hi.w, lo.w);
                    const int p = i * 4 + quarter;
                    sts_uint4(qs + piece<L::kN>(r, p), hi);
                    sts_uint4(qs + piece<L::kN>(R + r, p), lo);
                }
            }
            fence_proxy_async_smem();
            mbar_arrive(&bar[L::kQFull + buf]);
            if (self && run.r0 == 0 && t < a.rows_end) {  // the new row, where the cache keeps it
                const int seq = a.sequence ? __ldcg(a.sequence + run.row) : run.row;
                const int at = __ldcg(a.table + seq * a.stride + (t >> a.page_shift));
                if (at >= 0 && at < a.pages && u0 * 8 < 2 * D) {
                    const bool value = u0 * 8 >= D;
                    const int d = u0 * 8 - (value ? D : 0);
                    const float* src = (value ? a.v + static_cast<int64_t>(run.row) * a.G * D + run.head * D : kt) + d;
                    const float4 y0 = __ldcg(reinterpret_cast<const float4*>(src)), y1 = __ldcg(reinterpret_cast<const float4*>(src) + 1);
                    uint16_t* dst = (value ? a.value : a.key) + at * a.page_stride + run.head * a.head_stride +
                                    (t & (a.page_rows - 1)) * a.row_stride + d;
                    *reinterpret_cast<uint4*>(dst) = make_uint4(pack_h2(y0.x, y0.y), pack_h2(y0.z, y0.w), pack_h2(y1.x, y1.y), pack_h2(y1.z, y1.w));
                }
            }
            ++runs;
        }
        if (!ok) lost = 1;
    } else {
        // --------------------------------------- softmax and accumulation
        const int th = tid - 128;  // a key, later an output element
        const uint32_t mine = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        float* red = reinterpret_cast<float*>(smem + L::kRedOff);
        float* sums = reinterpret_cast<float*>(smem + L::kSumsOff);
        int runs = 0, tile = 0;  // counted over all runs
        JoinWork early{}, late{};  // items that the block shares: its first run's, its last run's
        while (walk.next(a, plan, run)) {
            const int buf = runs % L::kQBufs;
            const Sight<kTile> sight(a, plan.t[run.row]);
            const bool self = a.k && run.b == run.tiles;
            const int live = min(R, a.group - run.r0);
            const int64_t row0 = static_cast<int64_t>(run.row) * a.H + run.head * a.group + run.r0;
            const int seq = a.sequence ? __ldcg(a.sequence + run.row) : run.row;
            const int32_t* table = a.table + seq * a.stride;
            auto entry = [&](int t) {  // the page of this thread's key of tile t, -1 where it is not seen
                const int p = sight.first(t) * kTile + th;
                return t < run.b && sight.sees(p) ? __ldcg(table + (p >> a.page_shift)) : -1;
            };
            int next_page = entry(run.a);
            float vs[NH];
#pragma unroll
            for (int h = 0; h < NH; ++h)
                vs[h] = self && th + 128 * h < D
                            ? __half2float(__float2half_rn(__ldcg(a.v + (static_cast<int64_t>(run.row) * a.G + run.head) * D + th + 128 * h)))
                            : 0.f;
            // the gate of this warp's rows, where the block writes them out
            float4 z[NH == 1 ? R / 4 : 1];
            if (NH == 1) {
#pragma unroll
                for (int i = 0; i < R / 4; ++i) {
                    const int j = (warp & 3) + 4 * i;
                    z[i] = a.gate && run.whole() && j < live && 4 * lane < D ? __ldcg(reinterpret_cast<const float4*>(a.gate + (row0 + j) * D) + lane)
                                                                            : make_float4(0.f, 0.f, 0.f, 0.f);
                }
            }
            wait(L::kQFull + buf, runs / L::kQBufs);
            float sc[R], b[R], m[R], l[R], o[NH][R];
#pragma unroll
            for (int j = 0; j < R; ++j) {
                sc[j] = reinterpret_cast<float*>(smem + L::kScaleOff)[buf * 16 + j];
                const float dot = reinterpret_cast<float*>(smem + L::kSelfOff)[buf * 16 + j];
                // a score that is NaN or +infinity makes the sum NaN, -infinity counts as weight 0
                const bool counts = self && dot != kNegInf, fine = dot < INFINITY;
                m[j] = !counts ? kNegInf : fine ? dot : 0.f;
                b[j] = counts ? kOff - m[j] : INFINITY;
                l[j] = counts && th == 0 ? (fine ? 0x1p11f : NAN) : 0.f;  // 2^kOff
#pragma unroll
                for (int h = 0; h < NH; ++h) o[h][j] = counts ? 0x1p11f * vs[h] : 0.f;
            }
            bool fresh = !self;  // no reference yet
            auto drain = [&](int i) {  // adds the output tile i
                wait(L::kOFull + (i & 1), i >> 1);
                tc_fence_after();
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    float hi[R], lo[R];
                    load_rows(mine + 2 * L::kN + (i & 1) * L::kOCols + h * L::kN, hi);
                    load_rows(mine + 2 * L::kN + (i & 1) * L::kOCols + h * L::kN + R, lo);
                    tc_wait_ld(hi);
                    tc_wait_ld(lo);
#pragma unroll
                    for (int j = 0; j < R; ++j) o[h][j] += hi[j] + lo[j];
                }
                tc_fence_before();
            };
            for (int t = run.a; t < run.b; ++t, ++tile) {
                const int p0 = sight.first(t) * kTile, real = sight.real(p0);
                const bool seen = static_cast<uint32_t>(next_page) < static_cast<uint32_t>(a.pages);
                next_page = entry(t + 1);
                if (!seen && th < (max(real, 1) + 15) / 16 * 16) {  // the product must not meet what this V row holds
                    const int vi = 2 * tile + 1, st = vi % kNS;
                    wait(L::kFull + st, vi / kNS);
#pragma unroll
                    for (int c = 0; c < 8 * DB; ++c) sts_uint4(smem + st * L::kItem + piece<kTile>(th, c), make_uint4(0, 0, 0, 0));
                }
                __syncwarp();
                wait(L::kSFull + (tile & 1), tile >> 1);
                tc_fence_after();
                float s[R], x[R];
                if (t == run.b - 1) mbar_arrive(&bar[L::kQFree + buf]);  // no product reads this q any more
                load_rows(mine + (tile & 1) * L::kN, s);
                load_rows(mine + (tile & 1) * L::kN + R, x);
                tc_wait_ld(s);
                tc_wait_ld(x);
                float top = kNegInf;
#pragma unroll
                for (int j = 0; j < R; ++j) {
                    s[j] = seen ? (s[j] + x[j]) * sc[j] : kNegInf;
                    x[j] = s[j] + b[j];
                    top = fmaxf(top, x[j]);
                }
                bool drained = t == run.a;
                if (group_any(1, fresh || top > kMost)) {  // a new reference: the largest score so far
                    if (!drained) drain(tile - 1);
                    drained = true;
                    float v[R];
#pragma unroll
                    for (int j = 0; j < R; ++j) v[j] = s[j];
                    fold<R>(v, [](float p, float q) { return fmaxf(p, q); });
                    if ((lane & (32 / R - 1)) == 0) red[(warp & 3) * 16 + lane / (32 / R)] = v[0];
                    named_barrier_sync(1, 128);
                    if (th < R) red[th] = fmaxf(fmaxf(red[th], red[16 + th]), fmaxf(red[32 + th], red[48 + th]));
                    named_barrier_sync(1, 128);
#pragma unroll
                    for (int j = 0; j < R; ++j) {
                        const float mn = fmaxf(m[j], red[j]);
                        const float f = m[j] == kNegInf ? 0.f : ex2(m[j] - mn);
                        m[j] = mn;
                        b[j] = mn == kNegInf ? INFINITY : kOff - mn;  // no score yet: the next one asks again
                        l[j] *= f;
#pragma unroll
                        for (int h = 0; h < NH; ++h) o[h][j] *= f;
                        x[j] = s[j] == kNegInf ? kNegInf : s[j] + b[j];
                    }
                    named_barrier_sync(1, 128);  // red is free again
                    fresh = false;
                }
                uint32_t hi[R / 2], lo[R / 2];
#pragma unroll
                for (int j = 0; j < R; j += 2) {
                    const float p0v = seen ? ex2(x[j]) : 0.f, p1v = seen ? ex2(x[j + 1]) : 0.f;
                    l[j] += p0v;
                    l[j + 1] += p1v;
                    split2(p0v, p1v, hi[j / 2], lo[j / 2]);
                }
                uint8_t* pt = smem + L::kPOff + (tile & 1) * L::kPBytes + (th >> 3) * L::kKeyRow + (th & 7) * 16;
#pragma unroll
                for (int c = 0; c < R / 8; ++c) {
                    sts_uint4(pt + c * 128, make_uint4(hi[4 * c], hi[4 * c + 1], hi[4 * c + 2], hi[4 * c + 3]));
                    sts_uint4(pt + R / 8 * 128 + c * 128, make_uint4(lo[4 * c], lo[4 * c + 1], lo[4 * c + 2], lo[4 * c + 3]));
                }
                fence_proxy_async_smem();
                tc_fence_before();
                mbar_arrive(&bar[L::kPFull + (tile & 1)]);
                if (!drained) drain(tile - 1);
            }
            drain(tile - 1);
            ++runs;
            // the rows' sums over the keys' threads, then the result or this block's part of it
            fold<R>(l, [](float p, float q) { return p + q; });
            if ((lane & (32 / R - 1)) == 0) red[(warp & 3) * 16 + lane / (32 / R)] = l[0];
            if (!ok) lost = 1;
            named_barrier_sync(1, 128);
            // outputs by rows: an output element a thread, then a row a warp
            float* stage = reinterpret_cast<float*>(smem + L::kPOff);  // P's place is free: its last product is done
            constexpr int kStage = 128 * NH;
#pragma unroll
            for (int h = 0; h < NH; ++h)
#pragma unroll
                for (int j = 0; j < R; ++j) stage[j * kStage + 128 * h + th] = o[h][j];
            if (th < R) {
                float sum = (red[th] + red[16 + th]) + (red[32 + th] + red[48 + th]);
                if (lost != 0) sum = NAN;
                sums[th] = sum;
                float mine = m[0];
#pragma unroll
                for (int j = 1; j < R; ++j) mine = th == j ? m[j] : mine;
                sums[16 + th] = mine;
            }
            named_barrier_sync(1, 128);
            const bool whole = run.whole();
            const JoinWork work = join_work(a, walk, run);
            const int64_t part = static_cast<int64_t>(part_of(blockIdx.x, work.first)) * kPagedRows;
            auto write_row = [&](int j, int d, float4 gate) {
                float4 y = lds_float4(stage + j * kStage + d);
                const float sum = sums[j];
                if (whole) {
                    y = scaled(y, sum == 0.f ? 0.f : __fdividef(1.f, sum));
                    if (a.gate) y = gated4(y, gate);
                } else if (d == 0) {
                    a.part_ml[part + j] = make_float2(sums[16 + j], sum);
                }
                *reinterpret_cast<float4*>((whole ? work.out + j * D : a.part_o + (part + j) * D) + d) = y;
            };
            if (NH == 1) {
#pragma unroll
                for (int i = 0; i < R / 4; ++i) {
                    const int j = (warp & 3) + 4 * i;
                    if (j < live && 4 * lane < D) write_row(j, 4 * lane, z[i]);
                }
            } else {
                for (int j = warp & 3; j < live; j += 4)
                    each_piece(D, lane, [&](int d) {
                        write_row(j, d, whole && a.gate ? __ldcg(reinterpret_cast<const float4*>(work.gate + j * D + d)) : make_float4(0.f, 0.f, 0.f, 0.f));
                    });
            }
            if (!whole) {
                fence_proxy_async();  // the block that joins copies the part
                if (runs == 1) early = work;
                else late = work;
            }
            named_barrier_sync(1, 128);  // what was staged has been read; the part is written
        }
        // Joins: a shared item is its block's first or last one.  The parts come
        // as bulk copies into the stages, which are free now.
        constexpr uint32_t kRing = kNS * L::kItem, kSharesOff = kRing - 4096;
        float* const buffer = reinterpret_cast<float*>(smem);
        float2* const mls = reinterpret_cast<float2*>(smem + kSharesOff);                    // [parts][16]
        float* const shares = reinterpret_cast<float*>(smem + kSharesOff + 2048);            // [parts][16]
        float* const total = shares + 16 * kJoinMost;                                        // [16]
        static_assert(kJoinMost * 128 <= 2048 && 2048 + (kJoinMost + 1) * 64 <= 4096, "the shares fit");
        int copies = 0;  // waits on the copies' barrier
        auto join = [&](const JoinWork& w, int from, int step, int count, bool final) {
            const bool gate = final && w.gate;
            // rows whose parts fit the ring
            const int most = min(w.live, static_cast<int>(kSharesOff / (static_cast<uint32_t>(count + gate) * D * 4u)));
            auto place = [&](int i) { return static_cast<int64_t>(part_of(from + i * step, w.first)) * kPagedRows; };
            for (int r0 = 0; r0 < w.live; r0 += most) {
                const int rows = min(most, w.live - r0);
                const uint32_t bytes = static_cast<uint32_t>(rows) * D * 4u;
                named_barrier_sync(1, 128);  // what the ring held has been read
                if (th < 32) {
                    fence_proxy_async();
                    if (th == 0) mbar_arrive_expect_tx(&bar[L::kJoin], (count + gate) * bytes + (r0 == 0 ? count * 128u : 0u));
                    __syncwarp();
                    if (th < count) {
                        tma_load_1d(buffer + th * rows * D, w.part_o + (place(th) + r0) * D, bytes, &bar[L::kJoin]);
                        if (r0 == 0) tma_load_1d(mls + th * 16, w.part_ml + place(th), 128, &bar[L::kJoin]);
                    } else if (gate && th == count) {
                        tma_load_1d(buffer + th * rows * D, w.gate + r0 * D, bytes, &bar[L::kJoin]);
                    }
                }
                wait(L::kJoin, copies++);
                if (!ok && th == 0)  // the copies still write into this block's memory
                    mbar_wait_bounded(&bar[L::kJoin], static_cast<uint32_t>(copies - 1) & 1u, a.status, kDevStatusTxTimeout);
                if (r0 == 0) {  // eight threads a row, up to two parts each
                    const int j = th >> 3, i = th & 7;
                    const float2 e0 = i < count ? mls[i * 16 + j] : make_float2(kNegInf, 0.f);
                    const float2 e1 = i + 8 < count ? mls[(i + 8) * 16 + j] : make_float2(kNegInf, 0.f);
                    float m = fmaxf(e0.x, e1.x);
#pragma unroll
                    for (int o = 1; o < 8; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                    // -infinity: a part without rows, whose sums are not looked at
                    const float f0 = e0.x == kNegInf && e0.y == 0.f ? kNegInf : share(e0.x, m);
                    const float f1 = e1.x == kNegInf && e1.y == 0.f ? kNegInf : share(e1.x, m);
                    float l = (f0 == kNegInf ? 0.f : f0 * e0.y) + (f1 == kNegInf ? 0.f : f1 * e1.y);
#pragma unroll
                    for (int o = 1; o < 8; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
                    if (i < count) shares[i * 16 + j] = f0;
                    if (i + 8 < count) shares[(i + 8) * 16 + j] = f1;
                    if (i == 0) {
                        total[j] = l;
                        if (!final && j < w.live) w.part_ml[place(0) + j] = make_float2(m, l);
                    }
                    named_barrier_sync(1, 128);
                }
                for (int j = warp & 3; j < rows; j += 4)
                    each_piece(D, lane, [&](int d) {
                        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                        for (int i = 0; i < count; ++i) {
                            const float f = shares[i * 16 + r0 + j];
                            const float4 v = lds_float4(buffer + (i * rows + j) * D + d);
                            if (f != kNegInf) y = make_float4(fmaf(f, v.x, y.x), fmaf(f, v.y, y.y), fmaf(f, v.z, y.z), fmaf(f, v.w, y.w));
                        }
                        if (final) {
                            const float l = total[r0 + j];
                            y = scaled(y, l == 0.f ? 0.f : __fdividef(1.f, l));
                            if (gate) y = gated4(y, lds_float4(buffer + (count * rows + j) * D + d));
                        }
                        float* to = final ? w.out + (r0 + j) * D : w.part_o + (place(0) + r0 + j) * D;
                        if (ok) *reinterpret_cast<float4*>(to + d) = y;
                    });
            }
        };
        // An item of more than kJoinMost parts is joined by groups of `step` first.
        auto step_of = [](const JoinWork& w) {
            const int count = w.last - w.first + 1;
            int step = 1;
            if (count > kJoinMost)
                while (step * step < count) ++step;
            return step;
        };
        if ((th & 31) == 0 && th < 64) {  // both tickets at once
            const JoinWork& w = th == 0 ? early : late;
            uint32_t mine = 0;
            if (w.live > 0) {
                const int step = step_of(w), count = w.last - w.first + 1;
                const int from = w.first + (static_cast<int>(blockIdx.x) - w.first) / step * step;
                mine = step > 1 ? last_of(w.ticket + part_of(from, w.first), min(step, w.last - from + 1))
                                : last_of(w.ticket + 2 * kPagedMaxBlocks + w.first, count);
            }
            joining[th >> 5] = mine;
        }
        named_barrier_sync(1, 128);
#pragma unroll 1
        for (int it = 0; it < 2; ++it) {
            if (joining[it] == 0) continue;
            const JoinWork w = it == 0 ? early : late;
            const int count = w.last - w.first + 1, step = step_of(w), groups = (count + step - 1) / step;
            bool final = step == 1;
            int from = final ? w.first : w.first + (static_cast<int>(blockIdx.x) - w.first) / step * step;
            int stride = 1, parts = final ? count : min(step, w.last - from + 1);
#pragma unroll 1
            for (;;) {
                join(w, from, stride, parts, final);
                if (final) break;
                fence_proxy_async();
                named_barrier_sync(1, 128);
                if (th == 0) joining[it] = last_of(w.ticket + 2 * kPagedMaxBlocks + w.first, groups);
                named_barrier_sync(1, 128);
                if (joining[it] == 0) break;
                from = w.first;
                stride = step;
                parts = groups;
                final = true;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_free(tmem, L::kTmemCols);
    }
}

// The kernel's attribute, once per device.
template <int R, int DB>
bool ready() {
    struct Ready {};
    return device_once<R * 8 + DB, Ready>([](Ready&) {
               const cudaError_t e = cudaFuncSetAttribute(paged_tc_kernel<R, DB>, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<R, DB>::kBytes);
               return e == cudaSuccess ? static_cast<int>(MUSER_OK) : cuda_fail(e, "paged attention: cudaFuncSetAttribute");
           }) != nullptr;
}

template <int R, int DB>
int launch(const PagedArgs& a, const CUtensorMap& k, const CUtensorMap& v, int blocks, cudaStream_t s) {
    if (!ready<R, DB>()) return MUSER_ERR_CUDA;  // the message is set
    return launch_after("paged attention", paged_tc_kernel<R, DB>, dim3(static_cast<unsigned>(blocks)), kThreads,
                        Layout<R, DB>::kBytes, 1, s, a, k, v);
}

template <int R>
int launch_d(const PagedArgs& a, const CUtensorMap& k, const CUtensorMap& v, int blocks, cudaStream_t s) {
    if (a.D <= 64) return launch<R, 1>(a, k, v, blocks, s);
    if (a.D <= 128) return launch<R, 2>(a, k, v, blocks, s);
    return launch<R, 4>(a, k, v, blocks, s);
}

}  // namespace

bool paged_tc_supported(const PagedArgs& a) {
    constexpr int64_t kMost = int64_t{1} << 39;  // a tensor map's strides are below 2^40 bytes
    return a.D % 8 == 0 && a.D <= 256 && a.page_rows >= 8 && (a.page_rows & (a.page_rows - 1)) == 0 && is_aligned(a.key, 16) &&
           is_aligned(a.value, 16) && a.page_stride < kMost && (!a.k || is_aligned(a.k, 16)) && (!a.v || is_aligned(a.v, 16));
}

int launch_paged_tc(const PagedArgs& a, int blocks, cudaStream_t s) {
    CUtensorMap maps[2];
    const uint64_t dims[4] = {static_cast<uint64_t>(a.D), static_cast<uint64_t>(a.page_rows), static_cast<uint64_t>(a.G),
                              static_cast<uint64_t>(a.pages)};
    const uint64_t strides[3] = {static_cast<uint64_t>(a.row_stride) * 2, static_cast<uint64_t>(a.head_stride) * 2,
                                 static_cast<uint64_t>(a.page_stride) * 2};
    MUSER_TRY(encode_page_maps(a.key, a.value, dims, strides, std::min(a.page_rows, kTile), maps));
    return a.group <= 8 ? launch_d<8>(a, maps[0], maps[1], blocks, s) : launch_d<16>(a, maps[0], maps[1], blocks, s);
}

}  // namespace muser
