// pages.cu -- page tables of several sequences from their lengths, the copy of
// pages that no longer are shared, and the store of rows into pages.
#include <algorithm>

#include "kernels.cuh"
#include "pages.cuh"

namespace muser {
namespace {

// ------------------------------------------------------------- page tables
// Which pages are free is found anew in every call: a bit per page, set for
// every live entry of the new tables (mark), then counted (sweep).  No counts
// of references are kept between calls, so nothing can get out of step with
// the tables, and the same inputs give the same tables.  A page that a row goes
// on to fill is no mark of that row itself: if its bit is set in the end, or an
// earlier row fills it too, the row needs a copy.
//
// One cluster: its first block keeps the bits in shared memory, all blocks set
// them there (reductions over distributed shared memory), and the first one
// counts and gives pages out; then all blocks write the slots.
// Bound: latency, a dozen dependent steps of about 0.7 us (16 beams of 500 to
// 8,000 rows, one block: 7.8 us; 48 prompts, 48,000 new rows: 13.9 us with
// sixteen, 15.5 with eight).
//
// Sixteen blocks (or what the device can place) where the slots are many, since
// all of them write these; their marks cross to the first block's memory and are
// slower than its own, the slower the more entries live.  us, one block and
// sixteen: 48 sequences of 30 to 5,000 rows, pages of 16, 4,000 slots 11.0 and
// 12.2, 8,200 13.5 and 12.2, 48,000 31.9 and 13.9; without slots 16 of 500 to
// 8,000 in tables of 2,048 entries 7.6 and 9.4, of 30,000 to 120,000 (16,406
// live entries) 12.4 and 18.1, 128 of these 54 and 102.  Rows of more than 128
// sequences are marked in many turns: 256 of 250 to 1,000 rows 25.8 and 20.8,
// tables of 128 entries with 4,033 live ones 26.2 and 22.4, with 17,447 28.5 and
// 30.8; longer tables, when full, 41 and 63.
constexpr int kTabThreads = 1024, kTabWarps = kTabThreads / 32, kRows = kMaxSequences;

struct TabShared {
    int32_t parent[kRows], keep[kRows], rows[kRows], own[kRows];  // own: the page a row goes on in, or -1
    int32_t need_end[kRows];   // pages given to the rows up to this one
    int32_t copy[kRows];
    int32_t held[kRows];       // pages of the rows that stay
    int32_t new_end[kRows];    // new rows up to this one's; beyond 2^31 - 1 they are too many anyhow
    int32_t task_end[kRows];   // runs of entries of the rows up to this one
    int32_t copy_at[kRows];
    int32_t free_end[kTabThreads];  // free pages in the words of the threads up to this one
    int64_t warp64[kTabWarps][1];
    int32_t warp1[kTabWarps][1], warp3[kTabWarps][3];
    int64_t total_new;
    int32_t listed;            // new rows that get slots
    int32_t status, total_need, total_copy, free;
};
constexpr int kEach = 8;  // entries of a lane's turn

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// The first i in 0..n-1 with end[i] > x (there is one).
template <typename T>
__device__ __forceinline__ int find_row(const T* end, int n, T x) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (end[mid] > x) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

// Inclusive prefix sums of N values over the block's threads; `warp` has N
// entries a warp.
template <typename T, int N>
__device__ __forceinline__ void block_scan(T (&v)[N], T (*warp)[N]) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const T x = __shfl_up_sync(0xffffffffu, v[i], o);
            if (lane >= o) v[i] += x;
        }
    if (lane == 31)
#pragma unroll
        for (int i = 0; i < N; ++i) warp[w][i] = v[i];
    __syncthreads();
    T before[N] = {}, mine[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        mine[i] = lane < w ? warp[lane][i] : T{0};
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mine[i] += __shfl_xor_sync(0xffffffffu, mine[i], o);
        before[i] = mine[i];
        v[i] += before[i];
    }
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t map_first(uint32_t addr) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
    return r;
}
__device__ __forceinline__ void red_or(uint32_t addr, uint32_t v) {
    asm volatile("red.relaxed.cluster.shared::cluster.or.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__global__ void __launch_bounds__(kTabThreads, 1) page_tables_kernel(const __grid_constant__ PageTableArgs a) {
    extern __shared__ __align__(16) uint32_t bits[];
    __shared__ TabShared S;
    const int tid = threadIdx.x, lane = tid & 31;
    const int rank = static_cast<int>(cluster_rank()), ranks = static_cast<int>(cluster_size());
    const int R = a.page_rows, words = (a.pages + 31) / 32;
    pdl_launch_dependents();
    if (rank == 0)
        for (int w = tid; w < words; w += kTabThreads) {
            const int left = a.pages - 32 * w;  // bits behind the last page count as held
            bits[w] = left >= 32 ? 0u : 0xffffffffu << left;
        }
    if (tid == 0) S.status = 0;
    __syncthreads();
    pdl_wait();
    // the rows, in every block for itself
    int tasks = 0;
    if (tid < a.n) {
        int p = a.parent ? __ldcg(a.parent + tid) : tid;
        if (p < 0 || p >= a.n_old) p = -1;
        const int64_t most = a.stride * R;
        const int old = p < 0 ? 0 : static_cast<int>(min(static_cast<int64_t>(max(0, __ldcg(a.length + p))), most));
        const int64_t now = max(int64_t{0}, static_cast<int64_t>(old) + (a.add ? __ldcg(a.add + tid) : 1));
        const int keep = static_cast<int>(min(static_cast<int64_t>(old), now));
        if (now > most) S.status = 2;
        S.parent[tid] = p;
        S.keep[tid] = keep;
        S.rows[tid] = static_cast<int>(min(now, most));
        S.own[tid] = now > keep && keep % R != 0 ? __ldcg(a.table + p * a.stride + keep / R) : -1;
        if (now > keep && keep % R != 0 && (S.own[tid] < 0 || S.own[tid] >= a.pages)) S.own[tid] = -2;  // there is none: a new page, nothing to copy
        tasks = ceil_div(ceil_div(keep, R), 32 * kEach);
    }
    int task_end[1] = {tasks};
    block_scan(task_end, S.warp1);
    if (tid < a.n) S.task_end[tid] = task_end[0];
    if (ranks > 1) cluster_sync();  // the first block's bits are clear
    else __syncthreads();
    // mark, and copy the entries that stay
    const uint32_t first_bits = map_first(smem_u32(bits));
    const bool in_place = a.table_out == a.table;
    const int total_tasks = S.task_end[a.n - 1];
    for (int t = rank * kTabWarps + (tid >> 5); t < total_tasks; t += ranks * kTabWarps) {
        const int i = find_row(S.task_end, a.n, t);
        const int k0 = (t - (i == 0 ? 0 : S.task_end[i - 1])) * 32 * kEach + lane;
        const int keep = S.keep[i], held = ceil_div(keep, R);
        const bool grows = S.rows[i] > keep && keep % R != 0;
        const int32_t* src = a.table + S.parent[i] * a.stride;
        int32_t* dst = a.table_out + i * a.stride;
        int e[kEach];
#pragma unroll
        for (int u = 0; u < kEach; ++u) e[u] = k0 + 32 * u < held ? __ldcg(src + k0 + 32 * u) : -1;
#pragma unroll
        for (int u = 0; u < kEach; ++u) {
            const int k = k0 + 32 * u;
            if (k >= held) break;
            const int64_t end = (static_cast<int64_t>(k) + 1) * R;
            const bool live = a.window == 0 || end - R < a.n_sink || end > static_cast<int64_t>(keep) - a.window + 1;
            if (!live) {
                dst[k] = -1;
                continue;
            }
            if (!in_place) dst[k] = e[u];
            if (e[u] >= 0 && e[u] < a.pages && !(grows && k == held - 1))
                red_or(first_bits + (static_cast<uint32_t>(e[u]) >> 5) * 4u, 1u << (e[u] & 31));
        }
    }
    if (ranks > 1) cluster_sync();
    else __syncthreads();
    if (rank == 0) {
        // whose page is another's too
        const int own = tid < a.n ? S.own[tid] : -1;
        int copy = own == -2 ? 1 : 0;
        if (own >= 0) {
            copy = (bits[own >> 5] >> (own & 31)) & 1u;
            for (int j = 0; j < tid && !copy; ++j) copy = S.own[j] == own;
        }
        __syncthreads();
        if (own >= 0 && !copy) atomicOr(&bits[own >> 5], 1u << (own & 31));
        int need = 0;
        int64_t fresh = 0;
        if (tid < a.n) {
            need = min(copy + ceil_div(S.rows[tid], R) - ceil_div(S.keep[tid], R), a.pages + 1);  // more than there are is too many
            fresh = S.rows[tid] - S.keep[tid];
            S.copy[tid] = copy;
            S.held[tid] = ceil_div(S.keep[tid], R);
        }
        const bool listed = copy && own >= 0;
        __syncthreads();
        // sweep: a thread counts the free pages of a run of words
        const int per = ceil_div(words, kTabThreads), w0 = min(words, tid * per), w1 = min(words, w0 + per);
        int free = 0;
        for (int w = w0; w < w1; ++w) free += __popc(~bits[w]);
        int sums[3] = {need, listed ? 1 : 0, free};
        int64_t new_sum[1] = {fresh};
        block_scan(sums, S.warp3);
        block_scan(new_sum, S.warp64);
        const int64_t new_end = new_sum[0];
        if (tid < a.n) {
            S.need_end[tid] = sums[0];
            S.new_end[tid] = static_cast<int32_t>(min(new_end, int64_t{0x7fffffff}));
            S.copy_at[tid] = sums[1] - (listed ? 1 : 0);
        }
        S.free_end[tid] = sums[2];
        if (tid == kTabThreads - 1) {
            S.free = sums[2];
            S.total_need = sums[0];
            S.total_new = new_end;
            S.total_copy = sums[1];
            if (S.status == 0) {
                if (sums[1] > 0 && a.copies == nullptr) S.status = 4;
                else if (new_end > a.max_new && (a.slots || a.position || a.sequence)) S.status = 3;
                else if (sums[0] > sums[2]) S.status = 1;
            }
        }
        __syncthreads();
        const bool done = S.status == 0;
        const int give = done ? S.total_need : 0;
        // a warp takes a thread's words, a lane a page of each: its rank among the free ones
        for (int owner = tid >> 5; owner < kTabThreads; owner += kTabWarps) {
            int base = owner == 0 ? 0 : S.free_end[owner - 1];
            if (base >= give) break;
            const int end = min(words, (owner + 1) * per);
            for (int w = owner * per; w < end; ++w) {
                const uint32_t open = ~bits[w];
                const int at = base + __popc(open & ((1u << lane) - 1u));
                base += __popc(open);
                if (!((open >> lane) & 1u) || at >= give) continue;
                const int page = 32 * w + lane, i = find_row(S.need_end, a.n, at);
                const int j = at - (i == 0 ? 0 : S.need_end[i - 1]);
                a.table_out[i * a.stride + S.held[i] + j - S.copy[i]] = page;
                if (j == 0 && S.copy[i] && S.own[i] >= 0) {
                    int32_t* c = a.copies + 3 * S.copy_at[i];
                    c[0] = S.own[i];
                    c[1] = page;
                    c[2] = S.keep[i] % R;
                }
            }
        }
        if (tid < a.n) {
            const int keep = S.keep[tid], rows = done ? S.rows[tid] : keep;
            a.length_out[tid] = rows;
            if (a.last) a.last[tid] = rows > keep ? rows - 1 : -1;
            if (a.first) {
                if (tid == 0) a.first[0] = 0;
                a.first[tid + 1] = done ? static_cast<int32_t>(min(new_end, int64_t{0x7fffffff})) : 0;
            }
        }
        if (tid < 8) {
            const int v[8] = {S.status, done ? static_cast<int>(min(S.total_new, int64_t{0x7fffffff})) : 0,
                              done ? S.total_copy : 0, give, S.free - give, 0, 0, 0};
            int mine = 0;
#pragma unroll
            for (int u = 0; u < 8; ++u) mine = tid == u ? v[u] : mine;
            a.result[tid] = mine;
        }
        if (tid == 0) S.listed = done ? static_cast<int32_t>(min(S.total_new, int64_t{0x7fffffff})) : 0;
        __threadfence();  // the tables, for the other blocks
    }
    if (!(a.slots || a.position || a.sequence)) {
        return;  // no block reads another's memory from here on
    }
    if (ranks > 1) cluster_sync();
    else __syncthreads();
    if (rank != 0) {  // the rows' ends from the first block
        auto fetch = [](const int32_t* p) {
            int32_t v;
            asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(map_first(smem_u32(p))) : "memory");
            return v;
        };
        if (tid < a.n) S.new_end[tid] = fetch(&S.new_end[tid]);
        if (tid == 0) S.listed = fetch(&S.listed);
    }
    if (ranks > 1) cluster_sync();  // the first block leaves when its memory has been read
    else __syncthreads();
    // A warp takes 32 * kSlots new rows in a row: their sequence is searched for
    // once and followed from there, their table entries are on the way together.
    const int total = S.listed;
    constexpr int kSlots = 4;
    const int shift = (R & (R - 1)) == 0 ? __ffs(R) - 1 : -1;
    for (int64_t j0 = (static_cast<int64_t>(rank) * kTabWarps + (tid >> 5)) * 32 * kSlots; j0 < a.max_new;
         j0 += static_cast<int64_t>(ranks) * kTabThreads * kSlots) {
        int slot[kSlots], pos[kSlots], seq[kSlots], at = j0 < total ? find_row(S.new_end, a.n, static_cast<int>(j0)) : 0;
#pragma unroll
        for (int u = 0; u < kSlots; ++u) {
            const int64_t j = j0 + 32 * u + lane;
            slot[u] = pos[u] = seq[u] = -1;
            if (j < total) {
                while (S.new_end[at] <= j) ++at;
                seq[u] = at;
                pos[u] = S.keep[at] + static_cast<int>(j - (at == 0 ? 0 : S.new_end[at - 1]));
                slot[u] = __ldcg(a.table_out + at * a.stride + (shift >= 0 ? pos[u] >> shift : pos[u] / R));
            }
        }
#pragma unroll
        for (int u = 0; u < kSlots; ++u) {
            const int64_t j = j0 + 32 * u + lane;
            if (j >= a.max_new) break;
            if (a.slots) a.slots[j] = seq[u] < 0 ? -1 : slot[u] * R + (shift >= 0 ? pos[u] & (R - 1) : pos[u] % R);
            if (a.position) a.position[j] = pos[u];
            if (a.sequence) a.sequence[j] = seq[u];
        }
    }
}

// ------------------------------------------------------------------- copy
// Bound: the rows' bytes, read and written once (15 pages of 52 layers, 52 MB:
// 11.3 to 13.8 us, of which 4 are the launch and, one behind the other, the
// reads of the count and of a triple).  A block takes a part of a page of a
// layer's keys or values, all its loads in flight before the first store; blocks
// go round, since how many copies there are is known on the device only.
constexpr int kCopyThreads = 128;

template <int N>
struct PageCopyParams {
    PageCopyArgs a;  // its buffers are not used
    uint16_t* buffer[2 * N];
};

template <int N, bool VEC>
__global__ void __launch_bounds__(kCopyThreads) page_copy_kernel(const __grid_constant__ PageCopyParams<N> p, int parts) {
    const PageCopyArgs& a = p.a;
    pdl_launch_dependents();
    pdl_wait();
    const int count = min(max(0, __ldcg(a.count)), a.max_copies);
    const int64_t items = static_cast<int64_t>(count) * 2 * a.n_layers * parts;
    constexpr int kStep = VEC ? 8 : 1;
    const int row = a.run_dim / kStep;  // pieces of a row of a run
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int part = static_cast<int>(item % parts), which = static_cast<int>(item / parts % (2 * a.n_layers));
        const int32_t* c = a.copies + 3 * (item / parts / (2 * a.n_layers));
        const int src = __ldcg(c), dst = __ldcg(c + 1), rows = min(__ldcg(c + 2), a.page_rows);
        if (src < 0 || src >= a.pages || dst < 0 || dst >= a.pages || rows <= 0) continue;
        const int64_t page = static_cast<int64_t>(a.runs) * a.page_rows * a.run_dim;
        const uint16_t* from = p.buffer[which] + src * page;
        uint16_t* to = p.buffer[which] + dst * page;
        const unsigned run = static_cast<unsigned>(rows * row);  // pieces of a run; the next one is page_rows * row further
        const unsigned total = run * a.runs;
        const unsigned x0 = static_cast<unsigned>(static_cast<uint64_t>(total) * part / parts);
        const unsigned x1 = static_cast<unsigned>(static_cast<uint64_t>(total) * (part + 1) / parts);
        constexpr int U = 8;
        for (unsigned x = x0 + threadIdx.x; x < x1; x += U * kCopyThreads) {
            int at[U];
            uint4 v[U];
            uint16_t h[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const unsigned y = x + u * kCopyThreads;
                at[u] = y < x1 ? static_cast<int>((y / run * a.page_rows * row + y % run) * kStep) : -1;
                if (at[u] >= 0) {
                    if (VEC) v[u] = __ldcg(reinterpret_cast<const uint4*>(from + at[u]));
                    else h[u] = __ldcg(from + at[u]);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (at[u] >= 0) {
                    if (VEC) *reinterpret_cast<uint4*>(to + at[u]) = v[u];
                    else to[at[u]] = h[u];
                }
        }
    }
}

// ------------------------------------------------------------------ write
// Bound: 4 bytes read and 2 written an element (40,007 rows of 256, 123 MB:
// 20.4 us, 6.03 TB/s).  A thread takes 8 elements of a row of K and of V (or
// one, where rows are not 16-byte aligned).
constexpr int kWriteThreads = 256;

template <bool VEC>
__global__ void __launch_bounds__(kWriteThreads) page_write_kernel(const __grid_constant__ PageWriteArgs a) {
    pdl_launch_dependents();
    pdl_wait();
    constexpr int kStep = VEC ? 8 : 1;
    const int per = a.kv_dim / kStep;
    const int64_t total = a.rows * per;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kWriteThreads + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * kWriteThreads) {
        const int64_t j = i / per, src = i * kStep;
        const int e = static_cast<int>(i - j * per) * kStep;
        const int64_t slot = __ldcg(a.slots + j);
        if (slot < 0 || slot >= a.slot_end) continue;
        int64_t dst = slot * a.kv_dim + e;
        if (a.head_major) {
            const int64_t page = slot / a.page_rows;
            const int heads = a.kv_dim / a.head_dim, head = e / a.head_dim;
            dst = ((page * heads + head) * a.page_rows + (slot - page * a.page_rows)) * a.head_dim + (e - head * a.head_dim);
        }
        if (VEC) {
            const float4 k0 = __ldcg(reinterpret_cast<const float4*>(a.k + src)), k1 = __ldcg(reinterpret_cast<const float4*>(a.k + src + 4));
            const float4 v0 = __ldcg(reinterpret_cast<const float4*>(a.v + src)), v1 = __ldcg(reinterpret_cast<const float4*>(a.v + src + 4));
            const auto pack = [](float lo, float hi) {
                const __half2 h = __floats2half2_rn(lo, hi);
                return *reinterpret_cast<const uint32_t*>(&h);
            };
            *reinterpret_cast<uint4*>(a.key + dst) = make_uint4(pack(k0.x, k0.y), pack(k0.z, k0.w), pack(k1.x, k1.y), pack(k1.z, k1.w));
            *reinterpret_cast<uint4*>(a.value + dst) = make_uint4(pack(v0.x, v0.y), pack(v0.z, v0.w), pack(v1.x, v1.y), pack(v1.z, v1.w));
        } else {
            a.key[dst] = __half_as_ushort(__float2half_rn(__ldcg(a.k + src)));
            a.value[dst] = __half_as_ushort(__float2half_rn(__ldcg(a.v + src)));
        }
    }
}

struct Ready {
    int cluster;  // the most blocks that the device can place together
};

}  // namespace

int launch_page_tables(const PageTableArgs& a, cudaStream_t s) {
    const Ready* r = device_once<0, Ready>([](Ready& x) {
        constexpr int kSmem = static_cast<int>(kMaxPages / 8);
        cudaError_t e = cudaFuncSetAttribute(page_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(page_tables_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return cuda_fail(e, "page tables: cudaFuncSetAttribute");
        x.cluster = largest_cluster([](int size) {
            cudaLaunchConfig_t cfg{};
            cudaLaunchAttribute attr[1];
            cfg.gridDim = dim3(static_cast<unsigned>(size));
            cfg.blockDim = dim3(kTabThreads);
            cfg.dynamicSmemBytes = kSmem;
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = static_cast<unsigned>(size);
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            int clusters = 0;
            if (cudaOccupancyMaxActiveClusters(&clusters, page_tables_kernel, &cfg) != cudaSuccess) {
                cudaGetLastError();
                return false;
            }
            return clusters > 0;
        });
        return static_cast<int>(MUSER_OK);
    });
    if (r == nullptr) return MUSER_ERR_CUDA;  // the message is set
    const bool many = a.max_new > 8192 || (a.n > 128 && a.n * a.stride <= 32768);
    const int cluster = many ? r->cluster : 1;
    return launch_after("page tables", page_tables_kernel, dim3(static_cast<unsigned>(cluster)), kTabThreads,
                        static_cast<size_t>((a.pages + 31) / 32) * 4u, cluster, s, a);
}

int launch_page_copy(const PageCopyArgs& a, cudaStream_t s) {
    const int64_t most = static_cast<int64_t>(a.max_copies) * 2 * a.n_layers, page = static_cast<int64_t>(a.runs) * a.page_rows * a.run_dim;
    const int blocks = 8 * std::max(1, sm_count());
    // parts of at least 8 KB, while there are blocks for them
    const int parts = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({blocks / most, page / 4096, 64})));
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>(most * parts, blocks)));
    auto go = [&](auto size) {
        constexpr int N = decltype(size)::value;
        PageCopyParams<N> p;
        p.a = a;
        std::copy(a.buffer, a.buffer + 2 * a.n_layers, p.buffer);
        return a.vec ? launch_after("page copy", page_copy_kernel<N, true>, grid, kCopyThreads, 0, 1, s, p, parts)
                     : launch_after("page copy", page_copy_kernel<N, false>, grid, kCopyThreads, 0, 1, s, p, parts);
    };
    if (a.n_layers <= 64) return go(std::integral_constant<int, 64>{});
    return go(std::integral_constant<int, kPageCopyMaxLayers>{});
}

int launch_page_write(const PageWriteArgs& a, cudaStream_t s) {
    const int64_t items = a.rows * (a.kv_dim / (a.vec ? 8 : 1));
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>((items + kWriteThreads - 1) / kWriteThreads, 16 * std::max(1, sm_count()))));
    return a.vec ? launch_after("page write", page_write_kernel<true>, grid, kWriteThreads, 0, 1, s, a)
                 : launch_after("page write", page_write_kernel<false>, grid, kWriteThreads, 0, 1, s, a);
}

}  // namespace muser
