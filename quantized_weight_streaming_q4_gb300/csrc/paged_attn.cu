// paged_attn.cu -- attention of one token row each of several sequences over a
// paged K/V cache: the kernel for any head and page size, and the choice.
#include <algorithm>

#include "kernels.cuh"
#include "paged.cuh"

namespace muser {
namespace {

// ------------------------------------------------------- joining the parts
template <bool VEC>
__device__ __forceinline__ float4 load4(const float* p, int left) {
    if (VEC) return __ldcg(reinterpret_cast<const float4*>(p));
    return make_float4(__ldcg(p), left > 1 ? __ldcg(p + 1) : 0.f, left > 2 ? __ldcg(p + 2) : 0.f, left > 3 ? __ldcg(p + 3) : 0.f);
}
template <bool VEC>
__device__ __forceinline__ void store4(float* p, float4 v, int left) {
    if (VEC) {
        *reinterpret_cast<float4*>(p) = v;
        return;
    }
    p[0] = v.x;
    if (left > 1) p[1] = v.y;
    if (left > 2) p[2] = v.z;
    if (left > 3) p[3] = v.w;
}
// `count` parts, the first that of block `from` and each of a block `step`
// further, are joined, into the item's result or (!final) into the first part.
// A warp (w of W) takes every W-th row, two at a time; its lanes hold the
// parts' shares.
template <bool VEC>
__device__ __noinline__ void join_parts(const JoinWork a, int from, int step, int count, int w, int W, bool final) {
    constexpr int B = 10, U = 2;  // loads in flight of a row, rows
    const int lane = threadIdx.x & 31, live = a.live;
    // part i's row j
    auto place = [&](int i, int j) { return static_cast<int64_t>(part_of(from + i * step, a.first)) * kPagedRows + j; };
    for (int j0 = w; j0 < live; j0 += U * W) {
        float2 ml[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            ml[u] = lane < count && j0 + u * W < live ? __ldcg(a.part_ml + place(lane, j0 + u * W)) : make_float2(kNegInf, 0.f);
        for (int d = 4 * lane; d - 4 * lane < a.D; d += 128) {
            float4 z[U], o[U];
            float m[U], l[U], f[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                o[u] = z[u] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (final && a.gate && d < a.D && j0 + u * W < live) z[u] = load4<VEC>(a.gate + static_cast<int64_t>(j0 + u * W) * a.D + d, a.D - d);
            }
            for (int i0 = 0; i0 < count; i0 += B) {
                float4 v[U][B];
#pragma unroll
                for (int i = 0; i < B; ++i)
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        v[u][i] = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (i0 + i < count && d < a.D && j0 + u * W < live)
                            v[u][i] = load4<VEC>(a.part_o + place(i0 + i, j0 + u * W) * a.D + d, a.D - d);
                    }
                if (i0 == 0) {  // the shares, while the sums are on the way
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        m[u] = ml[u].x;
#pragma unroll
                        for (int x = 16; x > 0; x >>= 1) m[u] = fmaxf(m[u], __shfl_xor_sync(0xffffffffu, m[u], x));
                        const bool empty = ml[u].x == kNegInf && ml[u].y == 0.f;  // no rows there: its sums are not looked at
                        f[u] = empty ? kNegInf : share(ml[u].x, m[u]);
                        l[u] = warp_sum(empty ? 0.f : f[u] * ml[u].y);
                    }
                }
#pragma unroll
                for (int i = 0; i < B; ++i)
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const float fi = __shfl_sync(0xffffffffu, f[u], i0 + i);
                        if (i0 + i < count && fi != kNegInf)
                            o[u] = make_float4(fmaf(fi, v[u][i].x, o[u].x), fmaf(fi, v[u][i].y, o[u].y), fmaf(fi, v[u][i].z, o[u].z), fmaf(fi, v[u][i].w, o[u].w));
                    }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int j = j0 + u * W;
                if (d >= a.D || j >= live) continue;
                if (final) {
                    const float4 y = scaled(o[u], l[u] == 0.f ? 0.f : __fdividef(1.f, l[u]));
                    store4<VEC>(a.out + static_cast<int64_t>(j) * a.D + d, a.gate ? gated4(y, z[u]) : y, a.D - d);
                } else {
                    store4<VEC>(a.part_o + place(0, j) * a.D + d, o[u], a.D - d);
                    if (d == 0) a.part_ml[place(0, j)] = make_float2(m[u], l[u]);
                }
            }
        }
    }
}

// After the block's part of an item is written and a barrier passed: what is
// left to join, if this is the last block to get there.  All of the block's
// `threads` threads call it; `flag` is in shared memory.
template <bool VEC>
__device__ __noinline__ void finish_item(const JoinWork a, int tid, int threads, volatile uint32_t* flag) {
    const int count = a.last - a.first + 1, w = tid >> 5, W = threads >> 5;
    int step = 1, parts = count;
    if (count > kJoinMost) {
        while (step * step < count) ++step;  // as many groups as parts in each
        const int from = a.first + (static_cast<int>(blockIdx.x) - a.first) / step * step, size = min(step, a.last - from + 1);
        if (tid == 0) *flag = last_of(a.ticket + part_of(from, a.first), size);
        __syncthreads();
        if (!*flag) return;
        join_parts<VEC>(a, from, 1, size, w, W, false);
        parts = (count + step - 1) / step;
        __syncthreads();
    }
    if (tid == 0) *flag = last_of(a.ticket + 2 * kPagedMaxBlocks + a.first, parts);
    __syncthreads();
    if (*flag) join_parts<VEC>(a, a.first, step, parts, w, W, true);
}
// --------------------------------------------------- any size, CUDA cores
// As the tree attention's kernel for any head size: 32 rows at a time in shared
// memory as binary32, a lane scores one row, then owns the output elements d =
// lane, lane + 32, ...; one pass with the running maximum and sum.
constexpr int kTile = 32, kThreads = 256, kWarps = kThreads / 32, kQ = kPagedRows / kWarps;
constexpr int kMaxD = 256;
constexpr size_t smem_bytes(int D) {
    const size_t n = (2 * kTile * (D + 1) + kPagedRows * D) * sizeof(float);
    return n < 512 ? 512 : n;  // the plan's sums
}
static_assert(smem_bytes(128) <= 46 * 1024, "heads up to 128 need no attribute");

template <int ND>  // output elements per lane: D <= 32 * ND
__global__ void __launch_bounds__(kThreads) paged_generic_kernel(const __grid_constant__ PagedArgs a) {
    extern __shared__ float sm[];
    __shared__ PagedPlan plan;
    __shared__ int32_t slot[kTile];  // a row's page * page_rows + row, or -1
    __shared__ uint32_t flag;
    const int D = a.D, DP = D + 1;
    float* ks = sm;
    float* vs = ks + kTile * DP;
    float* qs = vs + kTile * DP;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_launch_dependents();
    pdl_wait();
    PagedWalk<kTile> walk(a, make_plan<kTile>(a, plan, reinterpret_cast<uint32_t*>(sm)));
    PagedRun run;
    while (walk.next(a, plan, run)) {
        __syncthreads();  // the plan's sums, and the run before, are done with what `sm` held
        const Sight<kTile> sight(a, plan.t[run.row]);
        const int live = min(kPagedRows, a.group - run.r0);
        const int seq = a.sequence ? __ldcg(a.sequence + run.row) : run.row;
        const int32_t* table = a.table + seq * a.stride;
        const int64_t row0 = static_cast<int64_t>(run.row) * a.H + run.head * a.group + run.r0;
        const float* kt = a.k + static_cast<int64_t>(run.row) * a.G * D + run.head * D;
        const float* vt = a.v + static_cast<int64_t>(run.row) * a.G * D + run.head * D;
        const bool self = a.k && run.b == run.tiles;
        for (int x = tid; x < kPagedRows * D; x += kThreads) qs[x] = x / D < live ? __ldcg(a.q + row0 * D + x) : 0.f;
        if (self && run.r0 == 0 && sight.t < a.rows_end) {  // the new row, where the cache keeps it
            const int page = __ldcg(table + sight.t / a.page_rows), r = sight.t % a.page_rows;
            if (page >= 0 && page < a.pages) {
                const int64_t at = page * a.page_stride + run.head * a.head_stride + r * a.row_stride;
                for (int d = tid; d < D; d += kThreads) {
                    a.key[at + d] = __half_as_ushort(__float2half_rn(__ldcg(kt + d)));
                    a.value[at + d] = __half_as_ushort(__float2half_rn(__ldcg(vt + d)));
                }
            }
        }
        float m[kQ], l[kQ], o[kQ][ND];
#pragma unroll
        for (int u = 0; u < kQ; ++u) {
            m[u] = kNegInf;
            l[u] = 0.f;
#pragma unroll
            for (int e = 0; e < ND; ++e) o[u][e] = 0.f;
        }
        for (int t = run.a; t < run.b + (self ? 1 : 0); ++t) {
            const bool own = t == run.b;
            const int p0 = sight.first(t) * kTile, n = own ? 1 : sight.real(p0);
            __syncthreads();
            if (tid < kTile && !own) {
                const int p = p0 + tid;
                int s = -1;
                if (tid < n && sight.sees(p)) {
                    const int page = __ldcg(table + p / a.page_rows);
                    if (page >= 0 && page < a.pages) s = page * a.page_rows + p % a.page_rows;
                }
                slot[tid] = s;
            }
            if (own && tid == 0) slot[0] = 0;
            __syncthreads();
            for (int x = tid; x < n * D; x += kThreads) {
                const int r = x / D, d = x - r * D;
                float k = 0.f, v = 0.f;
                if (own) {
                    k = __half2float(__float2half_rn(__ldcg(kt + d)));
                    v = __half2float(__float2half_rn(__ldcg(vt + d)));
                } else if (slot[r] >= 0) {
                    const int64_t at = (slot[r] / a.page_rows) * a.page_stride + run.head * a.head_stride +
                                       (slot[r] % a.page_rows) * a.row_stride + d;
                    k = h2f(__ldcg(a.key + at));
                    v = h2f(__ldcg(a.value + at));
                }
                ks[r * DP + d] = k;
                vs[r * DP + d] = v;
            }
            __syncthreads();
            const bool mine = lane < n && slot[lane] >= 0;
            const uint32_t seen = __ballot_sync(0xffffffffu, mine);
            if (seen == 0) continue;
#pragma unroll
            for (int u = 0; u < kQ; ++u) {
                const int r = warp * kQ + u;
                if (r >= live) break;
                float s = kNegInf;
                if (mine) {
                    float acc = 0.f;
                    for (int d = 0; d < D; ++d) acc = fmaf(qs[r * D + d], ks[lane * DP + d], acc);
                    s = acc * a.scale_log2;
                }
                float tm = s;
#pragma unroll
                for (int x = 16; x > 0; x >>= 1) tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, x));
                const float mn = fmaxf(m[u], tm);
                // all scores are -infinity so far: their weights are 0
                const float al = m[u] == kNegInf ? 0.f : exp2f(m[u] - mn);
                const float p = !mine || (s == kNegInf) ? 0.f : exp2f(s - mn);
                l[u] = l[u] * al + warp_sum(p);
                m[u] = mn;
#pragma unroll
                for (int e = 0; e < ND; ++e) o[u][e] *= al;
                for (uint32_t left = seen; left; left &= left - 1) {
                    const int k = __ffs(left) - 1;
                    const float pk = __shfl_sync(0xffffffffu, p, k);
#pragma unroll
                    for (int e = 0; e < ND; ++e)
                        if (lane + 32 * e < D) o[u][e] = fmaf(pk, vs[k * DP + lane + 32 * e], o[u][e]);
                }
            }
        }
        const int first = run.whole() ? 0 : walk.first_block(run);
#pragma unroll
        for (int u = 0; u < kQ; ++u) {
            const int r = warp * kQ + u;
            if (r >= live) break;
            const int64_t part = static_cast<int64_t>(part_of(blockIdx.x, first)) * kPagedRows + r;
            const float inv = l[u] == 0.f ? 0.f : __fdividef(1.f, l[u]);
            if (!run.whole() && lane == 0) a.part_ml[part] = make_float2(m[u], l[u]);
#pragma unroll
            for (int e = 0; e < ND; ++e) {
                const int d = lane + 32 * e;
                if (d >= D) break;
                if (!run.whole()) a.part_o[part * D + d] = o[u][e];
                else a.out[(row0 + r) * D + d] = a.gate ? gated(o[u][e] * inv, __ldcg(a.gate + (row0 + r) * D + d)) : o[u][e] * inv;
            }
        }
        __syncthreads();
        if (run.whole()) continue;
        if (D % 4 == 0) finish_item<true>(join_work(a, walk, run), tid, kThreads, &flag);
        else finish_item<false>(join_work(a, walk, run), tid, kThreads, &flag);
        __syncthreads();
    }
}

const int* generic_ready() {
    return device_once<0, int>([](int& most) {
        most = static_cast<int>(smem_bytes(kMaxD));
        const cudaError_t e = cudaFuncSetAttribute(paged_generic_kernel<8>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        return e == cudaSuccess ? static_cast<int>(MUSER_OK) : cuda_fail(e, "paged attention: cudaFuncSetAttribute");
    });
}

}  // namespace

size_t paged_scratch_bytes(int64_t head_dim) {
    const size_t rows = 2u * kPagedMaxBlocks * kPagedRows;
    return kPagedTicketBytes + rows * sizeof(float2) + (rows * static_cast<size_t>(head_dim) * 4u + 15u) / 16u * 16u;
}

int launch_paged_attention(PagedArgs a, void* scratch, cudaStream_t s) {
    uint8_t* p = static_cast<uint8_t*>(scratch);
    a.ticket = reinterpret_cast<unsigned*>(p);
    a.part_ml = reinterpret_cast<float2*>(p + kPagedTicketBytes);
    a.part_o = reinterpret_cast<float*>(p + kPagedTicketBytes + 2u * kPagedMaxBlocks * kPagedRows * sizeof(float2));
    a.blocks_per_head = (a.group + kPagedRows - 1) / kPagedRows;
    a.status = device_status_word();
    if (!a.status) return set_error(MUSER_ERR_CUDA, "paged attention: no device status word");
    const int blocks = std::min(kPagedMaxBlocks, std::max(1, sm_count()));
    if (paged_tc_supported(a)) return launch_paged_tc(a, blocks, s);
    if (a.D > 128 && generic_ready() == nullptr) return MUSER_ERR_CUDA;  // the message is set
    auto kern = a.D <= 64 ? paged_generic_kernel<2> : a.D <= 128 ? paged_generic_kernel<4> : paged_generic_kernel<8>;
    return launch_after("paged attention", kern, dim3(static_cast<unsigned>(blocks)), kThreads, smem_bytes(a.D), 1, s, a);
}

}  // namespace muser
