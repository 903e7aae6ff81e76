// paged_attn.cu -- attention of one token row each of several sequences over a
// paged K/V cache: the kernel for any head and page size, and the choice.
#include <algorithm>

#include "kernels.cuh"
#include "paged.cuh"

namespace muser {
namespace {

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
        for (int x = tid; x < kPagedRows * D; x += kThreads) qs[x] = x / D < live ? __ldg(a.q + row0 * D + x) : 0.f;
        if (self && run.r0 == 0 && sight.t < a.rows_end) {  // the new row, where the cache keeps it
            const int page = __ldcg(table + sight.t / a.page_rows), r = sight.t % a.page_rows;
            if (page >= 0 && page < a.pages) {
                const int64_t at = page * a.page_stride + run.head * a.head_stride + r * a.row_stride;
                for (int d = tid; d < D; d += kThreads) {
                    a.key[at + d] = __half_as_ushort(__float2half_rn(__ldg(kt + d)));
                    a.value[at + d] = __half_as_ushort(__float2half_rn(__ldg(vt + d)));
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
                    k = __half2float(__float2half_rn(__ldg(kt + d)));
                    v = __half2float(__float2half_rn(__ldg(vt + d)));
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
                else a.out[(row0 + r) * D + d] = a.gate ? gated(o[u][e] * inv, __ldg(a.gate + (row0 + r) * D + d)) : o[u][e] * inv;
            }
        }
        __syncthreads();
        if (run.whole()) continue;
        if (D % 4 == 0) finish_item<true>(join_work(a, walk, run), tid, kThreads, 1, &flag, true);
        else finish_item<false>(join_work(a, walk, run), tid, kThreads, 1, &flag, true);
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
