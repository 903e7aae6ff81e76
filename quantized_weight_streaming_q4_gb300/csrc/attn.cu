// attn.cu -- attention of M drafted (tree) rows over a K/V plane, with a
// sliding window and first tokens that stay visible.
#include <algorithm>

#include "attn.cuh"
#include "kernels.cuh"

namespace muser {
namespace {

constexpr float kNegInf = -INFINITY;

// ------------------------------------------------ any head size, CUDA cores
// softmax over base 2: s = scale * log2(e) * (q . k), m = running max of s,
// l = sum 2^(s - m), o = sum 2^(s - m) v; one pass over the rows.  A block
// takes one K/V head, one chunk of rows and 16 of the group's M * group query
// vectors; 32 rows at a time sit in shared memory as binary32, a lane scores
// one row, then owns the output elements d = lane, lane + 32, ...
constexpr int kGenWarps = 4, kGenQ = 4, kGenTile = 32, kGenMaxD = 256;

template <int ND>  // output elements per lane: D <= 32 * ND
__global__ void __launch_bounds__(kGenWarps * 32) attn_generic_kernel(const __grid_constant__ AttnArgs a) {
    extern __shared__ float sm[];
    const int D = a.D, DP = D + 1;
    float* ks = sm;                    // [32][D + 1]
    float* vs = ks + kGenTile * DP;    // [32][D + 1]
    float* qs = vs + kGenTile * DP;    // [16][D]
    const int g = blockIdx.y, c = blockIdx.x, rb = blockIdx.z;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rows = a.M * a.group;    // row r: tree row r / group, head g * group + r % group
    const int r0 = rb * kGenWarps * kGenQ;
    for (int x = threadIdx.x; x < kGenWarps * kGenQ * D; x += blockDim.x) {
        const int r = r0 + x / D, d = x % D;
        qs[x] = r < rows ? a.q[static_cast<int64_t>(r / a.group) * a.H * D + (g * a.group + r % a.group) * D + d] : 0.f;
    }
    float m[kGenQ], l[kGenQ], o[kGenQ][ND];
#pragma unroll
    for (int u = 0; u < kGenQ; ++u) {
        m[u] = kNegInf;
        l[u] = 0.f;
#pragma unroll
        for (int e = 0; e < ND; ++e) o[u][e] = 0.f;
    }
    const int first = c * a.chunk, last = min(first + a.chunk, a.n_common);
    const bool ragged = c == a.nchunks - 1;
    const int ncommon_tiles = (last - first + kGenTile - 1) / kGenTile;
    const int ntiles = ncommon_tiles + (ragged ? 1 : 0);
    for (int t = 0; t < ntiles; ++t) {
        const bool rag = t == ncommon_tiles;
        const int n = rag ? a.n_edge + a.M : min(kGenTile, last - first - t * kGenTile);
        __syncthreads();
        for (int x = threadIdx.x; x < n * D; x += blockDim.x) {
            const int r = x / D, d = x % D;
            if (rag) {
                ks[r * DP + d] = attn_ragged(a, g, r, d, false);
                vs[r * DP + d] = attn_ragged(a, g, r, d, true);
            } else {
                ks[r * DP + d] = h2f(ldg_u16(attn_row(a, g, first + t * kGenTile + r, false) + d));
                vs[r * DP + d] = h2f(ldg_u16(attn_row(a, g, first + t * kGenTile + r, true) + d));
            }
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kGenQ; ++u) {
            const int r = r0 + warp * kGenQ + u;
            if (r >= rows) break;
            const uint32_t seen = rag ? a.mask[r / a.group] : (n == 32 ? 0xffffffffu : (1u << n) - 1u);
            const bool mine = (seen >> lane) & 1u;
            float s = kNegInf;
            if (mine) {
                const float* qr = qs + (warp * kGenQ + u) * D;
                float acc = 0.f;
                for (int d = 0; d < D; ++d) acc = fmaf(qr[d], ks[lane * DP + d], acc);
                s = acc * a.scale_log2;
            }
            float tm = s;
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, x));
            const float mn = fmaxf(m[u], tm);
            if (seen == 0) continue;
            const float al = m[u] == kNegInf ? 0.f : exp2f(m[u] - mn);
            const float p = mine ? exp2f(s - mn) : 0.f;
            l[u] = l[u] * al + warp_sum(p);
            m[u] = mn;
#pragma unroll
            for (int e = 0; e < ND; ++e) o[u][e] *= al;
            // a row that this query does not see is skipped, whatever it holds
            for (uint32_t left = seen; left; left &= left - 1) {
                const int k = __ffs(left) - 1;
                const float pk = __shfl_sync(0xffffffffu, p, k);
#pragma unroll
                for (int e = 0; e < ND; ++e)
                    if (lane + 32 * e < D) o[u][e] = fmaf(pk, vs[k * DP + lane + 32 * e], o[u][e]);
            }
        }
    }
#pragma unroll
    for (int u = 0; u < kGenQ; ++u) {
        const int r = r0 + warp * kGenQ + u;
        if (r >= rows) break;
        const int64_t row = static_cast<int64_t>(r / a.group) * a.H + g * a.group + r % a.group;
        const int64_t slot = static_cast<int64_t>(c) * a.M * a.H + row;
        if (lane == 0) a.part_ml[slot] = make_float2(m[u], l[u]);
#pragma unroll
        for (int e = 0; e < ND; ++e)
            if (lane + 32 * e < D) a.part_o[slot * D + lane + 32 * e] = o[u][e];
    }
}

// Joins the parts: out = sum_c 2^(m_c - m) o_c / sum_c 2^(m_c - m) l_c, times
// sigmoid(gate).  One block per query vector; its threads are groups of
// ceil(D / 4) that take every kGroups-th part, eight loads in flight each, and
// are added in a fixed order.
constexpr int kJoinThreads = 256;
__global__ void __launch_bounds__(kJoinThreads) attn_combine_kernel(const __grid_constant__ AttnArgs a, int parts) {
    __shared__ float4 so[kJoinThreads];
    __shared__ float2 sl[kJoinThreads];
    pdl_launch_dependents();
    pdl_wait();
    const int64_t row = blockIdx.x, rows = static_cast<int64_t>(a.M) * a.H;
    const bool vec = a.D % 4 == 0;
    const int per = vec ? a.D / 4 : a.D, groups = max(1, kJoinThreads / per);
    const int group = threadIdx.x / per, e = threadIdx.x % per;
    float m = kNegInf, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f), z = o;
    const bool in = group < groups;
    if (in && group == 0 && a.gate) {
        if (vec) z = __ldcg(reinterpret_cast<const float4*>(a.gate + row * a.D) + e);
        else z.x = __ldcg(a.gate + row * a.D + e);
    }
    for (int c0 = group; in && c0 < parts; c0 += 8 * groups) {
        float2 w[8];
        float4 v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int c = c0 + k * groups;
            w[k] = make_float2(kNegInf, 0.f);
            v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (c < parts) {
                w[k] = __ldcg(a.part_ml + c * rows + row);
                const float* p = a.part_o + (c * rows + row) * a.D;
                if (vec) v[k] = __ldcg(reinterpret_cast<const float4*>(p) + e);
                else v[k].x = __ldcg(p + e);
            }
        }
        float mn = m;
#pragma unroll
        for (int k = 0; k < 8; ++k) mn = fmaxf(mn, w[k].x);
        const float f0 = m == kNegInf ? 0.f : exp2f(m - mn);
        m = mn;
        l *= f0;
        o = make_float4(o.x * f0, o.y * f0, o.z * f0, o.w * f0);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (w[k].x == kNegInf && w[k].y == 0.f) continue;  // a part without rows
            const float f = exp2f(w[k].x - m);
            l = fmaf(f, w[k].y, l);
            o = make_float4(fmaf(f, v[k].x, o.x), fmaf(f, v[k].y, o.y), fmaf(f, v[k].z, o.z), fmaf(f, v[k].w, o.w));
        }
    }
    so[threadIdx.x] = o;
    sl[threadIdx.x] = make_float2(m, l);
    __syncthreads();
    if (!in || group != 0) return;
    for (int k = 0; k < groups; ++k) m = fmaxf(m, sl[k * per + e].x);
    l = 0.f;
    o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < groups; ++k) {
        const float2 w = sl[k * per + e];
        if (w.x == kNegInf && w.y == 0.f) continue;
        const float4 v = so[k * per + e];
        const float f = exp2f(w.x - m);
        l = fmaf(f, w.y, l);
        o = make_float4(fmaf(f, v.x, o.x), fmaf(f, v.y, o.y), fmaf(f, v.z, o.z), fmaf(f, v.w, o.w));
    }
    const float inv = __fdividef(1.f, l);
    o = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
    if (a.gate) {
        o.x = __fdividef(o.x, 1.f + __expf(-z.x));
        o.y = __fdividef(o.y, 1.f + __expf(-z.y));
        o.z = __fdividef(o.z, 1.f + __expf(-z.z));
        o.w = __fdividef(o.w, 1.f + __expf(-z.w));
    }
    if (vec) reinterpret_cast<float4*>(a.out + row * a.D)[e] = o;
    else a.out[row * a.D + e] = o.x;
}

// Chunks of the common rows: about two blocks per SM, at least 64 rows each.
int generic_chunks(int G, int blocks_per_head, int n_common) {
    const int want = std::max(1, kAttnBlocks / std::max(1, G * blocks_per_head));
    return std::max(1, std::min(want, (n_common + 63) / 64));
}

}  // namespace

// The most parts a call leaves for the second kernel: of attn_tc.cu's, one for
// each pair of SMs.
static int64_t max_parts(int64_t G, int64_t rows, int64_t D) {
    const int64_t blocks = (rows + kGenWarps * kGenQ - 1) / (kGenWarps * kGenQ);
    const int64_t pairs = rows > 32 && D <= 128 ? 76 / (G * ((rows + 127) / 128)) : 0;
    return std::max<int64_t>({1, kAttnBlocks / std::max<int64_t>(1, G * blocks), pairs});
}

size_t attn_scratch_bytes(int64_t kv_dim, int64_t head_dim, int M, int n_heads) {
    const int64_t G = kv_dim / head_dim;
    const int64_t parts = max_parts(G, static_cast<int64_t>(M) * (n_heads / G), head_dim);
    return attn_part_layout(parts, static_cast<int64_t>(M) * n_heads, head_dim).bytes;
}

namespace {

void place_parts(AttnArgs& a, int parts, void* scratch) {
    a.part_ml = static_cast<float2*>(scratch);
    a.part_o = reinterpret_cast<float*>(static_cast<uint8_t*>(scratch) +
                                        attn_part_layout(parts, static_cast<int64_t>(a.M) * a.H, a.D).o);
}

int launch_combine(const AttnArgs& a, int parts, cudaStream_t s) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(a.M * a.H));
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, attn_combine_kernel, a, parts);
    if (e != cudaSuccess) return cuda_fail(e, "attention combine: cudaLaunchKernelEx");
    return check_launch("attention combine");
}

constexpr size_t generic_smem(int D) { return (2 * kGenTile * (D + 1) + kGenWarps * kGenQ * D) * sizeof(float); }
static_assert(generic_smem(128) <= 48 * 1024, "heads up to 128 need no attribute");

const int* generic_ready() {
    return device_once<0, int>([](int& most) {
        most = static_cast<int>(generic_smem(kGenMaxD));
        const cudaError_t e = cudaFuncSetAttribute(attn_generic_kernel<8>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        return e == cudaSuccess ? static_cast<int>(MUSER_OK) : cuda_fail(e, "attention: cudaFuncSetAttribute");
    });
}

int launch_generic(AttnArgs a, void* scratch, cudaStream_t s) {
    const int rows = a.M * a.group, blocks = (rows + kGenWarps * kGenQ - 1) / (kGenWarps * kGenQ);
    a.nchunks = generic_chunks(a.G, blocks, a.n_common);
    a.chunk = std::max(32, ((a.n_common + a.nchunks - 1) / a.nchunks + 31) / 32 * 32);
    a.nchunks = std::max(1, (a.n_common + a.chunk - 1) / a.chunk);
    place_parts(a, a.nchunks, scratch);
    const dim3 grid(static_cast<unsigned>(a.nchunks), static_cast<unsigned>(a.G), static_cast<unsigned>(blocks));
    auto kern = a.D <= 64 ? attn_generic_kernel<2> : a.D <= 128 ? attn_generic_kernel<4> : attn_generic_kernel<8>;
    if (a.D > 128 && generic_ready() == nullptr) return MUSER_ERR_CUDA;  // the message is set
    kern<<<grid, kGenWarps * 32, generic_smem(a.D), s>>>(a);
    MUSER_TRY(check_launch("attention"));
    return launch_combine(a, a.nchunks, s);
}

// The split of the common rows for the tensor-core kernels (tiles of 128 keys,
// one block per SM, `heads` K/V heads times row blocks): clusters of c blocks,
// k of them a head.  One cluster joins its blocks' results itself; more leave
// parts for a second kernel (2.7 us; 5.9 for 512 rows of 19 parts).  A tile takes a block `tile_us`, or
// `tile_full_us` where all SMs share the memory's rate, and beside its tiles 5
// us, or 3.5 where it joins no other; clusters beyond those that run at once wait for a turn (of 16 blocks
// 7 clusters are resident).  Measured, one token, 16 K/V heads of 64, 2,048
// rows: clusters of 16 in three turns 23.9 us, of 4 at once 11.2 us; 2 heads of
// 128: one cluster of 16 a head 8.4 us (11.0 with parts), and over 32,768 rows
// 21.4 us (14.0 with parts).
struct Split {
    int cluster, chunks;
};
Split choose_split(int heads, int tiles, int parts, double tile_us, double tile_full_us, const AttnResident& resident) {
    Split best{1, 1};
    double least = 1e30;
    for (int c = 16, e = 4; e >= 0; c /= 2, --e) {
        const int most = resident.clusters[e];
        if (most < 1 || (c > 1 && c / 2 >= tiles)) continue;
        for (const int k : {1, std::min(parts, most / heads)}) {
            if (k < 1) continue;
            const int chunks = std::min(c * k, std::max(1, tiles)), clusters = (chunks + c - 1) / c;
            const int waves = (heads * clusters + most - 1) / most, per = (std::max(1, tiles) + chunks - 1) / chunks;
            const double busy = std::min(1.0, heads * chunks / 144.0);
            const double us = waves * ((chunks > 1 ? 5.0 : 3.5) + per * std::max(tile_us, tile_full_us * busy)) + (clusters > 1 ? 2.7 : 0.0);
            if (us < least - 1e-9) {
                least = us;
                best = Split{c, chunks};
            }
        }
    }
    return best;
}

template <typename Launch>
int launch_tiles(AttnArgs a, int R, double tile_us, double tile_full_us, void* scratch, cudaStream_t s,
                 const AttnResident* resident, Launch&& launch) {
    if (resident == nullptr) return MUSER_ERR_CUDA;  // the message is set
    const int rows = a.M * a.group, blocks = (rows + R - 1) / R;
    // A tree's own rows are one more tile, of the last chunk, which therefore
    // takes 128 common rows less (16 rows, 2,037 common rows, 16 chunks: three
    // tiles in the last one 14.2 us, two in each 12.0).
    int n = a.n_common + (R == 128 || a.M > 1 ? 128 : 0);
    // Short runs at the start (kept first rows) are a tile each: chunk 0 takes
    // as many rows less as keep it to the others' tiles (one token, 4 kept rows
    // and a full ring of 2,048: 8.8 us, 8.0 so).
    int lead = 0, lead_rows = 0;
    while (lead < a.nseg - 1 && a.seg_end[lead] - lead_rows < 128) lead_rows = a.seg_end[lead++];
    n += lead * 128 - lead_rows;
    const Split split = choose_split(a.G * blocks, (n + 127) / 128, static_cast<int>(max_parts(a.G, rows, a.D)), tile_us,
                                     tile_full_us, *resident);
    a.cluster = split.cluster;
    a.chunk = std::max(16, ((n + split.chunks - 1) / split.chunks + 15) / 16 * 16);
    const int tiles = (a.chunk + 127) / 128, rows0 = lead_rows + std::max(0, tiles - lead) * 128;
    a.shift = lead == 0 ? 0 : std::min(std::max(0, a.chunk - rows0), lead * 128 - lead_rows);
    a.nchunks = std::max(1, (a.n_common + a.shift + a.chunk - 1) / a.chunk);
    if (a.nchunks == 1) a.cluster = 1;  // nothing to join; else blocks without rows share in the join
    const int clusters = (a.nchunks + a.cluster - 1) / a.cluster;
    place_parts(a, clusters, scratch);
    MUSER_TRY(launch(a, dim3(static_cast<unsigned>(clusters * a.cluster), static_cast<unsigned>(a.G), static_cast<unsigned>(blocks))));
    return clusters > 1 ? launch_combine(a, clusters, s) : MUSER_OK;
}

}  // namespace

int launch_attention(AttnArgs a, void* scratch, cudaStream_t s) {
    if (!attn_mma_supported(a)) return launch_generic(a, scratch, s);
    a.status = device_status_word();
    if (!a.status) return set_error(MUSER_ERR_CUDA, "attention: no device status word");
    if (a.D <= 128 && a.M * a.group <= 32) {
        const int rows = a.M * a.group;
        return launch_tiles(a, rows <= 16 ? 16 : 32, 0.85, a.D <= 64 ? 0.85 : 1.4, scratch, s,
                            attn_few_resident(rows), [&](const AttnArgs& b, dim3 grid) { return launch_attn_few(b, grid, s); });
    }
    if (a.D <= 128)
        return launch_tiles(a, 128, 1.35, 1.35, scratch, s, attn_tc_resident(a.D), [&](const AttnArgs& b, dim3 grid) { return launch_attn_tc(b, grid, s); });
    const int rows = a.M * a.group, rt = attn_mma_row_tiles(rows);
    const int blocks = (rows + 16 * rt - 1) / (16 * rt), heads = a.G * blocks;
    const int tiles = std::max(1, (a.n_common + 63) / 64);
    // up to 16 chunks of at least 128 keys: one cluster and no second kernel;
    // longer ones: as many clusters of 8 as run at once
    const int one = std::min(16, std::max(1, (tiles + 1) / 2));
    int chunks = one;
    a.cluster = 1;
    while (a.cluster < one) a.cluster *= 2;
    const int* resident = attn_mma_resident(rt);
    if (resident == nullptr) return MUSER_ERR_CUDA;  // the message is set
    if (tiles > 64) {
        const int most = *resident / heads;
        if (most > 2) {
            a.cluster = 8;
            chunks = std::min({8 * most, tiles / 2, static_cast<int>(8 * max_parts(a.G, rows, a.D))});
        }
    }
    a.chunk = std::max(64, ((a.n_common + chunks - 1) / chunks + 15) / 16 * 16);
    a.nchunks = std::max(1, (a.n_common + a.chunk - 1) / a.chunk);
    const int clusters = (a.nchunks + a.cluster - 1) / a.cluster;
    place_parts(a, clusters, scratch);
    MUSER_TRY(launch_attn_mma(a, dim3(static_cast<unsigned>(clusters * a.cluster), static_cast<unsigned>(a.G), static_cast<unsigned>(blocks)), rt, s));
    return clusters > 1 ? launch_combine(a, clusters, s) : MUSER_OK;
}

}  // namespace muser
