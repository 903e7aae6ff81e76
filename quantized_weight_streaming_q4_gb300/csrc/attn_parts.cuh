// attn_parts.cuh -- device code that the matrix-product attention kernels
// share: splitting binary32 values into two binary16 parts, the rows whose
// visibility differs, and the joining of a cluster's partial results.
#pragma once

#include "attn.cuh"
#include "kernels.cuh"

namespace muser {
namespace {

constexpr float kOffset = 14.f;  // p <= 2^14
constexpr float kNegInf = -INFINITY;

// Copies 16 bytes, or zeroes them where `real` is false (src is then not read).
__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void* src, bool real) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// The parts of two neighbouring elements: x = hi + lo to 22 bits.
__device__ __forceinline__ void split2(float x0, float x1, uint32_t& hi, uint32_t& lo) {
    const __half2 h = __floats2half2_rn(x0, x1);
    const float2 f = __half22float2(h);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    lo = pack_h2(x0 - f.x, x1 - f.y);
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
    cluster_arrive();
    cluster_wait();
}
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
__device__ __forceinline__ float2 ld_cluster2(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}
// `bytes` of this block's shared memory to another's, whose barrier counts them.
__device__ __forceinline__ void copy_to_block(uint32_t dst, uint32_t src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "r"(src), "r"(bytes), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
// The last barrier: nobody leaves while its shared memory is read.  What was
// read has arrived (it was used), and nothing needs the release, which would
// wait for the output's stores.
__device__ __forceinline__ void cluster_leave() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    cluster_wait();
}
// 2^(m - M) of a partial result with maximum m, 0 where it has no rows.
__device__ __forceinline__ float share(float m, float M) { return m == kNegInf ? 0.f : ex2(m - M); }

// Eight elements from d on of ragged row r (see attn_ragged), as they lie in
// memory: the loads of several go out before the first is packed, which waits
// for it.
struct RaggedRaw {
    uint4 a, b;
};
__device__ __forceinline__ RaggedRaw attn_ragged_load(const AttnArgs& a, int g, int r, int d, bool value) {
    RaggedRaw raw{make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (r < a.n_edge) {
        const int e = r < a.edge0 ? 0 : 1;
        const AttnSeg& S = a.edge[e];
        raw.a = __ldcg(reinterpret_cast<const uint4*>((value ? S.v : S.k) + g * S.head_stride + (r - (e ? a.edge0 : 0)) * S.row_stride + d));
    } else {
        const uint4* p = reinterpret_cast<const uint4*>((value ? a.vt : a.kt) + (r - a.n_edge) * a.G * a.D + g * a.D + d);
        raw.a = __ldcg(p);
        raw.b = __ldcg(p + 1);
    }
    return raw;
}
// The same as binary16.
__device__ __forceinline__ uint4 attn_ragged_pack(const AttnArgs& a, int r, const RaggedRaw& raw) {
    if (r < a.n_edge) return raw.a;
    auto two = [](uint32_t x, uint32_t y) { return pack_h2(__uint_as_float(x), __uint_as_float(y)); };
    return make_uint4(two(raw.a.x, raw.a.y), two(raw.a.z, raw.a.w), two(raw.b.x, raw.b.y), two(raw.b.z, raw.b.w));
}
// Whether one of eight binary16 values is infinite or NaN.
__device__ __forceinline__ bool not_finite8(uint4 v) {
    auto two = [](uint32_t w) { return (w & 0x7c00u) == 0x7c00u || (w & 0x7c000000u) == 0x7c000000u; };
    return two(v.x) || two(v.y) || two(v.z) || two(v.w);
}

// A box of a segment's rows into shared memory (see AttnMaps): elements
// [64 x, 64 x + 64), rows from `row` on, of head g.
__device__ __forceinline__ void tma_load_box(uint32_t dst, const CUtensorMap* map, int x, int row, int g, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::
            "r"(dst),
        "l"(map), "r"(x * 64), "r"(row), "r"(g), "r"(smem_u32(bar))
        : "memory");
}
// Byte offset of 16-byte piece c of row r in a tile of ROWS rows: blocks of 64
// elements, 128 bytes a row, the piece's low three bits exclusive-or the row's
// (the tensor maps' 128-byte swizzle; eight rows' pieces hit eight bank groups).
template <int ROWS>
__device__ __forceinline__ uint32_t piece(int r, int c) {
    return static_cast<uint32_t>((c >> 3) * ROWS * 128 + r * 128 + (((c ^ r) & 7) << 4));
}

// Touches the kernel's arguments, a lane each 64 bytes, so that later reads
// find them in the SM's constant cache.
__device__ __forceinline__ void touch_args(const AttnArgs& a, int lane) {
    const uint32_t* p = reinterpret_cast<const uint32_t*>(&a);
    for (int x = lane * 16; x < static_cast<int>(sizeof(AttnArgs) / 4); x += 32 * 16) {
        const uint32_t v = p[x];
        asm volatile("" ::"r"(v));
    }
}

// Brings the lines of the output gate that join_cluster will read into L2:
// LANES threads, those of the block's R rows that fall to its rank.
template <int R, int LANES>
__device__ __forceinline__ void prefetch_gate(const AttnArgs& a, int lane, int g, int r0, int rows) {
    if (a.gate == nullptr) return;
    const int n = a.cluster, rank = n > 1 ? static_cast<int>(cluster_rank()) : 0, lines = (a.D * 4 + 127) / 128;
    for (int x = lane + R * lines * rank / n; x < R * lines * (rank + 1) / n; x += LANES) {
        const int r = r0 + x / lines, i = r / a.group;
        if (r < rows) prefetch_l2(a.gate + (static_cast<int64_t>(i) * a.H + g * a.group + r - i * a.group) * a.D + x % lines * 32);
    }
}

// The cluster's result: the blocks hold the same R query rows' (maximum, sum)
// pairs at shared address mla and outputs at oa (row stride STRIDE floats);
// each joins a share of the elements and writes them out, final or as a part.
// Called by THREADS threads (tid counts them, whole warps) between two cluster
// barriers.  An element's blocks are shared by SPLIT neighbouring lanes (or n,
// if that is less), whose remote loads are all in flight together: one after
// another they took 16 round trips, about 5 us in a cluster of 16.
template <int DP, int STRIDE, int R, int THREADS, int SPLIT>
__device__ __forceinline__ void join_cluster(const AttnArgs& a, int tid, int c, int g, int r0, int rows, uint32_t mla,
                                             uint32_t oa) {
    constexpr int kEach = 16 / SPLIT < 8 ? 16 / SPLIT : 8;  // blocks of a lane loaded together
    const int n = a.cluster, rank = n > 1 ? static_cast<int>(cluster_rank()) : 0, split = min(n, SPLIT);
    const int units = R * DP / 4, u0 = units * rank / n, items = (units * (rank + 1) / n - u0) * split;
    const bool final = gridDim.x == static_cast<unsigned>(n);
    for (int item = tid; item < (items + 31) / 32 * 32; item += THREADS) {
        const int x = u0 + item / split, sub = item % split, r = x / (DP / 4), d = x % (DP / 4) * 4;
        const bool real = item < items && r0 + r < rows && d < a.D;
        const int i = (r0 + r) / a.group;
        const int64_t row = static_cast<int64_t>(i) * a.H + g * a.group + (r0 + r) - i * a.group;
        const uint32_t ma = mla + r * 8, va = oa + (r * STRIDE + d) * 4;
        float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
        if (real && final && a.gate) z = __ldcg(reinterpret_cast<const float4*>(a.gate + row * a.D + d));
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        float l = 0.f, M = kNegInf;
        for (int b0 = sub; b0 < n; b0 += kEach * split) {
            float2 w[kEach];
            float4 v[kEach];
#pragma unroll
            for (int k = 0; k < kEach; ++k) {
                const int b = b0 + k * split;
                w[k] = make_float2(kNegInf, 0.f);
                v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (real && b < n) {
                    w[k] = ld_cluster2(n > 1 ? map_rank(ma, b) : ma);
                    v[k] = ld_cluster4(n > 1 ? map_rank(va, b) : va);
                }
            }
            float mn = M;
#pragma unroll
            for (int k = 0; k < kEach; ++k) mn = fmaxf(mn, w[k].x);
            const float f0 = share(M, mn);
            M = mn;
            l *= f0;
            s.x *= f0;
            s.y *= f0;
            s.z *= f0;
            s.w *= f0;
#pragma unroll
            for (int k = 0; k < kEach; ++k) {
                const float f = share(w[k].x, M);
                if (w[k].x == kNegInf && w[k].y == 0.f) continue;  // no rows there
                l = fmaf(f, w[k].y, l);
                s.x = fmaf(f, v[k].x, s.x);
                s.y = fmaf(f, v[k].y, s.y);
                s.z = fmaf(f, v[k].z, s.z);
                s.w = fmaf(f, v[k].w, s.w);
            }
        }
        for (int o = 1; o < split; o <<= 1) {
            const float mo = __shfl_xor_sync(0xffffffffu, M, o), mn = fmaxf(M, mo);
            const float f = share(M, mn), fo = share(mo, mn);
            M = mn;
            l = fmaf(f, l, fo * __shfl_xor_sync(0xffffffffu, l, o));
            s.x = fmaf(f, s.x, fo * __shfl_xor_sync(0xffffffffu, s.x, o));
            s.y = fmaf(f, s.y, fo * __shfl_xor_sync(0xffffffffu, s.y, o));
            s.z = fmaf(f, s.z, fo * __shfl_xor_sync(0xffffffffu, s.z, o));
            s.w = fmaf(f, s.w, fo * __shfl_xor_sync(0xffffffffu, s.w, o));
        }
        if (!real || sub != 0) continue;
        if (final) {
            const float inv = __fdividef(1.f, l);  // l is between 2^-10 and 2^46: a step or two off
            float4 y = make_float4(s.x * inv, s.y * inv, s.z * inv, s.w * inv);
            if (a.gate) {
                y.x = __fdividef(y.x, 1.f + __expf(-z.x));
                y.y = __fdividef(y.y, 1.f + __expf(-z.y));
                y.z = __fdividef(y.z, 1.f + __expf(-z.z));
                y.w = __fdividef(y.w, 1.f + __expf(-z.w));
            }
            *reinterpret_cast<float4*>(a.out + row * a.D + d) = y;
        } else {
            const int64_t slot = static_cast<int64_t>(c / n) * a.M * a.H + row;
            *reinterpret_cast<float4*>(a.part_o + slot * a.D + d) = s;
            if (d == 0) a.part_ml[slot] = make_float2(M, l);
        }
    }
}

// The cluster's result from what its blocks have copied into this one's `out`:
// of n blocks, rank b's rows [rank R / n, (rank + 1) R / n) at row b R / n, each
// DP outputs, the maximum and the sum.  Every element is joined and written
// out, final or as a part.
template <int DP, int STRIDE, int R, int THREADS>
__device__ __forceinline__ void merge_cluster(const AttnArgs& a, int tid, int c, int g, int r0, int rows, const float* out) {
    const int n = a.cluster, rank = n > 1 ? static_cast<int>(cluster_rank()) : 0, per = R / n;
    const bool final = gridDim.x == static_cast<unsigned>(n);
    for (int x = tid; x < per * (DP / 4); x += THREADS) {
        const int own = x / (DP / 4), d = x % (DP / 4) * 4, r = r0 + rank * per + own, i = r / a.group;
        if (r >= rows || d >= a.D) continue;
        const int64_t row = static_cast<int64_t>(i) * a.H + g * a.group + r - i * a.group;
        float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
        if (final && a.gate) z = __ldcg(reinterpret_cast<const float4*>(a.gate + row * a.D + d));
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        float l = 0.f, M = kNegInf;
        const float* p = out + own * STRIDE;
#pragma unroll 2
        for (int b = 0; b < n; ++b, p += per * STRIDE) {
            const float2 w = *reinterpret_cast<const float2*>(p + DP);
            const float4 v = lds_float4(p + d);
            const float mn = fmaxf(M, w.x), f = share(M, mn), fb = share(w.x, mn);
            M = mn;
            l = fmaf(fb, w.y, l * f);
            s = make_float4(fmaf(fb, v.x, s.x * f), fmaf(fb, v.y, s.y * f), fmaf(fb, v.z, s.z * f), fmaf(fb, v.w, s.w * f));
        }
        if (final) {
            const float inv = __fdividef(1.f, l);  // l is between 2^-10 and 2^46: a step or two off
            float4 y = make_float4(s.x * inv, s.y * inv, s.z * inv, s.w * inv);
            if (a.gate) {
                y.x = __fdividef(y.x, 1.f + __expf(-z.x));
                y.y = __fdividef(y.y, 1.f + __expf(-z.y));
                y.z = __fdividef(y.z, 1.f + __expf(-z.z));
                y.w = __fdividef(y.w, 1.f + __expf(-z.w));
            }
            *reinterpret_cast<float4*>(a.out + row * a.D + d) = y;
        } else {
            const int64_t slot = static_cast<int64_t>(c / n) * a.M * a.H + row;
            *reinterpret_cast<float4*>(a.part_o + slot * a.D + d) = s;
            if (d == 0) a.part_ml[slot] = make_float2(M, l);
        }
    }
}

// Launch attributes: the cluster, and programmatic stream serialization (the
// blocks start while the kernel before them on the stream still runs and wait
// for it before their first global access).
inline cudaLaunchConfig_t cluster_config(int cluster, dim3 grid, int threads, size_t smem, cudaStream_t s,
                                         cudaLaunchAttribute* attr) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cfg;
}

}  // namespace
}  // namespace muser
