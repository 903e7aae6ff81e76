// attn_mma.cu -- tree attention on warp-level matrix products (mma.sync), for
// head sizes above 128 (multiples of 8, up to 256) and 16-byte aligned planes.
//
// A block takes one K/V head, 16 * RT of the group's M * group query vectors
// and one chunk of the cached rows; its four warps are RT row tiles times
// 4 / RT shares of every stage's keys.  K and V tiles come by TMA, two stages
// deep, in its 128-byte swizzle, so the fragment loads of eight rows hit eight
// different bank groups.
//
// Precision: the planes are binary16, q is binary32 and so is the result.  A
// query vector is scaled by a power of two and split into two binary16 parts
// (22 bits); p = 2^(s - m + 14) is split likewise (the offset keeps the low
// part of all but vanishing weights out of the subnormals), so both products
// run twice, and sums are binary32.  One part alone would be off by 2^-12.  The
// products' additions truncate: the outputs of every 16 keys are a fresh
// accumulator, added in registers.  Values of one sign over 8,125 keys a block
// were 2.9e-5 too small on one accumulator, 1.2e-7 off so, at 4 to 7 % of the
// time (16 rows, 16 heads of 256 on one, 130,000 rows: 541 -> 563 us).
//
// The blocks of a cluster hold neighbouring chunks of the same rows and join
// their (maximum, sum, output) triples through distributed shared memory; with
// one cluster per row block the result is final and there is no second kernel.
//
// Bound: mma.sync itself, about 16 cycles a 16 x 8 x 16 product and scheduler,
// an eighth of tcgen05's rate: heads up to 128 take attn_few.cu or attn_tc.cu.
// A head of 256 has 128 binary32 outputs a thread, which is why the q parts
// are read from shared memory for every key tile.
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>

#include "attn.cuh"
#include "attn_parts.cuh"
#include "kernels.cuh"

namespace muser {
namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kTileKeys = 64;

constexpr int DP = 256, kStages = 2;
constexpr int kTileBytes = kTileKeys * DP * 2;  // of K or of V
template <int RT>
struct Layout {
    static constexpr int R = 16 * RT, KW = kWarps / RT;
    static constexpr int kOutStride = DP + 8;  // floats; rows 32 bytes apart in the banks
    static constexpr int kOutOff = kStages * 2 * kTileBytes;            // q parts, then the block's output
    static constexpr int kMlOff = kOutOff + R * kOutStride * 4;                 // float2[R]: the block's maximum and sum
    static constexpr int kMlwOff = kMlOff + R * 8;                              // float2[KW][R]
    static constexpr int kScaleOff = kMlwOff + KW * R * 8;                      // float[R]
    static constexpr int kFlagOff = kScaleOff + R * 4;                          // uint32: ragged rows that are not finite
    static constexpr int kBarOff = kFlagOff + 16;                               // uint64[kStages]: a stage has landed
    static constexpr int kBytes = kBarOff + 8 * kStages;
    static_assert(R * kOutStride * 4 >= 2 * R * DP * 2, "the q parts fit under the output");
    static_assert(KW == 1 || KW * R * kOutStride * 4 <= kOutOff, "the warps' outputs fit under the stages");
};

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
template <int RT>
__global__ void __launch_bounds__(kThreads) attn_mma_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ AttnMaps maps) {
    using L = Layout<RT>;
    constexpr int R = L::R, KW = L::KW, NS = kStages;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t base = smem_u32(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rt = warp % RT, kw = warp / RT;
    const int c = blockIdx.x, g = blockIdx.y, r0 = blockIdx.z * R;
    const int rows = a.M * a.group;
    AttnWalk load(a, c), walk(a, c);
    const int ntiles = walk.count(a, kTileKeys);
    const bool ragged = c == a.nchunks - 1;
    float* cs = reinterpret_cast<float*>(smem + L::kScaleOff);
    uint32_t* flags = reinterpret_cast<uint32_t*>(smem + L::kFlagOff);
    uint64_t* bar = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
    // thread 0: the next tile's boxes into stage t % NS
    auto load_tile = [&](int t) {
        int s, row;
        load.next(a, kTileKeys, s, row);
        const uint32_t buf = base + (t % NS) * 2 * kTileBytes;
        mbar_arrive_expect_tx(&bar[t % NS], 2 * kTileBytes);
#pragma unroll
        for (int x = 0; x < DP / 64; ++x) {
            tma_load_box(buf + x * kTileKeys * 128, &maps.k[s], x, row, g, &bar[t % NS]);
            tma_load_box(buf + kTileBytes + x * kTileKeys * 128, &maps.v[s], x, row, g, &bar[t % NS]);
        }
    };
    pdl_launch_dependents();
    if (tid == 0) {
        *flags = 0;
        for (int i = 0; i < NS; ++i) mbar_init(&bar[i], 1);
        fence_mbar_init();
    }
    pdl_wait();  // no global access before this
    if (tid == 0) {
        // the last stage is left to the ragged rows
        for (int t = 0; t < NS - 1 && t < ntiles; ++t) load_tile(t);
    }

    // the ragged rows' loads (below) go out before q's
    constexpr int kPieces = DP / 8, kEach = 32 * kPieces / kThreads;  // 8-element pieces, of K and of V
    const int nragged = a.n_edge + a.M;
    uint4 kp[kEach], vp[kEach];
    if (ragged) {
        RaggedRaw kr[kEach], vr[kEach];
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            const int x = tid + j * kThreads, r = x / kPieces, d = x % kPieces * 8;
            if (r < nragged && d < a.D) {
                kr[j] = attn_ragged_load(a, g, r, d, false);
                vr[j] = attn_ragged_load(a, g, r, d, true);
            }
        }
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            const int x = tid + j * kThreads, r = x / kPieces, d = x % kPieces * 8;
            kp[j] = vp[j] = make_uint4(0, 0, 0, 0);
            if (r < nragged && d < a.D) {
                kp[j] = attn_ragged_pack(a, r, kr[j]);
                vp[j] = attn_ragged_pack(a, r, vr[j]);
            }
        }
    }

    prefetch_gate<R, kThreads>(a, tid, g, r0, rows);
    // q: scaled to base 2 and to [2^7, 2^8), split, into shared memory; a
    // warp's rows in batches whose loads are in flight together
    constexpr int kQRows = R / kWarps, kQBatch = 4, kQV = DP / 128;
#pragma unroll
    for (int b = 0; b < kQRows; b += kQBatch) {
        float4 x[kQBatch][kQV];
#pragma unroll
        for (int j = 0; j < kQBatch; ++j) {
            const int r = r0 + (b + j) * kWarps + warp;
            const float* row = a.q + (static_cast<int64_t>(r / a.group) * a.H + g * a.group + r % a.group) * a.D;
#pragma unroll
            for (int u = 0; u < kQV; ++u) {
                const int d = u * 128 + 4 * lane;
                x[j][u] = r < rows && d < a.D ? __ldcg(reinterpret_cast<const float4*>(row + d)) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
        }
#pragma unroll
        for (int j = 0; j < kQBatch; ++j) {
            const int rr = (b + j) * kWarps + warp;
            float mx = 0.f;
#pragma unroll
            for (int u = 0; u < kQV; ++u) {
                x[j][u].x *= a.scale_log2;
                x[j][u].y *= a.scale_log2;
                x[j][u].z *= a.scale_log2;
                x[j][u].w *= a.scale_log2;
                mx = fmaxf(fmaxf(mx, fmaxf(fabsf(x[j][u].x), fabsf(x[j][u].y))), fmaxf(fabsf(x[j][u].z), fabsf(x[j][u].w)));
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const int e = min(127, max(-119, ((__float_as_int(mx) >> 23) & 0xff) - 127)) - 7;
            const float f = __int_as_float((127 - e) << 23);
            if (lane == 0) cs[rr] = __int_as_float((127 + e) << 23);
#pragma unroll
            for (int u = 0; u < kQV; ++u) {
                const int d = u * 128 + 4 * lane;
                uint2 hi, lo;
                split2(x[j][u].x * f, x[j][u].y * f, hi.x, lo.x);
                split2(x[j][u].z * f, x[j][u].w * f, hi.y, lo.y);
                if (d < DP) {
                    const uint32_t at = piece<R>(rr, d >> 3) + (d & 7) * 2;
                    *reinterpret_cast<uint2*>(smem + L::kOutOff + at) = hi;
                    *reinterpret_cast<uint2*>(smem + L::kOutOff + R * DP * 2 + at) = lo;
                }
            }
        }
    }
    __syncthreads();

    const int gr = lane >> 2, qt = lane & 3;  // fragment row and column pair
    auto q_addr = [&](int ks) { return base + L::kOutOff + piece<R>(rt * 16 + (lane & 15), ks * 2 + (lane >> 4)); };
    const float c0 = cs[rt * 16 + gr], c1 = cs[rt * 16 + gr + 8];
    float m0 = kNegInf, m1 = kNegInf, l0 = 0.f, l1 = 0.f;
    float o[DP / 8][4];
#pragma unroll
    for (int n = 0; n < DP / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][e] = 0.f;

    // 16 keys of the tile at `kbuf`: keys k0..k0+15; bit j of see0/see1: the
    // two fragment rows see key k0 + j
    auto step = [&](uint32_t kbuf, int k0, uint32_t see0, uint32_t see1, bool all) {
        float sh[2][4], sl[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) sh[n][e] = sl[n][e] = 0.f;
#pragma unroll
        for (int ks = 0; ks < DP / 16; ++ks) {
            uint32_t kf[4];  // keys 0-7: d 0-7, 8-15; keys 8-15: the same
            ldsm4(kf, kbuf + piece<kTileKeys>(k0 + (lane & 7) + ((lane >> 4) << 3), ks * 2 + ((lane >> 3) & 1)));
            uint32_t f[4];
            ldsm4(f, q_addr(ks) + R * DP * 2);
            mma16816(sl[0], f, kf[0], kf[1]);
            mma16816(sl[1], f, kf[2], kf[3]);
            ldsm4(f, q_addr(ks));
            mma16816(sh[0], f, kf[0], kf[1]);
            mma16816(sh[1], f, kf[2], kf[3]);
        }
        float t0 = kNegInf, t1 = kNegInf;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int j = n * 8 + 2 * qt + e;
                sh[n][e] = all || ((see0 >> j) & 1u) ? (sh[n][e] + sl[n][e]) * c0 : kNegInf;
                sh[n][e + 2] = all || ((see1 >> j) & 1u) ? (sh[n][e + 2] + sl[n][e + 2]) * c1 : kNegInf;
                t0 = fmaxf(t0, sh[n][e]);
                t1 = fmaxf(t1, sh[n][e + 2]);
            }
#pragma unroll
        for (int x = 1; x < 4; x <<= 1) {
            t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, x));
            t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, x));
        }
        if (__any_sync(0xffffffffu, t0 > m0 || t1 > m1)) {
            const float n0 = fmaxf(m0, t0), n1 = fmaxf(m1, t1);
            const float a0 = m0 == kNegInf ? 0.f : ex2(m0 - n0), a1 = m1 == kNegInf ? 0.f : ex2(m1 - n1);
            m0 = n0;
            m1 = n1;
            l0 *= a0;
            l1 *= a1;
#pragma unroll
            for (int n = 0; n < DP / 8; ++n) {
                o[n][0] *= a0;
                o[n][1] *= a0;
                o[n][2] *= a1;
                o[n][3] *= a1;
            }
        }
        const float b0 = m0 == kNegInf ? 0.f : m0 - kOffset, b1 = m1 == kNegInf ? 0.f : m1 - kOffset;
        uint32_t ph[4], pl[4];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const float p0 = ex2(sh[n][0] - b0), p1 = ex2(sh[n][1] - b0);
            const float p2 = ex2(sh[n][2] - b1), p3 = ex2(sh[n][3] - b1);
            l0 += p0 + p1;
            l1 += p2 + p3;
            split2(p0, p1, ph[2 * n], pl[2 * n]);
            split2(p2, p3, ph[2 * n + 1], pl[2 * n + 1]);
        }
        const uint32_t vbuf = kbuf + kTileBytes;
#pragma unroll
        for (int n = 0; n < DP / 16; ++n) {
            uint32_t vf[4];  // d 0-7: keys 0-7, 8-15; d 8-15: the same
            ldsm4t(vf, vbuf + piece<kTileKeys>(k0 + (lane & 15), n * 2 + (lane >> 4)));
            float y[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
            mma16816(y[0], pl, vf[0], vf[1]);
            mma16816(y[1], pl, vf[2], vf[3]);
            mma16816(y[0], ph, vf[0], vf[1]);
            mma16816(y[1], ph, vf[2], vf[3]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                o[2 * n][e] += y[0][e];
                o[2 * n + 1][e] += y[1][e];
            }
        }
    };

    // the ragged rows: up to 31 keys with a mask for each query row.  A value
    // that is not finite is replaced by 0 and noted, so that it reaches no row
    // that does not see it; those that do become NaN at the end.
    bool spoiled0 = false, spoiled1 = false;
    if (ragged) {
        const uint32_t buf = (NS - 1) * 2 * kTileBytes;
        uint32_t bad = 0;
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            const int x = tid + j * kThreads, r = x / kPieces;
            if (not_finite8(kp[j]) || not_finite8(vp[j])) {
                bad |= 1u << r;
                kp[j] = vp[j] = make_uint4(0, 0, 0, 0);
            }
            const uint32_t at = buf + piece<kTileKeys>(r, x % kPieces);
            sts_uint4(smem + at, kp[j]);
            sts_uint4(smem + at + kTileBytes, vp[j]);
        }
        if (bad) atomicOr(flags, bad);
        __syncthreads();
        const int q0 = r0 + rt * 16 + gr, q1 = q0 + 8;
        const uint32_t see0 = q0 < rows ? a.mask[q0 / a.group] : 0u, see1 = q1 < rows ? a.mask[q1 / a.group] : 0u;
        for (int k0 = kw * 16; k0 < nragged; k0 += KW * 16) step(base + buf, k0, see0 >> k0, see1 >> k0, false);
        spoiled0 = (see0 & *flags) != 0;
        spoiled1 = (see1 & *flags) != 0;
        __syncthreads();
    }

    bool ok = true;
    int landed = 0;
    for (int t = 0; t < ntiles; ++t) {
        int sg, row;
        const int n = walk.next(a, kTileKeys, sg, row);  // keys of this tile: at least 1
        ok = ok && mbar_wait_bounded(&bar[t % NS], static_cast<uint32_t>(t / NS) & 1u, a.status, kDevStatusWaitTimeout);
        landed += ok ? 1 : 0;
        __syncthreads();
        if (tid == 0 && ok && t + NS - 1 < ntiles) {  // into the stage that every warp has left
            fence_proxy_async_smem();
            load_tile(t + NS - 1);
        }
        const uint32_t kbuf = base + (t % NS) * 2 * kTileBytes;
#pragma unroll
        for (int j = 0; j < RT; ++j) {
            const int k0 = (kw + j * KW) * 16;
            const uint32_t see = n - k0 >= 16 ? 0xffffu : (1u << max(0, n - k0)) - 1u;
            if (n > k0) step(kbuf, k0, see, see, n - k0 >= 16);
        }
    }
    if (tid == 0 && !ok)  // the copies under way still write into this block's memory
        for (int t = landed; t < min(ntiles, landed + NS); ++t)
            mbar_wait_bounded(&bar[t % NS], static_cast<uint32_t>(t / NS) & 1u, a.status, kDevStatusTxTimeout);
    ok = __syncthreads_and(ok);

    // the block's result: rows' maxima and sums over the warps that share them
#pragma unroll
    for (int x = 1; x < 4; x <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, x);
        l1 += __shfl_xor_sync(0xffffffffu, l1, x);
    }
    if (spoiled0) l0 = NAN;
    if (spoiled1) l1 = NAN;
    float2* ml = reinterpret_cast<float2*>(smem + L::kMlOff);
    float2* mlw = reinterpret_cast<float2*>(smem + L::kMlwOff);
    float* out = reinterpret_cast<float*>(smem + L::kOutOff);
    if (qt == 0) {
        mlw[kw * R + rt * 16 + gr] = make_float2(m0, l0);
        mlw[kw * R + rt * 16 + gr + 8] = make_float2(m1, l1);
    }
    __syncthreads();  // also: nobody reads the stages or q any more
    float* mine = KW == 1 ? out : reinterpret_cast<float*>(smem) + kw * R * L::kOutStride;
#pragma unroll
    for (int n = 0; n < DP / 8; ++n) {
        *reinterpret_cast<float2*>(mine + (rt * 16 + gr) * L::kOutStride + n * 8 + 2 * qt) = make_float2(o[n][0], o[n][1]);
        *reinterpret_cast<float2*>(mine + (rt * 16 + gr + 8) * L::kOutStride + n * 8 + 2 * qt) = make_float2(o[n][2], o[n][3]);
    }
    if constexpr (KW == 1) {
        if (tid < R) ml[tid] = mlw[tid];
    } else {
        __syncthreads();
        for (int x = tid; x < R * DP / 4; x += kThreads) {
            const int r = x / (DP / 4), d = x % (DP / 4) * 4;
            float M = kNegInf;
#pragma unroll
            for (int w = 0; w < KW; ++w) M = fmaxf(M, mlw[w * R + r].x);
            float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
            float l = 0.f;
#pragma unroll
            for (int w = 0; w < KW; ++w) {
                const float f = share(mlw[w * R + r].x, M);
                const float4 v = lds_float4(reinterpret_cast<const float*>(smem) + (w * R + r) * L::kOutStride + d);
                s.x = fmaf(f, v.x, s.x);
                s.y = fmaf(f, v.y, s.y);
                s.z = fmaf(f, v.z, s.z);
                s.w = fmaf(f, v.w, s.w);
                l = fmaf(f, mlw[w * R + r].y, l);
            }
            *reinterpret_cast<float4*>(out + r * L::kOutStride + d) = s;
            if (d == 0) ml[r] = make_float2(M, l);
        }
    }

    if (a.cluster > 1) cluster_sync();
    else __syncthreads();
    if (ok) join_cluster<DP, L::kOutStride, R, kThreads, 1>(a, tid, c, g, r0, rows, base + L::kMlOff, base + L::kOutOff);
    if (a.cluster > 1) cluster_leave();
}

// The kernel's attributes and its resident clusters of 8, once per device;
// null with the error set where that fails.
template <int RT>
const int* resident() {
    return device_once<RT, int>([](int& clusters) {
        cudaError_t e = cudaFuncSetAttribute(attn_mma_kernel<RT>, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<RT>::kBytes);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(attn_mma_kernel<RT>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return cuda_fail(e, "attention: cudaFuncSetAttribute");
        cudaLaunchAttribute attr[2];
        const cudaLaunchConfig_t cfg = cluster_config(8, dim3(8), kThreads, Layout<RT>::kBytes, nullptr, attr);
        if (cudaOccupancyMaxActiveClusters(&clusters, attn_mma_kernel<RT>, &cfg) != cudaSuccess) {
            cudaGetLastError();
            clusters = 0;
        }
        return static_cast<int>(MUSER_OK);
    });
}

template <int RT>
int launch(const AttnArgs& a, dim3 grid, cudaStream_t s) {
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = cluster_config(a.cluster, grid, kThreads, Layout<RT>::kBytes, s, attr);
    AttnMaps maps;
    MUSER_TRY(encode_attn_maps(a, kTileKeys, maps));
    const cudaError_t e = cudaLaunchKernelEx(&cfg, attn_mma_kernel<RT>, a, maps);
    if (e != cudaSuccess) return cuda_fail(e, "attention: cudaLaunchKernelEx");
    return check_launch("attention");
}

}  // namespace

// Whether TMA and 16-byte loads can read the planes' rows.
bool attn_mma_supported(const AttnArgs& a) {
    if (a.D % 8 != 0) return false;
    auto ok = [](const AttnSeg& s) {
        constexpr int64_t kMost = int64_t{1} << 39;  // a tensor map's strides are below 2^40 bytes
        return is_aligned(s.k, 16) && is_aligned(s.v, 16) && s.row_stride % 8 == 0 && s.head_stride % 8 == 0 &&
               s.row_stride < kMost && s.head_stride < kMost;
    };
    for (int i = 0; i < a.nseg; ++i)
        if (!ok(a.seg[i])) return false;
    for (int i = 0; i < 2 && a.n_edge > 0; ++i)
        if (i == 0 ? !ok(a.edge[0]) : (a.n_edge > a.edge0 && !ok(a.edge[1]))) return false;
    return true;
}

int attn_mma_row_tiles(int rows) { return rows <= 16 ? 1 : 2; }
const int* attn_mma_resident(int rt) { return rt == 1 ? resident<1>() : resident<2>(); }

// The driver's encoder, and its call that gives a map another address: V's map
// is K's but for that, and an encoding is 0.4 us of a call's host time.
struct MapEncoder {
    PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
    PFN_cuTensorMapReplaceAddress_v12000 readdress = nullptr;
};
static const MapEncoder& map_encoder() {
    static std::once_flag once;
    static MapEncoder m;
    std::call_once(once, [] {
        void *f = nullptr, *r = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess &&
            cudaGetDriverEntryPointByVersion("cuTensorMapReplaceAddress", &r, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess) {
            m.readdress = reinterpret_cast<PFN_cuTensorMapReplaceAddress_v12000>(r);
            m.encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
        }
    });
    return m;
}

// K's map of binary16 boxes in the 128-byte swizzle, and V's.
static int encode_pair(CUtensorMap& k, CUtensorMap& v, const uint16_t* key, const uint16_t* value, int rank,
                       const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box) {
    const MapEncoder& m = map_encoder();
    if (m.encode == nullptr) return set_error(MUSER_ERR_CUDA, "attention: cuTensorMapEncodeTiled is not available");
    const cuuint32_t one[4] = {1, 1, 1, 1};
    CUresult r = m.encode(&k, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, static_cast<cuuint32_t>(rank), const_cast<uint16_t*>(key), dims,
                          strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r == CUDA_SUCCESS) {
        v = k;
        r = m.readdress(&v, const_cast<uint16_t*>(value));
    }
    if (r != CUDA_SUCCESS) return set_error(MUSER_ERR_CUDA, "attention: a tensor map could not be made (%d)", static_cast<int>(r));
    return MUSER_OK;
}

int encode_attn_maps(const AttnArgs& a, int tile, AttnMaps& maps) {
    for (int i = 0; i < a.nseg; ++i) {
        const AttnSeg& S = a.seg[i];
        const cuuint64_t dims[3] = {static_cast<cuuint64_t>(a.D), static_cast<cuuint64_t>(S.rows), static_cast<cuuint64_t>(a.G)};
        const cuuint64_t strides[2] = {static_cast<cuuint64_t>(S.row_stride) * 2, static_cast<cuuint64_t>(S.head_stride) * 2};
        const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(tile), 1};
        MUSER_TRY(encode_pair(maps.k[i], maps.v[i], S.k, S.v, 3, dims, strides, box));
    }
    return MUSER_OK;
}

int encode_page_maps(uint16_t* key, uint16_t* value, const uint64_t (&dims)[4], const uint64_t (&strides)[3], int box_rows,
                     CUtensorMap (&maps)[2]) {
    cuuint64_t d[4], st[3];
    for (int i = 0; i < 4; ++i) d[i] = dims[i];
    for (int i = 0; i < 3; ++i) st[i] = strides[i];
    const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(box_rows), 1, 1};
    return encode_pair(maps[0], maps[1], key, value, 4, d, st, box);
}

int launch_attn_mma(const AttnArgs& a, dim3 grid, int rt, cudaStream_t s) {
    return rt == 1 ? launch<1>(a, grid, s) : launch<2>(a, grid, s);
}

}  // namespace muser
