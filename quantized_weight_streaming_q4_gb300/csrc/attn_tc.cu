// attn_tc.cu -- tree attention on the fifth-generation tensor cores, for head
// sizes that are multiples of 8 up to 128 and 16-byte aligned planes.
//
// A block takes one K/V head, 128 of the group's M * group query vectors (one
// per TMEM lane) and one chunk of the cached rows, in tiles of up to 128 keys:
//   S = Q K^T  (tcgen05.mma, A = Q in TMEM, B = K in shared memory)
//   p = 2^(S - m + 14), written over S in TMEM as the next product's A operand
//   O = P V    (B = V as it lies in the cache: keys along K, N contiguous)
// Even and odd tiles are two independent softmax streams, one warpgroup each: a
// thread owns a query row of its tiles, whose p are relative to the tile's own
// maximum, so a stream depends on nothing but its scores, and nothing passes
// between lanes.  A third warpgroup holds the rows' outputs (128 binary32
// registers a thread) and adds each tile's with its share.  While one stream's
// exponentials run, the tensor core works for the other.  Every O tile is a
// fresh accumulator added in registers: the tensor core's additions truncate,
// and a long chain of them drifts (8.4e-6 of the result after 3,456 keys on one
// accumulator; 8 steps do not show).
//
// Precision as in attn_mma.cu: q and p are each two binary16 parts, so both
// products run twice, low parts first.
//
// Warps: 0 issues the matrix products, 1 and 2 the TMA loads of K and of V
// (128-byte swizzle: K with d contiguous along the product's K, V along its
// N); 4-7 and 8-11 are the two streams, which also store the rows whose
// visibility differs; 12-15 the outputs.  K and V wait for their buffers apart:
// one thread for both held a free K buffer back behind V's.  The registers are
// split 40 : 144 : 144 : 184 a thread; a stream that held all 128 scores of its
// row spilled (83 us below).
//
// Bound: the tensor pipe, 32 products of 64 cycles a tile, 2,050 of about 2,700
// cycles; of the 57 to 60 us of 16 rows over 130,815 rows that is 38, beside 7.5
// from the launch to the first scores, 6.2 for the join and 5.9 for the second
// kernel.  For short caches what comes before the first product and behind the
// last (16 rows, 2,048 rows: 12 us).
#include <algorithm>

#include "attn.cuh"
#include "attn_parts.cuh"
#include "kernels.cuh"
#include "tc.cuh"

namespace muser {
namespace {

constexpr int kThreads = 512;
constexpr int kTile = 128;
constexpr uint32_t kTmemCols = 512, kColO = 256, kColQ = 384;  // S0, S1 at 0 and 128

template <int DP>
struct Layout {
    static constexpr uint32_t kItem = kTile * DP * 2;  // a K or a V tile
    static constexpr uint32_t kOutStride = DP + 4;     // floats: q, or outputs with their row's maximum and sum
    static constexpr uint32_t kOutOff = 4 * kItem;     // behind K0, K1, V0, V1: q, later the cluster's outputs
    static constexpr uint32_t kHalfOff = kOutOff + 128 * kOutStride * 4;  // float[2][128]
    static constexpr uint32_t kStatOff = kHalfOff + 128 * 8;  // float2[4][128]: four tiles' maxima and sums
    static constexpr uint32_t kBarOff = kStatOff + 4 * 128 * 8;
    static constexpr uint32_t kBytes = kBarOff + 256;
};
enum Bar { kKFull = 0, kVFull = 2, kVEmpty = 4, kSFull = 6, kPFull = 8, kOFull = 10, kQReady = 12, kRagged = 13, kJoin = 14, kBars = 15 };

template <int DP>
__global__ void __launch_bounds__(kThreads, 1) attn_tc_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ AttnMaps maps) {
    using L = Layout<DP>;
    constexpr uint32_t kHalf = kTile * 128;  // bytes from 64 elements of a tile's rows to the next 64
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t base = smem_u32(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint64_t* bar = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar + kBars);
    uint32_t* flags = tmem_slot + 1;
    volatile uint32_t* lost = tmem_slot + 2;  // a wait of the block ran out
    const int c = blockIdx.x, g = blockIdx.y, r0 = blockIdx.z * 128;
    const int rows = a.M * a.group;
    // tile 0 of the last chunk holds the ragged rows; the common ones follow
    const int ragged = c == a.nchunks - 1 ? 1 : 0, nragged = a.n_edge + a.M;

    pdl_launch_dependents();
    if (warp == 3) touch_args(a, lane);
    if (warp < 3 && lane == 0 && a.nseg > 0) prefetch_map(warp == 1 ? &maps.k[0] : &maps.v[0]);
    // q and the ragged rows: coalesced loads of the streams, all in flight
    // together and before the block's set-up, then through shared memory.
    // (Asynchronous 16-byte copies of q moved 12 bytes a clock, 512-byte bulk
    // copies 9.)
    constexpr int kStep = 256 / (DP / 4), kQ = 128 / kStep;  // rows of one pass, passes
    const int qd = tid % (DP / 4) * 4, q0 = (tid - 128) / (DP / 4);
    float4 q4[kQ];
    constexpr int kEach = 2 * 32 * (DP / 8) / 256;
    uint4 x[kEach];
    if (warp >= 4 && warp < 12) {
        pdl_wait();  // no global access before this
        RaggedRaw raw[kEach];
        auto ragged_at = [&](int u, int& r, int& p) {  // row and piece; of V where it returns true
            const int y = u * 256 + tid - 128, v = u >= kEach / 2 ? 1 : 0;
            r = y / (DP / 8) - v * 32;
            p = y % (DP / 8);
            return v != 0;
        };
        if (ragged) {
#pragma unroll
            for (int u = 0; u < kEach; ++u) {
                int r, p;
                const bool v = ragged_at(u, r, p);
                raw[u] = RaggedRaw{make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
                if (r < nragged && p * 8 < a.D) raw[u] = attn_ragged_load(a, g, r, p * 8, v);
            }
        }
        // row r0 + r of the block: tree row i, head j of the group
        int i = (r0 + q0) / a.group, j = r0 + q0 - i * a.group;
        const int skip = (a.H - a.group) * a.D;  // from one tree row's group to the next
        const float* src = a.q + static_cast<int64_t>(g * a.group + r0 + q0) * a.D + static_cast<int64_t>(i) * skip + qd;
#pragma unroll
        for (int u = 0; u < kQ; ++u) {
            q4[u] = r0 + q0 + u * kStep < rows && qd < a.D ? __ldcg(reinterpret_cast<const float4*>(src))
                                                           : make_float4(0.f, 0.f, 0.f, 0.f);
            src += kStep * a.D;
            for (j += kStep; j >= a.group; j -= a.group) src += skip;
        }
        if (ragged) {
#pragma unroll
            for (int u = 0; u < kEach; ++u) {
                int r, p;
                ragged_at(u, r, p);
                x[u] = attn_ragged_pack(a, r, raw[u]);
            }
        }
    }
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar[kKFull + i], 1);
            mbar_init(&bar[kVFull + i], 1);
            mbar_init(&bar[kVEmpty + i], 1);
            mbar_init(&bar[kSFull + i], 1);
            mbar_init(&bar[kPFull + i], 256);  // the stream's p, and the output tile before is read
            mbar_init(&bar[kOFull + i], 1);
        }
        mbar_init(&bar[kQReady], 256);
        mbar_init(&bar[kRagged], 256);
        mbar_init(&bar[kJoin], 1);
        *flags = 0;
        *lost = 0;
        fence_mbar_init();
        if (a.cluster > 1) mbar_arrive_expect_tx(&bar[kJoin], 128 * L::kOutStride * 4);
    }
    if (warp == 0) {
        tmem_alloc(tmem_slot, kTmemCols);
    }
    if (warp < 4 || warp >= 12) pdl_wait();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp >= 12) mbar_arrive(&bar[kPFull]);  // no output tile before the first
    AttnWalk walk(a, c);
    const int ntiles = ragged + walk.count(a, kTile);
    auto next_tile = [&](int t, int& s, int& row) { return t < ragged ? nragged : walk.next(a, kTile, s, row); };
    constexpr uint32_t tmem = 0;  // the address of an allocation of all columns
    // A thread whose wait has run out waits no more and goes on with what is
    // there, so that its warp stays together at the instructions that take all
    // of it.  The block's rows become NaN.
    bool ok = *tmem_slot == tmem;
    if (!ok) *lost = 1;
    auto wait = [&](int b, int phase) {
        if (!ok) return;
        ok = mbar_wait_bounded(&bar[b], static_cast<uint32_t>(phase & 1), a.status, kDevStatusWaitTimeout);
        if (!ok) *lost = 1;
    };
    float2* stat = reinterpret_cast<float2*>(smem + L::kStatOff);
    float* out = reinterpret_cast<float*>(smem + L::kOutOff);

    if (warp < 4) {
        set_regs_down<40>();
        if (a.cluster > 1) cluster_arrive();
        if (warp == 0) {
            // ------------------------------------------- matrix products
            // The whole warp runs the loop and one thread issues: under `lane ==
            // 0` alone every operand goes through a vector register, 130
            // cycles a product where the tensor core takes 64.
            const bool leader = elect_one();
            if (ntiles > 0) {
                int keys[2];  // of the tiles in the two score buffers, a multiple of 16
                auto scores = [&](int t) {
                    const int s = t & 1;
                    int sg, row;
                    keys[s] = (next_tile(t, sg, row) + 15) & ~15;
                    tc_fence_after();
                    const uint32_t id = idesc(static_cast<uint32_t>(keys[s]), false, false), d = tmem + s * 128, q = tmem + kColQ;
                    const uint64_t kd = desc_swizzle128(base + s * L::kItem, 16, 1024);
                    auto at = [&](int ks) { return kd + ((ks >> 2) * kHalf + (ks & 3) * 32 >> 4); };
                    if (leader) {
                        mma<false>(d, q + DP / 2, kd, id);  // the low part of q first
#pragma unroll
                        for (int ks = 1; ks < DP / 16; ++ks) mma<true>(d, q + DP / 2 + ks * 8, at(ks), id);
#pragma unroll
                        for (int ks = 0; ks < DP / 16; ++ks) mma<true>(d, q + ks * 8, at(ks), id);
                        mma_commit(&bar[kSFull + s]);
                    }
                    __syncwarp();
                };
                // Two waits at once, half of the lanes each.
                auto wait_both = [&](int b0, int phase0, int b1, int phase1) {
                    wait(lane & 1 ? b1 : b0, lane & 1 ? phase1 : phase0);
                    ok = __all_sync(0xffffffffu, ok);
                };
                wait_both(kQReady, 0, kKFull, 0);
                if (ok) scores(0);
                wait_both(kVFull, 0, ntiles > 1 ? kKFull + 1 : kVFull, 0);
                if (ok && ntiles > 1) scores(1);
#pragma unroll 1
                for (int t = 0; t < ntiles; ++t) {
                    const int s = t & 1;
                    wait(kPFull + s, t >> 1);  // and the output tile before is read
                    tc_fence_after();
                    const uint32_t id = idesc(DP, false, true), d = tmem + kColO, p = tmem + s * 128;
                    const uint64_t vd = desc_swizzle128(base + (2 + s) * L::kItem, kHalf, 1024);
                    const int steps = keys[s] / 16;
                    if (leader && ok) {
                        mma<false>(d, p + 8, vd, id);  // the low part of p first
#pragma unroll
                        for (int ks = 1; ks < kTile / 16; ++ks)
                            if (ks < steps) mma<true>(d, p + ks * 16 + 8, vd + (ks * 2048 >> 4), id);
#pragma unroll
                        for (int ks = 0; ks < kTile / 16; ++ks)
                            if (ks < steps) mma<true>(d, p + ks * 16, vd + (ks * 2048 >> 4), id);
                        mma_commit(&bar[kOFull + s]);
                        mma_commit(&bar[kVEmpty + s]);
                    }
                    __syncwarp();
                    // The queue holds about 330 cycles of products: what the warp
                    // does between them has to take less (a wait that is over takes
                    // 180).
                    if (t + 2 < ntiles) {
                        wait_both(kKFull + s, (t + 2) >> 1, kVFull + (s ^ 1), (t + 1) >> 1);
                        if (ok) scores(t + 2);
                    } else if (t + 1 < ntiles) {
                        wait(kVFull + (s ^ 1), (t + 1) >> 1);
                    }
                }
            }
        } else {
            // ------------------------------------------------- K, V loads
            if (warp == 3) prefetch_gate<128, 32>(a, lane, g, r0, rows);
            if (warp < 3 && lane == 0) {
                const int v = warp - 1, full = v ? kVFull : kKFull, empty = v ? kVEmpty : kSFull;
                int t = 0;
                for (; t < ntiles; ++t) {
                    const int s = t & 1;
                    int sg, row;
                    next_tile(t, sg, row);
                    if (t < ragged) {  // the streams store this one
                        wait(kRagged, 0);
                        if (!ok) break;
                        mbar_arrive(&bar[full + s]);
                        continue;
                    }
                    if (t >= 2) wait(empty + s, (t >> 1) - 1);
                    if (!ok) break;
                    const uint32_t dst = base + (v * 2 + s) * L::kItem;
                    const CUtensorMap* map = v ? &maps.v[sg] : &maps.k[sg];
                    mbar_arrive_expect_tx(&bar[full + s], L::kItem);
#pragma unroll
                    for (int x = 0; x < DP / 64; ++x) tma_load_box(dst + x * kHalf, map, x, row, g, &bar[full + s]);
                }
                for (int u = max(ragged, t - 2); u < t && !ok; ++u)  // copies under way still write into this block's memory
                    mbar_wait_bounded(&bar[full + (u & 1)], static_cast<uint32_t>(u >> 1) & 1u, a.status, kDevStatusTxTimeout);
            }
        }
        __syncwarp();
        // This warpgroup has 40 registers a thread: it shares no code with the
        // others from here on, only the barriers.
        tc_fence_before();
        if (a.cluster > 1) {
            cluster_wait();
            cluster_sync();
        } else {
            __syncthreads();
        }
        if (warp == 0) {
            tc_fence_after();
            tmem_free(tmem, kTmemCols);
        }
    } else {
        const int row = tid & 127;  // query row = TMEM lane
        const uint32_t mine = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint32_t mask = r0 + row < rows ? a.mask[(r0 + row) / a.group] : 0u;
        if (warp < 12) {
            set_regs_up<144>();
            // --------------------------------------------------- the streams
            const int w = (warp - 4) >> 2;
#pragma unroll
            for (int u = 0; u < kQ; ++u) sts_float4(out + (q0 + u * kStep) * L::kOutStride + qd, q4[u]);
            if (ragged) {  // stored as tile 0; a value that is not finite becomes 0 and is noted
#pragma unroll
                for (int u = 0; u < kEach; ++u) {
                    const int y = u * 256 + tid - 128, v = u >= kEach / 2 ? 1 : 0, r = y / (DP / 8) - v * 32, p = y % (DP / 8);
                    if (not_finite8(x[u])) {
                        atomicOr(flags, 1u << r);
                        x[u] = make_uint4(0, 0, 0, 0);
                    }
                    sts_uint4(smem + v * 2 * L::kItem + piece<kTile>(r, p), x[u]);
                }
                fence_proxy_async_smem();
                mbar_arrive(&bar[kRagged]);
            }
            named_barrier_sync(1, 256);
            // a thread takes half a row, the row's largest element from both
            float mx = 0.f;
#pragma unroll
            for (int i = 0; i < DP / 8; ++i) {
                q4[i] = lds_float4(out + row * L::kOutStride + w * (DP / 2) + i * 4);
                mx = fmaxf(fmaxf(mx, fmaxf(fabsf(q4[i].x), fabsf(q4[i].y))), fmaxf(fabsf(q4[i].z), fabsf(q4[i].w)));
            }
            float* half = reinterpret_cast<float*>(smem + L::kHalfOff);
            half[w * 128 + row] = mx;
            named_barrier_sync(1, 256);
            mx = fmaxf(mx, half[(w ^ 1) * 128 + row]);
            const int e = min(127, max(-119, ((__float_as_int(mx * fabsf(a.scale_log2)) >> 23) & 0xff) - 127)) - 7;
            const float qscale = a.scale_log2, up = __int_as_float((127 - e) << 23), down = __int_as_float((127 + e) << 23);
#pragma unroll
            for (int h = 0; h < DP / 64; ++h) {  // 32 elements: 16 columns of the high parts and 16 of the low ones
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float4 f = q4[h * 8 + i];
                    split2(f.x * qscale * up, f.y * qscale * up, hi[2 * i], lo[2 * i]);
                    split2(f.z * qscale * up, f.w * qscale * up, hi[2 * i + 1], lo[2 * i + 1]);
                }
                tmem_st16(mine + kColQ + w * (DP / 4) + h * 16, hi);
                tmem_st16(mine + kColQ + DP / 2 + w * (DP / 4) + h * 16, lo);
            }
            tc_wait_st();
            tc_fence_before();
            mbar_arrive(&bar[kQReady]);
            if (a.cluster > 1) cluster_arrive();  // q's place is free for the others' results

            const uint32_t scol = mine + w * 128;
#pragma unroll 1
            for (int t = 0; t < ntiles; ++t) {
                int sg, srow;
                const int real = next_tile(t, sg, srow), chunks = (real + 31) >> 5;
                if ((t & 1) != w) continue;
                wait(kSFull + w, t >> 1);
                tc_fence_after();
                // Columns [64 h, 64 h + 64) of the scores, -infinity where this
                // row does not see the key.  More at once did not fit the registers.
                float s[2][32];
                auto load = [&](int h) {
                    if (real == kTile && t >= ragged) {
                        tmem_ld32(scol + h * 64, s[0]);
                        tmem_ld32(scol + h * 64 + 32, s[1]);
                        tc_wait_ld(s[0]);
                        tc_wait_ld(s[1]);
                        return;
                    }
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int ch = 2 * h + k, left = min(32, max(0, real - ch * 32));
                        const uint32_t see = t < ragged ? (ch == 0 ? mask : 0u) : left == 32 ? 0xffffffffu : (1u << left) - 1u;
                        if (ch < chunks) tmem_ld32(scol + ch * 32, s[k]);
                        tc_wait_ld(s[k]);
#pragma unroll
                        for (int j = 0; j < 32; ++j) s[k][j] = (see >> j) & 1u ? s[k][j] : kNegInf;
                    }
                };
                float top[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
#pragma unroll 1
                for (int h = 1; h >= 0; --h) {
                    load(h);
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int j = 0; j < 32; j += 8)
#pragma unroll
                            for (int q = 0; q < 4; ++q) top[q] = fmaxf(top[q], fmaxf(s[k][j + q], s[k][j + q + 4]));
                }
                const float m = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * down;
                const float off = m == kNegInf ? 0.f : kOffset - m;
                // p: over the 32 columns read go, for each 16 keys, 8 columns of high
                // parts and 8 of low ones, the operand of one product
                float l0 = 0.f, l1 = 0.f;
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    if (2 * h >= chunks) break;
                    if (h == 1) load(1);  // the first half is still here
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        if (2 * h + k >= chunks) break;
                        uint32_t p[32];
#pragma unroll
                        for (int j = 0; j < 32; j += 2) {
                            const float p0 = ex2(fmaf(s[k][j], down, off)), p1 = ex2(fmaf(s[k][j + 1], down, off));
                            l0 += p0;
                            l1 += p1;
                            split2(p0, p1, p[(j & 16) + (j & 15) / 2], p[(j & 16) + 8 + (j & 15) / 2]);
                        }
                        tmem_st32(scol + h * 64 + k * 32, p);
                    }
                }
                // Read before tile t is: S(t) came after P V of t - 2, that after the
                // output of t - 3, hence after the use of t - 4's.
                stat[(t & 3) * 128 + row] = make_float2(m, l0 + l1);
                tc_wait_st();
                tc_fence_before();
                mbar_arrive(&bar[kPFull + w]);
            }
            if (a.cluster > 1) cluster_wait();
            else named_barrier_sync(2, 384);
        } else {
            // ---------------------------------------------------- the output
            set_regs_up<184>();
            if (a.cluster > 1) cluster_arrive();
            float m = kNegInf, l = 0.f;
            float o[DP];
#pragma unroll
            for (int d = 0; d < DP; ++d) o[d] = 0.f;
#pragma unroll 1
            for (int t = 0; t < ntiles; ++t) {
                const int s = t & 1;
                wait(kPFull + s, t >> 1);
                const float2 tile = stat[(t & 3) * 128 + row];
                const float mn = fmaxf(m, tile.x), f = share(m, mn), ft = share(tile.x, mn);
                m = mn;
                l = fmaf(l, f, tile.y * ft);
                wait(kOFull + s, t >> 1);
                tc_fence_after();
#pragma unroll
                for (int ch = 0; ch < DP / 32; ++ch) {
                    float x[32];
                    tmem_ld32(mine + kColO + ch * 32, x);
                    tc_wait_ld(x);
#pragma unroll
                    for (int j = 0; j < 32; ++j) o[ch * 32 + j] = fmaf(o[ch * 32 + j], f, x[j] * ft);
                }
                tc_fence_before();
                if (t + 1 < ntiles) mbar_arrive(&bar[kPFull + (s ^ 1)]);
            }
            // a wait ran out, or a ragged row that this row sees is not finite
            if (*lost || (mask & *flags)) l = NAN;
            // To the K and V tiles' place, and from there to the blocks that join
            // the rows.  (Reading the others' shared memory took 6,000 cycles in
            // a cluster of 4, storing there as long.)
            float* to = a.cluster > 1 ? reinterpret_cast<float*>(smem) : out;
            if (a.cluster > 1) cluster_wait();  // the others' q has been read
            else named_barrier_sync(2, 384);
            *reinterpret_cast<float2*>(to + row * L::kOutStride + DP) = make_float2(m, l);
#pragma unroll
            for (int d = 0; d < DP; d += 4) sts_float4(to + row * L::kOutStride + d, make_float4(o[d], o[d + 1], o[d + 2], o[d + 3]));
            if (a.cluster > 1) {
                fence_proxy_async_smem();
                named_barrier_sync(3, 128);
                if (row < a.cluster) {
                    const uint32_t bytes = 128 / a.cluster * L::kOutStride * 4;
                    copy_to_block(map_rank(base + L::kOutOff + cluster_rank() * bytes, row), base + row * bytes, bytes,
                                  map_rank(base + L::kBarOff + kJoin * 8, row));
                }
            }
        }
        tc_fence_before();
        if (a.cluster > 1) {
            wait(kJoin, 0);
            __syncwarp();
            cluster_arrive();
        } else {
            __syncthreads();
        }
        if (ok) merge_cluster<DP, L::kOutStride, 128, 384>(a, tid - 128, c, g, r0, rows, out);
        if (a.cluster > 1) {
            __syncwarp();
            cluster_wait();  // nobody leaves while copies read its shared memory
            // Every block has issued its copies by now: after a wait that ran out
            // they may still be on their way here.
            if (!ok) mbar_wait_bounded(&bar[kJoin], 0u, a.status, kDevStatusTxTimeout);
        }
    }
}

// The kernel's attributes and resident clusters, once per device; null with
// the error set where that fails.
template <int DP>
const AttnResident* resident() {
    return device_once<DP, AttnResident>([](AttnResident& r) {
        cudaError_t e = cudaFuncSetAttribute(attn_tc_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<DP>::kBytes);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(attn_tc_kernel<DP>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return cuda_fail(e, "attention: cudaFuncSetAttribute");
        for (int i = 0; i < 5; ++i) {
            cudaLaunchAttribute attr[2];
            const cudaLaunchConfig_t cfg = cluster_config(1 << i, dim3(1u << i), kThreads, Layout<DP>::kBytes, nullptr, attr);
            if (cudaOccupancyMaxActiveClusters(&r.clusters[i], attn_tc_kernel<DP>, &cfg) != cudaSuccess) {
                cudaGetLastError();
                r.clusters[i] = 0;
            }
        }
        return static_cast<int>(MUSER_OK);
    });
}

template <int DP>
int launch(const AttnArgs& a, dim3 grid, cudaStream_t s) {
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = cluster_config(a.cluster, grid, kThreads, Layout<DP>::kBytes, s, attr);
    AttnMaps maps;
    MUSER_TRY(encode_attn_maps(a, kTile, maps));
    const cudaError_t e = cudaLaunchKernelEx(&cfg, attn_tc_kernel<DP>, a, maps);
    if (e != cudaSuccess) return cuda_fail(e, "attention: cudaLaunchKernelEx");
    return check_launch("attention");
}

}  // namespace

const AttnResident* attn_tc_resident(int D) { return D <= 64 ? resident<64>() : resident<128>(); }

int launch_attn_tc(const AttnArgs& a, dim3 grid, cudaStream_t s) {
    return a.D <= 64 ? launch<64>(a, grid, s) : launch<128>(a, grid, s);
}

}  // namespace muser
