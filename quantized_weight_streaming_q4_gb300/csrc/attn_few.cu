// attn_few.cu -- tree attention of few query rows (up to 32 vectors a K/V
// head: single tokens, small trees) on the fifth-generation tensor cores, for
// head sizes that are multiples of 8 up to 128 and 16-byte aligned planes.
//
// With few rows the cached keys take the tile's 128 lanes and the rows its
// columns, so no lane idles: R rows are 2 R columns, the binary16 high parts of
// the scaled q beside the low ones, which come back as two sums and are added
// in binary32:
//   S^T = K Q^T   A = K [keys][d], B = Q [2 R][d]
//   O^T = V^T P^T A = V as it lies in the cache (M along its rows), B = P
//         [keys][2 R], high and low parts of p again
// (32 columns a tile of 128 keys cost 512 cycles of tensor core; mma.sync, at
// 16 cycles a 16 x 8 x 16 product, took 4,000 and held one token over 130,815
// rows at 31 us.)
//
// A thread of a softmax warpgroup holds one key's scores against 16 rows, and
// later one output element of the same rows.  The maximum over keys would be a
// reduction across lanes for every tile; instead p = 2^(s - m + 11) with a
// reference m per row that is the first tile's maximum and moves only when
// some s exceeds it by more than 4 (binary16 ends at 2^16), which all threads
// agree on with one barrier.  The result does not depend on m but for
// rounding.  O tiles are fresh accumulators added in registers.
//
// Bound: the planes' bytes for long caches (TMA, three stages of 64 KB in
// flight a block, two for 32 rows), latency for short ones.
#include <algorithm>

#include "attn.cuh"
#include "attn_parts.cuh"
#include "kernels.cuh"
#include "tc.cuh"

namespace muser {
namespace {

constexpr int kTile = 128;              // keys of a tile
constexpr uint32_t kItem = kTile * 256; // a K or a V tile: two blocks of 64 elements a row
constexpr uint32_t kHalf = kTile * 128;
constexpr float kOff = 11.f, kMost = 15.f;

template <int R>
struct Layout {
    static constexpr int kGroups = R / 16, kThreads = 128 + 128 * kGroups;
    static constexpr int kNS = R == 16 ? 3 : 2;             // stages
    static constexpr uint32_t kN = 2 * R;                   // columns
    static constexpr uint32_t kKeyRow = kN / 8 * 128;       // P: bytes from 8 keys to the next 8
    static constexpr uint32_t kPBytes = kTile / 8 * kKeyRow;
    static constexpr uint32_t kVOff = kNS * kItem, kPOff = 2 * kNS * kItem;
    static constexpr uint32_t kQOff = kPOff + 2 * kPBytes;  // [d / 64][2 R][128 bytes]
    static constexpr uint32_t kScaleOff = kQOff + 2 * kN * 128;      // float[R]
    static constexpr uint32_t kRedOff = kScaleOff + R * 4;           // float[kGroups][4][16]
    static constexpr uint32_t kMaxOff = kRedOff + kGroups * 256;     // float[R]: the rows' references
    static constexpr uint32_t kMlOff = kMaxOff + R * 4;              // float2[R]
    static constexpr uint32_t kBarOff = kMlOff + R * 8;
    static constexpr uint32_t kBytes = kBarOff + 256;
    static constexpr uint32_t kOutStride = 132;             // floats; the output takes P's and q's place
    static_assert(R * kOutStride * 4 <= kScaleOff - kPOff, "the output fits");
    static_assert(kBytes <= 227 * 1024, "a block's shared memory");
    static constexpr uint32_t kTmemCols = 4 * kN;           // S and O, two buffers each
};
enum Bar { kKFull = 0, kVFull = 3, kKEmpty = 6, kVEmpty = 9, kSFull = 12, kPFull = 14, kOFull = 16, kQReady = 18, kRagged = 19, kBars = 20 };

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

// v[j] joined over the warp's lanes, j = 0..15: afterwards v[0] of lane l holds
// that of j = l / 2 (each step halves what a lane keeps).
template <typename F>
__device__ __forceinline__ void fold16(float (&v)[16], F&& f) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int h = 8; h >= 1; h >>= 1) {
        const bool up = (lane & (2 * h)) != 0;
#pragma unroll
        for (int j = 0; j < h; ++j) {
            const float give = up ? v[j] : v[j + h], keep = up ? v[j + h] : v[j];
            v[j] = f(keep, __shfl_xor_sync(0xffffffffu, give, 2 * h));
        }
    }
    v[0] = f(v[0], __shfl_xor_sync(0xffffffffu, v[0], 1));
}

template <int R>
__global__ void __launch_bounds__(Layout<R>::kThreads, 1)
    attn_few_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ AttnMaps maps) {
    using L = Layout<R>;
    constexpr int kNS = L::kNS;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t base = smem_u32(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint64_t* bar = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar + kBars);
    uint32_t* flags = tmem_slot + 1;
    volatile uint32_t* lost = tmem_slot + 2;  // a wait of a softmax thread ran out
    float* cs = reinterpret_cast<float*>(smem + L::kScaleOff);
    const int c = blockIdx.x, g = blockIdx.y, r0 = blockIdx.z * R;
    const int rows = a.M * a.group;
    // A single token's own row starts the last chunk's sums (`self`).  A tree's
    // rows, and those at the windows' lower edge, are a tile of that chunk: the
    // last one, where every tile has a stage of its own (a reference taken from
    // the few ragged keys alone would soon have to move), else tile 0.
    AttnWalk walk(a, c);
    const bool self = c == a.nchunks - 1 && a.M == 1, ragged = c == a.nchunks - 1 && a.M > 1;
    const int nragged = a.n_edge + a.M, ntiles = (ragged ? 1 : 0) + walk.count(a, kTile);
    const int rt = !ragged ? -1 : ntiles <= kNS ? ntiles - 1 : 0;
    auto next_tile = [&](int t, int& s, int& row) { return t == rt ? nragged : walk.next(a, kTile, s, row); };

    // q and the ragged rows: the loads of the softmax warpgroups go out first.
    // Thread (row, 16 elements); row r of the block: tree row i, head j of the group
    pdl_launch_dependents();
    const int w = (warp - 4) >> 2, th = tid & 127, id = 1 + w;  // 16 rows from 16 w on; key, later element
    const int qr = th >> 3, d0 = (th & 7) * 16;
    float4 x4[4];
    RaggedRaw raw[8];
    float4 ks[4];
    float vs = 0.f;
    if (warp >= 4) {
        pdl_wait();  // no global access before this
        const int r = r0 + w * 16 + qr, i = r / a.group;
        const float* src = a.q + (static_cast<int64_t>(i) * a.H + g * a.group + r - i * a.group) * a.D + d0;
#pragma unroll
        for (int u = 0; u < 4; ++u)
            x4[u] = r < rows && d0 + 4 * u < a.D ? __ldcg(reinterpret_cast<const float4*>(src) + u) : make_float4(0.f, 0.f, 0.f, 0.f);
        if (self) {
#pragma unroll
            for (int u = 0; u < 4; ++u)
                ks[u] = d0 + 4 * u < a.D ? __ldcg(reinterpret_cast<const float4*>(a.kt + g * a.D + d0) + u) : make_float4(0.f, 0.f, 0.f, 0.f);
            if (th < a.D) vs = __ldcg(a.vt + g * a.D + th);
        }
        if (ragged && w == 0) {
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int rr = (u & 3) * 8 + (th >> 4), p = th & 15;
                raw[u] = RaggedRaw{make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
                if (rr < nragged && p * 8 < a.D) raw[u] = attn_ragged_load(a, g, rr, p * 8, u >= 4);
            }
        }
    }
    uint32_t ragged_see = 0;  // bit j: row j sees ragged key th
    if (warp >= 4 && ragged && th < 32) {
        int i = (r0 + w * 16) / a.group, k = r0 + w * 16 - i * a.group;
        uint32_t seen = i < a.M ? (a.mask[i] >> th) & 1u : 0u;
        for (int j = 0; j < 16; ++j) {
            ragged_see |= seen << j;
            if (++k == a.group) {
                k = 0;
                ++i;
                seen = i < a.M ? (a.mask[i] >> th) & 1u : 0u;
            }
        }
    }
    if (warp == 3) touch_args(a, lane);
    if (tid == 0) {
        for (int i = 0; i < 3; ++i) {
            mbar_init(&bar[kKFull + i], 1);
            mbar_init(&bar[kVFull + i], 1);
            mbar_init(&bar[kKEmpty + i], 1);
            mbar_init(&bar[kVEmpty + i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar[kSFull + i], 1);
            mbar_init(&bar[kPFull + i], 128 * L::kGroups);
            mbar_init(&bar[kOFull + i], 1);
        }
        mbar_init(&bar[kQReady], 128 * L::kGroups);
        mbar_init(&bar[kRagged], 128);
        *flags = 0;
        *lost = 0;
        fence_mbar_init();
    }
    if (warp == 0) tmem_alloc(tmem_slot, L::kTmemCols);
    if (warp < 4) pdl_wait();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // A thread whose wait has run out waits no more and goes on with what is
    // there: warps and warpgroups stay together at the instructions and barriers
    // that take all of them.  The block's rows become NaN; what it would have
    // joined is not written.
    bool ok = true;
    auto wait = [&](int b, int phase) {
        if (ok) ok = mbar_wait_bounded(&bar[b], static_cast<uint32_t>(phase & 1), a.status, kDevStatusWaitTimeout);
    };
    float2* ml = reinterpret_cast<float2*>(smem + L::kMlOff);
    float* out = reinterpret_cast<float*>(smem + L::kPOff);
    const int ksteps = (a.D + 15) / 16;  // along d; the rest of K's tile is zero

    if (warp == 0) {
        // --------------------------------------------- matrix products
        const bool leader = elect_one();
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint64_t qd = desc_swizzle128(base + L::kQOff, 16, 1024);
        const uint32_t ids = idesc(L::kN, false, false), ido = idesc(L::kN, true, true);
        int keys[2];
        auto scores = [&](int t) {
            const int s = t & 1, st = t % kNS;
            int sg, row;
            keys[s] = next_tile(t, sg, row);
            wait(kKFull + st, t / kNS);
            tc_fence_after();
            const uint64_t kd = desc_swizzle128(base + st * kItem, 16, 1024);
            const uint32_t d = tm + s * L::kN;
            if (leader && ok) {
#pragma unroll
                for (int ks = 0; ks < 8; ++ks)
                    if (ks < ksteps) {
                        const uint64_t ka = kd + ((ks >> 2) * kHalf + (ks & 3) * 32 >> 4), qb = qd + ((ks >> 2) * (L::kN * 128) + (ks & 3) * 32 >> 4);
                        if (ks == 0) mma_ss<false>(d, ka, qb, ids);
                        else mma_ss<true>(d, ka, qb, ids);
                    }
                mma_commit(&bar[kSFull + s]);
                mma_commit(&bar[kKEmpty + st]);
            }
            __syncwarp();
        };
        wait(kQReady, 0);
        tc_fence_after();
        if (ntiles > 0) scores(0);
        for (int t = 0; t < ntiles; ++t) {
            const int s = t & 1, st = t % kNS, steps = (keys[s] + 15) / 16;
            if (t + 1 < ntiles) scores(t + 1);
            wait(kPFull + s, t >> 1);
            wait(kVFull + st, t / kNS);
            tc_fence_after();
            const uint64_t vd = desc_swizzle128(base + L::kVOff + st * kItem, kHalf, 1024);
            const uint64_t pd = desc_bits(base + L::kPOff + s * L::kPBytes, L::kKeyRow, 128);
            const uint32_t d = tm + 2 * L::kN + s * L::kN;
            if (leader && ok) {
                mma_ss<false>(d, vd, pd, ido);
#pragma unroll
                for (int ks = 1; ks < kTile / 16; ++ks)
                    if (ks < steps) mma_ss<true>(d, vd + (ks * 2048 >> 4), pd + (ks * 2 * L::kKeyRow >> 4), ido);
                mma_commit(&bar[kOFull + s]);
                mma_commit(&bar[kVEmpty + st]);
            }
            __syncwarp();
        }
    } else if (warp < 3) {
        // ------------------------------------------------- K, V loads
        if (lane == 0) {
            const int v = warp - 1, full = v ? kVFull : kKFull, empty = v ? kVEmpty : kKEmpty;
            const uint32_t boxes = a.D <= 64 ? 1 : 2;
            int t = 0;
            for (; t < ntiles; ++t) {
                const int st = t % kNS;
                int sg, row;
                next_tile(t, sg, row);
                if (t == rt) {  // a softmax warpgroup stores this one
                    wait(kRagged, 0);
                    if (!ok) break;
                    mbar_arrive(&bar[full + st]);
                    continue;
                }
                if (t >= kNS) wait(empty + st, t / kNS - 1);
                if (!ok) break;
                const uint32_t dst = base + (v ? L::kVOff : 0u) + st * kItem;
                const CUtensorMap* map = v ? &maps.v[sg] : &maps.k[sg];
                mbar_arrive_expect_tx(&bar[full + st], boxes * kHalf);
                for (uint32_t x = 0; x < boxes; ++x) tma_load_box(dst + x * kHalf, map, static_cast<int>(x), row, g, &bar[full + st]);
            }
            for (int u = max(0, t - kNS); u < t && !ok; ++u)  // copies under way still write into this block's memory
                if (u != rt) mbar_wait_bounded(&bar[full + u % kNS], static_cast<uint32_t>(u / kNS) & 1u, a.status, kDevStatusTxTimeout);
        }
        __syncwarp();
    } else if (warp == 3) {
        prefetch_gate<R, 32>(a, lane, g, r0, rows);
    } else {
        // --------------------------------------- softmax and accumulation
        const uint32_t mine = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + w * 16;
        {
            float mx = 0.f;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                x4[u].x *= a.scale_log2;
                x4[u].y *= a.scale_log2;
                x4[u].z *= a.scale_log2;
                x4[u].w *= a.scale_log2;
                mx = fmaxf(fmaxf(mx, fmaxf(fabsf(x4[u].x), fabsf(x4[u].y))), fmaxf(fabsf(x4[u].z), fabsf(x4[u].w)));
            }
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            if (self) {  // the row's score against itself, K rounded as the cache will hold it
                float dot = 0.f;
                bool fine = true;
                auto add = [&](float q, float k) {
                    const float k16 = __half2float(__float2half_rn(k));
                    fine = fine && fabsf(k16) < INFINITY;
                    dot = fmaf(q, k16, dot);
                };
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    add(x4[u].x, ks[u].x);
                    add(x4[u].y, ks[u].y);
                    add(x4[u].z, ks[u].z);
                    add(x4[u].w, ks[u].w);
                }
#pragma unroll
                for (int o = 1; o < 8; o <<= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
                vs = __half2float(__float2half_rn(vs));
                fine = fine && fabsf(vs) < INFINITY;
                if (!fine) atomicOr(flags, 1u);
                if ((th & 7) == 0) reinterpret_cast<float*>(smem + L::kMaxOff)[w * 16 + qr] = dot;
            }
            const int e = min(127, max(-119, ((__float_as_int(mx) >> 23) & 0xff) - 127)) - 7;
            const float up = __int_as_float((127 - e) << 23);
            if ((th & 7) == 0) cs[w * 16 + qr] = __int_as_float((127 + e) << 23);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                uint4 hi, lo;
                split2(x4[2 * u].x * up, x4[2 * u].y * up, hi.x, lo.x);
                split2(x4[2 * u].z * up, x4[2 * u].w * up, hi.y, lo.y);
                split2(x4[2 * u + 1].x * up, x4[2 * u + 1].y * up, hi.z, lo.z);
                split2(x4[2 * u + 1].z * up, x4[2 * u + 1].w * up, hi.w, lo.w);
                const int p = (d0 >> 3) + u;
                sts_uint4(smem + L::kQOff + piece<L::kN>(w * 16 + qr, p), hi);
                sts_uint4(smem + L::kQOff + piece<L::kN>(R + w * 16 + qr, p), lo);
            }
            if (a.D <= 64) {  // V's second 64 elements are zero
                for (int z = tid - 128; z < kNS * static_cast<int>(kHalf / 16); z += 128 * L::kGroups)
                    sts_uint4(smem + L::kVOff + (z / (kHalf / 16)) * kItem + kHalf + z % (kHalf / 16) * 16, make_uint4(0, 0, 0, 0));
            }
            fence_proxy_async_smem();
            mbar_arrive(&bar[kQReady]);
            if (ragged && w == 0) {  // stored as tile rt; a value that is not finite becomes 0 and is noted
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const int rr = (u & 3) * 8 + (th >> 4), p = th & 15;
                    uint4 y = attn_ragged_pack(a, rr, raw[u]);
                    if (not_finite8(y)) {
                        atomicOr(flags, 1u << rr);
                        y = make_uint4(0, 0, 0, 0);
                    }
                    if (p < 8 || a.D > 64) sts_uint4(smem + (u >= 4 ? L::kVOff : 0u) + rt % kNS * kItem + piece<kTile>(rr, p), y);
                }
                fence_proxy_async_smem();
                mbar_arrive(&bar[kRagged]);
            }
        }
        named_barrier_sync(id, 128);  // the rows' scales
        const bool alone = gridDim.x == 1;  // nothing to join: straight to memory, a row at a time
        const int ti0 = (r0 + w * 16) / a.group, tk0 = r0 + w * 16 - ti0 * a.group;  // row r: tree row, head of the group
        const int live = th < a.D ? min(16, rows - r0 - w * 16) : 0;  // of this thread's rows
        const int64_t at0 = (static_cast<int64_t>(ti0) * a.H + g * a.group + tk0) * a.D + th;
        const int skip = (a.H - a.group) * a.D;  // from one tree row's group to the next
        float z[16];
        if (alone && a.gate) {
            const float* p = a.gate + at0;
#pragma unroll
            for (int j = 0, k = tk0; j < 16; ++j) {
                z[j] = j < live ? __ldcg(p) : 0.f;
                p += a.D;
                if (++k == a.group) k = 0, p += skip;
            }
        }
        float sc[16], b[16], m[16], l[16], o[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            sc[j] = cs[w * 16 + j];
            m[j] = self ? reinterpret_cast<float*>(smem + L::kMaxOff)[w * 16 + j] : kNegInf;
            b[j] = self ? kOff - m[j] : 0.f;
            l[j] = self && th == 0 ? 0x1p11f : 0.f;  // 2^kOff
            o[j] = self ? 0x1p11f * vs : 0.f;
        }
        if (self) named_barrier_sync(id, 128);  // before the references are written again
        auto drain = [&](int t) {  // adds the output tile t
            wait(kOFull + (t & 1), t >> 1);
            tc_fence_after();
            float hi[16], lo[16];
            tmem_ld16(mine + 2 * L::kN + (t & 1) * L::kN, hi);
            tmem_ld16(mine + 2 * L::kN + (t & 1) * L::kN + R, lo);
            tc_wait_ld(hi);
            tc_wait_ld(lo);
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] += hi[j] + lo[j];
            tc_fence_before();
        };
        for (int t = 0; t < ntiles; ++t) {
            int sg, srow;
            const int real = next_tile(t, sg, srow);
            uint32_t see = th < real ? 0xffffu : 0u;  // bit j: row j sees this thread's key
            if (t == rt) see = ragged_see;
            wait(kSFull + (t & 1), t >> 1);
            tc_fence_after();
            float s[16], x[16];
            tmem_ld16(mine + (t & 1) * L::kN, s);
            tmem_ld16(mine + (t & 1) * L::kN + R, x);
            tc_wait_ld(s);
            tc_wait_ld(x);
            float top = kNegInf;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                s[j] = (see >> j) & 1u ? (s[j] + x[j]) * sc[j] : kNegInf;
                x[j] = s[j] + b[j];
                top = fmaxf(top, x[j]);
            }
            bool drained = t == 0;
            const bool anew = group_any(id, (t == 0 && !self) || top > kMost);
            if (anew) {  // a new reference: the largest score so far
                if (!drained) drain(t - 1);
                drained = true;
                float* red = reinterpret_cast<float*>(smem + L::kRedOff) + w * 64;
                float v[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] = s[j];
                fold16(v, [](float p, float q) { return fmaxf(p, q); });
                if ((lane & 1) == 0) red[(warp & 3) * 16 + (lane >> 1)] = v[0];
                named_barrier_sync(id, 128);
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float mn = fmaxf(fmaxf(fmaxf(m[j], red[j]), fmaxf(red[16 + j], red[32 + j])), red[48 + j]);
                    const float f = m[j] == kNegInf ? 0.f : ex2(m[j] - mn);
                    m[j] = mn;
                    b[j] = mn == kNegInf ? INFINITY : kOff - mn;  // no score yet: the next one asks again
                    l[j] *= f;
                    o[j] *= f;
                    x[j] = s[j] == kNegInf ? kNegInf : s[j] + b[j];
                }
                if (th == 0) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) reinterpret_cast<float*>(smem + L::kMaxOff)[w * 16 + j] = m[j];
                }
                named_barrier_sync(id, 128);  // red is free again
            }
            // p, its parts to P [keys][2 R]
            uint32_t hi[8], lo[8];
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
                const float p0 = (see >> j) & 1u ? ex2(x[j]) : 0.f, p1 = (see >> (j + 1)) & 1u ? ex2(x[j + 1]) : 0.f;
                l[j] += p0;
                l[j + 1] += p1;
                split2(p0, p1, hi[j / 2], lo[j / 2]);
            }
            uint8_t* pt = smem + L::kPOff + (t & 1) * L::kPBytes + (th >> 3) * L::kKeyRow + (th & 7) * 16 + w * 256;
            sts_uint4(pt, make_uint4(hi[0], hi[1], hi[2], hi[3]));
            sts_uint4(pt + 128, make_uint4(hi[4], hi[5], hi[6], hi[7]));
            sts_uint4(pt + R / 8 * 128, make_uint4(lo[0], lo[1], lo[2], lo[3]));
            sts_uint4(pt + R / 8 * 128 + 128, make_uint4(lo[4], lo[5], lo[6], lo[7]));
            fence_proxy_async_smem();
            tc_fence_before();
            mbar_arrive(&bar[kPFull + (t & 1)]);
            if (!drained) drain(t - 1);
        }
        if (ntiles > 0) drain(ntiles - 1);
        // the rows' sums over the keys' threads, then this chunk's result
        float* red = reinterpret_cast<float*>(smem + L::kRedOff) + w * 64;
        fold16(l, [](float p, float q) { return p + q; });
        if ((lane & 1) == 0) red[(warp & 3) * 16 + (lane >> 1)] = l[0];
        if (!ok) *lost = 1;
        named_barrier_sync(id, 128);
        if (th < 16) {
            float sum = (red[th] + red[16 + th]) + (red[32 + th] + red[48 + th]);
            const int i = (r0 + w * 16 + th) / a.group;
            if ((ragged || self) && i < a.M && (a.mask[i] & *flags)) sum = NAN;  // it sees a ragged row that is not finite
            if (*lost) sum = NAN;
            if (alone) cs[w * 16 + th] = __fdividef(1.f, sum);
            else ml[w * 16 + th] = make_float2(ntiles > 0 || self ? reinterpret_cast<float*>(smem + L::kMaxOff)[w * 16 + th] : kNegInf, sum);
        }
        if (alone) {
            named_barrier_sync(1 + L::kGroups, 128 * L::kGroups);
            const bool any_lost = *lost != 0;  // the other warpgroup's too
            float* p = a.out + at0;
#pragma unroll
            for (int j = 0, k = tk0; j < 16; ++j) {
                float v = o[j] * cs[w * 16 + j];
                if (a.gate) v = __fdividef(v, 1.f + __expf(-z[j]));
                if (j < live) *p = any_lost ? NAN : v;
                p += a.D;
                if (++k == a.group) k = 0, p += skip;
            }
        }
        named_barrier_sync(1 + L::kGroups, 128 * L::kGroups);  // every group's last product is done: P and q are free
        if (!alone) {
#pragma unroll
            for (int j = 0; j < 16; ++j) out[(w * 16 + j) * L::kOutStride + th] = o[j];
        }
    }
    tc_fence_before();
    ok = __syncthreads_and(ok);
    if (warp == 0) {
        tc_fence_after();
        tmem_free(tmem, L::kTmemCols);
    }
    if (gridDim.x == 1) return;
    if (a.cluster > 1) cluster_sync();
    if (ok) join_cluster<128, L::kOutStride, R, L::kThreads, 8>(a, tid, c, g, r0, rows, base + L::kMlOff, base + L::kPOff);
    if (a.cluster > 1) cluster_leave();
}

// The kernel's attributes and resident clusters, once per device; null with
// the error set where that fails.
template <int R>
const AttnResident* resident() {
    return device_once<R, AttnResident>([](AttnResident& r) {
        cudaError_t e = cudaFuncSetAttribute(attn_few_kernel<R>, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<R>::kBytes);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(attn_few_kernel<R>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return cuda_fail(e, "attention: cudaFuncSetAttribute");
        for (int i = 0; i < 5; ++i) {
            cudaLaunchAttribute attr[2];
            const cudaLaunchConfig_t cfg = cluster_config(1 << i, dim3(1u << i), Layout<R>::kThreads, Layout<R>::kBytes, nullptr, attr);
            if (cudaOccupancyMaxActiveClusters(&r.clusters[i], attn_few_kernel<R>, &cfg) != cudaSuccess) {
                cudaGetLastError();
                r.clusters[i] = 0;
            }
        }
        return static_cast<int>(MUSER_OK);
    });
}

template <int R>
int launch(const AttnArgs& a, dim3 grid, cudaStream_t s) {
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = cluster_config(a.cluster, grid, Layout<R>::kThreads, Layout<R>::kBytes, s, attr);
    AttnMaps maps;
    MUSER_TRY(encode_attn_maps(a, kTile, maps));
    const cudaError_t e = cudaLaunchKernelEx(&cfg, attn_few_kernel<R>, a, maps);
    if (e != cudaSuccess) return cuda_fail(e, "attention: cudaLaunchKernelEx");
    return check_launch("attention");
}

}  // namespace

const AttnResident* attn_few_resident(int rows) { return rows <= 16 ? resident<16>() : resident<32>(); }

int launch_attn_few(const AttnArgs& a, dim3 grid, cudaStream_t s) {
    return a.M * a.group <= 16 ? launch<16>(a, grid, s) : launch<32>(a, grid, s);
}

}  // namespace muser
