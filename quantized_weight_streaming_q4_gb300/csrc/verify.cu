// verify.cu -- verification of drafted (tree) tokens against the target's
// probabilities from given random numbers, and the token that follows.
//
// Sampling is one cooperative launch, over few logits one cluster of 16 blocks:
//  1. Every row with children is streamed once, in slices that a warp each
//     sums (2^(l log2(e) / T), binary32).  The acceptance tests need no more:
//     an error of 1e-6 in p / q moves a decision with probability 1e-6.
//  2. After a grid barrier every block walks the tree by itself from the same
//     numbers, so all take the same path.
//  3. What needs the whole vocabulary of one node (a rejected child's
//     remainder, the next token) all blocks do together, each on its own slice
//     of tokens, whose weights stay in shared memory, with one barrier each.
// Temperature 0, and a single row, are ordinary launches: the last block to
// finish its maxima (its slice's sum) walks (finds the token).
//
// The next token comes from integer weights: with R an integer >= the largest
// exponent, round(2^(l log2(e) / T - R) * 2^42), good to about 2^-38.  Sums of
// integers do not depend on their order, so neither does the token; and a
// binary32 exponential (2^-23) would move some of the 2e5 borders of the
// cumulative sums far enough to pick a neighbour about once in a thousand
// draws.  FP64 has no rate to speak of on GB300: it is kept for a few scalars.
//
// Bound: the rows' bytes (24 MB for 15 drafts over 202,048 tokens: 3.6 us),
// then latency: a launch, two to four grid barriers of 1.5 us (0.2 us in a
// cluster) and the loads behind them.  Outside a graph a cooperative launch
// takes 2.6 us more than another one (15 drafts, 202,048 tokens: 18.4 us, 15.8
// as an ordinary launch), but only it makes the waiting safe beside other
// kernels.
#include <algorithm>
#include <cmath>
#include <mutex>

#include "kernels.cuh"

namespace muser {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kFrac = 42;  // fraction bits of a weight
constexpr int kRows = 2 * MUSER_MAX_M;
constexpr int kVerifyTable = 128;
constexpr int kMaxSlices = 256;  // of a row
constexpr int kClusterBlocks = 16;
constexpr int64_t kClusterVocab = 40000, kClusterLogits = 1000000;
constexpr int kMaxBlocks = 160;  // 152 SMs; a lane of the warp that joins the blocks' sums takes 5
constexpr float kMaxExponent = 32768.f;
constexpr int kBad = 1 << 24;  // exponent mark of a slice that holds a NaN or an infinity
constexpr uint64_t kGridWaitNs = 2000000000ull;

struct VerifyArgs {
    const float* target;   // [M][V]
    const float* draft;    // [M][V] or null
    const int32_t* tokens; // [M]
    const float* uniform;  // [M]
    int32_t* result;       // [M + 2]
    int M, V;
    float c_hi, c_lo;      // log2(e) / T
    int vec;               // rows are 16-byte aligned
    int parent[MUSER_MAX_M];
    uint32_t children[MUSER_MAX_M];
    int nrows;             // rows streamed first (greedy: all; else rows with children, targets then drafts)
    int row_node[kRows];   // their nodes
    int ntarget;           // how many of them are target rows
    int target_at[MUSER_MAX_M], draft_at[MUSER_MAX_M];  // row index of a node's rows, or -1
    int slices, slice_len; // of a row in the first pass
    int span;              // tokens per block in the passes over one node
    unsigned* sync;        // arrivals, exits
    unsigned* near;        // [MUSER_MAX_M] by node, see kFirst
    float2* part;          // [kRows][kMaxSlices] (sum, exponent); greedy: uint64 keys
    uint64_t* sums;        // [2][kMaxBlocks][4]: two passes' buffers in turn, a record a block
    int* exps;             // [kMaxBlocks]
    unsigned* status;
    uint64_t table[kVerifyTable];  // 2^(j / 128) * 2^kFrac
};

// round(2^(l * c - R) * 2^kFrac) for an integer R >= l * c; 0 where that is
// below 2^-20 of the last bit and for l = -inf.  l * c = n + j / 128 + r with
// r held as two floats, y = r ln 2 likewise (|y| < 2^-8), and 2^r - 1 = y +
// y^2/2 + y^3/6 + y^4/24 to 2^-46; that sum is turned into units of 2^-39 by
// adding numbers whose last bit has the wanted weight, in two parts.
__device__ __forceinline__ uint64_t weight(float l, float c_hi, float c_lo, int R, const uint64_t* table) {
    const float h = l * c_hi;
    const float e = fmaf(l, c_lo, fmaf(l, c_hi, -h));
    const float nj = rintf(h * static_cast<float>(kVerifyTable));
    const float r0 = fmaf(-1.f / kVerifyTable, nj, h);  // exact: h - nj / 128
    const float r = r0 + e, rl = e - (r - r0);
    constexpr float kLn2Hi = 0.693147182464599609375f, kLn2Lo = -1.904654323148236e-09f;
    const float y = r * kLn2Hi;
    const float yl = fmaf(rl, kLn2Hi, fmaf(r, kLn2Lo, fmaf(r, kLn2Hi, -y)));
    const float z = fmaf(y, fmaf(y, 1.f / 24.f, 1.f / 6.f), 0.5f);
    const float s = fmaf(y * y, z, yl);
    constexpr float kMagic1 = 1.5f * 0x1p-7f;   // last bit 2^-30
    constexpr float kMagic2 = 1.5f * 0x1p-16f;  // last bit 2^-39
    const float yb = y + kMagic1;
    const float rest = (y - (yb - kMagic1)) + s;
    const int g = ((__float_as_int(yb) - __float_as_int(kMagic1)) << 9) +
                  (__float_as_int(rest + kMagic2) - __float_as_int(kMagic2));
    const int i = static_cast<int>(nj);
    const uint64_t t = table[i & (kVerifyTable - 1)];
    // t * (1 + g 2^-39): t >> 11 has 32 bits
    const int64_t prod = static_cast<int64_t>(static_cast<uint32_t>(t >> 11)) * static_cast<int64_t>(g);
    const uint64_t w = t + static_cast<uint64_t>(prod >> (39 - 11));
    const int down = R - (i >> 7);
    if (!(h > static_cast<float>(R) - 62.f)) return 0;
    return down > 0 ? (w + (1ull << (down - 1))) >> down : w;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint64_t shifted(uint64_t s, int by) { return by < 64 ? s >> by : 0; }
__device__ __forceinline__ uint64_t warp_sum64(uint64_t v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ uint64_t ldcg64(const uint64_t* p) {
    return __ldcg(reinterpret_cast<const unsigned long long*>(p));
}
__device__ __forceinline__ const float* row_ptr(const VerifyArgs& a, int row) {
    return (row < a.ntarget ? a.target : a.draft) + static_cast<int64_t>(a.row_node[row]) * a.V;
}

// Every block has arrived `times` times.  False if it gave up waiting.  One
// cluster has the hardware's barrier (0.2 us, where the grid's takes 1.7).  The
// clock is read every 32nd poll: reading it each time doubled the wait.
template <bool CLUSTER>
__device__ __forceinline__ bool grid_barrier(const VerifyArgs& a, unsigned times, int* flag) {
    if constexpr (CLUSTER) {
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
        return true;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        asm volatile("fence.acq_rel.gpu;\n\tred.relaxed.gpu.global.add.u32 [%0], 1;" ::"l"(a.sync) : "memory");
        const unsigned want = gridDim.x * times;
        uint64_t t0 = 0;
        int ok = 1;
        for (unsigned poll = 1;; ++poll) {
            unsigned v;
            asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(a.sync) : "memory");
            if (v >= want) break;
            if (poll % 32 == 0) {
                const uint64_t t = global_ns();
                if (t0 == 0) t0 = t;
                if (t - t0 > kGridWaitNs) {
                    atomicOr(a.status, kDevStatusWaitTimeout);
                    ok = 0;
                    break;
                }
            }
        }
        *flag = ok;
    }
    __syncthreads();
    return *flag != 0;
}

// Calls f(x, i) for this lane's logits x = p[i], lo <= i < hi, in batches whose
// loads are in flight together (four at a time where `vec`, else one).
template <typename F>
__device__ __forceinline__ void for_slice(const float* p, int lo, int hi, bool vec, F&& f) {
    const int lane = threadIdx.x & 31;
    if (vec) {  // lo is a multiple of 4
        constexpr int kBatch = 8;
        const float4* p4 = reinterpret_cast<const float4*>(p + lo);
        const int n4 = (hi - lo) >> 2;
        int i = lane;
        for (; i + (kBatch - 1) * 32 < n4; i += kBatch * 32) {
            float4 v[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) v[u] = __ldcg(p4 + i + u * 32);
#pragma unroll
            for (int u = 0; u < kBatch; ++u) f(v[u], lo + 4 * (i + u * 32));
        }
        for (; i < n4; i += 32) f(__ldcg(p4 + i), lo + 4 * i);
        return;
    }
    for (int i = lo + lane; i < hi; i += 128) {
        float4 v;
        v.x = __ldcg(p + i);
        v.y = i + 32 < hi ? __ldcg(p + i + 32) : -INFINITY;
        v.z = i + 64 < hi ? __ldcg(p + i + 64) : -INFINITY;
        v.w = i + 96 < hi ? __ldcg(p + i + 96) : -INFINITY;
        f(v, i);
    }
}

// The warp's unit of the first pass: slice u % slices of row u / slices.
__device__ __forceinline__ bool my_unit(const VerifyArgs& a, int& row, int& lo, int& hi) {
    const int u = static_cast<int>((threadIdx.x >> 5) * gridDim.x + blockIdx.x);  // spread over the blocks
    row = u / a.slices;
    lo = (u - row * a.slices) * a.slice_len;
    hi = min(lo + a.slice_len, a.V);
    return row < a.nrows;
}

// ----------------------------------------------------------- temperature 0
// The first maximum of a row as one number: the value's bits in an order that
// integers share, then the index counted down.  A NaN or +infinity is above
// all.
__device__ __forceinline__ uint64_t max_key(float x, int i) {
    const uint32_t b = __float_as_uint(x == 0.f ? 0.f : x);
    const uint32_t o = b & 0x80000000u ? ~b : b | 0x80000000u;
    return x < INFINITY ? (static_cast<uint64_t>(o) << 32) | (0xffffffffu - static_cast<uint32_t>(i)) : ~0ull;
}

__global__ void __launch_bounds__(kThreads) verify_greedy_kernel(const __grid_constant__ VerifyArgs a) {
    __shared__ int s_last, s_arg[MUSER_MAX_M], s_token[MUSER_MAX_M];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint64_t* keys = reinterpret_cast<uint64_t*>(a.part);
    pdl_launch_dependents();
    pdl_wait();  // no global access before this
    int row, lo, hi;
    if (my_unit(a, row, lo, hi)) {
        float best = -INFINITY;
        int arg = 0x7fffffff;
        bool bad = false;
        const int step = a.vec ? 1 : 32;
        for_slice(row_ptr(a, row), lo, hi, a.vec, [&](float4 v, int i) {
            bad |= !(fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)) < INFINITY) | (v.x != v.x) | (v.y != v.y) | (v.z != v.z) | (v.w != v.w);
            if (v.x > best) best = v.x, arg = i;
            if (v.y > best) best = v.y, arg = i + step;
            if (v.z > best) best = v.z, arg = i + 2 * step;
            if (v.w > best) best = v.w, arg = i + 3 * step;
        });
        uint64_t key = bad ? ~0ull : max_key(best, arg);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const uint64_t other = __shfl_xor_sync(0xffffffffu, key, o);
            key = key > other ? key : other;
        }
        if (lane == 0) keys[row * kMaxSlices + lo / a.slice_len] = key;
    }
    __syncthreads();
    if (tid == 0) s_last = atom_add_acq_rel_gpu(a.sync, 1u) == gridDim.x - 1;
    __syncthreads();
    if (!s_last) return;
    if (tid >= 1 && tid < a.M) s_token[tid] = __ldcg(a.tokens + tid);
    for (int r = warp; r < a.nrows; r += kWarps) {
        uint64_t key = 0;
        for (int i = lane; i < a.slices; i += 32) {
            const uint64_t k = ldcg64(keys + r * kMaxSlices + i);
            key = key > k ? key : k;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const uint64_t other = __shfl_xor_sync(0xffffffffu, key, o);
            key = key > other ? key : other;
        }
        const uint64_t none = 0x00800000ull << 32;  // keys of -infinity lie below
        if (lane == 0) s_arg[r] = key == ~0ull || key < none ? -1 : static_cast<int>(0xffffffffu - static_cast<uint32_t>(key));
    }
    __syncthreads();
    if (tid == 0) {
        int cur = 0, n = 1;
        a.result[2] = 0;
        for (int i = 1; i < a.M; ++i)
            if (a.parent[i] == cur && s_arg[cur] >= 0 && s_token[i] == s_arg[cur]) a.result[2 + n++] = cur = i;
        a.result[0] = n;
        a.result[1] = s_arg[cur];
        for (; n < a.M; ++n) a.result[2 + n] = -1;
        a.sync[0] = 0;
    }
}

// ---------------------------------------------------------------- sampling
struct Shared {
    uint64_t table[kVerifyTable];
    uint64_t warp[4][kWarps];
    float warp_max[kWarps], warp_left[kWarps];
    int slice[MUSER_MAX_M], slices;  // those with a child's token
    uint32_t slice_kids[MUSER_MAX_M];
    float row_sum[kRows], row_exp[kRows];  // a row's sum (NaN: no distribution) and exponent
    float px[MUSER_MAX_M], qx[MUSER_MAX_M], u[MUSER_MAX_M];  // of node i: p(x_i), q(x_i) in its parent's rows
    int token[MUSER_MAX_M];
    uint32_t first, fine;  // bit i: node i passes the test of a first child; its parent's rows are distributions
    // the present node's remainder: sums of P, Q and of what is left; c (thread 0's, in binary64)
    uint64_t sum_p, sum_q, total;
    double c;
    float c_f, left_f;
    uint64_t fm;  // f = c sum_p / sum_q = fm 2^fe, fm in [2^63, 2^64)
    int fe;
    // the sampled point: its block (-1: nothing to sample, -2: no distribution), the place in its share
    int owner, exp;
    uint64_t before;
    unsigned near[MUSER_MAX_M], near_all;  // kFirst: draft weights near f0, the block's by node, all blocks'
    int flag, found;
    int cur, n;  // the walk along accepted first children
    uint32_t kept;
};

__device__ __forceinline__ void split_factor(double f, uint64_t& fm, int& fe) {
    const long long bits = __double_as_longlong(f);
    fm = (static_cast<uint64_t>(bits & 0xfffffffffffffll) | 0x10000000000000ull) << 11;
    fe = static_cast<int>((bits >> 52) & 0x7ff) - 1023 - 63;
}
__device__ __forceinline__ void split_factor(float f, uint64_t& fm, int& fe) {
    const int bits = __float_as_int(f);
    fm = static_cast<uint64_t>((bits & 0x7fffff) | 0x800000) << 40;
    fe = ((bits >> 23) & 0xff) - 127 - 63;
}
// p / q for p, q > 0, to about 2^-60: with s = q 2^z in [1/2, 1), r = 1/s from
// binary32 and two Newton steps r += r (1 - s r) in 64-bit fixed point.
__device__ __forceinline__ void split_quotient(uint64_t p, uint64_t q, uint64_t& fm, int& fe) {
    const int zp = __clzll(static_cast<long long>(p)), zq = __clzll(static_cast<long long>(q));
    const uint64_t pn = p << zp, s = q << zq;
    const float r0 = 1.f / (static_cast<float>(static_cast<uint32_t>(s >> 40)) * 0x1p-24f);
    uint64_t r = static_cast<uint64_t>(static_cast<uint32_t>(r0 * 0x1p30f)) << 32;  // r 2^62
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const long long e = static_cast<long long>((1ull << 62) - __umul64hi(s, r));  // small, either sign
        r += static_cast<uint64_t>(__mul64hi(static_cast<long long>(r >> 1), e << 3));
    }
    const uint64_t f = __umul64hi(pn, r);
    const int z = __clzll(static_cast<long long>(f));
    fm = f << z;
    fe = zq - zp - 62 - z;
}
__device__ __forceinline__ uint64_t scaled(uint64_t t, int sh) {
    return t == 0 ? 0 : sh <= 0 ? shifted(t, -sh) : sh >= __clzll(static_cast<long long>(t)) ? ~0ull >> 1 : t << sh;
}
// f q of a weight (at most 2^43: 19 bits are kept below the last one) and of a
// block's sum of them.
__device__ __forceinline__ uint64_t times_f(uint64_t q, uint64_t fm, int fe) { return scaled(__umul64hi(q << 19, fm), fe + 64 - 19); }
__device__ __forceinline__ uint64_t sum_times_f(uint64_t q, uint64_t fm, int fe) { return scaled(__umul64hi(q, fm), fe + 64); }

// The tokens v0..v0+n-1 are a block's in a pass; a thread's are `per`
// neighbouring ones.
struct Span {
    int v0, n, per, first, last;  // first..last: this thread's, relative to v0
    __device__ __forceinline__ Span(const VerifyArgs& a, int block) {
        v0 = min(block * a.span, a.V);
        n = min(a.span, a.V - v0);
        per = (a.span + kThreads - 1) / kThreads;
        first = min(static_cast<int>(threadIdx.x) * per, n);
        last = min(first + per, n);
    }
};

// The block's sums of N values, to its record of the pass's buffer.
template <int N>
__device__ __forceinline__ void publish(const VerifyArgs& a, Shared& S, const uint64_t (&v)[N], unsigned barriers) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const uint64_t x = warp_sum64(v[j]);
        if (lane == 0) S.warp[j][warp] = x;
    }
    __syncthreads();
    if (warp == 0) {
        uint64_t t[N];
#pragma unroll
        for (int j = 0; j < N; ++j) t[j] = warp_sum64(lane < kWarps ? S.warp[j][lane] : 0);
        if (lane == 0) {
            ulonglong2* to = reinterpret_cast<ulonglong2*>(a.sums + ((barriers & 1) * kMaxBlocks + blockIdx.x) * 4);
            __stcg(to, make_ulonglong2(t[0], N > 1 ? t[N > 1 ? 1 : 0] : 0));
            if (N > 2) __stcg(to + 1, make_ulonglong2(t[N > 2 ? 2 : 0], t[N > 2 ? 3 : 0]));
        }
    }
}

// floor(u * total) for a float u in [0, 1).
__device__ __forceinline__ uint64_t fraction_of(float u, uint64_t total) {
    if (!(u > 0.f)) return 0;
    u = fminf(u, 0x1.fffffep-1f);
    const int e = (__float_as_int(u) >> 23) & 0xff;  // u = mant * 2^(e - 150)
    const uint64_t mant = e ? ((__float_as_int(u) & 0x7fffff) | 0x800000) : (__float_as_int(u) & 0x7fffff);
    const int down = 150 - (e ? e : 1);              // 25.. for u < 1: at least 24
    const uint64_t lo = mant * total, hi = __umul64hi(mant, total);
    if (down >= 128) return 0;
    return down >= 64 ? hi >> (down - 64) : (lo >> down) | (hi << (64 - down));
}

// What a pass over the present node left, put together by warp 0 of every
// block from the blocks' published sums:
//  kLeaf   weights relative to each block's own exponent;
//  kFirst  the first rejected child: sums of P, of Q, and of both over the tokens
//          with P > f0 Q, f0 being f from the first pass's binary32 sums.  With
//          f = sum P / sum Q now exact, a block's share is sum P - f sum Q over
//          those tokens.  This saves the barrier between f and the shares, but
//          the tokens between f0 and f are on the wrong side, each off by at
//          most |f - f0| Q.  They are among those with |P - f0 Q| <= 2^-20 f0 Q,
//          whose Q the blocks that have any add up (expected is one of 202,048
//          tokens): where that could come to 2^-38 of the row or 2^-20 of what
//          is left, or f0 is further off (logits in the thousands), a pass with
//          f follows (rows that are nearly equal: 202,048 logits 1e-5 apart put
//          the next token off by five);
//  kNext   a further rejected child, or the row itself: the shares.
// Leaves the remainder's size, and the sampled point's block and place there.
enum PassKind { kLeaf, kFirst, kNext };
constexpr int kNearUnit = 16;             // bits of a unit in which Q near f0 is added up
constexpr unsigned kNearMost = 1u << 18;  // units of a token or a block: more counts as all of Q
template <PassKind KIND>
__device__ __forceinline__ void settle(const VerifyArgs& a, Shared& S, unsigned barriers) {
    if (threadIdx.x < 32) {
        constexpr int kEach = kMaxBlocks / 32;
        const int lane = threadIdx.x, nb = gridDim.x, each = (nb + 31) / 32;
        const ulonglong2* from = reinterpret_cast<const ulonglong2*>(a.sums + (barriers & 1) * 4 * kMaxBlocks);
        const float u = __ldcg(a.uniform);
        uint64_t x[kEach], fm = 0;
        int e[kEach], R = KIND == kLeaf ? -(1 << 23) : 0, fe = 0;
        ulonglong2 s0[kEach], s1[KIND == kFirst ? kEach : 1];
#pragma unroll
        for (int k = 0; k < kEach; ++k) {  // every load of the lane's blocks in flight together
            const int b = lane * each + k;
            const bool in = k < each && b < nb;
            s0[k] = make_ulonglong2(0, 0);
            if (KIND == kFirst) s1[KIND == kFirst ? k : 0] = make_ulonglong2(0, 0);
            e[k] = R;
            if (in) {
                s0[k] = __ldcg(from + 2 * b);
                if (KIND == kFirst) s1[KIND == kFirst ? k : 0] = __ldcg(from + 2 * b + 1);
                if (KIND == kLeaf) e[k] = __ldcg(a.exps + b);
            }
        }
        if constexpr (KIND == kFirst) {
            uint64_t sp = 0, sq = 0;
#pragma unroll
            for (int k = 0; k < kEach; ++k) {
                sp += s0[k].x;
                sq += s0[k].y;
            }
            sp = warp_sum64(sp);
            sq = warp_sum64(sq);
            split_quotient(sp, sq, fm, fe);  // c = 1
            if (lane == 0) {
                S.sum_p = sp;
                S.sum_q = sq;
                S.c = 1.0;
                S.c_f = 1.f;
                S.fm = fm;
                S.fe = fe;
            }
        }
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            if constexpr (KIND == kFirst) {
                const uint64_t q = sum_times_f(s1[k].y, fm, fe);
                x[k] = s1[k].x > q ? s1[k].x - q : 0;
            } else {
                x[k] = s0[k].x;
            }
        }
        if constexpr (KIND == kLeaf) {
#pragma unroll
            for (int k = 0; k < kEach; ++k) R = max(R, e[k]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) R = max(R, __shfl_xor_sync(0xffffffffu, R, o));
        }
        uint64_t mine = 0;
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            if constexpr (KIND == kLeaf) x[k] = shifted(x[k], R - e[k]);
            mine += x[k];
        }
        uint64_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint64_t v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        const uint64_t total = __shfl_sync(0xffffffffu, incl, 31);
        const uint64_t r = fraction_of(u, total);
        if (lane == 0) {
            S.exp = R;
            S.owner = R >= kBad ? -2 : -1;
            if constexpr (KIND != kLeaf) {
                S.total = total;
                S.left_f = static_cast<float>(total) / static_cast<float>(S.sum_p);
            }
        }
        __syncwarp();
        uint64_t before = incl - mine;
        if (R < kBad && r >= before && r < incl) {
#pragma unroll
            for (int k = 0; k < kEach; ++k) {
                if (r >= before && r - before < x[k]) {
                    S.owner = lane * each + k;
                    S.before = r - before;  // the point within the block's share
                    break;
                }
                before += x[k];
            }
        }
    }
    __syncthreads();
}

// The token at point r of this block's weights w(k), k = 0..n-1 (the last one
// with a weight, should r lie behind them).
template <typename W>
__device__ __forceinline__ int find_token(Shared& S, const Span& P, uint64_t r, W&& w) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint64_t mine = 0;
    for (int k = P.first; k < P.last; ++k) mine += w(k);
    uint64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) S.warp[0][warp] = incl;
    if (threadIdx.x == 0) S.found = P.v0;
    __syncthreads();
    uint64_t start = incl - mine, total = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        if (i == warp) start += total;
        total += S.warp[0][i];
    }
    if (r >= total) r = total ? total - 1 : 0;
    if (r >= start && r - start < mine) {
        uint64_t t = start;
        for (int k = P.first; k < P.last; ++k) {
            t += w(k);
            if (t > r) {
                S.found = P.v0 + k;
                break;
            }
        }
    }
    __syncthreads();
    return S.found;
}

// f(k, the logit) for this thread's tokens, in order, four loads at a time.
template <typename F>
__device__ __forceinline__ void each_logit(const Span& P, const float* row, F&& f) {
    for (int k = P.first; k < P.last; k += 4) {
        float x[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) x[u] = k + u < P.last ? __ldcg(row + P.v0 + k + u) : 0.f;
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (k + u < P.last) f(k + u, x[u]);
    }
}

// A row's weights relative to the block's own largest exponent, 0 for the
// tokens of the nodes in `removed`: to w, their sum and the exponent published.
// The removed tokens have no part in that exponent: the others' weights would
// lose as many bits as such a token is more likely than they are.
__device__ __forceinline__ void leaf_pass(const VerifyArgs& a, Shared& S, const Span& P, const float* row, uint32_t removed,
                                          uint64_t* w, float* logit, unsigned barriers) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    float mx = -INFINITY;
    bool bad = false;
    uint32_t mine = 0;  // of `removed`, those whose token is this thread's
    for (uint32_t r = removed; r; r &= r - 1) {
        const int k = S.token[__ffs(r) - 1] - P.v0;
        if (k >= P.first && k < P.last) mine |= r & -r;
    }
    each_logit(P, row, [&](int k, float x) {
        bad |= !(x < INFINITY);
        for (uint32_t r = mine; r; r &= r - 1)
            if (S.token[__ffs(r) - 1] == P.v0 + k) x = -INFINITY;
        mx = fmaxf(mx, x);
        logit[k] = x;
    });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (lane == 0) S.warp_max[warp] = mx;
    bad = __syncthreads_or(bad);
#pragma unroll
    for (int i = 0; i < kWarps; ++i) mx = fmaxf(mx, S.warp_max[i]);
    const float t = ceilf(mx * a.c_hi + 0.01f);
    const bool some = t >= -kMaxExponent && t <= kMaxExponent;
    const int R = some ? static_cast<int>(t) : -(1 << 23);
    uint64_t v[1] = {0};
    for (int k = P.first; k < P.last; ++k) {
        v[0] += w[k] = some ? weight(logit[k], a.c_hi, a.c_lo, R, S.table) : 0;
    }
    if (tid == 0) __stcg(a.exps + blockIdx.x, bad || t > kMaxExponent ? kBad : R);
    publish(a, S, v, barriers);
}

// One row and nothing drafted: the last block to finish its slice finds the
// token, on the owner's slice anew.
__global__ void __launch_bounds__(kThreads, 1) verify_sample_kernel(const __grid_constant__ VerifyArgs a) {
    __shared__ Shared S;
    extern __shared__ uint64_t held[];  // [span] weights, [span] logits
    const int tid = threadIdx.x;
    for (int j = tid; j < kVerifyTable; j += kThreads) S.table[j] = a.table[j];
    pdl_launch_dependents();
    pdl_wait();  // no global access before this
    __syncthreads();
    leaf_pass(a, S, Span(a, blockIdx.x), a.target, 0u, held, reinterpret_cast<float*>(held + a.span), 0);
    __syncthreads();
    if (tid == 0) S.flag = atom_add_acq_rel_gpu(a.sync, 1u) == gridDim.x - 1;
    __syncthreads();
    if (!S.flag) return;
    settle<kLeaf>(a, S, 0);
    int token = -1;
    if (S.owner >= 0) {
        const Span P(a, S.owner);
        const int R = __ldcg(a.exps + S.owner);
        each_logit(P, a.target, [&](int k, float x) { held[k] = weight(x, a.c_hi, a.c_lo, R, S.table); });
        token = find_token(S, P, S.before << (S.exp - R), [&](int k) { return held[k]; });
    }
    if (tid == 0) {
        a.result[0] = 1;
        a.result[1] = token;
        a.result[2] = 0;
        a.sync[0] = 0;
    }
}

// CLUSTER: the grid is one cluster.
template <bool CLUSTER>
__global__ void __launch_bounds__(kThreads, 1) verify_kernel(const __grid_constant__ VerifyArgs a) {
    __shared__ Shared S;
    extern __shared__ uint64_t held[];  // [span] target weights, [span] draft weights
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Span P(a, blockIdx.x);
    uint64_t* wp = held;
    uint64_t* wq = held + a.span;
    for (int j = tid; j < kVerifyTable; j += kThreads) S.table[j] = a.table[j];
    if (tid < MUSER_MAX_M) S.near[tid] = 0;
    pdl_wait();  // no global access before this
    unsigned barriers = 0;
    bool ok = true, any_near = false;
    int row, lo, hi;
    if (my_unit(a, row, lo, hi)) {
        float sum = 0.f, R = -kMaxExponent;
        for_slice(row_ptr(a, row), lo, hi, a.vec, [&](float4 v, int) {
            const float t = fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)) * a.c_hi;
            if (t > R) {
                const float Rn = ceilf(t);
                sum *= ex2(R - Rn);
                R = Rn;
            }
            sum += (ex2(fmaf(v.x, a.c_hi, -R)) + ex2(fmaf(v.y, a.c_hi, -R))) +
                   (ex2(fmaf(v.z, a.c_hi, -R)) + ex2(fmaf(v.w, a.c_hi, -R)));
        });
        float Rm = R;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) Rm = fmaxf(Rm, __shfl_xor_sync(0xffffffffu, Rm, o));
        sum = warp_sum(sum * ex2(R - Rm));  // a NaN or +infinity leaves a NaN here
        if (lane == 0) __stcg(a.part + row * kMaxSlices + lo / a.slice_len, make_float2(sum, Rm));
    }
    // the drafted tokens' logits, in flight during the barrier
    float lx = -INFINITY, ly = -INFINITY;
    if (tid >= 1 && tid < a.M) {
        const int x = __ldcg(a.tokens + tid), up = a.parent[tid];
        S.token[tid] = x;
        S.u[tid] = __ldcg(a.uniform + tid);
        if (x >= 0 && x < a.V) {
            lx = __ldcg(row_ptr(a, a.target_at[up]) + x);
            if (a.draft) ly = __ldcg(row_ptr(a, a.draft_at[up]) + x);
        }
    }
    ok = grid_barrier<CLUSTER>(a, ++barriers, &S.flag);
    // every block: the rows' sums and the drafted tokens' probabilities
    float2 x[2][kMaxSlices / 32];  // a warp has two rows at most: their loads go out together
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int r = warp + j * kWarps;
#pragma unroll
        for (int k = 0; k < kMaxSlices / 32; ++k)
            x[j][k] = r < a.nrows && lane + 32 * k < a.slices ? __ldcg(a.part + r * kMaxSlices + lane + 32 * k)
                                                              : make_float2(0.f, -kMaxExponent);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        float R = -kMaxExponent, sum = 0.f;
#pragma unroll
        for (int k = 0; k < kMaxSlices / 32; ++k) R = fmaxf(R, x[j][k].y);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) R = fmaxf(R, __shfl_xor_sync(0xffffffffu, R, o));
#pragma unroll
        for (int k = 0; k < kMaxSlices / 32; ++k) sum = fmaf(x[j][k].x, ex2(x[j][k].y - R), sum);
        sum = warp_sum(sum);
        if (lane == 0 && warp + j * kWarps < a.nrows) {
            S.row_sum[warp + j * kWarps] = sum > 0.f && R <= kMaxExponent ? sum : NAN;
            S.row_exp[warp + j * kWarps] = R;
        }
    }
    __syncthreads();
    if (warp == 0) {  // lane i: node i's probabilities, and whether it is accepted if it is its parent's first child
        bool first = false, fine = true;
        if (lane >= 1 && lane < a.M) {
            const int up = a.parent[lane], tr = a.target_at[up], dr = a.draft_at[up];
            const float p = ex2(fmaf(lx, a.c_hi, -S.row_exp[tr])) / S.row_sum[tr];
            const float q = a.draft ? ex2(fmaf(ly, a.c_hi, -S.row_exp[dr])) / S.row_sum[dr] : 1.f;
            S.px[lane] = p;
            S.qx[lane] = q;
            first = S.u[lane] * q < p;
            fine = S.row_sum[tr] == S.row_sum[tr] && (!a.draft || S.row_sum[dr] == S.row_sum[dr]);
        }
        const uint32_t f = __ballot_sync(0xffffffffu, first), g = __ballot_sync(0xffffffffu, fine);
        // The walk as long as first children are accepted: one warp's, a shuffle
        // a step (in all 16 warps a step took 270 cycles).
        const uint32_t mine = lane < a.M ? a.children[lane] : 0u;
        const int child = __ffs(mine) - 1, next = mine != 0 && ((f & g) >> child) & 1u ? child : -1;
        int cur = 0, n = 1;
        uint32_t kept = 1u;
        for (int i; (i = __shfl_sync(0xffffffffu, next, cur)) >= 0; cur = i, ++n) kept |= 1u << i;
        if (lane == 0) {
            S.first = f;
            S.fine = g;
            S.cur = cur;
            S.n = n;
            S.kept = kept;
        }
    }
    __syncthreads();

    // The walk: the same in every thread of every block.  Binary64 is thread
    // 0's alone: one division by all 512 threads holds an SM for 3 us.
    int cur = S.cur, n = S.n;
    uint32_t kept = S.kept, removed = 0u;
    const uint32_t first = S.first, fine = S.fine;
    bool valid = true, rejected = false;  // rejected: the node's weights are held, S describes its remainder
    float left = 1.f, c = 0.f, rest = -1.f;
    auto remainder = [&](int k) {  // max(P - f Q, 0)
        const uint64_t fq = S.fm ? times_f(wq[k], S.fm, S.fe) : 0;
        return wp[k] > fq ? wp[k] - fq : 0;
    };
    auto remainder_pass = [&]() {
        uint64_t v[1] = {0};
        for (int k = P.first; k < P.last; ++k) v[0] += remainder(k);
        publish(a, S, v, ++barriers);
        ok = grid_barrier<CLUSTER>(a, barriers, &S.flag);
        if (ok) settle<kNext>(a, S, barriers);
    };
    // Drafts that are certain: what is left of a row without the rejected tokens,
    // as a sum of the others, every block the same one.  As 1 - p it would be a
    // rounding error where p is nearly 1.  A node's sum over the tokens that are
    // no child's is made once: the slices without such a token are summed
    // already, the others are read anew.
    auto rest_of = [&](int row, uint32_t kids) {
        const float R = S.row_exp[row];
        const float* p = row_ptr(a, row);
        __syncthreads();  // the last call's sums have been read
        if (warp == 0) {
            const bool mine = lane < a.M && ((kids >> lane) & 1u) && S.token[lane] >= 0 && S.token[lane] < a.V;
            const int slice = mine ? S.token[lane] / a.slice_len : -1 - lane;
            const uint32_t same = __match_any_sync(0xffffffffu, slice);  // of every lane
            const bool lead = mine && (same & ((1u << lane) - 1u)) == 0;
            const uint32_t leads = __ballot_sync(0xffffffffu, lead);
            if (lead) {
                S.slice[__popc(leads & ((1u << lane) - 1u))] = slice;
                S.slice_kids[__popc(leads & ((1u << lane) - 1u))] = same;
            }
            if (lane == 0) S.slices = __popc(leads);
        }
        __syncthreads();
        float sum = 0.f;
        if (tid < a.slices) {
            bool whole = true;
            for (int i = 0; i < S.slices; ++i) whole = whole && S.slice[i] != tid;
            if (whole) {
                const float2 w = __ldcg(a.part + row * kMaxSlices + tid);
                sum = w.x * ex2(w.y - R);
            }
        }
        const int slices = S.slices, len = a.slice_len;
        constexpr int kBatch = 8;  // loads in flight together
        for (int k0 = tid; k0 < slices * len; k0 += kBatch * kThreads) {
            float x[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int k = k0 + u * kThreads, i = k / len;
                const int v = i < slices ? (S.slice[i] - i) * len + k : a.V;
                x[u] = v < a.V ? __ldcg(p + v) : -INFINITY;
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int k = k0 + u * kThreads, i = k / len;
                for (uint32_t e = i < slices ? S.slice_kids[i] : 0u; e; e &= e - 1)
                    if (S.token[__ffs(e) - 1] == (S.slice[i] - i) * len + k) x[u] = -INFINITY;
                sum += ex2(fmaf(x[u], a.c_hi, -R));
            }
        }
        sum = warp_sum(sum);
        if (lane == 0) S.warp_left[warp] = sum;
        __syncthreads();
        sum = 0.f;
        for (int w = 0; w < kWarps; ++w) sum += S.warp_left[w];
        return sum / S.row_sum[row];
    };
    uint32_t alike = 0;  // the node's children with this lane's child's token
    uint32_t children = a.children[cur];  // of the present node, not tried yet
    while (children && ok) {
        const int i = __ffs(children) - 1;
        valid = (fine >> i) & 1u;
        if (!valid) break;
        bool taken = (first >> i) & 1u, again = false;
        if (rejected || removed) {  // not a first child
            // a token that was certain, and rejected, has nothing left
            for (uint32_t r = removed; r; r &= r - 1) again = again || S.token[__ffs(r) - 1] == S.token[i];
            const float p = S.px[i], q = S.qx[i];
            taken = !again && S.u[i] * left * q < p - c * q;
        }
        if (taken) {
            cur = i;
            children = a.children[i];
            kept |= 1u << i;
            ++n;
            removed = 0;
            c = 0.f;
            left = 1.f;
            rest = -1.f;
            rejected = false;
            continue;
        }
        children &= children - 1;
        if (!a.draft) {
            removed |= 1u << i;
            if (children && !again) {  // a difference is as good as a sum while more than half of the row is left
                left -= S.px[i];
                if (left < 0.5f) {
                    const uint32_t kids = a.children[cur];
                    const bool child = lane < a.M && ((kids >> lane) & 1u);
                    if (rest < 0.f) {
                        rest = rest_of(a.target_at[cur], kids);
                        alike = __match_any_sync(0xffffffffu, child ? S.token[lane] : static_cast<int>(0x80000000u) + lane) & kids;
                    }
                    // and the probabilities of the other children's tokens, each once
                    left = rest + warp_sum(child && !(alike & removed) && !(alike & ((1u << lane) - 1u)) ? S.px[lane] : 0.f);
                }
            }
            continue;
        }
        const int tr = a.target_at[cur], dr = a.draft_at[cur];
        bool pass = rejected;
        if (!rejected) {  // the node's weights, to shared memory
            const int Rp = static_cast<int>(S.row_exp[tr]) + 1, Rq = static_cast<int>(S.row_exp[dr]) + 1;
            uint64_t fm, v[4] = {0, 0, 0, 0};
            unsigned near = 0;  // in units of 2^kNearUnit, upwards
            int fe;
            split_factor(S.row_sum[tr] / S.row_sum[dr], fm, fe);
            const float* pr = row_ptr(a, tr) + P.v0;
            const float* qr = row_ptr(a, dr) + P.v0;
            for (int k = P.first; k < P.last; k += 4) {  // eight loads in flight together
                float x[4], y[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[j] = k + j < P.last ? __ldcg(pr + k + j) : -INFINITY;
                    y[j] = k + j < P.last ? __ldcg(qr + k + j) : -INFINITY;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (k + j >= P.last) break;
                    const uint64_t w = weight(x[j], a.c_hi, a.c_lo, Rp, S.table), z = weight(y[j], a.c_hi, a.c_lo, Rq, S.table);
                    wp[k + j] = w;
                    wq[k + j] = z;
                    v[0] += w;
                    v[1] += z;
                    const uint64_t fz = times_f(z, fm, fe);
                    if (w > fz) {
                        v[2] += w;
                        v[3] += z;
                    }
                    // (below 2^20 units what such a token is off by is less than one)
                    if ((w > fz ? w - fz : fz - w) <= (fz >> 20) && z != 0) near += min(static_cast<unsigned>(z >> kNearUnit) + 1, kNearMost);
                }
            }
            if (__any_sync(0xffffffffu, near != 0)) {
                near = __reduce_add_sync(0xffffffffu, near);
                if (lane == 0) atomicAdd(&S.near[cur], near);
            }
            publish(a, S, v, ++barriers);
            if (tid == 0 && S.near[cur] != 0) atomicAdd(a.near + cur, min(S.near[cur], kNearMost));
            ok = grid_barrier<CLUSTER>(a, barriers, &S.flag);
            if (!ok) break;
            if (tid == 32) S.near_all = __ldcg(a.near + cur);  // beside warp 0
            settle<kFirst>(a, S, barriers);
            rejected = true;
            const uint64_t apart = S.fe == fe ? (S.fm > fm ? S.fm - fm : fm - S.fm)
                                 : fe == S.fe + 1 ? fm - (S.fm >> 1) : S.fe == fe + 1 ? S.fm - (fm >> 1) : ~0ull;
            const int one = S.fe == fe ? 63 : 62;  // |f - f0| / f = apart / 2^one at most
            pass = apart >> (one - 20) != 0;
            if (S.near_all != 0) {
                any_near = true;
                // the same times near / sum Q, each as a power of 2 not below it, then as it is
                const bool all = S.near_all >= kNearMost;
                const int bound = 64 - __clzll(static_cast<long long>(apart)) - one +
                                  (all ? 0 : 32 - __clz(static_cast<int>(S.near_all)) + kNearUnit - 63 + __clzll(static_cast<long long>(S.sum_q)));
                const int most = min(-38, -20 + (__float_as_int(S.left_f) >> 23) - 127);
                if (bound > most) {
                    const float off = static_cast<float>(apart) * __int_as_float((127 - one) << 23);
                    const float share = all ? 1.f : static_cast<float>(S.near_all) * (1 << kNearUnit) / static_cast<float>(S.sum_q);
                    pass = pass || off * share > fminf(0x1p-38f, 0x1p-20f * S.left_f);
                }
            }
        } else {
            __syncthreads();  // every thread has read the last remainder's c
            if (tid == 0) {
                S.c += static_cast<double>(S.total) / static_cast<double>(S.sum_p);
                S.c_f = static_cast<float>(S.c);
                split_factor(S.c * (static_cast<double>(S.sum_p) / static_cast<double>(S.sum_q)), S.fm, S.fe);
            }
            __syncthreads();
        }
        if (pass) {
            remainder_pass();
            if (!ok) break;
        }
        left = S.left_f;
        c = S.c_f;
    }

    // The next token.
    int token = -1;
    bool owner = blockIdx.x == 0;  // who writes it
    if (ok && valid) {
        if (rejected && S.owner == -1) {  // nothing is left of the target's row: the row itself
            __syncthreads();
            if (tid == 0) S.fm = 0;
            __syncthreads();
            remainder_pass();
        }
        // without rejections: weights relative to the block's own largest exponent
        const float* row = a.target + static_cast<int64_t>(cur) * a.V;
        for (int again = 0; !rejected && again < 2 && ok; ++again) {
            leaf_pass(a, S, P, row, removed, wp, reinterpret_cast<float*>(wq), ++barriers);
            ok = grid_barrier<CLUSTER>(a, barriers, &S.flag);
            if (!ok) break;
            settle<kLeaf>(a, S, barriers);
            if (S.owner != -1 || removed == 0) break;
            removed = 0;  // nothing is left: the row itself
            ok = grid_barrier<CLUSTER>(a, ++barriers, &S.flag);  // before exps are written again
        }
        if (ok && S.owner >= 0) {
            owner = S.owner == static_cast<int>(blockIdx.x);
            if (owner) {
                if (rejected) token = find_token(S, P, S.before, remainder);
                else token = find_token(S, P, S.before << (S.exp - __ldcg(a.exps + blockIdx.x)), [&](int k) { return wp[k]; });
            }
        }
    }
    if (ok && owner && tid == 0) a.result[1] = token;
    if (ok && blockIdx.x == 0 && tid == 0) {
        a.result[0] = n;
        int at = 2;
        for (int i = 0; i < a.M; ++i)
            if ((kept >> i) & 1u) a.result[at++] = i;
        for (; at < a.M + 2; ++at) a.result[at] = -1;
    }
    if constexpr (CLUSTER) {
        if (any_near) {  // in every block or in none
            ok = grid_barrier<CLUSTER>(a, ++barriers, &S.flag);  // all have read
            if (blockIdx.x == 0 && tid < MUSER_MAX_M) a.near[tid] = 0;
        }
        return;
    }
    // the last block to leave zeroes the counters for the next call
    __syncthreads();
    if (tid == 0 && atom_add_acq_rel_gpu(a.sync + 1, 1u) == gridDim.x - 1) {
        a.sync[0] = 0;
        a.sync[1] = 0;
        for (int i = 0; i < MUSER_MAX_M / 4; ++i) reinterpret_cast<uint4*>(a.near)[i] = make_uint4(0, 0, 0, 0);
    }
}

struct Scratch {
    size_t part, sums, exps, bytes;
};
constexpr Scratch layout() {
    Scratch s{};
    s.part = 256;
    s.sums = s.part + kRows * kMaxSlices * 8;
    s.exps = s.sums + 8 * kMaxBlocks * 8;
    s.bytes = s.exps + kMaxBlocks * 4;
    return s;
}

const uint64_t* weight_table() {
    static uint64_t table[kVerifyTable];
    static std::once_flag once;
    std::call_once(once, [] {
        for (int j = 0; j < kVerifyTable; ++j)
            table[j] = static_cast<uint64_t>(std::exp2(static_cast<double>(j) / kVerifyTable) * static_cast<double>(1ull << kFrac) + 0.5);
    });
    return table;
}

// The sampling kernels' attributes.  A block holds 16 bytes a token of its
// span, which is 1,024 tokens (a cluster's: 2,500) or a share of the vocabulary
// among all blocks.
const int* verify_ready() {
    return device_once<0, int>([](int& most) {
        const int blocks = std::min(sm_count(), kMaxBlocks);
        if (blocks < 1) return set_error(MUSER_ERR_CUDA, "tree_verify: cannot read the SM count");
        most = static_cast<int>(std::max<int64_t>((kVerifyMaxVocab + blocks - 1) / blocks, 1024) * 16);
        cudaError_t e = cudaFuncSetAttribute(verify_sample_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(verify_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(verify_kernel<true>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        return e == cudaSuccess ? static_cast<int>(MUSER_OK) : cuda_fail(e, "tree_verify: cudaFuncSetAttribute");
    });
}
static_assert((kClusterVocab + kClusterBlocks - 1) / kClusterBlocks * 16 + sizeof(Shared) <= 48 * 1024,
              "a cluster's blocks need no attribute for their shared memory");

}  // namespace

size_t verify_scratch_bytes() { return layout().bytes; }

int launch_verify(const float* target, const float* draft, const int32_t* tokens, const int32_t* parent, int M,
                  int64_t vocab, double temperature, const float* uniform, int32_t* result, void* scratch,
                  cudaStream_t s) {
    VerifyArgs a{};
    const bool greedy = temperature == 0.0;
    a.target = target;
    a.draft = greedy ? nullptr : draft;
    a.tokens = tokens;
    a.uniform = uniform;
    a.result = result;
    a.M = M;
    a.V = static_cast<int>(vocab);
    const double c = greedy ? 1.0 : 1.4426950408889634074 / temperature;
    a.c_hi = static_cast<float>(c);
    a.c_lo = static_cast<float>(c - static_cast<double>(a.c_hi));
    a.vec = vocab % 4 == 0;  // the matrices are 16-byte aligned
    bool inner[MUSER_MAX_M] = {};
    for (int i = 0; i < M; ++i) {
        a.parent[i] = i == 0 ? -1 : (parent ? parent[i] : i - 1);
        if (i > 0) {
            inner[a.parent[i]] = true;
            a.children[a.parent[i]] |= 1u << i;
        }
        a.target_at[i] = a.draft_at[i] = -1;
    }
    for (int i = 0; i < M; ++i)
        if (greedy || inner[i]) a.row_node[a.target_at[i] = a.nrows++] = i;
    a.ntarget = a.nrows;
    for (int i = 0; i < M && a.draft; ++i)
        if (inner[i]) a.row_node[a.draft_at[i] = a.nrows++] = i;
    // Few tokens: one cluster, whose barriers outweigh the other SMs.  Measured
    // in a graph, 15 drafts in a binary tree: 10,000 tokens 10.9 us in a cluster,
    // 14.0 on the grid; 32,768 14.4 and 15.1; 65,536 18.2 and 13.7.  A chain of
    // 15, whose first pass reads twice the rows: 20,000 tokens 12.7 and 13.1,
    // 32,768 13.7 and 12.6.  Outside a graph the cooperative launch adds to the
    // grid's: the chain of 15, 32,768 tokens 13.5 and 14.6, 39,999 17.3 and 15.2.
    const bool cluster = !greedy && M > 1 && vocab <= kClusterVocab && a.nrows * vocab <= kClusterLogits;
    const int sms = cluster ? kClusterBlocks : std::min(sm_count(), kMaxBlocks);
    if (sms < 1) return set_error(MUSER_ERR_CUDA, "tree_verify: cannot read the SM count");
    // The first pass gives every warp of the device one slice of a row, of 512
    // logits at least; the passes over one node give a block 1,024 tokens at
    // least (fewer blocks meet faster at a barrier).
    int blocks = greedy ? 1 : static_cast<int>(std::min<int64_t>(sms, (vocab + 1023) / 1024));
    if (a.nrows > 0) {
        const int64_t most = std::max<int64_t>(1, std::min<int64_t>(sms * kWarps / a.nrows, (vocab + 511) / 512));
        a.slices = static_cast<int>(std::min<int64_t>(most, kMaxSlices));
        a.slice_len = static_cast<int>(((vocab + a.slices - 1) / a.slices + 3) / 4 * 4);
        a.slices = static_cast<int>((vocab + a.slice_len - 1) / a.slice_len);
        blocks = std::max(blocks, std::min(sms, a.nrows * a.slices));
    }
    if (cluster) blocks = kClusterBlocks;
    a.span = static_cast<int>((vocab + blocks - 1) / blocks);
    const Scratch L = layout();
    uint8_t* p = static_cast<uint8_t*>(scratch);
    a.sync = reinterpret_cast<unsigned*>(p);
    a.near = reinterpret_cast<unsigned*>(p + 128);  // of the 256 bytes that are left zero
    a.part = reinterpret_cast<float2*>(p + L.part);
    a.sums = reinterpret_cast<uint64_t*>(p + L.sums);
    a.exps = reinterpret_cast<int*>(p + L.exps);
    a.status = device_status_word();
    if (!a.status) return set_error(MUSER_ERR_CUDA, "tree_verify: no device status word");
    std::copy(weight_table(), weight_table() + kVerifyTable, a.table);
    const size_t smem = static_cast<size_t>(a.span) * 16u;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = greedy ? 0 : smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    if (cluster) {
        cfg.gridDim.x = kClusterBlocks;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = kClusterBlocks;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    } else {
        attr[1].id = cudaLaunchAttributeCooperative;  // every block resident at once (grid barriers)
        attr[1].val.cooperative = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = greedy || M == 1 ? 1 : 2;
    auto kern = greedy ? verify_greedy_kernel : M == 1 ? verify_sample_kernel : cluster ? verify_kernel<true> : verify_kernel<false>;
    if (!greedy && verify_ready() == nullptr) return MUSER_ERR_CUDA;  // the message is set
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a);
    if (e != cudaSuccess) return cuda_fail(e, "tree_verify: cudaLaunchKernelEx");
    return check_launch("tree_verify");
}

}  // namespace muser
