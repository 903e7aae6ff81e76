// verify.cu -- verification of drafted (tree) tokens against the target's
// probabilities from given random numbers, and the token that follows.
//
// One cooperative launch.  All blocks first stream the logits once: per row
// the sum of 2^(l * log2(e) / T) (or, at temperature 0, the first maximum).
// After a grid barrier every block walks the tree by itself, from the same
// numbers, so all take the same path; only where a child is rejected, or at
// the end, do they pass over one pair of rows together, each over its own
// slice of the vocabulary.
//
// Weights are integers.  With R an integer >= the row's largest exponent, a
// token's weight is round(2^(l log2(e) / T - R) * 2^42): sums of integers do
// not depend on their order, so the sampled token is the same whatever the
// grid, and a token is decided by comparing integers.  The exponential is
// good to about 2^-38: a binary32 one (2^-23) would move some of the 2e5
// borders of the cumulative sums by enough to pick a neighbour about once in a
// thousand draws.  FP64 has no rate to speak of on GB300, so none of the
// per-token work uses it; it is kept for a few scalars per row.
#include <algorithm>
#include <cmath>

#include "kernels.cuh"

namespace muser {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kFrac = 42;             // fraction bits of a weight
constexpr int kRows = 2 * MUSER_MAX_M;  // target rows, then draft rows
constexpr int kTable = 128;
constexpr int kMaxParts = 256;        // blocks that can share one row
constexpr float kMaxExponent = 32768.f;
constexpr int kBadRow = 1 << 24;      // exponent mark of a row that holds a NaN or an infinity
constexpr uint64_t kGridWaitNs = 2000000000ull;

struct VerifyArgs {
    const float* target;   // [M][V]
    const float* draft;    // [M][V] or null
    const int32_t* tokens; // [M]
    const float* uniform;  // [M]
    int32_t* result;       // [M + 2]
    int M, V;
    float c_hi, c_lo;      // log2(e) / T
    int greedy, vec;       // vec: rows are 16-byte aligned
    int parent[MUSER_MAX_M];
    int nrows;             // rows that are read: target rows 0..M-1, then the draft rows listed
    int draft_row[MUSER_MAX_M];  // node whose draft row is row M + i
    int draft_at[MUSER_MAX_M];   // row index of node i's draft row, or -1
    int64_t per_block;     // logits per block of the first pass, a multiple of 4
    int slice;             // tokens per block of the walk's passes
    unsigned* sync;        // arrivals, exits
    uint64_t* part_sum;    // [kRows][kMaxParts]
    int* part_exp;         // [kRows][kMaxParts]
    uint64_t* pass_sum;    // [2][kMaxParts]: the walk's passes, two buffers in turn
    unsigned* status;
};

__device__ __forceinline__ const float* row_ptr(const VerifyArgs& a, int row) {
    return row < a.M ? a.target + static_cast<int64_t>(row) * a.V
                     : a.draft + static_cast<int64_t>(a.draft_row[row - a.M]) * a.V;
}

// 2^(j / 128) * 2^kFrac, j = 0..127, filled once per block in binary64.
__device__ void fill_table(uint64_t* table) {
    for (int j = threadIdx.x; j < kTable; j += blockDim.x)
        table[j] = static_cast<uint64_t>(exp2(static_cast<double>(j) / kTable) * static_cast<double>(1ull << kFrac) + 0.5);
}

// round(2^(l * c - R) * 2^kFrac) for an integer R >= l * c; 0 where that is
// below 2^-20 of the last bit and for l = -inf.  l * c = n + j / 128 + r with
// r held as two floats, y = r ln 2 likewise (|y| < 2^-8), and 2^r - 1 = y +
// y^2/2 + y^3/6 + y^4/24 to 2^-46; that sum is turned into units of 2^-39 by
// adding numbers whose last bit has the wanted weight, in two parts.
__device__ __forceinline__ uint64_t weight(float l, float c_hi, float c_lo, int R, const uint64_t* table) {
    const float h = l * c_hi;
    const float e = fmaf(l, c_lo, fmaf(l, c_hi, -h));
    const float nj = rintf(h * static_cast<float>(kTable));
    const float r0 = fmaf(-1.f / kTable, nj, h);  // exact: h - nj / 128
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
    const uint64_t t = table[i & (kTable - 1)];
    // t * (1 + g 2^-39): t >> 11 has 32 bits
    const int64_t prod = static_cast<int64_t>(static_cast<uint32_t>(t >> 11)) * static_cast<int64_t>(g);
    const uint64_t w = t + static_cast<uint64_t>(prod >> (39 - 11));
    const int down = R - (i >> 7);
    if (!(h > static_cast<float>(R) - 62.f)) return 0;
    return down > 0 ? (w + (1ull << (down - 1))) >> down : w;
}

// Thread-level running sum of weights with its own reference exponent.
struct Running {
    uint64_t sum;
    int R;
};
__device__ __forceinline__ uint64_t shifted(uint64_t s, int by) { return by < 64 ? s >> by : 0; }
__device__ __forceinline__ Running join(Running a, Running b) {
    const int R = max(a.R, b.R);
    return {shifted(a.sum, R - a.R) + shifted(b.sum, R - b.R), R};
}

// Every block has arrived `times` times.  False if it gave up waiting.
__device__ bool grid_barrier(const VerifyArgs& a, unsigned times, int* flag) {
    __syncthreads();
    if (threadIdx.x == 0) {
        atom_add_acq_rel_gpu(a.sync, 1u);
        const unsigned want = gridDim.x * times;
        const uint64_t t0 = global_ns();
        int ok = 1;
        for (;;) {
            unsigned v;
            asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(a.sync) : "memory");
            if (v >= want) break;
            if (global_ns() - t0 > kGridWaitNs) {
                atomicOr(a.status, kDevStatusWaitTimeout);
                ok = 0;
                break;
            }
        }
        *flag = ok;
    }
    __syncthreads();
    return *flag != 0;
}

struct Shared {
    uint64_t table[kTable];
    uint64_t warp_sum[kWarps];
    int warp_exp[kWarps];
    float warp_max[kWarps];
    int warp_arg[kWarps];
    uint64_t row_sum[kRows];  // weights' sum of a row, with its exponent
    int row_exp[kRows];
    double px[MUSER_MAX_M], qx[MUSER_MAX_M], u[MUSER_MAX_M];  // of node i: p(x_i), q(x_i) in its parent's rows
    int token[MUSER_MAX_M], arg[MUSER_MAX_M];
    uint64_t total;
    uint64_t blocks[kMaxParts];
    int flag;
    int found;
};

__device__ __forceinline__ uint64_t warp_sum64(uint64_t v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// ------------------------------------------------- first pass over all rows
// Block b streams logits [b * per_block, (b + 1) * per_block) of the rows laid
// end to end and leaves one partial per row it touches.
__device__ int first_block(const VerifyArgs& a, int row) {
    return static_cast<int>(static_cast<int64_t>(row) * a.V / a.per_block);
}
__device__ int last_block(const VerifyArgs& a, int row) {
    return static_cast<int>((static_cast<int64_t>(row + 1) * a.V - 1) / a.per_block);
}

template <bool GREEDY>
__device__ void stream_rows(const VerifyArgs& a, Shared& S) {
    const int64_t all = static_cast<int64_t>(a.nrows) * a.V;
    const int64_t b0 = blockIdx.x * a.per_block, b1 = min(b0 + a.per_block, all);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int64_t at = b0; at < b1;) {
        const int row = static_cast<int>(at / a.V);
        const int64_t base = static_cast<int64_t>(row) * a.V;
        const int lo = static_cast<int>(at - base), hi = static_cast<int>(min(b1 - base, static_cast<int64_t>(a.V)));
        const float* p = row_ptr(a, row);
        Running run{0, -(1 << 23)};
        float best = -INFINITY;
        int arg = 0x7fffffff, bad = 0;
        auto take4 = [&](const float (&x)[4], int n, int i) {
            if constexpr (GREEDY) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (k < n) {
                        bad |= !(x[k] < INFINITY);
                        if (x[k] > best) {
                            best = x[k];
                            arg = i + k;
                        }
                    }
            } else {
                float mx = -INFINITY;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (k < n) {
                        bad |= !(x[k] < INFINITY);
                        mx = fmaxf(mx, x[k]);
                    }
                const float t = ceilf(mx * a.c_hi + 0.01f);
                bad |= t > kMaxExponent;
                if (t >= -kMaxExponent && t <= kMaxExponent) {
                    const int R = static_cast<int>(t);
                    if (R > run.R) {
                        run.sum = shifted(run.sum, R - run.R);
                        run.R = R;
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (k < n) run.sum += weight(x[k], a.c_hi, a.c_lo, run.R, S.table);
                }
            }
        };
        if (a.vec && (lo & 3) == 0) {
            const int n4 = (hi - lo) >> 2;
            const float4* p4 = reinterpret_cast<const float4*>(p + lo);
#pragma unroll 4
            for (int i = threadIdx.x; i < n4; i += kThreads) {
                const float4 v = __ldcg(p4 + i);
                const float x[4] = {v.x, v.y, v.z, v.w};
                take4(x, 4, lo + 4 * i);
            }
            for (int i = lo + 4 * n4 + threadIdx.x; i < hi; i += kThreads) {
                const float x[4] = {__ldcg(p + i), 0.f, 0.f, 0.f};
                take4(x, 1, i);
            }
        } else {
            for (int i = lo + threadIdx.x; i < hi; i += kThreads) {
                const float x[4] = {__ldcg(p + i), 0.f, 0.f, 0.f};
                take4(x, 1, i);
            }
        }
        bad = __syncthreads_or(bad);
        const int slot = row * kMaxParts + static_cast<int>(blockIdx.x) - first_block(a, row);
        if constexpr (GREEDY) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const float ob = __shfl_xor_sync(0xffffffffu, best, o);
                const int oa = __shfl_xor_sync(0xffffffffu, arg, o);
                if (ob > best || (ob == best && oa < arg)) {
                    best = ob;
                    arg = oa;
                }
            }
            if (lane == 0) {
                S.warp_max[warp] = best;
                S.warp_arg[warp] = arg;
            }
            __syncthreads();
            if (threadIdx.x == 0) {
                for (int w = 1; w < kWarps; ++w)
                    if (S.warp_max[w] > best || (S.warp_max[w] == best && S.warp_arg[w] < arg)) {
                        best = S.warp_max[w];
                        arg = S.warp_arg[w];
                    }
                a.part_sum[slot] = (static_cast<uint64_t>(__float_as_uint(best)) << 32) | static_cast<uint32_t>(arg);
                a.part_exp[slot] = bad ? kBadRow : 0;
            }
        } else {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const Running other{__shfl_xor_sync(0xffffffffu, run.sum, o), __shfl_xor_sync(0xffffffffu, run.R, o)};
                run = join(run, other);
            }
            if (lane == 0) {
                S.warp_sum[warp] = run.sum;
                S.warp_exp[warp] = run.R;
            }
            __syncthreads();
            if (threadIdx.x == 0) {
                for (int w = 1; w < kWarps; ++w) run = join(run, Running{S.warp_sum[w], S.warp_exp[w]});
                a.part_sum[slot] = run.sum;
                a.part_exp[slot] = bad ? kBadRow : run.R;
            }
        }
        __syncthreads();
        at = base + hi;
    }
}

// ---------------------------------------------------- passes over one node
// w(v) = max(P(v) - f Q(v), 0) with P, Q the weights of the node's target and
// draft rows; without a draft row P(v), but 0 for the removed tokens.  f =
// fm * 2^fe with fm in [2^63, 2^64), or no Q at all (fm = 0).
struct Pass {
    int row, draft;   // row indexes; draft < 0: none
    uint64_t fm;
    int fe;
    uint32_t removed; // nodes whose tokens are removed (no draft row)
};

__device__ __forceinline__ uint64_t pass_weight(const VerifyArgs& a, const Shared& S, const Pass& P, int v) {
    uint64_t w = weight(__ldcg(row_ptr(a, P.row) + v), a.c_hi, a.c_lo, S.row_exp[P.row], S.table);
    if (P.fm) {
        // f Q = (Q 2^19) fm 2^-64 * 2^(fe + 45): Q 2^19 < 2^62
        const uint64_t q = weight(__ldcg(row_ptr(a, P.draft) + v), a.c_hi, a.c_lo, S.row_exp[P.draft], S.table);
        const uint64_t t = __umul64hi(q << 19, P.fm);
        const int sh = P.fe + 64 - 19;
        uint64_t fq;
        if (sh <= 0) fq = shifted(t, -sh);
        else fq = sh >= __clzll(static_cast<long long>(t)) ? ~0ull >> 1 : t << sh;
        if (t == 0) fq = 0;
        w = w > fq ? w - fq : 0;
    }
    for (uint32_t left = P.removed; left; left &= left - 1)
        if (S.token[__ffs(left) - 1] == v) w = 0;
    return w;
}

// This thread's part of the block's slice: tokens [v0, v1), in order.
__device__ __forceinline__ void my_tokens(const VerifyArgs& a, int& v0, int& v1) {
    const int s0 = static_cast<int>(blockIdx.x) * a.slice, s1 = min(s0 + a.slice, a.V);
    const int per = (a.slice + kThreads - 1) / kThreads;
    v0 = min(s0 + static_cast<int>(threadIdx.x) * per, s1);
    v1 = min(v0 + per, s1);
}

__device__ uint64_t thread_sum(const VerifyArgs& a, const Shared& S, const Pass& P) {
    int v0, v1;
    my_tokens(a, v0, v1);
    uint64_t sum = 0;
    for (int v = v0; v < v1; ++v) sum += pass_weight(a, S, P, v);
    return sum;
}

// The pass of all blocks: leaves every block's sum in S.blocks and the total
// in S.total; `mine` is this thread's sum.  False if a barrier gave up.
__device__ bool pass(const VerifyArgs& a, Shared& S, const Pass& P, unsigned& barriers, uint64_t& mine) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint64_t* sums = a.pass_sum + (barriers & 1) * kMaxParts;
    mine = thread_sum(a, S, P);
    const uint64_t w = warp_sum64(mine);
    if (lane == 0) S.warp_sum[warp] = w;
    __syncthreads();
    if (threadIdx.x == 0) {
        uint64_t t = 0;
        for (int i = 0; i < kWarps; ++i) t += S.warp_sum[i];
        __stcg(reinterpret_cast<unsigned long long*>(sums + blockIdx.x), static_cast<unsigned long long>(t));
    }
    if (!grid_barrier(a, ++barriers, &S.flag)) return false;
    for (int b = threadIdx.x; b < static_cast<int>(gridDim.x); b += kThreads)
        S.blocks[b] = __ldcg(reinterpret_cast<const unsigned long long*>(sums + b));
    __syncthreads();
    if (warp == 0) {
        uint64_t t = 0;
        for (int b = lane; b < static_cast<int>(gridDim.x); b += 32) t += S.blocks[b];
        t = warp_sum64(t);
        if (lane == 0) S.total = t;
    }
    __syncthreads();
    return true;
}

// floor(u * total) for a float u in [0, 1).
__device__ uint64_t fraction_of(float u, uint64_t total) {
    if (!(u > 0.f)) return 0;
    u = fminf(u, 0x1.fffffep-1f);
    const int e = (__float_as_int(u) >> 23) & 0xff;  // u = mant * 2^(e - 150)
    const uint64_t mant = e ? ((__float_as_int(u) & 0x7fffff) | 0x800000) : (__float_as_int(u) & 0x7fffff);
    const int down = 150 - (e ? e : 1);              // 25.. for u < 1: at least 24
    const uint64_t lo = mant * total, hi = __umul64hi(mant, total);
    if (down >= 128) return 0;
    return down >= 64 ? hi >> (down - 64) : (lo >> down) | (hi << (64 - down));
}

template <bool GREEDY>
__global__ void __launch_bounds__(kThreads) verify_kernel(const __grid_constant__ VerifyArgs a) {
    __shared__ Shared S;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    fill_table(S.table);
    __syncthreads();
    stream_rows<GREEDY>(a, S);
    unsigned barriers = 1;
    bool ok = grid_barrier(a, barriers, &S.flag);
    if (ok) {
        // every block: the rows' sums (or maxima) and the drafted tokens' probabilities
        for (int row = warp; row < a.nrows; row += kWarps) {
            const int n = last_block(a, row) - first_block(a, row) + 1;
            if constexpr (GREEDY) {
                float best = -INFINITY;
                int arg = 0x7fffffff, bad = 0;
                for (int i = lane; i < n; i += 32) {
                    const uint64_t v = __ldcg(reinterpret_cast<const unsigned long long*>(a.part_sum + row * kMaxParts + i));
                    bad |= __ldcg(a.part_exp + row * kMaxParts + i);
                    const float f = __uint_as_float(static_cast<uint32_t>(v >> 32));
                    const int x = static_cast<int>(v & 0xffffffffu);
                    if (f > best || (f == best && x < arg)) {
                        best = f;
                        arg = x;
                    }
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    const float ob = __shfl_xor_sync(0xffffffffu, best, o);
                    const int oa = __shfl_xor_sync(0xffffffffu, arg, o);
                    bad |= __shfl_xor_sync(0xffffffffu, bad, o);
                    if (ob > best || (ob == best && oa < arg)) {
                        best = ob;
                        arg = oa;
                    }
                }
                if (lane == 0) S.arg[row] = bad || arg == 0x7fffffff ? -1 : arg;
            } else {
                Running run{0, -(1 << 23)};
                int bad = 0;
                for (int i = lane; i < n; i += 32) {
                    const Running o{__ldcg(reinterpret_cast<const unsigned long long*>(a.part_sum + row * kMaxParts + i)),
                                    __ldcg(a.part_exp + row * kMaxParts + i)};
                    bad |= o.R == kBadRow;
                    run = join(run, o);
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    const Running other{__shfl_xor_sync(0xffffffffu, run.sum, o), __shfl_xor_sync(0xffffffffu, run.R, o)};
                    bad |= __shfl_xor_sync(0xffffffffu, bad, o);
                    run = join(run, other);
                }
                if (lane == 0) {
                    S.row_sum[row] = bad ? 0 : run.sum;
                    S.row_exp[row] = run.R;
                }
            }
        }
        if (tid >= 1 && tid < a.M) S.token[tid] = __ldg(a.tokens + tid);
        __syncthreads();
        if constexpr (!GREEDY) {
            if (tid < a.M) {
                S.u[tid] = static_cast<double>(__ldg(a.uniform + tid));
                const int x = tid ? S.token[tid] : -1;
                double p = 0.0, q = 0.0;
                if (x >= 0 && x < a.V) {
                    const int up = a.parent[tid], dr = a.draft ? a.draft_at[up] : -1;
                    if (S.row_sum[up])
                        p = static_cast<double>(weight(__ldcg(row_ptr(a, up) + x), a.c_hi, a.c_lo, S.row_exp[up], S.table)) /
                            static_cast<double>(S.row_sum[up]);
                    if (dr >= 0 && S.row_sum[dr])
                        q = static_cast<double>(weight(__ldcg(row_ptr(a, dr) + x), a.c_hi, a.c_lo, S.row_exp[dr], S.table)) /
                            static_cast<double>(S.row_sum[dr]);
                }
                S.px[tid] = p;
                S.qx[tid] = q;
            }
            __syncthreads();
        }

        // the walk: the same in every thread of every block
        int cur = 0, n = 1, next = -1;
        uint32_t kept = 1u;
        if constexpr (GREEDY) {
            for (int i = 1; i < a.M; ++i)
                if (a.parent[i] == cur && S.arg[cur] >= 0 && S.token[i] == S.arg[cur]) {
                    cur = i;
                    kept |= 1u << i;
                    ++n;
                }
            next = S.arg[cur];
        } else {
            double c = 0.0, left = 1.0;
            uint64_t mine = 0;
            bool passed = false;  // S.blocks, S.total and mine are those of this node's present state
            Pass P{0, -1, 0, 0, 0u};
            auto at_node = [&](int i) {
                cur = i;
                c = 0.0;
                left = 1.0;
                passed = false;
                P = Pass{i, a.draft ? a.draft_at[i] : -1, 0, 0, 0u};
            };
            at_node(0);
            bool valid = S.row_sum[0] != 0;
            for (int i = 1; i < a.M && valid && ok; ++i) {
                if (a.parent[i] != cur) continue;
                if (P.draft >= 0 && S.row_sum[P.draft] == 0) {
                    valid = false;
                    break;
                }
                if (P.draft >= 0) {
                    if (S.u[i] * left * S.qx[i] < S.px[i] - c * S.qx[i]) {
                        at_node(i);
                        kept |= 1u << i;
                        ++n;
                        valid = S.row_sum[i] != 0;
                        continue;
                    }
                    c += left;
                    const double f = c * (static_cast<double>(S.row_sum[P.row]) / static_cast<double>(S.row_sum[P.draft]));
                    const long long bits = __double_as_longlong(f);
                    P.fm = (static_cast<uint64_t>(bits & 0xfffffffffffffll) | 0x10000000000000ull) << 11;
                    P.fe = static_cast<int>((bits >> 52) & 0x7ff) - 1023 - 63;
                    ok = pass(a, S, P, barriers, mine);
                    passed = true;
                    left = static_cast<double>(S.total) / static_cast<double>(S.row_sum[P.row]);
                } else {
                    bool again = false;  // the token of a rejected sibling has nothing left
                    for (uint32_t r = P.removed; r; r &= r - 1) again = again || S.token[__ffs(r) - 1] == S.token[i];
                    if (!again && S.u[i] * left < S.px[i]) {
                        at_node(i);
                        kept |= 1u << i;
                        ++n;
                        valid = S.row_sum[i] != 0;
                        continue;
                    }
                    if (!again) left -= S.px[i];
                    P.removed |= 1u << i;
                }
            }
            if (ok && valid && !passed) ok = pass(a, S, P, barriers, mine);
            if (ok && valid && S.total == 0) {  // nothing is left of the target's row: the row itself
                P.fm = 0;
                P.removed = 0;
                ok = pass(a, S, P, barriers, mine);
            }
            if (ok && valid) {
                // the block that holds the token finds it; the others are done
                const uint64_t r = fraction_of(__ldg(a.uniform), S.total);
                uint64_t before = 0;
                int owner = 0;
                for (int b = 0; b < static_cast<int>(gridDim.x); ++b) {
                    if (before + S.blocks[b] > r) {
                        owner = b;
                        break;
                    }
                    before += S.blocks[b];
                }
                if (owner == static_cast<int>(blockIdx.x)) {
                    uint64_t incl = mine;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const uint64_t v = __shfl_up_sync(0xffffffffu, incl, o);
                        if (lane >= o) incl += v;
                    }
                    if (lane == 31) S.warp_sum[warp] = incl;
                    __syncthreads();
                    uint64_t start = before + incl - mine;
                    for (int w = 0; w < warp; ++w) start += S.warp_sum[w];
                    if (r >= start && r < start + mine) {
                        int v0, v1;
                        my_tokens(a, v0, v1);
                        uint64_t t = start;
                        for (int v = v0; v < v1; ++v) {
                            t += pass_weight(a, S, P, v);
                            if (t > r) {
                                S.found = v;
                                break;
                            }
                        }
                    }
                    __syncthreads();
                    next = S.found;
                    if (tid == 0) a.result[1] = next;
                }
            } else if (ok && blockIdx.x == 0 && tid == 0) {
                a.result[1] = -1;
            }
        }
        if (blockIdx.x == 0 && tid == 0 && ok) {
            a.result[0] = n;
            if constexpr (GREEDY) a.result[1] = next;
            int at = 0;
            for (int i = 0; i < a.M; ++i)
                if ((kept >> i) & 1u) a.result[2 + at++] = i;
            for (; at < a.M; ++at) a.result[2 + at] = -1;
        }
    }
    // the last block to leave zeroes the counters for the next call
    __syncthreads();
    if (tid == 0) {
        const unsigned left = atom_add_acq_rel_gpu(a.sync + 1, 1u);
        if (left == gridDim.x - 1) {
            a.sync[0] = 0;
            a.sync[1] = 0;
        }
    }
}

}  // namespace

size_t verify_scratch_bytes() {
    return 256 + static_cast<size_t>(kRows) * kMaxParts * (sizeof(uint64_t) + sizeof(int)) + 2 * kMaxParts * sizeof(uint64_t);
}

int launch_verify(const float* target, const float* draft, const int32_t* tokens, const int32_t* parent, int M,
                  int64_t vocab, double temperature, const float* uniform, int32_t* result, void* scratch,
                  cudaStream_t s) {
    VerifyArgs a{};
    a.greedy = temperature == 0.0;
    a.target = target;
    a.draft = a.greedy ? nullptr : draft;
    a.tokens = tokens;
    a.uniform = uniform;
    a.result = result;
    a.M = M;
    a.V = static_cast<int>(vocab);
    const double c = a.greedy ? 1.0 : 1.4426950408889634074 / temperature;
    a.c_hi = static_cast<float>(c);
    a.c_lo = static_cast<float>(c - static_cast<double>(a.c_hi));
    a.vec = vocab % 4 == 0 && is_aligned(target, 16) && (!a.draft || is_aligned(draft, 16));
    a.nrows = M;
    for (int i = 0; i < M; ++i) {
        a.parent[i] = i == 0 ? -1 : (parent ? parent[i] : i - 1);
        a.draft_at[i] = -1;
    }
    for (int i = 0; i < M && a.draft; ++i) {
        bool inner = false;
        for (int j = 1; j < M; ++j) inner = inner || a.parent[j] == i;
        if (!inner) continue;
        a.draft_row[a.nrows - M] = i;
        a.draft_at[i] = a.nrows++;
    }
    const int sms = sm_count();
    if (sms < 1) return set_error(MUSER_ERR_CUDA, "tree_verify: cannot read the SM count");
    const int64_t all = static_cast<int64_t>(a.nrows) * vocab;
    // at least 2,048 logits per block, one block per SM at most
    const int64_t blocks = std::max<int64_t>(1, std::min<int64_t>(std::min(sms, kMaxParts), all / 2048));
    a.per_block = ((all + blocks - 1) / blocks + 3) / 4 * 4;
    a.slice = static_cast<int>((vocab + blocks - 1) / blocks);
    uint8_t* p = static_cast<uint8_t*>(scratch);
    a.sync = reinterpret_cast<unsigned*>(p);
    a.part_sum = reinterpret_cast<uint64_t*>(p + 256);
    a.pass_sum = a.part_sum + kRows * kMaxParts;
    a.part_exp = reinterpret_cast<int*>(a.pass_sum + 2 * kMaxParts);
    a.status = device_status_word();
    if (!a.status) return set_error(MUSER_ERR_CUDA, "tree_verify: no device status word");
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;  // every block resident at once (grid barriers)
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = a.greedy ? cudaLaunchKernelEx(&cfg, verify_kernel<true>, a)
                                   : cudaLaunchKernelEx(&cfg, verify_kernel<false>, a);
    if (e != cudaSuccess) return cuda_fail(e, "tree_verify: cudaLaunchKernelEx");
    return check_launch("tree_verify");
}

}  // namespace muser
