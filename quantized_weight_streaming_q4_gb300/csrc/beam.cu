// beam.cu -- one step of beam search: log-probabilities, their sum with the
// beams' scores, and the largest n of a request's beams and tokens.
//
// One launch and one pass over the logits.  A row is cut into parts, one a
// block, which stay in registers: the sum of 2^(x log2(e) - E) with an integer
// E, in fixed point, and the part's n largest logits, in order (within a row
// the sum orders as the logit).  The last block of a request to finish joins
// them: the rows' log-sums (the parts' sums are shifted, exactly), and the n
// largest of beams * parts * n sums, of which only the parts whose largest is
// among the requests' largest are looked at further.
//
// Bound: latency, the logits being 1.9 us (16 beams of 202,048 tokens: 12.3 us:
// 2.3 until they are there, 1.1 for the sum, 3 for the part's largest, 0.7 for
// the ticket, 4 for the last block's work; 37 with binary64 sums).
// Two blocks an SM leave 64 registers a thread, of which 148 bytes spill; with
// one block, 123 registers and no spill the same takes 15.3 us, and 4 x 4 beams of
// 32,768 tokens 13.8 instead of 11.4.
// Binary64 is slow here and is left to a few operations a row: the sums
// score + x - log-sum are pairs of binary32 numbers (48 bits), compared as 64-bit
// keys.
//
// The n largest of many values: the values are dealt to 64 groups; the n-th
// largest of the groups' maxima is at most the n-th largest value, and few
// values are above it (of 10,000 random ones about 20 for n = 16).  These go to
// a list, where each counts how many come before it.  The last block's groups
// are of the parts' largest alone, dealt so that every group has some of them.
// Where these are fewer than n, the beams' scores far apart, or some groups
// empty (less than 2,048 logits), many values are above: what the list took of
// them is dealt to the groups again, for a closer bound.  Where the list would not
// take them even so (thousands of equal logits), the values are taken one by
// one, n times over (16 beams of 202,048 equal logits: 203 us; untied ones 12.3).
#include <algorithm>

#include "kernels.cuh"
#include "pages.cuh"

namespace muser {
namespace {

constexpr int kThreads = 512, kVec = 8, kPerThread = 4 * kVec;
constexpr int kMost = kThreads * kPerThread - 4;  // logits of a part; up to 3 elements before it share its first 16 bytes
constexpr int kGroups = 64, kGroupLanes = kThreads / kGroups, kList = 2048;
// Entries that are ranked as they are (n = 64 leaves about 270 of random values),
// and those that are ranked where a closer bound leaves more.  The ranking is
// quadratic: a call of 1,500 logits, n = 64, is 24 us narrowed, 262 with all of
// them ranked; of 1,500 equal ones, n = 4, 221 us ranked and 18 one by one.
constexpr int kShort = 512, kRanked = 1024;
constexpr float kNegInf = -INFINITY;
// log2(e) to 48 bits
constexpr float kLog2e = 1.44269502162933349609375f, kLog2eLow = 1.92596299112661746887e-8f;
constexpr float kFixed = 0x1p40f;     // a sum of 2^20 terms below 2 is below 2^61
constexpr float kMostLogit = 0x1p20f;  // beyond it binary32 leaves too little of a logit's fraction

struct Stat {
    float e;       // E, or NaN: no sum
    float pad;
    uint64_t sum;  // times 2^40
};
struct Cand {
    float x;
    int32_t index;  // the token
};

// Ordered as the numbers: a larger value has a larger key, and no key is 0
// but that of NaN, which counts as none.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);  // -0 as 0
    return x != x ? 0u : (b & 0x80000000u ? ~b : b | 0x80000000u);
}
__device__ __forceinline__ float from_key(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); }

// The key of a pair plus x, to 48 bits; 0 for -infinity and NaN.
__device__ __forceinline__ uint64_t sum_key(float2 base, float x) {
    const float s = base.x + x, t = s - base.x;
    const float err = (base.x - (s - t)) + (x - t) + base.y;  // what the first sum lost
    const float hi = s + err;
    if (!(hi > kNegInf)) return s > kNegInf ? static_cast<uint64_t>(key_of(s)) << 32 : 0;  // s may be +infinity: no low part
    return static_cast<uint64_t>(key_of(hi)) << 32 | key_of(err - (hi - s));
}

template <typename K>
struct Pick {
    K group[kGroups];      // the groups' maxima
    K list_key[kList];
    int32_t list_at[kList];
    K red_key[kThreads / 32];
    int32_t red_at[kThreads / 32];
    K floor;
    int32_t count;
};

// The n-th largest of the 64 groups' maxima (n <= 64); `top` is the thread's.
// A group's eight lanes compare its maximum with eight others each.
template <typename K>
__device__ __forceinline__ K floor_of(Pick<K>& S, int n, K top) {
    const int tid = threadIdx.x, g = tid / kGroupLanes;
    static_assert(kGroupLanes == 8 && kGroups == 64, "eight by eight");
#pragma unroll
    for (int o = 1; o < kGroupLanes; o <<= 1) {
        const K x = __shfl_xor_sync(0xffffffffu, top, o);
        top = x > top ? x : top;
    }
    if (tid % kGroupLanes == 0) S.group[g] = top;
    if (tid == 0) S.count = 0;
    __syncthreads();
    int before = 0;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        const int j = tid % kGroupLanes + 8 * u;
        before += (S.group[j] > top || (S.group[j] == top && j < g)) ? 1 : 0;
    }
#pragma unroll
    for (int o = 1; o < kGroupLanes; o <<= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
    if (before == n - 1) S.floor = top;
    __syncthreads();
    return S.floor;
}

template <typename K>
__device__ __forceinline__ void append(Pick<K>& S, K k, int at) {
    const int i = atomicAdd(&S.count, 1);
    if (i < kList) {
        S.list_key[i] = k;
        S.list_at[i] = at;
    }
}

// Puts the keys that are not below `least` on the list, as far as it takes
// them, and returns their number: each thread calls each(f), which calls
// f(key, at) for its values, key 0 for none.
template <typename K, typename Each>
__device__ __forceinline__ int collect(Pick<K>& S, K least, Each&& each) {
    each([&](K k, int at) {
        if (k != 0 && k >= least) append(S, k, at);
    });
    __syncthreads();
    return S.count;
}

// A list of more than kShort entries is cut down to those that are not below
// the bound that its own entries give; of a list that did not take all `count`
// of them this is only the bound, and the list is empty.
template <typename K>
__device__ __noinline__ int narrow(Pick<K>& S, int n, int count, K& least) {
    constexpr int kEach = kList / kThreads;
    const int tid = threadIdx.x;
    K k[kEach], top = 0;
    int at[kEach];
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
        const int i = tid + u * kThreads;
        k[u] = i < count ? S.list_key[i] : 0;
        at[u] = i < count ? S.list_at[i] : 0;
        top = k[u] > top ? k[u] : top;
    }
    __syncthreads();  // the count and the list have been read
    least = floor_of(S, n, top);
    if (count > kList) return count;
#pragma unroll
    for (int u = 0; u < kEach; ++u)
        if (k[u] != 0 && k[u] >= least) append(S, k[u], at[u]);
    __syncthreads();
    return S.count;
}

// The n largest keys (ties: the lower `at`) among what all threads hold, of
// which collect() found `count`.  put(rank, key, at) is called for rank
// 0..found-1, in some order; returns found.
template <typename K, typename Each, typename Put>
__device__ __forceinline__ int largest(Pick<K>& S, int n, int count, Each&& each, Put&& put) {
    const int tid = threadIdx.x;
    if (count <= kRanked) {
        for (int i = tid / 8; i < (count + 3) / 4 * 4; i += kThreads / 8) {  // eight lanes a value; whole warps
            const K k = i < count ? S.list_key[i] : 0;
            const int at = i < count ? S.list_at[i] : 0;
            int rank = 0;
            for (int j = tid % 8; j < count; j += 8) rank += (S.list_key[j] > k || (S.list_key[j] == k && S.list_at[j] < at)) ? 1 : 0;
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) rank += __shfl_xor_sync(0xffffffffu, rank, o);
            if (i < count && rank < n && tid % 8 == 0) put(rank, k, at);
        }
        return min(count, n);
    }
    // one after another: the first behind the last one taken
    K last = ~K{0};
    int last_at = -1;
    for (int rank = 0; rank < n; ++rank) {
        K best = 0;
        int best_at = 0x7fffffff;
        auto join = [&](K k, int at) {
            if (k > best || (k == best && at < best_at)) best = k, best_at = at;
        };
        each([&](K k, int at) {
            if (k != 0 && (k < last || (k == last && at > last_at))) join(k, at);
        });
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) join(__shfl_xor_sync(0xffffffffu, best, o), __shfl_xor_sync(0xffffffffu, best_at, o));
        if ((tid & 31) == 0) {
            S.red_key[tid >> 5] = best;
            S.red_at[tid >> 5] = best_at;
        }
        __syncthreads();
        for (int w = 0; w < kThreads / 32; ++w) join(S.red_key[w], S.red_at[w]);
        __syncthreads();
        if (best == 0) return rank;
        if (tid == 0) put(rank, best, best_at);
        last = best;
        last_at = best_at;
    }
    return n;
}

// Parts of a request: a beam's are at most 65 (2^20 tokens) or a share of 304.
constexpr int kHeads = 5, kMostLists = kHeads * kThreads;
static_assert(kBeamMaxBeams * ((kBeamMaxVocab + kMost - 1) / kMost) <= kMostLists && 304 <= kMostLists, "a request's parts");

struct BeamShared {
    union {
        Pick<uint32_t> part;
        Pick<uint64_t> all;
    };
    float2 base[kBeamMaxBeams];  // score - log-sum, as a pair
    float e[kBeamMaxBeams];      // the rows' largest E, and their sums
    uint64_t total[kBeamMaxBeams];
    int32_t ended[kBeamMaxBeams];
    uint16_t open[kMostLists];   // parts that may hold one of the n largest
    int32_t opened;
    float red_max[kThreads / 32];
    uint64_t red_sum[kThreads / 32];
    int32_t last;
};

__global__ void __launch_bounds__(kThreads, 2) beam_select_kernel(const __grid_constant__ BeamArgs a) {
    __shared__ BeamShared S;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int part = blockIdx.x, row = blockIdx.y, g = row / a.beams;
    Stat* const stat = static_cast<Stat*>(a.stat);
    Cand* const cand = static_cast<Cand*>(a.cand);
    pdl_launch_dependents();
    pdl_wait();
    const bool ended = a.ended && __ldcg(a.ended + row) != 0;
    Cand* const mine = cand + (static_cast<int64_t>(row) * a.parts + part) * a.n;
    const int v0 = static_cast<int>(static_cast<int64_t>(a.vocab) * part / a.parts);
    const int len = static_cast<int>(static_cast<int64_t>(a.vocab) * (part + 1) / a.parts) - v0;
    const float* p = a.logits + static_cast<int64_t>(row) * a.vocab + v0;
    const int off = static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15u) / 4u);
    p -= off;  // 16-byte aligned; element i of the part is p[off + i]
    float x[kPerThread];
#pragma unroll
    for (int u = 0; u < kVec; ++u) {
        const int i = 4 * (tid + u * kThreads) - off;
        if (i >= 0 && i + 4 <= len) {
            const float4 v = __ldcs(reinterpret_cast<const float4*>(p + off + i));
            x[4 * u] = v.x, x[4 * u + 1] = v.y, x[4 * u + 2] = v.z, x[4 * u + 3] = v.w;
        } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) x[4 * u + c] = i + c >= 0 && i + c < len ? __ldcs(p + off + i + c) : kNegInf;
        }
    }
    if (ended) {  // one way on, with probability 1
        if (tid < a.n) mine[tid] = Cand{part == 0 && tid == 0 ? 0.f : kNegInf, a.end_token};
        if (tid == 0) stat[row * a.parts + part] = Stat{0.f, 0.f, 1};
    } else {
        float m = kNegInf;
#pragma unroll
        for (int u = 0; u < kPerThread; ++u) m = fmaxf(m, x[u]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (lane == 0) S.red_max[warp] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) m = fmaxf(m, S.red_max[w]);
        // a part that is all below -2^20 (masked) adds nothing to a row that is not
        const bool some = m >= -kMostLogit;
        const float e = some && m <= kMostLogit ? floorf(m * kLog2e) : 0.f;
        float s = 0.f;
#pragma unroll
        for (int u = 0; u < kPerThread; ++u) s += exp2f(fmaf(x[u], kLog2eLow, fmaf(x[u], kLog2e, -e)));
        // NaN, or infinite: the row has no sum
        const bool bad = __syncthreads_or(!(s < INFINITY) || m > kMostLogit);
        if (!some) s = 0.f;
        uint64_t sum = bad ? 0 : __float2ull_rn(s * kFixed);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) S.red_sum[warp] = sum;
        float top = kNegInf;
#pragma unroll
        for (int u = 0; u < kPerThread; ++u) top = fmaxf(top, x[u]);
        const uint32_t least = floor_of(S.part, a.n, top == kNegInf ? 0u : key_of(top));
        if (tid < 32) {  // the warps' sums
            uint64_t total = lane < kThreads / 32 ? S.red_sum[lane] : 0;
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
            if (lane == 0) stat[row * a.parts + part] = Stat{bad ? NAN : e, 0.f, total};
        }
        const auto each = [&](auto&& f) {
            if (key_of(top) < least) return;  // most threads have none
#pragma unroll
            for (int u = 0; u < kPerThread; ++u)
                f(x[u] == kNegInf ? 0u : key_of(x[u]), 4 * (tid + u / 4 * kThreads) - off + u % 4);
        };
        int count = collect(S.part, least, each);
        if (count > kShort && count <= kList) {
            uint32_t closer;
            count = narrow(S.part, a.n, count, closer);
        }
        const int found = largest(S.part, a.n, count, each,
                                  [&](int rank, uint32_t k, int at) { mine[rank] = Cand{from_key(k), v0 + at}; });
        if (tid >= found && tid < a.n) mine[tid] = Cand{kNegInf, 0};
    }
    // the request's last block goes on
    __syncthreads();
    if (tid == 0) {
        const unsigned blocks = static_cast<unsigned>(a.beams * a.parts);
        S.last = atom_add_acq_rel_gpu(a.ticket + g, 1u) == blocks - 1u;
        if (S.last) a.ticket[g] = 0;
    }
    __syncthreads();
    if (!S.last) return;
    // the parts' largest, flags and scores, on the way while the rows' sums are made
    const int lists = a.beams * a.parts;
    const Cand* all = cand + static_cast<int64_t>(g) * lists * a.n;
    float head[kHeads];
    const int l0 = (threadIdx.x * kGroups | threadIdx.x / kGroupLanes) % kThreads;  // neighbours go to different groups
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
        const int l = l0 + i * kThreads;
        head[i] = l < lists ? __ldcg(&all[l * a.n].x) : kNegInf;
    }
    const int r = g * a.beams + tid;  // a beam a thread
    const bool end = tid < a.beams && a.ended && __ldcg(a.ended + r) != 0;
    const float score = tid < a.beams ? __ldcg(a.score + r) : 0.f;
    if (tid == 0) S.opened = 0;
    for (int b = warp; b < a.beams; b += kThreads / 32) {
        const Stat* st = stat + (g * a.beams + b) * a.parts;
        // the lane's first part stays in registers; beyond 32 the others are read twice
        auto read = [&](int i) {
            const uint4 w = __ldcg(reinterpret_cast<const uint4*>(st + i));
            return Stat{__uint_as_float(w.x), 0.f, static_cast<uint64_t>(w.w) << 32 | w.z};
        };
        const Stat mine = lane < a.parts ? read(lane) : Stat{0.f, 0.f, 0};
        float e = mine.sum != 0 ? mine.e : kNegInf;
        bool bad = mine.e != mine.e;
        for (int i = lane + 32; i < a.parts; i += 32) {
            const Stat p = read(i);
            bad = bad || p.e != p.e;
            if (p.sum != 0) e = fmaxf(e, p.e);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) e = fmaxf(e, __shfl_xor_sync(0xffffffffu, e, o));
        uint64_t s = 0;
        for (int i = lane; i < a.parts; i += 32) {
            const Stat p = i == lane ? mine : read(i);
            const float behind = e - p.e;
            if (behind < 64.f) s += p.sum >> static_cast<int>(fmaxf(behind, 0.f));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        bad = __any_sync(0xffffffffu, bad);
        if (lane == 0) {
            S.e[b] = bad ? NAN : e;
            S.total[b] = s;
        }
    }
    __syncthreads();
    if (tid < a.beams) {
        // ln(total 2^(e - 40)): the leading bit's place, and the logarithm of what follows it
        const uint64_t t = S.total[tid];
        const int place = 63 - __clzll(static_cast<long long>(t | 1));
        const float fraction = log2f(static_cast<float>(t << (63 - place)) * 0x1p-63f);
        double sum = score;
        if (!end) sum -= (static_cast<double>(S.e[tid] + static_cast<float>(place - 40)) + fraction) * 0.693147180559945309417;
        if (!end && t == 0) sum = NAN;
        const float hi = static_cast<float>(sum);
        S.base[tid] = make_float2(hi, fabsf(hi) < INFINITY ? static_cast<float>(sum - hi) : 0.f);
        S.ended[tid] = end;
    }
    __syncthreads();
    uint64_t key[kHeads], top = 0;
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
        key[i] = head[i] == kNegInf ? 0 : sum_key(S.base[(l0 + i * kThreads) / a.parts], head[i]);
        top = key[i] > top ? key[i] : top;
    }
    const uint64_t least = floor_of(S.all, a.n, top);
#pragma unroll
    for (int i = 0; i < kHeads; ++i)
        if (key[i] != 0 && key[i] >= least) S.open[atomicAdd(&S.opened, 1)] = static_cast<uint16_t>(l0 + i * kThreads);
    __syncthreads();
    const int out = g * a.n;
    const unsigned opened = S.opened, total = opened * a.n;
    // part by part, or, of many, the parts' largest first, then their second largest, ...
    const bool many = total > kShort;
    const unsigned inner = many ? opened : a.n;
    const auto each = [&](auto&& f) {
        for (unsigned e = tid; e < total; e += kThreads) {
            const unsigned y = e / inner, z = e - y * inner;
            const int l = S.open[many ? z : y], b = l / a.parts;
            const float2 c = __ldcg(reinterpret_cast<const float2*>(all + l * a.n + (many ? y : z)));
            f(c.x == kNegInf ? 0 : sum_key(S.base[b], c.x), b * a.vocab + __float_as_int(c.y));
        }
    };
    int count = collect(S.all, least, each);
    for (int round = 0; count > kShort && round < 2; ++round) {
        uint64_t closer;
        const int all_of_them = count;
        count = narrow(S.all, a.n, count, closer);
        if (all_of_them > kList) count = collect(S.all, closer, each);
    }
    const int found = largest(
        S.all, a.n, count, each,
        [&](int rank, uint64_t k, int at) {
            const int b = at / a.vocab, v = at - b * a.vocab;
            const bool end = S.ended[b] || v == a.end_token;
            a.parent[out + rank] = g * a.beams + b;
            a.token[out + rank] = v;
            a.score_out[out + rank] = from_key(static_cast<uint32_t>(k >> 32));
            if (a.ended_out) a.ended_out[out + rank] = end;
            if (a.add) a.add[out + rank] = !end;
        });
    for (int i = found + tid; i < a.n; i += kThreads) {
        a.parent[out + i] = -1;
        a.token[out + i] = -1;
        a.score_out[out + i] = kNegInf;
        if (a.ended_out) a.ended_out[out + i] = 1;
        if (a.add) a.add[out + i] = 0;
    }
}

// Parts of a row: two blocks an SM, at least 2,048 logits each.
int parts_of(int rows, int64_t vocab) {
    const int64_t least = (vocab + kMost - 1) / kMost, most = (vocab + 2047) / 2048;
    return static_cast<int>(std::max(least, std::min<int64_t>(most, std::max(1, 304 / rows))));
}
constexpr size_t kTicketBytes = 1024;
static_assert(kTicketBytes >= kMaxSequences * sizeof(unsigned), "a ticket a request");

}  // namespace

size_t beam_scratch_bytes(int groups, int beams, int64_t vocab, int n) {
    const size_t parts = static_cast<size_t>(groups) * beams * parts_of(groups * beams, vocab);
    return kTicketBytes + parts * sizeof(Stat) + (parts * n * sizeof(Cand) + 15u) / 16u * 16u;
}

int launch_beam_select(BeamArgs a, void* scratch, cudaStream_t s) {
    const int rows = a.groups * a.beams;
    a.parts = parts_of(rows, a.vocab);
    uint8_t* p = static_cast<uint8_t*>(scratch);
    a.ticket = reinterpret_cast<unsigned*>(p);
    a.stat = p + kTicketBytes;
    a.cand = p + kTicketBytes + static_cast<size_t>(rows) * a.parts * sizeof(Stat);
    return launch_after("beam selection", beam_select_kernel, dim3(static_cast<unsigned>(a.parts), static_cast<unsigned>(rows)),
                        kThreads, 0, 1, s, a);
}

}  // namespace muser
