// attn.cuh -- what the tree-attention kernels share: the call's arguments as
// the host lays them out, and the exact treatment of the rows whose
// visibility differs between query rows.
#pragma once

#include <cuda.h>  // CUtensorMap (types only)

#include "common.cuh"

namespace muser {

// A run of consecutive cache slots, read as rows of head_dim binary16 values:
// row r of K/V head g starts at k + g * head_stride + r * row_stride (the same
// for v).  Token-major planes have row_stride = kv_dim and head_stride =
// head_dim; head-major ones row_stride = head_dim and head_stride = capacity *
// head_dim.
struct AttnSeg {
    const uint16_t* k;
    const uint16_t* v;
    int64_t row_stride, head_stride;
    int32_t rows;
};
constexpr int kAttnMaxSeg = 6;   // sink plane, first rows, window: each may wrap once
constexpr int kAttnMaxRagged = MUSER_MAX_M - 1 + MUSER_MAX_M;  // fits a 32-bit mask
constexpr int kAttnBlocks = 304;  // blocks that a split aims at: two per SM
constexpr int kAttnMaxHeadDim = 256;

// One call.  The cached rows that every query row sees are the "common" rows
// 0..n_common-1, the segments one after another.  The rows only some query
// rows see are the "ragged" ones: up to 15 cached rows at the window's lower
// edge (deeper tree rows see less far back), then the M tree rows; bit r of
// mask[i] says that query row i sees ragged row r.
struct AttnArgs {
    const float* q;     // [M][H*D]
    const float* kt;    // [M][G*D] tree rows
    const float* vt;
    const float* gate;  // [M][H*D] or null
    float* out;
    int M, H, G, D, group;  // group = H / G query heads per K/V head
    float scale_log2;       // scale * log2(e)
    int nseg;
    AttnSeg seg[kAttnMaxSeg];
    int32_t seg_end[kAttnMaxSeg];  // common row index behind segment s
    int32_t n_common;
    AttnSeg edge[2];  // the ragged cached rows: at most one wrap
    int32_t edge0;    // rows of edge[0]
    int32_t n_edge;
    uint32_t mask[MUSER_MAX_M];
    // split: chunk c of the common rows is [c * chunk - shift, (c + 1) * chunk -
    // shift) within 0..n_common; the ragged rows belong to the last chunk
    int32_t chunk, nchunks, shift;
    int32_t cluster;  // blocks of a cluster; chunks behind nchunks are empty
    float* part_o;   // [parts][M*H][D]  unnormalised sums, one part per chunk or cluster
    float2* part_ml; // [parts][M*H]     maximum (base 2) and sum
    unsigned* status;  // device status word
};

// Where the parts lie in the scratch memory (bytes; it is 16-byte aligned): the
// (maximum, sum) pairs first, then the sums from the next 16-byte boundary on.
// Behind the sums, whose number may be odd, the pairs would miss their own 8.
struct AttnPartLayout {
    size_t o, bytes;
};
constexpr AttnPartLayout attn_part_layout(int64_t parts, int64_t rows, int64_t D) {
    const size_t o = (static_cast<size_t>(parts * rows) * 8u + 15u) / 16u * 16u;
    return AttnPartLayout{o, o + (static_cast<size_t>(parts * rows * D) * 4u + 15u) / 16u * 16u};
}

__device__ __forceinline__ const uint16_t* attn_row(const AttnArgs& a, int g, int r, bool value) {
    int s = 0;
#pragma unroll
    for (int i = 0; i < kAttnMaxSeg - 1; ++i) s += (i < a.nseg - 1 && r >= a.seg_end[i]) ? 1 : 0;
    const int r0 = s == 0 ? 0 : a.seg_end[s - 1];
    const AttnSeg& S = a.seg[s];
    return (value ? S.v : S.k) + g * S.head_stride + (r - r0) * S.row_stride;
}

// Element d of ragged row r of K/V head g, binary32.  A tree row's value is
// rounded to binary16 first: that is what the cache will hold of it.
__device__ __forceinline__ float attn_ragged(const AttnArgs& a, int g, int r, int d, bool value) {
    if (r < a.n_edge) {
        const int e = r < a.edge0 ? 0 : 1;
        const AttnSeg& S = a.edge[e];
        const uint16_t* p = (value ? S.v : S.k) + g * S.head_stride + (r - (e ? a.edge0 : 0)) * S.row_stride + d;
        return h2f(ldg_u16(p));
    }
    const float f = (value ? a.vt : a.kt)[(r - a.n_edge) * a.G * a.D + g * a.D + d];
    return __half2float(__float2half_rn(f));
}

// One tensor map per segment and of K and V each: (64 elements) x (tile rows)
// x (1 head) boxes of a segment's rows, 128-byte swizzle.  Rows behind the
// segment's end and elements behind the head's read as zero, so no row that
// is not in the segment gets into shared memory.
struct AttnMaps {
    CUtensorMap k[kAttnMaxSeg], v[kAttnMaxSeg];
};

// The tiles of one chunk: its common rows in runs of up to `tile` rows that do
// not cross a segment's end.
struct AttnWalk {
    int pos, end, seg, first, stop;  // first, stop: the segment's run, read when pos gets there
    __device__ __forceinline__ AttnWalk(const AttnArgs& a, int c)
        : pos(min(max(0, c * a.chunk - a.shift), a.n_common)), end(min((c + 1) * a.chunk - a.shift, a.n_common)), seg(0),
          first(0), stop(0) {}
    __device__ __forceinline__ int count(const AttnArgs& a, int tile) const {
        int n = 0, at = pos;
        for (int s = 0; at < end; ++s) {
            const int upto = min(end, a.seg_end[s]);
            if (upto > at) n += (upto - at + tile - 1) / tile, at = upto;
        }
        return n;
    }
    // The next tile's rows (it must exist), their segment and first row there.
    __device__ __forceinline__ int next(const AttnArgs& a, int tile, int& s, int& row) {
        if (pos >= stop) {
            while (pos >= a.seg_end[seg]) ++seg;
            first = seg == 0 ? 0 : a.seg_end[seg - 1];
            stop = min(end, a.seg_end[seg]);
        }
        s = seg;
        row = pos - first;
        const int n = min(tile, stop - pos);
        pos += n;
        return n;
    }
};

// Clusters of 2^e blocks of a kernel that the current device runs at once (0:
// none), found once per device.
struct AttnResident {
    int clusters[5];
};

// attn_mma.cu
bool attn_mma_supported(const AttnArgs& a);
int attn_mma_row_tiles(int rows);             // 16-row tiles of a block
const int* attn_mma_resident(int row_tiles);  // clusters of 8 blocks that run at once
int launch_attn_mma(const AttnArgs& a, dim3 grid, int row_tiles, cudaStream_t s);
// The segments' tensor maps, boxes of `tile` rows (attn_mma.cu).
int encode_attn_maps(const AttnArgs& a, int tile, AttnMaps& maps);
// The maps of a paged cache's keys and values: (64 elements) x (box rows) x (1
// head) x (1 page) boxes, 128-byte swizzle; what is not in the cache reads as zero.
int encode_page_maps(uint16_t* key, uint16_t* value, const uint64_t (&dims)[4], const uint64_t (&strides)[3], int box_rows,
                     CUtensorMap (&maps)[2]);
// attn_few.cu: up to 32 query rows a K/V head, planes as for attn_tc.cu
const AttnResident* attn_few_resident(int rows);
int launch_attn_few(const AttnArgs& a, dim3 grid, cudaStream_t s);
// attn_tc.cu: planes that attn_mma_supported() takes, head_dim <= 128
const AttnResident* attn_tc_resident(int D);
int launch_attn_tc(const AttnArgs& a, dim3 grid, cudaStream_t s);

}  // namespace muser
