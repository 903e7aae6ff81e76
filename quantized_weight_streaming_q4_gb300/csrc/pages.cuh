// pages.cuh -- launch interfaces of the calls on several sequences: page
// tables, paged K/V caches, beam selection.
#pragma once

#include "common.cuh"

namespace muser {

constexpr int kMaxSequences = MUSER_MAX_SEQUENCES;
constexpr int64_t kMaxPages = int64_t{1} << 20;
constexpr int64_t kMaxTableRows = int64_t{1} << 27;  // rows that a table's stride can name

// What runs a kernel with programmatic stream serialization (its blocks may
// start while the kernel before it still runs, and wait for it before their
// first global access) and, for cluster > 1, in clusters.
template <typename... Params, typename... Args>
int launch_after(const char* what, void (*kern)(Params...), dim3 grid, int threads, size_t smem, int cluster,
                 cudaStream_t s, Args&&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, static_cast<Args&&>(args)...);
    if (e != cudaSuccess) return cuda_fail(e, what);
    return check_launch(what);
}

// The largest cluster, of up to sixteen blocks, that fits(size) says can be placed.
template <typename F>
int largest_cluster(F&& fits) {
    for (int size : {16, 8, 4, 2})
        if (fits(size)) return size;
    return 1;
}

// pages.cu
struct PageTableArgs {
    const int32_t *table, *length, *parent, *add;
    int n_old, n;
    int64_t stride;
    int32_t pages, page_rows;
    int32_t window, n_sink;
    int32_t *table_out, *length_out, *last, *first, *slots, *position, *sequence, *copies, *result;
    int64_t max_new;
};
int launch_page_tables(const PageTableArgs& a, cudaStream_t s);

constexpr int kPageCopyMaxLayers = 128;
struct PageCopyArgs {
    int n_layers, max_copies;
    const int32_t *copies, *count;
    int32_t pages, page_rows, runs, run_dim;  // a page is `runs` runs of page_rows rows of run_dim elements
    int vec;
    uint16_t* buffer[2 * kPageCopyMaxLayers];  // the layers' keys, then their values
};
int launch_page_copy(const PageCopyArgs& a, cudaStream_t s);

struct PageWriteArgs {
    uint16_t *key, *value;
    const float *k, *v;
    const int32_t* slots;
    int64_t rows;
    int32_t page_rows, kv_dim, head_dim, head_major, vec;
    int64_t slot_end;
};
int launch_page_write(const PageWriteArgs& a, cudaStream_t s);

// beam.cu
constexpr int kBeamMaxBeams = 32, kBeamMaxOut = 64;
constexpr int64_t kBeamMaxVocab = int64_t{1} << 20;
struct BeamArgs {
    const float *logits, *score;
    const int32_t* ended;
    int groups, beams;
    int32_t vocab, n, end_token, parts;
    int32_t *parent, *token, *ended_out, *add;
    float* score_out;
    unsigned* ticket;
    void *stat, *cand;
};
size_t beam_scratch_bytes(int groups, int beams, int64_t vocab, int n);
int launch_beam_select(BeamArgs a, void* scratch, cudaStream_t s);

// paged_attn.cu
struct PagedArgs;
size_t paged_scratch_bytes(int64_t head_dim);
int launch_paged_attention(PagedArgs a, void* scratch, cudaStream_t s);

}  // namespace muser
