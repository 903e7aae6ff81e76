// api_pages.cu -- the C ABI's calls on several sequences (declared in
// include/muser.h): argument validation on the host, then launches on the
// caller's stream.
#include <algorithm>
#include <cmath>

#include "checks.cuh"
#include "paged.cuh"

namespace muser {
namespace {

constexpr int64_t kMostRows = int64_t{1} << 30;  // of a table; windows over its rows, and kept first rows, beyond it are all of them

// The checks of a paged cache that every call makes.
int check_cache(const char* fn, const muser_kv_pages* cache) {
    if (cache == nullptr) return set_error(MUSER_ERR_INVALID_ARG, "%s: cache is NULL", fn);
    const muser_kv_pages& C = *cache;
    if (C.key == nullptr || C.value == nullptr) return set_error(MUSER_ERR_INVALID_ARG, "%s: cache buffers are NULL", fn);
    if (!is_aligned(C.key, 2) || !is_aligned(C.value, 2))
        return set_error(MUSER_ERR_MISALIGNED, "%s: cache buffers must be 2-byte aligned", fn);
    if (C.pages < 1 || C.page_rows < 1) return set_error(MUSER_ERR_INVALID_ARG, "%s: pages and page_rows must be positive", fn);
    if (C.kv_dim < 1 || C.head_dim < 1 || C.kv_dim % C.head_dim != 0)
        return set_error(MUSER_ERR_INVALID_ARG, "%s: bad kv_dim/head_dim", fn);
    if (C.pages > kMaxPages || C.pages * C.page_rows > 0x7fffffff || int64_t{C.page_rows} * C.kv_dim > 0x7fffffff)
        return set_error(MUSER_ERR_UNSUPPORTED, "%s: at most 2^20 pages, 2^31-1 rows, and 2^31-1 elements a page", fn);
    return MUSER_OK;
}

size_t cache_bytes(const muser_kv_pages& C) { return static_cast<size_t>(C.pages) * C.page_rows * C.kv_dim * 2u; }

bool overlaps_cache(const muser_kv_pages& C, const void* p, size_t n) {
    return ranges_overlap(C.key, cache_bytes(C), p, n) || ranges_overlap(C.value, cache_bytes(C), p, n);
}

int check_own_overlap(const char* fn, const muser_kv_pages& C) {
    if (ranges_overlap(C.key, cache_bytes(C), C.value, cache_bytes(C)))
        return set_error(MUSER_ERR_INVALID_ARG, "%s: key and value must not overlap", fn);
    return MUSER_OK;
}

int check_ints(const char* fn, const char* name, const int32_t* p, bool required = true) {
    if (p == nullptr) return required ? set_error(MUSER_ERR_INVALID_ARG, "%s: %s is NULL", fn, name) : static_cast<int>(MUSER_OK);
    if (!is_aligned(p, 4)) return set_error(MUSER_ERR_MISALIGNED, "%s: %s must be 4-byte aligned", fn, name);
    return MUSER_OK;
}

int check_sequences(const char* fn, const char* name, int n) {
    if (n < 1 || n > kMaxSequences) return set_error(MUSER_ERR_INVALID_ARG, "%s: %s = %d outside 1..%d", fn, name, n, kMaxSequences);
    return MUSER_OK;
}

int check_table_rows(const char* fn, int64_t stride, int page_rows) {
    if (stride < 1) return set_error(MUSER_ERR_INVALID_ARG, "%s: stride = %lld", fn, (long long)stride);
    if (stride > kMaxTableRows || stride * page_rows > kMaxTableRows)
        return set_error(MUSER_ERR_UNSUPPORTED, "%s: a table of more than 2^27 rows", fn);
    return MUSER_OK;
}

int check_window(const char* fn, int64_t window, int64_t n_sink) {
    if (window < 0 || n_sink < 0) return set_error(MUSER_ERR_INVALID_ARG, "%s: window and n_sink must be >= 0", fn);
    return MUSER_OK;
}
int32_t clipped(int64_t rows) { return static_cast<int32_t>(std::min(rows, kMostRows)); }

int check_shape(const char* fn, int64_t kv_dim, int64_t head_dim, int n, int n_heads) {
    MUSER_TRY(check_sequences(fn, "n", n));
    if (head_dim < 1 || kv_dim < 1 || kv_dim % head_dim != 0) return set_error(MUSER_ERR_INVALID_ARG, "%s: bad kv_dim/head_dim", fn);
    if (n_heads < 1 || n_heads % (kv_dim / head_dim) != 0)
        return set_error(MUSER_ERR_INVALID_ARG, "%s: n_heads = %d is not a multiple of the %lld K/V heads", fn, n_heads,
                         (long long)(kv_dim / head_dim));
    if (head_dim > 256 || n_heads > 1024)
        return set_error(MUSER_ERR_UNSUPPORTED, "%s: head_dim <= 256 and n_heads <= 1024 only", fn);
    return MUSER_OK;
}

struct Range {
    const void* p;
    size_t n;
    const char* name;
};

// No output overlaps an input or another output; `same` names the one pair that may be equal.
template <size_t NI, size_t NO>
int check_apart(const char* fn, const Range (&in)[NI], const Range (&out)[NO]) {
    for (size_t i = 0; i < NO; ++i) {
        if (!out[i].p) continue;
        for (const Range& r : in)
            if (r.p && ranges_overlap(out[i].p, out[i].n, r.p, r.n))
                return set_error(MUSER_ERR_INVALID_ARG, "%s: %s and %s must not overlap", fn, out[i].name, r.name);
        for (size_t j = 0; j < i; ++j)
            if (out[j].p && ranges_overlap(out[i].p, out[i].n, out[j].p, out[j].n))
                return set_error(MUSER_ERR_INVALID_ARG, "%s: %s and %s must not overlap", fn, out[i].name, out[j].name);
    }
    return MUSER_OK;
}

int check_beams(const char* fn, int groups, int beams, int64_t vocab, int n) {
    if (groups < 1 || beams < 1 || n < 1 || vocab < 1)
        return set_error(MUSER_ERR_INVALID_ARG, "%s: groups, beams, vocab and n must be positive", fn);
    if (n > beams * std::min<int64_t>(vocab, kBeamMaxVocab))
        return set_error(MUSER_ERR_INVALID_ARG, "%s: n = %d of %d beams of %lld tokens", fn, n, beams, (long long)vocab);
    if (beams > kBeamMaxBeams || n > kBeamMaxOut || vocab > kBeamMaxVocab || int64_t{groups} * beams > kMaxSequences)
        return set_error(MUSER_ERR_UNSUPPORTED, "%s: beams <= %d, groups * beams <= %d, n <= %d and vocab <= 2^20 only", fn,
                         kBeamMaxBeams, kMaxSequences, kBeamMaxOut);
    return MUSER_OK;
}

}  // namespace
}  // namespace muser

using namespace muser;

extern "C" {

int muser_kv_page_tables(const int32_t* table, const int32_t* length, int n_old, const int32_t* parent,
                         const int32_t* add, int n, int64_t stride, int64_t pages, int page_rows, int64_t window,
                         int64_t n_sink, int32_t* table_out, int32_t* length_out, int32_t* last, int32_t* first,
                         int32_t* slots, int32_t* position, int32_t* sequence, int64_t max_new, int32_t* copies,
                         int32_t* result, void* stream) {
    clear_error();
    const char* fn = "muser_kv_page_tables";
    MUSER_TRY(check_sequences(fn, "n", n));
    MUSER_TRY(check_sequences(fn, "n_old", n_old));
    if (!parent && n != n_old) return set_error(MUSER_ERR_INVALID_ARG, "%s: parent is NULL and n differs from n_old", fn);
    if (pages < 1 || page_rows < 1) return set_error(MUSER_ERR_INVALID_ARG, "%s: pages and page_rows must be positive", fn);
    if (pages > kMaxPages || pages * page_rows > 0x7fffffff)
        return set_error(MUSER_ERR_UNSUPPORTED, "%s: at most 2^20 pages and 2^31-1 rows", fn);
    MUSER_TRY(check_table_rows(fn, stride, page_rows));
    MUSER_TRY(check_window(fn, window, n_sink));
    if (max_new < 0 || max_new > 0x7fffffff) return set_error(MUSER_ERR_INVALID_ARG, "%s: max_new = %lld", fn, (long long)max_new);
    const bool lists = slots || position || sequence;
    MUSER_TRY(check_ints(fn, "table", table));
    MUSER_TRY(check_ints(fn, "length", length));
    MUSER_TRY(check_ints(fn, "parent", parent, false));
    MUSER_TRY(check_ints(fn, "add", add, false));
    MUSER_TRY(check_ints(fn, "table_out", table_out));
    MUSER_TRY(check_ints(fn, "length_out", length_out));
    MUSER_TRY(check_ints(fn, "last", last, false));
    MUSER_TRY(check_ints(fn, "first", first, false));
    MUSER_TRY(check_ints(fn, "slots", slots, false));
    MUSER_TRY(check_ints(fn, "position", position, false));
    MUSER_TRY(check_ints(fn, "sequence", sequence, false));
    MUSER_TRY(check_ints(fn, "copies", copies, parent != nullptr));
    MUSER_TRY(check_ints(fn, "result", result));
    const size_t N = static_cast<size_t>(n) * 4u, old = static_cast<size_t>(n_old) * 4u, fresh = static_cast<size_t>(max_new) * 4u;
    const bool in_place = !parent && table_out == table, same_length = !parent && length_out == length;
    const Range in[] = {{in_place ? nullptr : table, old * static_cast<size_t>(stride), "table"},
                        {same_length ? nullptr : length, old, "length"},
                        {parent, N, "parent"},
                        {add, N, "add"}};
    const Range out[] = {{table_out, N * static_cast<size_t>(stride), "table_out"}, {length_out, N, "length_out"},
                         {last, N, "last"}, {first, N + 4u, "first"}, {slots, fresh, "slots"}, {position, fresh, "position"},
                         {sequence, fresh, "sequence"}, {copies, 3u * N, "copies"}, {result, 32, "result"}};
    MUSER_TRY(check_apart(fn, in, out));
    PageTableArgs a{};
    a.table = table;
    a.length = length;
    a.parent = parent;
    a.add = add;
    a.n_old = n_old;
    a.n = n;
    a.stride = stride;
    a.pages = static_cast<int32_t>(pages);
    a.page_rows = page_rows;
    a.window = clipped(window);
    a.n_sink = clipped(n_sink);
    a.table_out = table_out;
    a.length_out = length_out;
    a.last = last;
    a.first = first;
    a.slots = slots;
    a.position = position;
    a.sequence = sequence;
    a.copies = copies;
    a.result = result;
    a.max_new = lists ? max_new : 0;
    return launch_page_tables(a, as_stream(stream));
}

int muser_kv_page_copy(const muser_kv_pages* layers, int n_layers, const int32_t* copies, const int32_t* count,
                       int max_copies, void* stream) {
    clear_error();
    const char* fn = "muser_kv_page_copy";
    if (n_layers < 1 || n_layers > kPageCopyMaxLayers)
        return set_error(MUSER_ERR_INVALID_ARG, "%s: n_layers = %d outside 1..%d", fn, n_layers, kPageCopyMaxLayers);
    if (max_copies < 0 || max_copies > (1 << 20)) return set_error(MUSER_ERR_INVALID_ARG, "%s: max_copies = %d", fn, max_copies);
    MUSER_TRY(check_ints(fn, "copies", copies, max_copies > 0));
    MUSER_TRY(check_ints(fn, "count", count));
    PageCopyArgs a{};
    a.n_layers = n_layers;
    a.max_copies = max_copies;
    a.copies = copies;
    a.count = count;
    for (int i = 0; i < n_layers; ++i) {
        MUSER_TRY(check_cache(fn, layers ? layers + i : nullptr));
        const muser_kv_pages &C = layers[i], &F = layers[0];
        if (C.pages != F.pages || C.page_rows != F.page_rows || C.kv_dim != F.kv_dim || C.head_dim != F.head_dim ||
            (C.head_major != 0) != (F.head_major != 0))
            return set_error(MUSER_ERR_INVALID_ARG, "%s: layer %d differs from the first in more than its buffers", fn, i);
        a.buffer[i] = C.key;
        a.buffer[n_layers + i] = C.value;
    }
    const muser_kv_pages& F = layers[0];
    a.pages = static_cast<int32_t>(F.pages);
    a.page_rows = F.page_rows;
    a.runs = F.head_major ? F.kv_dim / F.head_dim : 1;
    a.run_dim = F.head_major ? F.head_dim : F.kv_dim;
    a.vec = a.run_dim % 8 == 0;
    for (int i = 0; i < 2 * n_layers; ++i) a.vec = a.vec && is_aligned(a.buffer[i], 16);
    const size_t bytes = cache_bytes(F);
    uint16_t* ordered[2 * kPageCopyMaxLayers];
    std::copy(a.buffer, a.buffer + 2 * n_layers, ordered);
    std::sort(ordered, ordered + 2 * n_layers);
    for (int i = 1; i < 2 * n_layers; ++i)
        if (reinterpret_cast<uintptr_t>(ordered[i]) - reinterpret_cast<uintptr_t>(ordered[i - 1]) < bytes)
            return set_error(MUSER_ERR_INVALID_ARG, "%s: two buffers share memory", fn);
    for (int i = 0; i < n_layers; ++i)
        if (overlaps_cache(layers[i], copies, static_cast<size_t>(max_copies) * 12u) || overlaps_cache(layers[i], count, 4))
            return set_error(MUSER_ERR_INVALID_ARG, "%s: copies and count must not overlap the caches", fn);
    if (max_copies == 0) return MUSER_OK;
    return launch_page_copy(a, as_stream(stream));
}

int muser_kv_page_write(const muser_kv_pages* cache, const float* k, const float* v, const int32_t* slots, int64_t rows,
                        void* stream) {
    clear_error();
    const char* fn = "muser_kv_page_write";
    MUSER_TRY(check_cache(fn, cache));
    const muser_kv_pages& C = *cache;
    MUSER_TRY(check_own_overlap(fn, C));
    if (rows < 0 || rows > 0x7fffffff) return set_error(MUSER_ERR_INVALID_ARG, "%s: rows = %lld", fn, (long long)rows);
    if (rows == 0) return MUSER_OK;
    if (!k || !v) return set_error(MUSER_ERR_INVALID_ARG, "%s: k/v NULL", fn);
    if (!is_aligned(k, 4) || !is_aligned(v, 4)) return set_error(MUSER_ERR_MISALIGNED, "%s: k/v must be 4-byte aligned", fn);
    MUSER_TRY(check_ints(fn, "slots", slots));
    const size_t bytes = static_cast<size_t>(rows) * C.kv_dim * 4u;
    if (overlaps_cache(C, k, bytes) || overlaps_cache(C, v, bytes) || overlaps_cache(C, slots, static_cast<size_t>(rows) * 4u))
        return set_error(MUSER_ERR_INVALID_ARG, "%s: k, v and slots must not overlap the cache", fn);
    PageWriteArgs a{};
    a.key = C.key;
    a.value = C.value;
    a.k = k;
    a.v = v;
    a.slots = slots;
    a.rows = rows;
    a.page_rows = C.page_rows;
    a.kv_dim = C.kv_dim;
    a.head_dim = C.head_dim;
    a.head_major = C.head_major;
    a.vec = (C.head_major ? C.head_dim : C.kv_dim) % 8 == 0 && is_aligned(C.key, 16) && is_aligned(C.value, 16) &&
            is_aligned(k, 16) && is_aligned(v, 16);
    a.slot_end = C.pages * C.page_rows;
    return launch_page_write(a, as_stream(stream));
}

size_t muser_kv_paged_attention_scratch_bytes(int64_t kv_dim, int64_t head_dim, int n, int n_heads) {
    clear_error();
    if (check_shape("muser_kv_paged_attention_scratch_bytes", kv_dim, head_dim, n, n_heads) != MUSER_OK) return 0;
    return paged_scratch_bytes(head_dim);
}

int muser_kv_paged_attention(const muser_kv_pages* cache, const int32_t* table, int64_t stride, int n_tables,
                             const int32_t* position, const int32_t* sequence, const float* q, const float* k,
                             const float* v, const float* gate, int n, int n_heads, int64_t window, int64_t n_sink,
                             float scale, float* out, void* scratch, size_t scratch_bytes, void* stream) {
    clear_error();
    const char* fn = "muser_kv_paged_attention";
    MUSER_TRY(check_cache(fn, cache));
    const muser_kv_pages& C = *cache;
    MUSER_TRY(check_own_overlap(fn, C));
    MUSER_TRY(check_shape(fn, C.kv_dim, C.head_dim, n, n_heads));
    MUSER_TRY(check_table_rows(fn, stride, C.page_rows));
    if (n_tables < 1) return set_error(MUSER_ERR_INVALID_ARG, "%s: n_tables = %d", fn, n_tables);
    MUSER_TRY(check_window(fn, window, n_sink));
    const float scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634074);
    if (!std::isfinite(scale_log2)) return set_error(MUSER_ERR_INVALID_ARG, "%s: scale * log2(e) must be finite", fn);
    MUSER_TRY(check_ints(fn, "table", table));
    MUSER_TRY(check_ints(fn, "position", position));
    MUSER_TRY(check_ints(fn, "sequence", sequence, false));
    MUSER_TRY(check_f32(fn, "q", q));
    if ((k == nullptr) != (v == nullptr)) return set_error(MUSER_ERR_INVALID_ARG, "%s: k and v are both given or both NULL", fn);
    if (k) MUSER_TRY(check_f32(fn, "k", k));
    if (v) MUSER_TRY(check_f32(fn, "v", v));
    if (gate) MUSER_TRY(check_f32(fn, "gate", gate));
    MUSER_TRY(check_f32(fn, "out", out));
    MUSER_TRY(check_f32(fn, "scratch", scratch));
    const size_t need = paged_scratch_bytes(C.head_dim);
    if (scratch_bytes < need) return set_error(MUSER_ERR_INVALID_ARG, "%s: scratch_bytes %zu < %zu", fn, scratch_bytes, need);
    const size_t N = static_cast<size_t>(n), nq = N * n_heads * C.head_dim * 4u, nk = N * C.kv_dim * 4u;
    const Range in[] = {{table, static_cast<size_t>(n_tables) * static_cast<size_t>(stride) * 4u, "table"},
                        {position, N * 4u, "position"}, {sequence, N * 4u, "sequence"}, {q, nq, "q"}, {k, nk, "k"},
                        {v, nk, "v"}, {gate, nq, "gate"}};
    const Range out_ranges[] = {{out, nq, "out"}, {scratch, scratch_bytes, "scratch"}, {C.key, cache_bytes(C), "the cache"},
                                {C.value, cache_bytes(C), "the cache"}};
    MUSER_TRY(check_apart(fn, in, out_ranges));

    PagedArgs a{};
    a.key = C.key;
    a.value = C.value;
    a.pages = static_cast<int32_t>(C.pages);
    a.page_rows = C.page_rows;
    while ((2 << a.page_shift) <= C.page_rows) ++a.page_shift;
    a.page_stride = int64_t{C.page_rows} * C.kv_dim;
    a.row_stride = C.head_major ? C.head_dim : C.kv_dim;
    a.head_stride = C.head_major ? int64_t{C.page_rows} * C.head_dim : C.head_dim;
    a.table = table;
    a.stride = stride;
    a.n_tables = n_tables;
    a.rows_end = static_cast<int32_t>(stride * C.page_rows);
    a.position = position;
    a.sequence = sequence;
    a.q = q;
    a.k = k;
    a.v = v;
    a.gate = gate;
    a.out = out;
    a.n = n;
    a.H = n_heads;
    a.D = C.head_dim;
    a.G = C.kv_dim / C.head_dim;
    a.group = n_heads / a.G;
    a.window = window > 0x7fffffff ? 0 : static_cast<int32_t>(window);  // no position is that far from another
    a.n_sink = clipped(n_sink);
    a.scale_log2 = scale_log2;
    return launch_paged_attention(a, scratch, as_stream(stream));
}

size_t muser_beam_select_scratch_bytes(int groups, int beams, int64_t vocab, int n) {
    clear_error();
    if (check_beams("muser_beam_select_scratch_bytes", groups, beams, vocab, n) != MUSER_OK) return 0;
    return beam_scratch_bytes(groups, beams, vocab, n);
}

int muser_beam_select(const float* logits, const float* score, const int32_t* ended, int groups, int beams,
                      int64_t vocab, int n, int32_t end_token, int32_t* parent, int32_t* token, float* score_out,
                      int32_t* ended_out, int32_t* add, void* scratch, size_t scratch_bytes, void* stream) {
    clear_error();
    const char* fn = "muser_beam_select";
    MUSER_TRY(check_beams(fn, groups, beams, vocab, n));
    if (end_token < -1 || end_token >= vocab) return set_error(MUSER_ERR_INVALID_ARG, "%s: end_token = %d", fn, end_token);
    if (ended && end_token < 0) return set_error(MUSER_ERR_INVALID_ARG, "%s: ended without an end_token", fn);
    MUSER_TRY(check_f32(fn, "logits", logits));
    if (!score || !score_out) return set_error(MUSER_ERR_INVALID_ARG, "%s: score/score_out NULL", fn);
    if (!is_aligned(score, 4) || !is_aligned(score_out, 4))
        return set_error(MUSER_ERR_MISALIGNED, "%s: score/score_out must be 4-byte aligned", fn);
    MUSER_TRY(check_ints(fn, "ended", ended, false));
    MUSER_TRY(check_ints(fn, "parent", parent));
    MUSER_TRY(check_ints(fn, "token", token));
    MUSER_TRY(check_ints(fn, "ended_out", ended_out, false));
    MUSER_TRY(check_ints(fn, "add", add, false));
    MUSER_TRY(check_f32(fn, "scratch", scratch));
    const size_t need = beam_scratch_bytes(groups, beams, vocab, n);
    if (scratch_bytes < need) return set_error(MUSER_ERR_INVALID_ARG, "%s: scratch_bytes %zu < %zu", fn, scratch_bytes, need);
    const size_t rows = static_cast<size_t>(groups) * beams, N = static_cast<size_t>(groups) * n * 4u;
    const Range in[] = {{logits, rows * static_cast<size_t>(vocab) * 4u, "logits"},
                        {n == beams && score_out == score ? nullptr : score, rows * 4u, "score"},
                        {n == beams && ended_out == ended ? nullptr : ended, rows * 4u, "ended"}};
    const Range out[] = {{parent, N, "parent"}, {token, N, "token"}, {score_out, N, "score_out"}, {ended_out, N, "ended_out"},
                         {add, N, "add"}, {scratch, scratch_bytes, "scratch"}};
    MUSER_TRY(check_apart(fn, in, out));
    BeamArgs a{};
    a.logits = logits;
    a.score = score;
    a.ended = ended;
    a.groups = groups;
    a.beams = beams;
    a.vocab = static_cast<int32_t>(vocab);
    a.n = n;
    a.end_token = end_token;
    a.parent = parent;
    a.token = token;
    a.score_out = score_out;
    a.ended_out = ended_out;
    a.add = add;
    return launch_beam_select(a, scratch, as_stream(stream));
}

}  // extern "C"
