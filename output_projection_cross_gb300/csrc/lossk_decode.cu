// lossk_decode.cu -- the extern "C" entry points of beam-search decoding
// (declared in include/lossk.h): argument checks in the documented order,
// workspace layout and launch sequence of each call.  No call synchronises
// and none allocates device memory.
#include "../../include/lossk.h"
#include "decode_internal.h"

#include <cmath>

using namespace lossk;

namespace {

constexpr int64_t MAX_DIM = int64_t(1) << 24;

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
bool misaligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }
bool dtype_ok(int32_t d) { return d == LOSSK_F32 || d == LOSSK_BF16 || d == LOSSK_F16; }
int64_t esize(int32_t d) { return d == LOSSK_F32 ? 4 : 2; }

struct BeamLayout {
    int n_split;
    size_t off_stat, off_cand, total;
};

int32_t beam_layout(int64_t batch, int64_t beams, int64_t vocab, int64_t n_out, BeamLayout *L)
{
    if (batch < 1 || beams < 1 || vocab < 1 || n_out < 1) return LOSSK_EMPTY_DIMENSION;
    // the rows are a grid dimension and the candidates' flat index is 63 bits
    if (batch > MAX_DIM || beams > LOSSK_BEAM_MAX_BEAMS || vocab > MAX_DIM || n_out > LOSSK_BEAM_MAX_OUT)
        return LOSSK_DIMENSION_TOO_LARGE;
    const int64_t rows = batch * beams;
    L->n_split = beam_splits(rows, vocab);
    L->off_stat = 256;
    L->off_cand = align256(L->off_stat + sizeof(BeamStat) * rows * L->n_split);
    L->total = align256(L->off_cand + sizeof(BeamCand) * rows * L->n_split * n_out);
    return LOSSK_OK;
}

// The scratch of the cache calls.
struct CacheLayout {
    int64_t slots;
    size_t off_hash, off_need, off_free, off_moves, off_id, total;
};

int32_t cache_layout(int64_t n_seq, int64_t n_pages, CacheLayout *L)
{
    if (n_seq < 1 || n_pages < 1) return LOSSK_EMPTY_DIMENSION;
    if (n_seq > MAX_DIM || n_pages > MAX_DIM) return LOSSK_DIMENSION_TOO_LARGE;
    L->slots = 2;
    while (L->slots < 2 * n_seq) L->slots *= 2;
    const int64_t moves = n_seq > n_pages / 2 + 1 ? n_seq : n_pages / 2 + 1;
    L->off_hash = 512;                                     // the header, then counters
    L->off_need = align256(L->off_hash + sizeof(SharerSlot) * L->slots);
    L->off_free = align256(L->off_need + sizeof(int4) * n_seq);
    L->off_moves = align256(L->off_free + sizeof(int32_t) * n_pages);
    L->off_id = align256(L->off_moves + sizeof(int2) * moves);
    L->total = align256(L->off_id + sizeof(int32_t) * n_pages);
    return LOSSK_OK;
}

// The sizes every cache call shares.
int32_t cache_sizes(int64_t n_seq, int64_t max_pages, int64_t page, int64_t n_pages)
{
    if (n_seq < 1 || max_pages < 1 || page < 1 || n_pages < 1) return LOSSK_EMPTY_DIMENSION;
    if (n_seq > MAX_DIM || max_pages > MAX_DIM || page > MAX_DIM || n_pages > MAX_DIM) return LOSSK_DIMENSION_TOO_LARGE;
    return LOSSK_OK;
}

bool table_short(int64_t n_seq, int64_t max_pages, const void *table, int64_t len, int64_t stride)
{
    return !table || stride < max_pages || stride > (int64_t(1) << 40) || len < (n_seq - 1) * stride + max_pages;
}

// A pool of n_planes planes of n_pages pages: 581, 582 or 591.
int32_t pool_check(int64_t n_pages, const void *pool, int64_t pool_bytes, int64_t n_planes, int64_t plane_stride,
                   int64_t page_stride, int64_t page_bytes)
{
    const int64_t most = int64_t(1) << 45;
    if (n_planes < 1 || page_bytes < 1) return LOSSK_EMPTY_DIMENSION;
    if (n_planes > MAX_DIM || page_bytes > most) return LOSSK_DIMENSION_TOO_LARGE;
    if (!pool || page_stride < page_bytes || page_stride > most / n_pages || plane_stride < 0 ||
        plane_stride > most / n_planes ||
        (n_planes > 1 && plane_stride < page_bytes) ||
        pool_bytes < (n_planes - 1) * plane_stride + (n_pages - 1) * page_stride + page_bytes)
        return LOSSK_LENGTH_MISMATCH;
    return LOSSK_OK;
}

bool pool_unaligned(const void *pool, int64_t plane_stride, int64_t page_stride, int64_t page_bytes)
{
    return misaligned(pool, 16) || ((plane_stride | page_stride | page_bytes) & 15) != 0;
}

// Key or value pages of one layer: element (page, token, head, i) at page
// page_stride + token tok_stride + head head_stride + i.
bool pages_short(int64_t n_pages, int64_t page, int64_t n_kv, int64_t hd, const void *p, int64_t len,
                 int64_t page_stride, int64_t tok_stride, int64_t head_stride)
{
    const int64_t most = int64_t(1) << 44;
    return !p || page_stride < 0 || tok_stride < 0 || head_stride < 0 || page_stride > most / n_pages ||
           tok_stride > most / page || head_stride > most / n_kv ||
           len < (n_pages - 1) * page_stride + (page - 1) * tok_stride + (n_kv - 1) * head_stride + hd;
}

CopyArgs copy_args(void *pool, int64_t n_planes, int64_t plane_stride, int64_t page_stride, int64_t page_bytes,
                   int64_t n_pages, int *fault)
{
    CopyArgs c{};
    c.pool = static_cast<char *>(pool);
    c.plane_stride = plane_stride;
    c.page_stride = page_stride;
    c.page_bytes = page_bytes;
    c.n_planes = static_cast<int>(n_planes);
    c.n_pages = static_cast<int>(n_pages);
    c.fault = fault;
    return c;
}

// The scratch of lossk_paged_attn.  Partial results take at most twice the query
// rows on either side (a group's shared rows are cut into items of mr rows,
// the last one less than full), and one item's rows more for each run.
struct AttnLayout {
    size_t off_shared, off_base, off_runs, off_part, total;
};

int32_t attn_layout(int64_t n_seq, int64_t n_q, int64_t n_kv, int64_t hd, AttnLayout *L)
{
    if (n_seq < 1 || n_q < 1 || n_kv < 1 || hd < 1) return LOSSK_EMPTY_DIMENSION;
    if (n_seq > MAX_DIM || n_q > MAX_DIM || n_kv > MAX_DIM || n_seq * n_q > MAX_DIM || hd > 256)
        return LOSSK_DIMENSION_TOO_LARGE;
    L->off_shared = 256;
    L->off_base = align256(L->off_shared + sizeof(int32_t) * n_seq);
    L->off_runs = align256(L->off_base + sizeof(long long) * (n_seq + 1));
    // (an item has at least one query row)
    L->off_part = align256(L->off_runs + sizeof(int2) * 2 * n_seq * n_q);
    const size_t rows = 4 * static_cast<size_t>(n_seq) * n_q + 2 * ATTN_MAX_ROWS;
    L->total = align256(L->off_part + sizeof(float) * rows * (hd + ATTN_ROW));
    return LOSSK_OK;
}

int32_t ws_check(const void *ws, int64_t bytes, size_t need)
{
    if (!ws || bytes < static_cast<int64_t>(need)) return LOSSK_LENGTH_MISMATCH;
    return LOSSK_OK;
}

int *fault_of(void *ws) { return &static_cast<WsHeader *>(ws)->pad[HDR_FAULT]; }

int32_t status_of(cudaError_t e) { return e == cudaSuccess ? LOSSK_OK : LOSSK_DEVICE_ERROR; }

} // namespace

extern "C" {

int64_t lossk_decode_workspace_bytes(int32_t kind, int64_t a, int64_t b, int64_t c, int64_t d)
{
    if (kind == LOSSK_KIND_BEAM_SELECT) {
        BeamLayout L;
        return beam_layout(a, b, c, d, &L) == LOSSK_OK ? static_cast<int64_t>(L.total) : -1;
    }
    if (kind == LOSSK_KIND_CACHE) {
        CacheLayout L;
        return cache_layout(a, b, &L) == LOSSK_OK ? static_cast<int64_t>(L.total) : -1;
    }
    if (kind == LOSSK_KIND_PAGED_ATTN) {
        AttnLayout L;
        return attn_layout(a, b, c, d, &L) == LOSSK_OK ? static_cast<int64_t>(L.total) : -1;
    }
    return -1;
}

int32_t lossk_beam_select(int64_t batch, int64_t beams, int64_t vocab, int64_t n_out, int32_t dtype,
                          const void *logits, int64_t logits_len, int64_t row_stride, const float *scores,
                          int64_t scores_len, double temperature, const uint32_t *allow, int64_t allow_len,
                          int64_t allow_stride, const uint8_t *finished, int64_t end_token, const int32_t *lengths,
                          double length_alpha, int32_t *parent_out, int64_t *token_out, float *score_out,
                          uint8_t *finished_out, int32_t *length_out, float *lse_out, void *workspace,
                          int64_t workspace_bytes, lossk_stream_t stream)
{
    BeamLayout L;
    int32_t s = beam_layout(batch, beams, vocab, n_out, &L);
    if (s != LOSSK_OK) return s;
    const int64_t rows = batch * beams, words = (vocab + 31) / 32;
    if (!dtype_ok(dtype) || !logits || !scores || !parent_out || !token_out || !score_out) return LOSSK_LENGTH_MISMATCH;
    if (row_stride < vocab || row_stride > (int64_t(1) << 40) || logits_len < (rows - 1) * row_stride + vocab ||
        scores_len < rows)
        return LOSSK_LENGTH_MISMATCH;
    if (allow && ((allow_stride != 0 && allow_stride < words) || allow_stride > (int64_t(1) << 40) ||
                  allow_len < (rows - 1) * allow_stride + words))
        return LOSSK_LENGTH_MISMATCH;
    if ((s = ws_check(workspace, workspace_bytes, L.total)) != LOSSK_OK) return s;
    if (misaligned(logits, 16) || misaligned(workspace, 256) || misaligned(scores, 4) || misaligned(allow, 4) ||
        misaligned(lengths, 4) || misaligned(parent_out, 4) || misaligned(token_out, 8) || misaligned(score_out, 4) ||
        misaligned(length_out, 4) || misaligned(lse_out, 4))
        return LOSSK_UNALIGNED;
    // (1 / temperature has to be a float with room for a logit's size)
    if (!(temperature >= 1e-30 && temperature <= 1e30) || !std::isfinite(length_alpha)) return LOSSK_NON_FINITE_SCALAR;
    if (end_token < -1 || end_token >= vocab) return LOSSK_TARGET_OUT_OF_RANGE;

    uint8_t *ws = static_cast<uint8_t *>(workspace);
    BeamArgs a{};
    a.logits = logits;
    a.row_stride = row_stride;
    a.batch = static_cast<int>(batch);
    a.beams = static_cast<int>(beams);
    a.vocab = static_cast<int>(vocab);
    a.n_out = static_cast<int>(n_out);
    a.dtype = dtype;
    // splits begin on 16-byte boundaries of an aligned row
    a.split_len = static_cast<int>(((vocab + L.n_split - 1) / L.n_split + 63) & ~int64_t(63));
    a.n_split = static_cast<int>((vocab + a.split_len - 1) / a.split_len);
    a.cap = beam_cap(dtype, a.n_out);
    a.c = static_cast<float>(LOG2E / temperature);
    a.inv_t = 1.0 / temperature;
    a.allow = allow;
    a.allow_stride = allow_stride;
    a.scores = scores;
    a.finished = finished;
    a.end_token = static_cast<int>(end_token);
    a.lengths = lengths;
    a.length_alpha = length_alpha;
    a.parent_out = parent_out;
    a.token_out = token_out;
    a.score_out = score_out;
    a.finished_out = finished_out;
    a.length_out = length_out;
    a.lse_out = lse_out;
    a.stat = reinterpret_cast<BeamStat *>(ws + L.off_stat);
    a.cand = reinterpret_cast<BeamCand *>(ws + L.off_cand);
    a.next = &static_cast<WsHeader *>(workspace)->pad[HDR_NEXT];
    a.err = &static_cast<WsHeader *>(workspace)->err;
    a.fault = fault_of(workspace);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    {
        Launch k(KK_BEAM_ROWS, st);
        if (launch_beam_rows(a, st) != cudaSuccess) return LOSSK_DEVICE_ERROR;
    }
    Launch k(KK_BEAM_MERGE, st);
    return status_of(launch_beam_merge(a, st));
}

int32_t lossk_beam_gather(int64_t n_group, int64_t n_src, int64_t n_dst, int64_t row_bytes, const int32_t *parent,
                          int64_t parent_len, const void *src, int64_t src_bytes, void *dst, int64_t dst_bytes,
                          void *workspace, int64_t workspace_bytes, lossk_stream_t stream)
{
    if (n_group < 1 || n_src < 1 || n_dst < 1 || row_bytes < 1) return LOSSK_EMPTY_DIMENSION;
    if (n_group > MAX_DIM || n_src > MAX_DIM || n_dst > MAX_DIM || n_group * n_src > MAX_DIM ||
        n_group * n_dst > MAX_DIM || row_bytes > (int64_t(1) << 38))
        return LOSSK_DIMENSION_TOO_LARGE;
    if (!parent || !src || !dst || parent_len < n_group * n_dst || src_bytes < n_group * n_src * row_bytes ||
        dst_bytes < n_group * n_dst * row_bytes)
        return LOSSK_LENGTH_MISMATCH;
    const int32_t s = ws_check(workspace, workspace_bytes, 256);
    if (s != LOSSK_OK) return s;
    if (misaligned(workspace, 256) || misaligned(parent, 4)) return LOSSK_UNALIGNED;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    Launch k(KK_BEAM_GATHER, st);
    return status_of(launch_beam_gather(n_group, n_src, n_dst, row_bytes, parent, src, dst, fault_of(workspace), st));
}

int32_t lossk_cache_fork(int64_t n_group, int64_t n_src, int64_t n_dst, int64_t max_pages, int64_t page_size,
                         int64_t n_pages, const int32_t *parent, int64_t parent_len, const int32_t *table,
                         int64_t table_len, int64_t table_stride, const int32_t *lens, int64_t lens_len, int32_t *ref,
                         int64_t ref_len, int32_t *table_out, int64_t table_out_len, int64_t table_out_stride,
                         int32_t *lens_out, int64_t lens_out_len, void *workspace, int64_t workspace_bytes,
                         lossk_stream_t stream)
{
    if (n_group < 1 || n_src < 1 || n_dst < 1) return LOSSK_EMPTY_DIMENSION;
    if (n_group > MAX_DIM || n_src > MAX_DIM || n_dst > MAX_DIM) return LOSSK_DIMENSION_TOO_LARGE;
    const int64_t rs = n_group * n_src, rd = n_group * n_dst;
    int32_t s = cache_sizes(rs > rd ? rs : rd, max_pages, page_size, n_pages);
    if (s != LOSSK_OK) return s;
    if (!parent || parent_len < rd || table_short(rs, max_pages, table, table_len, table_stride) || !lens ||
        lens_len < rs || !ref || ref_len < n_pages ||
        table_short(rd, max_pages, table_out, table_out_len, table_out_stride) || !lens_out || lens_out_len < rd ||
        table_out == table || lens_out == lens)
        return LOSSK_LENGTH_MISMATCH;
    if ((s = ws_check(workspace, workspace_bytes, 256)) != LOSSK_OK) return s;
    if (misaligned(workspace, 256) || misaligned(parent, 4) || misaligned(table, 4) || misaligned(lens, 4) ||
        misaligned(ref, 4) || misaligned(table_out, 4) || misaligned(lens_out, 4))
        return LOSSK_UNALIGNED;
    ForkArgs a{};
    a.n_group = static_cast<int>(n_group);
    a.n_src = static_cast<int>(n_src);
    a.n_dst = static_cast<int>(n_dst);
    a.max_pages = static_cast<int>(max_pages);
    a.page = static_cast<int>(page_size);
    a.n_pages = static_cast<int>(n_pages);
    a.parent = parent;
    a.table = table;
    a.lens = lens;
    a.table_stride = table_stride;
    a.table_out_stride = table_out_stride;
    a.ref = ref;
    a.table_out = table_out;
    a.lens_out = lens_out;
    a.fault = fault_of(workspace);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    Launch k(KK_CACHE_FORK, st);
    return status_of(launch_cache_fork(a, st));
}

int32_t lossk_cache_reserve(int64_t n_seq, int64_t max_pages, int64_t page_size, int64_t n_pages, int64_t n_new_all,
                            const int32_t *n_new, int64_t n_new_len, int32_t *table, int64_t table_len,
                            int64_t table_stride, const int32_t *lens, int64_t lens_len, int32_t *ref,
                            int64_t ref_len, void *pool, int64_t pool_bytes, int64_t n_planes, int64_t plane_stride,
                            int64_t page_stride, int64_t page_bytes, void *workspace, int64_t workspace_bytes,
                            lossk_stream_t stream)
{
    int32_t s = cache_sizes(n_seq, max_pages, page_size, n_pages);
    if (s != LOSSK_OK) return s;
    CacheLayout L;
    if ((s = cache_layout(n_seq, n_pages, &L)) != LOSSK_OK) return s;
    if ((s = pool_check(n_pages, pool, pool_bytes, n_planes, plane_stride, page_stride, page_bytes)) != LOSSK_OK)
        return s;
    if (n_new_all < 0 || n_new_all > MAX_DIM || (n_new && n_new_len < n_seq) ||
        table_short(n_seq, max_pages, table, table_len, table_stride) || !lens || lens_len < n_seq || !ref ||
        ref_len < n_pages)
        return LOSSK_LENGTH_MISMATCH;
    if ((s = ws_check(workspace, workspace_bytes, L.total)) != LOSSK_OK) return s;
    if (pool_unaligned(pool, plane_stride, page_stride, page_bytes) || misaligned(workspace, 256) ||
        misaligned(n_new, 4) || misaligned(table, 4) || misaligned(lens, 4) || misaligned(ref, 4))
        return LOSSK_UNALIGNED;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    ReserveArgs a{};
    a.n_seq = static_cast<int>(n_seq);
    a.max_pages = static_cast<int>(max_pages);
    a.page = static_cast<int>(page_size);
    a.n_pages = static_cast<int>(n_pages);
    a.n_new_all = static_cast<int>(n_new_all);
    a.n_new = n_new;
    a.lens = lens;
    a.table = table;
    a.ref = ref;
    a.table_stride = table_stride;
    a.hash = reinterpret_cast<SharerSlot *>(ws + L.off_hash);
    a.hash_mask = static_cast<int>(L.slots - 1);
    a.need = reinterpret_cast<int4 *>(ws + L.off_need);
    a.free_list = reinterpret_cast<int32_t *>(ws + L.off_free);
    a.moves = reinterpret_cast<int2 *>(ws + L.off_moves);
    a.n_copy = reinterpret_cast<int *>(ws + 256);
    a.fault = fault_of(workspace);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    {
        Launch k(KK_CACHE_PLAN, st);
        if (launch_cache_plan(a, st) != cudaSuccess) return LOSSK_DEVICE_ERROR;
    }
    CopyArgs c = copy_args(pool, n_planes, plane_stride, page_stride, page_bytes, n_pages, a.fault);
    c.moves = a.moves;
    c.n_dev = a.n_copy;
    Launch k(KK_CACHE_COPY, st);
    return status_of(launch_cache_copy(c, n_seq, st));
}

int32_t lossk_cache_free(int64_t n_seq, int64_t max_pages, int64_t page_size, int64_t n_pages, const uint8_t *drop,
                         int64_t drop_len, int32_t *table, int64_t table_len, int64_t table_stride, int32_t *lens,
                         int64_t lens_len, int32_t *ref, int64_t ref_len, void *workspace, int64_t workspace_bytes,
                         lossk_stream_t stream)
{
    int32_t s = cache_sizes(n_seq, max_pages, page_size, n_pages);
    if (s != LOSSK_OK) return s;
    if ((drop && drop_len < n_seq) || table_short(n_seq, max_pages, table, table_len, table_stride) || !lens ||
        lens_len < n_seq || !ref || ref_len < n_pages)
        return LOSSK_LENGTH_MISMATCH;
    if ((s = ws_check(workspace, workspace_bytes, 256)) != LOSSK_OK) return s;
    if (misaligned(workspace, 256) || misaligned(table, 4) || misaligned(lens, 4) || misaligned(ref, 4))
        return LOSSK_UNALIGNED;
    FreeArgs a{};
    a.n_seq = static_cast<int>(n_seq);
    a.max_pages = static_cast<int>(max_pages);
    a.page = static_cast<int>(page_size);
    a.n_pages = static_cast<int>(n_pages);
    a.drop = drop;
    a.table = table;
    a.lens = lens;
    a.ref = ref;
    a.table_stride = table_stride;
    a.fault = fault_of(workspace);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    Launch k(KK_CACHE_FREE, st);
    return status_of(launch_cache_free(a, st));
}

int32_t lossk_cache_compact(int64_t n_seq, int64_t max_pages, int64_t page_size, int64_t n_pages, const int32_t *table,
                            int64_t table_len, int64_t table_stride, const int32_t *lens, int64_t lens_len,
                            const int32_t *ref, int64_t ref_len, int32_t *table_out, int64_t table_out_len,
                            int64_t table_out_stride, int32_t *ref_out, int64_t ref_out_len, int32_t *n_live_out,
                            void *pool, int64_t pool_bytes, int64_t n_planes, int64_t plane_stride,
                            int64_t page_stride, int64_t page_bytes, void *workspace, int64_t workspace_bytes,
                            lossk_stream_t stream)
{
    int32_t s = cache_sizes(n_seq, max_pages, page_size, n_pages);
    if (s != LOSSK_OK) return s;
    CacheLayout L;
    if ((s = cache_layout(n_seq, n_pages, &L)) != LOSSK_OK) return s;
    if ((s = pool_check(n_pages, pool, pool_bytes, n_planes, plane_stride, page_stride, page_bytes)) != LOSSK_OK)
        return s;
    if (table_short(n_seq, max_pages, table, table_len, table_stride) || !lens || lens_len < n_seq || !ref ||
        ref_len < n_pages || table_short(n_seq, max_pages, table_out, table_out_len, table_out_stride) || !ref_out ||
        ref_out_len < n_pages || ref_out == ref || !n_live_out || (table_out == table && table_out_stride != table_stride))
        return LOSSK_LENGTH_MISMATCH;
    if ((s = ws_check(workspace, workspace_bytes, L.total)) != LOSSK_OK) return s;
    if (pool_unaligned(pool, plane_stride, page_stride, page_bytes) || misaligned(workspace, 256) ||
        misaligned(table, 4) || misaligned(lens, 4) || misaligned(ref, 4) || misaligned(table_out, 4) ||
        misaligned(ref_out, 4) || misaligned(n_live_out, 4))
        return LOSSK_UNALIGNED;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    CompactArgs a{};
    a.n_seq = static_cast<int>(n_seq);
    a.max_pages = static_cast<int>(max_pages);
    a.page = static_cast<int>(page_size);
    a.n_pages = static_cast<int>(n_pages);
    a.table = table;
    a.lens = lens;
    a.ref = ref;
    a.table_stride = table_stride;
    a.table_out_stride = table_out_stride;
    a.table_out = table_out;
    a.ref_out = ref_out;
    a.n_live_out = n_live_out;
    a.new_id = reinterpret_cast<int32_t *>(ws + L.off_id);
    a.moves = reinterpret_cast<int2 *>(ws + L.off_moves);
    a.n_copy = reinterpret_cast<int *>(ws + 256);
    a.fault = fault_of(workspace);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    {
        Launch k(KK_CACHE_RANK, st);
        if (launch_cache_rank(a, st) != cudaSuccess) return LOSSK_DEVICE_ERROR;
    }
    CopyArgs c = copy_args(pool, n_planes, plane_stride, page_stride, page_bytes, n_pages, a.fault);
    c.moves = a.moves;
    Launch k(KK_CACHE_COPY, st);
    return status_of(launch_cache_move(a, c, st));
}

int32_t lossk_cache_copy(int64_t n_copy, int64_t n_pages, const int32_t *src, int64_t src_len, const int32_t *dst,
                         int64_t dst_len, void *pool, int64_t pool_bytes, int64_t n_planes, int64_t plane_stride,
                         int64_t page_stride, int64_t page_bytes, void *workspace, int64_t workspace_bytes,
                         lossk_stream_t stream)
{
    if (n_copy < 1 || n_pages < 1) return LOSSK_EMPTY_DIMENSION;
    if (n_copy > MAX_DIM || n_pages > MAX_DIM) return LOSSK_DIMENSION_TOO_LARGE;
    int32_t s = pool_check(n_pages, pool, pool_bytes, n_planes, plane_stride, page_stride, page_bytes);
    if (s != LOSSK_OK) return s;
    if (!src || !dst || src_len < n_copy || dst_len < n_copy) return LOSSK_LENGTH_MISMATCH;
    if ((s = ws_check(workspace, workspace_bytes, 256)) != LOSSK_OK) return s;
    if (pool_unaligned(pool, plane_stride, page_stride, page_bytes) || misaligned(workspace, 256) ||
        misaligned(src, 4) || misaligned(dst, 4))
        return LOSSK_UNALIGNED;
    CopyArgs c = copy_args(pool, n_planes, plane_stride, page_stride, page_bytes, n_pages, fault_of(workspace));
    c.src = src;
    c.dst = dst;
    c.n = n_copy;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    Launch k(KK_CACHE_COPY, st);
    return status_of(launch_cache_copy(c, n_copy, st));
}

int32_t lossk_cache_write(int64_t n_tok, int64_t n_seq, int64_t n_kv_heads, int64_t head_dim, int64_t max_pages,
                          int64_t page_size, int64_t n_pages, int32_t dtype, const void *k_new, const void *v_new,
                          int64_t new_len, int64_t new_stride, void *k_pages, void *v_pages, int64_t pages_len,
                          int64_t page_stride, int64_t tok_stride, int64_t head_stride, const int32_t *table,
                          int64_t table_len, int64_t table_stride, const int32_t *lens, int64_t lens_len,
                          const int32_t *first, int64_t first_len, void *workspace, int64_t workspace_bytes,
                          lossk_stream_t stream)
{
    if (n_tok < 1 || n_kv_heads < 1 || head_dim < 1) return LOSSK_EMPTY_DIMENSION;
    if (n_tok > MAX_DIM || n_kv_heads > MAX_DIM || head_dim > MAX_DIM || n_kv_heads * head_dim > MAX_DIM)
        return LOSSK_DIMENSION_TOO_LARGE;
    int32_t s = cache_sizes(n_seq, max_pages, page_size, n_pages);
    if (s != LOSSK_OK) return s;
    const int64_t row = n_kv_heads * head_dim;
    if (!dtype_ok(dtype) || !k_new || !v_new || new_stride < row || new_stride > (int64_t(1) << 40) ||
        new_len < (n_tok - 1) * new_stride + row ||
        pages_short(n_pages, page_size, n_kv_heads, head_dim, k_pages, pages_len, page_stride, tok_stride,
                    head_stride) ||
        !v_pages || table_short(n_seq, max_pages, table, table_len, table_stride) || !lens || lens_len < n_seq ||
        (first ? first_len < n_seq + 1 : n_tok != n_seq))
        return LOSSK_LENGTH_MISMATCH;
    if ((s = ws_check(workspace, workspace_bytes, 256)) != LOSSK_OK) return s;
    const uintptr_t es = static_cast<uintptr_t>(esize(dtype));
    if (misaligned(workspace, 256) || misaligned(k_new, es) || misaligned(v_new, es) || misaligned(k_pages, es) ||
        misaligned(v_pages, es) || misaligned(table, 4) || misaligned(lens, 4) || misaligned(first, 4))
        return LOSSK_UNALIGNED;
    const int64_t e = esize(dtype);
    WriteArgs a{};
    a.n_tok = n_tok;
    a.n_seq = static_cast<int>(n_seq);
    a.n_kv = static_cast<int>(n_kv_heads);
    a.row_bytes = static_cast<int>(head_dim * e);
    a.page = static_cast<int>(page_size);
    a.n_pages = static_cast<int>(n_pages);
    a.max_pages = static_cast<int>(max_pages);
    a.k_new = static_cast<const char *>(k_new);
    a.v_new = static_cast<const char *>(v_new);
    a.k_row = a.v_row = new_stride * e;
    a.k = static_cast<char *>(k_pages);
    a.v = static_cast<char *>(v_pages);
    a.k_page = a.v_page = page_stride * e;
    a.k_tok = a.v_tok = tok_stride * e;
    a.k_head = a.v_head = head_stride * e;
    a.table = table;
    a.lens = lens;
    a.first = first;
    a.table_stride = table_stride;
    a.fault = fault_of(workspace);
    const uint64_t all = reinterpret_cast<uintptr_t>(k_new) | reinterpret_cast<uintptr_t>(v_new) |
                         reinterpret_cast<uintptr_t>(k_pages) | reinterpret_cast<uintptr_t>(v_pages) |
                         static_cast<uint64_t>(a.row_bytes | a.k_row | a.k_page | a.k_tok | a.k_head);
    const int word = all % 16 == 0 ? 16 : all % 4 == 0 ? 4 : 2;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    Launch k(KK_CACHE_WRITE, st);
    return status_of(launch_cache_write(a, word, st));
}

int32_t lossk_paged_attn(int64_t n_seq, int64_t n_q_heads, int64_t n_kv_heads, int64_t head_dim, int64_t max_pages,
                         int64_t page_size, int64_t n_pages, int64_t share, int32_t dtype, const void *q,
                         int64_t q_len, int64_t q_stride, const void *k_pages, const void *v_pages,
                         int64_t pages_len, int64_t page_stride, int64_t tok_stride, int64_t head_stride,
                         const int32_t *table, int64_t table_len, int64_t table_stride, const int32_t *lens,
                         int64_t lens_len, int64_t max_len, int64_t window, double scale, void *out, int64_t out_len,
                         float *lse_out, void *workspace, int64_t workspace_bytes, lossk_stream_t stream)
{
    AttnLayout L;
    int32_t s = attn_layout(n_seq, n_q_heads, n_kv_heads, head_dim, &L);
    if (s != LOSSK_OK) return s;
    if ((s = cache_sizes(n_seq, max_pages, page_size, n_pages)) != LOSSK_OK) return s;
    if (share < 1) return LOSSK_EMPTY_DIMENSION;
    if (max_pages * page_size > (int64_t(1) << 30)) return LOSSK_DIMENSION_TOO_LARGE;
    const int64_t row = n_q_heads * head_dim;
    if (!dtype_ok(dtype) || n_q_heads % n_kv_heads || n_seq % share || max_len < 0 || window < 0 || !q ||
        q_stride < row || q_stride > (int64_t(1) << 40) || q_len < (n_seq - 1) * q_stride + row || !out ||
        out_len < n_seq * row || !v_pages ||
        pages_short(n_pages, page_size, n_kv_heads, head_dim, k_pages, pages_len, page_stride, tok_stride,
                    head_stride) ||
        table_short(n_seq, max_pages, table, table_len, table_stride) || !lens || lens_len < n_seq)
        return LOSSK_LENGTH_MISMATCH;
    if ((s = ws_check(workspace, workspace_bytes, L.total)) != LOSSK_OK) return s;
    // rows are read 16 bytes at a time
    const int64_t e = esize(dtype);
    if (misaligned(q, 16) || misaligned(k_pages, 16) || misaligned(v_pages, 16) || misaligned(out, 16) ||
        misaligned(workspace, 256) || misaligned(table, 4) || misaligned(lens, 4) || misaligned(lse_out, 4) ||
        ((head_dim | q_stride | page_stride | tok_stride | head_stride) * e & 15) != 0)
        return LOSSK_UNALIGNED;
    if (!std::isfinite(scale) || !std::isfinite(static_cast<float>(scale * LOG2E))) return LOSSK_NON_FINITE_SCALAR;

    uint8_t *ws = static_cast<uint8_t *>(workspace);
    AttnArgs a{};
    a.n_group = static_cast<int>(n_seq / share);
    a.share = static_cast<int>(share);
    a.n_q = static_cast<int>(n_q_heads);
    a.n_kv = static_cast<int>(n_kv_heads);
    a.group = a.n_q / a.n_kv;
    a.hd = static_cast<int>(head_dim);
    a.max_pages = static_cast<int>(max_pages);
    a.page = static_cast<int>(page_size);
    a.n_pages = static_cast<int>(n_pages);
    a.window = static_cast<int>(window < (int64_t(1) << 30) ? window : 0);   // wider than any sequence: none
    a.scale_log2 = static_cast<float>(scale * LOG2E);
    a.q = q;
    a.k = k_pages;
    a.v = v_pages;
    a.q_stride = q_stride;
    a.page_stride = page_stride;
    a.tok_stride = tok_stride;
    a.head_stride = head_stride;
    a.table = table;
    a.lens = lens;
    a.table_stride = table_stride;
    a.out = out;
    a.lse = lse_out;
    const int rows_s = a.share * a.group;
    const AttnShape shape = attn_shape(dtype, a.hd, rows_s);
    a.kt = shape.kt;
    a.mr = shape.mr;
    a.cs = (rows_s + a.mr - 1) / a.mr;
    a.cp = (a.group + a.mr - 1) / a.mr;
    a.ra = rows_s < a.mr ? rows_s : a.mr;
    a.rb = a.group < a.mr ? a.group : a.mr;
    // no more runs than units there can be
    const int64_t cap = max_len > 0 && max_len < max_pages * page_size ? max_len : max_pages * page_size;
    const int64_t units = n_seq * n_kv_heads * a.cp * ((cap + a.kt - 1) / a.kt + 1);
    a.nw = static_cast<int>(units < 152 * shape.runs ? units : 152 * shape.runs);
    a.shared = reinterpret_cast<int32_t *>(ws + L.off_shared);
    a.base = reinterpret_cast<long long *>(ws + L.off_base);
    a.runs_a = reinterpret_cast<int2 *>(ws + L.off_runs);
    a.runs_b = a.runs_a + n_seq * n_q_heads;
    a.part_a = reinterpret_cast<float *>(ws + L.off_part);
    a.part_b = a.part_a + (static_cast<int64_t>(a.n_group) * a.n_kv * a.cs + a.nw) * a.ra * (a.hd + ATTN_ROW);
    a.fault = fault_of(workspace);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (attn_shares(a)) {
        Launch k(KK_ATTN_PLAN, st);
        if (launch_attn_share(a, st) != cudaSuccess) return LOSSK_DEVICE_ERROR;
    }
    if (attn_plans(a)) {
        Launch k(KK_ATTN_PLAN, st);
        if (launch_attn_plan(a, st) != cudaSuccess) return LOSSK_DEVICE_ERROR;
    }
    {
        Launch k(KK_ATTN, st);
        if (launch_attn(dtype, a, st) != cudaSuccess) return LOSSK_DEVICE_ERROR;
    }
    Launch k(KK_ATTN_JOIN, st);
    return status_of(launch_attn_join(dtype, a, st));
}

} // extern "C"
