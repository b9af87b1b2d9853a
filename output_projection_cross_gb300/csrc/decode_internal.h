// decode_internal.h -- shared between the host entry points and the kernels of
// beam-search decoding (k_beam.cu, k_pages.cu, k_attn.cu): argument records and
// launcher declarations.  Not part of the public ABI.
#pragma once
#include "lossk_internal.h"

namespace lossk {

// Leaves a lossk_status in the workspace header's fault word; the largest
// stays, so what is reported does not depend on which block came first.
__device__ __forceinline__ void raise_fault(int *fault, int status) { atomicMax(fault, status); }

// ---- beam selection ------------------------------------------------------------
// What the rows kernel leaves per (row, split): the largest kept logit m; the
// sum z + lost of 2^(c x + b) over the kept logits, c = log2(e) / T and b what
// -c ref rounds to (of 2^(c (x - ref)) where b is large; z NaN where a kept
// logit is a NaN or +infinity); and the split's n_out best (logit, token) pairs in
// falling order, token -1 filling the places left.
struct BeamStat {
    float z, lost, m, ref, b;
};
struct BeamCand {
    float x;
    int tok;
};

struct BeamArgs {
    const void *logits;
    int64_t row_stride;
    int dtype, batch, beams, vocab, n_out;
    int n_split, split_len; // tokens a split has (the last one less)
    int cap, depth;         // keys the rows kernel's buffer holds, the merge's of each split's list
    float c;                // log2(e) / T
    double inv_t;           // 1 / T
    const uint32_t *allow;
    int64_t allow_stride;
    const float *scores;
    const uint8_t *finished;
    int end_token;
    const int32_t *lengths;
    double length_alpha;
    int32_t *parent_out;
    int64_t *token_out;
    float *score_out;
    uint8_t *finished_out;
    int32_t *length_out;
    float *lse_out;
    BeamStat *stat;         // [rows][n_split]
    BeamCand *cand;         // [rows][n_split][n_out]
    int *next;              // the rows kernel's next item: 0 between calls
    int *err;               // the header's error word (expired waits)
    int *fault;
};

int beam_splits(int64_t rows, int64_t vocab);
int beam_cap(int dtype, int n_out);
cudaError_t launch_beam_rows(const BeamArgs &a, cudaStream_t st);
cudaError_t launch_beam_merge(const BeamArgs &a, cudaStream_t st);
cudaError_t launch_beam_gather(int64_t n_group, int64_t n_src, int64_t n_dst, int64_t row_bytes,
                               const int32_t *parent, const void *src, void *dst, int *fault, cudaStream_t st);

// ---- cache pages -----------------------------------------------------------------
struct ForkArgs {
    int n_group, n_src, n_dst, max_pages, page, n_pages;
    const int32_t *parent, *table, *lens;
    int64_t table_stride, table_out_stride;
    int32_t *ref, *table_out, *lens_out;
    int *fault;
};

struct SharerSlot {
    int page, count, top;
};
struct ReserveArgs {
    int n_seq, max_pages, page, n_pages, n_new_all;
    const int32_t *n_new, *lens;
    int32_t *table, *ref;
    int64_t table_stride;
    SharerSlot *hash;       // a power of two of slots, at least 2 n_seq
    int hash_mask;
    int4 *need;             // [n_seq]
    int32_t *free_list;     // [n_pages]
    int2 *moves;            // pages to copy (from, to) and their number
    int *n_copy;
    int *fault;
};

struct CopyArgs {
    char *pool;
    int64_t plane_stride, page_stride, page_bytes;   // bytes
    int n_planes, n_pages;
    const int2 *moves;      // or src and dst
    const int32_t *src, *dst;
    int64_t n;
    const int *n_dev;       // the number of moves where it is the device's (else n)
    int *fault;
};

struct FreeArgs {
    int n_seq, max_pages, page, n_pages;
    const uint8_t *drop;
    int32_t *table, *lens, *ref;
    int64_t table_stride;
    int *fault;
};

struct CompactArgs {
    int n_seq, max_pages, page, n_pages;
    const int32_t *table, *lens, *ref;
    int64_t table_stride, table_out_stride;
    int32_t *table_out, *ref_out, *n_live_out;
    int32_t *new_id;        // [n_pages]: a mover's new id
    int2 *moves;
    int *n_copy;
    int *fault;
};

struct WriteArgs {
    int64_t n_tok;
    int n_seq, n_kv, row_bytes, page, n_pages, max_pages;
    const char *k_new, *v_new;
    int64_t k_row, v_row;                                   // bytes from token to token
    char *k, *v;
    int64_t k_page, k_tok, k_head, v_page, v_tok, v_head;   // bytes
    const int32_t *table, *lens, *first;
    int64_t table_stride;
    int *fault;
};

cudaError_t launch_cache_fork(const ForkArgs &a, cudaStream_t st);
cudaError_t launch_cache_plan(const ReserveArgs &a, cudaStream_t st);
// most: the largest number of moves there can be
cudaError_t launch_cache_copy(const CopyArgs &a, int64_t most, cudaStream_t st);
cudaError_t launch_cache_free(const FreeArgs &a, cudaStream_t st);
cudaError_t launch_cache_rank(const CompactArgs &a, cudaStream_t st);
cudaError_t launch_cache_move(const CompactArgs &a, const CopyArgs &c, cudaStream_t st);
// word: bytes of the widest access every row allows (16, 4 or 2)
cudaError_t launch_cache_write(const WriteArgs &a, int word, cudaStream_t st);

// ---- paged attention ---------------------------------------------------------------
struct AttnArgs {
    int n_group, share, n_q, n_kv, group, hd;      // group: query heads per KV head
    int max_pages, page, n_pages;
    int window;                                    // 0: none
    float scale_log2;                              // scale * log2(e)
    const void *q, *k, *v;
    int64_t q_stride;                              // elements between sequences
    int64_t page_stride, tok_stride, head_stride;  // elements
    const int32_t *table, *lens;
    int64_t table_stride;
    void *out;
    float *lse;
    int kt, mr;                                    // tokens per unit, query rows per item
    int cs, cp;                                    // items per KV head: of a group's shared part, of a sequence
    int ra, rb;                                    // rows a partial result holds, shared and private
    int nw;                                        // runs at most
    int32_t *shared;                               // [n_group] shared tokens
    long long *base;                               // [n_group + 1] units before each group, where attn_plan leaves them
    int2 *runs_a, *runs_b;                         // per item of a group's shared part, of a sequence: first run, runs
    float *part_a, *part_b;                        // partial results per row: o[hd], m (log2 units), l, and 2 unused
    int *fault;
};

// The kernel that takes this type, head size and number of query rows per KV
// head: rows per item, tokens per unit, runs a block walks (one block per SM).
struct AttnShape {
    int mr, kt, runs;
};
constexpr int ATTN_MAX_ROWS = 152 * 12 * 16;       // runs x rows per item: a block has at most 12 warps of 16 rows
constexpr int ATTN_ROW = 4;            // floats a partial row holds beside o
AttnShape attn_shape(int dtype, int hd, int rows);
// Whether the split pass needs attn_share, and attn_plan, ahead of it.
bool attn_shares(const AttnArgs &a);
bool attn_plans(const AttnArgs &a);
cudaError_t launch_attn_share(const AttnArgs &a, cudaStream_t st);
cudaError_t launch_attn_plan(const AttnArgs &a, cudaStream_t st);
cudaError_t launch_attn(int dtype, const AttnArgs &a, cudaStream_t st);
// The tensor-core kernel (16-bit types) and the CUDA-core one (fp32).
AttnShape attn_ffma_shape(int hd, int rows);
cudaError_t launch_attn_ffma(const AttnArgs &a, cudaStream_t st);
AttnShape attn_mma_shape(int hd, int rows);
cudaError_t launch_attn_mma(bool f16, const AttnArgs &a, cudaStream_t st);
cudaError_t launch_attn_join(int dtype, const AttnArgs &a, cudaStream_t st);

} // namespace lossk
