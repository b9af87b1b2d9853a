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
// What the rows kernel leaves per (row, split): the largest kept logit m, the
// sum z of exp((x - m) / T) over the kept logits (NaN where one of them is a NaN
// or +infinity), and the split's n_out best (logit, token) pairs in any order,
// token -1 filling the places left.
struct BeamStat {
    double z;
    float m;
    int pad;
};
struct BeamCand {
    float x;
    int tok;
};

struct BeamArgs {
    const void *logits;
    int64_t row_stride;
    int batch, beams, vocab, n_out, n_split;
    float c_hi, c_lo;       // log2(e) / T as the sum of two floats
    double temperature;
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
    int *fault;
};

// Splits of a row: enough blocks for every SM, no split below 4096 tokens.
int beam_splits(int64_t rows, int64_t vocab);
cudaError_t launch_beam_rows(int dtype, const BeamArgs &a, cudaStream_t st);
cudaError_t launch_beam_merge(const BeamArgs &a, cudaStream_t st);
cudaError_t launch_beam_gather(int64_t n_group, int64_t n_src, int64_t n_dst, int64_t row_bytes,
                               const int32_t *parent, const void *src, void *dst, int *fault, cudaStream_t st);

} // namespace lossk
