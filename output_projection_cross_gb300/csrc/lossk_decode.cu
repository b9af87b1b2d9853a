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

// 581 or 583 for the first size outside [1, most].
int32_t size_check(int64_t v, int64_t most)
{
    return v < 1 ? LOSSK_EMPTY_DIMENSION : v > most ? LOSSK_DIMENSION_TOO_LARGE : LOSSK_OK;
}

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
        if (size_check(a, MAX_DIM) != LOSSK_OK || size_check(b, MAX_DIM) != LOSSK_OK) return -1;
        return 256;
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
    if (!std::isfinite(temperature) || temperature <= 0.0 || !std::isfinite(length_alpha)) return LOSSK_NON_FINITE_SCALAR;
    if (end_token < -1 || end_token >= vocab) return LOSSK_TARGET_OUT_OF_RANGE;

    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const double c = LOG2E / temperature;
    BeamArgs a{};
    a.logits = logits;
    a.row_stride = row_stride;
    a.batch = static_cast<int>(batch);
    a.beams = static_cast<int>(beams);
    a.vocab = static_cast<int>(vocab);
    a.n_out = static_cast<int>(n_out);
    a.n_split = L.n_split;
    a.c_hi = static_cast<float>(c);
    a.c_lo = static_cast<float>(c - static_cast<double>(a.c_hi));
    a.temperature = temperature;
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
    a.fault = fault_of(workspace);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    {
        Launch k(KK_BEAM_ROWS, st);
        if (launch_beam_rows(dtype, a, st) != cudaSuccess) return LOSSK_DEVICE_ERROR;
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

} // extern "C"
