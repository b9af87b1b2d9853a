// k_beam.cu -- beam search's selection over beams and vocabulary, and the
// reordering of states by parent.
//
//   beam_rows    per (row, split of the vocabulary): the statistics of the
//                log-sum-exp and the split's n_out best logits
//   beam_merge   per batch entry: log-sum-exps, scores, ranks, the n_out best
//   beam_gather  rows of a state by parent
//
// Within a row the candidates' order is the logits' (the log-sum-exp and the
// beam's score are constants of the row), so the rows kernel never needs a
// score; only the few survivors get one, in double, because candidates of
// different beams may lie closer together than floats resolve.
#include "../../include/lossk.h"
#include "decode_internal.h"
#include "ptx.cuh"

namespace lossk {

namespace {

constexpr int ROW_THREADS = 256;
constexpr int MERGE_THREADS = 256;

__device__ __forceinline__ float beam_f(float x) { return x + 0.f; }   // -0 to +0: they tie
__device__ __forceinline__ float beam_f(uint16_t x) { return __uint_as_float(static_cast<uint32_t>(x) << 16) + 0.f; }
__device__ __forceinline__ float beam_f(h16_t x) { return f16_to_f(x.bits) + 0.f; }

// A float's order as an unsigned integer's (no NaN).
__device__ __forceinline__ uint32_t order_of(float x)
{
    const uint32_t b = __float_as_uint(x);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o)
{
    return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}

// (logit, token) as one key: the larger logit first, then the lower token.
// 0 is below every key of a logit above -infinity.
__device__ __forceinline__ uint64_t key_of(float x, int tok)
{
    return (static_cast<uint64_t>(order_of(x)) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(tok));
}

// Whether beam k of entry b has logits to read: not finished, a finite score.
__device__ __forceinline__ bool beam_reads(const BeamArgs &a, int r)
{
    return !(a.finished && a.finished[r]) && isfinite(a.scores[r]);
}

template <typename T>
__global__ void __launch_bounds__(ROW_THREADS) beam_rows_kernel(BeamArgs a)
{
    __shared__ uint64_t s_key[ROW_THREADS / 32];
    __shared__ double s_z[ROW_THREADS / 32];
    __shared__ float s_m[ROW_THREADS / 32];
    const int r = blockIdx.x, split = blockIdx.y, t = threadIdx.x;
    if (!beam_reads(a, r)) return;
    const T *row = static_cast<const T *>(a.logits) + r * a.row_stride;
    const uint32_t *allow = a.allow ? a.allow + r * a.allow_stride : nullptr;
    const int v0 = static_cast<int>(static_cast<int64_t>(a.vocab) * split / a.n_split);
    const int v1 = static_cast<int>(static_cast<int64_t>(a.vocab) * (split + 1) / a.n_split);
    auto kept = [&](int v) { return !allow || ((allow[v >> 5] >> (v & 31)) & 1u); };

    float m = -INFINITY;
    bool bad = false;
    for (int v = v0 + t; v < v1; v += ROW_THREADS)
        if (kept(v)) {
            const float x = beam_f(row[v]);
            bad |= !(x < INFINITY);
            m = fmaxf(m, x);
        }
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    if ((t & 31) == 0) s_m[t >> 5] = m;
    bad = __syncthreads_or(bad);
    m = s_m[0];
    for (int i = 1; i < ROW_THREADS / 32; ++i) m = fmaxf(m, s_m[i]);

    BeamStat *stat = a.stat + static_cast<int64_t>(r) * a.n_split + split;
    BeamCand *cand = a.cand + (static_cast<int64_t>(r) * a.n_split + split) * a.n_out;
    if (bad) {
        if (t == 0) *stat = BeamStat{NAN, 0.f, 0};
        return;
    }
    double z = 0.0;
    for (int v = v0 + t; v < v1; v += ROW_THREADS)
        if (kept(v)) {
            const float d = beam_f(row[v]) - m;
            if (m > -INFINITY) z += exp2f(fmaf(d, a.c_hi, d * a.c_lo));
        }
    for (int o = 16; o; o >>= 1) z += __shfl_xor_sync(0xFFFFFFFFu, z, o);
    if ((t & 31) == 0) s_z[t >> 5] = z;
    __syncthreads();
    if (t == 0) {
        for (int i = 1; i < ROW_THREADS / 32; ++i) z += s_z[i];
        *stat = BeamStat{z, m, 0};
    }
    // n_out rounds, each the largest key below the last one's
    uint64_t last = ~0ull;
    for (int j = 0; j < a.n_out; ++j) {
        uint64_t best = 0;
        if (last)
            for (int v = v0 + t; v < v1; v += ROW_THREADS)
                if (kept(v)) {
                    const float x = beam_f(row[v]);
                    const uint64_t k = key_of(x, v);
                    if (x > -INFINITY && k < last && k > best) best = k;
                }
        for (int o = 16; o; o >>= 1) {
            const uint64_t other = __shfl_xor_sync(0xFFFFFFFFu, best, o);
            best = other > best ? other : best;
        }
        __syncthreads();
        if ((t & 31) == 0) s_key[t >> 5] = best;
        __syncthreads();
        for (int i = 0; i < ROW_THREADS / 32; ++i) best = s_key[i] > best ? s_key[i] : best;
        if (t == 0)
            cand[j] = best ? BeamCand{value_of(static_cast<uint32_t>(best >> 32)),
                                      static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(best))}
                           : BeamCand{0.f, -1};
        last = best;
    }
}

struct Ranked {
    double rank;
    int64_t flat;   // beam * vocab + token; -1: none
};
__device__ __forceinline__ bool better(const Ranked &x, const Ranked &y)
{
    if (x.flat < 0 || y.flat < 0) return x.flat >= 0 && y.flat < 0;
    return x.rank > y.rank || (x.rank == y.rank && x.flat < y.flat);
}

__global__ void __launch_bounds__(MERGE_THREADS) beam_merge_kernel(BeamArgs a)
{
    __shared__ double s_lse[LOSSK_BEAM_MAX_BEAMS], s_div[LOSSK_BEAM_MAX_BEAMS];
    __shared__ int s_kind[LOSSK_BEAM_MAX_BEAMS];       // 0: no candidates, 1: its own (finished), 2: the row's
    __shared__ Ranked s_best[MERGE_THREADS / 32];
    __shared__ double s_score[MERGE_THREADS / 32];
    const int b = blockIdx.x, t = threadIdx.x;
    for (int k = t; k < a.beams; k += MERGE_THREADS) {
        const int r = b * a.beams + k;
        const float start = a.scores[r];
        const bool done = a.finished && a.finished[r];
        int kind = done ? 1 : 2;
        double lse = -INFINITY;
        if (!isfinite(start)) {
            if (start != -INFINITY) raise_fault(a.fault, LOSSK_NON_FINITE_SCALAR);
            kind = 0;
        }
        if (kind == 2) {
            const BeamStat *st = a.stat + static_cast<int64_t>(r) * a.n_split;
            float m = -INFINITY;
            for (int i = 0; i < a.n_split; ++i) m = fmaxf(m, st[i].m);
            double z = 0.0;
            for (int i = 0; i < a.n_split; ++i)
                if (st[i].z != 0.0)
                    z += st[i].z * exp((static_cast<double>(st[i].m) - static_cast<double>(m)) / a.temperature);
            if (isnan(z)) raise_fault(a.fault, LOSSK_NON_FINITE_SCALAR);
            if (z > 0.0) lse = static_cast<double>(m) / a.temperature + log(z);
            else kind = 0;
        }
        if (a.lse_out) a.lse_out[r] = static_cast<float>(lse);
        const int len = (a.lengths ? a.lengths[r] : 0) + (done ? 0 : 1);
        s_lse[k] = lse;
        s_div[k] = a.length_alpha == 0.0 ? 1.0 : pow(static_cast<double>(len > 1 ? len : 1), a.length_alpha);
        s_kind[k] = kind;
    }
    __syncthreads();
    const int per_row = a.n_split * a.n_out;
    Ranked last{INFINITY, -1};
    for (int j = 0; j < a.n_out; ++j) {
        Ranked best{0.0, -1};
        double score = 0.0;
        for (int i = t; i < a.beams * per_row; i += MERGE_THREADS) {
            const int k = i / per_row, r = b * a.beams + k;
            Ranked c{0.0, -1};
            double s = a.scores[r];
            if (s_kind[k] == 1 && i % per_row == 0) {
                c.flat = static_cast<int64_t>(k) * a.vocab + (a.end_token < 0 ? 0 : a.end_token);
            } else if (s_kind[k] == 2) {
                const BeamCand q = a.cand[static_cast<int64_t>(r) * per_row + i % per_row];
                if (q.tok >= 0) c.flat = static_cast<int64_t>(k) * a.vocab + q.tok;
                s += static_cast<double>(q.x) / a.temperature - s_lse[k];
            }
            c.rank = s / s_div[k];
            if (c.flat >= 0 && (j == 0 || better(last, c)) && better(c, best)) {
                best = c;
                score = s;
            }
        }
        for (int o = 16; o; o >>= 1) {
            Ranked c{__shfl_xor_sync(0xFFFFFFFFu, best.rank, o), __shfl_xor_sync(0xFFFFFFFFu, best.flat, o)};
            const double s = __shfl_xor_sync(0xFFFFFFFFu, score, o);
            if (better(c, best)) {
                best = c;
                score = s;
            }
        }
        __syncthreads();
        if ((t & 31) == 0) {
            s_best[t >> 5] = best;
            s_score[t >> 5] = score;
        }
        __syncthreads();
        for (int i = 0; i < MERGE_THREADS / 32; ++i)
            if (better(s_best[i], best)) {
                best = s_best[i];
                score = s_score[i];
            }
        if (t == 0) {
            const int64_t o = static_cast<int64_t>(b) * a.n_out + j;
            const bool any = best.flat >= 0;
            const int k = any ? static_cast<int>(best.flat / a.vocab) : 0;
            const int r = b * a.beams + k;
            const bool was = any && s_kind[k] == 1;
            const int64_t tok = was ? a.end_token : best.flat - static_cast<int64_t>(k) * a.vocab;
            a.parent_out[o] = any ? k : -1;
            a.token_out[o] = any ? tok : -1;
            a.score_out[o] = any ? static_cast<float>(score) : -INFINITY;
            if (a.finished_out) a.finished_out[o] = any && (was || tok == a.end_token);
            if (a.length_out) a.length_out[o] = any ? (a.lengths ? a.lengths[r] : 0) + (was ? 0 : 1) : 0;
        }
        if (best.flat < 0) {
            // the places left
            for (int i = j + 1 + t; i < a.n_out; i += MERGE_THREADS) {
                const int64_t o = static_cast<int64_t>(b) * a.n_out + i;
                a.parent_out[o] = -1;
                a.token_out[o] = -1;
                a.score_out[o] = -INFINITY;
                if (a.finished_out) a.finished_out[o] = 0;
                if (a.length_out) a.length_out[o] = 0;
            }
            return;
        }
        last = best;
    }
}

template <typename V>
__global__ void beam_gather_kernel(int64_t n_src, int64_t n_dst, int64_t words, const int32_t *__restrict__ parent,
                                   const V *__restrict__ src, V *__restrict__ dst, int *fault)
{
    const int64_t j = blockIdx.x, g = j / n_dst;
    const int p = parent[j];
    const bool ok = p >= 0 && p < n_src;
    if (!ok && p != -1 && threadIdx.x == 0 && blockIdx.y == 0) raise_fault(fault, LOSSK_TARGET_OUT_OF_RANGE);
    const V *s = src + (g * n_src + (ok ? p : 0)) * words;
    V *d = dst + j * words;
    for (int64_t i = static_cast<int64_t>(blockIdx.y) * blockDim.x + threadIdx.x; i < words;
         i += static_cast<int64_t>(gridDim.y) * blockDim.x)
        d[i] = ok ? s[i] : V{};
}

} // namespace

int beam_splits(int64_t rows, int64_t vocab)
{
    const int64_t want = (2 * 152 + rows - 1) / rows, most = (vocab + 4095) / 4096;
    const int64_t n = want < most ? want : most;
    return static_cast<int>(n < 1 ? 1 : n > 64 ? 64 : n);
}

cudaError_t launch_beam_rows(int dtype, const BeamArgs &a, cudaStream_t st)
{
    const dim3 grid(static_cast<unsigned>(a.batch) * a.beams, a.n_split);
    if (dtype == LOSSK_F32) beam_rows_kernel<float><<<grid, ROW_THREADS, 0, st>>>(a);
    else if (dtype == LOSSK_BF16) beam_rows_kernel<uint16_t><<<grid, ROW_THREADS, 0, st>>>(a);
    else beam_rows_kernel<h16_t><<<grid, ROW_THREADS, 0, st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_beam_merge(const BeamArgs &a, cudaStream_t st)
{
    beam_merge_kernel<<<static_cast<unsigned>(a.batch), MERGE_THREADS, 0, st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_beam_gather(int64_t n_group, int64_t n_src, int64_t n_dst, int64_t row_bytes,
                               const int32_t *parent, const void *src, void *dst, int *fault, cudaStream_t st)
{
    const uintptr_t all = reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(dst) |
                          static_cast<uintptr_t>(row_bytes);
    const int64_t unit = all % 16 == 0 ? 16 : all % 4 == 0 ? 4 : 1, words = row_bytes / unit;
    // a row is cut into blocks of about 16 elements a thread, at most 64 of them
    const int64_t cut = (words + 256 * 16 - 1) / (256 * 16);
    const dim3 grid(static_cast<unsigned>(n_group * n_dst), static_cast<unsigned>(cut > 64 ? 64 : cut));
    if (unit == 16)
        beam_gather_kernel<uint4><<<grid, 256, 0, st>>>(n_src, n_dst, words, parent, static_cast<const uint4 *>(src),
                                                        static_cast<uint4 *>(dst), fault);
    else if (unit == 4)
        beam_gather_kernel<uint32_t><<<grid, 256, 0, st>>>(n_src, n_dst, words, parent,
                                                           static_cast<const uint32_t *>(src),
                                                           static_cast<uint32_t *>(dst), fault);
    else
        beam_gather_kernel<uint8_t><<<grid, 256, 0, st>>>(n_src, n_dst, words, parent,
                                                          static_cast<const uint8_t *>(src),
                                                          static_cast<uint8_t *>(dst), fault);
    return cudaGetLastError();
}

} // namespace lossk
