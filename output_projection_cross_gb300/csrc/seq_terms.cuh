// seq_terms.cuh -- the sequence losses' arithmetic per row, sequence and pair, and
// their scalars: device code that the coefficient kernel (k_seq.cu) and the passes over
// given logits (k_rows.cu) share.
#pragma once
#include "../../include/lossk.h"
#include "seq_internal.h"

namespace lossk {

__device__ __forceinline__ bool seq_refused(const WsHeader *hdr)
{
    return *reinterpret_cast<const volatile int *>(&hdr->bad_targets) != 0;
}

// log2 z to 2^-24 or so, of whatever size it is (log2f keeps that many of its own bits, 2^-18 at 64).
__device__ __forceinline__ double log2_of(float z)
{
    int e;
    const float f = frexpf(z, &e);
    return static_cast<double>(e) + static_cast<double>(log2f(f));
}

// ln 2 ((y - M) k2 - log2 z) - low, rounded once: a row's log-probability from its target's logit y, its
// largest logit M and the sum z.  Floats with their rounding errors carried along (Knuth's and Dekker's exact
// sums and products); doubles, a sixty-fourth as fast here and one after another in every row's chain,
// where those leave their range.
__device__ __forceinline__ float logp_of(float y, float M, float k2, float z, float low)
{
    const float d = y - M, b = d - y, d_low = (y - (d - b)) - (M + b);
    const float p = d * k2;
    if (!(p >= -0x1p40f && d >= -0x1p80f))
        return static_cast<float>(((static_cast<double>(y) - static_cast<double>(M)) * static_cast<double>(k2) - log2_of(z)) * LN2 -
                                  static_cast<double>(low));
    const float p_low = fmaf(d, k2, -p) + d_low * k2;
    int e;
    const float l = log2f(frexpf(z, &e)), fe = static_cast<float>(e);
    const float s = p - fe, c = s - p, s_low = (p - (s - c)) - (fe + c);
    constexpr float LN2F = static_cast<float>(LN2), LN2_LOW = static_cast<float>(LN2 - static_cast<double>(LN2F));
    return fmaf(s, LN2F, fmaf(s, LN2_LOW, fmaf(s_low + p_low - l, LN2F, -low)));
}

// What a log-probability is given back where the sum z of terms relative to the largest went through
// `exps` exponentials, that one's own terms aside.
__device__ __forceinline__ float ex2_low(float z, int exps) { return exps * static_cast<float>(EX2_LOW) * (1.f - 1.f / z); }

__device__ __forceinline__ int slots_before(int slot) { return slot < 0 ? ~slot : slot; }

// A counted row's weight in the mean: n_s its sequence's counted tokens.
__device__ __forceinline__ float row_weight(const SeqLoss &l, const WsHeader *hdr, int n_s)
{
    const bool sum = l.flags & LOSSK_REDUCE_SUM;
    if (l.flags & LOSSK_SEQ_MEAN)
        return sum ? 1.f / static_cast<float>(n_s)
                   : 1.f / (static_cast<float>(n_s) * static_cast<float>(hdr->pad[HDR_GROUPS]));
    return sum ? 1.f : 1.f / static_cast<float>(hdr->n_valid);
}

struct PolicyTerm {
    float loss, slope;      // P and dP / d(log ratio)
    bool clipped;
};

// log ratio `delta` (exp in float or, for ratios of sequences a few 1e-4 from 1, in double)
template <typename F> __device__ __forceinline__ PolicyTerm policy_term(const SeqLoss &l, F delta, float A)
{
    if (A == 0.f) return PolicyTerm{0.f, 0.f, false};
    const F r = exp(delta);
    const F edge = A > 0.f ? F(1) + static_cast<F>(l.high) : F(1) - static_cast<F>(l.low);
    const bool out = A > 0.f ? r > edge : r < edge;
    return PolicyTerm{static_cast<float>(-A * (out ? edge : r)), out ? 0.f : static_cast<float>(-A * r), out};
}

__device__ __forceinline__ float advantage(const SeqLoss &l, int row, int seq)
{
    return l.adv[(l.flags & LOSSK_SEQ_ADVANTAGES) ? seq : row];
}

// What a row leaves behind: its coefficient, and its terms of the three sums that the
// scalars are made of.
struct RowTerms {
    float coef, v[3];
};

// a_t from d total / d logp.
__device__ __forceinline__ float coefficient(const SeqLoss &l, float d_lp)
{
    return d_lp * l.per_t * l.per_t_up * l.per_t_up;
}

// What the policy loss reads for row t of sequence s (of n_s counted tokens).
struct RowInputs {
    float weight, adv, old, ref;
};
__device__ __forceinline__ RowInputs policy_inputs(const SeqLoss &l, const WsHeader *hdr, int t, int s, int n_s)
{
    return RowInputs{row_weight(l, hdr, n_s), advantage(l, t, s), l.old ? l.old[t] : 0.f, l.ref ? l.ref[t] : 0.f};
}

// Row t, counted, with log-probability lp.  By sequence (LOSSK_SEQ_RATIO): the log ratio
// `delta` of its sequence and what each token's logp moves the sequence's terms by, `slope`.
// write: the row's loss goes out.
__device__ __forceinline__ RowTerms policy_row(const SeqLoss &l, const RowInputs &in, int t, float lp, double delta,
                                               float slope, bool write = true)
{
    const float weight = in.weight, A = in.adv;
    PolicyTerm p;
    float d_lp;                                            // d total / d logp
    if (l.flags & LOSSK_SEQ_RATIO) {
        p = policy_term<double>(l, delta, A);
        d_lp = slope;
    } else {
        p = policy_term<float>(l, l.old ? lp - in.old : 0.f, A);
        d_lp = weight * p.slope;
    }
    float kl = 0.f, loss = p.loss;
    if (l.ref) {
        const float q = in.ref - lp, e = expm1f(q);
        kl = e == INFINITY ? e : e - q;                    // (of a token of probability 0: infinity, not infinity less itself)
        if (l.kl > 0.f) {
            loss = fmaf(l.kl, kl, loss);
            d_lp = fmaf(-l.kl * weight, e, d_lp);
        }
    }
    if (write && l.per_token) l.per_token[t] = loss;
    return RowTerms{coefficient(l, d_lp), {weight * p.loss, weight * kl, p.clipped ? weight : 0.f}};
}

__device__ __forceinline__ float softplus(float x) { return fmaxf(x, 0.f) + log1pf(expf(-fabsf(x))); }

// A pair's loss and d loss / du.
__device__ __forceinline__ void pair_term(const SeqLoss &l, double u, float &loss, float &slope)
{
    if (l.objective == LOSSK_PREF_SQUARED) {
        const float g = static_cast<float>(u - 0.5 / static_cast<double>(l.beta));
        loss = g * g;
        slope = 2.f * g;
        return;
    }
    const float h = static_cast<float>(static_cast<double>(l.beta) * u - static_cast<double>(l.margin));
    if (l.objective == LOSSK_PREF_HINGE) {
        loss = h >= 1.f ? 0.f : 1.f - h;
        slope = h >= 1.f ? 0.f : -l.beta;
    } else {
        loss = (1.f - l.smooth) * softplus(-h);
        if (l.smooth > 0.f) loss += l.smooth * softplus(h);
        slope = l.beta * (l.smooth / (1.f + expf(-h)) - (1.f - l.smooth) / (1.f + expf(h)));
    }
}

// A row of a pair of slope `slope` (0 where the pair does not count), n_s counted tokens in
// its sequence.
__device__ __forceinline__ RowTerms pair_row(const SeqLoss &l, const WsHeader *hdr, bool chosen, int n_s, float slope,
                                             float lp)
{
    const bool sum = l.flags & LOSSK_REDUCE_SUM;
    float d_lp = chosen ? slope : -slope;
    if (l.flags & LOSSK_LENGTH_MEAN) d_lp /= static_cast<float>(n_s);
    if (!sum && slope != 0.f) d_lp /= static_cast<float>(hdr->pad[HDR_GROUPS]);
    if (chosen && l.nll > 0.f) d_lp -= l.nll / (sum ? 1.f : static_cast<float>(hdr->pad[HDR_CHOSEN]));
    return RowTerms{coefficient(l, d_lp), {chosen ? -lp : 0.f, 0.f, 0.f}};
}

// The record that the passes over the logits read: {reference, a share, a, target}, where share
// 2^(x log2 e - reference) is a probability (given logits: share 2^(k2 (s - reference)), the reference
// being the largest of them); a row without any probability gets a zero gradient.
__device__ __forceinline__ float4 row_params(float ref, float share, float coef, int64_t y)
{
    const bool none = ref == -INFINITY && share == share;
    const float a = none ? 0.f : coef;
    return make_float4(none ? 0.f : ref, none ? 0.f : a * share, a, __int_as_float(static_cast<int>(y)));
}

// The scalars from their three sums.
__device__ __forceinline__ void write_scalars(const SeqLoss &l, const WsHeader *hdr, double v0, double v1, double v2)
{
    float *o = l.scalars;
    if (l.pairs > 0) {
        const int pairs = hdr->pad[HDR_GROUPS], chosen = hdr->pad[HDR_CHOSEN];
        if (!(l.flags & LOSSK_REDUCE_SUM)) {
            v0 = chosen > 0 ? v0 / chosen : 0.0;
            v1 = pairs > 0 ? v1 / pairs : 0.0;
            v2 = pairs > 0 ? v2 / pairs : 0.0;
        }
        // (without the likelihood term its infinities stay out of the total)
        o[0] = static_cast<float>(l.nll > 0.f ? v1 + static_cast<double>(l.nll) * v0 : v1);
        o[1] = static_cast<float>(v1);
        o[2] = static_cast<float>(v0);
        o[3] = static_cast<float>(v2);
    } else {
        o[0] = static_cast<float>(l.kl > 0.f ? v0 + static_cast<double>(l.kl) * v1 : v0);
        o[1] = static_cast<float>(v0);
        o[2] = static_cast<float>(v1);
        o[3] = static_cast<float>(v2);
    }
}

// From the coefficient kernel's blocks' sums, every T-th by a thread in their order, then a
// fixed tree.  All T threads of one block; no barrier is needed after it.
template <int T> __device__ __forceinline__ void seq_scalars(const SeqLoss &l, const SeqScratch &w)
{
    __shared__ double sh[3][T / 32];
    const int n = l.n_tok > l.n_seq ? l.n_tok : l.n_seq, blocks = (n + COEF_T - 1) / COEF_T;
    double v[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        v[k] = 0.0;
        for (int b = threadIdx.x; b < blocks; b += T) v[k] += w.acc[k * static_cast<int64_t>(blocks) + b];
        for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
        if ((threadIdx.x & 31) == 0) sh[k][threadIdx.x >> 5] = v[k];
    }
    __syncthreads();
    if (threadIdx.x != 0) return;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        v[k] = sh[k][0];
        for (int i = 1; i < T / 32; ++i) v[k] += sh[k][i];
    }
    write_scalars(l, w.hdr, v[0], v[1], v[2]);
}

// The sum of a value over the block's threads, in a fixed tree.  sh: a double per warp.
__device__ __forceinline__ double block_sum(double v, double *sh)
{
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    v = sh[0];
    for (unsigned i = 1; i < blockDim.x / 32; ++i) v += sh[i];
    return v;
}

} // namespace lossk
