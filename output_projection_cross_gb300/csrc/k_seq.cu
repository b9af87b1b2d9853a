// k_seq.cu -- the losses of sampled and compared sequences, all but their
// passes over logits: which rows count, log-probabilities from the passes'
// partial sums, sums over sequences, each row's loss and coefficient, the
// scalars, d_hidden from its partials.
//
// With x = s / T, logp_t = x_{t,y} - lse(x_t), every loss here is a function
// of the logp of the counted rows, so ds_t = a_t (softmax(x_t) - onehot_y), a_t =
// -grad_scale (d total / d logp_t) / T: one coefficient per row joins the loss to
// the passes over the logits.  These kernels handle a few floats per row; what
// bounds them is latency, one launch after another, so each starts while the
// one ahead of it ends (decode_launch.h).
#include "../../include/lossk.h"
#include "decode_internal.h"
#include "decode_launch.h"
#include "ptx.cuh"
#include "seq_terms.cuh"

#include <cfloat>
#include <type_traits>

namespace lossk {

namespace {

// The sequence that holds slot c: the last one whose slots start at or before it.  The
// whole warp calls it, each step reads 32 of the starts (a thread of its own would wait
// for log2 n_seq loads, one after another); slots rise from lane to lane, c < 0: none.  A lane
// behind the first goes on from there in doubling steps: one or none as a rule, but millions of
// sequences without a counted token may lie between (walked one by one, 1.3 s for 2^25).
__device__ __forceinline__ int seq_of(const int *seq_slot, int n_seq, int c, int lane)
{
    const unsigned some = __ballot_sync(0xffffffffu, c >= 0);
    if (!some) return 0;
    const int c0 = __shfl_sync(0xffffffffu, c, __ffs(some) - 1);
    int lo = 0, hi = n_seq;                                // the first slot's is in [lo, hi)
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) >> 5;
        const int at = lo + lane * step;
        const bool le = at < hi && seq_slot[at] <= c0;
        const int k = 31 - __clz(__ballot_sync(0xffffffffu, le) | 1u);
        lo += k * step;
        hi = min(hi, lo + step);
    }
    int s = lo, step = 1;
    while (s + step < n_seq && seq_slot[s + step] <= c) {
        s += step;
        step *= 2;
    }
    for (step /= 2; step > 0; step /= 2)
        if (s + step < n_seq && seq_slot[s + step] <= c) s += step;
    return s;
}

// The passes from hidden rows scale fp32 logits: the scaled ones' last bit is 2^6 at 2^30, and above that
// 2^(x log2 e - lse2) leaves fp32's range whatever x.  No number then, rather than one that means nothing.
__device__ __forceinline__ double lse2_or_nan(double lse2) { return fabs(lse2) <= 0x1p30 || lse2 == -INFINITY ? lse2 : NAN; }

__device__ __forceinline__ void put_lse2(const SeqScratch &w, int c, double lse2)
{
    const float ref = static_cast<float>(lse2);
    w.ref[c] = ref;
    w.share[c] = fabsf(ref) <= FLT_MAX ? exp2f(static_cast<float>(static_cast<double>(ref) - lse2)) : 1.f;
}

} // namespace

// One block: a prefix sum over the rows, 8192 in a round, in order, so that slots, and
// with them the order of every sum, are a function of the mask alone.  A chain of
// latencies: masks, targets and the sequences' ends are all asked for at once, before
// any of them is known to matter.  A warp's rows are consecutive, so that what it
// writes is too (eight rows in a row per thread took 25 us for 8192 rows, most of it
// stores of 32 sectors each).
constexpr int PREP_T = 1024, PREP_PER = 8;
__global__ void __launch_bounds__(PREP_T) seq_prep_kernel(const SeqLoss l, const SeqScratch w)
{
    wait_for_stream();
    let_next_start();
    static_assert(PREP_PER * 32 == 256, "a lane of a warp scans eight of the counts");
    __shared__ int s_count[PREP_PER * 32];
    __shared__ int s_groups;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int n = l.n_tok;
    // (what an earlier call left in the error or the fault word stays until lossk_device_status has
    // read it: refused)
    bool bad = *reinterpret_cast<volatile int *>(&w.hdr->err) != 0 ||
               is_fault(*reinterpret_cast<volatile int *>(&w.hdr->pad[HDR_FAULT]));
    unsigned on;
    int64_t y[PREP_PER];
    auto load = [&](int t0) {
        on = 0;
#pragma unroll
        for (int i = 0; i < PREP_PER; ++i) {
            const int r = t0 + i * PREP_T + tid;
            y[i] = r < n ? l.targets[r] : 0;
            on |= (r < n && (!l.mask || l.mask[r] != 0) ? 1u : 0u) << i;
        }
    };
    load(0);
    bool range = false;
    int lo = 0, hi = n, first0 = 0, first1 = 0;            // of sequence tid
    if (l.first) {
        lo = l.first[0];
        hi = l.first[l.n_seq];
        for (int s = tid; s < l.n_seq; s += PREP_T) {
            const int a = l.first[s], b = l.first[s + 1];
            range |= a < 0 || b < a || b > n;
            if (s == tid) first0 = a, first1 = b;
        }
    }
    if (tid == 0) s_groups = 0;
    const bool range_all = __syncthreads_or(range) != 0;
    if (range_all) lo = hi = first0 = first1 = 0;
    int done = 0;                                          // slots of the rounds before
    bool wrong = false;
    for (int t0 = 0; t0 < n; t0 += PREP_T * PREP_PER) {
        if (t0 > 0) load(t0);
        unsigned vote[PREP_PER];
#pragma unroll
        for (int i = 0; i < PREP_PER; ++i) {
            const int r = t0 + i * PREP_T + tid;
            const bool in = ((on >> i) & 1u) && r >= lo && r < hi;
            wrong |= in && (y[i] < 0 || y[i] >= l.vocab);
            vote[i] = __ballot_sync(0xffffffffu, in);
            if (lane == 0) s_count[i * 32 + warp] = __popc(vote[i]);
        }
        __syncthreads();
        // every warp scans the 256 counts, eight per lane
        int c[PREP_PER], sum = 0;
#pragma unroll
        for (int i = 0; i < PREP_PER; ++i) sum += c[i] = s_count[lane * PREP_PER + i];
        int inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        const int all = __shfl_sync(0xffffffffu, inc, 31);
        int before[PREP_PER];                              // counts before each of this lane's eight
        int run = inc - sum;
#pragma unroll
        for (int i = 0; i < PREP_PER; ++i) {
            before[i] = run;
            run += c[i];
        }
#pragma unroll
        for (int i = 0; i < PREP_PER; ++i) {
            // the count before (i, warp): entry i * 32 + warp lies with lane i * 4 + warp / 8
            int at = 0;
#pragma unroll
            for (int q = 0; q < PREP_PER; ++q) {
                const int v = __shfl_sync(0xffffffffu, before[q], i * 4 + (warp >> 3));
                if (q == (warp & 7)) at = v;
            }
            const int r = t0 + i * PREP_T + tid;
            const bool in = (vote[i] >> lane) & 1u;
            at += done + __popc(vote[i] & ((1u << lane) - 1u));
            if (r < n) w.slot[r] = in ? at : ~at;
            if (in) {
                w.row[at] = r;
                w.y[at] = y[i];
                w.tick[at] = 0;
            }
        }
        done += all;
        __syncthreads();
    }
    for (int i = tid; i < w.n_words; i += PREP_T) w.words[i] = 0;
    bad |= range_all || wrong;
    int groups = 0, chosen = 0;
    const bool any_bad = __syncthreads_or(bad) != 0;
    if (l.n_seq > 0) {
        auto slots = [&](int t) { return t < n ? slots_before(w.slot[t]) : done; };
        auto start = [&](int s) { return range_all ? 0 : l.first[s]; };
        for (int s = tid; s < l.n_seq; s += PREP_T) {
            const int a = slots(s == tid ? first0 : start(s)), b = slots(s == tid ? first1 : start(s + 1));
            w.seq_slot[s] = a;
            if (s == l.n_seq - 1) w.seq_slot[l.n_seq] = b;
            if (b == a) continue;
            if (l.pairs == 0 || (s < l.pairs && slots(start(l.pairs + s + 1)) > slots(start(l.pairs + s)))) ++groups;
        }
        if (l.pairs > 0 && tid == 0) chosen = slots(start(l.pairs));   // (rows before the first sequence do not count)
        groups = __reduce_add_sync(0xffffffffu, groups);
        if (lane == 0 && groups) atomicAdd(&s_groups, groups);
        __syncthreads();
    }
    if (tid == 0) {
        w.hdr->bad_targets = any_bad ? 1 : 0;
        w.hdr->n_valid = done;
        w.hdr->redo = 0;
        w.hdr->pad[HDR_GROUPS] = s_groups;
        w.hdr->pad[HDR_CHOSEN] = chosen;
        w.hdr->pad[HDR_COEF] = 0;
        int *fault = &w.hdr->pad[HDR_FAULT];
        if (any_bad && w.hdr->err == 0 && !is_fault(*fault)) *fault = LOSSK_TARGET_OUT_OF_RANGE;
    }
}

cudaError_t launch_seq_prep(const SeqLoss &l, const SeqScratch &w, cudaStream_t st)
{
    Launch k(KK_SEQ_PREP, st);
    return launch(seq_prep_kernel, dim3(1), dim3(PREP_T), 0, st, l, w);
}

// One warp per slot: the row's copy and, in the 16-bit types, its product with the
// target's weight row, near which the fused pass takes its exponents (the logit that
// counts is the pass's own).
template <typename T> // float, uint16_t (bf16 bits) or h16_t (fp16 bits)
__global__ void __launch_bounds__(256) seq_gather_kernel(const SeqLoss l, const SeqScratch w, const T *__restrict__ H,
                                                         const T *__restrict__ W, int64_t d, T *__restrict__ out)
{
    wait_for_stream();
    if (l.early_pass) let_next_start();
    if (seq_refused(w.hdr)) return;
    const int c = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int n_valid = w.hdr->n_valid;
    if (c >= max((n_valid + 255) & ~255, 256)) return;
    T *o = out + c * d;
    if constexpr (sizeof(T) == 4) {
        const T *h = c < n_valid ? H + w.row[c] * d : nullptr;
        for (int64_t k = lane; k < d; k += 32) o[k] = h ? h[k] : 0.f;
    } else {
        constexpr bool F16 = std::is_same<T, h16_t>::value;
        uint4 *ov = reinterpret_cast<uint4 *>(o);
        if (c >= n_valid) {
            for (int64_t k = lane; k < d / 8; k += 32) ov[k] = make_uint4(0, 0, 0, 0);
            return;
        }
        const uint4 *h = reinterpret_cast<const uint4 *>(H + w.row[c] * d);
        const uint4 *v = reinterpret_cast<const uint4 *>(W + w.y[c] * d);
        float s[8] = {};
#pragma unroll 4
        for (int64_t k = lane; k < d / 8; k += 32) {
            const uint4 a = h[k], b = v[k];
            ov[k] = a;
            const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[2 * i] = fmaf(h16_lo<F16>(aw[i]), h16_lo<F16>(bw[i]), s[2 * i]);
                s[2 * i + 1] = fmaf(h16_hi<F16>(aw[i]), h16_hi<F16>(bw[i]), s[2 * i + 1]);
            }
        }
        float acc = ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
        for (int q = 16; q > 0; q >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, q);
        if (lane == 0) {
            w.tokp[c] = make_float4(fmaf(acc, l.k2, FUSED_SHIFT), 0.f, 0.f, __int_as_float(static_cast<int>(w.y[c])));
        }
    }
}

cudaError_t launch_seq_gather(int dtype, const SeqLoss &l, const SeqScratch &w, const void *H, const void *W, int64_t d,
                              void *out, cudaStream_t st)
{
    Launch k(KK_SEQ_GATHER, st);
    const dim3 grid(static_cast<unsigned>((((static_cast<int64_t>(l.n_tok) + 255) & ~int64_t(255)) + 7) / 8));
    if (dtype == LOSSK_F32)
        return launch(seq_gather_kernel<float>, grid, dim3(256), 0, st, l, w, static_cast<const float *>(H),
                      static_cast<const float *>(W), d, static_cast<float *>(out));
    if (dtype == LOSSK_F16)
        return launch(seq_gather_kernel<h16_t>, grid, dim3(256), 0, st, l, w, static_cast<const h16_t *>(H),
                      static_cast<const h16_t *>(W), d, static_cast<h16_t *>(out));
    return launch(seq_gather_kernel<uint16_t>, grid, dim3(256), 0, st, l, w, static_cast<const uint16_t *>(H),
                  static_cast<const uint16_t *>(W), d, static_cast<uint16_t *>(out));
}

// One thread per slot.  With r the row's reference (its target at about 64 in log2
// units) and Z the sum of 2^(x log2 e - r): lse2 = r + log2 Z, logp = ln 2 (x_y log2 e - r -
// log2 Z).  The difference is taken in double: r's own rounding, 4e-6 at 64, is in Z
// as well and must not be in the result.  The passes take 2^(x log2 e - lse2) with lse2 a
// float: what its rounding moves every probability of the row by (2e-6 at 64, 7e-5 at 3000)
// is given back in `share`.  x_y comes from the pass as the sum does: the
// tensor cores' sums are truncated, logits come out low by 1e-9 of their size per unit of
// d_model, and an exact x_y against such a sum was 2.5e-5 off at d_model 4096, the same
// way for every token of a sequence.
__global__ void __launch_bounds__(32) seq_merge_fused_kernel(const SeqLoss l, const SeqScratch w,
                                                             const float *__restrict__ zpart, int64_t nz)
{
    wait_for_stream();
    if (l.early) let_next_start();
    if (seq_refused(w.hdr)) return;
    const int c = blockIdx.x * 32 + threadIdx.x;
    if (c >= w.hdr->n_valid) return;
    float Z = 0.f;
    int64_t j = 0;
    for (; j + 16 <= nz; j += 16) {
        float v[16];
#pragma unroll
        for (int q = 0; q < 16; ++q) v[q] = zpart[(j + q) * w.n_pad + c];
#pragma unroll
        for (int q = 0; q < 16; ++q) Z += v[q];
    }
    for (; j < nz; ++j) Z += zpart[j * w.n_pad + c];
    // outside, the largest shifted term may be near the end of fp32's range (or not a number)
    if (!(Z >= 0x1p-80f && Z <= 0x1p90f)) w.hdr->redo = 1;
    const float r = w.tokp[c].x;
    const double lz = log2_of(Z), lse2 = lse2_or_nan(static_cast<double>(r) + lz);
    const double gap = static_cast<double>(w.tgt[c]) * static_cast<double>(l.k2) - static_cast<double>(r);
    put_lse2(w, c, lse2);
    w.z[c] = Z;
    // (the exponentials are of -64 for the target, as exact as of 0, and anything for the others)
    const double lp = lse2 == lse2 ? (gap - lz) * LN2 : NAN;
    w.lp[c] = static_cast<float>(lp - EX2_LOW * static_cast<double>(1.f - expf(fminf(static_cast<float>(lp), 0.f))));
}

cudaError_t launch_seq_merge_fused(const SeqLoss &l, const SeqScratch &w, const float *zpart, int64_t nz,
                                   cudaStream_t st)
{
    Launch k(KK_SEQ_MERGE, st);
    return launch(seq_merge_fused_kernel, dim3(static_cast<unsigned>((l.n_tok + 31) / 32)), dim3(32), 0, st, l, w, zpart,
                  nz);
}

// 32 slots per block, their tiles dealt to eight warps in runs.
constexpr int MT_W = 8;
__global__ void __launch_bounds__(32 * MT_W) seq_merge_tiles_kernel(const SeqLoss l, const SeqScratch w,
                                                                    const float *__restrict__ part, int64_t n_ct,
                                                                    const int *only_if)
{
    wait_for_stream();
    if (l.early) let_next_start();
    if (seq_refused(w.hdr) || (only_if && !*reinterpret_cast<const volatile int *>(only_if))) return;
    __shared__ float s_max[MT_W][32];
    __shared__ double s_sum[MT_W][32];
    const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    const bool live = c < w.hdr->n_valid;
    const float *m2 = part, *zz = part + n_ct * w.n_pad;
    const int64_t c0 = n_ct * g / MT_W, c1 = n_ct * (g + 1) / MT_W;
    float M = -INFINITY;
    if (live)
        for (int64_t i = c0; i < c1; ++i) M = fmaxf(M, m2[i * w.n_pad + c]);
    s_max[g][lane] = M;
    __syncthreads();
    for (int q = 0; q < MT_W; ++q) M = fmaxf(M, s_max[q][lane]);
    double Z = 0.0;
    if (live)                                  // (a row without any probability: 0, or the NaNs that maxima pass over)
        for (int64_t i = c0; i < c1; ++i)
            Z += static_cast<double>(zz[i * w.n_pad + c] * (M > -INFINITY ? exp2f(m2[i * w.n_pad + c] - M) : 1.f));
    s_sum[g][lane] = Z;
    __syncthreads();
    if (g != 0 || !live) return;
    Z = 0.0;
    for (int q = 0; q < MT_W; ++q) Z += s_sum[q][lane];
    const double lse2 = lse2_or_nan(static_cast<double>(M) + (M > -INFINITY && Z == 0.0 ? NAN : log2(Z)));
    put_lse2(w, c, lse2);
    w.z[c] = 1.f;
    w.lp[c] = static_cast<float>((static_cast<double>(w.tgt[c]) * static_cast<double>(l.k2) - lse2) * LN2 -
                                 static_cast<double>(ex2_low(static_cast<float>(Z), 2)));
}

cudaError_t launch_seq_merge_tiles(const SeqLoss &l, const SeqScratch &w, const float *part, int64_t n_ct,
                                   const int *only_if, cudaStream_t st)
{
    Launch k(KK_SEQ_MERGE, st);
    return launch(seq_merge_tiles_kernel, dim3(static_cast<unsigned>((l.n_tok + 31) / 32)), dim3(32 * MT_W), 0, st, l, w,
                  part, n_ct, only_if);
}

// One block per sequence; the order of the sum is a function of its length.
constexpr int SUM_T = 256;
__global__ void __launch_bounds__(SUM_T) seq_sum_kernel(const SeqLoss l, const SeqScratch w)
{
    wait_for_stream();
    if (l.early) let_next_start();
    if (seq_refused(w.hdr)) return;
    __shared__ double sh[SUM_T / 32];
    const int s = blockIdx.x, a = w.seq_slot[s], b = w.seq_slot[s + 1];
    const float *base = l.pairs > 0 ? l.ref : l.old;
    double v = 0.0;
    if (l.pairs > 0 || l.old)
        for (int c = a + static_cast<int>(threadIdx.x); c < b; c += SUM_T)
            v += static_cast<double>(w.lp[c]) - (base ? static_cast<double>(base[w.row[c]]) : 0.0);
    v = block_sum(v, sh);
    if (threadIdx.x == 0) w.sum[s] = v;
    if (l.pairs > 0 || a == b) return;
    // the policy loss by sequence: every token's term moves the one ratio
    const double delta = v / (b - a), weight = row_weight(l, w.hdr, b - a);
    double slope = 0.0;
    for (int c = a + static_cast<int>(threadIdx.x); c < b; c += SUM_T)
        slope += weight * static_cast<double>(policy_term<double>(l, delta, advantage(l, w.row[c], s)).slope);
    slope = block_sum(slope, sh);
    if (threadIdx.x == 0) w.slope[s] = slope;
}

cudaError_t launch_seq_sum(const SeqLoss &l, const SeqScratch &w, cudaStream_t st)
{
    Launch k(KK_SEQ_SUM, st);
    return launch(seq_sum_kernel, dim3(static_cast<unsigned>(l.n_seq)), dim3(SUM_T), 0, st, l, w);
}

namespace {

__device__ __forceinline__ double log_ratio(const SeqLoss &l, const SeqScratch &w, int s, int &count)
{
    count = w.seq_slot[s + 1] - w.seq_slot[s];
    const double v = w.sum[s];
    return (l.flags & LOSSK_LENGTH_MEAN) && count > 0 ? v / count : v;
}

} // namespace

// One thread per row, and per sequence and pair.  Each block adds up its threads' terms
// of the three means; the first block of the kernel after it adds the blocks' sums
// (seq_scalars).  (Doubles run at a sixty-fourth of floats here: one block that summed
// every row took 34 us.  The last block to arrive, here, held the next kernel up for 3.)
__global__ void __launch_bounds__(COEF_T) seq_coef_kernel(const SeqLoss l, const SeqScratch w)
{
    wait_for_stream();
    if (l.early_pass) let_next_start();
    if (seq_refused(w.hdr)) return;
    const int t = blockIdx.x * COEF_T + threadIdx.x;
    const bool pref = l.pairs > 0;
    float coef = 0.f;
    double v[3] = {0.0, 0.0, 0.0};
    if (pref && t < l.n_seq && l.log_ratio) {
        int n_s;
        l.log_ratio[t] = static_cast<float>(log_ratio(l, w, t, n_s));
    }
    if (pref && t < l.pairs) {
        int nc, nr;
        const double u = log_ratio(l, w, t, nc) - log_ratio(l, w, l.pairs + t, nr);
        float loss = 0.f, slope;
        const bool live = nc > 0 && nr > 0;
        if (live) pair_term(l, u, loss, slope);
        if (l.per_token) l.per_token[t] = loss;
        v[1] = static_cast<double>(loss);
        v[2] = live && u > 0.0 ? 1.0 : 0.0;
    }
    const int c = t < l.n_tok ? w.slot[t] : -1;
    const int s = l.n_seq > 0 ? seq_of(w.seq_slot, l.n_seq, c, threadIdx.x & 31) : 0;
    if (t < l.n_tok) {
        if (c < 0) {
            if (l.logp) l.logp[t] = 0.f;
            if (!pref && l.per_token) l.per_token[t] = 0.f;
        } else {
            const float lp = w.lp[c];
            const int n_s = l.n_seq > 0 ? w.seq_slot[s + 1] - w.seq_slot[s] : 0;
            RowTerms r;
            if (pref) {
                const bool chosen = s < l.pairs;
                const int i = chosen ? s : s - l.pairs;
                int nc, nr;
                const double u = log_ratio(l, w, i, nc) - log_ratio(l, w, l.pairs + i, nr);
                float loss, slope = 0.f;
                if (nc > 0 && nr > 0) pair_term(l, u, loss, slope);
                r = pair_row(l, w.hdr, chosen, n_s, slope, lp);
                v[0] = r.v[0];
            } else {
                const bool by_seq = l.flags & LOSSK_SEQ_RATIO;
                r = policy_row(l, policy_inputs(l, w.hdr, t, s, n_s), t, lp, by_seq ? w.sum[s] / n_s : 0.0,
                               by_seq ? static_cast<float>(w.slope[s] / n_s) : 0.f);
#pragma unroll
                for (int k = 0; k < 3; ++k) v[k] = r.v[k];
            }
            if (l.logp) l.logp[t] = lp;
            const float4 P = row_params(w.ref[c], w.share[c], r.coef, w.y[c]);
            w.tokp[c] = P;
            coef = P.z;
        }
    }
    // the largest finite |coefficient| (fp16's d_weight pass scales by it): positive floats order as integers
    unsigned m = isfinite(coef) ? __float_as_uint(fabsf(coef)) : 0;
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0 && m) atomicMax(reinterpret_cast<unsigned *>(&w.hdr->pad[HDR_COEF]), m);

    __shared__ double sh[3][COEF_T / 32];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
        if ((threadIdx.x & 31) == 0) sh[k][threadIdx.x >> 5] = v[k];
    }
    __syncthreads();
    if (threadIdx.x < 3) {
        double x = sh[threadIdx.x][0];
        for (int i = 1; i < COEF_T / 32; ++i) x += sh[threadIdx.x][i];
        w.acc[threadIdx.x * static_cast<int64_t>(gridDim.x) + blockIdx.x] = x;
    }
}

cudaError_t launch_seq_coef(const SeqLoss &l, const SeqScratch &w, cudaStream_t st)
{
    Launch k(KK_SEQ_COEF, st);
    const int n = l.n_tok > l.n_seq ? l.n_tok : l.n_seq;
    return launch(seq_coef_kernel, dim3(static_cast<unsigned>((n + COEF_T - 1) / COEF_T)), dim3(COEF_T), 0, st, l, w);
}

__global__ void __launch_bounds__(256) seq_scalars_kernel(const SeqLoss l, const SeqScratch w)
{
    wait_for_stream();
    if (l.early) let_next_start();
    if (seq_refused(w.hdr)) return;
    seq_scalars<256>(l, w);
}

cudaError_t launch_seq_scalars(const SeqLoss &l, const SeqScratch &w, cudaStream_t st)
{
    Launch k(KK_REDUCE, st);
    return launch(seq_scalars_kernel, dim3(1), dim3(256), 0, st, l, w);
}

namespace {

__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(uint16_t *p, float v) { *p = static_cast<uint16_t>(pack_bf16x2(v, 0.f)); }
__device__ __forceinline__ void put(h16_t *p, float v) { p->bits = static_cast<uint16_t>(pack_f16x2(v, 0.f)); }
__device__ __forceinline__ void put4(float *p, const float (&v)[4])
{
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void put4(uint16_t *p, const float (&v)[4])
{
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}
__device__ __forceinline__ void put4(h16_t *p, const float (&v)[4])
{
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3]));
}

} // namespace

// Four elements per thread where d_model is a multiple of 4, else one, and with few elements
// LANES threads for each, which share the splits.  The splits are added in their order, or each
// thread's every LANES-th in order and then the threads' sums: a function of the sizes.
template <typename O, int N, int LANES>
__global__ void __launch_bounds__(256) seq_dh_kernel(const SeqLoss l, const SeqScratch w, const float *__restrict__ part,
                                                     int64_t nsplit, int64_t d, const uint16_t *__restrict__ W, int fused,
                                                     const int *only_if, O *out, int add, int by_row, int scalars)
{
    wait_for_stream();
    if (l.early) let_next_start();
    if (seq_refused(w.hdr)) return;
    if (only_if && !*reinterpret_cast<const volatile int *>(only_if)) return;
    if (scalars && blockIdx.x == 0) seq_scalars<256>(l, w);
    const int64_t dn = d / N, count = l.n_tok * dn, plane = l.n_tok * d;
    const int sub = threadIdx.x % LANES;
    bool bad = false;
    for (int64_t i0 = blockIdx.x * int64_t(256 / LANES); i0 < count; i0 += int64_t(256 / LANES) * gridDim.x) {
        const int64_t i = i0 + threadIdx.x / LANES;
        const bool in = i < count;
        const int64_t t = in ? i / dn : 0, k = in ? (i - t * dn) * N : 0;
        const int c = in ? w.slot[t] : -1;
        float v[N] = {};
        if (c >= 0) {
            const float *p = part + (by_row ? t : c) * d + k;
            auto load = [&](int64_t s, float (&x)[N]) {
                if constexpr (N == 4) {
                    const float4 q = __ldcs(reinterpret_cast<const float4 *>(p + s * plane));
                    x[0] = q.x; x[1] = q.y; x[2] = q.z; x[3] = q.w;
                } else {
                    x[0] = __ldcs(p + s * plane);
                }
            };
            int64_t s = sub;
            for (; s + 7 * LANES < nsplit; s += 8 * LANES) {
                float x[8][N];
#pragma unroll
                for (int q = 0; q < 8; ++q) load(s + q * LANES, x[q]);
#pragma unroll
                for (int q = 0; q < 8; ++q)
#pragma unroll
                    for (int e = 0; e < N; ++e) v[e] += x[q][e];
            }
            for (; s < nsplit; s += LANES) {
                float x[N];
                load(s, x);
#pragma unroll
                for (int e = 0; e < N; ++e) v[e] += x[e];
            }
        }
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1)
#pragma unroll
            for (int e = 0; e < N; ++e) v[e] += __shfl_xor_sync(0xffffffffu, v[e], o);
        if (!in || sub != 0) continue;
        if (fused && c >= 0) {
            if constexpr (N == 4) {
                // (the fused pass runs on bf16 inputs)
                const float a = w.tokp[c].z, az = a / w.z[c];
                const uint2 b = *reinterpret_cast<const uint2 *>(W + w.y[c] * d + k);
                const float wv[4] = {h16_lo<false>(b.x), h16_hi<false>(b.x), h16_lo<false>(b.y), h16_hi<false>(b.y)};
#pragma unroll
                for (int e = 0; e < N; ++e) v[e] = a == 0.f ? 0.f : fmaf(az, v[e], -a * wv[e]);
            }
#pragma unroll
            for (int e = 0; e < N; ++e) bad |= !isfinite(v[e]);
        }
        O *o = out + t * d + k;
        if constexpr (std::is_same<O, float>::value) {
            if (add) {
                if (c < 0) continue;
#pragma unroll
                for (int e = 0; e < N; ++e) v[e] += o[e];
            }
        }
        if constexpr (N == 4) put4(o, v);
        else put(o, v[0]);
    }
    if (bad) w.hdr->redo = 1;
}

template <typename O>
static cudaError_t dh_one(const SeqLoss &l, const SeqScratch &w, const float *part, int64_t nsplit, int64_t d,
                          const void *W, bool fused, const int *only_if, void *out, bool add, bool by_row,
                          bool scalars, cudaStream_t st)
{
    const bool four = d % 4 == 0;
    const int64_t items = l.n_tok * (four ? d / 4 : d);
    // fewer elements than eight threads for each would fill the GPU with
    const bool few = items < 152 * 256 && nsplit >= 16;
    int64_t grid = (items * (few ? 8 : 1) + 255) / 256;
    if (grid > 4096) grid = 4096;
    auto kern = four ? (few ? seq_dh_kernel<O, 4, 8> : seq_dh_kernel<O, 4, 1>)
                     : (few ? seq_dh_kernel<O, 1, 8> : seq_dh_kernel<O, 1, 1>);
    return launch(kern, dim3(static_cast<unsigned>(grid)), dim3(256), 0, st, l, w, part, nsplit, d,
                  static_cast<const uint16_t *>(W), fused ? 1 : 0, only_if, static_cast<O *>(out), add ? 1 : 0,
                  by_row ? 1 : 0, scalars ? 1 : 0);
}

cudaError_t launch_seq_dh(int out_dtype, const SeqLoss &l, const SeqScratch &w, const float *part, int64_t nsplit,
                          int64_t d, const void *W, bool fused, const int *only_if, void *out, bool add, bool by_row,
                          bool scalars, cudaStream_t st)
{
    Launch k(KK_SEQ_DH, st);
    if (out_dtype == LOSSK_F32) return dh_one<float>(l, w, part, nsplit, d, W, fused, only_if, out, add, by_row, scalars, st);
    if (out_dtype == LOSSK_F16) return dh_one<h16_t>(l, w, part, nsplit, d, W, fused, only_if, out, add, by_row, scalars, st);
    return dh_one<uint16_t>(l, w, part, nsplit, d, W, fused, only_if, out, add, by_row, scalars, st);
}

} // namespace lossk
