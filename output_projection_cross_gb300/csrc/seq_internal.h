// seq_internal.h -- the losses of sampled and compared sequences: what their
// host side (lossk_seq.cu) and kernels (k_seq.cu, k_rows.cu) share.
#pragma once
#include "lossk_internal.h"

namespace lossk {

// Rows that count are numbered in order: "slots" 0 .. n_valid - 1.  Every
// per-row array below but `slot` is indexed by slot, and the fused passes see
// the rows of a gathered copy of `hidden`, so rows that do not count cost them
// nothing.
struct SeqScratch {
    WsHeader *hdr;
    int *slot;          // [n_pad] by row: its slot, or ~(slots before it) where it does not count
    int *row;           // [n_pad] the slot's row
    int64_t *y;         // [n_pad] its target
    int *seq_slot;      // [n_seq + 1] slots before each sequence (and all of them)
    float *tgt;         // [n_pad] its target's logit (the forms from hidden rows, as the pass has it)
    float *lp;          // [n_pad] logp
    float *ref;         // [n_pad] from hidden rows log2 sum 2^(x log2 e), given logits the largest of them
    float *share;       // [n_pad] a term relative to the reference times this is a probability
    float *z;           // [n_pad] fused pass: the sum of its shifted terms
    float4 *tokp;       // [n_pad] {ref, a share, a, target}: softmax and one-hot coefficients
    double *sum;        // [n_seq] sum over the sequence of logp minus its base
    double *slope;      // [n_seq] LOSSK_SEQ_RATIO: sum over the sequence of w dP/d(log ratio)
    double *acc;        // [3][blocks] the coefficient kernel's blocks' terms of the scalars
    float4 *terms;      // forms from logits, policy loss by token: [n_tok] each row's terms of the scalars
    int *tick;          // [n_pad] forms from logits: pieces of the row that are done
    unsigned *words;    // [n_words] forms from hidden rows: zeroed by seq_prep, the group passes' hand-off counters
    int n_words;
    float2 *part;       // forms from logits: [n_pad][seq_stat_splits] (max, sum) of the row's pieces
    int64_t n_pad;
};

// ex2.approx comes out low by 5e-8 of its value on average (measured over [-80, 0]:
// 4.9e-8 to 5.2e-8), and so does a sum of exponentials, once per exponential that a
// term has gone through.  That much is given back to the log-probabilities: sequences sum
// hundreds of them against a reference's, and it would add up.  A largest term's own exponentials are of 0,
// and exact: what is given back is of the other terms' share of the sum (a token that is all but
// certain has logp 0, not 1e-7).
constexpr double EX2_LOW = 5e-8;

// The tensor cores drop what lies below an fp32 sum's last bit at each step of 16
// products: a logit comes out low by so much of itself per unit of d_model (measured, d_model
// 256 to 4096): 0.9e-9 to 1.2e-9 where its sum grows evenly along d_model or is carried by a few
// channels anywhere, 0.1e-9 to 0.3e-9 where the last channel carries it, 1.5e-9 to 2.3e-9 where
// the first one does or they fall in size.  The passes' scale makes up for the middle of that
// range, 1e-9: a softmax over 4096-wide products is then not 2.5e-5 flatter than the logits', and
// at the ends of the range, either way, half as far off as the lowest was (logp of 4096-wide rows, root mean
// square, with and without it: even 6e-6 and 1.2e-5, last channel 9e-6 and 7e-6, falling 1.2e-5 and 2.1e-5).
constexpr double TC_LOW = 1e-9;

// The loss: fields of the policy loss, then of the preference loss.
struct SeqLoss {
    int n_tok, n_seq, pairs;       // n_seq 0: no sequences; pairs > 0: the preference loss
    int64_t vocab;
    const int64_t *targets;
    const uint8_t *mask;
    const int32_t *first;
    const float *adv, *old, *ref;
    float low, high, kl;
    float k2;                      // log2(e) / temperature
    float per_t, per_t_up;         // -grad_scale / temperature as per_t per_t_up^2, per_t_up a power of two (the
                                   // quotient is beyond floats where both are at their ends)
    uint32_t flags;
    int objective;
    float beta, margin, smooth, nll;
    float *scalars, *per_token, *logp;      // per_token: per_pair for the preference loss
    float *log_ratio;
    // Each kernel's blocks are set up while the kernel ahead runs, not while it ends; those of the passes
    // over the logits.
    bool early, early_pass;
};

// dtype: lossk_dtype.  All enqueue on `st`.
// Counts and numbers the rows, checks targets and `first`, clears the header's
// words of one call; 586 into the header, and every later kernel returns at once.
cudaError_t launch_seq_prep(const SeqLoss &l, const SeqScratch &w, cudaStream_t st);
// Copies the counted rows of hidden to out (rows up to the next multiple of 256
// as zeros); 16-bit types: tokp.x, the fused pass's reference target logit * k2 +
// FUSED_SHIFT, and the target in tokp.w.
cudaError_t launch_seq_gather(int dtype, const SeqLoss &l, const SeqScratch &w, const void *H, const void *W, int64_t d,
                              void *out, cudaStream_t st);
// The fused pass's sums -> logp, ref, share (redo where a row left the range).
cudaError_t launch_seq_merge_fused(const SeqLoss &l, const SeqScratch &w, const float *zpart, int64_t nz,
                                   cudaStream_t st);
// The forward pass's (max, sum) partials of n_ct tiles -> logp, ref, share.  only_if: or
// NULL; zero: not needed.
cudaError_t launch_seq_merge_tiles(const SeqLoss &l, const SeqScratch &w, const float *part, int64_t n_ct,
                                   const int *only_if, cudaStream_t st);
// Per sequence the sum of log ratios (and the slope of LOSSK_SEQ_RATIO).
cudaError_t launch_seq_sum(const SeqLoss &l, const SeqScratch &w, cudaStream_t st);
// Per row its loss, outputs and coefficient; per pair its loss.  The scalars: by a kernel of their
// own where none follows, else by the one that does.
constexpr int COEF_T = 128;
cudaError_t launch_seq_coef(const SeqLoss &l, const SeqScratch &w, cudaStream_t st);
cudaError_t launch_seq_scalars(const SeqLoss &l, const SeqScratch &w, cudaStream_t st);
// Given logits: logp, ref, share, a row in `splits` pieces; grad_logits of every row, and the scalars.
int seq_stat_splits(int64_t n, int64_t vocab, int dtype);
cudaError_t launch_seq_stats(int dtype, const SeqLoss &l, const SeqScratch &w, const void *logits, int splits,
                             cudaStream_t st);
cudaError_t launch_seq_grad(int dtype, const SeqLoss &l, const SeqScratch &w, const void *logits, void *grad,
                            bool accumulate, cudaStream_t st);
// The policy loss by token in one launch, a row's logits on the chip from its statistics to
// its gradient (grad NULL: none); blocks of a cluster that take a row, 0 where a row does not fit.
int policy_rows_cluster(int64_t n, int64_t vocab, int dtype);
bool policy_rows_early(int64_t n, int64_t vocab, int dtype, int cluster);
cudaError_t launch_policy_rows(int dtype, const SeqLoss &l, const SeqScratch &w, const void *logits, void *grad,
                               bool accumulate, int cluster, cudaStream_t st);
// d_hidden of every row from the passes' split partials [nsplit][n_tok][d], indexed by
// slot: fused, a_t / Z_t times their sum minus a_t W[y_t] (a value that is not
// finite asks for the separate passes, redo), else their sum.  out: out_dtype.
// add: added to it (float).  by_row: the partials are indexed by row.
// scalars: writes them too.
cudaError_t launch_seq_dh(int out_dtype, const SeqLoss &l, const SeqScratch &w, const float *part, int64_t nsplit,
                          int64_t d, const void *W, bool fused, const int *only_if, void *out, bool add,
                          bool by_row, bool scalars, cudaStream_t st);

} // namespace lossk
