// lossk_seq.cu -- the extern "C" entry points of the losses of sampled and
// compared sequences (declared in include/lossk.h): argument checks in the
// documented order, workspace layout and launch sequence.  No call synchronises
// and none allocates device memory.
#include "../../include/lossk.h"
#include "host_internal.h"
#include "seq_internal.h"

#include <cmath>
#include <cstring>
#include <limits>
#include <mutex>

using namespace lossk;

namespace {

constexpr int64_t MAX_DIM = int64_t(1) << 24;

bool is16(int32_t dtype) { return dtype == LOSSK_BF16 || dtype == LOSSK_F16; }
bool dtype_ok(int32_t dtype) { return dtype == LOSSK_F32 || is16(dtype); }

// hand-off counters of a group pass
constexpr int GSIG_WORDS = 2 * G_MAX_CTAS * G_SLOTS;

struct Layout {
    int64_t n_pad, n_ct, nsplit;
    bool small;
    int splits, cluster;
    size_t off_slot, off_row, off_y, off_seq, off_tgt, off_lp, off_ref, off_share, off_z, off_tokp, off_sum, off_slope, off_acc,
        off_terms, off_tick, off_rows, off_hidden, off_part, off_dhpart, off_zpart, off_gring, off_gsig, off_dhacc, total;
};

// 580, or why there is no layout.
int32_t layout(int32_t kind, int64_t n, int64_t d, int64_t V, int64_t n_seq, int32_t dtype, Layout *L)
{
    const bool head = kind == LOSSK_KIND_SEQUENCE_HEAD;
    const int32_t s = lossk_dims_check(n, head ? d : 1, V);
    if (s != LOSSK_OK) return s;
    if (n_seq < 0) return LOSSK_EMPTY_DIMENSION;
    if (n_seq > 2 * MAX_DIM) return LOSSK_DIMENSION_TOO_LARGE;
    if (!dtype_ok(dtype)) return LOSSK_LENGTH_MISMATCH;
    std::memset(L, 0, sizeof(*L));
    L->n_pad = cdiv(n, 256) * 256;
    const size_t np = static_cast<size_t>(L->n_pad), ns = static_cast<size_t>(n_seq);
    size_t off = 256;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = align256(off + bytes);
        return at;
    };
    L->off_slot = take(sizeof(int) * np);
    L->off_row = take(sizeof(int) * np);
    L->off_y = take(sizeof(int64_t) * np);
    L->off_seq = take(sizeof(int) * (ns + 1));
    L->off_tgt = take(sizeof(float) * np);
    L->off_lp = take(sizeof(float) * np);
    L->off_ref = take(sizeof(float) * np);
    L->off_share = take(sizeof(float) * np);
    L->off_z = take(sizeof(float) * np);
    L->off_tokp = take(sizeof(float4) * np);
    L->off_sum = take(sizeof(double) * ns);
    L->off_slope = take(sizeof(double) * ns);
    L->off_acc = take(sizeof(double) * 3 * static_cast<size_t>(cdiv(n > n_seq ? n : n_seq, 128)));
    L->off_tick = take(sizeof(int) * np);
    if (head) {
        const bool tc = is16(dtype);
        // fp32: small tiles where those of 64 x 64 would be fewer than two for each SM
        L->small = !tc && cdiv(n, FP_BM) * cdiv(V, FP_BN) < 304;
        const int64_t edge = L->small ? FP_SMALL : FP_BM, slice = L->small ? FP_SMALL_SLICE : FP_SLICE;
        L->n_ct = cdiv(V, tc ? TC_BN_FWD : edge);
        L->nsplit = dh_splits(n, d, V, dtype);
        if (!tc) {
            // d_hidden in as many splits of the vocabulary as make two blocks per SM, down to one tile
            // each: 64 x 64 x 1000 takes 72 us in the two splits of the label loss's rule (eight tiles one
            // after another)
            const int64_t base = cdiv(n, edge) * cdiv(d, slice), most = cdiv(304, base);
            L->nsplit = most < L->n_ct ? most : L->n_ct;
        }
        const size_t nd = static_cast<size_t>(n) * static_cast<size_t>(d);
        L->off_hidden = take((tc ? 2 : 4) * np * static_cast<size_t>(d));
        L->off_part = take(sizeof(float) * NSTAT_CE * static_cast<size_t>(L->n_ct) * np);
        L->off_dhpart = take(sizeof(float) * static_cast<size_t>(L->nsplit) * nd);
        if (dtype == LOSSK_BF16) {
            L->off_zpart = take(sizeof(float) * static_cast<size_t>(L->nsplit) * BWD_MAX_CL * np);
            L->off_dhacc = take(sizeof(float) * nd);
        }
        if (tc) {
            L->off_gring = take(sizeof(uint16_t) * 128 * static_cast<size_t>(G_RING_ROWS));
            L->off_gsig = take(sizeof(unsigned) * 3 * GSIG_WORDS);      // one set for each pass of a call
        }
    } else {
        L->splits = seq_stat_splits(n, V, dtype);
        L->cluster = policy_rows_cluster(n, V, dtype);
        L->off_rows = take(sizeof(float2) * np * static_cast<size_t>(L->splits));
        L->off_terms = take(sizeof(float4) * np);
    }
    L->total = off;
    return LOSSK_OK;
}

SeqScratch scratch(const Layout &L, void *ws)
{
    uint8_t *b = static_cast<uint8_t *>(ws);
    SeqScratch w;
    std::memset(&w, 0, sizeof(w));
    w.hdr = reinterpret_cast<WsHeader *>(b);
    w.slot = reinterpret_cast<int *>(b + L.off_slot);
    w.row = reinterpret_cast<int *>(b + L.off_row);
    w.y = reinterpret_cast<int64_t *>(b + L.off_y);
    w.seq_slot = reinterpret_cast<int *>(b + L.off_seq);
    w.tgt = reinterpret_cast<float *>(b + L.off_tgt);
    w.lp = reinterpret_cast<float *>(b + L.off_lp);
    w.ref = reinterpret_cast<float *>(b + L.off_ref);
    w.share = reinterpret_cast<float *>(b + L.off_share);
    w.z = reinterpret_cast<float *>(b + L.off_z);
    w.tokp = reinterpret_cast<float4 *>(b + L.off_tokp);
    w.sum = reinterpret_cast<double *>(b + L.off_sum);
    w.slope = reinterpret_cast<double *>(b + L.off_slope);
    w.acc = reinterpret_cast<double *>(b + L.off_acc);
    w.tick = reinterpret_cast<int *>(b + L.off_tick);
    w.terms = reinterpret_cast<float4 *>(b + L.off_terms);
    w.part = reinterpret_cast<float2 *>(b + L.off_rows);
    w.words = reinterpret_cast<unsigned *>(b + L.off_gsig);
    w.n_words = L.off_gsig ? 3 * GSIG_WORDS : 0;
    w.n_pad = L.n_pad;
    return w;
}

// One call of either loss in either form.
struct Call {
    bool head;
    int64_t n, d, V, n_seq, n_pairs;      // n_pairs 0: the policy loss
    int32_t dtype;
    const void *X;                        // hidden or logits
    int64_t x_len;
    const void *W;
    int64_t w_len;
    const int64_t *targets;
    int64_t targets_len;
    const uint8_t *mask;
    const int32_t *first;
    int64_t first_len;
    const float *adv, *old, *ref;
    int64_t adv_len, old_len, ref_len;
    double low, high, kl, temperature, beta, margin, smooth, nll, grad_scale;
    int32_t objective;
    uint32_t flags;
    float *scalars, *per_item, *log_ratio, *logp;
    int32_t grad_dtype;
    void *g0, *g1;                        // d_hidden and d_weight, or grad_logits
    int64_t g_len;
    void *ws;
    int64_t ws_bytes;
    cudaStream_t st;
};

// Finite, as the floats that the kernels take too.
bool finite(std::initializer_list<double> v)
{
    for (double x : v)
        if (!(std::fabs(x) <= std::numeric_limits<float>::max())) return false;
    return true;
}

int32_t check(const Call &c, Layout *L)
{
    const bool pref = c.n_pairs != 0;
    if (pref && (c.n_pairs < 1 || c.n < 1)) return LOSSK_EMPTY_DIMENSION;
    if (c.n_pairs > MAX_DIM || c.n_seq > 2 * MAX_DIM) return LOSSK_DIMENSION_TOO_LARGE;
    const int32_t s = layout(c.head ? LOSSK_KIND_SEQUENCE_HEAD : LOSSK_KIND_SEQUENCE_LOGITS, c.n, c.d, c.V, c.n_seq,
                             c.dtype, L);
    if (s != LOSSK_OK) return s;
    const int64_t cells = c.n * (c.head ? c.d : c.V);
    if (!c.X || c.x_len < cells || (c.head && (!c.W || c.w_len < c.V * c.d)) || !c.targets || c.targets_len < c.n ||
        !c.scalars || !c.ws || c.ws_bytes < static_cast<int64_t>(L->total))
        return LOSSK_LENGTH_MISMATCH;
    if (!c.head && c.g0 && c.g_len < cells) return LOSSK_LENGTH_MISMATCH;
    if (c.head && c.grad_dtype != LOSSK_F32 && c.grad_dtype != c.dtype) return LOSSK_LENGTH_MISMATCH;
    if ((c.first != nullptr) != (c.n_seq > 0) || (c.first && c.first_len < c.n_seq + 1)) return LOSSK_LENGTH_MISMATCH;
    if ((c.old && c.old_len < c.n) || (c.ref && c.ref_len < c.n)) return LOSSK_LENGTH_MISMATCH;
    if (!pref) {
        const uint32_t need = LOSSK_SEQ_RATIO | LOSSK_SEQ_MEAN | LOSSK_SEQ_ADVANTAGES;
        if ((c.flags & need) && !c.first) return LOSSK_LENGTH_MISMATCH;
        if (!c.adv || c.adv_len < ((c.flags & LOSSK_SEQ_ADVANTAGES) ? c.n_seq : c.n)) return LOSSK_LENGTH_MISMATCH;
        if (c.kl > 0.0 && !c.ref) return LOSSK_LENGTH_MISMATCH;
    }
    if (!aligned16(c.X) || (c.head && !aligned16(c.W)) || (c.g0 && !aligned16(c.g0)) || (c.g1 && !aligned16(c.g1)) ||
        (reinterpret_cast<uintptr_t>(c.ws) & 255u) || (c.head && is16(c.dtype) && c.d % 8 != 0))
        return LOSSK_UNALIGNED;
    if (!finite({c.grad_scale})) return LOSSK_NON_FINITE_SCALAR;
    if (pref) {
        if (!finite({c.beta, c.margin, c.smooth, c.nll}) || c.beta < 1e-30 || c.smooth < 0.0 || c.smooth > 1.0 ||
            c.nll < 0.0)
            return LOSSK_NON_FINITE_SCALAR;
        if (c.objective < LOSSK_PREF_SIGMOID || c.objective > LOSSK_PREF_SQUARED) return LOSSK_UNKNOWN_OBJECTIVE;
        if (c.objective != LOSSK_PREF_SIGMOID && (c.margin != 0.0 || c.smooth != 0.0)) return LOSSK_NON_FINITE_SCALAR;
    } else if (!finite({c.low, c.high, c.kl, c.temperature}) || c.low < 0.0 || c.low > 1.0 || c.high < 0.0 ||
               c.kl < 0.0 || c.temperature < 1e-30 || c.temperature > 1e30) {
        return LOSSK_NON_FINITE_SCALAR;
    }
    const uint32_t known = LOSSK_ACCUMULATE_GRADS | LOSSK_REDUCE_SUM |
                           (pref ? LOSSK_LENGTH_MEAN : LOSSK_SEQ_RATIO | LOSSK_SEQ_MEAN | LOSSK_SEQ_ADVANTAGES);
    if (c.flags & ~known) return LOSSK_UNKNOWN_FLAGS;
    if (c.head && (c.flags & LOSSK_ACCUMULATE_GRADS) && (c.g0 || c.g1) && c.grad_dtype != LOSSK_F32)
        return LOSSK_UNKNOWN_FLAGS;
    return LOSSK_OK;
}

#define TRY(x)                                                                                                        \
    do {                                                                                                              \
        if ((x) != cudaSuccess) return LOSSK_DEVICE_ERROR;                                                            \
    } while (0)

// The forward statistics pass over the gathered rows (16-bit inputs).
int32_t run_forward(const Call &c, const Layout &L, const SeqLoss &l, const SeqScratch &w, const void *hid,
                    const int *only_if)
{
    uint8_t *b = static_cast<uint8_t *>(c.ws);
    float *part = reinterpret_cast<float *>(b + L.off_part);
    TcArgs a;
    std::memset(&a, 0, sizeof(a));
    if (!make_map(&a.map_x, hid, c.d, L.n_pad, 64, TC_BM) || !make_map(&a.map_y, c.W, c.d, c.V, 64, 128))
        return LOSSK_DEVICE_ERROR;
    a.n_x = a.n_tok = static_cast<int>(c.n);
    a.n_y = a.vocab = static_cast<int>(c.V);
    a.d = static_cast<int>(c.d);
    a.n_xt = static_cast<int>(cdiv(c.n, TC_BM));
    a.n_yt = static_cast<int>(L.n_ct);
    a.n_items = static_cast<int>(cdiv(a.n_xt, 2)) * a.n_yt;
    a.inv_t_l2e = l.k2;
    a.n_dev = &w.hdr->n_valid;
    a.refused = &w.hdr->bad_targets;
    a.only_if = only_if;
    a.chained = 1;
    a.targets = w.y;
    a.tgt_out = w.tgt;
    a.part = part;
    a.part_stride = L.n_pad;
    a.part_plane = L.n_ct * L.n_pad;
    a.err = &w.hdr->err;
    const int pairs = a.n_items < sm_count() / 2 ? a.n_items : sm_count() / 2;
    {
        Launch k(KK_TC_STATS, c.st);
        TRY(launch_fwd2(a, false, c.dtype == LOSSK_F16, 2 * pairs, c.st));
    }
    TRY(launch_seq_merge_tiles(l, w, part, L.n_ct, only_if, c.st));
    return LOSSK_OK;
}

// The caller's stream's helper, forked from it where `want`: aux, until join().  (Without
// a helper aux is the caller's stream.)
struct Fork {
    cudaStream_t st, aux;
    SideStream *sd;
    std::unique_lock<std::mutex> lk;
    bool ok = true;

    Fork(bool want, cudaStream_t s) : st(s), aux(s), sd(want ? side_stream(s) : nullptr)
    {
        if (!sd) return;
        lk = std::unique_lock<std::mutex>(sd->mu);
        if (!sd->ready()) return;
        ok = cudaEventRecord(sd->fork, st) == cudaSuccess && cudaStreamWaitEvent(sd->s, sd->fork, 0) == cudaSuccess;
        if (ok) aux = sd->s;
    }
    bool join()
    {
        if (aux == st) return true;
        return cudaEventRecord(sd->join, aux) == cudaSuccess && cudaStreamWaitEvent(st, sd->join, 0) == cudaSuccess;
    }
};

// What follows the log-probabilities: sums over sequences, coefficients.
int32_t run_losses(const Call &c, const SeqLoss &l, const SeqScratch &w)
{
    if (l.pairs > 0 || (l.flags & LOSSK_SEQ_RATIO)) TRY(launch_seq_sum(l, w, c.st));
    TRY(launch_seq_coef(l, w, c.st));
    return LOSSK_OK;
}

int32_t run_head(const Call &c, const Layout &L, const SeqLoss &l, const SeqScratch &w)
{
    uint8_t *b = static_cast<uint8_t *>(c.ws);
    void *hid = b + L.off_hidden;
    float *part = reinterpret_cast<float *>(b + L.off_part);
    float *dhpart = reinterpret_cast<float *>(b + L.off_dhpart);
    const bool acc = (c.flags & LOSSK_ACCUMULATE_GRADS) != 0, f16 = c.dtype == LOSSK_F16;
    const int *n_dev = &w.hdr->n_valid, *bad = &w.hdr->bad_targets;
    const int n = static_cast<int>(c.n), V = static_cast<int>(c.V), d = static_cast<int>(c.d);
    cudaStream_t st = c.st;
    TRY(launch_seq_gather(c.dtype, l, w, c.X, c.W, c.d, hid, st));
    if (!is16(c.dtype)) {
        const float inv_t = static_cast<float>(1.0 / c.temperature);
        {
            Launch k(KK_FP_STATS, st);
            TRY(launch_fp(TC_STATS, false, hid, c.W, nullptr, n, V, d, n, V, 1, 0, inv_t, w.y, nullptr, nullptr, part,
                          w.tgt, L.n_pad, L.n_ct * L.n_pad, nullptr, 0, st, false, n_dev, bad, L.small));
        }
        TRY(launch_seq_merge_tiles(l, w, part, L.n_ct, nullptr, st));
        int32_t s = run_losses(c, l, w);
        if (s != LOSSK_OK) return s;
        if (!c.g0) TRY(launch_seq_scalars(l, w, st));
        // d_hidden beside d_weight
        Fork f(c.g0 && c.g1, st);
        if (!f.ok) return LOSSK_DEVICE_ERROR;
        cudaError_t e = cudaSuccess;
        if (c.g0) {
            {
                Launch k(KK_FP_ROWS, f.aux);
                e = launch_fp(TC_ROWS, false, hid, c.W, nullptr, n, V, d, n, V, static_cast<int>(L.nsplit), 0, inv_t,
                              nullptr, w.tokp, nullptr, nullptr, nullptr, 0, 0, dhpart, c.n * c.d, f.aux, false, n_dev,
                              bad, L.small);
            }
            if (e == cudaSuccess)
                e = launch_seq_dh(LOSSK_F32, l, w, dhpart, L.nsplit, c.d, c.W, false, nullptr, c.g0, acc, false, true,
                                  f.aux);
        }
        if (c.g1 && e == cudaSuccess) {
            Launch k(KK_FP_COLS, st);
            e = launch_fp(TC_COLS, false, c.W, hid, nullptr, V, n, d, n, V, 1, 0, inv_t, nullptr, w.tokp, nullptr,
                          nullptr, nullptr, 0, 0, static_cast<float *>(c.g1), 0, st, acc, n_dev, bad, L.small);
        }
        return f.join() && e == cudaSuccess ? LOSSK_OK : LOSSK_DEVICE_ERROR;
    }

    const BwdScratch bs{reinterpret_cast<uint16_t *>(b + L.off_gring), reinterpret_cast<unsigned *>(b + L.off_gsig),
                        w.tokp, w.hdr};
    // The passes' maps span the gathered rows up to a multiple of 256 (zeros past the last).
    auto rows_args = [&](BwdArgs *a, int pass) {
        if (!bwd_args(bs, true, L.n_pad, c.d, c.V, hid, c.W, a)) return false;
        a->gsig = w.words + pass * GSIG_WORDS;
        a->chained = 1;
        a->n_tok = n;
        a->n_split = static_cast<int>(L.nsplit);
        a->inv_t_l2e = l.k2;
        a->n_dev = n_dev;
        a->out = dhpart;
        a->out_split_stride = c.n * c.d;
        a->out3_tma = make_map_out3_f32(&a->map_out3, dhpart, c.d, c.n, L.nsplit) ? 1 : 0;
        a->out_scale = 1.f;
        if (f16) a->coef_max = reinterpret_cast<const unsigned *>(&w.hdr->pad[HDR_COEF]);
        return true;
    };
    const bool fused = c.g0 && !f16;
    int *redo = &w.hdr->redo;
    BwdArgs a;
    if (fused) {
        // forward and d_hidden in one pass; a row that left the range of its
        // reference asks for the separate forward
        float *zpart = reinterpret_cast<float *>(b + L.off_zpart);
        if (!rows_args(&a, 0)) return LOSSK_DEVICE_ERROR;
        a.zpart = zpart;
        a.zpart_stride = L.n_pad;
        a.tgt_out = w.tgt;
        {
            Launch k(KK_TC_FUSED, st);
            TRY(launch_bwp(BWD_FUSED, false, false, a, a.n_fixed * a.n_split * a.n_dg, st));
        }
        TRY(launch_seq_merge_fused(l, w, zpart, L.nsplit * a.n_cl, st));
    }
    int32_t s = run_forward(c, L, l, w, hid, fused ? redo : nullptr);
    if (s == LOSSK_OK) s = run_losses(c, l, w);
    if (s != LOSSK_OK) return s;
    if (!c.g0) TRY(launch_seq_scalars(l, w, st));

    // d_hidden from the fused pass, beside the d_weight pass.
    Fork f(fused && c.g1, st);
    if (!f.ok) return LOSSK_DEVICE_ERROR;
    void *dh_to = fused && acc ? static_cast<void *>(b + L.off_dhacc) : c.g0;
    if (fused &&
        launch_seq_dh(c.grad_dtype, l, w, dhpart, L.nsplit, c.d, c.W, true, nullptr, dh_to, false, false, true, f.aux) !=
            cudaSuccess)
        s = LOSSK_DEVICE_ERROR;
    if (s == LOSSK_OK && c.g1) {
        BwdArgs q;
        if (!bwd_args(bs, false, L.n_pad, c.d, c.V, hid, c.W, &q)) {
            s = LOSSK_DEVICE_ERROR;
        } else {
            q.n_tok = n;
            q.gsig = w.words + GSIG_WORDS;
            q.chained = 1;
            q.inv_t_l2e = l.k2;
            q.n_dev = n_dev;
            q.out = static_cast<float *>(c.g1);
            q.accumulate = acc ? 1 : 0;
            q.out_scale = 1.f;
            if (f16) q.coef_max = reinterpret_cast<const unsigned *>(&w.hdr->pad[HDR_COEF]);
            q.out16 = c.grad_dtype != LOSSK_F32 ? 1 : 0;
            q.out_tma = (q.out16 ? make_map_out_16(&q.map_out, c.g1, c.d, c.V)
                                 : make_map_out_f32(&q.map_out, c.g1, c.d, c.V)) ? 1 : 0;
            Launch k(KK_TC_COLS, st);
            if (!q.out_tma || launch_bwp(BWD_COLS, false, f16, q, q.n_fixed * q.n_dg, st) != cudaSuccess)
                s = LOSSK_DEVICE_ERROR;
        }
    }
    if (!f.join()) return LOSSK_DEVICE_ERROR;
    if (s != LOSSK_OK || !c.g0) return s;
    // d_hidden as a pass of its own: fp16, whose tiles need the log-sum-exp, and
    // bf16 where the fused pass's could not be used
    const int *only_if = fused ? redo : nullptr;
    if (!rows_args(&a, 2)) return LOSSK_DEVICE_ERROR;
    a.only_if = only_if;
    {
        Launch k(KK_TC_ROWS, st);
        TRY(launch_bwp(BWD_ROWS, false, f16, a, a.n_fixed * a.n_split * a.n_dg, st));
    }
    TRY(launch_seq_dh(c.grad_dtype, l, w, dhpart, L.nsplit, c.d, c.W, false, only_if, dh_to, !fused && acc, false, !fused,
                      st));
    if (fused && acc)
        TRY(launch_seq_dh(LOSSK_F32, l, w, static_cast<float *>(dh_to), 1, c.d, c.W, false, nullptr, c.g0, true, true,
                          false, st));
    return LOSSK_OK;
}

bool one_launch(const Call &c, const Layout &L)
{
    return c.n_pairs == 0 && !(c.flags & LOSSK_SEQ_RATIO) && L.cluster > 0;
}

int32_t run_rows(const Call &c, const Layout &L, const SeqLoss &l, const SeqScratch &w)
{
    const bool acc = (c.flags & LOSSK_ACCUMULATE_GRADS) != 0;
    if (one_launch(c, L)) {
        TRY(launch_policy_rows(c.dtype, l, w, c.X, c.g0, acc, L.cluster, c.st));
        return LOSSK_OK;
    }
    TRY(launch_seq_stats(c.dtype, l, w, c.X, L.splits, c.st));
    const int32_t s = run_losses(c, l, w);
    if (s != LOSSK_OK) return s;
    if (c.g0) TRY(launch_seq_grad(c.dtype, l, w, c.X, c.g0, acc, c.st));
    else TRY(launch_seq_scalars(l, w, c.st));
    return LOSSK_OK;
}

int32_t run(const Call &c)
{
    Layout L;
    const int32_t s = check(c, &L);
    if (s != LOSSK_OK) return s;
    const SeqScratch w = scratch(L, c.ws);
    SeqLoss l;
    std::memset(&l, 0, sizeof(l));
    l.n_tok = static_cast<int>(c.n);
    l.n_seq = static_cast<int>(c.n_seq);
    l.pairs = static_cast<int>(c.n_pairs);
    l.vocab = c.V;
    l.targets = c.targets;
    l.mask = c.mask;
    l.first = c.first;
    l.adv = c.adv;
    l.old = c.old;
    l.ref = c.ref;
    l.low = static_cast<float>(c.low);
    l.high = static_cast<float>(c.high);
    l.kl = static_cast<float>(c.kl);
    l.k2 = static_cast<float>(LOG2E / c.temperature *
                              (c.head && is16(c.dtype) ? 1.0 + TC_LOW * static_cast<double>(c.d) : 1.0));
    // (as the fp32 passes have it: the target's logit is scaled by what the sum's are)
    if (c.head && !is16(c.dtype)) l.k2 = static_cast<float>(LOG2E) * static_cast<float>(1.0 / c.temperature);
    int up = 0;
    l.per_t = static_cast<float>(std::frexp(-c.grad_scale / c.temperature, &up));
    if (up & 1) l.per_t *= 2.f, --up;
    l.per_t_up = static_cast<float>(std::ldexp(1.0, up / 2));
    l.flags = c.flags;
    l.objective = c.objective;
    l.beta = static_cast<float>(c.beta);
    l.margin = static_cast<float>(c.margin);
    l.smooth = static_cast<float>(c.smooth);
    l.nll = static_cast<float>(c.nll);
    l.scalars = c.scalars;
    l.per_token = c.per_item;
    l.log_ratio = c.log_ratio;
    l.logp = c.logp;
    // (Which kernels are set up while the one ahead runs; the rows' numbering always lets its next one be.)
    // Not the gradients of given logits by sequence and pair: 0 to 2 us slower with it.  The group passes'
    // own hand-overs up to 2^25 logits: 203 x 264 x 5000 in fp16 86 -> 80 us a call, 512 x 1024 x 32000 in bf16 164.5
    // -> 163.7, 8192 x 4096 x 128256 17190 -> 17260 (pairs whose blocks came as others left).
    l.early = c.head || (one_launch(c, L) && policy_rows_early(c.n, c.V, c.dtype, L.cluster));
    l.early_pass = c.head && (!is16(c.dtype) || c.n * c.V <= (int64_t(1) << 25));
    TRY(launch_seq_prep(l, w, c.st));
    return c.head ? run_head(c, L, l, w) : run_rows(c, L, l, w);
}

} // namespace

extern "C" {

int64_t lossk_sequence_workspace_bytes(int32_t kind, int64_t n, int64_t d, int64_t V, int64_t n_seq, int32_t dtype)
{
    Layout L;
    if (kind != LOSSK_KIND_SEQUENCE_HEAD && kind != LOSSK_KIND_SEQUENCE_LOGITS) return -1;
    return layout(kind, n, d, V, n_seq, dtype, &L) == LOSSK_OK ? static_cast<int64_t>(L.total) : -1;
}

int32_t lossk_policy_fwd_bwd(int64_t n, int64_t d, int64_t V, int64_t n_seq, int32_t dtype, const void *hidden,
                             int64_t hidden_len, const void *weight, int64_t weight_len, const int64_t *targets,
                             int64_t targets_len, const uint8_t *loss_mask, const int32_t *first, int64_t first_len,
                             const float *advantages, int64_t advantages_len, const float *old_logp, int64_t old_len,
                             const float *ref_logp, int64_t ref_len, double clip_low, double clip_high,
                             double kl_weight, double temperature, double grad_scale, uint32_t flags,
                             float *scalars_out, float *per_token_out, float *logp_out, int32_t grad_dtype,
                             void *d_hidden, void *d_weight, void *workspace, int64_t workspace_bytes,
                             lossk_stream_t stream)
{
    Call c{};
    c.head = true;
    c.n = n, c.d = d, c.V = V, c.n_seq = n_seq, c.dtype = dtype;
    c.X = hidden, c.x_len = hidden_len, c.W = weight, c.w_len = weight_len;
    c.targets = targets, c.targets_len = targets_len, c.mask = loss_mask, c.first = first, c.first_len = first_len;
    c.adv = advantages, c.adv_len = advantages_len, c.old = old_logp, c.old_len = old_len;
    c.ref = ref_logp, c.ref_len = ref_len;
    c.low = clip_low, c.high = clip_high, c.kl = kl_weight, c.temperature = temperature, c.grad_scale = grad_scale;
    c.flags = flags, c.scalars = scalars_out, c.per_item = per_token_out, c.logp = logp_out;
    c.grad_dtype = grad_dtype, c.g0 = d_hidden, c.g1 = d_weight;
    c.ws = workspace, c.ws_bytes = workspace_bytes, c.st = reinterpret_cast<cudaStream_t>(stream);
    return run(c);
}

int32_t lossk_policy_from_logits(int64_t n, int64_t V, int64_t n_seq, int32_t dtype, const void *logits,
                                 int64_t logits_len, const int64_t *targets, int64_t targets_len,
                                 const uint8_t *loss_mask, const int32_t *first, int64_t first_len,
                                 const float *advantages, int64_t advantages_len, const float *old_logp,
                                 int64_t old_len, const float *ref_logp, int64_t ref_len, double clip_low,
                                 double clip_high, double kl_weight, double temperature, double grad_scale,
                                 uint32_t flags, float *scalars_out, float *per_token_out, float *logp_out,
                                 void *grad_logits, int64_t grad_len, void *workspace, int64_t workspace_bytes,
                                 lossk_stream_t stream)
{
    Call c{};
    c.n = n, c.V = V, c.n_seq = n_seq, c.dtype = dtype, c.X = logits, c.x_len = logits_len;
    c.targets = targets, c.targets_len = targets_len, c.mask = loss_mask, c.first = first, c.first_len = first_len;
    c.adv = advantages, c.adv_len = advantages_len, c.old = old_logp, c.old_len = old_len;
    c.ref = ref_logp, c.ref_len = ref_len;
    c.low = clip_low, c.high = clip_high, c.kl = kl_weight, c.temperature = temperature, c.grad_scale = grad_scale;
    c.flags = flags, c.scalars = scalars_out, c.per_item = per_token_out, c.logp = logp_out;
    c.g0 = grad_logits, c.g_len = grad_len;
    c.ws = workspace, c.ws_bytes = workspace_bytes, c.st = reinterpret_cast<cudaStream_t>(stream);
    return run(c);
}

int32_t lossk_preference_fwd_bwd(int64_t n, int64_t d, int64_t V, int64_t n_pairs, int32_t dtype, const void *hidden,
                                 int64_t hidden_len, const void *weight, int64_t weight_len, const int64_t *targets,
                                 int64_t targets_len, const uint8_t *loss_mask, const int32_t *first,
                                 int64_t first_len, const float *ref_logp, int64_t ref_len, int32_t objective,
                                 double beta, double margin, double label_smoothing, double nll_weight,
                                 double grad_scale, uint32_t flags, float *scalars_out, float *per_pair_out,
                                 float *log_ratio_out, float *logp_out, int32_t grad_dtype, void *d_hidden,
                                 void *d_weight, void *workspace, int64_t workspace_bytes, lossk_stream_t stream)
{
    if (n_pairs < 1) return LOSSK_EMPTY_DIMENSION;
    if (n_pairs > MAX_DIM) return LOSSK_DIMENSION_TOO_LARGE;
    Call c{};
    c.head = true;
    c.n = n, c.d = d, c.V = V, c.n_seq = 2 * n_pairs, c.n_pairs = n_pairs, c.dtype = dtype;
    c.X = hidden, c.x_len = hidden_len, c.W = weight, c.w_len = weight_len;
    c.targets = targets, c.targets_len = targets_len, c.mask = loss_mask, c.first = first, c.first_len = first_len;
    c.ref = ref_logp, c.ref_len = ref_len, c.temperature = 1.0;
    c.objective = objective, c.beta = beta, c.margin = margin, c.smooth = label_smoothing, c.nll = nll_weight;
    c.grad_scale = grad_scale, c.flags = flags, c.scalars = scalars_out, c.per_item = per_pair_out;
    c.log_ratio = log_ratio_out, c.logp = logp_out, c.grad_dtype = grad_dtype, c.g0 = d_hidden, c.g1 = d_weight;
    c.ws = workspace, c.ws_bytes = workspace_bytes, c.st = reinterpret_cast<cudaStream_t>(stream);
    return run(c);
}

int32_t lossk_preference_from_logits(int64_t n, int64_t V, int64_t n_pairs, int32_t dtype, const void *logits,
                                     int64_t logits_len, const int64_t *targets, int64_t targets_len,
                                     const uint8_t *loss_mask, const int32_t *first, int64_t first_len,
                                     const float *ref_logp, int64_t ref_len, int32_t objective, double beta,
                                     double margin, double label_smoothing, double nll_weight, double grad_scale,
                                     uint32_t flags, float *scalars_out, float *per_pair_out, float *log_ratio_out,
                                     float *logp_out, void *grad_logits, int64_t grad_len, void *workspace,
                                     int64_t workspace_bytes, lossk_stream_t stream)
{
    if (n_pairs < 1) return LOSSK_EMPTY_DIMENSION;
    if (n_pairs > MAX_DIM) return LOSSK_DIMENSION_TOO_LARGE;
    Call c{};
    c.n = n, c.V = V, c.n_seq = 2 * n_pairs, c.n_pairs = n_pairs, c.dtype = dtype;
    c.X = logits, c.x_len = logits_len;
    c.targets = targets, c.targets_len = targets_len, c.mask = loss_mask, c.first = first, c.first_len = first_len;
    c.ref = ref_logp, c.ref_len = ref_len, c.temperature = 1.0;
    c.objective = objective, c.beta = beta, c.margin = margin, c.smooth = label_smoothing, c.nll = nll_weight;
    c.grad_scale = grad_scale, c.flags = flags, c.scalars = scalars_out, c.per_item = per_pair_out;
    c.log_ratio = log_ratio_out, c.logp = logp_out, c.g0 = grad_logits, c.g_len = grad_len;
    c.ws = workspace, c.ws_bytes = workspace_bytes, c.st = reinterpret_cast<cudaStream_t>(stream);
    return run(c);
}

} // extern "C"
