// k_rows.cu -- the sequence losses' passes over given logits.
//
// The policy loss by token: a row's coefficient needs its own log-probability only, so
// a cluster of blocks takes a row through all of it, the row's logits in shared memory
// from its statistics to its gradient: each logit is read once and written once
// (policy_rows).  The losses by sequence and pair need the log-probabilities of whole
// sequences before any gradient, more than fits on the chip: a pass for the rows' statistics and
// one for the gradients (row_stats, row_grad).
//
// All are streams over HBM.  A row may start anywhere (an odd vocabulary): its 16-byte
// vectors are those of the address space, the first and the last of them partly outside
// the row and read element by element.
#include "../../include/lossk.h"
#include "decode_launch.h"
#include "float2.cuh"
#include "ptx.cuh"
#include "seq_terms.cuh"

#include <type_traits>

namespace lossk {

namespace {

// Threads per block and 16-byte loads in flight per thread.  Statistics: eight loads, 154 us
// for 2867 rows of 151936 in bf16 and 5.7 for 210 of 32003, against 157 and 9.3 with four;
// blocks of 512 took 165.  Gradients: blocks of 128, 307 us and 7.3, against 307 and 9.4 in
// blocks of 256; of 512 345.
constexpr int ROW_T = 256, ROW_U = 8;
constexpr int GRAD_T = 128, GRAD_U = 4;
// The policy loss by token: two blocks of 512 on an SM with 76 KB of a row each took 212 us for
// 2048 rows of 151936 in bf16 (217 with exponents as scaled distances, which all shapes share); 38 KB in blocks of 256, five to an SM, 231, of 512, four to an
// SM, 249; blocks of 768 247 and of 1024 262.
constexpr int POLICY_T = 512, POLICY_BLOCKS = 2;
constexpr int POLICY_CHUNKS = 4;               // copies that a block's share of a row arrives in
// Rows of up to so many bytes are a warp's each, four or eight to a block (3967 rows of 1086 in bf16, two
// pairs: 47 -> 33 us; a block of 256 threads has half a vector for each of its threads there).
constexpr int64_t SMALL_ROW = 8192;
constexpr int SMALL_U = 4;

template <typename T> constexpr int NVEC = 16 / sizeof(T);

__device__ __forceinline__ float value(float x) { return x; }
__device__ __forceinline__ float value(uint16_t x) { return __uint_as_float(static_cast<uint32_t>(x) << 16); }
__device__ __forceinline__ float value(h16_t x) { return f16_to_f(x.bits); }

template <typename T> __device__ __forceinline__ void unpack(const uint4 &v, float (&f)[NVEC<T>])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(w[i]);
    } else {
        constexpr bool F16 = std::is_same<T, h16_t>::value;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = h16_lo<F16>(w[i]);
            f[2 * i + 1] = h16_hi<F16>(w[i]);
        }
    }
}

template <typename T> __device__ __forceinline__ uint4 pack(const float (&f)[NVEC<T>])
{
    if constexpr (sizeof(T) == 4) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    } else {
        constexpr bool F16 = std::is_same<T, h16_t>::value;
        return make_uint4(pack_16x2<F16>(f[0], f[1]), pack_16x2<F16>(f[2], f[3]), pack_16x2<F16>(f[4], f[5]),
                          pack_16x2<F16>(f[6], f[7]));
    }
}

__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(uint16_t *p, float v) { *p = static_cast<uint16_t>(pack_bf16x2(v, 0.f)); }
__device__ __forceinline__ void put(h16_t *p, float v) { p->bits = static_cast<uint16_t>(pack_f16x2(v, 0.f)); }

// A row's vectors: `n` of them, element e of the row at element skip + e of them.
template <typename T> struct RowVecs {
    const T *row;
    int skip, n, vocab;                        // (a row has at most 2^24 elements)
    __device__ RowVecs(const T *r, int64_t V) : row(r), vocab(static_cast<int>(V))
    {
        skip = static_cast<int>((reinterpret_cast<uintptr_t>(r) & 15) / sizeof(T));
        n = (skip + vocab + NVEC<T> - 1) / NVEC<T>;
    }
    // first element of vector j in the row (negative for the first one of a row that starts inside it)
    __device__ int at(int j) const { return j * NVEC<T> - skip; }
    __device__ bool whole(int e) const { return e >= 0 && e + NVEC<T> <= vocab; }
    // first vector of piece p of `pieces`
    __device__ int piece(int p, int pieces) const { return static_cast<int>(static_cast<int64_t>(n) * p / pieces); }
    // the vector of element e, elements outside the row as -infinity
    __device__ void load_part(int e, float (&f)[NVEC<T>]) const
    {
#pragma unroll
        for (int i = 0; i < NVEC<T>; ++i) f[i] = e + i >= 0 && e + i < vocab ? value(row[e + i]) : -INFINITY;
    }
};

// The largest of a vector's values (of 16-bit ones two an instruction), past NaNs.
template <typename T> __device__ __forceinline__ float vec_max(const uint4 &v)
{
    if constexpr (sizeof(T) == 4) {
        return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
    } else {
        constexpr bool F16 = std::is_same<T, h16_t>::value;
        uint32_t a, b, m;
        if constexpr (F16) {
            asm("max.f16x2 %0, %1, %2;" : "=r"(a) : "r"(v.x), "r"(v.y));
            asm("max.f16x2 %0, %1, %2;" : "=r"(b) : "r"(v.z), "r"(v.w));
            asm("max.f16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
        } else {
            asm("max.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(v.x), "r"(v.y));
            asm("max.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(v.z), "r"(v.w));
            asm("max.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
        }
        return fmaxf(h16_lo<F16>(m), h16_hi<F16>(m));
    }
}

// One vector's terms (f its values, lm the largest) into a running (max m, sum z of 2^(k2 (f - m))):
// one rescale if the maximum rose, then exponentials that do not depend on one another, their
// arguments and sums two an instruction.  m is one of the logits itself, and what is scaled is the
// distance to it: k2 f - k2 m would end where k2 f does (a mask of bf16's or fp32's lowest value, a
// temperature far below 1), and there be no number.
template <int N> __device__ __forceinline__ void add_vec(float &m, float &z, const float (&f)[N], float lm, float k2)
{
    if (lm == -INFINITY) {
        // every term is zero, unless there is a NaN, which the maximum passes over
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (f[i] != f[i]) z = f[i];
        return;
    }
    if (lm > m) {
        z *= ex2_approx((m - lm) * k2);
        m = lm;
    }
    const uint64_t kk = pack2(k2, k2), mm = pack2(-m, -m);
    uint64_t s = 0;
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        float a, b;
        unpack2(mul2(add2(pack2(f[i], f[i + 1]), mm), kk), a, b);
        const uint64_t e = pack2(ex2_approx(a), ex2_approx(b));
        s = i ? add2(s, e) : e;
    }
    float a, b;
    unpack2(s, a, b);
    z += a + b;
}

// The same of a vector partly outside its row.
template <int N> __device__ __forceinline__ void add_part(float &m, float &z, const float (&f)[N], float k2)
{
    float lm = f[0];
#pragma unroll
    for (int i = 1; i < N; ++i) lm = fmaxf(lm, f[i]);
    add_vec<N>(m, z, f, lm, k2);
}

// The block's (max, sum) from its threads': its maximum, one rescale of each thread's sum, then
// plain sums in a fixed order.  Valid in thread 0.
template <int T>
__device__ __forceinline__ void block_stats(float &m, float &z, float k2, float (&sm)[T / 32], float (&sz)[T / 32])
{
    float M = m;
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = M;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < T / 32; ++i) M = fmaxf(M, sm[i]);
    if (M > -INFINITY) z *= ex2_approx((m - M) * k2);  // (a NaN of a row of nothing else stays)
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    if ((threadIdx.x & 31) == 0) sz[threadIdx.x >> 5] = z;
    __syncthreads();
    m = M;
    if (threadIdx.x == 0)
        for (int i = 1; i < T / 32; ++i) z += sz[i];
}

// logp from a row's (max, sum) and its target's logit y.  exps: exponentials that all
// but a maximum's own terms have gone through.
__device__ __forceinline__ float row_logp(const SeqLoss &l, float M, float z, float y, int exps)
{
    return y == -INFINITY && z == z ? y : logp_of(y, M, l.k2, z, ex2_low(z, exps));
}

// A warp's (max, sum) from its lanes', as block_stats; valid in every lane.
__device__ __forceinline__ void warp_stats(float &m, float &z, float k2)
{
    float M = m;
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if (M > -INFINITY) z *= ex2_approx((m - M) * k2);
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    m = M;
}

// Thread tid of a team's (max, sum) over vectors [v0, v1) of a row, U loads in flight.
template <typename T, int TEAM, int U>
__device__ __forceinline__ void scan_row(const RowVecs<T> &r, int v0, int v1, int tid, float k2, float &m, float &z)
{
    constexpr int N = NVEC<T>;
    for (int j0 = v0; j0 < v1; j0 += TEAM * U) {
        uint4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int j = j0 + u * TEAM + tid, e = r.at(j);
            if (j < v1 && r.whole(e)) v[u] = __ldg(reinterpret_cast<const uint4 *>(r.row + e));
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int j = j0 + u * TEAM + tid, e = r.at(j);
            if (j >= v1) continue;
            float f[N];
            if (r.whole(e)) {
                unpack<T>(v[u], f);
                add_vec<N>(m, z, f, vec_max<T>(v[u]), k2);
            } else {
                r.load_part(e, f);
                add_part<N>(m, z, f, k2);
            }
        }
    }
}

// A vector of the gradient from its logits f: a (softmax - onehot), the row's parameters P (its largest
// logit as the reference, so that a common offset of the logits costs no bits).
template <int N> __device__ __forceinline__ void grad_vec(float (&f)[N], const float4 &P, float k2, int e)
{
    const uint64_t kk = pack2(k2, k2), mm = pack2(-P.x, -P.x), pp = pack2(P.y, P.y);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        float a, b;
        unpack2(mul2(add2(pack2(f[i], f[i + 1]), mm), kk), a, b);
        unpack2(mul2(pp, pack2(ex2_approx(a), ex2_approx(b))), f[i], f[i + 1]);
    }
    const int dy = __float_as_int(P.w) - e;                // the one-hot term, in one vector of the row
    if (dy >= 0 && dy < N) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i == dy) f[i] -= P.z;
    }
}

// The elements of a vector that lie in the row, written (ADD: added to what is there).
template <typename T, bool ADD> __device__ __forceinline__ void put_part(const RowVecs<T> &r, T *g, int e, const float (&f)[NVEC<T>])
{
#pragma unroll
    for (int i = 0; i < NVEC<T>; ++i)
        if (e + i >= 0 && e + i < r.vocab) put(g + e + i, ADD ? f[i] + value(g[e + i]) : f[i]);
}

// Vectors [v0, v1) of a row's gradient by thread tid of a team.
template <typename T, bool ADD, int TEAM, int U>
__device__ __forceinline__ void write_row(const RowVecs<T> &r, T *g, int v0, int v1, int tid, const float4 &P, float k2)
{
    constexpr int N = NVEC<T>;
    for (int j0 = v0; j0 < v1; j0 += TEAM * U) {
        uint4 v[U], old[ADD ? U : 1];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int j = j0 + u * TEAM + tid, e = r.at(j);
            if (j < v1 && P.z != 0.f && r.whole(e)) {
                v[u] = __ldcs(reinterpret_cast<const uint4 *>(r.row + e));
                if (ADD) old[ADD ? u : 0] = __ldcs(reinterpret_cast<const uint4 *>(g + e));
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int j = j0 + u * TEAM + tid, e = r.at(j);
            if (j >= v1) continue;
            float f[N] = {};
            const bool whole = r.whole(e);
            if (P.z != 0.f) {
                if (whole) unpack<T>(v[u], f);
                else r.load_part(e, f);
                grad_vec<N>(f, P, k2, e);
            }
            if (!whole) {
                put_part<T, ADD>(r, g, e, f);
                continue;
            }
            if (ADD) {
                float o[N];
                unpack<T>(old[ADD ? u : 0], o);
#pragma unroll
                for (int i = 0; i < N; ++i) f[i] += o[i];
            }
            __stcs(reinterpret_cast<uint4 *>(g + e), pack<T>(f));
        }
    }
}

} // namespace

// Whether row t counts, from the call's inputs (`first` may be wrong still).
__device__ __forceinline__ bool row_counts(const SeqLoss &l, int64_t t)
{
    return (!l.mask || l.mask[t] != 0) && (!l.first || (t >= l.first[0] && t < l.first[l.n_seq]));
}

// logp, largest logit and sum of a counted row, which comes in pieces of one block each; the last piece to
// arrive joins them all, in their order.  SMALL: a warp per row.  The rows' numbering runs beside
// the first rows: all that their statistics read is the call's inputs, which were there before it
// began (let_next_start), and results wait for it: 1531 rows of 32003 in fp32, by sequence, 108.9 -> 103.8
// us a call, 300 in fp16, in pairs, 30.9 -> 27.8.
template <typename T, bool SMALL>
__global__ void __launch_bounds__(ROW_T) row_stats_kernel(const SeqLoss l, const SeqScratch w,
                                                          const T *__restrict__ logits, int splits)
{
    constexpr int TEAM = SMALL ? 32 : ROW_T;
    const int64_t at = SMALL ? static_cast<int64_t>(blockIdx.x) * (ROW_T / 32) + (threadIdx.x >> 5) : blockIdx.x;
    const int64_t t = SMALL ? at : at / splits;
    const int piece = SMALL ? 0 : static_cast<int>(at - t * splits), tid = threadIdx.x % TEAM;
    if (t >= l.n_tok || !row_counts(l, t)) {
        wait_for_stream();                     // (this kernel must not end before the one ahead)
        return;
    }
    const RowVecs<T> r(logits + t * l.vocab, l.vocab);
    float y = 0.f;
    if (tid == 0) {
        const int64_t target = l.targets[t];
        if (target >= 0 && target < l.vocab) y = value(r.row[target]);
    }
    float m = -INFINITY, z = 0.f;
    if constexpr (SMALL) {
        scan_row<T, 32, SMALL_U>(r, 0, r.n, tid, l.k2, m, z);
        warp_stats(m, z, l.k2);
    } else {
        scan_row<T, ROW_T, ROW_U>(r, r.piece(piece, splits), r.piece(piece + 1, splits), tid, l.k2, m, z);
        __shared__ float sm[ROW_T / 32], sz[ROW_T / 32];
        block_stats<ROW_T>(m, z, l.k2, sm, sz);
    }
    if (tid != 0) return;
    wait_for_stream();
    const int c = w.slot[t];
    if (seq_refused(w.hdr)) return;
    if (splits > 1) {
        float2 *p = w.part + static_cast<int64_t>(c) * splits;
        p[piece] = make_float2(m, z);
        __threadfence();
        if (atomicAdd(&w.tick[c], 1) != splits - 1) return;
        __threadfence();
        m = -INFINITY;
        for (int i = 0; i < splits; ++i) m = fmaxf(m, __ldcg(&p[i].x));
        z = 0.f;
        for (int i = 0; i < splits; ++i) {
            const float2 q = __ldcg(p + i);
            z += m > -INFINITY ? q.y * ex2_approx((q.x - m) * l.k2) : q.y;
        }
    }
    w.lp[c] = row_logp(l, m, z, y, splits > 1 ? 3 : 2);
    w.ref[c] = m;
    w.share[c] = 1.f / z;
}

int seq_stat_splits(int64_t n, int64_t vocab, int dtype)
{
    const int64_t bytes = vocab * (dtype == LOSSK_F32 ? 4 : 2);
    // a row whole, or, where that makes fewer than four blocks for each of 152 SMs, in pieces of down
    // to 16 KB
    int64_t s = (608 + n - 1) / n;
    const int64_t most = bytes / 16384;
    if (s > most) s = most;
    return static_cast<int>(s < 1 ? 1 : (s > 64 ? 64 : s));
}

template <typename T>
static cudaError_t stats_one(const SeqLoss &l, const SeqScratch &w, const void *logits, int splits, cudaStream_t st)
{
    const bool small = l.vocab * static_cast<int64_t>(sizeof(T)) <= SMALL_ROW;
    const int64_t grid = small ? (l.n_tok + ROW_T / 32 - 1) / (ROW_T / 32) : static_cast<int64_t>(l.n_tok) * splits;
    return launch(small ? row_stats_kernel<T, true> : row_stats_kernel<T, false>, dim3(static_cast<unsigned>(grid)),
                  dim3(ROW_T), 0, st, l, w, static_cast<const T *>(logits), splits);
}

cudaError_t launch_seq_stats(int dtype, const SeqLoss &l, const SeqScratch &w, const void *logits, int splits,
                             cudaStream_t st)
{
    Launch k(KK_SEQ_STATS, st);
    if (dtype == LOSSK_F32) return stats_one<float>(l, w, logits, splits, st);
    if (dtype == LOSSK_F16) return stats_one<h16_t>(l, w, logits, splits, st);
    return stats_one<uint16_t>(l, w, logits, splits, st);
}

// grad_logits of a piece of a row.  A coefficient of 0 (a row that does not
// count, a clipped token) writes zeros and reads nothing.
template <typename T, bool ADD, bool SMALL>
__global__ void __launch_bounds__(GRAD_T) row_grad_kernel(const SeqLoss l, const SeqScratch w,
                                                         const T *logits, T *grad, int splits)
{
    wait_for_stream();
    if (seq_refused(w.hdr)) return;
    if (blockIdx.x == 0) seq_scalars<GRAD_T>(l, w);
    if constexpr (SMALL) {
        const int t = blockIdx.x * (GRAD_T / 32) + (threadIdx.x >> 5);
        if (t >= l.n_tok) return;
        const int c = w.slot[t];
        const float4 P = c >= 0 ? w.tokp[c] : make_float4(0.f, 0.f, 0.f, __int_as_float(-1));
        if (ADD && P.z == 0.f) return;
        const RowVecs<T> r(logits + t * l.vocab, l.vocab);
        write_row<T, ADD, 32, SMALL_U>(r, grad + t * l.vocab, 0, r.n, threadIdx.x & 31, P, l.k2);
        return;
    }
    // the last rows first: the statistics pass has just read them, and the L2 holds them still
    const unsigned at = gridDim.x - 1 - blockIdx.x;
    const int64_t t = at / splits;
    const int piece = at - static_cast<unsigned>(t) * splits;
    const int c = w.slot[t];
    const float4 P = c >= 0 ? w.tokp[c] : make_float4(0.f, 0.f, 0.f, __int_as_float(-1));
    if (ADD && P.z == 0.f) return;
    const RowVecs<T> r(logits + t * l.vocab, l.vocab);
    T *g = grad + t * l.vocab;
    const int v0 = r.piece(piece, splits), v1 = r.piece(piece + 1, splits);
    write_row<T, ADD, GRAD_T, GRAD_U>(r, g, v0, v1, threadIdx.x, P, l.k2);
}

template <typename T>
static cudaError_t grad_one(const SeqLoss &l, const SeqScratch &w, const void *logits, void *grad, bool add,
                            cudaStream_t st)
{
    // pieces of 16 KB: two rounds of loads
    int64_t s = l.vocab * static_cast<int64_t>(sizeof(T)) / (2 * GRAD_T * GRAD_U * 16);
    const int splits = static_cast<int>(s < 1 ? 1 : (s > 1024 ? 1024 : s));
    const bool small = l.vocab * static_cast<int64_t>(sizeof(T)) <= SMALL_ROW;
    const int64_t grid = small ? (l.n_tok + GRAD_T / 32 - 1) / (GRAD_T / 32) : static_cast<int64_t>(l.n_tok) * splits;
    auto kern = small ? (add ? row_grad_kernel<T, true, true> : row_grad_kernel<T, false, true>)
                      : (add ? row_grad_kernel<T, true, false> : row_grad_kernel<T, false, false>);
    return launch(kern, dim3(static_cast<unsigned>(grid)), dim3(GRAD_T), 0, st, l, w, static_cast<const T *>(logits),
                  static_cast<T *>(grad), splits);
}

cudaError_t launch_seq_grad(int dtype, const SeqLoss &l, const SeqScratch &w, const void *logits, void *grad,
                            bool accumulate, cudaStream_t st)
{
    Launch k(KK_SEQ_GRAD, st);
    if (dtype == LOSSK_F32) return grad_one<float>(l, w, logits, grad, accumulate, st);
    if (dtype == LOSSK_F16) return grad_one<h16_t>(l, w, logits, grad, accumulate, st);
    return grad_one<uint16_t>(l, w, logits, grad, accumulate, st);
}

// ---- the policy loss by token ------------------------------------------------------
// A cluster of C blocks per row, each with its share of the row in shared memory: it arrives in
// bulk copies, its statistics are taken on the way in, the blocks' (max, sum) exchanged through
// one another's shared memory, then the coefficient, then the gradient from shared memory.  What
// bounds it is HBM, one read and one write a logit (5.3 TB/s of 6.8), and what keeps it from that
// is a row's chain: copy, sums, exchange, coefficient, stores, with two rows in flight on an SM.
constexpr int64_t POLICY_SHARE = 80000, POLICY_MOST = 112640;      // bytes of a row per block: as a rule, and at most

int policy_rows_cluster(int64_t n, int64_t vocab, int dtype)
{
    const int64_t bytes = vocab * (dtype == LOSSK_F32 ? 4 : 2);
    int c = 1;
    while (c < 8 && bytes > c * POLICY_SHARE) c *= 2;
    // few rows: more blocks for each, down to 8 KB
    while (c < 8 && n * c < 304 && bytes > 2 * c * 8192) c *= 2;
    return bytes > c * POLICY_MOST ? 0 : c;
}

// Every block has its place at once: the rows' copies and statistics run beside the kernel that
// numbers the rows (48 rows of 32000 in bf16 17.9 -> 15.0 us a call).  With more rows than that what
// comes after the wait would be in every row's chain (2048 of 151936: 226 -> 234).
bool policy_rows_early(int64_t n, int64_t vocab, int dtype, int cluster)
{
    return vocab * (dtype == LOSSK_F32 ? 4 : 2) > SMALL_ROW && n * cluster <= 152 * POLICY_BLOCKS;
}

namespace {

// What the policy loss reads for row t, counted.
__device__ __forceinline__ RowInputs slot_inputs(const SeqLoss &l, const SeqScratch &w, int t)
{
    int s = 0, n_s = 0;
    if (l.n_seq > 0 && (l.flags & (LOSSK_SEQ_MEAN | LOSSK_SEQ_ADVANTAGES))) {
        const int c = w.slot[t];
        int hi = l.n_seq;                      // the last sequence that starts at or before slot c
        while (hi - s > 1) {
            const int mid = (s + hi) >> 1;
            if (w.seq_slot[mid] <= c) s = mid;
            else hi = mid;
        }
        n_s = w.seq_slot[s + 1] - w.seq_slot[s];
    }
    return policy_inputs(l, w.hdr, t, s, n_s);
}

} // namespace

// Small rows, a warp each: the second read finds them in the L1 or L2.  GRAD: 0 none, 1
// written, 2 added to what is there.
template <typename T, int GRAD>
__global__ void __launch_bounds__(GRAD_T) policy_small_kernel(const SeqLoss l, const SeqScratch w, const T *logits, T *grad)
{
    wait_for_stream();
    const int t = blockIdx.x * (GRAD_T / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int c = t < l.n_tok ? w.slot[t] : -1;
    if (t >= l.n_tok || seq_refused(w.hdr)) return;
    const RowVecs<T> r(logits + t * l.vocab, l.vocab);
    float4 P = make_float4(0.f, 0.f, 0.f, __int_as_float(-1)), terms = make_float4(0.f, 0.f, 0.f, 0.f);
    if (c >= 0) {
        RowInputs in{};
        int64_t target = 0;
        float y = 0.f;
        if (lane == 0) {
            target = w.y[c];
            y = value(r.row[target]);
            in = slot_inputs(l, w, t);
        }
        float m = -INFINITY, z = 0.f;
        scan_row<T, 32, SMALL_U>(r, 0, r.n, lane, l.k2, m, z);
        warp_stats(m, z, l.k2);
        if (lane == 0) {
            const float lp = row_logp(l, m, z, y, 2);
            const RowTerms x = policy_row(l, in, t, lp, 0.0, 0.f);
            if (l.logp) l.logp[t] = lp;
            P = row_params(m, 1.f / z, x.coef, target);
            terms = make_float4(x.v[0], x.v[1], x.v[2], 0.f);
        }
        P.x = __shfl_sync(0xffffffffu, P.x, 0);
        P.y = __shfl_sync(0xffffffffu, P.y, 0);
        P.z = __shfl_sync(0xffffffffu, P.z, 0);
        P.w = __shfl_sync(0xffffffffu, P.w, 0);
    } else if (lane == 0) {
        if (l.logp) l.logp[t] = 0.f;
        if (l.per_token) l.per_token[t] = 0.f;
    }
    if (lane == 0) w.terms[t] = terms;
    if (GRAD == 1 || (GRAD == 2 && P.z != 0.f))
        write_row<T, GRAD == 2, 32, SMALL_U>(r, grad + t * l.vocab, 0, r.n, lane, P, l.k2);
}

// GRAD: 0 none, 1 written, 2 added to what is there.  EARLY: policy_rows_early().
template <typename T, int GRAD, bool EARLY>
__global__ void __launch_bounds__(POLICY_T, POLICY_BLOCKS) policy_rows_kernel(const SeqLoss l, const SeqScratch w, const T *logits, T *grad,
                                                            int cluster)
{
    constexpr int N = NVEC<T>;
    constexpr bool ADD = GRAD == 2;
    extern __shared__ uint4 s_row[];
    __shared__ uint64_t s_bar[POLICY_CHUNKS];
    __shared__ float sm[POLICY_T / 32], sz[POLICY_T / 32];
    __shared__ float2 s_part[8];
    __shared__ float4 s_param;
    if (threadIdx.x == 0) {
        for (int i = 0; i < POLICY_CHUNKS; ++i) mbar_init(&s_bar[i], 1);
        fence_mbarrier_init();
    }
    __syncthreads();
    // (waited for beside the row's copies, ahead of the first store into another block's memory)
    if (cluster > 1) cluster_arrive_started();
    const int t = blockIdx.x / cluster, rank = blockIdx.x - t * cluster, tid = threadIdx.x;
    // Early: all that the copies and the statistics read is the call's inputs, which were there before
    // the kernel ahead began (let_next_start), and which row counts follows from them.
    bool on;
    if constexpr (!EARLY) {
        wait_for_stream();
        on = w.slot[t] >= 0;                   // (asked for beside the refusal)
        if (seq_refused(w.hdr)) {
            if (cluster > 1) cluster_wait_started();
            return;
        }
    } else {
        on = row_counts(l, t);
    }
    const RowVecs<T> r(logits + t * l.vocab, l.vocab);
    const int v0 = r.piece(rank, cluster), v1 = r.piece(rank + 1, cluster);
    T *g = GRAD ? grad + t * l.vocab : nullptr;
    float4 P = make_float4(0.f, 0.f, 0.f, __int_as_float(-1));
    float4 terms = make_float4(0.f, 0.f, 0.f, 0.f);
    float m = -INFINITY, z = 0.f, y = 0.f;
    int64_t target = 0;
    RowInputs in{};
    if (on) {
        // the share's whole vectors arrive in chunks
        const int va = v0 < v1 && !r.whole(r.at(v0)) ? v0 + 1 : v0;
        const int vb = v1 > va && !r.whole(r.at(v1 - 1)) ? v1 - 1 : v1, nv = max(vb - va, 0);
        auto chunk = [&](int k) { return va + nv * k / POLICY_CHUNKS; };
        if (tid == 0)
            for (int k = 0; k < POLICY_CHUNKS; ++k) {
                const uint32_t bytes = static_cast<uint32_t>(chunk(k + 1) - chunk(k)) * 16;
                mbar_arrive_expect_tx(&s_bar[k], bytes);
                if (bytes) bulk_copy_g2s(s_row + chunk(k) - v0, r.row + r.at(chunk(k)), bytes, &s_bar[k]);
            }
        // what does not come from the row's statistics, asked for before they are taken
        if (tid == 0) {
            target = l.targets[t];
            y = !EARLY || (target >= 0 && target < l.vocab) ? value(r.row[target]) : 0.f;
            if (!EARLY) in = slot_inputs(l, w, t);
        }
        // the first and the last vector where they are partly outside the row
        if ((tid == 0 && va > v0) || (tid == 1 && vb < v1)) {
            float f[N];
            r.load_part(r.at(tid == 0 ? v0 : v1 - 1), f);
            add_part<N>(m, z, f, l.k2);
        }
        for (int k = 0; k < POLICY_CHUNKS; ++k) {
            // (a wait that ran out: the error word says so, and the call's status)
            if (!mbar_wait(&s_bar[k], 0, &w.hdr->err)) mbar_drain(&s_bar[k], 0);
            for (int j = chunk(k) + tid; j < chunk(k + 1); j += POLICY_T) {
                const uint4 v = s_row[j - v0];
                float f[N];
                unpack<T>(v, f);
                add_vec<N>(m, z, f, vec_max<T>(v), l.k2);
            }
        }
        block_stats<POLICY_T>(m, z, l.k2, sm, sz);
        if (cluster > 1) {
            __syncwarp();
            cluster_wait_started();
            if (tid == 0)
                for (int q = 0; q < cluster; ++q)
                    st_cluster_f2(mapa_shared(smem_u32(&s_part[rank]), q), make_float2(m, z));
            __syncwarp();
            cluster_sync();
            if (tid == 0) {
                m = -INFINITY;
                for (int q = 0; q < cluster; ++q) m = fmaxf(m, s_part[q].x);
                z = 0.f;
                for (int q = 0; q < cluster; ++q)
                    z += m > -INFINITY ? s_part[q].y * ex2_approx((s_part[q].x - m) * l.k2) : s_part[q].y;
            }
        }
    } else if (cluster > 1) {
        cluster_wait_started();                // (a row counts in all blocks of its cluster, or in none)
    }
    if constexpr (EARLY) {
        wait_for_stream();
        let_next_start();
        if (seq_refused(w.hdr)) return;
        if (on && tid == 0) in = slot_inputs(l, w, t);
    }
    if (on) {
        if (tid == 0) {
            const float lp = row_logp(l, m, z, y, cluster > 1 ? 3 : 2);
            const RowTerms x = policy_row(l, in, t, lp, 0.0, 0.f, rank == 0);
            if (rank == 0 && l.logp) l.logp[t] = lp;
            s_param = row_params(m, 1.f / z, x.coef, target);
            terms = make_float4(x.v[0], x.v[1], x.v[2], 0.f);
        }
        __syncthreads();
        P = s_param;
    } else if (rank == 0 && tid == 0) {
        if (l.logp) l.logp[t] = 0.f;
        if (l.per_token) l.per_token[t] = 0.f;
    }
    if (GRAD == 1 || (GRAD == 2 && P.z != 0.f)) {
        for (int j = v0 + tid; j < v1; j += POLICY_T) {
            const int e = r.at(j);
            const bool whole = r.whole(e);
            float f[N] = {};
            if (P.z != 0.f) {
                if (whole) unpack<T>(s_row[j - v0], f);
                else r.load_part(e, f);
                grad_vec<N>(f, P, l.k2, e);
            }
            if (!whole) {
                put_part<T, ADD>(r, g, e, f);
                continue;
            }
            if (ADD) {
                float o[N];
                unpack<T>(__ldcs(reinterpret_cast<const uint4 *>(g + e)), o);
#pragma unroll
                for (int i = 0; i < N; ++i) f[i] += o[i];
            }
            __stcs(reinterpret_cast<uint4 *>(g + e), pack<T>(f));
        }
    }
    if (rank == 0 && tid == 0) w.terms[t] = terms;
}

// The scalars: every thread every 1024th row's terms in order, then a fixed tree.  (Added by the
// last row to arrive they cost every row a fence and an atomic, with its shared memory held.)
__global__ void __launch_bounds__(1024) policy_scalars_kernel(const SeqLoss l, const SeqScratch w)
{
    wait_for_stream();
    if (seq_refused(w.hdr)) return;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    double v[3] = {0.0, 0.0, 0.0};
    int n = 0;
    for (int i = threadIdx.x; i < l.n_tok; i += 1024) {
        const float4 x = w.terms[i];
        a.x += x.x;
        a.y += x.y;
        a.z += x.z;
        if (++n == 8) {                        // eight in floats, then doubles, which are slow here
            v[0] += a.x;
            v[1] += a.y;
            v[2] += a.z;
            a = make_float4(0.f, 0.f, 0.f, 0.f);
            n = 0;
        }
    }
    v[0] += a.x;
    v[1] += a.y;
    v[2] += a.z;
#pragma unroll
    for (int k = 0; k < 3; ++k)
        for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    __shared__ double s_sum[3][32];
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int k = 0; k < 3; ++k) s_sum[k][threadIdx.x >> 5] = v[k];
    __syncthreads();
    if (threadIdx.x >= 32) return;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        v[k] = s_sum[k][threadIdx.x];
        for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    }
    if (threadIdx.x == 0) write_scalars(l, w.hdr, v[0], v[1], v[2]);
}

template <typename T, int GRAD, bool EARLY>
static cudaError_t policy_one(const SeqLoss &l, const SeqScratch &w, const void *logits, void *grad, int cluster,
                              cudaStream_t st)
{
    if constexpr (!EARLY)
        if (l.vocab * static_cast<int64_t>(sizeof(T)) <= SMALL_ROW)
            return launch(policy_small_kernel<T, GRAD>, dim3(static_cast<unsigned>((l.n_tok + GRAD_T / 32 - 1) / (GRAD_T / 32))),
                          dim3(GRAD_T), 0, st, l, w, static_cast<const T *>(logits), static_cast<T *>(grad));
    constexpr auto K = policy_rows_kernel<T, GRAD, EARLY>;
    // a share of the row's vectors, rounded up, and the one that a row may begin in
    const size_t smem = static_cast<size_t>((l.vocab / NVEC<T> + 2) / cluster + 2) * 16;
    cudaError_t e = raise_smem<K>(smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(static_cast<int64_t>(l.n_tok) * cluster));
    cfg.blockDim = dim3(POLICY_T);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, K, l, w, static_cast<const T *>(logits), static_cast<T *>(grad), cluster);
}

template <typename T>
static cudaError_t policy_type(const SeqLoss &l, const SeqScratch &w, const void *logits, void *grad, bool add,
                               int cluster, cudaStream_t st)
{
    auto one = [&](auto early) {
        constexpr bool E = decltype(early)::value;
        if (!grad) return policy_one<T, 0, E>(l, w, logits, grad, cluster, st);
        return add ? policy_one<T, 2, E>(l, w, logits, grad, cluster, st)
                   : policy_one<T, 1, E>(l, w, logits, grad, cluster, st);
    };
    return l.early ? one(std::true_type{}) : one(std::false_type{});
}

cudaError_t launch_policy_rows(int dtype, const SeqLoss &l, const SeqScratch &w, const void *logits, void *grad,
                               bool accumulate, int cluster, cudaStream_t st)
{
    cudaError_t e;
    {
        Launch k(KK_POLICY_ROWS, st);
        if (dtype == LOSSK_F32) e = policy_type<float>(l, w, logits, grad, accumulate, cluster, st);
        else if (dtype == LOSSK_F16) e = policy_type<h16_t>(l, w, logits, grad, accumulate, cluster, st);
        else e = policy_type<uint16_t>(l, w, logits, grad, accumulate, cluster, st);
    }
    if (e != cudaSuccess) return e;
    Launch k(KK_REDUCE, st);
    return launch(policy_scalars_kernel, dim3(1), dim3(1024), 0, st, l, w);
}

} // namespace lossk
