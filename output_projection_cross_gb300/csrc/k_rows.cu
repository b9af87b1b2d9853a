// k_rows.cu -- the sequence losses' passes over given logits: per row the
// (max, sum of exponentials) of its logits, and grad_logits = a (softmax - onehot)
// once the row's coefficient a is known.
//
// Both are streams over HBM: 2 bytes read per 16-bit logit and pass, 2 written
// in the second.  Rows are cut into pieces of whole 16-byte vectors, one block
// each, so that few rows fill the GPU and many rows leave no tail.  A row may
// start anywhere (an odd vocabulary): its vectors are those of the address
// space, the first and the last of them partly outside the row and read element by
// element.
#include "../../include/lossk.h"
#include "decode_launch.h"
#include "ptx.cuh"
#include "seq_scalars.cuh"

#include <type_traits>

namespace lossk {

namespace {

constexpr int ROW_T = 256;         // threads per block
constexpr int ROW_U = 4;           // 16-byte loads in flight per thread

__device__ __forceinline__ bool refused(const WsHeader *hdr)
{
    return *reinterpret_cast<const volatile int *>(&hdr->bad_targets) != 0;
}

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

// A row's vectors: `n` of them from `base`, element e of the row at element
// skip + e of them.
template <typename T> struct RowVecs {
    const T *row;
    int skip;
    int64_t n, vocab;
    __device__ RowVecs(const T *r, int64_t V) : row(r), vocab(V)
    {
        skip = static_cast<int>((reinterpret_cast<uintptr_t>(r) & 15) / sizeof(T));
        n = (skip + V + NVEC<T> - 1) / NVEC<T>;
    }
    // first element of vector j in the row (negative for the first one of a row that starts inside it)
    __device__ int64_t at(int64_t j) const { return j * NVEC<T> - skip; }
    __device__ bool whole(int64_t e) const { return e >= 0 && e + NVEC<T> <= vocab; }
};

} // namespace

// (max, sum) in log2 units of x = k2 s over a counted row, or a piece of it.  Each
// vector's maximum first, one rescale if it rose, then its exponentials,
// which do not depend on one another.  fp32 sums of at most a few thousand terms per
// thread.
template <typename T>
__global__ void __launch_bounds__(ROW_T) row_stats_kernel(const SeqLoss l, const SeqScratch w,
                                                          const T *__restrict__ logits, int splits)
{
    constexpr int N = NVEC<T>;
    wait_for_stream();
    if (refused(w.hdr)) return;
    const int c = blockIdx.x / splits, piece = blockIdx.x - c * splits;
    if (c >= w.hdr->n_valid) return;
    const RowVecs<T> r(logits + w.row[c] * l.vocab, l.vocab);
    const int64_t v0 = r.n * piece / splits, v1 = r.n * (piece + 1) / splits;
    float m = -INFINITY, z = 0.f;
    auto vec = [&](const float (&f)[N]) {
        float lm = f[0];
#pragma unroll
        for (int i = 1; i < N; ++i) lm = fmaxf(lm, f[i]);
        if (lm == -INFINITY) {
            // every term is zero, unless there is a NaN, which the maximum passes over
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (f[i] != f[i]) z = f[i];
            return;
        }
        lm *= l.k2;
        if (lm > m) {
            z *= ex2_approx(m - lm);
            m = lm;
        }
        float a = 0.f, b = 0.f;
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            a += ex2_approx(fmaf(f[i], l.k2, -m));
            b += ex2_approx(fmaf(f[i + 1], l.k2, -m));
        }
        z += a + b;
    };
    for (int64_t j0 = v0; j0 < v1; j0 += ROW_T * ROW_U) {
        uint4 v[ROW_U];
#pragma unroll
        for (int u = 0; u < ROW_U; ++u) {
            const int64_t j = j0 + u * ROW_T + threadIdx.x, e = r.at(j);
            if (j < v1 && r.whole(e)) v[u] = __ldg(reinterpret_cast<const uint4 *>(r.row + e));
        }
#pragma unroll
        for (int u = 0; u < ROW_U; ++u) {
            const int64_t j = j0 + u * ROW_T + threadIdx.x, e = r.at(j);
            if (j >= v1) continue;
            float f[N];
            if (r.whole(e)) {
                unpack<T>(v[u], f);
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i) f[i] = e + i >= 0 && e + i < r.vocab ? value(r.row[e + i]) : -INFINITY;
            }
            vec(f);
        }
    }
    // the block's maximum, one rescale of each thread's sum, then plain sums in a fixed order
    __shared__ float sm[ROW_T / 32], sz[ROW_T / 32];
    float M = m;
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = M;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < ROW_T / 32; ++i) M = fmaxf(M, sm[i]);
    if (M > -INFINITY) z *= ex2_approx(m - M);         // (a NaN of a row of nothing else stays)
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    if ((threadIdx.x & 31) == 0) sz[threadIdx.x >> 5] = z;
    __syncthreads();
    if (threadIdx.x != 0) return;
    for (int i = 1; i < ROW_T / 32; ++i) z += sz[i];
    // exponentials that all but a maximum's own terms have gone through: the element's and the
    // thread's, and where a row has several pieces the piece's
    double low = 2 * EX2_LOW;
    if (splits > 1) {
        float2 *p = w.part + static_cast<int64_t>(c) * splits;
        p[piece] = make_float2(M, z);
        __threadfence();
        if (atomicAdd(&w.tick[c], 1) != splits - 1) return;
        // the last piece to arrive joins them all, in their order
        __threadfence();
        M = -INFINITY;
        for (int i = 0; i < splits; ++i) M = fmaxf(M, __ldcg(&p[i].x));
        z = 0.f;
        for (int i = 0; i < splits; ++i) {
            const float2 q = __ldcg(p + i);
            z += M > -INFINITY ? q.y * ex2_approx(q.x - M) : q.y;
        }
        low = 3 * EX2_LOW;
    }
    const float y = value(r.row[w.y[c]]);
    const double lse2 = static_cast<double>(M) + static_cast<double>(log2f(z));
    w.lse2[c] = static_cast<float>(lse2);
    w.lp[c] = y == -INFINITY && z == z
                  ? y
                  : static_cast<float>((static_cast<double>(y) * static_cast<double>(l.k2) - lse2) * LN2 - low);
}

int seq_stat_splits(int64_t n, int64_t vocab, int dtype)
{
    const int64_t bytes = vocab * (dtype == LOSSK_F32 ? 4 : 2);
    // four blocks for each of 152 SMs, pieces of 16 KB (a round of loads) and more; but pieces of
    // 64 KB also where there are many rows, whose last wave of blocks is short then
    int64_t s = (608 + n - 1) / n;
    const int64_t most = bytes / (ROW_T * ROW_U * 16), some = bytes / 65536;
    if (s > most) s = most;
    if (s < some) s = some;
    return static_cast<int>(s < 1 ? 1 : (s > 64 ? 64 : s));
}

cudaError_t launch_seq_stats(int dtype, const SeqLoss &l, const SeqScratch &w, const void *logits, int splits,
                             cudaStream_t st)
{
    Launch k(KK_SEQ_STATS, st);
    const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(l.n_tok) * splits));
    if (dtype == LOSSK_F32)
        return launch(row_stats_kernel<float>, grid, dim3(ROW_T), 0, st, l, w, static_cast<const float *>(logits), splits);
    if (dtype == LOSSK_F16)
        return launch(row_stats_kernel<h16_t>, grid, dim3(ROW_T), 0, st, l, w, static_cast<const h16_t *>(logits), splits);
    return launch(row_stats_kernel<uint16_t>, grid, dim3(ROW_T), 0, st, l, w, static_cast<const uint16_t *>(logits),
                  splits);
}

// grad_logits of a piece of a row.  A coefficient of 0 (a row that does not
// count, a clipped token) writes zeros and reads nothing.
template <typename T, bool ADD>
__global__ void __launch_bounds__(ROW_T) row_grad_kernel(const SeqLoss l, const SeqScratch w,
                                                         const T *__restrict__ logits, T *__restrict__ grad, int splits)
{
    constexpr int N = NVEC<T>;
    wait_for_stream();
    if (refused(w.hdr)) return;
    if (blockIdx.x == 0) seq_scalars<ROW_T>(l, w);
    // the last rows first: the statistics pass has just read them, and the L2 holds them still
    const unsigned at = gridDim.x - 1 - blockIdx.x;
    const int64_t t = at / splits;
    const int piece = at - static_cast<unsigned>(t) * splits;
    const int c = w.slot[t];
    const float4 P = c >= 0 ? w.tokp[c] : make_float4(0.f, 0.f, 0.f, __int_as_float(-1));
    if (ADD && P.y == 0.f) return;
    const RowVecs<T> r(logits + t * l.vocab, l.vocab);
    T *g = grad + t * l.vocab;
    const int64_t v0 = r.n * piece / splits, v1 = r.n * (piece + 1) / splits;
    const int y = __float_as_int(P.w);
    for (int64_t j0 = v0; j0 < v1; j0 += ROW_T * ROW_U) {
        uint4 v[ROW_U], old[ADD ? ROW_U : 1];
#pragma unroll
        for (int u = 0; u < ROW_U; ++u) {
            const int64_t j = j0 + u * ROW_T + threadIdx.x, e = r.at(j);
            if (j < v1 && P.y != 0.f && r.whole(e)) {
                v[u] = __ldcs(reinterpret_cast<const uint4 *>(r.row + e));
                if (ADD) old[ADD ? u : 0] = __ldcs(reinterpret_cast<const uint4 *>(g + e));
            }
        }
#pragma unroll
        for (int u = 0; u < ROW_U; ++u) {
            const int64_t j = j0 + u * ROW_T + threadIdx.x, e = r.at(j);
            if (j >= v1) continue;
            if (!r.whole(e)) {
                for (int i = 0; i < N; ++i) {
                    if (e + i < 0 || e + i >= r.vocab) continue;
                    float x = 0.f;
                    if (P.y != 0.f) {
                        x = P.y * ex2_approx(fmaf(value(r.row[e + i]), l.k2, -P.x));
                        if (e + i == y) x -= P.z;
                        if (ADD) x += value(g[e + i]);
                    }
                    put(g + e + i, x);
                }
                continue;
            }
            float f[N];
            if (P.y != 0.f) {
                unpack<T>(v[u], f);
#pragma unroll
                for (int i = 0; i < N; ++i) f[i] = P.y * ex2_approx(fmaf(f[i], l.k2, -P.x));
                const int64_t dy = y - e;                  // the one-hot term, in one vector of the row
                if (dy >= 0 && dy < N) {
#pragma unroll
                    for (int i = 0; i < N; ++i)
                        if (i == dy) f[i] -= P.z;
                }
                if (ADD) {
                    float o[N];
                    unpack<T>(old[ADD ? u : 0], o);
#pragma unroll
                    for (int i = 0; i < N; ++i) f[i] += o[i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i) f[i] = 0.f;
            }
            __stcs(reinterpret_cast<uint4 *>(g + e), pack<T>(f));
        }
    }
}

template <typename T>
static cudaError_t grad_one(const SeqLoss &l, const SeqScratch &w, const void *logits, void *grad, bool add,
                            cudaStream_t st)
{
    // pieces of 32 KB: two rounds of loads
    int64_t s = l.vocab * static_cast<int64_t>(sizeof(T)) / (2 * ROW_T * ROW_U * 16);
    const int splits = static_cast<int>(s < 1 ? 1 : (s > 1024 ? 1024 : s));
    const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(l.n_tok) * splits));
    return launch(add ? row_grad_kernel<T, true> : row_grad_kernel<T, false>, grid, dim3(ROW_T), 0, st, l, w,
                  static_cast<const T *>(logits), static_cast<T *>(grad), splits);
}

cudaError_t launch_seq_grad(int dtype, const SeqLoss &l, const SeqScratch &w, const void *logits, void *grad,
                            bool accumulate, cudaStream_t st)
{
    Launch k(KK_SEQ_GRAD, st);
    if (dtype == LOSSK_F32) return grad_one<float>(l, w, logits, grad, accumulate, st);
    if (dtype == LOSSK_F16) return grad_one<h16_t>(l, w, logits, grad, accumulate, st);
    return grad_one<uint16_t>(l, w, logits, grad, accumulate, st);
}

} // namespace lossk
