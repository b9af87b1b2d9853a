// k_attn.cu -- attention of one new token per sequence over a paged key-value
// cache, split over the cache's length and joined.
//
//   attn_plan   per group of sequences: how many leading pages they share, and
//               the work in units
//   attn        the split pass
//   attn_join   the partial results of each output row joined
//
// For query row q of a sequence with tokens j in [lo, len):
//   x_j = scale q.k_j,   out = sum_j e^(x_j - m) v_j / sum_j e^(x_j - m)
// computed online: a running maximum m, the sum l and the unnormalised output
// o are rescaled when m rises, so one pass over the keys and values is enough
// and any cut of the tokens into pieces (m, l, o) can be joined afterwards.
//
// The split.  A unit is a tile of KT tokens of one item; an item is a KV head
// of a sequence with up to MR of the query rows that read it, or, where the
// sequences of a group share their leading pages, of the group's shared tokens
// with the rows of all its sequences (read once for all of them).  The units
// are numbered in a row and every warp takes an equal run of them, whatever the
// lengths: a long sequence is cut over many warps, short ones share a warp.
#include "attn_split.cuh"

namespace lossk {

namespace {

constexpr int PLAN_T = 256;
constexpr int ATTN_WARPS = 4;
constexpr int JOIN_WARPS = 8;
constexpr int JOIN_THREADS = JOIN_WARPS * 32;
constexpr int JOIN_W = 1024;

// Shared tokens of each group: the leading pages whose ids agree in all its
// rows, full in all of them.  With a window the rows have to be equally long,
// for the first token read depends on the length.
__global__ void __launch_bounds__(PLAN_T) attn_share_kernel(AttnArgs a)
{
    __shared__ int s_first, s_min, s_max;
    const int g = blockIdx.x, t = threadIdx.x;
    if (t == 0) {
        int mn = 1 << 30, mx = 0;
        for (int i = 0; i < a.share; ++i) {
            const int n = attn_len(a, g * a.share + i);
            mn = n < mn ? n : mn;
            mx = n > mx ? n : mx;
        }
        s_min = mn;
        s_max = mx;
        s_first = mn / a.page;
    }
    __syncthreads();
    const int full = s_min / a.page;
    if (a.window > 0 && s_min != s_max) {
        if (t == 0) a.shared[g] = 0;
        return;
    }
    const int32_t *row0 = a.table + static_cast<int64_t>(g) * a.share * a.table_stride;
    for (int base = 0; base < full; base += PLAN_T) {
        const int c = base + t;
        bool differ = false;
        if (c < full)
            for (int i = 1; i < a.share; ++i) differ |= row0[i * a.table_stride + c] != row0[c];
        if (differ) atomicMin(&s_first, c);
        __syncthreads();
        if (s_first < base + PLAN_T) break;
        __syncthreads();
    }
    __syncthreads();
    if (t == 0) a.shared[g] = (s_first < full ? s_first : full) * a.page;
}

// One block: the units before each group (a prefix sum), base[n_group] their number.
__global__ void __launch_bounds__(PLAN_T) attn_plan_kernel(AttnArgs a)
{
    __shared__ long long s_warp[PLAN_T / 32];
    const int t = threadIdx.x, lane = t & 31;
    long long done = 0;
    for (int base = 0; base < a.n_group; base += PLAN_T) {
        const int g = base + t;
        const long long x = g < a.n_group ? group_units(a, g) : 0;
        if (g < a.n_group)
            for (int i = 0; i < a.share; ++i) {
                const int n = a.lens[g * a.share + i];
                if (n < 0 || n > static_cast<int64_t>(a.max_pages) * a.page)
                    raise_fault(a.fault, LOSSK_TARGET_OUT_OF_RANGE);
            }
        long long inc = x;
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xFFFFFFFFu, inc, o);
            if (lane >= o) inc += y;
        }
        __syncthreads();
        if (lane == 31) s_warp[t >> 5] = inc;
        __syncthreads();
        long long before = 0, all = 0;
        for (int w = 0; w < PLAN_T / 32; ++w) {
            if (w < (t >> 5)) before += s_warp[w];
            all += s_warp[w];
        }
        if (g < a.n_group) a.base[g] = done + before + inc - x;
        done += all;
    }
    if (t == 0) a.base[a.n_group] = done;
}

// ---- CUDA cores ---------------------------------------------------------------------
// One key at a time per warp, a lane holding elements lane, lane + 32, ... of
// the head.
constexpr int SIMT_MR = 4;

template <typename T> __global__ void __launch_bounds__(ATTN_WARPS * 32) attn_simt_kernel(AttnArgs a)
{
    const int lane = threadIdx.x & 31, w = blockIdx.x * ATTN_WARPS + (threadIdx.x >> 5);
    walk_run(a, w, [&](const Piece &p) {
        float q[SIMT_MR][8], o[SIMT_MR][8], m[SIMT_MR], l[SIMT_MR];
        for (int i = 0; i < SIMT_MR; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
            const T *row = static_cast<const T *>(a.q) +
                           (i < p.rows ? row_seq(a, p, i) * a.q_stride + static_cast<int64_t>(row_head(a, p, i)) * a.hd : 0);
            for (int e = 0; e < 8; ++e) {
                q[i][e] = i < p.rows && lane + 32 * e < a.hd ? attn_f(row[lane + 32 * e]) : 0.f;
                o[i][e] = 0.f;
            }
        }
        for (int j = p.t0; j < p.t1; ++j) {
            const int64_t at = token_at(a, p.seq, j);
            if (at < 0) continue;
            const T *k = static_cast<const T *>(a.k) + at + p.head * a.head_stride;
            const T *v = static_cast<const T *>(a.v) + at + p.head * a.head_stride;
            float kv[8], vv[8];
            for (int e = 0; e < 8; ++e) {
                kv[e] = lane + 32 * e < a.hd ? attn_f(k[lane + 32 * e]) : 0.f;
                vv[e] = lane + 32 * e < a.hd ? attn_f(v[lane + 32 * e]) : 0.f;
            }
            for (int i = 0; i < SIMT_MR; ++i) {
                float x = 0.f;
                for (int e = 0; e < 8; ++e) x = fmaf(q[i][e], kv[e], x);
                for (int s = 16; s; s >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, s);
                x *= a.scale_log2;
                const float mn = fmaxf(m[i], x), mz = mn == -INFINITY ? 0.f : mn;
                const float f = exp2f(m[i] - mz), pr = exp2f(x - mz);
                l[i] = l[i] * f + pr;
                for (int e = 0; e < 8; ++e) o[i][e] = o[i][e] * f + pr * vv[e];
                m[i] = mn;
            }
        }
        for (int i = 0; i < p.rows; ++i) {
            if (p.slot < 0) {
                const float inv = l[i] > 0.f ? 1.f / l[i] : 1.f;
                const int64_t row = static_cast<int64_t>(row_seq(a, p, i)) * a.n_q + row_head(a, p, i);
                T *out = static_cast<T *>(a.out) + row * a.hd;
                for (int e = 0; e < 8; ++e)
                    if (lane + 32 * e < a.hd) attn_put(out + lane + 32 * e, o[i][e] * inv);
                if (a.lse && lane == 0) a.lse[row] = (m[i] == -INFINITY ? 0.f : m[i]) * float(LN2) + logf(l[i]);
            } else {
                float *d = p.part + static_cast<int64_t>(i) * (a.hd + ATTN_ROW);
                for (int e = 0; e < 8; ++e)
                    if (lane + 32 * e < a.hd) d[lane + 32 * e] = o[i][e];
                if (lane == 0) {
                    d[a.hd] = m[i];
                    d[a.hd + 1] = l[i];
                }
            }
        }
    });
}

// ---- joining -----------------------------------------------------------------------
// One block per output row: the row's pieces, from the group's shared tokens
// and from its own, weighted by e^(m - M).  A row that one piece covers was
// written by it.
template <typename T> __global__ void __launch_bounds__(JOIN_THREADS) attn_join_kernel(AttnArgs a)
{
    __shared__ __align__(16) float s_o[JOIN_WARPS][256];
    __shared__ float s_w[JOIN_W], s_x[JOIN_WARPS], s_l[JOIN_WARPS];
    const int s = blockIdx.x / a.n_q, hq = blockIdx.x % a.n_q, g = s / a.share;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int head = hq / a.group, r = hq % a.group;
    const long long units = a.base[a.n_group];
    const int nw = warps_used(units, a.nw);
    const int ts = shared_tiles(a, g);
    const Span own = attn_span(a, s, g);
    const int tp = tiles_of(own.hi - own.mid, a.kt);
    // the pieces: n_a of the shared item (from slot a0 on), then n_b of its own
    const int ri = (s % a.share) * a.group + r, ca = ri / a.mr, cb = r / a.mr;
    int n_a = 0, n_b = 0;
    int64_t a0 = 0, b0 = 0;
    if (ts > 0) {
        const long long u = a.base[g] + (static_cast<long long>(head) * a.cs + ca) * units_of(ts) + ITEM_COST;
        const int w0 = warp_of(units, nw, u), w1 = warp_of(units, nw, u + ts - 1);
        n_a = w1 - w0 + 1;
        a0 = (static_cast<int64_t>(g) * a.n_kv + head) * a.cs + ca + w0;
    }
    if (tp > 0) {
        long long u = a.base[g] + static_cast<long long>(units_of(ts)) * a.n_kv * a.cs;
        for (int i = g * a.share; i < s; ++i) {
            const Span x = attn_span(a, i, g);
            u += static_cast<long long>(units_of(tiles_of(x.hi - x.mid, a.kt))) * a.n_kv * a.cp;
        }
        u += (static_cast<long long>(head) * a.cp + cb) * units_of(tp) + ITEM_COST;
        const int w0 = warp_of(units, nw, u), w1 = warp_of(units, nw, u + tp - 1);
        n_b = w1 - w0 + 1;
        b0 = (static_cast<int64_t>(s) * a.n_kv + head) * a.cp + cb + w0;
    }
    if (n_a == 0 && n_b == 1) return;
    const int n = n_a + n_b;
    const int64_t stride = a.hd + ATTN_ROW;
    const float *pa = a.part_a + (a0 * a.ra + ri % a.mr) * stride, *pb = a.part_b + (b0 * a.rb + r % a.mr) * stride;
    const int64_t sa = a.ra * stride, sb = a.rb * stride;
    auto piece = [&](int i) { return i < n_a ? pa + i * sa : pb + (i - n_a) * sb; };
    // the largest m, then each piece's weight e^(m - M), kept for the first JOIN_W pieces
    float M = -INFINITY;
    for (int i = t; i < n; i += JOIN_THREADS) {
        const float m = piece(i)[a.hd];
        if (i < JOIN_W) s_w[i] = m;
        M = fmaxf(M, m);
    }
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
    if (lane == 0) s_x[warp] = M;
    __syncthreads();
    for (int i = 0; i < JOIN_WARPS; ++i) M = fmaxf(M, s_x[i]);
    const float mz = M == -INFINITY ? 0.f : M;
    // each warp adds up its share of the pieces, a lane holding elements 4 lane.. and 128 + 4 lane..
    float4 acc[2] = {};
    float L = 0.f;
    const int words = a.hd >> 2;
#pragma unroll 4
    for (int i = warp; i < n; i += JOIN_WARPS) {
        const float *d = piece(i);
        const float f = exp2f((i < JOIN_W ? s_w[i] : d[a.hd]) - mz);
        L += f * d[a.hd + 1];
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (lane + 32 * h < words) {
                const float4 x = *reinterpret_cast<const float4 *>(d + 4 * (lane + 32 * h));
                acc[h].x += f * x.x;
                acc[h].y += f * x.y;
                acc[h].z += f * x.z;
                acc[h].w += f * x.w;
            }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
        if (lane + 32 * h < words) *reinterpret_cast<float4 *>(&s_o[warp][4 * (lane + 32 * h)]) = acc[h];
    if (lane == 0) s_l[warp] = L;
    __syncthreads();
    L = 0.f;
    for (int i = 0; i < JOIN_WARPS; ++i) L += s_l[i];
    const float inv = L > 0.f ? 1.f / L : 1.f;
    const int64_t row = static_cast<int64_t>(s) * a.n_q + hq;
    for (int e = t; e < a.hd; e += JOIN_THREADS) {
        float x = 0.f;
        for (int i = 0; i < JOIN_WARPS; ++i) x += s_o[i][e];
        attn_put(static_cast<T *>(a.out) + row * a.hd + e, x * inv);
    }
    if (a.lse && t == 0) a.lse[row] = mz * float(LN2) + logf(L);
}

} // namespace

AttnShape attn_shape(int dtype, int hd, int rows)
{
    if (dtype != LOSSK_F32) return attn_mma_shape(hd, rows);
    return AttnShape{SIMT_MR, 32, 8};
}

cudaError_t launch_attn_plan(const AttnArgs &a, cudaStream_t st)
{
    if (a.share > 1) attn_share_kernel<<<static_cast<unsigned>(a.n_group), PLAN_T, 0, st>>>(a);
    attn_plan_kernel<<<1, PLAN_T, 0, st>>>(a);
    return cudaGetLastError();
}
cudaError_t launch_attn(int dtype, const AttnArgs &a, cudaStream_t st)
{
    const unsigned grid = static_cast<unsigned>((a.nw + ATTN_WARPS - 1) / ATTN_WARPS);
    if (dtype != LOSSK_F32) return launch_attn_mma(dtype == LOSSK_F16, a, st);
    attn_simt_kernel<float><<<grid, ATTN_WARPS * 32, 0, st>>>(a);
    return cudaGetLastError();
}
cudaError_t launch_attn_join(int dtype, const AttnArgs &a, cudaStream_t st)
{
    const unsigned grid = static_cast<unsigned>(a.n_group) * a.share * a.n_q;
    if (dtype == LOSSK_F32) attn_join_kernel<float><<<grid, JOIN_THREADS, 0, st>>>(a);
    else if (dtype == LOSSK_BF16) attn_join_kernel<uint16_t><<<grid, JOIN_THREADS, 0, st>>>(a);
    else attn_join_kernel<h16_t><<<grid, JOIN_THREADS, 0, st>>>(a);
    return cudaGetLastError();
}

} // namespace lossk
