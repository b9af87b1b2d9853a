// k_attn.cu -- attention of one new token per sequence over a paged key-value
// cache, split over the cache's length and joined.
//
//   attn_share  per group of sequences: how many leading pages they share
//   attn_plan   the work in units, where there are many groups
//   attn        the split pass (k_attn_mma.cu, k_attn_ffma.cu)
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
// The split pass then ends everywhere at much the same time, and its results
// are few: a run has a partial one only where it begins or ends inside an item.
//
// Measured: a single sequence of 512 tokens takes 9 us (two launches and a
// chain of dependent loads each: lengths, table, tokens), of 131072 tokens 96 us
// (k_attn_mma.cu).  The join's own share is 3 us of the first, 4 us of the second
// (32 rows in 152 pieces) and 6 us for 2048 rows in 2 to 14 pieces: its loads'
// latency, twice (which runs have pieces, then the pieces).  Where it worked out
// the runs itself from the lengths it took 4, 9 and 10 us.
#include "attn_split.cuh"

namespace lossk {

namespace {

constexpr int PLAN_T = 256;
constexpr int SHARE_U = 4;
constexpr int JOIN_FEW = 3, JOIN_MANY = 16;

// Shared tokens of each group: the leading pages whose ids agree in all its
// rows, full in all of them.  With a window the rows have to be equally long,
// for the first token read depends on the length.
// A thread looks at SHARE_U columns at a time (one, in blocks of 256: 16 us
// instead of 5 for one group of 4 beams of 3750 pages).
template <int T> __global__ void __launch_bounds__(T) attn_share_kernel(AttnArgs a)
{
    __shared__ int s_first, s_min, s_max;
    const int g = blockIdx.x, t = threadIdx.x;
    wait_for_stream();
    let_next_start();
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
    for (int base = 0; base < full; base += T * SHARE_U) {
        int32_t v[SHARE_U];
        bool differ[SHARE_U];
#pragma unroll
        for (int u = 0; u < SHARE_U; ++u) {
            const int c = base + u * T + t;
            v[u] = c < full ? row0[c] : 0;
            differ[u] = false;
        }
#pragma unroll 4
        for (int i = 1; i < a.share; ++i)
#pragma unroll
            for (int u = 0; u < SHARE_U; ++u) {
                const int c = base + u * T + t;
                if (c < full) differ[u] |= row0[i * a.table_stride + c] != v[u];
            }
#pragma unroll
        for (int u = 0; u < SHARE_U; ++u)
            if (differ[u]) atomicMin(&s_first, base + u * T + t);
        __syncthreads();
        // (what others find meanwhile lies beyond these columns)
        if (s_first < base + T * SHARE_U) break;
    }
    __syncthreads();
    if (t == 0) a.shared[g] = (s_first < full ? s_first : full) * a.page;
}

// One block: the units before each group, where they are too many for every
// block of the split pass to sum up for itself.
__global__ void __launch_bounds__(PLAN_T) attn_plan_kernel(AttnArgs a)
{
    __shared__ long long s_warp[PLAN_T / 32];
    wait_for_stream();
    let_next_start();
    check_lens(a);
    sum_units(a, a.base, s_warp);
}

// ---- joining -----------------------------------------------------------------------
// An output row's pieces, from its group's shared tokens and from its own,
// weighted by e^(m - M).  A row that one piece covers was written by it.
struct RowPieces {
    const float *pa, *pb;       // this row of the first shared and the first own piece
    int64_t sa, sb;             // floats from piece to piece
    int n_a, n;
    __device__ __forceinline__ const float *at(int i) const { return i < n_a ? pa + i * sa : pb + (i - n_a) * sb; }
};
__device__ __forceinline__ RowPieces row_pieces(const AttnArgs &a, int s, int hq)
{
    const int g = s / a.share, head = hq / a.group, r = hq % a.group;
    const int ri = (s % a.share) * a.group + r, ca = ri / a.mr, cb = r / a.mr;
    const int64_t ia = shared_item(a, g, head, ca), ib = own_item(a, s, head, cb), stride = a.hd + ATTN_ROW;
    // (read before it is known whether there are such items: one wait for all of it)
    const int2 wa = a.share > 1 ? a.runs_a[ia] : make_int2(0, 0), wb = a.runs_b[ib];
    const Span own = attn_span(a, s, g);
    RowPieces p;
    p.sa = a.ra * stride;
    p.sb = a.rb * stride;
    p.pa = a.part_a + ((ia + wa.x) * a.ra + ri % a.mr) * stride;
    p.pb = a.part_b + ((ib + wb.x) * a.rb + r % a.mr) * stride;
    p.n_a = shared_tiles(a, g) > 0 ? wa.y : 0;
    p.n = p.n_a + (own.hi > own.mid ? wb.y : 0);
    if (p.n_a == 0 && p.n == 1) p.n = -1;
    return p;
}

// A row by WPR warps (a block of WPR warps, or of eight rows where it is 1); H
// vectors of four columns a lane.  A warp takes every WPR-th piece, B at a time,
// all their loads in flight together; its maximum runs on as in the split pass.
template <typename T, int H, int WPR>
__global__ void __launch_bounds__(WPR == 1 ? 256 : WPR * 32) attn_join_kernel(AttnArgs a)
{
    constexpr int B = (WPR == 1 ? 4 : 8) / H;              // (a row of one warp has few pieces)
    __shared__ float4 s_o[WPR > 1 ? WPR : 1][32 * H];
    __shared__ float2 s_ml[WPR > 1 ? WPR : 1];
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5, k0 = WPR == 1 ? 0 : warp;
    wait_for_stream();
    // (there are fewer than 2^31 rows)
    const unsigned row = WPR == 1 ? blockIdx.x * 8 + warp : blockIdx.x, n_q = a.n_q;
    if (row >= static_cast<unsigned>(a.n_group) * a.share * n_q) return;
    const RowPieces p = row_pieces(a, static_cast<int>(row / n_q), static_cast<int>(row % n_q));
    if (p.n < 0) return;
    const int words = a.hd >> 2;
    float M = -INFINITY, mz = 0.f, l = 0.f;
    float4 o[H] = {};
    for (int i0 = k0; i0 < p.n; i0 += WPR * B) {
        float2 ml[B];
        float4 x[B][H];
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const int i = i0 + b * WPR;
            ml[b] = make_float2(-INFINITY, 0.f);
            if (i < p.n) {
                const float *d = p.at(i);
                ml[b] = *reinterpret_cast<const float2 *>(d + a.hd);
#pragma unroll
                for (int h = 0; h < H; ++h)
                    if (lane + 32 * h < words) x[b][h] = *reinterpret_cast<const float4 *>(d + 4 * (lane + 32 * h));
            }
        }
        float top = M;
#pragma unroll
        for (int b = 0; b < B; ++b) top = fmaxf(top, ml[b].x);
        mz = top == -INFINITY ? 0.f : top;
        const float old = exp2f(M - mz);
        M = top;
        l *= old;
#pragma unroll
        for (int h = 0; h < H; ++h) o[h] = make_float4(o[h].x * old, o[h].y * old, o[h].z * old, o[h].w * old);
#pragma unroll
        for (int b = 0; b < B; ++b)
            if (i0 + b * WPR < p.n) {
                const float f = exp2f(ml[b].x - mz);
                l += f * ml[b].y;
#pragma unroll
                for (int h = 0; h < H; ++h)
                    if (lane + 32 * h < words) {
                        o[h].x += f * x[b][h].x;
                        o[h].y += f * x[b][h].y;
                        o[h].z += f * x[b][h].z;
                        o[h].w += f * x[b][h].w;
                    }
            }
    }
    T *out = static_cast<T *>(a.out) + static_cast<int64_t>(row) * a.hd;
    if constexpr (WPR == 1) {
        const float inv = l > 0.f ? 1.f / l : 1.f;
#pragma unroll
        for (int h = 0; h < H; ++h)
            if (lane + 32 * h < words) attn_put4(out + 4 * (lane + 32 * h), o[h], inv);
        if (a.lse && lane == 0) a.lse[row] = mz * float(LN2) + logf(l);
    } else {
#pragma unroll
        for (int h = 0; h < H; ++h) s_o[warp][lane + 32 * h] = o[h];
        if (lane == 0) s_ml[warp] = make_float2(M, l);
        __syncthreads();
        // warp h joins the sums of vector h of every lane
        if (warp >= H) return;
        const float2 mine = lane < WPR ? s_ml[lane] : make_float2(-INFINITY, 0.f);
        float top = mine.x;
        for (int x = 16; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
        mz = top == -INFINITY ? 0.f : top;
        const float f = exp2f(mine.x - mz);
        l = f * mine.y;
        for (int x = 16; x; x >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, x);
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < WPR; ++k) {
            const float fk = __shfl_sync(0xFFFFFFFFu, f, k);
            const float4 x = s_o[k][t];
            sum.x += fk * x.x;
            sum.y += fk * x.y;
            sum.z += fk * x.z;
            sum.w += fk * x.w;
        }
        const float inv = l > 0.f ? 1.f / l : 1.f;
        if (t < words) attn_put4(out + 4 * t, sum, inv);
        if (a.lse && t == 0) a.lse[row] = mz * float(LN2) + logf(l);
    }
}

template <typename T, int H> cudaError_t launch_join_h(const AttnArgs &a, cudaStream_t st)
{
    const int64_t rows = static_cast<int64_t>(a.n_group) * a.share * a.n_q;
    const int64_t pieces = a.nw / (static_cast<int64_t>(a.n_group) * a.share * a.n_kv * a.cp) + 1;
    // pieces a row has where lengths are equal.  One, 4 and 16 warps a row take, split pass and join:
    // 52, 54 and 82 us (64 sequences in groups of 8, 2048 rows, pieces 3); 41, 37 and 46 us (33 sequences of
    // up to 9000 tokens, 1056 rows, pieces 5); 100, 100 and 96 us (one of 131072, 32 rows, pieces 153)
    if (pieces > JOIN_MANY)
        return launch(attn_join_kernel<T, H, 16>, dim3(static_cast<unsigned>(rows)), dim3(512), 0, st, a);
    if (pieces > JOIN_FEW)
        return launch(attn_join_kernel<T, H, 4>, dim3(static_cast<unsigned>(rows)), dim3(128), 0, st, a);
    return launch(attn_join_kernel<T, H, 1>, dim3(static_cast<unsigned>((rows + 7) / 8)), dim3(256), 0, st, a);
}
template <typename T> cudaError_t launch_join(const AttnArgs &a, cudaStream_t st)
{
    return a.hd <= 128 ? launch_join_h<T, 1>(a, st) : launch_join_h<T, 2>(a, st);
}

} // namespace

AttnShape attn_shape(int dtype, int hd, int rows)
{
    return dtype == LOSSK_F32 ? attn_ffma_shape(hd, rows) : attn_mma_shape(hd, rows);
}

bool attn_shares(const AttnArgs &a) { return a.share > 1; }
bool attn_plans(const AttnArgs &a) { return a.n_group > BASE_GROUPS; }

cudaError_t launch_attn_share(const AttnArgs &a, cudaStream_t st)
{
    // the more threads the fewer rounds over a long table, and the later a short one is done: 4 beams of
    // 3750 pages took 8 us with 256 threads and 4 with 1024, 8 x 8 of 136 pages 4 and 5
    const dim3 groups(static_cast<unsigned>(a.n_group));
    return a.max_pages <= 256 * SHARE_U ? launch(attn_share_kernel<256>, groups, dim3(256), 0, st, a)
                                        : launch(attn_share_kernel<1024>, groups, dim3(1024), 0, st, a);
}
cudaError_t launch_attn_plan(const AttnArgs &a, cudaStream_t st)
{
    return launch(attn_plan_kernel, dim3(1), dim3(PLAN_T), 0, st, a);
}
cudaError_t launch_attn(int dtype, const AttnArgs &a, cudaStream_t st)
{
    return dtype == LOSSK_F32 ? launch_attn_ffma(a, st) : launch_attn_mma(dtype == LOSSK_F16, a, st);
}
cudaError_t launch_attn_join(int dtype, const AttnArgs &a, cudaStream_t st)
{
    return dtype == LOSSK_F32 ? launch_join<float>(a, st)
         : dtype == LOSSK_BF16 ? launch_join<uint16_t>(a, st) : launch_join<h16_t>(a, st);
}

} // namespace lossk
