// k_attn.cu -- attention of one new token per sequence over a paged key-value
// cache, split over the cache's length and joined.
//
//   attn_plan   per group of sequences: how many leading pages they share, and
//               the work in units
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
// Measured: a single sequence of 512 tokens takes 10 us (two launches and a
// chain of dependent loads each: lengths, table, tokens), of 131072 tokens 99 to
// 103 us (k_attn_mma.cu); the join takes 4 us of the first and 9 us for 2048 rows
// in 2 to 14 pieces.
#include "attn_split.cuh"

namespace lossk {

namespace {

constexpr int PLAN_T = 256;
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
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
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

// One block: the units before each group, where they are too many for every
// block of the split pass to sum up for itself.
__global__ void __launch_bounds__(PLAN_T) attn_plan_kernel(AttnArgs a)
{
    __shared__ long long s_warp[PLAN_T / 32];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
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
    const long long units = a.base[a.n_group];
    const Runs runs(units, a.nw);
    const int ts = shared_tiles(a, g);
    const Span own = attn_span(a, s, g);
    const int tp = tiles_of(own.hi - own.mid, a.kt);
    const int ri = (s % a.share) * a.group + r, ca = ri / a.mr, cb = r / a.mr;
    const int64_t stride = a.hd + ATTN_ROW;
    RowPieces p{nullptr, nullptr, a.ra * stride, a.rb * stride, 0, 0};
    if (ts > 0) {
        const long long u = a.base[g] + (static_cast<long long>(head) * a.cs + ca) * units_of(ts) + ITEM_COST;
        const int w0 = runs.of(u), w1 = runs.of(u + ts - 1);
        p.n_a = w1 - w0 + 1;
        p.pa = a.part_a + (((static_cast<int64_t>(g) * a.n_kv + head) * a.cs + ca + w0) * a.ra + ri % a.mr) * stride;
    }
    p.n = p.n_a;
    if (tp > 0) {
        long long u = a.base[g] + static_cast<long long>(units_of(ts)) * a.n_kv * a.cs;
        for (int i = g * a.share; i < s; ++i) {
            const Span x = attn_span(a, i, g);
            u += static_cast<long long>(units_of(tiles_of(x.hi - x.mid, a.kt))) * a.n_kv * a.cp;
        }
        u += (static_cast<long long>(head) * a.cp + cb) * units_of(tp) + ITEM_COST;
        const int w0 = runs.of(u), w1 = runs.of(u + tp - 1);
        p.n += w1 - w0 + 1;
        p.pb = a.part_b + (((static_cast<int64_t>(s) * a.n_kv + head) * a.cp + cb + w0) * a.rb + r % a.mr) * stride;
    }
    if (p.n_a == 0 && p.n == 1) p.n = -1;
    return p;
}

// The weighted sum of pieces i0, i0 + step, ...: a lane holds elements 4 lane..
// and 128 + 4 lane..
struct RowSum {
    float4 o[2];
    float l;
};
template <typename W>
__device__ __forceinline__ RowSum sum_pieces(const RowPieces &p, int hd, int i0, int step, int lane, W &&weight)
{
    RowSum r = {};
    const int words = hd >> 2;
#pragma unroll 4
    for (int i = i0; i < p.n; i += step) {
        const float *d = p.at(i);
        const float f = weight(i, d);
        r.l += f * d[hd + 1];
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (lane + 32 * h < words) {
                const float4 x = *reinterpret_cast<const float4 *>(d + 4 * (lane + 32 * h));
                r.o[h].x += f * x.x;
                r.o[h].y += f * x.y;
                r.o[h].z += f * x.z;
                r.o[h].w += f * x.w;
            }
    }
    return r;
}

template <typename T>
__device__ __forceinline__ void put_row(const AttnArgs &a, int64_t row, int lane, const RowSum &r, float mz)
{
    const float inv = r.l > 0.f ? 1.f / r.l : 1.f;
    T *out = static_cast<T *>(a.out) + row * a.hd;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int e = 4 * (lane + 32 * h);
        if (e < a.hd) {
            attn_put(out + e, r.o[h].x * inv);
            attn_put(out + e + 1, r.o[h].y * inv);
            attn_put(out + e + 2, r.o[h].z * inv);
            attn_put(out + e + 3, r.o[h].w * inv);
        }
    }
    if (a.lse && lane == 0) a.lse[row] = mz * float(LN2) + logf(r.l);
}

// A warp per output row: many rows, of few pieces each.
template <typename T> __global__ void __launch_bounds__(JOIN_THREADS) attn_join_rows_kernel(AttnArgs a)
{
    const int lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * JOIN_WARPS + (threadIdx.x >> 5);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (row >= static_cast<int64_t>(a.n_group) * a.share * a.n_q) return;
    const RowPieces p = row_pieces(a, static_cast<int>(row / a.n_q), static_cast<int>(row % a.n_q));
    if (p.n < 0) return;
    float M = -INFINITY;
    for (int i = lane; i < p.n; i += 32) M = fmaxf(M, p.at(i)[a.hd]);
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
    const float mz = M == -INFINITY ? 0.f : M;
    const RowSum r = sum_pieces(p, a.hd, 0, 1, lane, [&](int, const float *d) { return exp2f(d[a.hd] - mz); });
    put_row<T>(a, row, lane, r, mz);
}

// A block per output row: few rows, cut into many pieces.
template <typename T> __global__ void __launch_bounds__(JOIN_THREADS) attn_join_kernel(AttnArgs a)
{
    __shared__ float4 s_o[JOIN_WARPS][64];
    __shared__ float s_w[JOIN_W], s_x[JOIN_WARPS], s_l[JOIN_WARPS];
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const RowPieces p = row_pieces(a, blockIdx.x / a.n_q, blockIdx.x % a.n_q);
    if (p.n < 0) return;
    // the largest m; the pieces' m are kept for the weights
    float M = -INFINITY;
    for (int i = t; i < p.n; i += JOIN_THREADS) {
        const float m = p.at(i)[a.hd];
        if (i < JOIN_W) s_w[i] = m;
        M = fmaxf(M, m);
    }
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
    if (lane == 0) s_x[warp] = M;
    __syncthreads();
    for (int i = 0; i < JOIN_WARPS; ++i) M = fmaxf(M, s_x[i]);
    const float mz = M == -INFINITY ? 0.f : M;
    RowSum r = sum_pieces(p, a.hd, warp, JOIN_WARPS, lane,
                          [&](int i, const float *d) { return exp2f((i < JOIN_W ? s_w[i] : d[a.hd]) - mz); });
    s_o[warp][lane] = r.o[0];
    s_o[warp][lane + 32] = r.o[1];
    if (lane == 0) s_l[warp] = r.l;
    __syncthreads();
    if (warp) return;
    for (int i = 1; i < JOIN_WARPS; ++i) {
        r.l += s_l[i];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float4 x = s_o[i][lane + 32 * h];
            r.o[h].x += x.x;
            r.o[h].y += x.y;
            r.o[h].z += x.z;
            r.o[h].w += x.w;
        }
    }
    put_row<T>(a, blockIdx.x, lane, r, mz);
}

template <typename T> cudaError_t launch_join(const AttnArgs &a, cudaStream_t st)
{
    const int64_t rows = static_cast<int64_t>(a.n_group) * a.share * a.n_q;
    // a block per row while all blocks fit at once (8 per SM): 1056 rows of up to 28 pieces took
    // 7 us less than a warp per row, 2048 rows of 2 to 14 pieces 10 us more
    if (rows <= 8 * 152) return launch_after(true, attn_join_kernel<T>, dim3(static_cast<unsigned>(rows)), dim3(JOIN_THREADS), 0, st, a);
    return launch_after(true, attn_join_rows_kernel<T>, dim3(static_cast<unsigned>((rows + JOIN_WARPS - 1) / JOIN_WARPS)),
                        dim3(JOIN_THREADS), 0, st, a);
}

} // namespace

AttnShape attn_shape(int dtype, int hd, int rows)
{
    return dtype == LOSSK_F32 ? attn_ffma_shape(hd, rows) : attn_mma_shape(hd, rows);
}

bool attn_plans(const AttnArgs &a) { return a.share > 1 || a.n_group > BASE_GROUPS; }

cudaError_t launch_attn_plan(const AttnArgs &a, cudaStream_t st)
{
    if (a.share > 1) {
        attn_share_kernel<<<static_cast<unsigned>(a.n_group), PLAN_T, 0, st>>>(a);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess || a.n_group <= BASE_GROUPS) return e;
    }
    return launch_after(a.share > 1, attn_plan_kernel, dim3(1), dim3(PLAN_T), 0, st, a);
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
