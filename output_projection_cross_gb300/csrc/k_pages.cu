// k_pages.cu -- the page side of a paged key-value cache: forking sequences,
// reserving places for new tokens, freeing, compacting and copying pages,
// writing tokens' rows.
//
//   cache_fork    table rows by parent; reference counts
//   cache_plan    (reserve) which sequences need a page, which get a copy of
//                 a shared one, and the free pages for them
//   cache_copy    the pages of a list, in every plane of the pool
//   cache_free    drops sequences
//   cache_rank    (compact) a pool's live pages counted and ranked
//   cache_write   key and value rows of new tokens into their pages
//
// A page is free while its reference count is 0: the lowest free pages are
// found by scanning the counts (4 bytes a page, read once), which keeps no
// list that could disagree with the counts and makes every allocation a
// function of the inputs alone.
//
// Copies and moves are bound by HBM (compaction of 8192 pages, 515 MB read and
// written: 87 us in all; cache_move alone 77 us = 6.7 TB/s), everything else by
// the latency of its few dependent loads and scans: a fork or a write 2 to 5 us,
// the plan of a reservation 6 us for 4 sequences and 160 pages, 10 us for 512
// sequences and 13312 pages.  Plan and copies are two launches: one launch whose
// blocks wait for the first one's plan made that decoding step (fork,
// reservation and writes for 512 sequences) 38 us instead of 30, a compaction of
// 331 pages 15 instead of 8.
#include "../../include/lossk.h"
#include "decode_internal.h"
#include "decode_launch.h"
#include "ptx.cuh"

namespace lossk {

namespace {

__device__ __forceinline__ bool page_ok(int p, int n_pages) { return p >= 0 && p < n_pages; }

// A length of the table's: 0 and a fault where it is out of range.
__device__ __forceinline__ int len_checked(int len, int max_pages, int page, int *fault)
{
    if (len >= 0 && len <= static_cast<int64_t>(max_pages) * page) return len;
    raise_fault(fault, LOSSK_TARGET_OUT_OF_RANGE);
    return 0;
}
__device__ __forceinline__ int pages_of(int len, int page) { return len / page + (len % page != 0); }

// ---- fork ----------------------------------------------------------------------
// The first n_dst blocks write a row each; the others each take one source row
// and add (children - 1) to the counts of its pages, children being how many
// rows of the group took it: the row itself goes, each child holds it once.
__global__ void __launch_bounds__(128) cache_fork_kernel(ForkArgs a)
{
    __shared__ int s_n;
    const int t = threadIdx.x, b = blockIdx.x;
    const int rows_dst = a.n_group * a.n_dst;
    wait_for_stream();
    if (b < rows_dst) {
        const int g = b / a.n_dst, p = a.parent[b];
        const bool ok = p >= 0 && p < a.n_src;
        if (!ok && p != -1 && t == 0) raise_fault(a.fault, LOSSK_TARGET_OUT_OF_RANGE);
        const int s = g * a.n_src + (ok ? p : 0);
        const int len = ok ? len_checked(a.lens[s], a.max_pages, a.page, a.fault) : 0;
        const int used = pages_of(len, a.page);
        const int32_t *from = a.table + s * a.table_stride;
        int32_t *to = a.table_out + b * a.table_out_stride;
        for (int c = t; c < a.max_pages; c += 128) {
            int v = -1;
            if (c < used) {
                v = from[c];
                if (!page_ok(v, a.n_pages)) {
                    raise_fault(a.fault, LOSSK_TARGET_OUT_OF_RANGE);
                    v = -1;
                }
            }
            to[c] = v;
        }
        if (t == 0) a.lens_out[b] = len;
        return;
    }
    const int s = b - rows_dst, g = s / a.n_src, me = s % a.n_src;
    if (t == 0) s_n = 0;
    __syncthreads();
    int n = 0;
    for (int j = t; j < a.n_dst; j += 128) n += a.parent[g * a.n_dst + j] == me;
    if (n) atomicAdd(&s_n, n);
    __syncthreads();
    const int delta = s_n - 1;
    if (delta == 0) return;
    const int used = pages_of(len_checked(a.lens[s], a.max_pages, a.page, a.fault), a.page);
    for (int c = t; c < used; c += 128) {
        const int p = a.table[s * a.table_stride + c];
        if (page_ok(p, a.n_pages)) atomicAdd(a.ref + p, delta);
        else raise_fault(a.fault, LOSSK_TARGET_OUT_OF_RANGE);
    }
}

// ---- reserve ---------------------------------------------------------------------
constexpr int PLAN_THREADS = 1024;

// Exclusive sum over the block of x; *total its sum.  All threads call it.
template <typename I> __device__ __forceinline__ I block_scan(I x, I *s_warp, I *total)
{
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    I inc = x;
    for (int o = 1; o < 32; o <<= 1) {
        const I y = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += y;
    }
    __syncthreads();
    if (lane == 31) s_warp[w] = inc;
    __syncthreads();
    if (w == 0) {
        I v = s_warp[lane];
        for (int o = 1; o < 32; o <<= 1) {
            const I y = __shfl_up_sync(0xFFFFFFFFu, v, o);
            if (lane >= o) v += y;
        }
        s_warp[lane] = v;
    }
    __syncthreads();
    *total = s_warp[31];
    return inc - x + (w ? s_warp[w - 1] : 0);
}

// Eight counts from ref[p0] on (of pages past the last one: `past`).
constexpr int PER = 8;
__device__ __forceinline__ void load_counts(const int32_t *ref, int p0, int n_pages, int past, int (&r)[PER])
{
    if (p0 + PER <= n_pages && (reinterpret_cast<uintptr_t>(ref + p0) & 15) == 0) {
        const int4 x = *reinterpret_cast<const int4 *>(ref + p0), y = *reinterpret_cast<const int4 *>(ref + p0 + 4);
        r[0] = x.x; r[1] = x.y; r[2] = x.z; r[3] = x.w;
        r[4] = y.x; r[5] = y.y; r[6] = y.z; r[7] = y.w;
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) r[i] = p0 + i < n_pages ? ref[p0 + i] : past;
    }
}

// One slot of the sharers' table: how many sequences of the call have this
// page as their partial last one, and the highest of them.
__device__ __forceinline__ int sharer_slot(SharerSlot *h, int mask, int page)
{
    unsigned i = static_cast<unsigned>(page) * 2654435761u & mask;
    while (true) {
        const int was = atomicCAS(&h[i].page, -1, page);
        if (was == -1 || was == page) return static_cast<int>(i);
        i = (i + 1) & mask;
    }
}

// One block.  For each sequence with n > 0 new tokens: a copy of its last
// page where that is partial and shared, and a page for each that the tokens
// open.  Among the sharers of a page the lower ones get copies; the highest
// keeps the page itself when no other row holds it.  Pages are given in
// sequence order, the lowest free ones first.  Nothing is changed unless every
// sequence can be served: a bad id or length leaves 586, too few free pages
// or too short a table 584.
__global__ void __launch_bounds__(PLAN_THREADS) cache_plan_kernel(ReserveArgs a)
{
    __shared__ int s_warp[32];
    __shared__ long long s_long[32];
    __shared__ int s_status;
    const int t = threadIdx.x;
    wait_for_stream();
    if (t == 0) {
        s_status = 0;
        *a.n_copy = 0;
    }
    for (int i = t; i <= a.hash_mask; i += PLAN_THREADS) a.hash[i] = SharerSlot{-1, 0, -1};
    __syncthreads();
    // what each sequence asks for, and who shares its last page
    for (int i = t; i < a.n_seq; i += PLAN_THREADS) {
        const int n = a.n_new ? a.n_new[i] : a.n_new_all, len = a.lens[i];
        if (n == 0) continue;
        if (n < 0 || len < 0 || len > static_cast<int64_t>(a.max_pages) * a.page) {
            atomicMax(&s_status, LOSSK_TARGET_OUT_OF_RANGE);
            continue;
        }
        if (static_cast<int64_t>(len) + n > static_cast<int64_t>(a.max_pages) * a.page) {
            atomicMax(&s_status, LOSSK_WORK_BUDGET_EXCEEDED);
            continue;
        }
        if (len % a.page == 0) continue;
        const int p = a.table[i * a.table_stride + len / a.page];
        if (!page_ok(p, a.n_pages)) {
            atomicMax(&s_status, LOSSK_TARGET_OUT_OF_RANGE);
            continue;
        }
        const int h = sharer_slot(a.hash, a.hash_mask, p);
        atomicAdd(&a.hash[h].count, 1);
        atomicMax(&a.hash[h].top, i);
    }
    __syncthreads();
    if (s_status) {
        if (t == 0) raise_fault(a.fault, s_status);
        return;
    }
    // each sequence's place among the pages given out: need[i] = (first page, pages, copy)
    // (64-bit sums: sequences may ask for more pages than an int counts)
    int given = 0, n_copy = 0;
    for (int base = 0; base < a.n_seq; base += PLAN_THREADS) {
        const int i = base + t;
        int pages = 0, copy = 0;
        if (i < a.n_seq) {
            const int n = a.n_new ? a.n_new[i] : a.n_new_all, len = a.lens[i];
            if (n > 0) {
                pages = pages_of(len + n, a.page) - pages_of(len, a.page);
                if (len % a.page) {
                    const int p = a.table[i * a.table_stride + len / a.page];
                    const SharerSlot h = a.hash[sharer_slot(a.hash, a.hash_mask, p)];
                    copy = !(a.ref[p] <= h.count && h.top == i);
                }
            }
        }
        long long sum;
        const long long first = block_scan(static_cast<long long>(pages) + copy, s_long, &sum);
        if (given + sum > a.n_pages) {
            if (t == 0) raise_fault(a.fault, LOSSK_WORK_BUDGET_EXCEEDED);
            return;
        }
        if (i < a.n_seq) a.need[i] = make_int4(given + static_cast<int>(first), pages, copy, 0);
        given += static_cast<int>(sum);
    }
    __syncthreads();
    // the lowest `given` free pages
    int found = 0;
    for (int base = 0; base < a.n_pages && found < given; base += PLAN_THREADS * PER) {
        int r[PER], free = 0, sum;
        const int p0 = base + t * PER;
        load_counts(a.ref, p0, a.n_pages, 1, r);
#pragma unroll
        for (int i = 0; i < PER; ++i) free += r[i] == 0;
        int at = found + block_scan(free, s_warp, &sum);
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (r[i] == 0 && at < given) a.free_list[at++] = p0 + i;
        found += sum;
    }
    if (found < given) {
        if (t == 0) raise_fault(a.fault, LOSSK_WORK_BUDGET_EXCEEDED);
        return;
    }
    __syncthreads();
    for (int base = 0; base < a.n_seq; base += PLAN_THREADS) {
        const int i = base + t;
        int copy = 0, pages = 0, first = 0;
        if (i < a.n_seq) {
            const int4 nd = a.need[i];
            first = nd.x;
            pages = nd.y;
            copy = nd.z;
        }
        int sum;
        const int at = n_copy + block_scan(copy, s_warp, &sum);
        n_copy += sum;
        if (copy + pages) {
            int32_t *row = a.table + i * a.table_stride;
            const int len = a.lens[i];
            if (copy) {
                const int p = row[len / a.page], q = a.free_list[first];
                a.moves[at] = make_int2(p, q);
                atomicSub(a.ref + p, 1);
                a.ref[q] = 1;
                row[len / a.page] = q;
            }
            const int c0 = pages_of(len, a.page);
            for (int j = 0; j < pages; ++j) {
                const int q = a.free_list[first + copy + j];
                a.ref[q] = 1;
                row[c0 + j] = q;
            }
        }
    }
    if (t == 0) *a.n_copy = n_copy;
}

// ---- copying pages ----------------------------------------------------------------
// moves[i] = (from, to), n of them (*n_dev where the count is the device's).  A
// block takes pieces of a page; a piece is 256 threads x 4 loads of 16 bytes
// (four blocks of it in flight on an SM are the 64 KB that HBM's latency asks for).
constexpr int COPY_THREADS = 256;
constexpr int COPY_U = 4;

template <typename V>
__device__ __forceinline__ void copy_piece(const V *s, V *d, int64_t at, int64_t words)
{
    V v[COPY_U];
#pragma unroll
    for (int u = 0; u < COPY_U; ++u) {
        const int64_t i = at + u * COPY_THREADS + threadIdx.x;
        if (i < words) v[u] = s[i];
    }
#pragma unroll
    for (int u = 0; u < COPY_U; ++u) {
        const int64_t i = at + u * COPY_THREADS + threadIdx.x;
        if (i < words) d[i] = v[u];
    }
}

__device__ __forceinline__ void copy_moves(const CopyArgs &a, int64_t n, int block, int blocks)
{
    const int64_t words = a.page_bytes >> 4;
    const int64_t pieces = (words + COPY_THREADS * COPY_U - 1) / (COPY_THREADS * COPY_U);
    const int64_t total = n * a.n_planes * pieces;
    for (int64_t w = block; w < total; w += blocks) {
        const int64_t piece = w % pieces, plane = w / pieces % a.n_planes, i = w / pieces / a.n_planes;
        int2 m;
        if (a.moves) m = a.moves[i];
        else m = make_int2(a.src[i], a.dst[i]);
        if (!page_ok(m.x, a.n_pages) || !page_ok(m.y, a.n_pages)) {
            if (threadIdx.x == 0 && !(m.x == -1 && m.y == -1)) raise_fault(a.fault, LOSSK_TARGET_OUT_OF_RANGE);
            continue;
        }
        if (m.x == m.y) continue;
        char *base = a.pool + plane * a.plane_stride;
        copy_piece(reinterpret_cast<const uint4 *>(base + m.x * a.page_stride),
                   reinterpret_cast<uint4 *>(base + m.y * a.page_stride), piece * COPY_THREADS * COPY_U, words);
    }
}

__global__ void __launch_bounds__(COPY_THREADS) cache_copy_kernel(CopyArgs a)
{
    wait_for_stream();
    copy_moves(a, a.n_dev ? *a.n_dev : a.n, blockIdx.x, gridDim.x);
}

// ---- free -------------------------------------------------------------------------
__global__ void __launch_bounds__(128) cache_free_kernel(FreeArgs a)
{
    const int i = blockIdx.x, t = threadIdx.x;
    wait_for_stream();
    if (a.drop && !a.drop[i]) return;
    int32_t *row = a.table + i * a.table_stride;
    const int used = pages_of(len_checked(a.lens[i], a.max_pages, a.page, a.fault), a.page);
    for (int c = t; c < a.max_pages; c += 128) {
        if (c < used) {
            const int p = row[c];
            if (page_ok(p, a.n_pages)) atomicSub(a.ref + p, 1);
            else raise_fault(a.fault, LOSSK_TARGET_OUT_OF_RANGE);
        }
        row[c] = -1;
    }
    __syncthreads();
    if (t == 0) a.lens[i] = 0;
}

// ---- compact ------------------------------------------------------------------------
// With n_live pages live in all, the k-th live page at or above n_live moves
// to the k-th free page below it: the fewest moves that leave the live pages in
// front.  cache_rank (one block) lists both sides in order and notes each
// mover's new id; cache_move copies the pages, renames the table's entries
// and writes the new counts.
__global__ void __launch_bounds__(PLAN_THREADS) cache_rank_kernel(CompactArgs a)
{
    __shared__ int s_warp[32];
    __shared__ long long s_long[32];
    const int t = threadIdx.x;
    wait_for_stream();
    int live = 0, n_live;
    for (int base = 0; base < a.n_pages; base += PLAN_THREADS * PER) {
        int r[PER];
        load_counts(a.ref, base + t * PER, a.n_pages, 0, r);
#pragma unroll
        for (int i = 0; i < PER; ++i) live += r[i] > 0;
    }
    block_scan(live, s_warp, &n_live);
    // (both sums at once: holes in the low half, movers in the high one)
    long long done = 0;
    for (int base = 0; base < a.n_pages; base += PLAN_THREADS * PER) {
        int r[PER];
        const int p0 = base + t * PER;
        load_counts(a.ref, p0, a.n_pages, 0, r);
        long long mine = 0, sum;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            mine += r[i] > 0 ? (p0 + i >= n_live ? 1ll << 32 : 0) : p0 + i < n_live ? 1 : 0;
        const long long at = done + block_scan(mine, s_long, &sum);
        int h = static_cast<int>(at & 0xFFFFFFFF), m = static_cast<int>(at >> 32);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (r[i] > 0) {
                if (p0 + i >= n_live) a.moves[m++].x = p0 + i;
            } else if (p0 + i < n_live) {
                a.moves[h++].y = p0 + i;
            }
        }
        done += sum;
    }
    const int movers = static_cast<int>(done >> 32);
    __syncthreads();
    for (int k = t; k < movers; k += PLAN_THREADS) a.new_id[a.moves[k].x] = a.moves[k].y;
    if (t == 0) {
        *a.n_copy = movers;
        *a.n_live_out = n_live;
    }
}

__global__ void __launch_bounds__(COPY_THREADS) cache_move_kernel(CompactArgs a, CopyArgs c)
{
    wait_for_stream();
    const int n_live = *a.n_live_out, n = *a.n_copy;
    const int64_t gt = static_cast<int64_t>(blockIdx.x) * COPY_THREADS + threadIdx.x;
    const int64_t all = static_cast<int64_t>(gridDim.x) * COPY_THREADS;
    // a hole's count comes from its mover, which cache_rank listed beside it
    for (int64_t p = gt; p < a.n_pages; p += all) {
        const int r = a.ref[p];
        if (p >= n_live) a.ref_out[p] = 0;
        else if (r > 0) a.ref_out[p] = r;
    }
    for (int64_t k = gt; k < n; k += all) a.ref_out[a.moves[k].y] = a.ref[a.moves[k].x];
    for (int64_t e = gt; e < static_cast<int64_t>(a.n_seq) * a.max_pages; e += all) {
        const int i = static_cast<int>(e / a.max_pages), col = static_cast<int>(e % a.max_pages);
        const int used = pages_of(len_checked(a.lens[i], a.max_pages, a.page, a.fault), a.page);
        int v = -1;
        if (col < used) {
            v = a.table[i * a.table_stride + col];
            if (!page_ok(v, a.n_pages) || a.ref[v] <= 0) {
                raise_fault(a.fault, LOSSK_TARGET_OUT_OF_RANGE);
                v = -1;
            } else if (v >= n_live) {
                v = a.new_id[v];
            }
        }
        a.table_out[i * a.table_out_stride + col] = v;
    }
    copy_moves(c, n, blockIdx.x, gridDim.x);
}

// ---- writing rows -----------------------------------------------------------------
// One warp per (token, key or value).  V is the widest word that the rows'
// sizes, strides and addresses allow.
template <typename V>
__global__ void __launch_bounds__(128) cache_write_kernel(WriteArgs a)
{
    const int64_t w = (static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    const int64_t tok = w >> 1;
    wait_for_stream();
    if (tok >= a.n_tok) return;
    int seq = static_cast<int>(tok), off = 0;
    if (a.first) {
        // the sequence whose rows [first[i], first[i + 1]) hold tok
        int lo = 0, hi = a.n_seq;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (a.first[mid] <= tok) lo = mid;
            else hi = mid;
        }
        seq = lo;
        if (tok < a.first[lo] || tok >= a.first[lo + 1]) return;   // a row of no sequence
        off = static_cast<int>(tok - a.first[lo]);
    }
    const int64_t pos = static_cast<int64_t>(a.lens[seq]) + off;
    const int64_t col = pos / a.page;
    int p = -1;
    if (a.lens[seq] >= 0 && col < a.max_pages) p = a.table[seq * a.table_stride + col];
    if (!page_ok(p, a.n_pages)) {
        if (lane == 0) raise_fault(a.fault, LOSSK_TARGET_OUT_OF_RANGE);
        return;
    }
    const bool is_v = w & 1;
    const char *src = (is_v ? a.v_new : a.k_new) + tok * (is_v ? a.v_row : a.k_row);
    char *dst = (is_v ? a.v : a.k) + p * (is_v ? a.v_page : a.k_page) + (pos % a.page) * (is_v ? a.v_tok : a.k_tok);
    const int64_t head = is_v ? a.v_head : a.k_head;
    const int words = a.row_bytes / static_cast<int>(sizeof(V));
    for (int i = lane; i < a.n_kv * words; i += 32) {
        const int h = i / words, c = i % words;
        *reinterpret_cast<V *>(dst + h * head + c * static_cast<int>(sizeof(V))) =
            *reinterpret_cast<const V *>(src + (static_cast<int64_t>(h) * words + c) * static_cast<int>(sizeof(V)));
    }
}

int copy_blocks(int64_t most)
{
    const int64_t b = most < 152 * 8 ? most : 152 * 8;
    return static_cast<int>(b < 1 ? 1 : b);
}
int64_t pieces_of(const CopyArgs &c)
{
    return (c.page_bytes / 16 + COPY_THREADS * COPY_U - 1) / (COPY_THREADS * COPY_U) * c.n_planes;
}

} // namespace

cudaError_t launch_cache_fork(const ForkArgs &a, cudaStream_t st)
{
    return launch(cache_fork_kernel, dim3(static_cast<unsigned>(a.n_group) * (a.n_dst + a.n_src)), dim3(128), 0, st, a);
}
cudaError_t launch_cache_plan(const ReserveArgs &a, cudaStream_t st)
{
    return launch(cache_plan_kernel, dim3(1), dim3(PLAN_THREADS), 0, st, a);
}
cudaError_t launch_cache_copy(const CopyArgs &a, int64_t most, cudaStream_t st)
{
    return launch(cache_copy_kernel, dim3(copy_blocks(most * pieces_of(a))), dim3(COPY_THREADS), 0, st, a);
}
cudaError_t launch_cache_free(const FreeArgs &a, cudaStream_t st)
{
    return launch(cache_free_kernel, dim3(static_cast<unsigned>(a.n_seq)), dim3(128), 0, st, a);
}
cudaError_t launch_cache_rank(const CompactArgs &a, cudaStream_t st)
{
    return launch(cache_rank_kernel, dim3(1), dim3(PLAN_THREADS), 0, st, a);
}
cudaError_t launch_cache_move(const CompactArgs &a, const CopyArgs &c, cudaStream_t st)
{
    return launch(cache_move_kernel, dim3(copy_blocks((a.n_pages / 2 + 1) * pieces_of(c))), dim3(COPY_THREADS), 0, st, a, c);
}
cudaError_t launch_cache_write(const WriteArgs &a, int word, cudaStream_t st)
{
    const unsigned grid = static_cast<unsigned>((a.n_tok * 2 + 3) / 4);
    return launch(word == 16 ? cache_write_kernel<uint4> : word == 4 ? cache_write_kernel<uint32_t> : cache_write_kernel<uint16_t>,
                  dim3(grid), dim3(128), 0, st, a);
}

} // namespace lossk
