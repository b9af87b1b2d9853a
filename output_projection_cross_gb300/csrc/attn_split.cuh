// attn_split.cuh -- how attention over a paged cache is split into units, items
// and runs (see k_attn.cu), shared by its kernels.
#pragma once
#include "../../include/lossk.h"
#include "decode_internal.h"
#include "decode_launch.h"
#include "ptx.cuh"

namespace lossk {

__device__ __forceinline__ void attn_put4(float *p, float4 v, float f)
{
    *reinterpret_cast<float4 *>(p) = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
}
__device__ __forceinline__ void attn_put4(uint16_t *p, float4 v, float f)
{
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16x2(v.x * f, v.y * f), pack_bf16x2(v.z * f, v.w * f));
}
__device__ __forceinline__ void attn_put4(h16_t *p, float4 v, float f)
{
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_f16x2(v.x * f, v.y * f), pack_f16x2(v.z * f, v.w * f));
}

// A sequence's length as the kernels use it: 0 where it is out of range.
__device__ __forceinline__ int attn_len(const AttnArgs &a, int s)
{
    const int n = a.lens[s];
    return n >= 0 && n <= static_cast<int64_t>(a.max_pages) * a.page ? n : 0;
}

// What of a sequence is read: tokens [lo, hi) with its group (the leading
// `shared` tokens, lo on), then [mid, hi) by itself.
struct Span {
    int lo, mid, hi;
};
__device__ __forceinline__ Span attn_span(const AttnArgs &a, int s, int g)
{
    Span r;
    r.hi = attn_len(a, s);
    r.lo = a.window > 0 && r.hi > a.window ? r.hi - a.window : 0;
    const int shared = a.share > 1 ? a.shared[g] : 0;
    r.mid = shared > r.lo ? shared : r.lo;
    return r;
}
__device__ __forceinline__ int tiles_of(int n, int kt) { return (n + kt - 1) / kt; }

// Starting an item (its query rows, its first tile's latency, its result) takes
// a warp about as long as ITEM_COST tiles; counting it so keeps runs of many
// short items from lagging behind.  An item's units are ITEM_COST for its
// start, then one per tile.  (Counted as 2, 3, 4 and 6: 55, 50, 51 and 51 us for
// 8 x 8 beams on 4096 shared tokens, 137, 133, 134 and 140 for 64 x 8 of 1501.)
constexpr int ITEM_COST = 3;
__device__ __forceinline__ int units_of(int tiles) { return tiles > 0 ? tiles + ITEM_COST : 0; }

// Units of a group's shared part, per item.
__device__ __forceinline__ int shared_tiles(const AttnArgs &a, int g)
{
    if (a.share <= 1) return 0;
    const Span r = attn_span(a, g * a.share, g);
    return tiles_of(r.mid - r.lo, a.kt);
}
__device__ __forceinline__ long long group_units(const AttnArgs &a, int g)
{
    long long u = static_cast<long long>(units_of(shared_tiles(a, g))) * a.n_kv * a.cs;
    for (int i = 0; i < a.share; ++i) {
        const Span r = attn_span(a, g * a.share + i, g);
        u += static_cast<long long>(units_of(tiles_of(r.hi - r.mid, a.kt))) * a.n_kv * a.cp;
    }
    return u;
}

// Groups whose prefix sum a block keeps in shared memory; more take attn_plan.
constexpr int BASE_GROUPS = 1024;
constexpr int BASE_BYTES = 10 * 1024;              // that array and some to spare

// Exclusive prefix sum of the groups' units into out[0 .. n_group], by the whole
// block; s_warp holds one value per warp.
__device__ __forceinline__ void sum_units(const AttnArgs &a, long long *out, long long *s_warp)
{
    const int t = threadIdx.x, lane = t & 31, nt = blockDim.x;
    long long done = 0;
    for (int base = 0; base < a.n_group; base += nt) {
        const int g = base + t;
        const long long x = g < a.n_group ? group_units(a, g) : 0;
        long long inc = x;
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xFFFFFFFFu, inc, o);
            if (lane >= o) inc += y;
        }
        __syncthreads();
        if (lane == 31) s_warp[t >> 5] = inc;
        __syncthreads();
        long long before = 0, all = 0;
        for (int w = 0; w < nt / 32; ++w) {
            if (w < (t >> 5)) before += s_warp[w];
            all += s_warp[w];
        }
        if (g < a.n_group) out[g] = done + before + inc - x;
        done += all;
    }
    if (t == 0) out[a.n_group] = done;
    __syncthreads();
}
// Lengths out of range leave their fault (they count as 0 everywhere).
__device__ __forceinline__ void check_lens(const AttnArgs &a)
{
    for (int s = threadIdx.x; s < a.n_group * a.share; s += blockDim.x)
        if (a.lens[s] < 0 || a.lens[s] > static_cast<int64_t>(a.max_pages) * a.page)
            raise_fault(a.fault, LOSSK_TARGET_OUT_OF_RANGE);
}

// The units before each group, for the split pass: summed by every block for
// itself unless attn_plan already did.
__device__ __forceinline__ const long long *unit_bases(const AttnArgs &a, long long *s_base)
{
    __shared__ long long s_warp[32];
    // what share or plan left is complete after the wait (the join is not let in early: its blocks,
    // resident and waiting, cost the pass 2.5 us)
    wait_for_stream();
    if (a.n_group > BASE_GROUPS) return a.base;
    sum_units(a, s_base, s_warp);
    if (blockIdx.x == 0) check_lens(a);
    return s_base;
}

// a / b, mostly in 32 bits (a 64-bit division is a long routine).
__device__ __forceinline__ int quotient(long long a, int b)
{
    return a <= 0xFFFFFFFFll ? static_cast<int>(static_cast<unsigned>(a) / static_cast<unsigned>(b))
                             : static_cast<int>(a / b);
}

// How the units fall into runs: n runs (no more than there are units), the
// first `more` of q + 1 units, the others of q.
struct Runs {
    int n;
    long long q;
    int more;
    __device__ __forceinline__ Runs(long long units, int most)
    {
        n = units < most ? static_cast<int>(units) : most;
        if (n < 1) n = 1;
        q = units <= 0xFFFFFFFFll ? static_cast<unsigned>(units) / static_cast<unsigned>(n) : units / n;
        more = static_cast<int>(units - q * n);
    }
    __device__ __forceinline__ long long start(int w) const { return q * w + (w < more ? w : more); }
    // the run that has unit u
    __device__ __forceinline__ int of(long long u) const
    {
        const long long big = (q + 1) * more;
        return u < big ? over(u, q + 1) : more + over(u - big, q);
    }
    static __device__ __forceinline__ int over(long long a, long long b)
    {
        return a <= 0xFFFFFFFFll && b <= 0xFFFFFFFFll ? static_cast<int>(static_cast<unsigned>(a) / static_cast<unsigned>(b))
                                                      : static_cast<int>(a / b);
    }
};

// One item's piece as a warp computes it.
struct Piece {
    int first_row;      // its rows are rows first_row.. of sequences from seq on, counted group rows of heads
    int rows;
    int seq;            // the sequence (private) or the group's first one (shared)
    int head;           // KV head
    int t0, t1;         // tokens [t0, t1)
    int64_t slot;       // where a partial result goes; -1: the whole row is here
    float *part;
};

// Items numbered: of a group's shared part, of a sequence.
__device__ __forceinline__ int64_t shared_item(const AttnArgs &a, int g, int head, int c)
{
    return (static_cast<int64_t>(g) * a.n_kv + head) * a.cs + c;
}
__device__ __forceinline__ int64_t own_item(const AttnArgs &a, int s, int head, int c)
{
    return (static_cast<int64_t>(s) * a.n_kv + head) * a.cp + c;
}

// Query row i of a piece: sequence and query head.
__device__ __forceinline__ int row_seq(const AttnArgs &a, const Piece &p, int i)
{
    return p.seq + (p.first_row + i) / a.group;
}
__device__ __forceinline__ int row_head(const AttnArgs &a, const Piece &p, int i)
{
    return p.head * a.group + (p.first_row + i) % a.group;
}

// Walks run w; body(piece) computes each piece.  The run that has an item's first
// tile also notes for the join which runs have the others.
template <typename F>
__device__ __forceinline__ void walk_run(const AttnArgs &a, const long long *base, int w, F &&body)
{
    const long long units = base[a.n_group];
    const Runs runs(units, a.nw);
    if (w >= runs.n || units == 0) return;
    long long u = runs.start(w);
    const long long u1 = runs.start(w + 1);
    int g = 0;
    for (int lo = 0, hi = a.n_group; hi - lo > 1;) {
        const int mid = (lo + hi) >> 1;
        if (base[mid] <= u) lo = mid;
        else hi = mid;
        g = lo;
    }
    while (u < u1) {
        while (base[g + 1] <= u) ++g;
        long long in = u - base[g];
        const int ts = shared_tiles(a, g), us = units_of(ts);
        const long long su = static_cast<long long>(us) * a.n_kv * a.cs;
        Piece p;
        int at, tiles, lo, hi;                      // the run goes on `at` units into the item
        int2 *runs_of;
        if (in < su) {
            const int item = quotient(in, us), c = item % a.cs;
            at = static_cast<int>(in - static_cast<long long>(item) * us);
            tiles = ts;
            p.head = item / a.cs;
            p.seq = g * a.share;
            p.first_row = c * a.mr;
            p.rows = min(a.mr, a.share * a.group - p.first_row);
            const Span r = attn_span(a, p.seq, g);
            lo = r.lo;
            hi = r.mid;
            p.slot = shared_item(a, g, p.head, c);
            runs_of = a.runs_a + p.slot;
            p.slot += w;
            p.part = a.part_a + p.slot * a.ra * (a.hd + ATTN_ROW);
        } else {
            in -= su;
            int s = g * a.share;
            Span r = attn_span(a, s, g);
            tiles = tiles_of(r.hi - r.mid, a.kt);
            for (long long all; in >= (all = static_cast<long long>(units_of(tiles)) * a.n_kv * a.cp);) {
                in -= all;
                r = attn_span(a, ++s, g);
                tiles = tiles_of(r.hi - r.mid, a.kt);
            }
            const int up = units_of(tiles), item = quotient(in, up), c = item % a.cp;
            at = static_cast<int>(in - static_cast<long long>(item) * up);
            p.head = item / a.cp;
            p.seq = s;
            p.first_row = c * a.mr;
            p.rows = min(a.mr, a.group - p.first_row);
            lo = r.mid;
            hi = r.hi;
            p.slot = own_item(a, s, p.head, c);
            runs_of = a.runs_b + p.slot;
            p.slot += w;
            p.part = a.part_b + p.slot * a.rb * (a.hd + ATTN_ROW);
        }
        const int n = static_cast<int>(min(static_cast<long long>(units_of(tiles) - at), u1 - u));
        const int tile0 = max(at - ITEM_COST, 0), tile1 = at + n - ITEM_COST;
        u += n;
        if (tile1 <= 0) continue;                   // the run ends within the item's start
        // (every warp of a ring notes the same)
        if (tile0 == 0 && (threadIdx.x & 31) == 0)
            *runs_of = make_int2(w, tile1 == tiles ? 1 : runs.of(u + (tiles - tile1) - 1) - w + 1);
        if (ts == 0 && tile0 == 0 && tile1 == tiles) p.slot = -1;
        p.t0 = lo + tile0 * a.kt;
        p.t1 = min(hi, lo + tile1 * a.kt);
        body(p);
    }
}

// ---- tiles of keys and values --------------------------------------------------------
__device__ __forceinline__ void cp16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// bytes 0: zeros, src is not read
__device__ __forceinline__ void cp16_or_zero(uint32_t dst, const void *src, int bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }


// The tiles of a piece, copied into a ring of V::STAGES of them in shared memory
// (each V::KT tokens' keys, then their values, rows V::RS bytes apart): start()
// sends for the first tiles, next(i) for tile i + STAGES - 1, once every warp of
// the ring is past tile i - 1.  Each of the ring's V::W warps copies its share
// of the rows and leaves the tile's valid tokens as a mask in valid[stage].
template <typename V> struct TileStream {
    static constexpr int KT = V::KT, STEP = 32 / V::LPR, MINE = KT / STEP / V::W;
    static constexpr int NO_TOKEN = -2;                // beside pages, of which -1 stands for every negative id
    static constexpr uint32_t FULL = KT == 32 ? 0xFFFFFFFFu : (1u << KT) - 1u;
    const AttnArgs &a;
    const Piece &p;
    const int lane, c, first, words;
    const uint32_t ring;
    uint32_t *valid;
    const int32_t *row;
    const char *kb, *vb;
    // lane < KT: this lane's token of the tile to be looked up next, its page's column and its
    // place in the page; the page itself is loaded a tile before it is needed
    int t, col, off, pg, place;
    const int step_col, step_off;       // a tile is that many pages and tokens long

    __device__ __forceinline__ TileStream(const AttnArgs &a_, const Piece &p_, int sub, int lane_, uint32_t ring_,
                                          uint32_t *valid_)
        : a(a_), p(p_), lane(lane_), c(lane_ % V::LPR), first(sub * MINE * STEP + lane_ / V::LPR),
          words(a_.hd * V::ESIZE / 16), ring(ring_), valid(valid_), step_col(KT / a_.page), step_off(KT % a_.page)
    {
        row = a.table + p.seq * a.table_stride;
        kb = static_cast<const char *>(a.k) + p.head * a.head_stride * V::ESIZE + c * 16;
        vb = static_cast<const char *>(a.v) + p.head * a.head_stride * V::ESIZE + c * 16;
        t = p.t0 + lane;
        col = t / a.page;
        off = t % a.page;
        look_up();
    }
    __device__ __forceinline__ void look_up()
    {
        const bool in = lane < KT && t < p.t1;
        pg = in ? max(row[col], -1) : NO_TOKEN;
        place = off;
        t += KT;
        off += step_off;
        col += step_col;
        if (off >= a.page) {
            off -= a.page;
            ++col;
        }
    }
    // Tile i, whose pages are pg_ and places place_.
    __device__ __forceinline__ void fetch(int i, int pg_, int place_)
    {
        const int st = i % V::STAGES;
        const bool ok = pg_ >= 0 && pg_ < a.n_pages;
        if (!ok && pg_ != NO_TOKEN) raise_fault(a.fault, LOSSK_TARGET_OUT_OF_RANGE);
        const int64_t at = ok ? (pg_ * a.page_stride + place_ * a.tok_stride) * V::ESIZE : -1;
        const uint32_t mask = __ballot_sync(0xFFFFFFFFu, ok);
        if (lane == 0) valid[st] = mask;
        const uint32_t kd = ring + st * 2 * V::TILE + first * V::RS + c * 16, vd = kd + V::TILE;
        // a whole tile inside one page: its rows are tok_stride apart
        if (mask == FULL && __shfl_sync(0xFFFFFFFFu, place_, 0) + KT <= a.page) {
            const int64_t step = a.tok_stride * V::ESIZE;
            const int64_t o = __shfl_sync(0xFFFFFFFFu, at, 0) + first * step;
#pragma unroll
            for (int x = 0; x < V::CPL; ++x)
                if (c + x * V::LPR < words) {
                    const char *ks = kb + o + x * V::LPR * 16, *vs = vb + o + x * V::LPR * 16;
#pragma unroll
                    for (int j = 0; j < MINE; ++j) {
                        cp16(kd + j * STEP * V::RS + x * V::LPR * 16, ks);
                        cp16(vd + j * STEP * V::RS + x * V::LPR * 16, vs);
                        ks += STEP * step;
                        vs += STEP * step;
                    }
                }
            return;
        }
#pragma unroll
        for (int j = 0; j < MINE; ++j) {
            const int64_t o = __shfl_sync(0xFFFFFFFFu, at, j * STEP + first);
            const int bytes = o >= 0 ? 16 : 0;
#pragma unroll
            for (int x = 0; x < V::CPL; ++x)
                if (c + x * V::LPR < words) {
                    cp16_or_zero(kd + j * STEP * V::RS + x * V::LPR * 16, kb + (o >= 0 ? o : 0) + x * V::LPR * 16, bytes);
                    cp16_or_zero(vd + j * STEP * V::RS + x * V::LPR * 16, vb + (o >= 0 ? o : 0) + x * V::LPR * 16, bytes);
                }
        }
    }
    __device__ __forceinline__ void send(int i, int n_tiles)
    {
        const int pg_ = pg, place_ = place;
        look_up();
        if (i < n_tiles) fetch(i, pg_, place_);
        cp_commit();
    }
    __device__ __forceinline__ void start(int n_tiles)
    {
#pragma unroll
        for (int i = 0; i < V::STAGES - 1; ++i) send(i, n_tiles);
    }
    __device__ __forceinline__ void next(int i, int n_tiles) { send(i + V::STAGES - 1, n_tiles); }
};

} // namespace lossk
