// k_beam.cu -- beam search's selection over beams and vocabulary, and the
// reordering of states by parent.
//
//   beam_rows    per (row, split of the vocabulary): the statistics of the
//                log-sum-exp and the split's n_out best logits
//   beam_merge   per batch entry: log-sum-exps, scores, ranks, the n_out best
//   beam_gather  rows of a state by parent
//
// Within a row the candidates' order is the logits' (the log-sum-exp and the
// beam's score are constants of the row), so the rows kernel never needs a
// score; only the few survivors get one, in double, because candidates of
// different beams may lie closer together than floats resolve.
//
// A row is read once: 65 us for 128 x 8 beams over 151936 tokens (272 MB of
// live rows, 4.2 TB/s over both kernels), 18 us for 16 x 4, 11 us for one entry
// of 4 beams over 32000 tokens, which is two launches and their chains of
// dependent steps (rows 7 us, merge 4).
#include "../../include/lossk.h"
#include "decode_internal.h"
#include "decode_launch.h"
#include "float2.cuh"
#include "ptx.cuh"

#include <type_traits>

namespace lossk {

namespace {

constexpr int NT = 256;                    // threads of a block, here throughout
constexpr int WARPS = NT / 32;

// A barrier of those threads (the rows kernel has a loading warp beside them).
__device__ __forceinline__ void block_sync() { named_bar_sync(1, NT); }

// ---- the n best of many -----------------------------------------------------------
// A block streams keys past a threshold into a buffer in shared memory.  The
// threshold comes from the first chunk: cut the block into groups of threads;
// the n-th largest of the groups' largest keys has n keys at or above it, so
// nothing below it can be among the n best.  Keys are unique, so at most n
// groups hold keys that pass.  When the buffer fills up, it is cut back to its
// n best and the threshold raised to the last of them.
//
// A key orders by logit, then by falling token.  0 stands for none.
using Key = uint64_t;

__device__ __forceinline__ uint32_t order_of(float x)
{
    const uint32_t b = __float_as_uint(x);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o)
{
    return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}
__device__ __forceinline__ Key key_of(float x, int tok)
{
    return (static_cast<uint64_t>(order_of(x)) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(tok));
}

__device__ __forceinline__ uint64_t order_of(double x)
{
    const uint64_t b = __double_as_longlong(x + 0.0);
    return b >> 63 ? ~b : b | (1ull << 63);
}

// Groups of threads a threshold is taken over: at least 4 n of them where
// there are that many threads (fewer keys to rank; with 4 n groups about n / 7
// keys more than n pass).
__host__ __device__ constexpr int groups_for(int n) { return n <= 16 ? 64 : n <= 32 ? 128 : 256; }

// The n-th largest of the groups' largest keys (none where fewer groups have
// any).  All threads call it with their largest key; s_keys holds NT keys.
__device__ __forceinline__ Key nth_of_groups(Key mine, int n, Key *s_keys, Key *s_nth)
{
    const int t = threadIdx.x, groups = groups_for(n), per = NT / groups;
    for (int o = 1; o < per; o <<= 1) {
        const Key other = __shfl_xor_sync(0xFFFFFFFFu, mine, o);
        if (other > mine) mine = other;
    }
    block_sync();
    if (t == 0) *s_nth = 0;
    if (t % per == 0) s_keys[t / per] = mine;
    block_sync();
    // `per` threads count the keys above each group's, a part each
    mine = s_keys[t / per];
    int above = 0;
    const int part = groups / per, first = (t % per) * part;
#pragma unroll 8
    for (int i = 0; i < part; ++i) above += s_keys[first + i] > mine;
    for (int o = 1; o < per; o <<= 1) above += __shfl_xor_sync(0xFFFFFFFFu, above, o);
    if (t % per == 0 && above == n - 1 && mine) *s_nth = mine;
    block_sync();
    return *s_nth;
}

// The n best of buf[0 .. cnt), in falling order, into buf[0 ..); returns how
// many there are.  tmp holds as many keys as buf.
__device__ __forceinline__ int keep_best(Key *buf, Key *tmp, int cnt, int n, Key *s_keys, Key *s_nth, int *s_cnt)
{
    const int t = threadIdx.x;
    Key mine = 0;
    for (int i = t; i < cnt; i += NT)
        if (buf[i] > mine) mine = buf[i];
    const Key nth = nth_of_groups(mine, n, s_keys, s_nth);
    if (t == 0) *s_cnt = 0;
    block_sync();
    for (int i = t; i < cnt; i += NT)
        if (buf[i] && buf[i] >= nth) tmp[atomicAdd(s_cnt, 1)] = buf[i];
    block_sync();
    const int left = *s_cnt;
    for (int i = t; i < left; i += NT) {
        const Key k = tmp[i];
        int above = 0;
#pragma unroll 4
        for (int j = 0; j < left; ++j) above += tmp[j] > k;
        if (above < n) buf[above] = k;
    }
    block_sync();
    return left < n ? left : n;
}

// ---- rows --------------------------------------------------------------------------
template <typename T> struct Elem;
template <> struct Elem<float> {
    static constexpr int NV = 4;
};
template <> struct Elem<uint16_t> {
    static constexpr int NV = 8;
};
template <> struct Elem<h16_t> {
    static constexpr int NV = 8;
};
constexpr int U = 4;                       // 16-byte vectors a thread holds of a chunk
constexpr int CHUNK = NT * U;
constexpr int STAGES = 3, STAGE_BYTES = (CHUNK + 1) * 16;
constexpr int STEADY = 32;

__device__ __forceinline__ float beam_f(float x) { return x + 0.f; }   // -0 to +0: they tie
__device__ __forceinline__ float beam_f(uint16_t x) { return __uint_as_float(static_cast<uint32_t>(x) << 16) + 0.f; }
__device__ __forceinline__ float beam_f(h16_t x) { return f16_to_f(x.bits) + 0.f; }

template <typename T> __device__ __forceinline__ void unpack(const uint4 &v, float *f)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(w[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = h16_lo<std::is_same<T, h16_t>::value>(w[i]);
            f[2 * i + 1] = h16_hi<std::is_same<T, h16_t>::value>(w[i]);
        }
    }
}

// max that a NaN goes through
__device__ __forceinline__ float max_nan(float x, float y)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}
template <typename T> __device__ __forceinline__ uint32_t max_nan2(uint32_t x, uint32_t y)
{
    uint32_t r;
    if constexpr (std::is_same<T, h16_t>::value) asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
    else asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
    return r;
}
// The largest of a vector (of 16-bit types two at a time, before they are unpacked).
template <typename T> __device__ __forceinline__ float vec_max(const uint4 &v)
{
    if constexpr (sizeof(T) == 4) {
        return max_nan(max_nan(__uint_as_float(v.x), __uint_as_float(v.y)),
                       max_nan(__uint_as_float(v.z), __uint_as_float(v.w)));
    } else {
        constexpr bool F16 = std::is_same<T, h16_t>::value;
        const uint32_t x = max_nan2<T>(max_nan2<T>(v.x, v.y), max_nan2<T>(v.z, v.w));
        return max_nan(h16_lo<F16>(x), h16_hi<F16>(x));
    }
}

// A thread's running sum of 2^(c x + b), c = log2(e) / T.  b follows the
// largest logit only once that is FAR above it (in log2 units), so a warp
// seldom rescales.  The sum's true base is what b says, rounded or not: it is
// taken off again in double.  Below 2^30 the rounding moves the exponents by 32
// at most, which the sum's range has room for (2^(32 + FAR) a logit).  From
// LARGE on it could take the sum to infinity or 0; there a float next to ref is
// 64 or more off in the exponent, so only logits equal to ref count.  z is two
// floats, sum and what its roundings lost.
struct RowStat {
    float m, ref, b, z, lost;
};
constexpr float FAR = 24.f, LARGE = 0x1p30f;

__device__ __forceinline__ bool plain(float b) { return fabsf(b) < LARGE; }
// 2^(the base of a sum (ref, b) - the base `top` of one at least as high)
__device__ __forceinline__ float to_base(float ref, float b, float top_ref, float top_b)
{
    return plain(top_b) ? (plain(b) ? ex2_approx(top_b - b) : 0.f) : ref == top_ref ? 1.f : 0.f;
}
__device__ __forceinline__ void rebase(RowStat &r, float lm, float c)
{
    const float b = -lm * c;
    if (r.ref > -INFINITY) {
        const float g = to_base(r.ref, r.b, lm, b);
        r.z *= g;
        r.lost *= g;
    }
    r.ref = lm;
    r.b = b;
}
// (z, lost) += (x, rest)
__device__ __forceinline__ void add_z(float &z, float &lost, float x, float rest)
{
    const float s = z + x, y = s - z;
    lost += (z - (s - y)) + (x - y) + rest;
    z = s;
}
__device__ __forceinline__ bool far_above(const RowStat &r, float lm, float c)
{
    return !((lm - r.ref) * c < FAR);          // (a NaN is, too)
}

// A vector of -infinity.
template <typename T> __device__ __forceinline__ uint4 all_low()
{
    const uint32_t w = sizeof(T) == 4 ? 0xFF800000u : std::is_same<T, h16_t>::value ? 0xFC00FC00u : 0xFF80FF80u;
    return make_uint4(w, w, w, w);
}

// A vector with -infinity where its token's bit is 0.
template <typename T> __device__ __forceinline__ uint4 masked(const uint4 &v, uint32_t bits)
{
    const uint4 low = all_low<T>();
    auto word = [&](uint32_t w, int i) {
        uint32_t keep;
        if constexpr (sizeof(T) == 4) {
            keep = (bits >> i) & 1u ? 0xFFFFFFFFu : 0u;
        } else {
            const uint32_t x = (bits >> (2 * i)) & 3u;
            keep = ((x | (x << 15)) & 0x10001u) * 0xFFFFu;
        }
        return (w & keep) | (low.x & ~keep);
    };
    return make_uint4(word(v.x, 0), word(v.y, 1), word(v.z, 2), word(v.w, 3));
}

// 32 bits of a row's mask from token v on.
__device__ __forceinline__ uint32_t allow_bits(const uint32_t *allow, int words, int v)
{
    const int w = v >> 5;
    const uint32_t lo = __ldg(allow + w), hi = w + 1 < words ? __ldg(allow + w + 1) : 0u;
    return __funnelshift_r(lo, hi, v & 31);
}

// Whether beam k of entry b has logits to read: not finished, a finite score.
__device__ __forceinline__ bool beam_reads(const BeamArgs &a, int r)
{
    return !(a.finished && a.finished[r]) && isfinite(a.scores[r]);
}

// Bytes [skew, skew + 16) of two vectors.
__device__ __forceinline__ uint4 joined(uint4 x, uint4 y, int skew)
{
    if (skew & 8) {
        x = make_uint4(x.z, x.w, y.x, y.y);
        y.x = y.z;
        y.y = y.w;
    }
    if (skew & 4) {
        x = make_uint4(x.y, x.z, x.w, y.x);
        y.x = y.y;
    }
    const int bits = (skew & 3) * 8;
    return make_uint4(__funnelshift_r(x.x, x.y, bits), __funnelshift_r(x.y, x.z, bits),
                      __funnelshift_r(x.z, x.w, bits), __funnelshift_r(x.w, y.x, bits));
}

// ---- a row's items ------------------------------------------------------------------
// An item is a split of a row.  Vectors are cut from the split's start on
// whatever the row's alignment, so that equal rows have equal sums and tie; a
// vector of a row that is off by `skew` bytes is put together from two aligned
// ones.  The last NV to 2 NV - 1 tokens go one by one, so that the second of
// those always ends inside the row.
template <typename T> struct Item {
    static constexpr int NV = Elem<T>::NV;
    int r, v0, v1, n_vec, tail, skew;
    const T *row;
    const char *from;                      // the first aligned vector
    __device__ __forceinline__ Item(const BeamArgs &a, int item)
    {
        r = item / a.n_split;
        const int split = item % a.n_split;
        row = static_cast<const T *>(a.logits) + r * a.row_stride;
        v0 = min(split * a.split_len, a.vocab);
        v1 = min(v0 + a.split_len, a.vocab);
        n_vec = max((v1 - v0) / NV - 1, 0);
        tail = v0 + n_vec * NV;
        skew = static_cast<int>(reinterpret_cast<uintptr_t>(row + v0) & 15);
        from = reinterpret_cast<const char *>(row + v0) - skew;
    }
    __device__ __forceinline__ int chunks() const { return n_vec > CHUNK ? (n_vec + CHUNK - 1) / CHUNK : 1; }
};

// mbar_wait, asleep for up to 20 us at a try: the block's warps wait for memory
// most of the time, and a warp that polls takes issue slots from those that work.
__device__ __forceinline__ void wait_for(uint64_t *bar, uint32_t parity, int *err)
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok)
                 : "r"(smem_u32(bar)), "r"(parity), "r"(20000u)
                 : "memory");
    if (!ok) mbar_wait(bar, parity, err);
}

__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

// The n best of a split once more, step by step with a barrier each, for data
// that ran over the buffer (logits that keep rising): where a step's keys do
// not fit, the buffer is cut to its best and the threshold raised first.
template <typename T, bool MASK>
__device__ __noinline__ int best_by_steps(const BeamArgs &a, const Item<T> &it, Key *buf, Key *tmp, Key *s_keys,
                                          Key *s_nth, int *s_cnt, int *s_kept)
{
    constexpr int NV = Elem<T>::NV;
    const int t = threadIdx.x, words = (a.vocab + 31) >> 5;
    const uint32_t *allow = MASK ? a.allow + it.r * a.allow_stride : nullptr;
    const uint4 *vec = reinterpret_cast<const uint4 *>(it.from);
    block_sync();
    if (t == 0) *s_cnt = 0;
    Key limit = 0;
    // step -1: the tokens after the last vector
    for (int base = -NT; base < it.n_vec; base += NT) {
        float f[NV];
        const int i = base + t;
        int v = it.tail + t;
#pragma unroll
        for (int e = 0; e < NV; ++e) f[e] = -INFINITY;
        if (base < 0) {
            if (v < it.v1) f[0] = beam_f(it.row[v]);
        } else if (i < it.n_vec) {
            v = it.v0 + i * NV;
            uint4 x = vec[i];
            if (it.skew) x = joined(x, vec[i + 1], it.skew);
            unpack<T>(x, f);
        }
        if constexpr (MASK) {
            const uint32_t bits = v < it.v1 ? allow_bits(allow, words, v) : 0u;
#pragma unroll
            for (int e = 0; e < NV; ++e)
                if (!((bits >> e) & 1u)) f[e] = -INFINITY;
        }
        Key k[NV], best = 0;
        int mine = 0;
#pragma unroll
        for (int e = 0; e < NV; ++e) {
            k[e] = f[e] > -INFINITY ? key_of(f[e] + 0.f, v + e) : 0;
            best = k[e] > best ? k[e] : best;
            mine += k[e] && k[e] >= limit;
        }
        block_sync();
        const int before = *s_cnt;
        block_sync();
        int at = mine ? atomicAdd(s_cnt, mine) : 0;
        block_sync();
        if (*s_cnt > a.cap) {
            const int kept = keep_best(buf, tmp, before, a.n_out, s_keys, s_nth, s_kept);
            if (kept == a.n_out && buf[kept - 1] > limit) limit = buf[kept - 1];
            const Key nth = nth_of_groups(best, a.n_out, s_keys, s_nth);
            if (nth > limit) limit = nth;
            mine = 0;
#pragma unroll
            for (int e = 0; e < NV; ++e) mine += k[e] && k[e] >= limit;
            if (t == 0) *s_cnt = kept;
            block_sync();
            at = mine ? atomicAdd(s_cnt, mine) : 0;
        }
#pragma unroll
        for (int e = 0; e < NV; ++e)
            if (k[e] && k[e] >= limit) buf[at++] = k[e];
    }
    block_sync();
    return *s_cnt;
}

// Persistent blocks of eight warps that work and one that loads.  After a
// block's first item the loading warp takes items from a common counter; it keeps a ring of STAGES chunks
// full with bulk copies, across items, so that the ends of one item (its
// threshold, its lists) cost no memory time.  In a chunk a thread has U
// vectors; the working warps meet at a barrier only for thresholds.  The first
// chunk's threshold stays for the item while n <= STEADY (of random logits
// every chunk then brings n keys, at most 19 chunks; raising it as keys come in
// cost 17 us of 127 at 896 rows of 151936 with n = 16 where the block cut its
// buffer, and 3 of 65 where one warp did while the others went on); for larger
// n the buffer is cut to its n best after the 2nd, 4th, 8th ... chunk.  Keys that
// do not fit the buffer are dropped, and the item's best are found by
// best_by_steps.
//
// Measured at 1024 rows of 151936 bf16, 896 of them alive (272 MB), n = 16: 59 us
// = 4.6 TB/s, where the loads alone take 45.  The rest is what ring and blocks do
// not hide: the first chunk's threshold 2 us, keys past it 4, exponentials 4 (two
// floats an instruction; 5 with one), an item's end 5 (each of 456 blocks has two
// items, all end at much the same time).
template <typename T, bool MASK> __global__ void __launch_bounds__(NT + 32, 3) beam_rows_kernel(BeamArgs a)
{
    constexpr int NV = Elem<T>::NV;
    extern __shared__ __align__(16) unsigned char smem[];
    Key *buf = reinterpret_cast<Key *>(smem + STAGES * STAGE_BYTES), *tmp = buf + a.cap;
    __shared__ __align__(8) uint64_t s_full[STAGES], s_empty[STAGES];
    __shared__ Key s_keys[NT], s_nth;
    __shared__ float4 s_part[WARPS];
    __shared__ float2 s_z[WARPS];
    __shared__ int s_item[STAGES], s_cnt, s_kept, s_over;
    const int t = threadIdx.x, lane = t & 31;
    if (t == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&s_empty[i], WARPS);
        }
        fence_mbarrier_init();
    }
    wait_for_stream();
    __syncthreads();

    if (t >= NT) {
        if (lane) return;
        int k = 0;                                     // stages filled so far
        // an expired wait leaves its error and the loop runs on without waiting
        auto stage = [&] {
            const int st = k % STAGES;
            if (k >= STAGES) wait_for(&s_empty[st], (k / STAGES - 1) & 1, a.err);
            ++k;
            return st;
        };
        const int items = a.batch * a.beams * a.n_split;
        // an item is followed by one look at the counter: the items-th look is the last of the launch and
        // puts it back, so that the next call finds 0 whatever becomes of the kernels after this one
        auto following = [&] {
            const int n = atomicAdd(a.next, 1);
            if (n == items - 1) *a.next = 0;
            return static_cast<int>(gridDim.x) + n;
        };
        for (int i = blockIdx.x; i < items; i = following()) {
            const Item<T> it(a, i);
            if (!beam_reads(a, it.r)) continue;
            for (int c = 0; c < it.chunks(); ++c) {
                const int st = stage();
                s_item[st] = i;
                const int n = min(it.n_vec - c * CHUNK, CHUNK);
                if (n > 0) {
                    const uint32_t bytes = static_cast<uint32_t>(n + (it.skew ? 1 : 0)) * 16;
                    mbar_arrive_expect_tx(&s_full[st], bytes);
                    bulk_load(smem + st * STAGE_BYTES, it.from + static_cast<int64_t>(c) * CHUNK * 16, bytes, &s_full[st]);
                } else {
                    mbar_arrive(&s_full[st]);
                }
            }
        }
        const int st = stage();
        s_item[st] = -1;
        mbar_arrive(&s_full[st]);
        // no copy of this block is in flight when it ends
        for (int i = max(k - STAGES, 0); i < k; ++i) wait_for(&s_full[i % STAGES], (i / STAGES) & 1, a.err);
        return;
    }

    const float c = a.c;
    const int words = (a.vocab + 31) >> 5;
    int k = 0;                                         // stages used so far
    while (true) {
        wait_for(&s_full[k % STAGES], (k / STAGES) & 1, a.err);
        const int item = s_item[k % STAGES];
        if (item < 0) return;
        const Item<T> it(a, item);
        const uint32_t *allow = MASK ? a.allow + it.r * a.allow_stride : nullptr;
        if (t == 0) s_cnt = s_over = 0;
        RowStat st{-INFINITY, -INFINITY, 0.f, 0.f, 0.f};
        float one = -INFINITY;                         // used after the first chunk's sum
        const int one_v = it.tail + t;
        if (one_v < it.v1 && (!MASK || (allow[one_v >> 5] >> (one_v & 31)) & 1u)) one = beam_f(it.row[one_v]);
        Key limit = 0;                                 // keys below it are not among the best
        float limit_x = -INFINITY;
        const int chunks = it.chunks();
        for (int j = 0; j < chunks; ++j, ++k) {
            const int sg = k % STAGES, base = j * CHUNK;
            uint32_t bits[U];                          // MASK: which of a vector's tokens are allowed
            if constexpr (MASK) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int i = base + u * NT + t;
                    bits[u] = i < it.n_vec ? allow_bits(allow, words, it.v0 + i * NV) : 0u;
                }
            }
            if (j) wait_for(&s_full[sg], (k / STAGES) & 1, a.err);
            const uint4 *tile = reinterpret_cast<const uint4 *>(smem + sg * STAGE_BYTES);
            uint4 cur[U];
            if (base + CHUNK <= it.n_vec) {
#pragma unroll
                for (int u = 0; u < U; ++u) cur[u] = tile[u * NT + t];
            } else {
#pragma unroll
                for (int u = 0; u < U; ++u) cur[u] = base + u * NT + t < it.n_vec ? tile[u * NT + t] : all_low<T>();
            }
            if (it.skew) {
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (base + u * NT + t < it.n_vec) cur[u] = joined(cur[u], tile[u * NT + t + 1], it.skew);
            }
            if constexpr (MASK) {
#pragma unroll
                for (int u = 0; u < U; ++u) cur[u] = masked<T>(cur[u], bits[u]);
            }
            static_assert(U == 4, "the chunk's largest in pairs");
            float top;
            if constexpr (sizeof(T) == 4) {
                top = max_nan(max_nan(vec_max<T>(cur[0]), vec_max<T>(cur[1])), max_nan(vec_max<T>(cur[2]), vec_max<T>(cur[3])));
            } else {
                const auto both = [](const uint4 &x, const uint4 &y) {
                    return make_uint4(max_nan2<T>(x.x, y.x), max_nan2<T>(x.y, y.y), max_nan2<T>(x.z, y.z),
                                      max_nan2<T>(x.w, y.w));
                };
                top = vec_max<T>(both(both(cur[0], cur[1]), both(cur[2], cur[3])));
            }
            if (!(top == -INFINITY)) {
                st.m = max_nan(st.m, top);
                if (far_above(st, top, c)) rebase(st, top, c);
                float sum = 0.f;
                // (two floats an instruction)
                const auto add = [&](auto term) {
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        float f[NV];
                        unpack<T>(cur[u], f);
                        uint64_t p[NV / 2];
#pragma unroll
                        for (int e = 0; e < NV / 2; ++e) p[e] = term(f[2 * e], f[2 * e + 1]);
#pragma unroll
                        for (int h = NV / 4; h; h >>= 1)
#pragma unroll
                            for (int e = 0; e < h; ++e) p[e] = add2(p[e], p[e + h]);
                        float x, y;
                        unpack2(p[0], x, y);
                        sum += x + y;
                    }
                };
                if (plain(st.b)) {
                    const uint64_t c2 = pack2(c, c), b2 = pack2(st.b, st.b);
                    add([&](float x, float y) {
                        unpack2(fma2(pack2(x, y), c2, b2), x, y);
                        return pack2(ex2_approx(x), ex2_approx(y));
                    });
                } else {
                    add([&](float x, float y) { return pack2(x == st.ref ? 1.f : 0.f, y == st.ref ? 1.f : 0.f); });
                }
                add_z(st.z, st.lost, sum, 0.f);
            }
            const auto token = [&](int x) { return it.v0 + (base + (x / NV) * NT + t) * NV + x % NV; };   // of value x
            if (j == 0) {
                if (!(one == -INFINITY)) {
                    st.m = max_nan(st.m, one);
                    if (far_above(st, one, c)) rebase(st, one, c);
                    add_z(st.z, st.lost, plain(st.b) ? ex2_approx(fmaf(one, c, st.b)) : one == st.ref ? 1.f : 0.f, 0.f);
                }
                // the first threshold, from each thread's best
                Key best = one > -INFINITY ? key_of(one, one_v) : 0;
                if (top > -INFINITY) {
                    int at = -1;
#pragma unroll
                    for (int u = U - 1; u >= 0; --u) {
                        float f[NV];
                        unpack<T>(cur[u], f);
#pragma unroll
                        for (int e = NV - 1; e >= 0; --e)
                            if (f[e] == top) at = u * NV + e;
                    }
                    const Key q = at >= 0 ? key_of(top + 0.f, token(at)) : 0;    // (none: a NaN was the largest)
                    best = q > best ? q : best;
                }
                limit = nth_of_groups(best, a.n_out, s_keys, &s_nth);
                if (limit) limit_x = value_of(static_cast<uint32_t>(limit >> 32));
            }
            // keys from the limit on go to the buffer.  Few threads have any, so a warp looks through one such
            // thread's values together, a value a lane
            const auto put = [&](float x, int v) {
                const Key q = key_of(x, v);
                if (q < limit) return;
                const int at = atomicAdd(&s_cnt, 1);
                if (at < a.cap) buf[at] = q;
                else s_over = 1;
            };
            if (j == 0 && one >= limit_x && one > -INFINITY) put(one, one_v);
            const T *mine = reinterpret_cast<const T *>(smem + sg * STAGE_BYTES + it.skew) +
                            ((lane / NV) * NT + (t - lane)) * NV + lane % NV;
            for (uint32_t who = __ballot_sync(0xFFFFFFFFu, top >= limit_x && top > -INFINITY); who; who &= who - 1) {
                const int from = __ffs(who) - 1, i = base + (lane / NV) * NT + t - lane + from;
                float x = -INFINITY;
                if (lane < U * NV && i < it.n_vec) x = beam_f(mine[from * NV]);
                if constexpr (MASK) {
                    uint32_t w = 0;
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const uint32_t y = __shfl_sync(0xFFFFFFFFu, bits[u], from);
                        if (lane / NV == u) w = y;
                    }
                    if (!((w >> (lane % NV)) & 1u)) x = -INFINITY;
                }
                if (x >= limit_x && x > -INFINITY) put(x, it.v0 + i * NV + lane % NV);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_empty[sg]);  // this warp is done with the chunk
            if (a.n_out > STEADY && j && (j & (j + 1)) == 0 && j + 1 < chunks) {
                block_sync();
                if (!s_over) {
                    const int kept = keep_best(buf, tmp, s_cnt, a.n_out, s_keys, &s_nth, &s_kept);
                    if (kept == a.n_out && buf[kept - 1] > limit) {
                        limit = buf[kept - 1];
                        limit_x = value_of(static_cast<uint32_t>(limit >> 32));
                    }
                    if (t == 0) s_cnt = kept;
                    block_sync();
                }
            }
        }
        // the split's highest base, its keys cut to the best, its sum: every thread's sum is brought to that
        // base and added up in two floats (a double addition runs at a sixty-fourth of a float's rate)
        float m = st.m, ref = st.ref, bb = st.b;
        auto higher = [&](float x, float y) {
            if (x > ref) {
                ref = x;
                bb = y;
            }
        };
        for (int o = 16; o; o >>= 1) {
            m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
            higher(__shfl_xor_sync(0xFFFFFFFFu, ref, o), __shfl_xor_sync(0xFFFFFFFFu, bb, o));
        }
        if (lane == 0) s_part[t >> 5] = make_float4(m, ref, bb, 0.f);
        block_sync();
        int cnt = s_cnt;
        if (s_over) cnt = best_by_steps<T, MASK>(a, it, buf, tmp, s_keys, &s_nth, &s_cnt, &s_kept);
#pragma unroll
        for (int i = 0; i < WARPS; ++i) {
            const float4 x = s_part[i];
            m = max_nan(m, x.x);
            higher(x.y, x.z);
        }
        float z = 0.f, lost = 0.f;
        if (st.ref > -INFINITY) {
            const float g = to_base(st.ref, st.b, ref, bb);
            z = st.z * g;
            lost = st.lost * g;
        }
        for (int o = 16; o; o >>= 1) {
            const float x = __shfl_xor_sync(0xFFFFFFFFu, z, o), y = __shfl_xor_sync(0xFFFFFFFFu, lost, o);
            add_z(z, lost, x, y);
        }
        if (lane == 0) s_z[t >> 5] = make_float2(z, lost);
        const int kept = keep_best(buf, tmp, cnt, a.n_out, s_keys, &s_nth, &s_kept);
        for (int i = t; i < a.n_out; i += NT)
            a.cand[static_cast<int64_t>(item) * a.n_out + i] =
                i < kept ? BeamCand{value_of(static_cast<uint32_t>(buf[i] >> 32)),
                                    static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(buf[i]))}
                         : BeamCand{0.f, -1};
        if (t == NT - 32) {
            z = lost = 0.f;
            for (int i = 0; i < WARPS; ++i) add_z(z, lost, s_z[i].x, s_z[i].y);
            a.stat[item] = BeamStat{m < INFINITY ? z : NAN, lost, m, ref, bb};
        }
    }
}

// ---- rows of few tokens ----------------------------------------------------------------
// A warp per row, SMALL / 32 tokens a lane: the rows kernel's blocks, each with
// its thresholds and barriers per item, took 42 us for 1560 rows of 20 tokens.
constexpr int SMALL = 512;
template <typename T> __global__ void __launch_bounds__(128) beam_small_kernel(BeamArgs a)
{
    constexpr int N = SMALL / 32;
    const int r = static_cast<int>((static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x) >> 5), lane = threadIdx.x & 31;
    wait_for_stream();
    if (r >= a.batch * a.beams || !beam_reads(a, r)) return;
    const T *row = static_cast<const T *>(a.logits) + r * a.row_stride;
    const uint32_t *allow = a.allow ? a.allow + r * a.allow_stride : nullptr;
    float x[N], m = -INFINITY;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int v = lane + 32 * i;
        x[i] = -INFINITY;
        if (v < a.vocab && (!allow || (allow[i] >> lane) & 1u)) x[i] = beam_f(row[v]);
        m = max_nan(m, x[i]);
    }
    for (int o = 16; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    const float b = -m * a.c;
    float z = 0.f, lost = 0.f;
    if (m > -INFINITY) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            add_z(z, lost, plain(b) ? ex2_approx(fmaf(x[i], a.c, b)) : x[i] == m ? 1.f : 0.f, 0.f);
        for (int o = 16; o; o >>= 1) {
            const float p = __shfl_xor_sync(0xFFFFFFFFu, z, o), q = __shfl_xor_sync(0xFFFFFFFFu, lost, o);
            add_z(z, lost, p, q);
        }
    }
    if (lane == 0) a.stat[r] = BeamStat{m < INFINITY ? z : NAN, lost, m, m, b};
    // the best one by one: the largest logit, the lowest of its tokens
    BeamCand *cand = a.cand + static_cast<int64_t>(r) * a.n_out;
    for (int j = 0; j < a.n_out; ++j) {
        float best = -INFINITY;
        int at = 0;
#pragma unroll
        for (int i = N - 1; i >= 0; --i)
            if (x[i] >= best) {
                best = x[i];
                at = i;
            }
        const uint32_t mine = best > -INFINITY ? order_of(best) : 0u;
        const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, mine);
        const uint32_t tok = __reduce_min_sync(0xFFFFFFFFu, top && mine == top ? lane + 32u * at : 0xFFFFFFFFu);
        if (lane == 0) cand[j] = top ? BeamCand{value_of(top), static_cast<int>(tok)} : BeamCand{0.f, -1};
        if (!top) {
            for (int i = j + 1 + lane; i < a.n_out; i += 32) cand[i] = BeamCand{0.f, -1};
            break;
        }
        if (tok == lane + 32u * at) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (i == at) x[i] = -INFINITY;
        }
    }
}

// ---- merge -------------------------------------------------------------------------
// One block per batch entry.  A warp per beam joins the sums of its splits; the
// lists are joined while lane k of another warp forms beam k's log-sum-exp in
// double (one after the other 2 to 3 us more of 4 to 7); then every beam's candidates are ranked.  A list is in falling order,
// so a candidate's place among all is its place in its list and what a binary
// search counts in each other list, a thread for each (candidate, list).  Doubles run at a
// sixty-fourth of a float's rate here, so only what orders the beams is one:
// two logarithms and an exponential per beam, a quotient and two sums per candidate.  (The
// quotient itself, not a product by 1 / length ^ alpha, which puts -49 / 49 a step
// beside -1 / 1: equal ranks have to be equal.)
// The lists are joined by a warp per beam (up to 16 at a time) while one more
// warp does the logarithms, a lane per beam, and another the divisors.
constexpr int LIST_WARPS = 16, MERGE_WARPS = LIST_WARPS + 2, MERGE_NT = MERGE_WARPS * 32;

struct BeamRow {
    float z, lost, m, ref, b, start;
    int kind, len;                         // kind 0: no candidates, 1: its own (finished), 2: the row's
};

__device__ __forceinline__ void put_out(const BeamArgs &a, int b, int j, int k, int64_t tok, float score, bool was, int len)
{
    const int64_t o = static_cast<int64_t>(b) * a.n_out + j;
    a.parent_out[o] = k;
    a.token_out[o] = tok;
    a.score_out[o] = score;
    if (a.finished_out) a.finished_out[o] = k >= 0 && (was || tok == a.end_token);
    if (a.length_out) a.length_out[o] = len;
}

// x / T, rounded: joined with a sum to one instruction it would be exact on one side of x / T - lse and rounded
// on the other, 1e22 apart where logits lie at -3e38 (a row of which everything is masked).
__device__ __forceinline__ double scaled(float x, double inv_t) { return __dmul_rn(x, inv_t); }

// n^alpha; of multiples of a half (1 among them) exact wherever that is a double, so that ranks that are
// equal come out so.  Of others by a logarithm and an exponential, some steps of a double off: lengths that
// differ give no equal ranks there.  (By pow: 1.7 us more a selection.)
__device__ __forceinline__ double length_power(double n, double alpha)
{
    const double halves = 2.0 * fabs(alpha);
    if (!(halves <= 8.0 && halves == floor(halves))) return exp(alpha * log(n));
    const int j = static_cast<int>(halves);
    double p = j & 1 ? sqrt(n) : 1.0;
    for (int i = 0; i < j / 2; ++i) p *= n;
    return alpha < 0.0 ? 1.0 / p : p;
}

__global__ void __launch_bounds__(MERGE_NT) beam_merge_kernel(BeamArgs a)
{
    extern __shared__ __align__(16) unsigned char smem[];
    const int all = a.beams * a.n_out;
    Key *lists = reinterpret_cast<Key *>(smem);        // [beams][n_out]
    uint64_t *ranks = lists + all;                     // the same places: order of the rank, 0: no candidate
    Key *heads = ranks + all;                          // a warp's splits' lists, `depth` of each, and then:
    float *score = reinterpret_cast<float *>(heads);
    int *place = reinterpret_cast<int *>(score + all);
    __shared__ BeamRow s_row[LOSSK_BEAM_MAX_BEAMS];
    __shared__ double s_lse[LOSSK_BEAM_MAX_BEAMS], s_div[LOSSK_BEAM_MAX_BEAMS];
    __shared__ int s_valid[MERGE_WARPS];
    const int b = blockIdx.x, t = threadIdx.x, lane = t & 31, warp = t >> 5;
    wait_for_stream();
    // the splits' lists, each in falling order, from shared memory (what lies deeper than `depth` from
    // where it is); asked for before it is known whether the beam has any
    const int depth = a.n_split > 1 ? a.depth : a.n_out;
    Key *mine = heads + warp * a.n_split * depth;
    auto entry = [&](int k, int i, int j) {
        if (i >= a.n_split || j >= a.n_out) return Key(0);
        const BeamCand x = a.cand[(static_cast<int64_t>(b) * a.beams + k) * a.n_split * a.n_out + i * a.n_out + j];
        return x.tok >= 0 ? key_of(x.x, x.tok) : Key(0);
    };
    auto fetch = [&](int k) {
        if (a.n_split == 1)
            for (int j = lane; j < a.n_out; j += 32) lists[k * a.n_out + j] = entry(k, 0, j);
        else
            for (int i = lane; i < a.n_split * depth; i += 32) mine[i] = entry(k, i / depth, i % depth);
    };
    if (warp < LIST_WARPS && warp < a.beams) fetch(warp);
    for (int k = warp; k < a.beams; k += MERGE_WARPS) {
        const int r = b * a.beams + k;
        const float start = a.scores[r];
        const bool done = a.finished && a.finished[r];
        const int len = (a.lengths ? a.lengths[r] : 0) + (done ? 0 : 1);
        // lane i has splits i and i + 32
        BeamStat st[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            st[h] = BeamStat{0.f, 0.f, -INFINITY, -INFINITY, 0.f};
            if (lane + 32 * h < a.n_split) st[h] = a.stat[static_cast<int64_t>(r) * a.n_split + lane + 32 * h];
        }
        BeamRow row{0.f, 0.f, -INFINITY, -INFINITY, 0.f, start, isfinite(start) ? (done ? 1 : 2) : 0, len};
        if (!isfinite(start) && start != -INFINITY && lane == 0) raise_fault(a.fault, LOSSK_NON_FINITE_SCALAR);
        if (row.kind == 2) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                row.m = fmaxf(row.m, st[h].m);
                if (st[h].ref > row.ref) {
                    row.ref = st[h].ref;
                    row.b = st[h].b;
                }
            }
            for (int o = 16; o; o >>= 1) {
                row.m = fmaxf(row.m, __shfl_xor_sync(0xFFFFFFFFu, row.m, o));
                const float x = __shfl_xor_sync(0xFFFFFFFFu, row.ref, o), y = __shfl_xor_sync(0xFFFFFFFFu, row.b, o);
                if (x > row.ref) {
                    row.ref = x;
                    row.b = y;
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (st[h].ref > -INFINITY || isnan(st[h].z)) {
                    const float g = isnan(st[h].z) ? NAN : to_base(st[h].ref, st[h].b, row.ref, row.b);
                    add_z(row.z, row.lost, st[h].z * g, st[h].lost * g);
                }
            for (int o = 16; o; o >>= 1) {
                const float x = __shfl_xor_sync(0xFFFFFFFFu, row.z, o), y = __shfl_xor_sync(0xFFFFFFFFu, row.lost, o);
                add_z(row.z, row.lost, x, y);
            }
            if (!(row.z == row.z) && lane == 0) raise_fault(a.fault, LOSSK_NON_FINITE_SCALAR);
            if (!(row.z > 0.f)) row.kind = 0;
        }
        if (lane == 0) s_row[k] = row;
    }
    __syncthreads();
    if (warp == LIST_WARPS) {
        for (int k = lane; k < a.beams; k += 32) {
            const BeamRow row = s_row[k];
            double lse = -INFINITY;
            if (row.kind == 2) {
                // the sum's base in log2 units; the logits' own scale 1 / T about their largest, c about that
                const double base = plain(row.b) ? -static_cast<double>(row.b) : static_cast<double>(row.ref) * a.c;
                const double m = row.m;
                lse = scaled(row.m, a.inv_t) + (log(static_cast<double>(row.z) + row.lost) + LN2 * (base - m * a.c));
            }
            s_lse[k] = lse;
            if (a.lse_out) a.lse_out[b * a.beams + k] = static_cast<float>(lse);
        }
    } else if (warp > LIST_WARPS) {
        for (int k = lane; k < a.beams; k += 32) {
            const double n = s_row[k].len > 1 ? s_row[k].len : 1;
            s_div[k] = length_power(n, a.length_alpha);
        }
    } else {
        for (int k = warp; k < a.beams; k += LIST_WARPS) {
            if (k != warp) {
                __syncwarp();
                fetch(k);
            }
            const int kind = s_row[k].kind;
            __syncwarp();
            if (kind != 2) {
                // a finished beam's candidate is itself (its logit is not used)
                const int tok = a.end_token < 0 ? 0 : a.end_token;
                for (int j = lane; j < a.n_out; j += 32) lists[k * a.n_out + j] = kind == 1 && j == 0 ? key_of(0.f, tok) : 0;
            } else if (a.n_split > 1) {
                // lane i keeps the heads of lists i and i + 32
                auto at = [&](int i, int j) { return i < a.n_split && j < depth ? mine[i * depth + j] : entry(k, i, j); };
                int j0 = 0, j1 = 0;
                Key q0 = at(lane, 0), q1 = at(lane + 32, 0);
                for (int j = 0; j < a.n_out; ++j) {
                    const Key q = q1 > q0 ? q1 : q0;
                    const uint32_t hi = __reduce_max_sync(0xFFFFFFFFu, static_cast<uint32_t>(q >> 32));
                    const uint32_t lo = __reduce_max_sync(
                        0xFFFFFFFFu, static_cast<uint32_t>(q >> 32) == hi ? static_cast<uint32_t>(q) : 0u);
                    const Key best = (static_cast<uint64_t>(hi) << 32) | lo;
                    if (lane == 0) lists[k * a.n_out + j] = best;
                    if (best && q0 == best) q0 = at(lane, ++j0);
                    else if (best && q1 == best) q1 = at(lane + 32, ++j1);
                }
            }
        }
    }
    __syncthreads();
    auto score_of = [&](int i, int k) {
        const double s = s_row[k].start;
        return s_row[k].kind == 2 ? s + (scaled(value_of(static_cast<uint32_t>(lists[i] >> 32)), a.inv_t) - s_lse[k]) : s;
    };
    int valid = 0;
    for (int i = t; i < all; i += MERGE_NT) {
        const int k = i / a.n_out;
        const double s = lists[i] ? score_of(i, k) : 0.0;
        ranks[i] = lists[i] ? order_of(a.length_alpha == 0.0 ? s : s / s_div[k]) : 0;
        score[i] = static_cast<float>(s);
        place[i] = i - k * a.n_out;
        valid += lists[i] != 0;
    }
    for (int o = 16; o; o >>= 1) valid += __shfl_xor_sync(0xFFFFFFFFu, valid, o);
    if (lane == 0) s_valid[warp] = valid;
    __syncthreads();
    // A candidate's place: equal ranks go by the lower beam, then by the order of its list (the
    // larger logit, the lower token).
    for (int x = t; x < all * a.beams; x += MERGE_NT) {
        const int o = x / all, i = x - o * all, k = i / a.n_out;
        const uint64_t rank = ranks[i];
        if (o == k || !rank || place[i] >= a.n_out) continue;   // (another thread may just be adding to it)
        const uint64_t *list = ranks + o * a.n_out;
        int lo = 0, hi = a.n_out;                      // the first entry that does not come before mine
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (list[mid] > rank || (list[mid] == rank && o < k)) lo = mid + 1;
            else hi = mid;
        }
        if (lo) atomicAdd(&place[i], lo);
    }
    __syncthreads();
    for (int i = t; i < all; i += MERGE_NT) {
        if (!ranks[i] || place[i] >= a.n_out) continue;
        const int k = i / a.n_out;
        const bool was = s_row[k].kind == 1;
        put_out(a, b, place[i], k, was ? a.end_token : static_cast<int64_t>(0xFFFFFFFFu - static_cast<uint32_t>(lists[i])),
                score[i], was, s_row[k].len);
    }
    valid = 0;
    for (int i = 0; i < MERGE_WARPS; ++i) valid += s_valid[i];
    for (int j = valid + t; j < a.n_out; j += MERGE_NT) put_out(a, b, j, -1, -1, -INFINITY, false, 0);
}

template <typename V>
__global__ void beam_gather_kernel(int64_t n_src, int64_t n_dst, int64_t words, const int32_t *__restrict__ parent,
                                   const V *__restrict__ src, V *__restrict__ dst, int *fault)
{
    const int64_t j = blockIdx.x, g = j / n_dst;
    wait_for_stream();
    const int p = parent[j];
    const bool ok = p >= 0 && p < n_src;
    if (!ok && p != -1 && threadIdx.x == 0 && blockIdx.y == 0) raise_fault(fault, LOSSK_TARGET_OUT_OF_RANGE);
    const V *s = src + (g * n_src + (ok ? p : 0)) * words;
    V *d = dst + j * words;
    for (int64_t i = static_cast<int64_t>(blockIdx.y) * blockDim.x + threadIdx.x; i < words;
         i += static_cast<int64_t>(gridDim.y) * blockDim.x)
        d[i] = ok ? s[i] : V{};
}

} // namespace

// Blocks take items as they get free.  A row is cut where that makes the last
// round of items fuller; an item's fixed work (its thresholds, lists and
// sums) is about that of ITEM_TOKENS tokens, and a split has a chunk of 16-bit
// logits at least (smaller ones make the merge's lists more, not the rows' time less).
constexpr int ROW_BLOCKS = 3 * 152;
constexpr double ITEM_TOKENS = 32000.0;
int beam_splits(int64_t rows, int64_t vocab)
{
    int64_t most = (vocab + CHUNK * 8 - 1) / (CHUNK * 8);
    if (most > 64) most = 64;
    int64_t best = 1;
    double cost = 0.0;
    for (int64_t n = 1; n <= most; ++n) {
        const double c = static_cast<double>((rows * n + ROW_BLOCKS - 1) / ROW_BLOCKS) *
                         (static_cast<double>(vocab) / n + ITEM_TOKENS);
        if (n == 1 || c < cost * 0.97) {
            cost = c;
            best = n;
        }
    }
    return static_cast<int>(best);
}

// Keys the rows kernel's buffer holds: what passes one step's threshold of
// best_by_steps at most (n groups' every key) beside the n best, and room for
// a first chunk of random logits.
int beam_cap(int dtype, int n_out)
{
    const int keys = n_out + n_out * (NT / groups_for(n_out)) * (dtype == LOSSK_F32 ? 4 : 8);
    return keys > 1024 ? keys : 1024;
}

template <typename T, bool MASK> cudaError_t launch_rows(const BeamArgs &a, cudaStream_t st)
{
    const size_t bytes = STAGES * STAGE_BYTES + 2 * sizeof(Key) * static_cast<size_t>(a.cap);
    const cudaError_t e = raise_smem<beam_rows_kernel<T, MASK>>(bytes);
    if (e != cudaSuccess) return e;
    const int64_t items = static_cast<int64_t>(a.batch) * a.beams * a.n_split;
    return launch(beam_rows_kernel<T, MASK>, dim3(static_cast<unsigned>(items < ROW_BLOCKS ? items : ROW_BLOCKS)),
                  dim3(NT + 32), bytes, st, a);
}

template <typename T> cudaError_t launch_small(const BeamArgs &a, cudaStream_t st)
{
    return launch(beam_small_kernel<T>, dim3(static_cast<unsigned>((static_cast<int64_t>(a.batch) * a.beams + 3) / 4)),
                  dim3(128), 0, st, a);
}

cudaError_t launch_beam_rows(const BeamArgs &a, cudaStream_t st)
{
    if (a.vocab <= SMALL)
        return a.dtype == LOSSK_F32 ? launch_small<float>(a, st)
             : a.dtype == LOSSK_BF16 ? launch_small<uint16_t>(a, st) : launch_small<h16_t>(a, st);
    if (a.dtype == LOSSK_F32) return a.allow ? launch_rows<float, true>(a, st) : launch_rows<float, false>(a, st);
    if (a.dtype == LOSSK_BF16) return a.allow ? launch_rows<uint16_t, true>(a, st) : launch_rows<uint16_t, false>(a, st);
    return a.allow ? launch_rows<h16_t, true>(a, st) : launch_rows<h16_t, false>(a, st);
}

cudaError_t launch_beam_merge(const BeamArgs &a0, cudaStream_t st)
{
    BeamArgs a = a0;
    const size_t all = static_cast<size_t>(a.beams) * a.n_out;
    // at most 512 entries of a beam's splits in shared memory
    a.depth = a.n_split == 1 ? 0 : a.n_out < 512 / a.n_split ? a.n_out : 512 / a.n_split;
    const size_t heads = LIST_WARPS * static_cast<size_t>(a.n_split) * a.depth;
    const size_t bytes = sizeof(Key) * (2 * all + (heads > all ? heads : all));
    const cudaError_t e = raise_smem<beam_merge_kernel>(bytes);
    if (e != cudaSuccess) return e;
    return launch(beam_merge_kernel, dim3(static_cast<unsigned>(a.batch)), dim3(MERGE_NT), bytes, st, a);
}

cudaError_t launch_beam_gather(int64_t n_group, int64_t n_src, int64_t n_dst, int64_t row_bytes,
                               const int32_t *parent, const void *src, void *dst, int *fault, cudaStream_t st)
{
    const uintptr_t all = reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(dst) |
                          static_cast<uintptr_t>(row_bytes);
    const int64_t unit = all % 16 == 0 ? 16 : all % 4 == 0 ? 4 : 1, words = row_bytes / unit;
    // a row is cut into blocks of about 16 elements a thread, at most 64 of them
    const int64_t cut = (words + 256 * 16 - 1) / (256 * 16);
    const dim3 grid(static_cast<unsigned>(n_group * n_dst), static_cast<unsigned>(cut > 64 ? 64 : cut));
    if (unit == 16)
        return launch(beam_gather_kernel<uint4>, grid, dim3(256), 0, st, n_src, n_dst, words, parent,
                      static_cast<const uint4 *>(src), static_cast<uint4 *>(dst), fault);
    if (unit == 4)
        return launch(beam_gather_kernel<uint32_t>, grid, dim3(256), 0, st, n_src, n_dst, words, parent,
                      static_cast<const uint32_t *>(src), static_cast<uint32_t *>(dst), fault);
    return launch(beam_gather_kernel<uint8_t>, grid, dim3(256), 0, st, n_src, n_dst, words, parent,
                  static_cast<const uint8_t *>(src), static_cast<uint8_t *>(dst), fault);
}

} // namespace lossk
