// k_attn_mma.cu -- the split pass of attention over a paged cache for 16-bit
// types, on the tensor cores.
//
// One new token per sequence makes the pass a stream: every key and value is
// read once from HBM and meets only the query rows of its KV head (and, for
// shared pages, of its group).  With 2 to 32 rows to a key tcgen05 would spend
// tiles of 128 on them, so the products run as mma.sync m16n8k16 with 16 query
// rows (the tensor pipe is 23 to 29 % active while HBM is read at 83 to 86 % of
// the copy rate), and the kernel is built around the loads.  (From 64 rows on the
// products bound it: 8 x 8 beams of 64 query heads 76 us, of 128 124.)
//
//  - every warp walks its own run of units with its own ring of STAGES tiles
//    of KT tokens in shared memory, filled by 16-byte asynchronous copies two
//    tiles ahead; no barrier joins warps, so a warp that rescales or starts a
//    new item never stops another's stream.
//  - a lane finds a token's page once per tile and hands its offset to the
//    lanes that copy the row; rows of no token, or of a page out of range, are
//    filled with zeros and masked, whatever the page holds there.
//  - scores stay in the accumulators' registers, where they already have the
//    layout of the second product's left operand.
//  - a weight goes to the tensor cores as the sum of two 16-bit values: two
//    instructions instead of one, which the stream hides.  Of bf16 that keeps
//    16 bits of every weight.  Of fp16 it keeps 22 of those above 2^-14, and
//    below that what lies above 2^-25, so the exponents' reference follows the
//    tiles' maxima both up and down (see Reference): every weight is within 2^-22 of
//    the largest in its tile, and the output's sums stay those of fp32.
//
// Measured, split pass and join: one sequence of 131072 tokens (8 KV heads of
// 128, bf16, 537 MB) 96 us, the pass alone 92 us = 5.8 TB/s; 33 sequences of 1 to
// 9000 tokens (160 MB, fp16) 37 us; 8 x 8 beams on 4096 shared tokens (170 MB) 50 us.
// What bounds it: the stream at 6.2 TB/s at the margin, and about 9 us before
// the first tile and after the last; with many short items also their products
// (8 x 8 beams: 37 us without the products, 32 without the loads, 42 with both).
// Two or four stages are within 2 % of three.
#include "attn_split.cuh"

namespace lossk {

namespace {

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t at)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t at)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if constexpr (F16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                     "{%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                     "{%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// m, the reference that a row's exponents are taken against, is not the running
// maximum: any m gives the same result, and rescaling the outputs for every new
// maximum would cost most tiles one (with 16 rows some maximum rises).  It moves
// to x - LIFT where a tile's maximum x is more than TOP above it, or LOW below.
//   bf16: up alone, TOP 8 and LIFT 0: weights of 2^8 at most.
//   fp16: LIFT 7 and TOP 15, so weights are up to 2^15 and a tile's largest is
//   2^7 when m moves.  m moves down as well: behind a token that outweighs the
//   rest by 2^26 their weights would be 0 to the tensor cores, while the sum of
//   weights in fp32 counts them (an output of 6 % off at 2^23, of 0 at 2^26, where
//   the heavy token's value is 0).  It stops where the weights so far add up to
//   2^MOST, which leaves the outputs' sums floats (values are below 2^16); what
//   weighs that much less is under any fp16 output's step.
template <bool F16> struct Reference {
    static constexpr float LIFT = F16 ? 7.f : 0.f, TOP = F16 ? 15.f : 8.f, LOW = 3.f, MOST = 70.f;
    // whether a tile of maximum x moves m (a row without tokens so far has m -infinity: it does)
    static __device__ __forceinline__ bool moves(float m, float x)
    {
        if constexpr (F16) return fabsf(x - m - (TOP - LOW) / 2) > (TOP + LOW) / 2;
        else return x > m + TOP;
    }
    // where to; l: the row's weights so far, against m
    static __device__ __forceinline__ float place(float m, float x, float l)
    {
        if (x > m + TOP) return x - LIFT;
        if constexpr (F16)
            if (x < m - LOW && x > -INFINITY) return fminf(m, fmaxf(x - LIFT, m - MOST + log2f(l)));
        return m;
    }
};

// A variant: head sizes up to HDP (a multiple of 32) and W warps on a ring.
// The warps of a ring share its tiles and its run of units, each with 16 query
// rows of its own: where more than 16 rows meet a key (a wide group of heads,
// beams over shared pages) it is still read once, and no warp carries more than
// 16 rows' outputs in registers.
template <int HDP_, int W_> struct Variant {
    static constexpr int HDP = HDP_, W = W_;
    static constexpr int KT = 16;
    static constexpr int STAGES = 3;
    // rows an odd number of 16-byte words apart: the 8 rows of a matrix load lie in different banks
    static constexpr int RS = HDP * 2 + 16;
    static constexpr int TILE = KT * RS;
    static constexpr int LPR = HDP <= 64 ? 8 : HDP <= 128 ? 16 : 32;   // lanes that copy a row
    static constexpr int CPL = 1, ESIZE = 2;                           // 16-byte words each, bytes an element
    static constexpr bool QREG = W == 1 && HDP <= 128;                // query rows in registers
    static constexpr int QBYTES = W * 16 * RS;
    static constexpr int RING_BYTES = STAGES * 2 * TILE + QBYTES + 16 * W;
    static constexpr int SPACE = 227 * 1024 - BASE_BYTES;
    // warps whose registers fit (9 of heads of 96 have 168 each, as 12 have, and spill: 33 ragged sequences 32 us, 8 25)
    static constexpr int MOST = HDP <= 64 ? 12 : HDP <= 96 && W == 1 ? 8 : HDP <= 128 ? 12 : 8;
    static constexpr int RINGS = SPACE / RING_BYTES < MOST / W ? SPACE / RING_BYTES : MOST / W;
    static constexpr int THREADS = RINGS * W * 32;
};

// Where a warp works: its ring's place in shared memory, its own masks of valid
// tokens there, its number in the ring, and the ring's barrier.
struct Seat {
    uint32_t ring;
    uint32_t *valid;
    int sub, bar;
};
template <typename V> __device__ __forceinline__ void ring_sync(const Seat &at)
{
    if constexpr (V::W == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(at.bar), "n"(V::W * 32) : "memory");
}
// Whether x holds in any thread of the ring; a barrier, too.
template <typename V> __device__ __forceinline__ bool ring_any(const Seat &at, bool x)
{
    if constexpr (V::W == 1) {
        return __any_sync(0xFFFFFFFFu, x) != 0;
    } else {
        uint32_t r;
        asm volatile("{\n\t.reg .pred p, q;\n\t"
                     "setp.ne.u32 p, %1, 0;\n\t"
                     "bar.red.or.pred q, %2, %3, p;\n\t"
                     "selp.u32 %0, 1, 0, q;\n\t}"
                     : "=r"(r)
                     : "r"(static_cast<uint32_t>(x)), "r"(at.bar), "n"(V::W * 32)
                     : "memory");
        return r != 0;
    }
}
__device__ __forceinline__ float unless_nan(float x, float other) { return x == x ? x : other; }

// One piece; returns whether one of this lane's outputs is NaN.
// An infinite value times a weight's low part, which may be negative or 0, takes
// from what its high part gave: NaN instead of infinity.  So a run that leaves a
// NaN is walked once more with AGAIN, where every weight above 0 is 1, twice, and
// what that gives is stored where a NaN was.
template <typename V, bool F16, bool AGAIN>
__device__ __forceinline__ bool attn_piece(const AttnArgs &a, const Piece &p, const Seat &at)
{
    constexpr int HDP = V::HDP, KT = V::KT, STAGES = V::STAGES, RS = V::RS;
    constexpr int KS = HDP / 16, NT = KT / 8, DT = HDP / 8;
    static_assert(KT == 16 && DT % 4 == 0, "one step of keys, column tiles in fours");
    constexpr uint32_t FULL = KT == 32 ? 0xFFFFFFFFu : (1u << KT) - 1u;
    const int lane = threadIdx.x & 31, sub = at.sub;
    const uint32_t ring = at.ring, qs = ring + STAGES * 2 * V::TILE + sub * 16 * RS;
    uint32_t *valid = at.valid;
    const int ch = a.hd >> 3;                              // 16-byte words of a row
    // matrix loads: K rows (tokens) lane % 8 + 8 (lane / 16), word (lane / 8) % 2; V and Q rows lane % 16, word lane / 16
    const uint32_t k_off = ((lane & 7) + ((lane >> 4) << 3)) * RS + ((lane >> 3) & 1) * 16;
    const uint32_t v_off = (lane & 15) * RS + (lane >> 4) * 16;
    const int mine0 = sub * 16;                        // this warp's first row of the item
    const bool active = mine0 < p.rows;
    const int n_tiles = (p.t1 - p.t0 + KT - 1) / KT;
    TileStream<V> in(a, p, sub, lane, ring, valid);
    // the query rows, zeros past the last one, come with the first tile (loaded and stored one after the
    // other: 132 instead of 105 us for 200 groups of 4 sequences of 120 to 320 tokens)
#pragma unroll 4
    for (int i = lane; i < 16 * (HDP / 8); i += 32) {
        const int rr = i / (HDP / 8), cc = i % (HDP / 8);
        const bool in_row = mine0 + rr < p.rows && cc < ch;
        const uint16_t *from = static_cast<const uint16_t *>(a.q);
        if (in_row)
            from += row_seq(a, p, mine0 + rr) * a.q_stride + static_cast<int64_t>(row_head(a, p, mine0 + rr)) * a.hd + cc * 8;
        cp16_or_zero(qs + rr * RS + cc * 16, from, in_row ? 16 : 0);
    }
    in.start(n_tiles);
    cp_wait<STAGES - 2>();
    __syncwarp();
    uint32_t qf[V::QREG ? KS : 1][4];
    if constexpr (V::QREG) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) ldsm4(qf[ks], qs + v_off + ks * 32);
    }
    float o[DT][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[d][e] = 0.f;

    for (int i = 0; i < n_tiles; ++i) {
        // once every warp of the ring is here, tile i has landed and tile i - 1's stage is free
        cp_wait<STAGES - 2>();
        ring_sync<V>(at);
        in.next(i, n_tiles);
        const int st = i % STAGES;
        if (active) {
            const uint32_t kt = ring + st * 2 * V::TILE, vt = kt + V::TILE;
            const uint32_t mask = valid[st];
            // scores; even and odd steps add up apart: four sums in flight, not two
            float s[2][NT][4];
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[x][j][e] = 0.f;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                uint32_t q4[4];
                if constexpr (V::QREG) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) q4[e] = qf[ks][e];
                } else {
                    ldsm4(q4, qs + v_off + ks * 32);
                }
#pragma unroll
                for (int j = 0; j < NT; j += 2) {
                    uint32_t b[4];
                    ldsm4(b, kt + j * 8 * RS + k_off + ks * 32);
                    mma16816<F16>(s[ks & 1][j], q4, b[0], b[1]);
                    mma16816<F16>(s[ks & 1][j + 1], q4, b[2], b[3]);
                }
            }
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[0][j][e] = (s[0][j][e] + s[1][j][e]) * a.scale_log2;
            if (mask != FULL) {
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (!((mask >> (j * 8 + (lane & 3) * 2 + (e & 1))) & 1u)) s[0][j][e] = -INFINITY;
            }
            float z[2];
            bool moves = false;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float x = fmaxf(fmaxf(s[0][0][2 * h], s[0][0][2 * h + 1]), fmaxf(s[0][1][2 * h], s[0][1][2 * h + 1]));
                x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 1));
                x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 2));
                moves |= Reference<F16>::moves(m[h], x);
                z[h] = x;
            }
            if (__any_sync(0xFFFFFFFFu, moves)) {
                float f[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float sum = l[h];                  // of this lane's keys, then of the row's
                    sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
                    sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
                    const float to = Reference<F16>::place(m[h], z[h], sum);
                    f[h] = m[h] == -INFINITY ? 0.f : ex2_approx(m[h] - to);
                    m[h] = to;
                    l[h] *= f[h];
                }
#pragma unroll
                for (int d = 0; d < DT; ++d) {
                    o[d][0] *= f[0];
                    o[d][1] *= f[0];
                    o[d][2] *= f[1];
                    o[d][3] *= f[1];
                }
            }
            z[0] = m[0] == -INFINITY ? 0.f : m[0];
            z[1] = m[1] == -INFINITY ? 0.f : m[1];
            uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float x = ex2_approx(s[0][j][2 * h] - z[h]), y = ex2_approx(s[0][j][2 * h + 1] - z[h]);
                    l[h] += x + y;
                    if constexpr (AGAIN) {
                        ph[j][h] = pl[j][h] = pack_16x2<F16>(x > 0.f ? 1.f : x, y > 0.f ? 1.f : y);
                    } else {
                        const uint32_t hi = pack_16x2<F16>(x, y);
                        ph[j][h] = hi;
                        pl[j][h] = pack_16x2<F16>(x - h16_lo<F16>(hi), y - h16_hi<F16>(hi));
                    }
                }
            // weights times values, two pairs of column tiles at a time: four sums in flight
#pragma unroll
            for (int d = 0; d < DT; d += 4) {
                uint32_t b[2][4];
                ldsm4_t(b[0], vt + v_off + d * 16);
                ldsm4_t(b[1], vt + v_off + (d + 2) * 16);
                const uint32_t hi[4] = {ph[0][0], ph[0][1], ph[1][0], ph[1][1]};
                const uint32_t lo[4] = {pl[0][0], pl[0][1], pl[1][0], pl[1][1]};
#pragma unroll
                for (int x = 0; x < 4; ++x) mma16816<F16>(o[d + x], hi, b[x >> 1][2 * (x & 1)], b[x >> 1][2 * (x & 1) + 1]);
#pragma unroll
                for (int x = 0; x < 4; ++x) mma16816<F16>(o[d + x], lo, b[x >> 1][2 * (x & 1)], b[x >> 1][2 * (x & 1) + 1]);
            }
        }
    }
    cp_wait<0>();
    bool none = false;                                     // whether one of this warp's outputs is NaN
    if (active) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float sum = l[h];
            sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
            sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
            const int i = mine0 + h * 8 + (lane >> 2);
            if (i >= p.rows) continue;
            const int col0 = (lane & 3) * 2;
#pragma unroll
            for (int d = 0; d < DT; ++d) none |= o[d][2 * h] != o[d][2 * h] || o[d][2 * h + 1] != o[d][2 * h + 1];
            if (p.slot < 0) {
                const float inv = sum > 0.f ? 1.f / sum : 1.f;
                const int64_t r = static_cast<int64_t>(row_seq(a, p, i)) * a.n_q + row_head(a, p, i);
                uint16_t *out = static_cast<uint16_t *>(a.out) + r * a.hd;
#pragma unroll
                for (int d = 0; d < DT; ++d)
                    if (d * 8 < a.hd) {
                        uint32_t *to = reinterpret_cast<uint32_t *>(out + d * 8 + col0);
                        float x = o[d][2 * h] * inv, y = o[d][2 * h + 1] * inv;
                        if constexpr (AGAIN) {
                            x = unless_nan(h16_lo<F16>(*to), x);
                            y = unless_nan(h16_hi<F16>(*to), y);
                        }
                        *to = pack_16x2<F16>(x, y);
                    }
                if (a.lse && col0 == 0) a.lse[r] = (m[h] == -INFINITY ? 0.f : m[h]) * float(LN2) + logf(sum);
            } else {
                float *d0 = p.part + static_cast<int64_t>(i) * (a.hd + ATTN_ROW);
#pragma unroll
                for (int d = 0; d < DT; ++d)
                    if (d * 8 < a.hd) {
                        float2 *to = reinterpret_cast<float2 *>(d0 + d * 8 + col0);
                        float2 x = make_float2(o[d][2 * h], o[d][2 * h + 1]);
                        if constexpr (AGAIN) x = make_float2(unless_nan(to->x, x.x), unless_nan(to->y, x.y));
                        *to = x;
                    }
                if (col0 == 0) *reinterpret_cast<float2 *>(d0 + a.hd) = make_float2(m[h], sum);
            }
        }
    }
    ring_sync<V>(at);
    return none;
}

// (a function of its own, so that its registers are not the first walk's; with a piece at a time walked
// again, what it needs stayed in registers throughout the first walk)
template <typename V, bool F16>
__device__ __noinline__ void attn_run_again(const AttnArgs &a, const long long *base, int w, Seat at)
{
    walk_run(a, base, w, [&](const Piece &p) { attn_piece<V, F16, true>(a, p, at); });
}

template <typename V, bool F16>
__global__ void __launch_bounds__(V::THREADS, 1) attn_mma_kernel(const __grid_constant__ AttnArgs a)
{
    constexpr int W = V::W;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ long long s_base[BASE_GROUPS + 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, ring_i = warp / W, sub = warp % W;
    unsigned char *mine = smem + ring_i * V::RING_BYTES;
    const Seat at{smem_u32(mine), reinterpret_cast<uint32_t *>(mine + V::STAGES * 2 * V::TILE + V::QBYTES) + 4 * sub, sub,
                  1 + ring_i};
    // the columns between the head's size and HDP are zero in every tile and stay so
    if (a.hd != V::HDP) {
        for (int i = sub * 32 + lane; i < V::RING_BYTES / 16; i += W * 32)
            reinterpret_cast<uint4 *>(mine)[i] = make_uint4(0, 0, 0, 0);
        ring_sync<V>(at);
    }
    const long long *base = unit_bases(a, s_base);
    // rings are numbered across the blocks first, so that few units still use every SM
    const int w = ring_i * gridDim.x + blockIdx.x;
    bool none = false;
    walk_run(a, base, w, [&](const Piece &p) { none |= attn_piece<V, F16, false>(a, p, at); });
    if (ring_any<V>(at, none)) attn_run_again<V, F16>(a, base, w, at);
}

template <int HDP, int W> cudaError_t launch_variant(bool f16, const AttnArgs &a, cudaStream_t st)
{
    using V = Variant<HDP, W>;
    constexpr int bytes = V::RINGS * V::RING_BYTES;
    const cudaError_t e = f16 ? raise_smem<attn_mma_kernel<V, true>>(bytes) : raise_smem<attn_mma_kernel<V, false>>(bytes);
    if (e != cudaSuccess) return e;
    auto kern = f16 ? attn_mma_kernel<V, true> : attn_mma_kernel<V, false>;
    return launch(kern, dim3(a.nw < 152 ? a.nw : 152),
                        dim3(V::THREADS), bytes, st, a);
}

template <int HDP> cudaError_t launch_hdp(bool f16, const AttnArgs &a, cudaStream_t st)
{
    return a.mr == 64 ? launch_variant<HDP, 4>(f16, a, st)
         : a.mr == 32 ? launch_variant<HDP, 2>(f16, a, st) : launch_variant<HDP, 1>(f16, a, st);
}

template <int HDP> AttnShape shape_hdp(int rows)
{
    return rows > 32 ? AttnShape{64, Variant<HDP, 4>::KT, Variant<HDP, 4>::RINGS}
         : rows > 16 ? AttnShape{32, Variant<HDP, 2>::KT, Variant<HDP, 2>::RINGS}
                     : AttnShape{16, Variant<HDP, 1>::KT, Variant<HDP, 1>::RINGS};
}

} // namespace

AttnShape attn_mma_shape(int hd, int rows)
{
    return hd <= 64 ? shape_hdp<64>(rows) : hd <= 96 ? shape_hdp<96>(rows) : hd <= 128 ? shape_hdp<128>(rows)
         : hd <= 192 ? shape_hdp<192>(rows) : shape_hdp<256>(rows);
}

cudaError_t launch_attn_mma(bool f16, const AttnArgs &a, cudaStream_t st)
{
    return a.hd <= 64 ? launch_hdp<64>(f16, a, st) : a.hd <= 96 ? launch_hdp<96>(f16, a, st)
         : a.hd <= 128 ? launch_hdp<128>(f16, a, st) : a.hd <= 192 ? launch_hdp<192>(f16, a, st)
                       : launch_hdp<256>(f16, a, st);
}

} // namespace lossk
