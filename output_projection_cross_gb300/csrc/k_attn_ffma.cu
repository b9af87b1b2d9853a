// k_attn_ffma.cu -- the split pass of attention over a paged cache for fp32, on
// the CUDA cores (the tensor cores' tf32 alone would drop 13 of 24 bits; operands
// split into parts, which would keep them, are not built).
//
// As in k_attn_mma.cu every warp walks its own run of units with its own ring
// of tiles.  A tile's KT tokens lie across the lanes for the scores, 32 / KT
// lanes to a token, each with its part of the head; the head's columns lie
// across the lanes for the output (of heads up to 64 wide across half the
// lanes, the other half with the next token; the halves are added at the end).
// Each element of a tile is read from shared memory once and meets R query rows
// (scores: broadcast reads of q; output: of the weights).
//
// A warp's chain from a tile's scores to its output is longer than its loads, so
// warps are worth more than deep rings: two stages of small tiles, and as many
// warps as fit (12 where R rows leave them registers, 8 for R = 16).  Against
// three stages of 16 tokens (4 warps for heads of 128): 34 -> 28 us for 64
// sequences of 20 to 500 tokens with 8 KV heads of 128 and 32 query heads,
// 301 -> 238 us for 4 of 20000 with 128 query heads.  Products and sums go two
// floats an instruction (219 instead of 237 us at 128 query heads).
//
// Measured at 4 sequences of 20000 tokens, 8 KV heads of 128 (655 MB): 110 us =
// 6.0 TB/s for 8 query heads, 112 for 32, 133 for 64, 214 for 128.  Up to 4 rows to a KV head
// the stream bounds it, beyond that the multiply-adds and their reads of q and
// of the weights.
#include "attn_split.cuh"
#include "float2.cuh"

namespace lossk {

namespace {

constexpr float RISE = 8.f;                // a row's reference moves once its maximum is that far above it

template <int HDP_, int R_> struct FVariant {
    static constexpr int HDP = HDP_, R = R_, W = 1;
    // (a tile of 8 tokens of 256 columns for 8 rows: 172 us, of 4: 159; for 4 rows 121 and 123)
    static constexpr int KT = HDP <= 64 ? 16 : HDP <= 128 || R < 8 ? 8 : 4;
    static constexpr int STAGES = 2;
    static constexpr int RS = HDP * 4 + 16;            // an odd number of 16-byte words
    static constexpr int TILE = KT * RS;
    static constexpr int LPR = HDP <= 64 ? 16 : 32, CPL = HDP <= 128 ? 1 : 2, ESIZE = 4;
    static constexpr int QBYTES = R * HDP * 4, PBYTES = KT * R * 4;
    static constexpr int WARP_BYTES = STAGES * 2 * TILE + QBYTES + PBYTES + 16;
    static constexpr int SPACE = 227 * 1024 - BASE_BYTES;
    static constexpr int MOST = R == 16 ? 8 : 12;
    static constexpr int WARPS = SPACE / WARP_BYTES < MOST ? SPACE / WARP_BYTES : MOST;
};

template <typename V> __global__ void __launch_bounds__(V::WARPS * 32, 1) attn_ffma_kernel(AttnArgs a)
{
    constexpr int HDP = V::HDP, R = V::R, KT = V::KT, STAGES = V::STAGES, PARTS = 32 / KT, C = HDP <= 128 ? 1 : 2;
    constexpr int SETS = HDP <= 64 ? 128 / HDP : 1, COLS = 32 / SETS;   // a set of lanes has every SETS-th token's columns
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ long long s_base[BASE_GROUPS + 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned char *mine = smem + warp * V::WARP_BYTES;
    float *qs = reinterpret_cast<float *>(mine + STAGES * 2 * V::TILE), *ps = qs + R * HDP;
    uint32_t *valid = reinterpret_cast<uint32_t *>(ps + KT * R);
    // columns from the head's size on are zero in every tile and stay so
    if (a.hd != HDP) {
        for (int i = lane; i < V::WARP_BYTES / 16; i += 32) reinterpret_cast<uint4 *>(mine)[i] = make_uint4(0, 0, 0, 0);
        __syncwarp();
    }
    const long long *base = unit_bases(a, s_base);
    const int tok = lane % KT, part = lane / KT, set = lane / COLS, col = lane % COLS;
    const int steps = (a.hd + 4 * PARTS - 1) / (4 * PARTS);      // of four elements a lane
    const int w = warp * gridDim.x + blockIdx.x;

    walk_run(a, base, w, [&](const Piece &p) {
        const int n_tiles = (p.t1 - p.t0 + KT - 1) / KT;
        TileStream<V> in(a, p, 0, lane, smem_u32(mine), valid);
        // the query rows, zeros past the last one, come with the first tile
#pragma unroll 4
        for (int i = lane; i < R * (HDP / 4); i += 32) {
            const int r = i / (HDP / 4), e = i % (HDP / 4) * 4;
            const bool in_row = r < p.rows && e < a.hd;
            const float *from = static_cast<const float *>(a.q);
            if (in_row) from += row_seq(a, p, r) * a.q_stride + static_cast<int64_t>(row_head(a, p, r)) * a.hd + e;
            cp16_or_zero(smem_u32(qs + r * HDP + e), from, in_row ? 16 : 0);
        }
        in.start(n_tiles);
        ulonglong2 o[R][C];                                // four columns, in pairs
        float m[R], l[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            m[r] = -INFINITY;
            l[r] = 0.f;
#pragma unroll
            for (int x = 0; x < C; ++x) o[r][x] = make_ulonglong2(0, 0);
        }
        for (int i = 0; i < n_tiles; ++i) {
            cp_wait<STAGES - 2>();
            __syncwarp();
            in.next(i, n_tiles);
            const int st = i % STAGES;
            const unsigned char *kt = mine + st * 2 * V::TILE, *vt = kt + V::TILE;
            // (two products an instruction)
            uint64_t s2[R];
#pragma unroll
            for (int r = 0; r < R; ++r) s2[r] = 0;
            const float *kr = reinterpret_cast<const float *>(kt + tok * V::RS);
#pragma unroll 2
            for (int e = 0; e < steps; ++e) {
                const int at = (e * PARTS + part) * 4;
                const ulonglong2 x = *reinterpret_cast<const ulonglong2 *>(kr + at);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const ulonglong2 q = *reinterpret_cast<const ulonglong2 *>(qs + r * HDP + at);
                    s2[r] = fma2(q.x, x.x, s2[r]);
                    s2[r] = fma2(q.y, x.y, s2[r]);
                }
            }
            float s[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float y;
                unpack2(s2[r], s[r], y);
                s[r] += y;
            }
            const bool ok = (valid[st] >> tok) & 1u;
            bool rose = false;
            float top[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
#pragma unroll
                for (int x = KT; x < 32; x <<= 1) s[r] += __shfl_xor_sync(0xFFFFFFFFu, s[r], x);
                s[r] = ok ? s[r] * a.scale_log2 : -INFINITY;
                top[r] = s[r];
#pragma unroll
                for (int x = 1; x < KT; x <<= 1) top[r] = fmaxf(top[r], __shfl_xor_sync(0xFFFFFFFFu, top[r], x));
                rose |= top[r] > m[r] + RISE;
            }
            if (rose) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float y = top[r] > m[r] + RISE ? top[r] : m[r];
                    const float f = m[r] == -INFINITY ? 0.f : exp2f(m[r] - y);
                    m[r] = y;
                    l[r] *= f;
#pragma unroll
                    for (int x = 0; x < C; ++x) {
                        o[r][x].x = mul2(o[r][x].x, pack2(f, f));
                        o[r][x].y = mul2(o[r][x].y, pack2(f, f));
                    }
                }
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                s[r] = exp2f(s[r] - (m[r] == -INFINITY ? 0.f : m[r]));
                if (part == 0) l[r] += s[r];
            }
            __syncwarp();
            if (part == 0) {
#pragma unroll
                for (int r = 0; r < R; r += 4)
                    *reinterpret_cast<float4 *>(ps + tok * R + r) = make_float4(s[r], s[r + 1], s[r + 2], s[r + 3]);
            }
            __syncwarp();
#pragma unroll 4
            for (int jj = 0; jj < KT; jj += SETS) {
                const int j = jj + set;
                float pr[R];
#pragma unroll
                for (int r = 0; r < R; r += 4)
                    *reinterpret_cast<float4 *>(pr + r) = *reinterpret_cast<const float4 *>(ps + j * R + r);
#pragma unroll
                for (int x = 0; x < C; ++x)
                    if (SETS > 1 || lane * 4 + 128 * x < HDP) {
                        const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(vt + j * V::RS + col * 16 + 512 * x);
#pragma unroll
                        for (int r = 0; r < R; ++r) {
                            const uint64_t w2 = pack2(pr[r], pr[r]);
                            o[r][x].x = fma2(w2, v.x, o[r][x].x);
                            o[r][x].y = fma2(w2, v.y, o[r][x].y);
                        }
                    }
            }
        }
        cp_wait<0>();
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (r >= p.rows) break;
#pragma unroll
            for (int x = COLS; x < 32; x <<= 1) {
                o[r][0].x = add2(o[r][0].x, __shfl_xor_sync(0xFFFFFFFFu, o[r][0].x, x));
                o[r][0].y = add2(o[r][0].y, __shfl_xor_sync(0xFFFFFFFFu, o[r][0].y, x));
            }
            float sum = l[r];
            for (int x = 16; x; x >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, x);
            const int64_t row = static_cast<int64_t>(row_seq(a, p, r)) * a.n_q + row_head(a, p, r);
            const float inv = sum > 0.f ? 1.f / sum : 1.f;
            float *d = p.slot < 0 ? static_cast<float *>(a.out) + row * a.hd : p.part + static_cast<int64_t>(r) * (a.hd + ATTN_ROW);
            const float f = p.slot < 0 ? inv : 1.f;
#pragma unroll
            for (int x = 0; x < C; ++x) {
                const int e = col * 4 + 128 * x;
                if (set == 0 && e < a.hd)
                    *reinterpret_cast<ulonglong2 *>(d + e) =
                        make_ulonglong2(mul2(o[r][x].x, pack2(f, f)), mul2(o[r][x].y, pack2(f, f)));
            }
            if (lane == 0) {
                if (p.slot >= 0) *reinterpret_cast<float2 *>(d + a.hd) = make_float2(m[r], sum);
                else if (a.lse) a.lse[row] = (m[r] == -INFINITY ? 0.f : m[r]) * float(LN2) + logf(sum);
            }
        }
        __syncwarp();
    });
}

template <int HDP, int R> cudaError_t launch_fvariant(const AttnArgs &a, cudaStream_t st)
{
    using V = FVariant<HDP, R>;
    constexpr int bytes = V::WARPS * V::WARP_BYTES;
    const cudaError_t e = raise_smem<attn_ffma_kernel<V>>(bytes);
    if (e != cudaSuccess) return e;
    return launch(attn_ffma_kernel<V>, dim3(a.nw < 152 ? a.nw : 152), dim3(V::WARPS * 32), bytes, st, a);
}

template <int HDP> cudaError_t launch_fhdp(const AttnArgs &a, cudaStream_t st)
{
    if (a.mr == 4) return launch_fvariant<HDP, 4>(a, st);
    if constexpr (HDP <= 128)
        if (a.mr == 16) return launch_fvariant<HDP, 16>(a, st);
    return launch_fvariant<HDP, 8>(a, st);
}

template <int HDP> AttnShape fshape(int rows)
{
    if (rows <= 4) return AttnShape{4, FVariant<HDP, 4>::KT, FVariant<HDP, 4>::WARPS};
    if constexpr (HDP <= 128)                          // (16 rows of 256 columns do not fit the registers)
        if (rows > 8) return AttnShape{16, FVariant<HDP, 16>::KT, FVariant<HDP, 16>::WARPS};
    return AttnShape{8, FVariant<HDP, 8>::KT, FVariant<HDP, 8>::WARPS};
}

} // namespace

AttnShape attn_ffma_shape(int hd, int rows)
{
    return hd <= 64 ? fshape<64>(rows) : hd <= 128 ? fshape<128>(rows) : fshape<256>(rows);
}

cudaError_t launch_attn_ffma(const AttnArgs &a, cudaStream_t st)
{
    return a.hd <= 64 ? launch_fhdp<64>(a, st) : a.hd <= 128 ? launch_fhdp<128>(a, st) : launch_fhdp<256>(a, st);
}

} // namespace lossk
