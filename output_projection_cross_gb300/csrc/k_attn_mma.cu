// k_attn_mma.cu -- the split pass of attention over a paged cache for 16-bit
// types, on the tensor cores.
//
// One new token per sequence makes the pass a stream: every key and value is
// read once from HBM and meets only the query rows of its KV head (and, for
// shared pages, of its group), 2 to 32 multiply-adds a byte.  That is far below
// what tcgen05 needs to be worth its 128-row tiles, so the products run as
// mma.sync m16n8k16 with 16 query rows (1.5 of 16 tensor instructions per
// issue slot would be needed to keep HBM waiting), and the kernel is built
// around the loads:
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
//  - a weight goes to the tensor cores as the sum of two 16-bit values, so
//    that it keeps 16 (bf16) or 22 (fp16) bits: two instructions instead of
//    one, which the stream hides, for an output that is rounded once.
#include "attn_split.cuh"

#include <atomic>
#include <type_traits>

namespace lossk {

namespace {

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

// A variant: head sizes up to HDP (a multiple of 32), MT tiles of 16 query
// rows, KT tokens a unit, STAGES tiles in a warp's ring, WARPS warps a block.
template <int HDP_, int MT_> struct Variant {
    static constexpr int HDP = HDP_, MT = MT_;
    static constexpr int KT = 16;
    static constexpr int STAGES = 3;
    // rows an odd number of 16-byte words apart: the 8 rows of a matrix load lie in different banks
    static constexpr int RS = HDP * 2 + 16;
    static constexpr int TILE = KT * RS;
    static constexpr int LPR = HDP <= 64 ? 8 : HDP <= 128 ? 16 : 32;   // lanes that copy a row
    static constexpr bool QREG = MT * HDP <= 128;                     // query rows in registers
    static constexpr int QBYTES = MT * 16 * RS;
    static constexpr int WARP_BYTES = STAGES * 2 * TILE + QBYTES + 16 * ((STAGES + 3) / 4);
    static constexpr int WARPS = 227 * 1024 / WARP_BYTES > 8 ? 8 : 227 * 1024 / WARP_BYTES;
};

template <typename V, bool F16>
__global__ void __launch_bounds__(V::WARPS * 32, 1) attn_mma_kernel(AttnArgs a)
{
    constexpr int HDP = V::HDP, MT = V::MT, KT = V::KT, STAGES = V::STAGES, RS = V::RS;
    constexpr int KS = HDP / 16, NT = KT / 8, DT = HDP / 8;
    constexpr uint32_t FULL = KT == 32 ? 0xFFFFFFFFu : (1u << KT) - 1u;
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned char *mine = smem + warp * V::WARP_BYTES;
    const uint32_t ring = smem_u32(mine), qs = ring + STAGES * 2 * V::TILE;
    uint32_t *valid = reinterpret_cast<uint32_t *>(mine + STAGES * 2 * V::TILE + V::QBYTES);
    // the columns between the head's size and HDP are zero in every tile and stay so
    if (a.hd != HDP) {
        for (int i = lane; i < V::WARP_BYTES / 16; i += 32)
            reinterpret_cast<uint4 *>(mine)[i] = make_uint4(0, 0, 0, 0);
        __syncwarp();
    }
    const int ch = a.hd >> 3;                              // 16-byte words of a row
    const int c = lane % V::LPR, r0 = lane / V::LPR;
    const bool copies = c < ch;
    const uint16_t *kb = static_cast<const uint16_t *>(a.k) + c * 8;
    const uint16_t *vb = static_cast<const uint16_t *>(a.v) + c * 8;
    // matrix loads: K rows (tokens) lane % 8 + 8 (lane / 16), word (lane / 8) % 2; V and Q rows lane % 16, word lane / 16
    const uint32_t k_off = ((lane & 7) + ((lane >> 4) << 3)) * RS + ((lane >> 3) & 1) * 16;
    const uint32_t v_off = (lane & 15) * RS + (lane >> 4) * 16;
    // warps are numbered across the blocks first, so that few units still use every SM
    const int w = warp * gridDim.x + blockIdx.x;

    walk_run(a, w, [&](const Piece &p) {
        const int n_tiles = (p.t1 - p.t0 + KT - 1) / KT;
        const int64_t head = p.head * a.head_stride;
        const int32_t *row = a.table + p.seq * a.table_stride;
        // lane < KT: this lane's token of the tile to be looked up next, its page's column and its
        // place in the page; the page itself is loaded a tile before it is needed
        int t = p.t0 + lane, col = t / a.page, off = t % a.page;
        auto look_up = [&](int &pg, int &place) {
            const bool in = lane < KT && t < p.t1;
            pg = in ? row[col] : -2;
            place = off;
            t += KT;
            off += KT;
            while (off >= a.page) {
                off -= a.page;
                ++col;
            }
        };
        auto fetch = [&](int i, int pg, int place) {
            const int st = i % STAGES;
            const bool ok = pg >= 0 && pg < a.n_pages;
            if (!ok && pg != -2) raise_fault(a.fault, LOSSK_TARGET_OUT_OF_RANGE);
            const int64_t at = ok ? pg * a.page_stride + place * a.tok_stride + head : -1;
            const uint32_t mask = __ballot_sync(0xFFFFFFFFu, ok);
            if (lane == 0) valid[st] = mask;
            const uint32_t kd = ring + st * 2 * V::TILE + r0 * RS + c * 16, vd = kd + V::TILE;
            constexpr int STEP = 32 / V::LPR;
            // a whole tile inside one page: its rows are tok_stride apart
            if (mask == FULL && __shfl_sync(0xFFFFFFFFu, place, 0) + KT <= a.page) {
                const int64_t o = __shfl_sync(0xFFFFFFFFu, at, 0) + r0 * a.tok_stride;
                if (copies) {
                    const uint16_t *ks = kb + o, *vs = vb + o;
#pragma unroll
                    for (int j = 0; j < KT / STEP; ++j) {
                        cp16(kd + j * STEP * RS, ks);
                        cp16(vd + j * STEP * RS, vs);
                        ks += STEP * a.tok_stride;
                        vs += STEP * a.tok_stride;
                    }
                }
                return;
            }
#pragma unroll
            for (int j = 0; j < KT / STEP; ++j) {
                const int64_t o = __shfl_sync(0xFFFFFFFFu, at, j * STEP + r0);
                if (copies) {
                    const int bytes = o >= 0 ? 16 : 0;
                    cp16_or_zero(kd + j * STEP * RS, kb + (o >= 0 ? o : 0), bytes);
                    cp16_or_zero(vd + j * STEP * RS, vb + (o >= 0 ? o : 0), bytes);
                }
            }
        };
        int pg, place;
        look_up(pg, place);
#pragma unroll
        for (int i = 0; i < STAGES - 1; ++i) {
            int pg2, place2;
            look_up(pg2, place2);
            if (i < n_tiles) fetch(i, pg, place);
            cp_commit();
            pg = pg2;
            place = place2;
        }
        // the query rows, zeros past the last one
        uint32_t qf[V::QREG ? MT : 1][V::QREG ? KS : 1][4];
#pragma unroll
        for (int i = 0; i < MT * 16 * (HDP / 8); i += 32) {
            const int rr = (i + lane) / (HDP / 8), cc = (i + lane) % (HDP / 8);
            uint4 x = make_uint4(0, 0, 0, 0);
            if (rr < p.rows && cc < ch)
                x = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.q) +
                                                          row_seq(a, p, rr) * a.q_stride +
                                                          static_cast<int64_t>(row_head(a, p, rr)) * a.hd) + cc);
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(qs + rr * RS + cc * 16), "r"(x.x), "r"(x.y),
                         "r"(x.z), "r"(x.w)
                         : "memory");
        }
        __syncwarp();
        if constexpr (V::QREG) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) ldsm4(qf[mt][ks], qs + mt * 16 * RS + v_off + ks * 32);
        }
        float o[MT][DT][4], m[MT][2], l[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[mt][d][e] = 0.f;
            m[mt][0] = m[mt][1] = -INFINITY;
            l[mt][0] = l[mt][1] = 0.f;
        }
        // one tile's scores, weights and products for the first U tiles of query rows
        auto tile = [&](auto u_, int st) {
            constexpr int U = decltype(u_)::value;
            const uint32_t kt = ring + st * 2 * V::TILE, vt = kt + V::TILE;
            const uint32_t mask = valid[st];
            // with one tile of rows the even and odd steps add up apart: four sums in flight, not two
            constexpr int C = U == 1 ? 2 : 1;
            float s[U][C][NT][4];
#pragma unroll
            for (int mt = 0; mt < U; ++mt)
#pragma unroll
                for (int x = 0; x < C; ++x)
#pragma unroll
                    for (int j = 0; j < NT; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[mt][x][j][e] = 0.f;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                uint32_t q4[U][4];
#pragma unroll
                for (int mt = 0; mt < U; ++mt) {
                    if constexpr (V::QREG) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) q4[mt][e] = qf[mt][ks][e];
                    } else {
                        ldsm4(q4[mt], qs + mt * 16 * RS + v_off + ks * 32);
                    }
                }
#pragma unroll
                for (int j = 0; j < NT; j += 2) {
                    uint32_t b[4];
                    ldsm4(b, kt + j * 8 * RS + k_off + ks * 32);
#pragma unroll
                    for (int mt = 0; mt < U; ++mt) {
                        mma16816<F16>(s[mt][ks % C][j], q4[mt], b[0], b[1]);
                        mma16816<F16>(s[mt][ks % C][j + 1], q4[mt], b[2], b[3]);
                    }
                }
            }
            uint32_t ph[U][NT][2], pl[U][NT][2];
            float mx[U][2];
#pragma unroll
            for (int mt = 0; mt < U; ++mt) {
                mx[mt][0] = mx[mt][1] = -INFINITY;
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if constexpr (C == 2) s[mt][0][j][e] += s[mt][1][j][e];
                        s[mt][0][j][e] *= a.scale_log2;
                    }
            }
            if (mask != FULL) {
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (!((mask >> (j * 8 + (lane & 3) * 2 + (e & 1))) & 1u))
#pragma unroll
                            for (int mt = 0; mt < U; ++mt) s[mt][0][j][e] = -INFINITY;
            }
#pragma unroll
            for (int mt = 0; mt < U; ++mt) {
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) mx[mt][e >> 1] = fmaxf(mx[mt][e >> 1], s[mt][0][j][e]);
            }
            float f[U][2];
            bool rose = false;
#pragma unroll
            for (int mt = 0; mt < U; ++mt)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float x = mx[mt][h];
                    x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 1));
                    x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 2));
                    x = fmaxf(x, m[mt][h]);
                    const float z = x == -INFINITY ? 0.f : x;
                    f[mt][h] = ex2_approx(m[mt][h] - z);
                    rose |= f[mt][h] != 1.f;
                    m[mt][h] = x;
                    mx[mt][h] = z;
                }
            // the outputs are rescaled only where some row's maximum rose
            if (__any_sync(0xFFFFFFFFu, rose)) {
#pragma unroll
                for (int mt = 0; mt < U; ++mt) {
                    l[mt][0] *= f[mt][0];
                    l[mt][1] *= f[mt][1];
#pragma unroll
                    for (int d = 0; d < DT; ++d) {
                        o[mt][d][0] *= f[mt][0];
                        o[mt][d][1] *= f[mt][0];
                        o[mt][d][2] *= f[mt][1];
                        o[mt][d][3] *= f[mt][1];
                    }
                }
            }
#pragma unroll
            for (int mt = 0; mt < U; ++mt)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float x = ex2_approx(s[mt][0][j][2 * h] - mx[mt][h]);
                        const float y = ex2_approx(s[mt][0][j][2 * h + 1] - mx[mt][h]);
                        l[mt][h] += x + y;
                        const uint32_t hi = pack_16x2<F16>(x, y);
                        ph[mt][j][h] = hi;
                        pl[mt][j][h] = pack_16x2<F16>(x - h16_lo<F16>(hi), y - h16_hi<F16>(hi));
                    }
            // weights times values
#pragma unroll
            for (int kk = 0; kk < KT / 16; ++kk)
#pragma unroll
                for (int d = 0; d < DT; d += 2) {
                    uint32_t b[4];
                    ldsm4_t(b, vt + kk * 16 * RS + v_off + d * 16);
#pragma unroll
                    for (int mt = 0; mt < U; ++mt) {
                        const uint32_t hi[4] = {ph[mt][2 * kk][0], ph[mt][2 * kk][1], ph[mt][2 * kk + 1][0],
                                                ph[mt][2 * kk + 1][1]};
                        const uint32_t lo[4] = {pl[mt][2 * kk][0], pl[mt][2 * kk][1], pl[mt][2 * kk + 1][0],
                                                pl[mt][2 * kk + 1][1]};
                        mma16816<F16>(o[mt][d], hi, b[0], b[1]);
                        mma16816<F16>(o[mt][d + 1], hi, b[2], b[3]);
                        mma16816<F16>(o[mt][d], lo, b[0], b[1]);
                        mma16816<F16>(o[mt][d + 1], lo, b[2], b[3]);
                    }
                }
        };
        const int used = MT == 1 || p.rows <= 16 ? 1 : MT;
        for (int i = 0; i < n_tiles; ++i) {
            cp_wait<STAGES - 2>();
            __syncwarp();
            if (MT == 1 || used == 1) tile(std::integral_constant<int, 1>(), i % STAGES);
            else tile(std::integral_constant<int, MT>(), i % STAGES);
            __syncwarp();
            int pg2, place2;
            look_up(pg2, place2);
            if (i + STAGES - 1 < n_tiles) fetch(i + STAGES - 1, pg, place);
            cp_commit();
            pg = pg2;
            place = place2;
        }
        cp_wait<0>();
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            if (mt >= used) break;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float sum = l[mt][h];
                sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
                sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
                const int i = mt * 16 + h * 8 + (lane >> 2);
                if (i >= p.rows) continue;
                const int col = (lane & 3) * 2;
                if (p.slot < 0) {
                    const float inv = sum > 0.f ? 1.f / sum : 1.f;
                    const int64_t r = static_cast<int64_t>(row_seq(a, p, i)) * a.n_q + row_head(a, p, i);
                    uint16_t *out = static_cast<uint16_t *>(a.out) + r * a.hd;
#pragma unroll
                    for (int d = 0; d < DT; ++d)
                        if (d * 8 < a.hd)
                            *reinterpret_cast<uint32_t *>(out + d * 8 + col) =
                                pack_16x2<F16>(o[mt][d][2 * h] * inv, o[mt][d][2 * h + 1] * inv);
                    if (a.lse && col == 0)
                        a.lse[r] = (m[mt][h] == -INFINITY ? 0.f : m[mt][h]) * float(LN2) + logf(sum);
                } else {
                    float *d0 = p.part + static_cast<int64_t>(i) * (a.hd + ATTN_ROW);
#pragma unroll
                    for (int d = 0; d < DT; ++d)
                        if (d * 8 < a.hd)
                            *reinterpret_cast<float2 *>(d0 + d * 8 + col) = make_float2(o[mt][d][2 * h], o[mt][d][2 * h + 1]);
                    if (col == 0) *reinterpret_cast<float2 *>(d0 + a.hd) = make_float2(m[mt][h], sum);
                }
            }
        }
        __syncwarp();
    });
}

template <int HDP, int MT> cudaError_t launch_variant(bool f16, const AttnArgs &a, cudaStream_t st)
{
    using V = Variant<HDP, MT>;
    constexpr int bytes = V::WARPS * V::WARP_BYTES;
    auto kern = f16 ? attn_mma_kernel<V, true> : attn_mma_kernel<V, false>;
    // the shared-memory attribute is set once per device
    static std::atomic<int> ready[2][64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !ready[f16][dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) ready[f16][dev].store(1, std::memory_order_release);
    }
    const int grid = a.nw < 152 ? a.nw : 152;
    kern<<<grid, V::WARPS * 32, bytes, st>>>(a);
    return cudaGetLastError();
}

template <int HDP, int MT> constexpr AttnShape shape_of()
{
    using V = Variant<HDP, MT>;
    return AttnShape{16 * MT, V::KT, V::WARPS};
}

} // namespace

// Two tiles of query rows where more than 16 rows meet a key (a wide group of
// heads, or beams over shared pages) and the outputs still fit the registers.
AttnShape attn_mma_shape(int hd, int rows)
{
    const bool two = rows > 16;
    if (hd <= 64) return two ? shape_of<64, 2>() : shape_of<64, 1>();
    if (hd <= 96) return two ? shape_of<96, 2>() : shape_of<96, 1>();
    if (hd <= 128) return two ? shape_of<128, 2>() : shape_of<128, 1>();
    return hd <= 192 ? shape_of<192, 1>() : shape_of<256, 1>();
}

cudaError_t launch_attn_mma(bool f16, const AttnArgs &a, cudaStream_t st)
{
    const bool two = a.mr > 16;
    if (a.hd <= 64) return two ? launch_variant<64, 2>(f16, a, st) : launch_variant<64, 1>(f16, a, st);
    if (a.hd <= 96) return two ? launch_variant<96, 2>(f16, a, st) : launch_variant<96, 1>(f16, a, st);
    if (a.hd <= 128) return two ? launch_variant<128, 2>(f16, a, st) : launch_variant<128, 1>(f16, a, st);
    return a.hd <= 192 ? launch_variant<192, 1>(f16, a, st) : launch_variant<256, 1>(f16, a, st);
}

} // namespace lossk
