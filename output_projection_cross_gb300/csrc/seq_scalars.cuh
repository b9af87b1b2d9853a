// seq_scalars.cuh -- the sequence losses' scalars, by one block of a kernel that runs
// after seq_coef.
#pragma once
#include "../../include/lossk.h"
#include "seq_internal.h"

namespace lossk {

// The coefficient kernel's blocks' sums, every T-th by a thread in their order, then a
// fixed tree.  All T threads of one block; no barrier is needed after it.
template <int T> __device__ __forceinline__ void seq_scalars(const SeqLoss &l, const SeqScratch &w)
{
    __shared__ double sh[3][T / 32];
    const int n = l.n_tok > l.n_seq ? l.n_tok : l.n_seq, blocks = (n + COEF_T - 1) / COEF_T;
    double v[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        v[k] = 0.0;
        for (int b = threadIdx.x; b < blocks; b += T) v[k] += w.acc[k * static_cast<int64_t>(blocks) + b];
        for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
        if ((threadIdx.x & 31) == 0) sh[k][threadIdx.x >> 5] = v[k];
    }
    __syncthreads();
    if (threadIdx.x != 0) return;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        v[k] = sh[k][0];
        for (int i = 1; i < T / 32; ++i) v[k] += sh[k][i];
    }
    float *o = l.scalars;
    if (l.pairs > 0) {
        const int pairs = w.hdr->pad[HDR_GROUPS], chosen = w.hdr->pad[HDR_CHOSEN];
        if (!(l.flags & LOSSK_REDUCE_SUM)) {
            v[0] = chosen > 0 ? v[0] / chosen : 0.0;
            v[1] = pairs > 0 ? v[1] / pairs : 0.0;
            v[2] = pairs > 0 ? v[2] / pairs : 0.0;
        }
        // (without the likelihood term its infinities stay out of the total)
        o[0] = static_cast<float>(l.nll > 0.f ? v[1] + static_cast<double>(l.nll) * v[0] : v[1]);
        o[1] = static_cast<float>(v[1]);
        o[2] = static_cast<float>(v[0]);
        o[3] = static_cast<float>(v[2]);
    } else {
        o[0] = static_cast<float>(l.kl > 0.f ? v[0] + static_cast<double>(l.kl) * v[1] : v[0]);
        o[1] = static_cast<float>(v[0]);
        o[2] = static_cast<float>(v[1]);
        o[3] = static_cast<float>(v[2]);
    }
}

} // namespace lossk
