// host_internal.h -- host-side pieces that the losses' entry points share:
// tensor maps, the group passes' arguments, the helper streams.
#pragma once
#include "lossk_internal.h"

#include <mutex>

namespace lossk {

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int sm_count();

// Tensor maps (lossk_abi.cu says what each one is).
bool make_map_plain(CUtensorMap *m, const void *base, int64_t inner, int64_t outer, uint32_t box_inner,
                    uint32_t box_outer);
bool make_map(CUtensorMap *m, const void *base, int64_t inner, int64_t outer, uint32_t box_inner, uint32_t box_outer);
bool make_map_out_f32(CUtensorMap *m, void *base, int64_t inner, int64_t outer);
bool make_map_out_16(CUtensorMap *m, void *base, int64_t inner, int64_t outer);
bool make_map_out3_f32(CUtensorMap *m, void *base, int64_t inner, int64_t rows, int64_t planes);

// What the group passes need of a workspace.
struct BwdScratch {
    uint16_t *gring;
    unsigned *gsig;
    float4 *tokp;
    WsHeader *hdr;
};

// Tensor maps and shape fields of a cluster pass.  rows: d_hidden / fused
// (fixed = hidden token tiles, loop = vocabulary); otherwise d_weight (fixed =
// weight vocabulary tiles, loop = tokens).
bool bwd_args(const BwdScratch &w, bool rows, int64_t n, int64_t d, int64_t V, const void *H, const void *W,
              BwdArgs *a);

// A helper stream per (device, caller stream): the training step's small
// kernels that nothing after them waits for (the token mean, d_hidden's
// combine) run on it beside the d_weight pass, on the SMs its groups leave
// free; the call joins it back into the caller's stream before it returns.
// Calls on different caller streams get different helper streams, so neither
// waits for the other's helper work.  Up to SIDE_PER_DEV caller streams per
// device get one; a call on a further stream runs those kernels on its own
// stream (the same results, without the overlap).
struct SideStream {
    std::mutex mu;
    cudaStream_t owner = nullptr;      // the caller stream this helper serves
    bool used = false;
    cudaStream_t s = nullptr;
    cudaEvent_t fork = nullptr, join = nullptr;
    bool ready()
    {
        if (s) return true;
        if (cudaStreamCreateWithFlags(&s, cudaStreamNonBlocking) != cudaSuccess ||
            cudaEventCreateWithFlags(&fork, cudaEventDisableTiming) != cudaSuccess ||
            cudaEventCreateWithFlags(&join, cudaEventDisableTiming) != cudaSuccess) {
            (void)cudaGetLastError();
            s = nullptr;
            return false;
        }
        return true;
    }
};

SideStream *side_stream(cudaStream_t caller);

} // namespace lossk
