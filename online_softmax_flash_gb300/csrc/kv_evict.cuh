// Eviction from a K/V cache by accumulated attention weight: choice of the rows to keep, and the move.
#pragma once

#include "osf_internal.cuh"

namespace osf {

struct EvictProblem {
    const float *w;             // [B, Hkv, S]
    float *w_out;               // [B, Hkv, S_out]
    const int *lens;            // nullable: S
    int *lens_out;              // nullable
    int *idx;                   // [B, Hkv, budget]
    const unsigned char *src[2];   // [B, Hkv, S, row_bytes]; src[1] nullable
    unsigned char *dst[2];         // [B, Hkv, S_out, row_bytes]
    long long row_bytes[2];
    int B, Hkv, S, S_out, budget, sinks, recent;
    int *status;
};
cudaError_t launch_kv_evict(const EvictProblem &p, int sm_count, cudaStream_t s);

}  // namespace osf
