// Accumulated attention weight of every key (osf_attn_key_weights).
#pragma once

#include "osf_internal.cuh"

namespace osf {

struct KeyWeightsProblem {
    const void *q, *k;
    const float *lse;           // [B, Hq, Sq] natural log; -inf: the row sees no key
    float *w;                   // [B, Hkv, Sk]
    int dtype, B, Hq, Hkv, Sq, Sk, D;
    int causal, causal_off;     // key j is visible to row i iff !causal or j <= i + causal_off
    float scale_log2;           // scale * log2(e)
    long long q_sb, q_sh, q_ss, k_sb, k_sh, k_ss;
    int accumulate;
    int splits;                 // most parts of a key block's rows; each has partial sums in [splits][B * Hkv * Sk]
    long long tiles_per_part;   // row tiles of one part
    float *part;
    int *status;
};

// Base-2 exponent offset of a row with this log-sum-exp: a row that sees nothing adds nothing.
__device__ __forceinline__ float row_offset(float lse) { return lse == -INFINITY ? -INFINITY : -lse * kLog2e; }

// CUDA-core kernel: any type, head dimension and strides.
void key_weights_simt_plan(KeyWeightsProblem &p, int sm_count);   // sets splits and tiles_per_part
cudaError_t launch_key_weights_simt(const KeyWeightsProblem &p, cudaStream_t s);
// Tensor-core kernels (bf16): a few rows per kv head (D 32, 64, 96, 128), and any number of them (D 64, 128).
bool key_weights_rows_supported(const KeyWeightsProblem &p);
cudaError_t launch_key_weights_rows(const KeyWeightsProblem &p, int sm_count, cudaStream_t s);
bool key_weights_tc_supported(const KeyWeightsProblem &p);
size_t key_weights_tc_floats(int sm_count);   // partial sums it keeps in `part`
cudaError_t launch_key_weights_tc(const KeyWeightsProblem &p, int sm_count, cudaStream_t s);
// w (+)= the sum of the splits' parts, in split order.
cudaError_t launch_key_weights_reduce(const KeyWeightsProblem &p, cudaStream_t s);

}  // namespace osf
