// The 4-bit K/V cache: record format, problem descriptions and launchers.
//
// A record holds K and V of one token of one kv head in 1.25 D bytes (D a multiple of 32):
//   [0, D/2)            codes of K          [D, D + D/8)          (scale, minimum) pairs of K
//   [D/2, D)            codes of V          [D + D/8, D + D/4)    (scale, minimum) pairs of V
// Channels are quantised in groups of 32 with one bfloat16 pair per group; a code c in 0..15 stands
// for minimum + scale * c.  The eight codes of channels 8w .. 8w+7 fill one little-endian 32-bit word
// (channel 8w+i in bits 4i .. 4i+3), and word w is word number (w % 4) * (D/32) + w / 4 of its half.
// That order lets the attention kernel's lane t of a row read its words of every group (the four lanes
// of a row of a 16-row MMA tile take 8 channels of each group) with one wide load, and spreads the
// V words that one lane needs over 8 bytes.
#pragma once

#include "osf_internal.cuh"

namespace osf {

constexpr int kKv4Group = 32;

__host__ __device__ __forceinline__ int kv4_record_bytes(int D) { return D + D / 4; }
// Word number, within a half, of the codes of channels 8w .. 8w+7.
__host__ __device__ __forceinline__ int kv4_word_at(int D, int w) { return (w & 3) * (D / 32) + (w >> 2); }

struct Kv4StoreProblem {
    const void *k, *v;          // append: rows to store
    void *ko, *vo;              // read: rows to write
    unsigned char *cache;       // [B, Hkv, S, 1.25 D]
    const int *lens;            // append: tokens already there; read: tokens that are valid (nullable)
    const int *counts;          // append: new tokens of each sequence (nullable: n)
    const int *starts;          // read: first token of each sequence (nullable: 0)
    int dtype, B, Hkv, n, S, D;
    long long k_sb, k_sh, k_ss, v_sb, v_sh, v_ss;
    int *status;
};
cudaError_t launch_kv4_append(const Kv4StoreProblem &p, int sm_count, cudaStream_t s);
cudaError_t launch_kv4_read(const Kv4StoreProblem &p, int sm_count, cudaStream_t s);

// Attention over records: the AttnProblem's q, o, lse, sizes (Sk = records per sequence), strides and
// split workspace; k, v and their strides are unused, as is causal_off (the mask follows each length).
struct Kv4AttnProblem {
    AttnProblem a;
    const unsigned char *cache;
    const int *lens;            // nullable: every record is valid
    float *weights;             // nullable [B, Hkv, Sk]
    int accumulate;             // add to weights instead of overwriting them
    float *scores;              // with weights: base-2 scores [B * Hkv][G * Sq][Sk]
    float *part;                // tensor-core kernel: numerators of items that several CTAs share,
    float2 *part_ml;            //   and their maxima and denominators
};
// Bytes of partial states that the call keeps in `partials`.
size_t kv4_attn_partial_bytes(const Kv4AttnProblem &p, int sm_count);
cudaError_t launch_attn_kv4(const Kv4AttnProblem &p, void *partials, int sm_count, cudaStream_t s);

// Valid records of sequence b; a length outside [0, S] is cut to it and recorded in the status word.
__device__ __forceinline__ int kv4_length(const int *lens, int b, int S, int *status) {
    if (!lens) return S;
    const int n = lens[b];
    if (n < 0 || n > S) atomicExch(status, (int)OSF_ERR_INVALID);
    return min(max(n, 0), S);
}

}  // namespace osf
