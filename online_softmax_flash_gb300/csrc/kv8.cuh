// The paged 8-bit K/V cache: format, problem descriptions and launchers.
//
// pages [n_pages][2][Hkv][P][D]: e4m3 codes (K, then V) of P tokens, a token's D channels in a row; P 16, 32, 64 or 128.
// scales [n_pages][2][Hkv]: float32 powers of two.  A value is code * scale.
// table [B][per_seq]: page of tokens P i .. P i + P - 1 of a sequence.
#pragma once

#include "osf_internal.cuh"

namespace osf {

constexpr int kKv8MinExp = -110;   // smallest exponent of a scale: the smallest code times it stays a normal bfloat16

struct Kv8Cache {
    unsigned char *pages;
    float *scales;
    const int *table;
    int n_pages, P, log2_p, per_seq, Hkv, D;
};

struct Kv8StoreProblem {
    Kv8Cache c;
    const void *k, *v, *q;      // append: rows to store, and queries to rotate (nullable)
    void *qo;
    void *ko, *vo;              // read: rows to write
    const int *lens;            // append: tokens already there (nullable: 0); read: tokens that are valid (nullable: all)
    const int *counts;          // append: new tokens of each sequence (nullable: n)
    const int *starts;          // read: first token of each sequence (nullable: 0)
    const float *cos, *sin;     // [max_pos][R / 2], or null
    int max_pos, R, interleaved;
    unsigned units_inv;         // for divisions by the units of a row
    int units_shift;
    int table_vec;              // the tables' rows can be read 16 bytes at a time
    int dtype, B, Hq, n;
    long long k_sb, k_sh, k_ss, v_sb, v_sh, v_ss, q_sb, q_sh, q_ss, o_sb, o_sh, o_ss;
    int *status;
};
cudaError_t launch_kv8_append(const Kv8StoreProblem &p, int sm_count, cudaStream_t s);
cudaError_t launch_kv8_read(const Kv8StoreProblem &p, int sm_count, cudaStream_t s);

// Attention over pages: the AttnProblem's q, o, lse, sizes (Sk = per_seq * P), strides, window (0: none) and sinks, and
// split workspace; the rows of a sequence are its last Sq tokens.
struct Kv8AttnProblem {
    AttnProblem a;
    Kv8Cache c;
    const int *lens;            // nullable: every slot of the table is valid
    float *part;                // tensor-core kernel: numerators of items that several CTAs share,
    float2 *part_ml;            //   and their maxima and denominators
};
size_t kv8_attn_partial_bytes(const Kv8AttnProblem &p, int sm_count);
cudaError_t launch_attn_kv8(const Kv8AttnProblem &p, void *partials, int sm_count, cudaStream_t s);

// Valid tokens of sequence b; a length outside [0, most] is cut to it and recorded in the status word.
__device__ __forceinline__ int kv8_length(const int *lens, int b, int most, int *status) {
    if (!lens) return most;
    const int n = lens[b];
    if (n < 0 || n > most) atomicExch(status, (int)OSF_ERR_INVALID);
    return min(max(n, 0), most);
}
// Page of token `tok` (within the table) of sequence b; -1, recorded, where the table holds no page of the cache.  In two
// steps, so that an entry can be on its way while others are worked with.
__device__ __forceinline__ int kv8_entry(const Kv8Cache &c, int b, int tok) {
    return c.table[(long long)b * c.per_seq + (tok >> c.log2_p)];
}
__device__ __forceinline__ int kv8_checked(const Kv8Cache &c, int entry, int *status) {
    if (entry >= 0 && entry < c.n_pages) return entry;
    atomicExch(status, (int)OSF_ERR_INVALID);
    return -1;
}
__device__ __forceinline__ int kv8_page(const Kv8Cache &c, int b, int tok, int *status) {
    return kv8_checked(c, kv8_entry(c, b, tok), status);
}
// Exponent of a scale (one that is no power of two counts as the next below), and the power of two of an exponent.
__device__ __forceinline__ int kv8_exponent(float scale) {
    return min(max((int)(__float_as_uint(scale) >> 23 & 255u) - 127, kKv8MinExp), 120);
}
__device__ __forceinline__ float pow2_of(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Two e4m3 codes (low byte first) as float32, and two float32 (|x| <= 448) as e4m3 codes, to the nearest, ties to even.
__device__ __forceinline__ float2 e4m3x2_to_f32(uint32_t codes) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)codes));
    float2 r;
    asm("{\n .reg .b16 l, u;\n mov.b32 {l, u}, %2;\n cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, u;\n}"
        : "=f"(r.x), "=f"(r.y)
        : "r"(h));
    return r;
}
__device__ __forceinline__ uint32_t f32_to_e4m3x2(float lo, float hi) {
    unsigned short r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two float16 as e5m2 codes (low byte first), to the nearest, ties to even, and back: the upper bytes of float16.
__device__ __forceinline__ uint32_t f16x2_to_e5m2x2(uint32_t h) {
    unsigned short r;
    asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
    return r;
}
__device__ __forceinline__ uint32_t e5m2x2_to_f16x2(uint32_t codes) { return __byte_perm(codes, 0, 0x1404); }
__device__ __forceinline__ uint32_t f16x2_min(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t f32_to_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// (a - b) f of float16 pairs, exact where a - b is and f a power of two.
__device__ __forceinline__ uint32_t f16x2_rest(uint32_t a, uint32_t b, uint32_t f) {
    uint32_t r;
    asm("{\n .reg .b32 t;\n sub.rn.f16x2 t, %1, %2;\n mul.rn.f16x2 %0, t, %3;\n}" : "=r"(r) : "r"(a), "r"(b), "r"(f));
    return r;
}

}  // namespace osf
