// Storing rows in the 4-bit K/V cache and reading them back (format: kv4.cuh).
//
// Quantisation of a group of 32 channels x: m = the largest bfloat16 <= min x, s = the smallest
// bfloat16 >= (max x - m) / 15, code = round-half-even((x - m) / s).  Rounding m down and s up makes
// m .. m + 15 s cover the group, so no code is clamped and the error is at most s / 2.  All
// three are decided exactly, whatever float32 rounds on the way: x - m is kept as a float32 and its
// rounding error (Knuth's two-sum), and the comparisons that settle s and a code near a tie use
// 15 s and (c +- 1/2) s, which float32 holds exactly (8 significant bits times at most 5).
// A group with a NaN, an infinity or a range past float32 is stored as s = m = NaN: it reads back NaN.
//
// Both directions move bytes: 4 D + 1.25 D per bf16 token and kv head.  Four lanes share a group, eight
// channels each, so a warp reads 16-byte pieces (bf16) and writes one code word per lane; at D = 128
// the 32 lanes hold exactly one token, K in lanes 0-15 and V in lanes 16-31.
#include "kv4.cuh"

namespace osf {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float bf16_bits_to_f32(uint32_t b) { return __uint_as_float(b << 16); }

// Eight channels of a row as float32.
__device__ __forceinline__ void load8(const float *p, bool vec, float (&x)[8]) {
    if (vec) {
        const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = p[i];
    }
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, bool vec, float (&x)[8]) {
    if (vec) {
        const uint4 a = *reinterpret_cast<const uint4 *>(p);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __bfloat162float(p[i]);
    }
}
__device__ __forceinline__ void store8(float *p, bool vec, const float (&x)[8]) {
    if (vec) {
        *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<float4 *>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = x[i];
    }
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, bool vec, const float (&x)[8]) {
    if (vec) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = __float2bfloat16_rn(x[i]);
    }
}

// d + e = a - b exactly, d the float32 nearest to it.
__device__ __forceinline__ void diff_exact(float a, float b, float &d, float &e) {
    d = __fsub_rn(a, b);
    const float bb = __fsub_rn(a, d);
    e = __fadd_rn(__fsub_rn(a, __fadd_rn(d, bb)), __fsub_rn(bb, b));
}
// Sign of (d + e) - t, where d is the float32 nearest to d + e.
__device__ __forceinline__ int cmp_exact(float d, float e, float t) {
    if (d != t) return d > t ? 1 : -1;
    return e > 0.f ? 1 : e < 0.f ? -1 : 0;
}

// The largest bfloat16 <= x, as float32 (a NaN stays a NaN).
__device__ __forceinline__ float bf16_floor(float x) {
    const uint32_t u = __float_as_uint(x);
    if (!(u & 0xffffu) || x != x) return x;
    return __uint_as_float((u & 0xffff0000u) + ((u >> 31) ? 0x10000u : 0u));
}

// (scale, minimum) of a group with the smallest value lo and the largest hi.
__device__ __forceinline__ void group_scale(float lo, float hi, float &s, float &m) {
    m = __fadd_rn(bf16_floor(lo), 0.f);   // a minimum of -0 is stored as 0
    float d, e;
    diff_exact(hi, m, d, e);
    if (!(fabsf(d) <= 3.0e38f) || !(fabsf(m) <= 3.39e38f)) {
        s = m = __uint_as_float(0x7fc00000u);
        return;
    }
    // the float32 quotient is at most the wanted bfloat16, and above the one before it
    s = __uint_as_float(__float_as_uint(__fdiv_rn(d, 15.f)) & 0xffff0000u);
    if (cmp_exact(d, e, 15.f * s) > 0) s = __uint_as_float(__float_as_uint(s) + 0x10000u);
}

// Codes of eight channels as one word.
__device__ __forceinline__ uint32_t quantise8(const float (&x)[8], float s, float m) {
    if (!(s > 0.f)) return 0u;   // a constant group, or NaN
    // a scale whose reciprocal could overflow is lifted first
    const float up = s < 0x1p-100f ? 0x1p60f : 1.f;
    const float inv = __frcp_rn(s * up);
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float d = __fsub_rn(x[i], m);
        const float t = d * up * inv;   // within 2^-21 of (x - m) / s
        float c = rintf(t);
        if (fabsf(t - c) > 0.4999f) {   // near a tie: settle it exactly
            float e;
            diff_exact(x[i], m, d, e);
            c = floorf(t);   // the tie is at c + 1/2
            const int side = cmp_exact(d, e, (c + 0.5f) * s);
            if (side > 0 || (side == 0 && ((int)c & 1))) c += 1.f;
        }
        w |= (uint32_t)(int)c << (4 * i);
    }
    return w;
}

// One group of four lanes per (token, half, group of 32 channels): flat index over
// [token of (b, h)][K groups, V groups].
template <typename T>
__global__ void __launch_bounds__(kThreads)
kv4_append_kernel(const Kv4StoreProblem p, int k_vec, int v_vec) {
    const int gph = p.D / kKv4Group, per_token = 2 * gph;
    const long long per_head = (long long)p.n * per_token;
    const int bh = blockIdx.y, b = bh / p.Hkv, h = bh % p.Hkv;
    const int n_new = p.counts ? p.counts[b] : p.n;
    const int base = p.lens ? p.lens[b] : 0;
    // new tokens that fit: the rest is left out, and recorded
    const int fit = base < 0 ? 0 : (int)min((long long)min(n_new, p.n), (long long)p.S - base);
    if (blockIdx.x == 0 && threadIdx.x == 0 && (base < 0 || n_new < 0 || n_new > p.n || fit < n_new))
        atomicExch(p.status, (int)OSF_ERR_INVALID);
    const int R = kv4_record_bytes(p.D);
    const int t = threadIdx.x & 3;
    unsigned char *head = p.cache + (long long)bh * p.S * R;
    const long long live = (long long)max(fit, 0) * per_token;
    for (long long i0 = (long long)blockIdx.x * (kThreads / 4); i0 < per_head; i0 += (long long)gridDim.x * (kThreads / 4)) {
        if (i0 >= live) break;   // the whole block is done
        const long long i = i0 + (threadIdx.x >> 2);
        const bool on = i < live;
        const long long at = on ? i : live - 1;   // idle lanes repeat the last group: shuffles need them
        const int tok = (int)(at / per_token), r = (int)(at - (long long)tok * per_token);
        const int half = r >= gph, n = r - half * gph;
        const T *src = half ? static_cast<const T *>(p.v) + b * p.v_sb + h * p.v_sh + tok * p.v_ss
                            : static_cast<const T *>(p.k) + b * p.k_sb + h * p.k_sh + tok * p.k_ss;
        float x[8];
        load8(src + n * kKv4Group + 8 * t, half ? v_vec : k_vec, x);
        float lo = x[0], hi = x[0];
        bool bad = false;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            lo = fminf(lo, x[e]);
            hi = fmaxf(hi, x[e]);
            bad |= x[e] != x[e];
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
            hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
            bad |= __shfl_xor_sync(0xffffffffu, (int)bad, o) != 0;
        }
        if (bad) lo = __uint_as_float(0x7fc00000u);
        float s, m;
        group_scale(lo, hi, s, m);
        const uint32_t w = quantise8(x, s, m);
        if (!on) continue;
        unsigned char *rec = head + (long long)(base + tok) * R;
        reinterpret_cast<uint32_t *>(rec + half * (p.D / 2))[kv4_word_at(p.D, n * 4 + t)] = w;
        if (t == 0)
            reinterpret_cast<uint32_t *>(rec + p.D + half * (p.D / 8))[n] =
                (__float_as_uint(s) >> 16) | (__float_as_uint(m) & 0xffff0000u);
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
kv4_read_kernel(const Kv4StoreProblem p, int k_vec, int v_vec) {
    const int wph = p.D / 8, per_token = 2 * wph;
    const int bh = blockIdx.y, b = bh / p.Hkv;
    const int len = kv4_length(p.lens, b, p.S, p.status);
    const int start = p.starts ? p.starts[b] : 0;
    const int R = kv4_record_bytes(p.D);
    const unsigned char *head = p.cache + (long long)bh * p.S * R;
    T *ko = static_cast<T *>(p.ko) + (long long)bh * p.n * p.D, *vo = static_cast<T *>(p.vo) + (long long)bh * p.n * p.D;
    const long long total = (long long)p.n * per_token;
    for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < total; i += (long long)gridDim.x * kThreads) {
        const int tok = (int)(i / per_token), r = (int)(i - (long long)tok * per_token);
        const int half = r >= wph, w = r - half * wph;
        const long long pos = (long long)start + tok;
        float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (pos >= 0 && pos < len) {
            const unsigned char *rec = head + pos * R;
            const uint32_t c = reinterpret_cast<const uint32_t *>(rec + half * (p.D / 2))[kv4_word_at(p.D, w)];
            const uint32_t sm = reinterpret_cast<const uint32_t *>(rec + p.D + half * (p.D / 8))[w >> 2];
            const float s = bf16_bits_to_f32(sm & 0xffffu), m = __uint_as_float(sm & 0xffff0000u);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = fmaf((float)((c >> (4 * e)) & 15u), s, m);
        }
        store8((half ? vo : ko) + (long long)tok * p.D + 8 * w, half ? v_vec : k_vec, x);
    }
}

// Blocks along a head's work: enough to fill the GPU several times over all heads, none idle.
unsigned store_blocks(long long work, int heads, int sm_count) {
    long long want = ((long long)sm_count * 16 + heads - 1) / heads;
    want = want < work ? want : work;
    return (unsigned)(want < 1 ? 1 : want);
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4StoreProblem &p, int sm_count, cudaStream_t s) {
    const long long groups = (long long)p.n * 2 * (p.D / kKv4Group);
    const dim3 grid(store_blocks((groups + kThreads / 4 - 1) / (kThreads / 4), p.B * p.Hkv, sm_count), p.B * p.Hkv);
    const int es = p.dtype == OSF_F32 ? 4 : 2, unit = 16 / es;
    auto vec = [&](const void *q, long long a, long long b, long long c) {
        return (reinterpret_cast<uintptr_t>(q) & 15u) == 0 && ((a | b | c) % unit) == 0;
    };
    const int kvec = vec(p.k, p.k_sb, p.k_sh, p.k_ss), vvec = vec(p.v, p.v_sb, p.v_sh, p.v_ss);
    if (p.dtype == OSF_F32) kv4_append_kernel<float><<<grid, kThreads, 0, s>>>(p, kvec, vvec);
    else kv4_append_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(p, kvec, vvec);
    count_launches(1);
    return cudaGetLastError();
}

cudaError_t launch_kv4_read(const Kv4StoreProblem &p, int sm_count, cudaStream_t s) {
    const long long words = (long long)p.n * 2 * (p.D / 8);
    const dim3 grid(store_blocks((words + kThreads - 1) / kThreads, p.B * p.Hkv, sm_count), p.B * p.Hkv);
    const int kvec = (reinterpret_cast<uintptr_t>(p.ko) & 15u) == 0, vvec = (reinterpret_cast<uintptr_t>(p.vo) & 15u) == 0;
    if (p.dtype == OSF_F32) kv4_read_kernel<float><<<grid, kThreads, 0, s>>>(p, kvec, vvec);
    else kv4_read_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(p, kvec, vvec);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace osf
