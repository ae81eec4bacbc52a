// Storing rows in the 4-bit K/V cache and reading them back (format: kv4.cuh).
//
// Quantisation of a group of 32 channels x: m = the largest bfloat16 <= min x, s = the smallest
// bfloat16 >= (max x - m) / 15, code = round-half-even((x - m) / s).  Rounding m down and s up makes
// m .. m + 15 s cover the group, so no code is clamped and the error is at most s / 2.  All
// three are decided exactly, whatever float32 rounds on the way: x - m is kept as a float32 and its
// rounding error (Knuth's two-sum), and the comparisons that settle s and a code near a tie use
// 15 s and (c +- 1/2) s, which float32 holds exactly (8 significant bits times at most 5).
// A group with a NaN, an infinity or a value below the least finite bfloat16 (m would be -inf) is stored as s = m = NaN: it
// reads back NaN.  Ranges near float32's end, or past it, are worked out in halves.
//
// Both directions move bytes: 4 D + 1.25 D per bf16 token and kv head.  Two lanes share a group when storing, sixteen
// channels (a 32-byte sector of bf16) each, with the next token's row in flight; that leaves 16 instructions
// per channel, and takes 43 us for the 176 MB of B=8 Hkv=8 n=4096 D=128 bf16, bound by their issue (26 us at the copy's
// rate).
// Reading back writes the same bytes at 6.4 TB/s, 27.5 us.  (Storing with four lanes to a group, eight channels
// each, in scalar float32: 68 us.)
#include "kv4.cuh"
#include "sm100_ptx.cuh"

namespace osf {
namespace {

constexpr int kThreads = 256;

// The two bfloat16 of a word as float32.
__device__ __forceinline__ float lo_bf16(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// Eight channels of a row from float32.
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

// Smallest and largest of three, a NaN among them giving a NaN.
__device__ __forceinline__ float min3_nan(float a, float b, float c) {
    float d;
    asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// (scale, minimum) of a group whose largest value is hi and whose minimum, a bfloat16, is m.
constexpr float kMaxF32 = 3.4028235e38f;
__device__ __forceinline__ void group_scale(float hi, float &s, float &m) {
    m = __fadd_rn(m, 0.f);   // a minimum of -0 is stored as 0
    float d, e, unit = 1.f;
    diff_exact(hi, m, d, e);
    if (!(fabsf(d) <= 3.0e38f)) {   // 15 s could overflow, or hi - m did: in halves (of e the sign is enough)
        if (!(fabsf(hi) <= kMaxF32 && fabsf(m) <= kMaxF32)) {
            s = m = __uint_as_float(0x7fc00000u);
            return;
        }
        if (fabsf(d) <= kMaxF32) d *= 0.5f;
        else diff_exact(0.5f * hi, 0.5f * m, d, e);   // (both far from the subnormals, so exact)
        unit = 2.f;
    }
    // 0x1.11111p-4 is below 1/15 by 2^-22: the truncated product is the wanted bfloat16, the first with
    // 15 s >= d + e, or at most two below it
    uint32_t u = __float_as_uint(d * 0x1.11111p-4f) & 0xffff0000u;
    if (cmp_exact(d, e, 15.f * __uint_as_float(u)) > 0) u += 0x10000u;
    if (cmp_exact(d, e, 15.f * __uint_as_float(u)) > 0) u += 0x10000u;
    s = __uint_as_float(u) * unit;
}

// Codes of eight channels as one word.  t + 1.5 * 2^23 has the rounded t in its low bits, so a code needs no
// conversion: the eight sums of those bits times 16^i make the word and a constant.
constexpr float kMagic = 12582912.f;   // 0x4b400000
__device__ __forceinline__ uint32_t word_of(const float (&r)[8]) {
    uint32_t w = 0u - 0x4b400000u * 0x11111111u, place = 1u;
#pragma unroll
    for (int i = 0; i < 8; ++i, place <<= 4) w += __float_as_uint(r[i]) * place;
    return w;
}

// Any group.  t is off by up to 2^-20; what is left over, (x - m) - code * s, is exact, and only where it
// reaches s / 2 is the code looked at again.  From kWideScale on, where x - m may overflow, all in halves.
constexpr float kWideScale = 0x1p123f;
__device__ __noinline__ uint32_t quantise8_any(float x0, float x1, float x2, float x3, float x4, float x5, float x6, float x7,
                                               float s, float m) {
    const float x[8] = {x0, x1, x2, x3, x4, x5, x6, x7};
    const float h = s >= kWideScale ? 0.5f : 1.f, sh = s * h, mh = m * h;
    const float up = s < 0x1p-100f ? 0x1p60f : 1.f;   // a reciprocal that could overflow: lifted first
    const float inv = rcp_approx(sh * up), half = 0.5f * sh;
    float r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float d = fmaf(x[i], h, -mh), e;
        r[i] = __fadd_rn(d * up * inv, kMagic);
        const float c = __fsub_rn(r[i], kMagic), rest = fmaf(-c, sh, d);
        if (fabsf(rest) >= half) {
            diff_exact(x[i], m, d, e);
            if (!(fabsf(d) <= kMaxF32)) diff_exact(x[i] * h, mh, d, e);   // (of e the sign is enough)
            // at the tie (rest = +- s / 2) the side is that of e, or the even code; past it the neighbour
            const float over = fabsf(rest) > half ? 1.f : rest > 0.f ? e : -e;
            if (over > 0.f || (over == 0.f && ((int)c & 1))) r[i] += rest > 0.f ? 1.f : -1.f;
        }
    }
    return word_of(r);
}

// A group of bfloat16 values of which, with m, every one that is not 0 is at least 2^-11 s in magnitude: they are
// multiples of 2^-19 s, so x - m (< 16 s) is exact, and (x - m) / s is a tie or at least 2^-20 off one.  The
// correctly rounded quotient (a product with the rounded reciprocal and one remainder step, Markstein) then rounds to
// the right code, ties to even among them, which bfloat16's coarse grid makes common: one code in some hundred.
// v: four pairs of channels.  Packed float32 pairs: half the instructions.
__device__ __forceinline__ uint32_t quantise8_coarse(const uint32_t *v, float s, float m, float inv) {
    const uint64_t ns2 = ptx::f2_pack(-s, -s), nm2 = ptx::f2_pack(-m, -m), inv2 = ptx::f2_pack(inv, inv);
    const uint64_t magic2 = ptx::f2_pack(kMagic, kMagic);
    float r[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint64_t d = ptx::f2_add(ptx::f2_pack(lo_bf16(v[i]), hi_bf16(v[i])), nm2), t = ptx::f2_mul(d, inv2);
        ptx::f2_unpack(ptx::f2_add(ptx::f2_fma(ptx::f2_fma(t, ns2, d), inv2, t), magic2), r[2 * i], r[2 * i + 1]);
    }
    return word_of(r);
}

__device__ __forceinline__ uint32_t min_nan_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t min_s16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("min.s16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Sixteen channels of a row, half a group; the other half is the neighbouring lane's.  `range` gives the group's
// minimum, rounded down to a bfloat16, and its largest value (NaN if it has one); `codes` the channels' two words.
template <typename T>
struct Half;

template <>
struct Half<float> {
    float x[16];
    __device__ __forceinline__ void load(const float *p, bool vec) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (vec) {
                const float4 a = *reinterpret_cast<const float4 *>(p + 4 * i);
                x[4 * i] = a.x; x[4 * i + 1] = a.y; x[4 * i + 2] = a.z; x[4 * i + 3] = a.w;
            } else {
                x[4 * i] = p[4 * i]; x[4 * i + 1] = p[4 * i + 1]; x[4 * i + 2] = p[4 * i + 2]; x[4 * i + 3] = p[4 * i + 3];
            }
        }
    }
    __device__ __forceinline__ void range(float &m, float &hi) const {
        float lo = x[0];
        hi = x[0];
#pragma unroll
        for (int i = 1; i < 16; i += 2) {
            lo = min3_nan(lo, x[i], x[min(i + 1, 15)]);
            hi = max3_nan(hi, x[i], x[min(i + 1, 15)]);
        }
        lo = min3_nan(lo, lo, __shfl_xor_sync(0xffffffffu, lo, 1));
        hi = max3_nan(hi, hi, __shfl_xor_sync(0xffffffffu, hi, 1));
        m = bf16_floor(lo);
    }
    __device__ __forceinline__ void codes(float s, float m, uint32_t &a, uint32_t &b) const {
        a = quantise8_any(x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7], s, m);
        b = quantise8_any(x[8], x[9], x[10], x[11], x[12], x[13], x[14], x[15], s, m);
    }
};

template <>
struct Half<__nv_bfloat16> {
    uint32_t v[8];   // two channels each
    __device__ __forceinline__ void load(const __nv_bfloat16 *p, bool vec) {
        if (vec) {
            const uint4 a = *reinterpret_cast<const uint4 *>(p), b = *reinterpret_cast<const uint4 *>(p + 8);
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        } else {
            const unsigned short *h = reinterpret_cast<const unsigned short *>(p);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = h[2 * i] | (uint32_t)h[2 * i + 1] << 16;
        }
    }
    __device__ __forceinline__ void range(float &m, float &hi) const {
        uint32_t a = v[0], b = v[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) {
            a = min_nan_bf16x2(a, v[i]);
            b = max_nan_bf16x2(b, v[i]);
        }
        b ^= 0x80008000u;   // minima of -x: one pair (smallest, -largest) holds both from here on
        uint32_t r = min_nan_bf16x2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
        r = min_nan_bf16x2(r, __shfl_xor_sync(0xffffffffu, r, 1));
        m = lo_bf16(r);
        hi = -hi_bf16(r);
    }
    __device__ __forceinline__ void codes(float s, float m, uint32_t &a, uint32_t &b) const {
        // |x| - 1 of the smallest that is not 0, as 16 bits (0 wraps to the largest): magnitudes ordered by setting
        // the sign bit first, so that the subtraction does not borrow across halves
        uint32_t w = (v[0] | 0x80008000u) - 0x00010001u;
#pragma unroll
        for (int i = 1; i < 8; ++i) w = min_s16x2(w, (v[i] | 0x80008000u) - 0x00010001u);
        const int least = min((int)(short)w, (int)w >> 16) + 0x8000;
        const int bound = (int)(__float_as_uint(s) >> 16) - (11 << 7);   // 2^-11 s as a bfloat16's bits
        if (least >= bound - 1 && (m == 0.f || fabsf(m) >= 0x1p-11f * s) && s >= 0x1p-80f && s < kWideScale) {
            const float inv = __frcp_rn(s);
            a = quantise8_coarse(v, s, m, inv);
            b = quantise8_coarse(v + 4, s, m, inv);
        } else {
            a = quantise8_any(lo_bf16(v[0]), hi_bf16(v[0]), lo_bf16(v[1]), hi_bf16(v[1]), lo_bf16(v[2]), hi_bf16(v[2]),
                              lo_bf16(v[3]), hi_bf16(v[3]), s, m);
            b = quantise8_any(lo_bf16(v[4]), hi_bf16(v[4]), lo_bf16(v[5]), hi_bf16(v[5]), lo_bf16(v[6]), hi_bf16(v[6]),
                              lo_bf16(v[7]), hi_bf16(v[7]), s, m);
        }
    }
};

// Groups of a token, K's and then V's, lie along neighbouring lane pairs; a block takes the tokens that fit its
// threads, and a thread keeps its group.  DC: the head dimension where the compiler is to know it, or 0.
__host__ __device__ __forceinline__ int append_tokens(int D) { return kThreads / 2 / (2 * (D / kKv4Group)); }

template <typename T, int DC>
__global__ void __launch_bounds__(kThreads)
kv4_append_kernel(const Kv4StoreProblem p, int k_vec, int v_vec) {
    const int D = DC ? DC : p.D;
    const int NG = D / kKv4Group, tokens = append_tokens(D);
    const int bh = blockIdx.y, b = bh / p.Hkv, h = bh % p.Hkv;
    const int n_new = p.counts ? p.counts[b] : p.n;
    const int base = p.lens ? p.lens[b] : 0;
    // new tokens that fit: the rest is left out, and recorded
    const int fit = base < 0 ? 0 : (int)min((long long)min(n_new, p.n), (long long)p.S - base);
    if (blockIdx.x == 0 && threadIdx.x == 0 && (base < 0 || n_new < 0 || n_new > p.n || fit < n_new))
        atomicExch(p.status, (int)OSF_ERR_INVALID);
    if (fit <= 0) return;
    const int R = kv4_record_bytes(D);
    const int u = threadIdx.x & 1, unit = threadIdx.x >> 1;
    const int tl = unit / (2 * NG), group = unit % (2 * NG);
    const bool v_side = group >= NG;
    const int n = v_side ? group - NG : group;
    const T *rows = (v_side ? static_cast<const T *>(p.v) + b * p.v_sb + h * p.v_sh
                            : static_cast<const T *>(p.k) + b * p.k_sb + h * p.k_sh) + n * kKv4Group + 16 * u;
    const long long ss = v_side ? p.v_ss : p.k_ss;
    const bool vec = v_side ? v_vec : k_vec;
    unsigned char *head = p.cache + ((long long)bh * p.S + base) * R + (v_side ? D / 2 : 0) + 4 * kv4_word_at(D, n * 4 + 2 * u);
    unsigned char *pair = p.cache + ((long long)bh * p.S + base) * R + D + (v_side ? D / 8 : 0) + 4 * n;
    const int step = gridDim.x * tokens;
    // idle lanes repeat the last token: shuffles need them
    auto token = [&](int t0) { return min(t0 + tl, fit - 1); };
    Half<T> next;
    next.load(rows + token(blockIdx.x * tokens) * ss, vec);
    for (int t0 = blockIdx.x * tokens; t0 < fit; t0 += step) {
        const bool on = tl < tokens && t0 + tl < fit;
        const int tok = token(t0);
        const Half<T> x = next;
        if (t0 < fit - step) next.load(rows + token(t0 + step) * ss, vec);
        float s, m, hi;
        x.range(m, hi);
        group_scale(hi, s, m);
        uint32_t w0 = 0, w1 = 0;   // a constant group, or NaN
        if (s > 0.f) x.codes(s, m, w0, w1);
        if (!on) continue;
        unsigned char *rec = head + (long long)tok * R;
        *reinterpret_cast<uint32_t *>(rec) = w0;
        *reinterpret_cast<uint32_t *>(rec + 4 * NG) = w1;
        if (u == 0)
            *reinterpret_cast<uint32_t *>(pair + (long long)tok * R) =
                (__float_as_uint(s) >> 16) | (__float_as_uint(m) & 0xffff0000u);
    }
}

// A thread takes one word (8 channels) of four tokens: their loads are in flight together.
constexpr int kReadTokens = 4;
template <typename T, int DC>
__global__ void __launch_bounds__(kThreads)
kv4_read_kernel(const Kv4StoreProblem p, int k_vec, int v_vec) {
    const int D = DC ? DC : p.D;
    const unsigned wph = D / 8, per_token = 2 * wph;
    const int bh = blockIdx.y, b = bh / p.Hkv;
    const int len = kv4_length(p.lens, b, p.S, p.status);
    const int start = p.starts ? p.starts[b] : 0;
    const int R = kv4_record_bytes(D);
    const unsigned char *head = p.cache + (long long)bh * p.S * R;
    T *ko = static_cast<T *>(p.ko) + (long long)bh * p.n * D, *vo = static_cast<T *>(p.vo) + (long long)bh * p.n * D;
    const unsigned quads = (unsigned)(p.n + kReadTokens - 1) / kReadTokens, total = quads * per_token;   // n * D < 2^31
    for (unsigned i = blockIdx.x * kThreads + threadIdx.x; i < total; i += gridDim.x * kThreads) {
        const unsigned quad = i / per_token, r = i - quad * per_token;
        const bool half = r >= wph;
        const unsigned w = half ? r - wph : r;
        const unsigned code_at = (half ? D / 2 : 0) + 4 * kv4_word_at(D, w), pair_at = D + (half ? D / 8 : 0) + (w >> 2) * 4;
        uint32_t c[kReadTokens], sm[kReadTokens];
#pragma unroll
        for (int e = 0; e < kReadTokens; ++e) {
            const long long pos = (long long)start + quad * kReadTokens + e;
            c[e] = sm[e] = 0;   // scale and minimum 0: the value 0
            if (pos >= 0 && pos < len) {
                const unsigned char *rec = head + pos * R;
                c[e] = *reinterpret_cast<const uint32_t *>(rec + code_at);
                sm[e] = *reinterpret_cast<const uint32_t *>(rec + pair_at);
            }
        }
#pragma unroll
        for (int e = 0; e < kReadTokens; ++e) {
            const unsigned tok = quad * kReadTokens + e;
            if (tok >= (unsigned)p.n) break;
            const float s = lo_bf16(sm[e]), m = hi_bf16(sm[e]);
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = fmaf((float)((c[e] >> (4 * j)) & 15u), s, m);
            store8((half ? vo : ko) + (long long)tok * D + 8 * w, half ? v_vec : k_vec, x);
        }
    }
}

// Blocks along a head's work: `per_sm` for every SM over all heads, none idle.
unsigned store_blocks(long long work, int heads, int sm_count, int per_sm) {
    long long want = ((long long)sm_count * per_sm + heads - 1) / heads;
    want = want < work ? want : work;
    return (unsigned)(want < 1 ? 1 : want);
}

}  // namespace

template <typename T>
static cudaError_t append_t(const Kv4StoreProblem &p, dim3 grid, int kvec, int vvec, cudaStream_t s) {
    auto kernel = p.D == 128 ? kv4_append_kernel<T, 128> : p.D == 64 ? kv4_append_kernel<T, 64> : kv4_append_kernel<T, 0>;
    kernel<<<grid, kThreads, 0, s>>>(p, kvec, vvec);
    count_launches(1);
    return cudaGetLastError();
}

template <typename T>
static cudaError_t read_t(const Kv4StoreProblem &p, dim3 grid, int kvec, int vvec, cudaStream_t s) {
    auto kernel = p.D == 128 ? kv4_read_kernel<T, 128> : p.D == 64 ? kv4_read_kernel<T, 64> : kv4_read_kernel<T, 0>;
    kernel<<<grid, kThreads, 0, s>>>(p, kvec, vvec);
    count_launches(1);
    return cudaGetLastError();
}

cudaError_t launch_kv4_append(const Kv4StoreProblem &p, int sm_count, cudaStream_t s) {
    const int tokens = append_tokens(p.D);
    // (with 3, 5, 8, 16 and 32 blocks to an SM the prompt of the top and its reading back: 76, 84, 73, 74 and 77 us)
    const dim3 grid(store_blocks(((long long)p.n + tokens - 1) / tokens, p.B * p.Hkv, sm_count, 8), p.B * p.Hkv);
    const int es = p.dtype == OSF_F32 ? 4 : 2, unit = 16 / es;
    auto vec = [&](const void *q, long long a, long long b, long long c) {
        return (reinterpret_cast<uintptr_t>(q) & 15u) == 0 && ((a | b | c) % unit) == 0;
    };
    const int kvec = vec(p.k, p.k_sb, p.k_sh, p.k_ss), vvec = vec(p.v, p.v_sb, p.v_sh, p.v_ss);
    return p.dtype == OSF_F32 ? append_t<float>(p, grid, kvec, vvec, s) : append_t<__nv_bfloat16>(p, grid, kvec, vvec, s);
}

cudaError_t launch_kv4_read(const Kv4StoreProblem &p, int sm_count, cudaStream_t s) {
    const long long words = (long long)((p.n + kReadTokens - 1) / kReadTokens) * 2 * (p.D / 8);
    const dim3 grid(store_blocks((words + kThreads - 1) / kThreads, p.B * p.Hkv, sm_count, 16), p.B * p.Hkv);
    const int kvec = (reinterpret_cast<uintptr_t>(p.ko) & 15u) == 0, vvec = (reinterpret_cast<uintptr_t>(p.vo) & 15u) == 0;
    return p.dtype == OSF_F32 ? read_t<float>(p, grid, kvec, vvec, s) : read_t<__nv_bfloat16>(p, grid, kvec, vvec, s);
}

}  // namespace osf
