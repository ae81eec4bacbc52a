// Storing rows in the paged 8-bit K/V cache, with the position rotation on the way, and reading them back (format:
// kv8.cuh).
//
// Appending: a block takes one page of one kv head, K or V.  K's rows are rotated: channels a, b of a pair by the angle of
// their position become a c - b s and b c + a s, rounded once to float32 (both products and their difference are kept with
// their rounding errors, so the codes are those of the formulas and not of some order of float32 operations).  The page's
// scale is 2^e with the least e for which its largest magnitude is at most 448 * 2^e; a page that holds earlier tokens
// keeps its scale unless the new ones need a larger one, and then the codes there are rounded again: e4m3 codes only
// change their exponent, so that is exact but for those that fall among the subnormals.  NaN and infinities are stored as
// NaN and leave the scale alone.
#include "kv8.cuh"
#include "sm100_ptx.cuh"

namespace osf {
namespace {

constexpr int kThreads = 256;
constexpr float kMaxF32 = 3.4028235e38f;

__device__ __forceinline__ float lo_bf16(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// Four neighbouring channels of a row.
__device__ __forceinline__ void load4(const float *p, bool vec, float *x) {
    if (vec) {
        const float4 v = *reinterpret_cast<const float4 *>(p);
        x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = p[i];
    }
}
__device__ __forceinline__ void load4(const __nv_bfloat16 *p, bool vec, float *x) {
    if (vec) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        x[0] = lo_bf16(v.x); x[1] = hi_bf16(v.x); x[2] = lo_bf16(v.y); x[3] = hi_bf16(v.y);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = __bfloat162float(p[i]);
    }
}
__device__ __forceinline__ void store4(float *p, bool vec, const float *x) {
    if (vec) {
        *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = x[i];
    }
}
__device__ __forceinline__ void store4(__nv_bfloat16 *p, bool vec, const float *x) {
    if (vec) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(ptx::pack_bf16x2(x[0], x[1]), ptx::pack_bf16x2(x[2], x[3]));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = __float2bfloat16_rn(x[i]);
    }
}

// The float32 nearest to a c - b s.
__device__ __forceinline__ float rotate1(float a, float c, float b, float s) {
    const float p = __fmul_rn(a, c), q = __fmul_rn(b, s);
    const float pe = __fmaf_rn(a, c, -p), qe = __fmaf_rn(b, s, -q);
    const float h = __fsub_rn(p, q), t = __fsub_rn(h, p);
    const float he = __fsub_rn(__fsub_rn(p, __fsub_rn(h, t)), __fadd_rn(q, t));   // h + he = p - q
    return fabsf(h) <= kMaxF32 ? __fadd_rn(h, __fadd_rn(he, __fsub_rn(pe, qe))) : h;
}

// Where the eight channels of unit u of a row lie: two runs of four, at first and second.
struct Unit {
    int first, second;
    bool rotated;
    int angle;   // of the four pairs: columns angle .. angle + 3 of the tables
};
__device__ __forceinline__ Unit unit_of(int u, int R, bool interleaved) {
    Unit w;
    w.rotated = 8 * u < R;
    w.angle = 4 * u;
    const bool halves = w.rotated && !interleaved;
    w.first = halves ? 4 * u : 8 * u;
    w.second = halves ? R / 2 + 4 * u : 8 * u + 4;
    return w;
}

// The eight channels of a unit of a row at position pos, rotated where they are to be.
template <typename T>
__device__ __forceinline__ void load_unit(const Kv8StoreProblem &p, const T *row, const Unit &w, int pos, bool vec, float (&x)[8]) {
    load4(row + w.first, vec, x);
    load4(row + w.second, vec, x + 4);
    if (!w.rotated) return;
    float c[4], s[4];
    const bool tv = ((reinterpret_cast<uintptr_t>(p.cos) | reinterpret_cast<uintptr_t>(p.sin)) & 15u) == 0 && p.R % 8 == 0;
    load4(p.cos + (long long)pos * (p.R / 2) + w.angle, tv, c);
    load4(p.sin + (long long)pos * (p.R / 2) + w.angle, tv, s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float &a = p.interleaved ? x[2 * i] : x[i], &b = p.interleaved ? x[2 * i + 1] : x[i + 4];
        const float ra = rotate1(a, c[i], b, s[i]), rb = rotate1(b, c[i], -a, s[i]);
        a = ra;
        b = rb;
    }
}

__device__ __forceinline__ uint32_t code4(const float *x, float inv) {
    uint32_t w = f32_to_e4m3x2(x[0] * inv, x[1] * inv) | f32_to_e4m3x2(x[2] * inv, x[3] * inv) << 16;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (!(fabsf(x[i]) <= kMaxF32)) w = (w & ~(0xffu << 8 * i)) | 0x7fu << 8 * i;
    return w;
}

// Blocks: [0, pages) x (b, kv head) x (K, V): the page-th page that new tokens of the sequence may fall into.
template <typename T>
__global__ void __launch_bounds__(kThreads)
kv8_append_kernel(const Kv8StoreProblem p, int k_vec, int v_vec) {
    __shared__ float sh_max[kThreads / 32];
    const Kv8Cache &c = p.c;
    const int D = c.D, P = c.P, units = D / 8;
    const int bh = blockIdx.y, b = bh / c.Hkv, h = bh % c.Hkv, half = blockIdx.z;
    const int n_new = p.counts ? p.counts[b] : p.n;
    const int base = p.lens ? p.lens[b] : 0, most = c.per_seq * P;
    // new tokens that fit: the rest is left out, and recorded
    const int fit = base < 0 ? 0 : (int)min((long long)min(n_new, p.n), (long long)most - base);
    if (blockIdx.x == 0 && h == 0 && half == 0 && threadIdx.x == 0) {
        if (base < 0 || n_new < 0 || n_new > p.n || fit < n_new) atomicExch(p.status, (int)OSF_ERR_INVALID);
        if (p.R && fit > 0 && base + fit > p.max_pos) atomicExch(p.status, (int)OSF_ERR_INVALID);
    }
    if (fit <= 0) return;
    const int first = (base / P + blockIdx.x) * P;        // first token of the page
    if (first >= base + fit) return;
    const int t0 = max(base, first), t1 = min(base + fit, first + P);   // its new tokens
    const int page = kv8_page(c, b, first, p.status);
    if (page < 0) return;
    const T *rows = half ? static_cast<const T *>(p.v) + b * p.v_sb + h * p.v_sh
                         : static_cast<const T *>(p.k) + b * p.k_sb + h * p.k_sh;
    const long long ss = half ? p.v_ss : p.k_ss;
    const bool vec = half ? v_vec : k_vec;
    const int R = half ? 0 : p.R;
    const long long at = ((long long)page * 2 + half) * c.Hkv + h;
    unsigned char *codes = c.pages + at * P * D;
    const int work = (t1 - t0) * units;
    float x[8], mx = 0.f;
    for (int i = threadIdx.x; i < work; i += blockDim.x) {
        const int tok = t0 + i / units;
        load_unit(p, rows + (tok - base) * ss, unit_of(i % units, R, p.interleaved), min(tok, p.max_pos - 1), vec, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float a = fabsf(x[e]);
            mx = a <= kMaxF32 ? fmaxf(mx, a) : mx;
        }
    }
    mx = warp_max(mx);
    if ((threadIdx.x & 31) == 0) sh_max[threadIdx.x >> 5] = mx;
    const float old_scale = c.scales[at];
    __syncthreads();
    for (int w = 0; w < (int)blockDim.x / 32; ++w) mx = fmaxf(mx, sh_max[w]);
    // mx = (1 + m / 2^23) 2^x: the least e with mx <= 1.75 * 2^(8 + e)
    const uint32_t bits = __float_as_uint(mx);
    int e = max((int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0), kKv8MinExp);
    if (t0 > first) {   // earlier tokens: the scale only grows, and their codes follow it
        const int old = kv8_exponent(old_scale);
        if (e > old) {
            const float f = pow2_of(max(old - e, -126));
            const int words = (t0 - first) * D / 4;
            for (int i = threadIdx.x; i < words; i += blockDim.x) {
                uint32_t *w = reinterpret_cast<uint32_t *>(codes) + i;
                const float2 lo = e4m3x2_to_f32(*w), hi = e4m3x2_to_f32(*w >> 16);
                *w = f32_to_e4m3x2(lo.x * f, lo.y * f) | f32_to_e4m3x2(hi.x * f, hi.y * f) << 16;
            }
        }
        e = max(e, old);
    }
    const float inv = pow2_of(-e);
    for (int i = threadIdx.x; i < work; i += blockDim.x) {
        const int tok = t0 + i / units;
        const Unit w = unit_of(i % units, R, p.interleaved);
        load_unit(p, rows + (tok - base) * ss, w, min(tok, p.max_pos - 1), vec, x);
        unsigned char *row = codes + (long long)(tok - first) * D;
        *reinterpret_cast<uint32_t *>(row + w.first) = code4(x, inv);
        *reinterpret_cast<uint32_t *>(row + w.second) = code4(x + 4, inv);
    }
    if (threadIdx.x == 0) c.scales[at] = pow2_of(e);
}

// The queries of the new tokens, rotated.  A thread takes a unit of a row.
template <typename T>
__global__ void __launch_bounds__(kThreads)
kv8_rotate_kernel(const Kv8StoreProblem p, int q_vec, int o_vec) {
    const int units = p.c.D / 8;
    const int bh = blockIdx.y, b = bh / p.Hq, h = bh % p.Hq;
    const int count = min(p.counts ? p.counts[b] : p.n, p.n), base = p.lens ? p.lens[b] : 0;
    const T *src = static_cast<const T *>(p.q) + b * p.q_sb + h * p.q_sh;
    T *dst = static_cast<T *>(p.qo) + b * p.o_sb + h * p.o_sh;
    for (int i = blockIdx.x * kThreads + threadIdx.x; i < count * units; i += gridDim.x * kThreads) {
        const int t = i / units;
        const Unit w = unit_of(i % units, p.R, p.interleaved);
        float x[8];
        load_unit(p, src + t * p.q_ss, w, min(max(base + t, 0), p.max_pos - 1), q_vec, x);
        store4(dst + t * p.o_ss + w.first, o_vec, x);
        store4(dst + t * p.o_ss + w.second, o_vec, x + 4);
    }
}

// A thread takes 16 channels of a token.
template <typename T>
__global__ void __launch_bounds__(kThreads)
kv8_read_kernel(const Kv8StoreProblem p, int k_vec, int v_vec) {
    const Kv8Cache &c = p.c;
    const int D = c.D, per = D / 16;
    const int bh = blockIdx.y, b = bh / c.Hkv, h = bh % c.Hkv, half = blockIdx.z;
    const int len = kv8_length(p.lens, b, c.per_seq * c.P, p.status), start = p.starts ? p.starts[b] : 0;
    T *out = static_cast<T *>(half ? p.vo : p.ko) + (long long)bh * p.n * D;
    const bool vec = half ? v_vec : k_vec;
    for (int i = blockIdx.x * kThreads + threadIdx.x; i < p.n * per; i += gridDim.x * kThreads) {
        const int t = i / per, ch = i % per * 16;
        const long long pos = (long long)start + t;
        const int page = pos >= 0 && pos < len ? kv8_page(c, b, (int)pos, p.status) : -1;
        uint4 w = make_uint4(0, 0, 0, 0);
        float scale = 0.f;
        if (page >= 0) {
            const long long at = ((long long)page * 2 + half) * c.Hkv + h;
            w = *reinterpret_cast<const uint4 *>(c.pages + (at * c.P + pos % c.P) * D + ch);
            scale = pow2_of(kv8_exponent(c.scales[at]));
        }
        const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 lo = e4m3x2_to_f32(v[e]), hi = e4m3x2_to_f32(v[e] >> 16);
            const float x[4] = {lo.x * scale, lo.y * scale, hi.x * scale, hi.y * scale};
            store4(out + (long long)t * D + ch + 4 * e, vec, x);
        }
    }
}

bool rows_vec(const void *q, long long a, long long b, long long c, int es) {
    const int unit = 4 * es;   // four channels
    return (reinterpret_cast<uintptr_t>(q) % unit) == 0 && (a | b | c) % 4 == 0;
}

template <typename T>
cudaError_t append_t(const Kv8StoreProblem &p, int sm_count, cudaStream_t s) {
    const Kv8Cache &c = p.c;
    const int es = sizeof(T);
    const long long pages = ((long long)p.n + 2 * c.P - 2) / c.P;
    const int tokens = p.n < c.P ? p.n : c.P, want = (tokens * (c.D / 8) + 31) / 32 * 32;
    const dim3 grid((unsigned)(pages < c.per_seq ? pages : c.per_seq), (unsigned)(p.B * c.Hkv), 2);
    kv8_append_kernel<T><<<grid, want < kThreads ? want : kThreads, 0, s>>>(
        p, rows_vec(p.k, p.k_sb, p.k_sh, p.k_ss, es), rows_vec(p.v, p.v_sb, p.v_sh, p.v_ss, es));
    count_launches(1);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !p.q) return e;
    const long long work = ((long long)p.n * (c.D / 8) + kThreads - 1) / kThreads;
    const long long most = (16LL * sm_count + p.B * p.Hq - 1) / (p.B * p.Hq);
    const dim3 gq((unsigned)(work < most ? work : most), (unsigned)(p.B * p.Hq));
    kv8_rotate_kernel<T><<<gq, kThreads, 0, s>>>(p, rows_vec(p.q, p.q_sb, p.q_sh, p.q_ss, es),
                                                 rows_vec(p.qo, p.o_sb, p.o_sh, p.o_ss, es));
    count_launches(1);
    return cudaGetLastError();
}

template <typename T>
cudaError_t read_t(const Kv8StoreProblem &p, int sm_count, cudaStream_t s) {
    const Kv8Cache &c = p.c;
    const long long work = ((long long)p.n * (c.D / 16) + kThreads - 1) / kThreads;
    const long long most = (16LL * sm_count + p.B * c.Hkv * 2 - 1) / (p.B * c.Hkv * 2);
    const dim3 grid((unsigned)(work < most ? work : most), (unsigned)(p.B * c.Hkv), 2);
    kv8_read_kernel<T><<<grid, kThreads, 0, s>>>(p, rows_vec(p.ko, 0, 0, 0, sizeof(T)), rows_vec(p.vo, 0, 0, 0, sizeof(T)));
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv8_append(const Kv8StoreProblem &p, int sm_count, cudaStream_t s) {
    return p.dtype == OSF_F32 ? append_t<float>(p, sm_count, s) : append_t<__nv_bfloat16>(p, sm_count, s);
}
cudaError_t launch_kv8_read(const Kv8StoreProblem &p, int sm_count, cudaStream_t s) {
    return p.dtype == OSF_F32 ? read_t<float>(p, sm_count, s) : read_t<__nv_bfloat16>(p, sm_count, s);
}

}  // namespace osf
