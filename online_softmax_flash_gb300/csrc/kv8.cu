// Storing rows in the paged 8-bit K/V cache, with the position rotation on the way, and reading them back (format:
// kv8.cuh).
//
// Appending: a block (or, of few tokens, a warp) takes one page of one kv head, K or V.  K's rows are rotated: channels a, b of
// a pair by the angle of their position become a c - b s and b c + a s, rounded once to float32, so the codes are those of the
// formulas and not of some order of float32 operations (rotate1; all but the few values near a tie need only rotate2).  The
// page's scale is 2^e with the least e for which its largest magnitude is at most 448 * 2^e; a page that holds earlier tokens
// keeps its scale unless the new ones need a larger one, and then the codes there are rounded again: e4m3 codes only
// change their exponent, so that is exact but for those that fall among the subnormals.  NaN and infinities are stored as
// NaN and leave the scale alone.
// A block goes through one chain: lengths and table, then rows and angles, then the scale; the reduction; the stores.  That, not
// DRAM, bounds it: three blocks of 256 threads to an SM hide most of it (8 prompts of 4096 tokens, 8 heads of 128, 201 MB
// without queries: 74 us, 2.7 TB/s; two or four blocks 87, 107; two blocks of 512 threads 111; angles loaded behind the
// check of the table's entry 85; every value by rotate1 2 us more).  With the queries of 32 heads, 738 MB: 138 us, 5.3 TB/s.
#include "kv8.cuh"
#include "sm100_ptx.cuh"

namespace osf {
namespace {

constexpr int kThreads = 256;
constexpr float kMaxF32 = 3.4028235e38f;

__device__ __forceinline__ float lo_bf16(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// W (4 or 8) neighbouring channels of a row.
template <int W>
__device__ __forceinline__ void load_run(const float *p, bool vec, float *x) {
    if (vec) {
#pragma unroll
        for (int i = 0; i < W; i += 4) {
            const float4 v = *reinterpret_cast<const float4 *>(p + i);
            x[i] = v.x; x[i + 1] = v.y; x[i + 2] = v.z; x[i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i) x[i] = p[i];
    }
}
template <int W>
__device__ __forceinline__ void load_run(const __nv_bfloat16 *p, bool vec, float *x) {
    if (vec) {
        uint32_t v[W / 2];
        if constexpr (W == 8) {
            const uint4 q = *reinterpret_cast<const uint4 *>(p);
            v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
        } else {
            const uint2 q = *reinterpret_cast<const uint2 *>(p);
            v[0] = q.x; v[1] = q.y;
        }
#pragma unroll
        for (int i = 0; i < W / 2; ++i) {
            x[2 * i] = lo_bf16(v[i]);
            x[2 * i + 1] = hi_bf16(v[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i) x[i] = __bfloat162float(p[i]);
    }
}
template <int W>
__device__ __forceinline__ void store_run(float *p, bool vec, const float *x) {
    if (vec) {
#pragma unroll
        for (int i = 0; i < W; i += 4) *reinterpret_cast<float4 *>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i) p[i] = x[i];
    }
}
template <int W>
__device__ __forceinline__ void store_run(__nv_bfloat16 *p, bool vec, const float *x) {
    if (vec) {
        uint32_t v[W / 2];
#pragma unroll
        for (int i = 0; i < W / 2; ++i) v[i] = ptx::pack_bf16x2(x[2 * i], x[2 * i + 1]);
        if constexpr (W == 8) *reinterpret_cast<uint4 *>(p) = make_uint4(v[0], v[1], v[2], v[3]);
        else *reinterpret_cast<uint2 *>(p) = make_uint2(v[0], v[1]);
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i) p[i] = __float2bfloat16_rn(x[i]);
    }
}

// A run as it is in memory, and its values.
template <typename T, int W>
struct Raw;
template <int W>
struct Raw<float, W> {
    float v[W];
    __device__ __forceinline__ void load(const float *p, bool vec) { load_run<W>(p, vec, v); }
    __device__ __forceinline__ void values(float *x) const {
#pragma unroll
        for (int i = 0; i < W; ++i) x[i] = v[i];
    }
};
template <int W>
struct Raw<__nv_bfloat16, W> {
    uint32_t v[W / 2];
    __device__ __forceinline__ void load(const __nv_bfloat16 *p, bool vec) {
        if (!vec) {
            const unsigned short *h = reinterpret_cast<const unsigned short *>(p);
#pragma unroll
            for (int i = 0; i < W / 2; ++i) v[i] = h[2 * i] | (uint32_t)h[2 * i + 1] << 16;
        } else if constexpr (W == 8) {
            const uint4 q = *reinterpret_cast<const uint4 *>(p);
            v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
        } else {
            const uint2 q = *reinterpret_cast<const uint2 *>(p);
            v[0] = q.x; v[1] = q.y;
        }
    }
    __device__ __forceinline__ void values(float *x) const {
#pragma unroll
        for (int i = 0; i < W / 2; ++i) {
            x[2 * i] = lo_bf16(v[i]);
            x[2 * i + 1] = hi_bf16(v[i]);
        }
    }
};

// The float32 nearest to a c - b s.
__device__ __forceinline__ float rotate1(float a, float c, float b, float s) {
    const float p = __fmul_rn(a, c), q = __fmul_rn(b, s);
    const float pe = __fmaf_rn(a, c, -p), qe = __fmaf_rn(b, s, -q);
    const float h = __fsub_rn(p, q), t = __fsub_rn(h, p);
    const float he = __fsub_rn(__fsub_rn(p, __fsub_rn(h, t)), __fadd_rn(q, t));   // h + he = p - q
    return fabsf(h) <= kMaxF32 ? __fadd_rn(h, __fadd_rn(he, __fsub_rn(pe, qe))) : h;
}
// a c - b s within 2 units in the last place, whatever cancels (Kahan's): the rounding error of b s, exact, is added back.
__device__ __forceinline__ float rotate2(float a, float c, float b, float s) {
    const float q = __fmul_rn(b, s);
    return __fadd_rn(__fmaf_rn(a, c, -q), __fmaf_rn(-b, s, q));
}
// Whether the code (or the page's scale) could be another if x were up to 8 units off.  An e4m3 code keeps 3 bits of the
// fraction or fewer, so ties have zeros in the last 19 (of a coarser code more of them), and so have 448 * 2^e, infinity and NaN
// (its last bits are ones).
__device__ __forceinline__ bool near_tie(float x) { return ((__float_as_uint(x) + 8u) & 0x7ffffu) < 16u; }

// i / d, exact for 0 <= i < 2^31: with 2^(s - 1) < d <= 2^s and inv = floor(2^(31 + s) / d) + 1, inv * d - 2^(31 + s) is in
// 1 .. d, which moves i * inv / 2^(31 + s) away from i / d by less than 2^31 / 2^(31 + s) <= 1 / d.
__device__ __forceinline__ int quotient(int i, uint32_t inv, int shift) { return (int)(__umulhi((uint32_t)i, inv) >> shift); }

// Where the 2 W channels of unit u of a row lie: two runs of W, at first and second.  The W pairs of a unit that is rotated
// have the angles in columns angle .. angle + W - 1 of the tables.
struct Unit {
    int first, second, angle;
    bool rotated;
};
template <int W>
__device__ __forceinline__ Unit unit_of(int u, int R, bool interleaved) {
    Unit w;
    w.rotated = 2 * W * u < R;
    w.angle = W * u;
    const bool halves = w.rotated && !interleaved;
    w.first = halves ? W * u : 2 * W * u;
    w.second = halves ? R / 2 + W * u : 2 * W * u + W;
    return w;
}
// cos and sin of a unit's angles at position pos.
template <int W>
__device__ __forceinline__ void load_angles(const Kv8StoreProblem &p, const Unit &w, int pos, float (&c)[W], float (&s)[W]) {
    load_run<W>(p.cos + (long long)pos * (p.R / 2) + w.angle, p.table_vec, c);
    load_run<W>(p.sin + (long long)pos * (p.R / 2) + w.angle, p.table_vec, s);
}
// The first and second channels of a unit's pairs, and back.
template <int W>
__device__ __forceinline__ void split_pairs(const float (&x)[2 * W], bool interleaved, float (&a)[W], float (&b)[W]) {
#pragma unroll
    for (int i = 0; i < W; ++i) {
        a[i] = interleaved ? x[2 * i] : x[i];
        b[i] = interleaved ? x[2 * i + 1] : x[i + W];
    }
}
template <int W>
__device__ __forceinline__ void join_pairs(float (&x)[2 * W], bool interleaved, const float (&a)[W], const float (&b)[W]) {
#pragma unroll
    for (int i = 0; i < W; ++i) {
        x[i] = interleaved ? (i & 1 ? b[i / 2] : a[i / 2]) : a[i];
        x[i + W] = interleaved ? (i & 1 ? b[(i + W) / 2] : a[(i + W) / 2]) : b[i];
    }
}

// A unit of K, rotated: the values that near_tie lets through give the codes that the exact ones would give.
template <int W>
__device__ __forceinline__ void rotate_unit(bool interleaved, const float (&c)[W], const float (&s)[W], float (&x)[2 * W]) {
    float a[W], b[W];
    split_pairs<W>(x, interleaved, a, b);
#pragma unroll
    for (int i = 0; i < W; ++i) {
        float ra = rotate2(a[i], c[i], b[i], s[i]), rb = rotate2(b[i], c[i], -a[i], s[i]);
        if (near_tie(ra) || near_tie(rb)) {
            ra = rotate1(a[i], c[i], b[i], s[i]);
            rb = rotate1(b[i], c[i], -a[i], s[i]);
        }
        a[i] = ra;
        b[i] = rb;
    }
    join_pairs<W>(x, interleaved, a, b);
}

// Codes of four values.  ODD: some of the page's are NaN or infinite.
template <bool ODD>
__device__ __forceinline__ uint32_t code4(const float *x, float inv) {
    uint32_t w = f32_to_e4m3x2(x[0] * inv, x[1] * inv) | f32_to_e4m3x2(x[2] * inv, x[3] * inv) << 16;
    if constexpr (ODD) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (!(fabsf(x[i]) <= kMaxF32)) w = (w & ~(0xffu << 8 * i)) | 0x7fu << 8 * i;
    }
    return w;
}
template <int W, bool ODD>
__device__ __forceinline__ void store_codes(unsigned char *p, const float *x, float inv) {
    if constexpr (W == 8) *reinterpret_cast<uint2 *>(p) = make_uint2(code4<ODD>(x, inv), code4<ODD>(x + 4, inv));
    else *reinterpret_cast<uint32_t *>(p) = code4<ODD>(x, inv);
}

// The new tokens of one page of one kv head, K or V, by `size` threads: a warp (few tokens) or a block.  K units per thread
// stay in registers between the search for the largest magnitude and the rounding.
template <typename T, int W, bool BLOCK>
__device__ __forceinline__ void append_page(const Kv8StoreProblem &p, bool interleaved, int bh, int half, int page_no, int me, int size,
                                            bool vec) {
    constexpr int KEEP = W == 8 ? 2 : 4;
    __shared__ uint32_t sh_max[kThreads / 32];
    const Kv8Cache &c = p.c;
    const int D = c.D, P = c.P, units = D / (2 * W);
    const int b = bh / c.Hkv, h = bh % c.Hkv;
    const int n_new = p.counts ? p.counts[b] : p.n;
    const int base = p.lens ? p.lens[b] : 0, most = c.per_seq * P;
    // new tokens that fit: the rest is left out, and recorded
    const int fit = base < 0 ? 0 : (int)min((long long)min(n_new, p.n), (long long)most - base);
    if (page_no == 0 && h == 0 && half == 0 && me == 0) {
        if (base < 0 || n_new < 0 || n_new > p.n || fit < n_new) atomicExch(p.status, (int)OSF_ERR_INVALID);
        if (p.R && fit > 0 && base + fit > p.max_pos) atomicExch(p.status, (int)OSF_ERR_INVALID);
    }
    if (fit <= 0) return;
    const int first = (base / P + page_no) * P;           // first token of the page
    if (first >= base + fit) return;
    const int t0 = max(base, first), t1 = min(base + fit, first + P);   // its new tokens
    const int entry = kv8_entry(c, b, first);
    const T *rows = half ? static_cast<const T *>(p.v) + b * p.v_sb + h * p.v_sh
                         : static_cast<const T *>(p.k) + b * p.k_sb + h * p.k_sh;
    const long long ss = half ? p.v_ss : p.k_ss;
    const int R = half ? 0 : p.R, work = (t1 - t0) * units;
    rows += (t0 - base) * ss;
    struct Spot {
        int t;   // token behind t0
        Unit w;
    };
    auto spot_of = [&](int i) {
        const int t = quotient(i, p.units_inv, p.units_shift);
        return Spot{t, unit_of<W>(i - t * units, R, interleaved)};
    };
    auto angles = [&](const Spot &o, float (&c)[W], float (&s)[W]) {
        if (o.w.rotated) load_angles<W>(p, o.w, min(t0 + o.t, p.max_pos - 1), c, s);
    };
    auto load = [&](const Spot &o, float (&x)[2 * W]) {
        const T *row = rows + o.t * ss;
        float c[W], s[W];
        load_run<W>(row + o.w.first, vec, x);
        load_run<W>(row + o.w.second, vec, x + W);
        angles(o, c, s);
        if (o.w.rotated) rotate_unit<W>(interleaved, c, s, x);
    };
    // the largest magnitude, as bits: a NaN or an infinity shows
    constexpr uint32_t INF = 0x7f800000u;
    uint32_t mx = 0;
    auto largest = [&](const float (&x)[2 * W]) {
#pragma unroll
        for (int e = 0; e < 2 * W; ++e) mx = max(mx, __float_as_uint(x[e]) & 0x7fffffffu);
    };
    auto of_all = [&](uint32_t m) {
        m = __reduce_max_sync(0xffffffffu, m);
        if constexpr (BLOCK) {
            __syncthreads();
            if ((me & 31) == 0) sh_max[me >> 5] = m;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < kThreads / 32; ++w) m = max(m, sh_max[w]);
        }
        return m;
    };
    int page;
    long long at;
    float old_scale;
    // (rows, angles and the table's entry on their way together)
    float kept[KEEP][2 * W];
    Spot spot[KEEP];
    {
        Raw<T, W> lo[KEEP], hi[KEEP];
        float c[KEEP][W], s[KEEP][W];
#pragma unroll
        for (int k = 0; k < KEEP; ++k) {
            spot[k] = spot_of(me + k * size);
            if (me + k * size < work) {
                const T *row = rows + spot[k].t * ss;
                lo[k].load(row + spot[k].w.first, vec);
                hi[k].load(row + spot[k].w.second, vec);
                angles(spot[k], c[k], s[k]);
            }
        }
        page = kv8_checked(p.c, entry, p.status);
        if (page < 0) return;
        at = ((long long)page * 2 + half) * p.c.Hkv + h;
        old_scale = p.c.scales[at];
#pragma unroll
        for (int k = 0; k < KEEP; ++k)
            if (me + k * size < work) {
                lo[k].values(kept[k]);
                hi[k].values(kept[k] + W);
                if (spot[k].w.rotated) rotate_unit<W>(interleaved, c[k], s[k], kept[k]);
                largest(kept[k]);
            }
    }
    for (int i = me + KEEP * size; i < work; i += size) {
        float x[2 * W];
        const Spot o = spot_of(i);
        load(o, x);
        largest(x);
    }
    mx = of_all(mx);
    const bool odd = mx >= INF;
    if (odd) {   // once more, without them
        mx = 0;
        for (int i = me; i < work; i += size) {
            float x[2 * W];
            const Spot o = spot_of(i);
            load(o, x);
#pragma unroll
            for (int e = 0; e < 2 * W; ++e) {
                const uint32_t u = __float_as_uint(x[e]) & 0x7fffffffu;
                mx = max(mx, u < INF ? u : 0u);
            }
        }
        mx = of_all(mx);
    }
    // mx = (1 + m / 2^23) 2^x: the least e with mx <= 1.75 * 2^(8 + e)
    int e = max((int)(mx >> 23) - 127 - 8 + ((mx & 0x7fffffu) > 0x600000u ? 1 : 0), kKv8MinExp);
    unsigned char *codes = c.pages + at * P * D;
    if (t0 > first) {   // earlier tokens: the scale only grows, and their codes follow it
        const int old = kv8_exponent(old_scale);
        if (e > old) {
            const float f = pow2_of(max(old - e, -126));
            const int words = (t0 - first) * D / 4;
            for (int i = me; i < words; i += size) {
                uint32_t *w = reinterpret_cast<uint32_t *>(codes) + i;
                const float2 lo = e4m3x2_to_f32(*w), hi = e4m3x2_to_f32(*w >> 16);
                *w = f32_to_e4m3x2(lo.x * f, lo.y * f) | f32_to_e4m3x2(hi.x * f, hi.y * f) << 16;
            }
        }
        e = max(e, old);
    }
    const float inv = pow2_of(-e);
    auto store = [&](const Spot &o, const float (&x)[2 * W]) {
        unsigned char *row = codes + (t0 - first + o.t) * D;
        if (odd) {
            store_codes<W, true>(row + o.w.first, x, inv);
            store_codes<W, true>(row + o.w.second, x + W, inv);
        } else {
            store_codes<W, false>(row + o.w.first, x, inv);
            store_codes<W, false>(row + o.w.second, x + W, inv);
        }
    };
#pragma unroll
    for (int k = 0; k < KEEP; ++k)
        if (me + k * size < work) store(spot[k], kept[k]);
    for (int i = me + KEEP * size; i < work; i += size) {   // pages of more: once more from the start
        float x[2 * W];
        const Spot o = spot_of(i);
        load(o, x);
        store(o, x);
    }
    if constexpr (BLOCK) __syncthreads();   // (every thread has read the old scale)
    else __syncwarp();
    if (me == 0) c.scales[at] = pow2_of(e);
}

// The queries of the new tokens, rotated in float32.  A thread takes a unit of a token for HB heads: the angles are read once.
template <typename T, int W, int HB>
__device__ __forceinline__ void rotate_queries(const Kv8StoreProblem &p, bool interleaved, int bc, int i, int q_vec, int o_vec) {
    const int units = p.c.D / (2 * W), chunks = (p.Hq + HB - 1) / HB;
    const int b = bc / chunks, h0 = bc % chunks * HB, t = quotient(i, p.units_inv, p.units_shift), u = i - t * units;
    if (t >= (p.counts ? min(p.counts[b], p.n) : p.n)) return;
    const Unit w = unit_of<W>(u, p.R, interleaved);
    const T *src = static_cast<const T *>(p.q) + b * p.q_sb + h0 * p.q_sh + t * p.q_ss;
    T *dst = static_cast<T *>(p.qo) + b * p.o_sb + h0 * p.o_sh + t * p.o_ss;
    float c[W], s[W];
    if (w.rotated) load_angles<W>(p, w, min(max((p.lens ? p.lens[b] : 0) + t, 0), p.max_pos - 1), c, s);
    Raw<T, W> lo[HB], hi[HB];
#pragma unroll
    for (int k = 0; k < HB; ++k)
        if (h0 + k < p.Hq) {
            lo[k].load(src + k * p.q_sh + w.first, q_vec);
            hi[k].load(src + k * p.q_sh + w.second, q_vec);
        }
#pragma unroll
    for (int k = 0; k < HB; ++k)
        if (h0 + k < p.Hq) {
            float x[2 * W];
            lo[k].values(x);
            hi[k].values(x + W);
            if (w.rotated) {
                float a[W], b2[W];
                split_pairs<W>(x, interleaved, a, b2);
#pragma unroll
                for (int e = 0; e < W; ++e) {
                    const float ra = fmaf(a[e], c[e], -(b2[e] * s[e])), rb = fmaf(b2[e], c[e], a[e] * s[e]);
                    a[e] = ra;
                    b2[e] = rb;
                }
                join_pairs<W>(x, interleaved, a, b2);
            }
            store_run<W>(dst + k * p.o_sh + w.first, o_vec, x);
            store_run<W>(dst + k * p.o_sh + w.second, o_vec, x + W);
        }
}

// One launch: blocks for the pages that new tokens may fall into, and among them, spread evenly, blocks for the queries; the
// former wait on their chain of loads, a reduction and stores, and the latter are bound by memory.  Of the blocks before block i,
// i * page_share / 2^32 have pages.
// INTER: whether pairs are interleaved (2: to be seen at run time).
template <typename T, int W, bool BLOCK, int HB, int INTER>
__global__ void __launch_bounds__(kThreads, 3)
kv8_append_kernel(const Kv8StoreProblem p, int pages_per_seq, unsigned long long page_share, unsigned q_blocks, int k_vec,
                  int v_vec, int q_vec, int o_vec) {
    const Kv8Cache &c = p.c;
    const bool inter = INTER == 2 ? p.interleaved != 0 : INTER != 0;
    const unsigned page_block = (unsigned)(blockIdx.x * page_share >> 32);
    if ((unsigned)((blockIdx.x + 1) * page_share >> 32) == page_block) {
        // q_blocks blocks to each (batch, HB heads), or several of those to a block (a token of 32 sequences: 10.9 us with a block
        // for each, 8.8)
        const unsigned qb = blockIdx.x - page_block, each = (unsigned)p.n * (c.D / (2 * W));
        unsigned bc, i;
        if (each * 2 <= kThreads) {
            const unsigned per = kThreads / each, k = threadIdx.x / each;
            bc = qb * per + k;
            i = threadIdx.x - k * each;
            if (k >= per || bc >= (unsigned)p.B * ((p.Hq + HB - 1) / HB)) return;
        } else {
            bc = qb / q_blocks;
            i = (qb - bc * q_blocks) * kThreads + threadIdx.x;
        }
        rotate_queries<T, W, HB>(p, inter, (int)bc, (int)i, q_vec, o_vec);
        return;
    }
    const unsigned task = BLOCK ? page_block : page_block * (kThreads / 32) + (threadIdx.x >> 5);
    const unsigned bhh = task / pages_per_seq;
    const int page_no = (int)(task - bhh * pages_per_seq), half = (int)(bhh & 1), bh = (int)(bhh >> 1);
    if (bh >= p.B * c.Hkv) return;
    append_page<T, W, BLOCK>(p, inter, bh, half, page_no, BLOCK ? threadIdx.x : threadIdx.x & 31, BLOCK ? kThreads : 32,
                             half ? v_vec : k_vec);
}

// A thread takes CH channels of kReadTokens tokens at a time: 16 bytes to write of each, so that a warp's stores are whole lines
// (32 bytes of bfloat16: 47 us for 8 prompts of 4096 tokens, 8 heads of 128), and all loads in flight together (1, 2, 4, 8
// tokens: 42, 40, 42, 42 us there, and of one token in 32 sequences 11, 11, 11, 15).  201 MB in 40 us: 5.0 TB/s.
constexpr int kReadTokens = 2;
template <typename T>
__global__ void __launch_bounds__(kThreads)
kv8_read_kernel(const Kv8StoreProblem p, int k_vec, int v_vec) {
    constexpr int CH = 16 / sizeof(T);
    const Kv8Cache &c = p.c;
    const int D = c.D, per = D / CH;
    const int bh = blockIdx.y, b = bh / c.Hkv, h = bh % c.Hkv, half = blockIdx.z;
    const int len = kv8_length(p.lens, b, c.per_seq * c.P, p.status), start = p.starts ? p.starts[b] : 0;
    T *out = static_cast<T *>(half ? p.vo : p.ko) + (long long)bh * p.n * D;
    const bool vec = half ? v_vec : k_vec;
    const int total = p.n * per, step = gridDim.x * kThreads;
    for (int i0 = blockIdx.x * kThreads + threadIdx.x; i0 < total; i0 += kReadTokens * step) {
        int entry[kReadTokens], at[kReadTokens];   // page (-1: none), and the piece's place in it
#pragma unroll
        for (int e = 0; e < kReadTokens; ++e) {
            const int i = i0 + e * step, t = quotient(i, p.units_inv, p.units_shift);
            const long long pos = (long long)start + t;
            const bool have = i < total && pos >= 0 && pos < len;
            entry[e] = have ? kv8_entry(c, b, (int)pos) : -1;
            at[e] = have ? ((int)pos & (c.P - 1)) * D + (i - t * per) * CH : -1;
        }
        uint32_t v[kReadTokens][CH / 4];
        float scale[kReadTokens];
#pragma unroll
        for (int e = 0; e < kReadTokens; ++e) {
            const int page = at[e] >= 0 ? kv8_checked(c, entry[e], p.status) : -1;
#pragma unroll
            for (int k = 0; k < CH / 4; ++k) v[e][k] = 0;
            scale[e] = 1.f;
            if (page >= 0) {
                const long long row = ((long long)page * 2 + half) * c.Hkv + h;
                const unsigned char *src = c.pages + row * c.P * D + at[e];
                if constexpr (CH == 8) {
                    const uint2 w = *reinterpret_cast<const uint2 *>(src);
                    v[e][0] = w.x;
                    v[e][CH / 4 - 1] = w.y;
                } else {
                    v[e][0] = *reinterpret_cast<const uint32_t *>(src);
                }
                scale[e] = c.scales[row];
            }
        }
#pragma unroll
        for (int e = 0; e < kReadTokens; ++e) {
            const int i = i0 + e * step;
            if (i >= total) break;
            const float f = pow2_of(kv8_exponent(scale[e]));
            float x[CH];
#pragma unroll
            for (int k = 0; k < CH / 4; ++k) {
                const float2 lo = e4m3x2_to_f32(v[e][k]), hi = e4m3x2_to_f32(v[e][k] >> 16);
                x[4 * k] = lo.x * f; x[4 * k + 1] = lo.y * f; x[4 * k + 2] = hi.x * f; x[4 * k + 3] = hi.y * f;
            }
            store_run<CH>(out + (long long)i * CH, vec, x);
        }
    }
}

// Whether runs of W channels of every row can be read or written 16 (bfloat16 and W = 4: 8) bytes at a time.
bool rows_vec(const void *q, long long a, long long b, long long c, int es, int W) {
    const int bytes = W * es < 16 ? W * es : 16, elems = bytes / es;
    return (reinterpret_cast<uintptr_t>(q) % bytes) == 0 && (a | b | c) % elems == 0;
}

template <typename T, int W, bool BLOCK, int HB, int INTER>
cudaError_t append_k(const Kv8StoreProblem &p, int pages_per_seq, cudaStream_t s) {
    const Kv8Cache &c = p.c;
    const int es = sizeof(T);
    const long long tasks = (long long)p.B * c.Hkv * 2 * pages_per_seq;
    const long long page_blocks = BLOCK ? tasks : (tasks + kThreads / 32 - 1) / (kThreads / 32);
    const long long each = (long long)p.n * (c.D / (2 * W)), q_blocks = (each + kThreads - 1) / kThreads;
    const long long heads = (long long)p.B * ((p.Hq + HB - 1) / HB), per = each * 2 <= kThreads ? kThreads / each : 0;
    const long long blocks = page_blocks + (!p.q ? 0 : per ? (heads + per - 1) / per : heads * q_blocks);
    if (blocks >= (1LL << 31) || tasks >= (1LL << 31)) return cudaErrorInvalidValue;
    kv8_append_kernel<T, W, BLOCK, HB, INTER><<<(unsigned)blocks, kThreads, 0, s>>>(
        p, pages_per_seq, (((unsigned long long)page_blocks << 32) + blocks - 1) / blocks, (unsigned)q_blocks,
        rows_vec(p.k, p.k_sb, p.k_sh, p.k_ss, es, W), rows_vec(p.v, p.v_sb, p.v_sh, p.v_ss, es, W), rows_vec(p.q, p.q_sb, p.q_sh, p.q_ss, es, W),
        rows_vec(p.qo, p.o_sb, p.o_sh, p.o_ss, es, W));
    count_launches(1);
    return cudaGetLastError();
}

// The division by the `units` (2 .. 64) of a row.
void set_units(Kv8StoreProblem &p, int units) {
    p.units_shift = 31 - __builtin_clz(units - 1);
    p.units_inv = (unsigned)((1ULL << (32 + p.units_shift)) / units + 1);
}

template <typename T, int W>
cudaError_t append_w(Kv8StoreProblem p, int sm_count, cudaStream_t s) {
    const Kv8Cache &c = p.c;
    set_units(p, c.D / (2 * W));
    const long long pages = ((long long)p.n + 2 * c.P - 2) / c.P;
    const int per_seq = (int)(pages < c.per_seq ? pages : c.per_seq);
    // a warp to a page while a page's new tokens fit its lanes' registers
    const bool block = (long long)(p.n < c.P ? p.n : c.P) * (c.D / (2 * W)) > (W == 8 ? 64 : 128);
    // four heads to a thread once there are threads enough (queries of 8 prompts of 4096 tokens, 32 heads of 128: with 2, 4, 8
    // heads the call took 177, 154, 195 us)
    const bool heads = (long long)p.B * p.Hq * p.n * (c.D / (2 * W)) >= 8LL * 1024 * sm_count;
    if (!block) return heads ? append_k<T, W, false, 4, 2>(p, per_seq, s) : append_k<T, W, false, 1, 2>(p, per_seq, s);
    if (p.interleaved) return heads ? append_k<T, W, true, 4, 1>(p, per_seq, s) : append_k<T, W, true, 1, 1>(p, per_seq, s);
    return heads ? append_k<T, W, true, 4, 0>(p, per_seq, s) : append_k<T, W, true, 1, 0>(p, per_seq, s);
}

template <typename T>
cudaError_t read_t(Kv8StoreProblem p, int sm_count, cudaStream_t s) {
    constexpr int CH = 16 / sizeof(T);
    const Kv8Cache &c = p.c;
    set_units(p, c.D / CH);
    const long long work = ((long long)p.n * (c.D / CH) + kThreads - 1) / kThreads;
    const long long heads = (long long)p.B * c.Hkv * 2, most = (16LL * sm_count + heads - 1) / heads;
    // (32 sequences of 64 tokens: 8.8 us; a block to each kThreads pieces 10.9)
    const long long few = (work + kReadTokens - 1) / kReadTokens;
    const dim3 grid((unsigned)(few < most ? few : most), (unsigned)(p.B * c.Hkv), 2);
    kv8_read_kernel<T><<<grid, kThreads, 0, s>>>(p, rows_vec(p.ko, 0, 0, 0, sizeof(T), CH), rows_vec(p.vo, 0, 0, 0, sizeof(T), CH));
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv8_append(const Kv8StoreProblem &p0, int sm_count, cudaStream_t s) {
    Kv8StoreProblem p = p0;
    const bool wide = p.R % 16 == 0;   // units of 16 channels; else (multiples of 8) of 8
    p.table_vec = ((reinterpret_cast<uintptr_t>(p.cos) | reinterpret_cast<uintptr_t>(p.sin)) & 15u) == 0;
    if (p.dtype == OSF_F32) return wide ? append_w<float, 8>(p, sm_count, s) : append_w<float, 4>(p, sm_count, s);
    return wide ? append_w<__nv_bfloat16, 8>(p, sm_count, s) : append_w<__nv_bfloat16, 4>(p, sm_count, s);
}
cudaError_t launch_kv8_read(const Kv8StoreProblem &p, int sm_count, cudaStream_t s) {
    return p.dtype == OSF_F32 ? read_t<float>(p, sm_count, s) : read_t<__nv_bfloat16>(p, sm_count, s);
}

}  // namespace osf
