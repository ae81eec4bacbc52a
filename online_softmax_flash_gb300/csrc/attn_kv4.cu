// Attention over the 4-bit K/V cache (record format: kv4.cuh): a few query rows per sequence against
// a long cache, the decode step.  Like the bf16 decode kernel, one CTA takes the query rows of one
// (batch, kv head) against one part of its keys, so a record leaves HBM once; every part yields a partial
// online-softmax state (m, l, acc), and the log-sum-exp combine merges them.  The parts are cut from each
// sequence's own length, on the device, so a ragged batch splits every sequence evenly.
//
// Two kernels.  The tensor-core one (bfloat16 queries, D 64 or 128) is described where it starts.  The
// general one takes any D that is a multiple of 32 and float32 or bfloat16 queries.  There a warp copies the records of
// 32 keys to shared memory and takes a key per lane (its whole dot product with up to 4 query rows), then a channel of
// each group per lane: B=2 Hq=12 Hkv=4, 284 records of D=128, float32, 12 us, latency.  (Each lane reading its own
// record from memory, and every record again for V: 25 us.)
#include "kv4.cuh"
#include "sm100_ptx.cuh"

namespace osf {
namespace {

using namespace ptx;

constexpr int GW = 4;        // warps per CTA
constexpr int RB = 4;        // query rows per CTA
constexpr int MAXG = 8;      // groups of 32 channels: D <= 256
constexpr int WS_D = 256;

template <bool B>
struct Flag {
    static constexpr bool value = B;
};

__device__ __forceinline__ float lo_bf16(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// Keys [begin, end) that part `split` of `splits` has of a sequence of n keys, in steps of `unit`.
__device__ __forceinline__ void part_of(int n, int unit, int split, int splits, int &begin, int &end) {
    const long long units = ((long long)n + unit - 1) / unit;
    begin = (int)(units * split / splits) * unit;
    end = min(n, (int)(units * (split + 1) / splits) * unit);
}

// Words between the staged records of two keys: one more than a record, so that 32 lanes that read the same word of
// their keys hit 32 banks.
__host__ __device__ __forceinline__ int stage_stride(int D) { return kv4_record_bytes(D) / 4 + 1; }
__host__ __device__ __forceinline__ int general_smem(int D) {
    const int stage = GW * 32 * stage_stride(D) * 4, out = GW * RB * D * 4;
    return stage > out ? stage : out;
}

// NGC: groups of a head dimension where the compiler is to know them (D up to 128), or 0.
template <typename T, int NGC>
__global__ void __launch_bounds__(GW * 32)
attn_kv4_kernel(const Kv4AttnProblem kp) {
    constexpr int MG = NGC ? NGC : MAXG;
    const AttnProblem &p = kp.a;
    extern __shared__ __align__(16) uint32_t stage[];   // [GW][32][stride] words; at the end [GW][RB][D] outputs
    __shared__ __align__(16) float sq[RB][WS_D];
    __shared__ __align__(16) float sp[GW][32][RB];      // weights of a warp's 32 keys
    __shared__ float sm[GW][RB], sl[GW][RB];
    griddep_launch();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = p.Hq / p.Hkv, R = G * p.Sq;
    const int kvbh = blockIdx.x, b = kvbh / p.Hkv, kvh = kvbh % p.Hkv;
    const int r0 = blockIdx.z * RB, rows = min(RB, R - r0);
    const int n = kv4_length(kp.lens, b, p.Sk, p.status);
    const int NG = NGC ? NGC : p.D / kKv4Group, D = 32 * NG, rec = kv4_record_bytes(D), stride = stage_stride(D);
    for (int i = tid; i < RB * D; i += GW * 32) {
        const int r = i / D, c = i % D;
        float x = 0.f;
        if (r < rows) {
            const int gr = r0 + r;
            x = to_f32(static_cast<const T *>(p.q)[q_at(p, b, kvh * G + gr / p.Sq, gr % p.Sq) + c]);
        }
        sq[r][c] = x;
    }
    __syncthreads();
    int lim[RB], lim_all = n;   // keys below lim_all are seen by every row
#pragma unroll
    for (int r = 0; r < RB; ++r) {
        const int i = (r0 + min(r, rows - 1)) % p.Sq;
        lim[r] = r >= rows ? 0 : p.causal ? min(n, max(0, n - p.Sq + i + 1)) : n;
        if (r < rows) lim_all = min(lim_all, lim[r]);
    }
    int begin, end;
    part_of(n, 32, blockIdx.y, p.splits, begin, end);
    const unsigned char *head = kp.cache + (long long)kvbh * p.Sk * rec;
    uint32_t *mine = stage + warp * 32 * stride;
    float m[RB], l[RB], acc[RB][MG];
#pragma unroll
    for (int r = 0; r < RB; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.f;
#pragma unroll
        for (int g = 0; g < MG; ++g) acc[r][g] = 0.f;
    }
    for (int k0 = begin + warp * 32; k0 < end; k0 += GW * 32) {
        const int key = k0 + lane, cnt = min(32, end - k0);
        // the keys' records, 8 bytes at a time (their alignment), ten loads of a lane in flight
        const uint2 *src = reinterpret_cast<const uint2 *>(head + (long long)k0 * rec);
        const int per = 5 * NG;   // 8-byte pieces of a record
#pragma unroll
        for (int c0 = 0; c0 < 5 * MG; c0 += 10) {
            if (c0 >= per) break;
            uint2 v[10];
#pragma unroll
            for (int c = 0; c < 10; ++c) {
                const int i = (c0 + c) * 32 + lane;
                if (i < cnt * per) v[c] = __ldcs(src + i);
            }
#pragma unroll
            for (int c = 0; c < 10; ++c) {
                const int i = (c0 + c) * 32 + lane, k = i / per;
                if (i < cnt * per) {
                    mine[k * stride + 2 * (i - k * per)] = v[c].x;
                    mine[k * stride + 2 * (i - k * per) + 1] = v[c].y;
                }
            }
        }
        __syncwarp();
        float s[RB] = {0.f, 0.f, 0.f, 0.f};
        if (key < end) {
            const uint32_t *codes = mine + lane * stride, *pairs = codes + 8 * NG;
#pragma unroll
            for (int g = 0; g < MG; ++g) {
                if (g >= NG) break;
                const uint32_t sp2 = pairs[g];
                const float sc = lo_bf16(sp2), mn = hi_bf16(sp2);
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const uint32_t w = codes[t * NG + g];
                    float x[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = fmaf((float)((w >> (4 * e)) & 15u), sc, mn);
#pragma unroll
                    for (int r = 0; r < RB; ++r) {
                        const float4 a = *reinterpret_cast<const float4 *>(&sq[r][g * 32 + t * 8]);
                        const float4 c = *reinterpret_cast<const float4 *>(&sq[r][g * 32 + t * 8 + 4]);
                        s[r] = fmaf(x[0], a.x, s[r]); s[r] = fmaf(x[1], a.y, s[r]);
                        s[r] = fmaf(x[2], a.z, s[r]); s[r] = fmaf(x[3], a.w, s[r]);
                        s[r] = fmaf(x[4], c.x, s[r]); s[r] = fmaf(x[5], c.y, s[r]);
                        s[r] = fmaf(x[6], c.z, s[r]); s[r] = fmaf(x[7], c.w, s[r]);
                    }
                }
            }
        }
        float pr[RB];
#pragma unroll
        for (int r = 0; r < RB; ++r) {
            const float y = key < lim[r] ? s[r] * p.scale_log2 : -INFINITY;
            if (kp.scores && r < rows && key < end)
                kp.scores[((long long)kvbh * R + r0 + r) * p.Sk + key] = y;
            const float mx = fmaxf(m[r], warp_max(y));
            const float ref = mx == -INFINITY ? 0.f : mx;
            const float a = ex2_approx(m[r] - ref);
            pr[r] = ex2_approx(y - ref);
            l[r] = l[r] * a + warp_sum(pr[r]);
            m[r] = mx;
#pragma unroll
            for (int g = 0; g < MG; ++g) acc[r][g] *= a;
        }
        *reinterpret_cast<float4 *>(sp[warp][lane]) = make_float4(pr[0], pr[1], pr[2], pr[3]);
        __syncwarp();
        const bool all_seen = k0 + cnt <= lim_all;
        auto values = [&](auto masked) {
#pragma unroll 4
            for (int kk = 0; kk < cnt; ++kk) {
                const float4 pk4 = *reinterpret_cast<const float4 *>(sp[warp][kk]);
                const float pk[RB] = {pk4.x, pk4.y, pk4.z, pk4.w};
                const uint32_t *codes = mine + kk * stride + 4 * NG, *pairs = codes + 5 * NG;
#pragma unroll
                for (int g = 0; g < MG; ++g) {
                    if (g >= NG) break;
                    const uint32_t sp2 = pairs[g], w = codes[(lane >> 3) * NG + g];
                    const float x = fmaf((float)((w >> (4 * (lane & 7))) & 15u), lo_bf16(sp2), hi_bf16(sp2));
#pragma unroll
                    for (int r = 0; r < RB; ++r)   // a NaN value must not reach a row that does not see its key
                        acc[r][g] = masked.value && k0 + kk >= lim[r] ? acc[r][g] : fmaf(pk[r], x, acc[r][g]);
                }
            }
        };
        if (all_seen) values(Flag<false>{});
        else values(Flag<true>{});
        __syncwarp();
    }
    __syncthreads();   // the records are done with: their memory takes the outputs
    float *sacc = reinterpret_cast<float *>(stage);
#pragma unroll
    for (int r = 0; r < RB; ++r) {
        if (lane == 0) {
            sm[warp][r] = m[r];
            sl[warp][r] = l[r];
        }
#pragma unroll
        for (int g = 0; g < MG; ++g)
            if (g < NG) sacc[(warp * RB + r) * D + g * 32 + lane] = acc[r][g];
    }
    __syncthreads();
    const long long rows_total = (long long)p.B * p.Hq * p.Sq;
    for (int i = tid; i < rows * D; i += GW * 32) {
        const int r = i / D, c = i % D, gr = r0 + r;
        float M = -INFINITY, L = 0.f, A = 0.f;
#pragma unroll
        for (int w = 0; w < GW; ++w) M = fmaxf(M, sm[w][r]);
        const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
        for (int w = 0; w < GW; ++w) {
            const float wt = ex2_approx(sm[w][r] - ref);
            A += wt * sacc[(w * RB + r) * D + c];
            L += wt * sl[w][r];
        }
        const int hq = kvh * G + gr / p.Sq, qi = gr % p.Sq;
        const long long grow = ((long long)b * p.Hq + hq) * p.Sq + qi;
        if (p.splits == 1) {
            static_cast<T *>(p.o)[o_at(p, b, hq, qi) + c] = from_f32<T>(L > 0.f || L != L ? A / L : 0.f);
            if (p.lse && c == 0) p.lse[grow] = L > 0.f ? (M + __log2f(L)) * kLn2 : L != L ? L : -INFINITY;
        } else {
            p.part_acc[((size_t)blockIdx.y * rows_total + grow) * D + c] = A;
            if (c == 0) {
                p.part_m[(size_t)blockIdx.y * rows_total + grow] = M;
                p.part_l[(size_t)blockIdx.y * rows_total + grow] = L;
            }
        }
    }
}

// ============================================================================ tensor-core kernel
// Keys are the M rows of warp-level MMAs (m16n8k16) and query rows the N columns, so eight query rows
// cost one MMA column block and the dequantised operand is always A, built in registers:
//   S^T[16 keys x 8 rows]      = sum over groups of  scale * (codes . Q) + minimum * sum Q
//   O^T[16 channels x 8 rows] += V^T[16 channels x 16 keys] P^T[16 keys x 8 rows]
// K: a code masked out of its word is the float16 subnormal code * 2^-24 (nibbles 0, 4) or
// code * 2^-20 (nibbles 1, 5; Q is scaled by 2^-4 there), so one AND per pair makes an exact operand.  Q is
// held in float16 after an exact power-of-two scaling per row that puts its largest entry at 2^13 .. 2^14:
// 8 significant bits fit, down to entries 2^-28 of the row's largest.  A group's two k-steps go to a
// fresh accumulator, and the scale is applied to it in float32; the sum of minimum * (sum Q of the group) is
// one more MMA, bfloat16, whose k index runs over the groups three times, for three bfloat16 parts of sum Q.
// V: likewise, with scale and minimum moved to the other side of the product: for the channels of one group
//   sum_k P_k (minimum_k + scale_k code_kc) = sum_k P_k minimum_k + sum_k (P_k scale_k) code_kc,
// the first sum in float32 (one per row and group), the second an MMA whose B operand is P * scale in
// float16, 11 bits.  One byte permute interleaves the halves of two keys' words, after which one AND makes the pair
// (code of key k, code of key k') of a channel.  P <= 1 and scale < 2^e, e following the largest V scale that the warp
// has met, so P * scale is lifted by 2^(14 - e); what float16 cannot hold of a key is then at most 2^(e - 39).  That
// is little beside the scales of a tile that are at least 2^(e - 6).  A tile with a smaller one (groups or keys
// whose values lie far apart) takes P * scale in two bfloat16 parts, 16 bits, lifted by 2^109 more, against the codes
// as bfloat16 subnormals (code * 2^-133): two MMAs, the same unit in the accumulators, all 16 bits down to P * scale =
// 2^(e - 108) and none below 2^(e - 116).  (Always in float16: with equal weights a scale 2^-28 of the largest had
// 12 % error, one of 2^-32 was gone.  Always in two parts: the decode step below 88 us.)
// P moves from the S^T accumulator layout to the B operand by movmatrix.
//
// Each warp streams its own 5120-byte runs of records through a ring of bulk copies (one instruction
// per run, since K and V of a token are adjacent) and keeps its own softmax state; the eight states merge
// through shared memory at the end.  The running maximum is lazy: a row's reference starts 4 (in base 2) above its
// largest score and moves when a score passes it, so most tiles need no cross-lane reduction and no rescale, and
// P <= 1.  References are whole numbers: rescaling is exact, and log2 of the denominator meets no large number whose
// rounding it would share.
//
// B=8 Hq=32 Hkv=8, 32768 records of D=128: 336 MB in 72 us (4.7 TB/s of 6.8), 76 us with the join, against 631 us for the
// general kernel's layout on the CUDA cores.  Bound by the integer pipe, busy 53 % of the time (the masks that take codes
// out of their words run at half rate), and by the latency of a warp's chain from scores to products: 2.8
// instructions per code, the matrix pipe busy 22 %.  tcgen05 takes its operands from shared memory or TMEM, so the
// codes would have to be expanded there and read again, for at most 16 rows.  Two slots to a warp keep 80 KB in
// flight per CTA, two CTAs to an SM; smaller slots 86 us.
constexpr int TW = 8;                     // warps per CTA
constexpr uint32_t kSlot = 5120;          // bytes of one ring slot: 32 records at D = 128, 64 at D = 64
constexpr float kRowFloor = -3.4028235e38f;   // reference of a row that has seen nothing
// Scales this far below the largest still go through float16: a row's heaviest key has P >= 2^-5, so float16's least step
// (2^(e - 38) of P * scale) is at most 2^-27 of that key's P * scale.  (The decode step above with every tile past it
// 92 us, with none 82, caches cold.)
constexpr float kNarrow = 0x1p-6f;
constexpr float kHeadroom = 4.f;              // what a new reference is above the largest score (8 takes the same time)

template <int D, int NT>
struct TcCfg {
    static constexpr int REC = D + D / 4;
    static constexpr int TK = (int)kSlot / REC;
    static constexpr int STAGES = 2;
    static constexpr int NG = D / 32;
    static constexpr uint32_t RING = TW * STAGES * kSlot;
    static constexpr uint32_t MERGE = TW * 8 * NT * D * 4;
    static constexpr uint32_t SMEM = RING > MERGE ? RING : MERGE;
};

// Key of a 16-key tile that MMA row m (or k index m) stands for, m < 8 (m + 8: 8 more).  With 160-byte
// records the 16-byte K reads of rows m, m + 1 and the V reads of k = 0, 2, 4, 6 (and 1, 3, 5, 7)
// then fall on different banks (measured: no load conflicts).
__device__ __forceinline__ int tile_key(int m) { return ((m >> 1) & 1) | (((m & 1) ^ (m >> 2)) << 1) | (m & 4); }

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float trunc_bf16(float x) { return __uint_as_float(__float_as_uint(x) & 0xffff0000u); }
// D = A B, no accumulator.
__device__ __forceinline__ void mma_bf16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                               uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
// Two values as the sum of two bfloat16 pairs: 16 bits of each.
__device__ __forceinline__ void split_bf16x2(float a, float b, uint32_t &hi, uint32_t &lo) {
    hi = pack_bf16x2(a, b);
    lo = pack_bf16x2(a - lo_bf16(hi), b - hi_bf16(hi));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Channels c .. c+3 of a finished row with maximum M, denominator L and numerator A.
__device__ __forceinline__ void write_row(const AttnProblem &p, int b, int hq, int qi, int c, float4 A, float M, float L) {
    const float inv = L > 0.f || L != L ? 1.f / L : 0.f;   // a row that saw nothing gives 0
    __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(p.o) + o_at(p, b, hq, qi) + c;
    o[0] = __float2bfloat16_rn(A.x * inv); o[1] = __float2bfloat16_rn(A.y * inv);
    o[2] = __float2bfloat16_rn(A.z * inv); o[3] = __float2bfloat16_rn(A.w * inv);
    if (p.lse && c == 0)
        p.lse[((long long)b * p.Hq + hq) * p.Sq + qi] = L > 0.f ? (M + log2f(L)) * kLn2 : L != L ? L : -INFINITY;
}

template <int N>
struct Words {
    uint32_t w[N];
};
template <int N>
__device__ __forceinline__ Words<N> lds_words(const unsigned char *p) {
    Words<N> r;
    if (N == 4) {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        r.w[0] = v.x; r.w[1] = v.y; r.w[N > 2 ? 2 : 0] = v.z; r.w[N > 3 ? 3 : 0] = v.w;
    } else if (N == 2) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        r.w[0] = v.x; r.w[N > 1 ? 1 : 0] = v.y;
    } else {
        r.w[0] = *reinterpret_cast<const uint32_t *>(p);
    }
    return r;
}

// Work is cut flat: an item is one block of query rows of one (batch, kv head), worth max(1, ceil(length / TK))
// tiles and kItemCost more for what it costs besides them; the items lie one after another (batch, kv head, row
// block), and CTA c of nc takes the c-th part of the whole, whatever items it spans.  So every CTA gets the same
// work, in one wave, for any mix of lengths.  (Without kItemCost a CTA full of short sequences ran 60 us where
// the average took 30: B=16 Hkv=8 Sq=4 D=64, lengths 4 .. 8192.)  An item whose tiles all lie in one part is finished
// there; of the others a CTA holds at most two pieces, the end of one that began before (slot 2c of the partial
// states) and the start of one that goes on (slot 2c + 1).
struct FlatWork {
    long long total, base;   // units of all items, and of the batches before b
    int nc;                  // CTAs that take part
};
// Tiles worth a CTA: one for every warp (Hq=32 Hkv=8 D=128, 4096 records: B=1 11.6 us, B=4 16.2 us; two for every warp 14.7 and
// 19.3 us, three 14.9 and 16.7 us).
constexpr int kMinTiles = TW;
// Tiles that an item's set-up and merge are counted as.  (Hkv=8, D=128, 16 lengths even up to 8192: 34.9 us with 8, 41.5
// with 4, 33.7 with 16; 32 lengths, most of them short: 42.7, 59.3, 30.6; 4 equal ones of 4096, 12 rows of D=64: 19.7,
// 25.6, 25.3.)
constexpr int kItemCost = 8;

__device__ __forceinline__ int item_tiles(const Kv4AttnProblem &kp, int b, int tk) {
    return max(1, (kv4_length(kp.lens, b, kp.a.Sk, kp.a.status) + tk - 1) / tk);
}
// Called by a whole warp.
__device__ __forceinline__ FlatWork flat_work(const Kv4AttnProblem &kp, int tk, int items_per_b, int b, int grid) {
    const int lane = threadIdx.x & 31;
    long long all = 0, before = 0;
    for (int i = lane; i < kp.a.B; i += 32) {
        const long long n = item_tiles(kp, i, tk) + kItemCost;
        all += n;
        before += i < b ? n : 0;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        all += __shfl_xor_sync(0xffffffffu, all, o);
        before += __shfl_xor_sync(0xffffffffu, before, o);
    }
    FlatWork f;
    f.total = all * items_per_b;
    f.base = before * items_per_b;
    f.nc = (int)max(1LL, min((long long)grid, f.total / (kMinTiles + kItemCost)));
    return f;
}
// The CTA that has unit x: the last one whose part begins at or before it.
__device__ __forceinline__ int cta_of(const FlatWork &w, long long x) { return (int)(((x + 1) * w.nc - 1) / w.total); }

template <int D, int NT, bool SCORES>
__global__ void __launch_bounds__(TW * 32, NT == 1 || D == 64 ? 2 : 1)
attn_kv4_tc_kernel(const Kv4AttnProblem kp, int q_vec, int row_blocks, int flat) {
    using C = TcCfg<D, NT>;
    constexpr int NG = C::NG, REC = C::REC, TK = C::TK, STAGES = C::STAGES;
    const AttnProblem &p = kp.a;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ uint64_t full[TW][STAGES];
    __shared__ float sm_m[TW][8 * NT], sm_l[TW][8 * NT];
    __shared__ volatile int abort_flag;
    griddep_launch();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t = lane & 3;
    const int G = p.Hq / p.Hkv, R = G * p.Sq;
    unsigned char *ring = smem + warp * (STAGES * kSlot);
    if (lane == 0) {
        for (int s = 0; s < STAGES; ++s) mbar_init(smem_u32(&full[warp][s]), 1);
        mbar_init_fence();
        if (warp == 0) abort_flag = 0;
    }
    __syncthreads();
    const int items_per_b = p.Hkv * row_blocks;
    int rest = 0;                     // units that this CTA still has to take
    int b = 0, item = 0, unit0 = 0;   // the next piece: item of batch b, from unit0 on
    if (flat) {
        const FlatWork w = flat_work(kp, TK, items_per_b, 0, gridDim.x);
        if ((int)blockIdx.x >= w.nc) return;
        const long long pos = w.total * blockIdx.x / w.nc;
        rest = (int)(w.total * (blockIdx.x + 1) / w.nc - pos);
        long long at = 0;   // units before batch b: 32 batches at a time, a lane each
        for (int b0 = 0;; b0 += 32) {
            const int bi = b0 + lane;
            const long long ub = bi < p.B ? (long long)(item_tiles(kp, bi, TK) + kItemCost) * items_per_b : 0;
            long long upto = ub;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += y;
            }
            const uint32_t past = __ballot_sync(0xffffffffu, pos < at + upto);
            if (past) {
                const int f = __ffs(past) - 1;
                b = b0 + f;
                at += __shfl_sync(0xffffffffu, upto - ub, f);
                break;
            }
            at += __shfl_sync(0xffffffffu, upto, 31);
        }
        const int ui = item_tiles(kp, b, TK) + kItemCost;
        item = (int)((pos - at) / ui);
        unit0 = (int)((pos - at) % ui);
    } else {   // one whole item per CTA
        b = blockIdx.x / items_per_b;
        item = blockIdx.x % items_per_b;
    }
    int phase = 0;   // bit s: parity of the next wait on ring slot s
    bool ok = true;
    for (;;) {
    const int kvh = item / row_blocks, kvbh = b * p.Hkv + kvh;
    const int r0 = item % row_blocks * (8 * NT), rows = min(8 * NT, R - r0);
    const int n = kv4_length(kp.lens, b, p.Sk, p.status);
    const int nb = max(1, (n + TK - 1) / TK);
    // units [unit0, unit0 + take) of the item: its first kItemCost units hold no tiles
    const int take = flat ? min(nb + kItemCost - unit0, rest) : nb + kItemCost;
    const int tile0 = max(0, unit0 - kItemCost), tile1 = unit0 + take - kItemCost;
    if (tile1 <= tile0) {   // the part ends before the item's first tile
        rest -= take;
        break;
    }
    const bool whole = tile1 - tile0 == nb;
    const int begin = tile0 * TK, end = min(n, tile1 * TK);
    // this warp's tiles of the piece: warp, warp + 8, ...
    const int tiles = (end - begin + TK - 1) / TK;
    const int mine = tiles > warp ? (tiles - warp + TW - 1) / TW : 0;
    const unsigned char *src = kp.cache + ((long long)kvbh * p.Sk + begin + warp * TK) * REC;   // the next tile to copy
    int left = end - begin - warp * TK;                                                       // records from there on
    auto issue = [&](int slot) {
        const uint32_t bytes = (uint32_t)min(TK, left) * REC, bar = smem_u32(&full[warp][slot]);
        mbar_expect_tx(bar, bytes);
        bulk_load(smem_u32(ring + slot * kSlot), src, bytes, bar);
        src += TW * TK * REC;
        left -= TW * TK;
    };
    if (lane == 0)
        for (int i = 0; i < min(STAGES, mine); ++i) issue(i);

    // Q as the B operand: column n = query row, lane (g, t) holds row g's channels 8t .. 8t+7 of each group
    uint32_t qb[NT][NG][4];
    uint32_t qm[NT][2];         // sums of Q over the groups, as the B operand of the minima
    float f[NT][2];             // S to base-2 score: undoes the scalings, times scale * log2 e
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int r = nt * 8 + g, gr = r0 + r;
        const __nv_bfloat16 *Q = static_cast<const __nv_bfloat16 *>(p.q);
        if (r < rows) Q += q_at(p, b, kvh * G + gr / p.Sq, gr % p.Sq);
        float x[NG][8];
        float mx = 0.f;
#pragma unroll
        for (int gi = 0; gi < NG; ++gi) {
            if (r >= rows) {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[gi][e] = 0.f;
            } else if (q_vec) {
                const uint4 v = *reinterpret_cast<const uint4 *>(Q + 32 * gi + 8 * t);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[gi][2 * e] = lo_bf16(w[e]);
                    x[gi][2 * e + 1] = hi_bf16(w[e]);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[gi][e] = __bfloat162float(Q[32 * gi + 8 * t + e]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(x[gi][e]));
        }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const int ex = max(-90, min(100, 13 - ((int)(__float_as_uint(mx) >> 23) - 127)));
        const float up = __uint_as_float((uint32_t)(ex + 127) << 23);
        float sum[NG];
#pragma unroll
        for (int gi = 0; gi < NG; ++gi) {
            float s = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x[gi][e] *= up;
                s += x[gi][e];
            }
            qb[nt][gi][0] = pack_f16x2(x[gi][0], x[gi][4]);
            qb[nt][gi][1] = pack_f16x2(x[gi][1] * 0.0625f, x[gi][5] * 0.0625f);
            qb[nt][gi][2] = pack_f16x2(x[gi][2], x[gi][6]);
            qb[nt][gi][3] = pack_f16x2(x[gi][3] * 0.0625f, x[gi][7] * 0.0625f);
            s += __shfl_xor_sync(0xffffffffu, s, 1);
            s += __shfl_xor_sync(0xffffffffu, s, 2);
            sum[gi] = s * 0x1p-24f;   // in the unit of the code products
        }
        // k = 2t, 2t + 1: lanes t < 2 the leading parts of groups 2t, 2t + 1, lanes t >= 2 the next parts of
        // groups 2t - 4, 2t - 3;  k + 8: lanes t < 2 the last parts, else 0.  (D = 64: groups 0, 1 only.)
        float s0 = sum[0], s1 = sum[1];
        if (NG == 4 && (t & 1)) s0 = sum[NG - 2], s1 = sum[NG - 1];
        if (NG == 2 && (t & 1)) s0 = s1 = 0.f;
        const float h0 = trunc_bf16(s0), h1 = trunc_bf16(s1), e0 = s0 - h0, e1 = s1 - h1;
        const float d0 = trunc_bf16(e0), d1 = trunc_bf16(e1);
        qm[nt][0] = t < 2 ? pack_bf16x2(h0, h1) : pack_bf16x2(d0, d1);
        qm[nt][1] = t < 2 ? pack_bf16x2(e0 - d0, e1 - d1) : 0u;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int back = 24 - __shfl_sync(0xffffffffu, ex, 8 * t + 4 * c);   // -76 .. 114
            f[nt][c] = __uint_as_float((uint32_t)(back + 127) << 23) * p.scale_log2;
        }
    }
    const int lim_all = p.causal ? n - p.Sq + 1 : n;   // keys below this are visible to every row

    // o: code sums, tile (group, h), row g (+ 8) = channel 32 group + 4 g + 2 h (+ 1), in units of 2^(e - 38)
    // (2^(e - 34)), 2^e = s_top; om: sums of P * minimum of a group
    float o[NT][NG * 2][4], om[NT][NG][2], m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int j = 0; j < NG * 2; ++j) o[nt][j][0] = o[nt][j][1] = o[nt][j][2] = o[nt][j][3] = 0.f;
#pragma unroll
        for (int gi = 0; gi < NG; ++gi) om[nt][gi][0] = om[nt][gi][1] = 0.f;
        m[nt][0] = m[nt][1] = kRowFloor;
        l[nt][0] = l[nt][1] = 0.f;
    }
    float s_top = 0x1p-100f;   // V scales so far are below it: 2^e
    float lift = 0x1p114f;     // 2^(14 - e)
    const int ka = tile_key(g);
    const int off_a = ka * REC;                                                // K, and both halves' pairs: keys ka, ka + 8
    const int off_m = off_a + D + (NG == 4 ? (t & 1) * 8 : 0);                 // K pairs whose minima this lane feeds
    const int off_v0 = tile_key(2 * t) * REC + D / 2 + (g >> 1) * (D / 8);     // V codes: keys of k = 2t, 2t + 1 (+ 8)
    const int off_v1 = tile_key(2 * t + 1) * REC + D / 2 + (g >> 1) * (D / 8);
    const uint32_t pick = (g & 1) ? 0x7632u : 0x5410u;                         // lane's half of a word, of two keys
    float *sc_out = SCORES ? kp.scores + ((long long)kvbh * R + r0 + 2 * t) * p.Sk : nullptr;
    int i = 0;
    for (; i < mine; ++i) {
        const int st = i % STAGES;
        ok = mbar_wait(smem_u32(&full[warp][st]), (phase >> st) & 1, &abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        phase ^= 1 << st;
        unsigned char *slot = ring + st * kSlot;
        const int k0 = begin + (warp + TW * i) * TK;
        const int subs = min(TK / 16, (end - k0 + 15) / 16);
        if (end - k0 < TK) {
            // the sequence ends inside the tile (its last one): records behind it are zeroed, so that stale
            // scales cannot turn a weight of zero into a NaN
            for (int x = (end - k0) * REC / 16 + lane; x < subs * REC; x += 32)
                reinterpret_cast<uint4 *>(slot)[x] = make_uint4(0, 0, 0, 0);
            __syncwarp();
        }
        // The tile's largest and smallest V scale, a key per lane.  (A scale of 0 counts as small: right, only slower.)
        float s_max = 0.f, s_min = INFINITY;
#pragma unroll
        for (int r = 0; r < TK; r += 32) {
            if (r + lane < end - k0) {
                const Words<NG> w = lds_words<NG>(slot + (r + lane) * REC + D + D / 8);
#pragma unroll
                for (int gi = 0; gi < NG; gi += 2) {
                    s_max = fmax3(s_max, lo_bf16(w.w[gi]), lo_bf16(w.w[gi + 1]));
                    s_min = fminf(s_min, fminf(lo_bf16(w.w[gi]), lo_bf16(w.w[gi + 1])));
                }
            }
        }
        bool wide = false;
        if (__any_sync(0xffffffffu, s_max >= s_top || s_min < s_top * kNarrow)) {
            const int e = __reduce_max_sync(0xffffffffu, min(254, (int)(__float_as_uint(s_max) >> 23) + 1));
            const float top = __uint_as_float((uint32_t)e << 23);   // the power of two above the tile's scales, at most 2^127
            if (top > s_top) {
                const float a = s_top / top;
                s_top = top;
                lift = 0x1p14f / top;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < NG * 2; ++j)
#pragma unroll
                        for (int q = 0; q < 4; ++q) o[nt][j][q] *= a;
            }
            wide = __any_sync(0xffffffffu, s_min < s_top * kNarrow);
        }
        auto sub_tiles = [&](auto two_parts) {
#pragma unroll 1
        for (int sub = 0; sub < subs; ++sub) {
            const unsigned char *tile = slot + sub * 16 * REC;
            const int key = k0 + sub * 16 + ka;
            float y[NT][4];
            const unsigned char *ra = tile + off_a, *rb = ra + 8 * REC;
            {
                const Words<2> ma = lds_words<2>(tile + off_m), mb = lds_words<2>(tile + off_m + 8 * REC);
                const uint32_t a0 = __byte_perm(ma.w[0], ma.w[1], 0x7632), a1 = __byte_perm(mb.w[0], mb.w[1], 0x7632);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma_bf16_first(y[nt], a0, a1, a0, a1, qm[nt][0], qm[nt][1]);
                const Words<NG> xa = lds_words<NG>(ra + t * (D / 8)), xb = lds_words<NG>(rb + t * (D / 8));
                const Words<NG> pa = lds_words<NG>(ra + D), pb = lds_words<NG>(rb + D);
#pragma unroll
                for (int gi = 0; gi < NG; ++gi) {
                    const uint32_t a = xa.w[gi], c = xb.w[gi], a8 = a >> 8, c8 = c >> 8;
                    const float s0 = lo_bf16(pa.w[gi]), s1 = lo_bf16(pb.w[gi]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float d[4];
                        mma_f16_first(d, a & 0x000f000fu, c & 0x000f000fu, a & 0x00f000f0u, c & 0x00f000f0u, qb[nt][gi][0],
                                      qb[nt][gi][1]);
                        mma_f16(d, a8 & 0x000f000fu, c8 & 0x000f000fu, a8 & 0x00f000f0u, c8 & 0x00f000f0u, qb[nt][gi][2],
                                qb[nt][gi][3]);
                        y[nt][0] = fmaf(s0, d[0], y[nt][0]);
                        y[nt][1] = fmaf(s0, d[1], y[nt][1]);
                        y[nt][2] = fmaf(s1, d[2], y[nt][2]);
                        y[nt][3] = fmaf(s1, d[3], y[nt][3]);
                    }
                }
            }
            // base-2 scores; -inf where the row does not see the key
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) y[nt][e] *= f[nt][e & 1];
            const bool masked = k0 + sub * 16 + 16 > lim_all;   // some row does not see some key
            if (masked) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int row = r0 + nt * 8 + 2 * t + (e & 1);
                        const int lim = p.causal ? n - p.Sq + row % p.Sq + 1 : n;
                        if (key + (e >> 1) * 8 >= lim) y[nt][e] = -INFINITY;
                    }
            }
            if (SCORES) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (nt * 8 + 2 * t + (e & 1) < rows && key + (e >> 1) * 8 < end)
                            sc_out[(long long)(nt * 8 + (e & 1)) * p.Sk + key + (e >> 1) * 8] = y[nt][e];
            }
            float top = -INFINITY;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                top = fmax3(top, y[nt][0] - m[nt][0], y[nt][1] - m[nt][1]);
                top = fmax3(top, y[nt][2] - m[nt][0], y[nt][3] - m[nt][1]);
            }
            if (__any_sync(0xffffffffu, top > 0.f)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float mx = fmaxf(y[nt][c], y[nt][c + 2]);
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                        mx = fmaxf(m[nt][c], ceilf(mx) + kHeadroom);
                        const float a = ex2_approx(m[nt][c] - mx);
                        m[nt][c] = mx;
                        l[nt][c] *= a;
#pragma unroll
                        for (int j = 0; j < NG * 2; ++j) {
                            o[nt][j][c] *= a;
                            o[nt][j][c + 2] *= a;
                        }
#pragma unroll
                        for (int gi = 0; gi < NG; ++gi) om[nt][gi][c] *= a;
                    }
            }
            // V scales and minima of this lane's two keys
            float vs[2][NG], vm[2][NG];
            {
                const Words<NG> pa = lds_words<NG>(ra + D + D / 8), pb = lds_words<NG>(rb + D + D / 8);
#pragma unroll
                for (int gi = 0; gi < NG; ++gi) {
                    vs[0][gi] = lo_bf16(pa.w[gi]); vm[0][gi] = hi_bf16(pa.w[gi]);
                    vs[1][gi] = lo_bf16(pb.w[gi]); vm[1][gi] = hi_bf16(pb.w[gi]);
                }
            }
            float pr[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int e = 0; e < 4; ++e) pr[nt][e] = ex2_approx(y[nt][e] - m[nt][e & 1]);
                l[nt][0] += pr[nt][0] + pr[nt][2];
                l[nt][1] += pr[nt][1] + pr[nt][3];
            }
            if (!masked) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int gi = 0; gi < NG; ++gi) {
                        om[nt][gi][0] = fmaf(pr[nt][0], vm[0][gi], fmaf(pr[nt][2], vm[1][gi], om[nt][gi][0]));
                        om[nt][gi][1] = fmaf(pr[nt][1], vm[0][gi], fmaf(pr[nt][3], vm[1][gi], om[nt][gi][1]));
                    }
            } else {
                // a NaN group (scale and minimum) must not reach a row that does not see its key: through the minimum it
                // comes where the row sees it, through the scale nowhere
#pragma unroll
                for (int gi = 0; gi < NG; ++gi) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (y[nt][e] != -INFINITY) om[nt][gi][e & 1] = fmaf(pr[nt][e], vm[e >> 1][gi], om[nt][gi][e & 1]);
                    vs[0][gi] = vs[0][gi] == vs[0][gi] ? vs[0][gi] : 0.f;
                    vs[1][gi] = vs[1][gi] == vs[1][gi] ? vs[1][gi] : 0.f;
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; e += 2)
                    f2_unpack(f2_mul(f2_pack(pr[nt][e], pr[nt][e + 1]), f2_pack(lift, lift)), pr[nt][e], pr[nt][e + 1]);
            const Words<NG> w0 = lds_words<NG>(tile + off_v0), w1 = lds_words<NG>(tile + off_v1);
            const Words<NG> w2 = lds_words<NG>(tile + off_v0 + 8 * REC), w3 = lds_words<NG>(tile + off_v1 + 8 * REC);
#pragma unroll
            for (int gi = 0; gi < NG; ++gi) {
                const uint32_t u = __byte_perm(w0.w[gi], w1.w[gi], pick), v = __byte_perm(w2.w[gi], w3.w[gi], pick);
                const uint32_t u8 = u >> 8, v8 = v >> 8;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float(&oa)[4] = o[nt][2 * gi], (&ob)[4] = o[nt][2 * gi + 1];
                    const float p0 = pr[nt][0] * vs[0][gi], p1 = pr[nt][1] * vs[0][gi];
                    const float p2 = pr[nt][2] * vs[1][gi], p3 = pr[nt][3] * vs[1][gi];
                    if constexpr (two_parts.value) {
                        uint32_t b0, b1, c0, c1;
                        split_bf16x2(p0 * 0x1p109f, p1 * 0x1p109f, b0, c0);
                        split_bf16x2(p2 * 0x1p109f, p3 * 0x1p109f, b1, c1);
                        b0 = transpose_8x8(b0); b1 = transpose_8x8(b1);
                        c0 = transpose_8x8(c0); c1 = transpose_8x8(c1);
                        mma_bf16(oa, u & 0x000f000fu, u & 0x00f000f0u, v & 0x000f000fu, v & 0x00f000f0u, b0, b1);
                        mma_bf16(ob, u8 & 0x000f000fu, u8 & 0x00f000f0u, v8 & 0x000f000fu, v8 & 0x00f000f0u, b0, b1);
                        mma_bf16(oa, u & 0x000f000fu, u & 0x00f000f0u, v & 0x000f000fu, v & 0x00f000f0u, c0, c1);
                        mma_bf16(ob, u8 & 0x000f000fu, u8 & 0x00f000f0u, v8 & 0x000f000fu, v8 & 0x00f000f0u, c0, c1);
                    } else {
                        const uint32_t b0 = transpose_8x8(pack_f16x2(p0, p1)), b1 = transpose_8x8(pack_f16x2(p2, p3));
                        mma_f16(oa, u & 0x000f000fu, u & 0x00f000f0u, v & 0x000f000fu, v & 0x00f000f0u, b0, b1);
                        mma_f16(ob, u8 & 0x000f000fu, u8 & 0x00f000f0u, v8 & 0x000f000fu, v8 & 0x00f000f0u, b0, b1);
                    }
                }
            }
        }
        };
        if (wide) sub_tiles(Flag<true>{});
        else sub_tiles(Flag<false>{});
        __syncwarp();
        if (lane == 0 && i + STAGES < mine) issue(st);
    }
    if (!ok) {
        abort_flag = 1;
        if (lane == 0) {
            atomicExch(p.status, kStatusTimeout);
            for (int j = i; j < min(i + STAGES, mine); ++j)   // let issued copies land before the ring is reused
                mbar_wait(smem_u32(&full[warp][j % STAGES]), (phase >> (j % STAGES)) & 1, nullptr, 20000000ull);
        }
    }
    // ------------------------------------------------------------- merge the warps' states
    __syncthreads();   // the rings are drained: their memory takes the outputs
    float *so = reinterpret_cast<float *>(smem);
    const float back = s_top * 0x1p-6f;   // 2^(e + 10) in two steps, each within float32's range
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            float v = l[nt][c];
            v += __shfl_xor_sync(0xffffffffu, v, 4);
            v += __shfl_xor_sync(0xffffffffu, v, 8);
            v += __shfl_xor_sync(0xffffffffu, v, 16);
            const int r = nt * 8 + 2 * t + c;
            if (g == 0) {
                sm_m[warp][r] = v > 0.f || v != v ? m[nt][c] : -INFINITY;
                sm_l[warp][r] = v;
            }
#pragma unroll
            for (int gi = 0; gi < NG; ++gi) {
                float mn = om[nt][gi][c];
                mn += __shfl_xor_sync(0xffffffffu, mn, 4);
                mn += __shfl_xor_sync(0xffffffffu, mn, 8);
                mn += __shfl_xor_sync(0xffffffffu, mn, 16);
                const float *lo = o[nt][2 * gi], *hi = o[nt][2 * gi + 1];
                *reinterpret_cast<float4 *>(so + (warp * 8 * NT + r) * D + 32 * gi + 4 * g) =
                    make_float4(fmaf(lo[c] * 0x1p16f, back, mn), fmaf(lo[c + 2] * 0x1p12f, back, mn),
                                fmaf(hi[c] * 0x1p16f, back, mn), fmaf(hi[c + 2] * 0x1p12f, back, mn));
            }
        }
    }
    __syncthreads();
    const size_t slot = 2 * (size_t)blockIdx.x + (tile0 == 0 ? 1 : 0);
    for (int x = tid; x < rows * (D / 4); x += TW * 32) {
        const int r = x / (D / 4), c = x % (D / 4) * 4, gr = r0 + r;
        float M = -INFINITY, L = 0.f;
        float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < TW; ++w) M = fmaxf(M, sm_m[w][r]);
        const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
        for (int w = 0; w < TW; ++w) {
            const float wt = ex2_approx(sm_m[w][r] - ref);
            const float4 v = *reinterpret_cast<const float4 *>(so + (w * 8 * NT + r) * D + c);
            A.x = fmaf(wt, v.x, A.x); A.y = fmaf(wt, v.y, A.y);
            A.z = fmaf(wt, v.z, A.z); A.w = fmaf(wt, v.w, A.w);
            L = fmaf(wt, sm_l[w][r], L);
        }
        if (whole) write_row(p, b, kvh * G + gr / p.Sq, gr % p.Sq, c, A, M, L);
        else {
            *reinterpret_cast<float4 *>(kp.part + (slot * 8 * NT + r) * D + c) = A;
            if (c == 0) kp.part_ml[slot * 8 * NT + r] = make_float2(M, L);
        }
    }
    if (!flat) break;
    rest -= take;
    if (rest <= 0 || abort_flag) break;   // (after a timeout the copies are settled; the rest is left)
    unit0 = 0;
    if (++item == items_per_b) {
        item = 0;
        ++b;
    }
    fence_proxy_async_smem();   // the merge buffer becomes ring again: its accesses before the next copies
    __syncthreads();
    }
}

// Rows of the items that several CTAs shared: a block per item, the same cut of the work as above.  Latency: 4 us for the
// 64 items of the problem above, its pieces' loads eight at a time.
template <int D, int NT>
__global__ void __launch_bounds__(256) kv4_combine_kernel(const Kv4AttnProblem kp, int row_blocks, int grid) {
    griddep_launch();
    constexpr int TK = TcCfg<D, NT>::TK;
    const AttnProblem &p = kp.a;
    const int G = p.Hq / p.Hkv, R = G * p.Sq, items_per_b = p.Hkv * row_blocks;
    const int b = blockIdx.x / items_per_b, item = blockIdx.x % items_per_b;
    const FlatWork w = flat_work(kp, TK, items_per_b, b, grid);
    const int ui = item_tiles(kp, b, TK) + kItemCost;
    const long long p0 = w.base + (long long)item * ui;
    const int c0 = cta_of(w, p0 + kItemCost), c1 = cta_of(w, p0 + ui - 1);   // CTAs of the first and the last tile
    griddep_wait();
    if (c0 == c1) return;
    const int r0 = item % row_blocks * (8 * NT), rows = min(8 * NT, R - r0);
    constexpr int KG = 8;   // pieces whose states are loaded together
    for (int x = threadIdx.x; x < rows * (D / 4); x += blockDim.x) {
        const int r = x / (D / 4), c = x % (D / 4) * 4, gr = r0 + r;
        float M = -INFINITY, L = 0.f;
        float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k0 = c0; k0 <= c1; k0 += KG) {
            float2 ml[KG];
            float4 v[KG];
            float mx = M;
#pragma unroll
            for (int e = 0; e < KG; ++e) {
                const size_t slot = 2 * (size_t)min(k0 + e, c1) + (k0 + e == c0 ? 1 : 0);
                ml[e] = k0 + e <= c1 ? kp.part_ml[slot * 8 * NT + r] : make_float2(-INFINITY, 0.f);
                v[e] = k0 + e <= c1 ? *reinterpret_cast<const float4 *>(kp.part + (slot * 8 * NT + r) * D + c)
                                    : make_float4(0.f, 0.f, 0.f, 0.f);
                mx = fmaxf(mx, ml[e].x);
            }
            const float ref = mx == -INFINITY ? 0.f : mx, a = ex2_approx(M - ref);
            A.x *= a; A.y *= a; A.z *= a; A.w *= a;
            L *= a;
            M = mx;
#pragma unroll
            for (int e = 0; e < KG; ++e) {
                const float wt = ex2_approx(ml[e].x - ref);
                A.x = fmaf(wt, v[e].x, A.x); A.y = fmaf(wt, v[e].y, A.y);
                A.z = fmaf(wt, v[e].z, A.z); A.w = fmaf(wt, v[e].w, A.w);
                L = fmaf(wt, ml[e].y, L);
            }
        }
        write_row(p, b, item / row_blocks * G + gr / p.Sq, gr % p.Sq, c, A, M, L);
    }
}

// Weights from the stored scores, once every row's log-sum-exp is known: a thread sums the rows of V neighbouring
// keys, RG rows' loads in flight together.  Bound by the latency of reading the scores once: 32 MB (B=16 Hkv=8, 16 rows,
// lengths 4 .. 8192) in 9 us.  (RG = 8: that call 43.2 us against 42.8, B=8 Hkv=8 Hq=32 over 32768 records 94.5 against 92.3.)
constexpr int RG = 4;
template <int V>
__global__ void __launch_bounds__(256) kv4_weights_kernel(const Kv4AttnProblem kp) {
    const AttnProblem &p = kp.a;
    const int G = p.Hq / p.Hkv, R = G * p.Sq;
    const int kvbh = blockIdx.y, b = kvbh / p.Hkv, kvh = kvbh % p.Hkv;
    const int n = kv4_length(kp.lens, b, p.Sk, p.status);
    const int key = (blockIdx.x * 256 + threadIdx.x) * V;
    float *w = kp.weights + (long long)kvbh * p.Sk + key;
    float sum[V];
#pragma unroll
    for (int i = 0; i < V; ++i) sum[i] = 0.f;
    griddep_wait();
    if (key >= p.Sk) return;
    if (key < n) {
        const float *lse = p.lse + ((long long)b * p.Hq + kvh * G) * p.Sq;   // the R rows of a kv head are consecutive
        const float *sc = kp.scores + (long long)kvbh * R * p.Sk + key;
        for (int r0 = 0; r0 < R; r0 += RG) {
            float x[RG][V], off[RG];
            bool nan = false;
#pragma unroll
            for (int e = 0; e < RG; ++e) {
                const int r = min(r0 + e, R - 1);
                off[e] = lse[r];
                const float *at = sc + (long long)r * p.Sk;
                if (V == 4) {
                    const float4 v = __ldcs(reinterpret_cast<const float4 *>(at));
                    x[e][0] = v.x; x[e][V > 1 ? 1 : 0] = v.y; x[e][V > 2 ? 2 : 0] = v.z; x[e][V > 3 ? 3 : 0] = v.w;
                } else {
                    x[e][0] = __ldcs(at);
                }
            }
#pragma unroll
            for (int e = 0; e < RG; ++e) {
                // a row that saw nothing, or a repeated one past the last, adds 0
                off[e] = r0 + e < R && off[e] != -INFINITY ? -off[e] * kLog2e : -INFINITY;
                nan |= off[e] != off[e];
            }
            if (!nan) {
#pragma unroll
                for (int e = 0; e < RG; ++e)
#pragma unroll
                    for (int i = 0; i < V; ++i) sum[i] += ex2_approx(x[e][i] + off[e]);
            } else {   // the NaN of a row is for the keys that it sees alone (the others' scores are -inf)
#pragma unroll
                for (int e = 0; e < RG; ++e)
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        if (!p.causal || key + i <= n - p.Sq + (r0 + e) % p.Sq) sum[i] += ex2_approx(x[e][i] + off[e]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (key + i >= p.Sk || (key + i >= n && kp.accumulate)) continue;
        const float v = key + i < n ? sum[i] : 0.f;   // scores behind the length were never written
        w[i] = kp.accumulate ? w[i] + v : v;
    }
}

}  // namespace

static bool use_tc(const AttnProblem &p) { return p.dtype == OSF_BF16 && (p.D == 64 || p.D == 128); }

// Launch shape of the tensor-core kernel.  Items of few tiles are not cut: a CTA each, one launch, no combine.  Else one wave
// of CTAs shares all tiles, as many as the longest possible lengths are worth.  Few is 28 tiles, 48 where the items fill a
// quarter of the SMs, 64 where they fill half.  (Hq=32 Hkv=8 D=128, whole against cut, us: 8 items of 24 tiles 9.1 against
// 10.3, of 32 10.4 against 10.4, of 48 13.1 against 10.6; 64 of 40 12.5 against 14.2, of 48 14.0 against 15.0, of 64 16.8
// against 16.1; 128 of 64 17.4 against 23.1; 256 of 64 26.0 against 31.7.  D=64 crosses at the same numbers, 16 rows of
// 32 items at 28 tiles and, D=128, 36.  Longer items are cut so that ragged batches stay even: 16 x 8 of up to 64 tiles 17.2
// against 18.4, of up to 96 22.4 against 21.8.)
struct TcPlan {
    int nt, row_blocks, flat, grid;
};
static TcPlan tc_plan(const AttnProblem &p, int sm_count) {
    TcPlan t;
    const int R = p.Hq / p.Hkv * p.Sq, tk = (int)kSlot / kv4_record_bytes(p.D);
    t.nt = R <= 8 ? 1 : 2;
    t.row_blocks = (R + 8 * t.nt - 1) / (8 * t.nt);
    const long long items = (long long)p.B * p.Hkv * t.row_blocks, per = ((long long)p.Sk + tk - 1) / tk;
    const long long wave = (long long)sm_count * (t.nt == 1 || p.D == 64 ? 2 : 1);
    t.flat = per > (items * 2 > sm_count ? 64 : items * 4 > sm_count ? 48 : 28);
    const long long worth = items * per / kMinTiles;
    t.grid = (int)(!t.flat ? items : worth < wave ? (worth < 1 ? 1 : worth) : wave);
    return t;
}

static int simt_splits(const AttnProblem &p, int sm_count) {
    const int R = p.Hq / p.Hkv * p.Sq;
    const long long items = (long long)p.B * p.Hkv * ((R + RB - 1) / RB);
    const long long units = ((long long)p.Sk + 31) / 32;
    long long s = (8LL * sm_count + items - 1) / items;
    const long long most = (units + GW - 1) / GW;   // at least one step of every warp per part
    s = s < most ? s : most;
    return (int)(s < 1 ? 1 : s > 1024 ? 1024 : s);
}

static size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

size_t kv4_attn_partial_bytes(const Kv4AttnProblem &kp, int sm_count) {
    const AttnProblem &p = kp.a;
    if (use_tc(p)) {
        const TcPlan t = tc_plan(p, sm_count);
        const size_t rows = 2 * (size_t)t.grid * 8 * t.nt;
        return t.flat ? round256(rows * p.D * sizeof(float)) + round256(rows * sizeof(float2)) : 0;
    }
    const int splits = simt_splits(p, sm_count);
    const size_t rows = (size_t)splits * p.B * p.Hq * p.Sq;
    return splits > 1 ? round256(rows * p.D * sizeof(float)) + 2 * round256(rows * sizeof(float)) : 0;
}

template <int D, int NT>
static cudaError_t launch_tc_t(Kv4AttnProblem kp, const TcPlan &t, char *partials, cudaStream_t s) {
    using C = TcCfg<D, NT>;
    const AttnProblem &p = kp.a;
    auto kernel = kp.scores ? attn_kv4_tc_kernel<D, NT, true> : attn_kv4_tc_kernel<D, NT, false>;
    cudaError_t e = set_max_dynamic_smem((const void *)kernel, (int)C::SMEM);
    if (e != cudaSuccess) return e;
    kp.part = reinterpret_cast<float *>(partials);
    kp.part_ml = reinterpret_cast<float2 *>(partials + round256(2 * (size_t)t.grid * 8 * NT * D * sizeof(float)));
    const int q_vec = (reinterpret_cast<uintptr_t>(p.q) & 15u) == 0 && ((p.q_sb | p.q_sh | p.q_ss) & 7) == 0;
    kernel<<<t.grid, TW * 32, C::SMEM, s>>>(kp, q_vec, t.row_blocks, t.flat);
    count_launches(1);
    e = cudaGetLastError();
    if (e != cudaSuccess || !t.flat) return e;
    count_launches(1);
    return launch_dependent(kv4_combine_kernel<D, NT>, dim3((unsigned)(p.B * p.Hkv * t.row_blocks)), dim3(256), 0, s, kp,
                            t.row_blocks, t.grid);
}

template <typename T>
static cudaError_t launch_general(const Kv4AttnProblem &kp, dim3 grid, cudaStream_t s) {
    const int D = kp.a.D, smem = general_smem(D);
    auto kernel = D == 96 ? attn_kv4_kernel<T, 3> : attn_kv4_kernel<T, 0>;
    if constexpr (sizeof(T) == 4) {   // (bfloat16 with these goes to the tensor cores)
        if (D == 64) kernel = attn_kv4_kernel<T, 2>;
        if (D == 128) kernel = attn_kv4_kernel<T, 4>;
    }
    const cudaError_t e = set_max_dynamic_smem((const void *)kernel, smem);
    if (e != cudaSuccess) return e;
    kernel<<<grid, GW * 32, smem, s>>>(kp);
    count_launches(1);
    return cudaGetLastError();
}

cudaError_t launch_attn_kv4(const Kv4AttnProblem &kp0, void *partials, int sm_count, cudaStream_t s) {
    Kv4AttnProblem kp = kp0;
    AttnProblem &p = kp.a;
    const int R = p.Hq / p.Hkv * p.Sq;
    cudaError_t e;
    if (use_tc(p)) {
        const TcPlan t = tc_plan(p, sm_count);
        char *at = static_cast<char *>(partials);
        e = p.D == 64 ? (t.nt == 1 ? launch_tc_t<64, 1>(kp, t, at, s) : launch_tc_t<64, 2>(kp, t, at, s))
                      : (t.nt == 1 ? launch_tc_t<128, 1>(kp, t, at, s) : launch_tc_t<128, 2>(kp, t, at, s));
    } else {
        p.splits = simt_splits(p, sm_count);
        p.keep_nan = 1;
        const size_t rows = (size_t)p.splits * p.B * p.Hq * p.Sq;
        char *at = static_cast<char *>(partials);
        p.part_acc = reinterpret_cast<float *>(at);
        p.part_m = reinterpret_cast<float *>(at + round256(rows * p.D * sizeof(float)));
        p.part_l = reinterpret_cast<float *>(at + round256(rows * p.D * sizeof(float)) + round256(rows * sizeof(float)));
        const dim3 grid((unsigned)(p.B * p.Hkv), (unsigned)p.splits, (unsigned)((R + RB - 1) / RB));
        e = p.dtype == OSF_F32 ? launch_general<float>(kp, grid, s) : launch_general<__nv_bfloat16>(kp, grid, s);
        if (e == cudaSuccess && p.splits > 1) e = launch_attn_combine(p, s);
    }
    if (e == cudaSuccess && kp.weights && p.Sk > 0) {
        count_launches(1);
        // four keys per thread where a row of scores keeps 16-byte alignment
        const int v = p.Sk % 4 == 0 ? 4 : 1;
        const dim3 grid((unsigned)((p.Sk + 256 * v - 1) / (256 * v)), (unsigned)(p.B * p.Hkv));
        e = launch_dependent(v == 4 ? kv4_weights_kernel<4> : kv4_weights_kernel<1>, grid, dim3(256), 0, s, kp);
    }
    return e;
}

}  // namespace osf
