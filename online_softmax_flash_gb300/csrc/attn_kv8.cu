// Attention over the paged 8-bit K/V cache (format: kv8.cuh): the last Sq tokens of each sequence against it, with or
// without a window and sinks.
//
// General kernel (float32 queries, which e4m3 parts do not hold, or D above 128): a CTA takes up to 4 query rows of one (b, kv
// head) and a part of the keys that they see; a warp copies the rows of 32 keys to shared memory, takes a key per lane
// (its whole dot product with the rows), then a channel of every 32 per lane.  Bound by its reads of shared memory and the
// conversions of codes, a few instructions to each four multiplications: float32, 16 sequences of 20000 tokens, 8 kv heads of 8 rows,
// D = 128, 655 MB: 515 us, 1.3 TB/s.  A short one is a chain of loads and a join: 2 sequences of 777 tokens, D = 96: 14 us.
#include "kv8.cuh"
#include "sm100_ptx.cuh"
#include "tma_host.cuh"

namespace osf {
namespace {

using namespace ptx;

constexpr int GW = 4;        // warps per CTA
constexpr int RB = 4;        // query rows per CTA
constexpr int MAXG = 8;      // D <= 256

// Tokens of a sequence's rows: position of the first and of the last row among its n tokens.
__device__ __forceinline__ KeyStream kv8_stream(const Kv8AttnProblem &kp, int n, int tile) {
    const AttnProblem &p = kp.a;
    return key_stream(n - p.Sq, n - 1, n, p.window ? p.window : n, p.sinks, tile);
}

__host__ __device__ __forceinline__ int general_smem(int D) {
    const int stage = GW * 32 * 2 * (D + 16), out = GW * RB * D * 4;   // a row's pitch: an odd number of 16-byte pieces
    return stage > out ? stage : out;
}

template <typename T>
__global__ void __launch_bounds__(GW * 32)
attn_kv8_kernel(const Kv8AttnProblem kp) {
    const AttnProblem &p = kp.a;
    const Kv8Cache &c = kp.c;
    extern __shared__ __align__(16) unsigned char stage[];   // [GW][K, V][32][D + 16]; at the end [GW][RB][D] outputs
    __shared__ __align__(16) float sq[RB][32 * MAXG];
    __shared__ __align__(16) float sp[GW][32][RB];      // weights of a warp's 32 keys, -1 where a row does not see one
    __shared__ float sm[GW][RB], sl[GW][RB];
    griddep_launch();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = p.Hq / p.Hkv, R = G * p.Sq, D = p.D, NG = D / 32, pitch = D + 16;
    const int kvbh = blockIdx.x, b = kvbh / p.Hkv, kvh = kvbh % p.Hkv;
    const int r0 = blockIdx.z * RB, rows = min(RB, R - r0);
    const int n = kv8_length(kp.lens, b, p.Sk, p.status);
    for (int i = tid; i < RB * D; i += GW * 32) {
        const int r = i / D, ch = i % D, gr = r0 + r;
        sq[r][ch] = r < rows ? to_f32(static_cast<const T *>(p.q)[q_at(p, b, kvh * G + gr / p.Sq, gr % p.Sq) + ch]) : 0.f;
    }
    __syncthreads();
    const KeyStream ks = kv8_stream(kp, n, 32);
    const int units = n > 0 ? ks.n : 0;
    const int u0 = (int)((long long)units * blockIdx.y / p.splits), u1 = (int)((long long)units * (blockIdx.y + 1) / p.splits);
    unsigned char *mine = stage + warp * 64 * pitch;
    float m[RB], l[RB], acc[RB][MAXG];
#pragma unroll
    for (int r = 0; r < RB; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.f;
#pragma unroll
        for (int g = 0; g < MAXG; ++g) acc[r][g] = 0.f;
    }
    for (int u = u0 + warp; u < u1; u += GW) {
        const int k0 = ks.tile(u) * 32, key = k0 + lane;
        // (a page that no row of the sequence sees need not be there)
        const bool wanted = key < n && (!p.window || key > n - p.Sq - p.window || key < p.sinks);
        const int page = wanted ? kv8_page(c, b, key, p.status) : -1;
        long long at = 0;
        float kscale = 0.f, vscale = 0.f;
        if (page >= 0) {
            const long long s = (long long)page * 2 * c.Hkv + kvh;
            kscale = pow2_of(kv8_exponent(c.scales[s])) * p.scale_log2;
            vscale = pow2_of(kv8_exponent(c.scales[s + c.Hkv]));
            at = (s * c.P + (key & (c.P - 1))) * D;
        }
        const long long v_off = (long long)c.Hkv * c.P * D;
        const int per = 2 * D / 16, inv = 65536 / per + 1;   // 16-byte pieces of a key: K's, then V's (i / per = i * inv >> 16)
        for (int i0 = 0; i0 < 32 * per; i0 += 32 * 8) {
            uint4 v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int i = i0 + 32 * e + lane, q = i * inv >> 16, k = q % 32, w = i - q * per;
                const long long from = __shfl_sync(0xffffffffu, at, k);
                const int have = __shfl_sync(0xffffffffu, page, k);
                v[e] = make_uint4(0, 0, 0, 0);
                if (i < 32 * per && have >= 0)
                    v[e] = *reinterpret_cast<const uint4 *>(c.pages + from + (w < per / 2 ? w * 16 : v_off + (w - per / 2) * 16));
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int i = i0 + 32 * e + lane, k = i * inv >> 16, w = i - k * per;
                if (i < 32 * per)
                    *reinterpret_cast<uint4 *>(mine + (w < per / 2 ? k * pitch + w * 16 : (32 + k) * pitch + (w - per / 2) * 16)) = v[e];
            }
        }
        __syncwarp();
        float s[RB] = {0.f, 0.f, 0.f, 0.f};
        for (int w = 0; w < D / 16; ++w) {
            const uint4 v = *reinterpret_cast<const uint4 *>(mine + lane * pitch + w * 16);
            const uint32_t x4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 lo = e4m3x2_to_f32(x4[e]), hi = e4m3x2_to_f32(x4[e] >> 16);
#pragma unroll
                for (int r = 0; r < RB; ++r) {
                    const float4 a = *reinterpret_cast<const float4 *>(&sq[r][w * 16 + e * 4]);
                    s[r] = fmaf(lo.x, a.x, s[r]); s[r] = fmaf(lo.y, a.y, s[r]);
                    s[r] = fmaf(hi.x, a.z, s[r]); s[r] = fmaf(hi.y, a.w, s[r]);
                }
            }
        }
        float pr[RB];
#pragma unroll
        for (int r = 0; r < RB; ++r) {
            const int pos = n - p.Sq + (r0 + min(r, rows - 1)) % p.Sq;
            const bool sees = r < rows && page >= 0 && key <= pos && (!p.window || key > pos - p.window || key < p.sinks);
            const float y = sees ? s[r] * kscale : -INFINITY;
            const float mx = fmaxf(m[r], warp_max(y));
            const float ref = mx == -INFINITY ? 0.f : mx;
            const float a = ex2_approx(m[r] - ref), e = ex2_approx(y - ref);
            l[r] = l[r] * a + warp_sum(e);
            pr[r] = sees ? e * vscale : -1.f;
            m[r] = mx;
#pragma unroll
            for (int g = 0; g < MAXG; ++g) acc[r][g] *= a;
        }
        *reinterpret_cast<float4 *>(sp[warp][lane]) = make_float4(pr[0], pr[1], pr[2], pr[3]);
        __syncwarp();
#pragma unroll 8
        for (int k = 0; k < 32; ++k) {   // (keys behind the last: no row sees them)
            const float4 pk4 = *reinterpret_cast<const float4 *>(sp[warp][k]);
            const float pk[RB] = {pk4.x, pk4.y, pk4.z, pk4.w};
            const unsigned char *row = mine + (32 + k) * pitch + lane;
#pragma unroll
            for (int g = 0; g < MAXG; ++g) {
                if (g >= NG) break;
                const float x = e4m3x2_to_f32(row[32 * g]).x;
#pragma unroll
                for (int r = 0; r < RB; ++r)   // a NaN value must not reach a row that does not see its key
                    acc[r][g] = pk[r] < 0.f ? acc[r][g] : fmaf(pk[r], x, acc[r][g]);
            }
        }
        __syncwarp();
    }
    __syncthreads();   // the codes are done with: their memory takes the outputs
    float *sacc = reinterpret_cast<float *>(stage);
#pragma unroll
    for (int r = 0; r < RB; ++r) {
        if (lane == 0) {
            sm[warp][r] = m[r];
            sl[warp][r] = l[r];
        }
#pragma unroll
        for (int g = 0; g < MAXG; ++g)
            if (g < NG) sacc[(warp * RB + r) * D + g * 32 + lane] = acc[r][g];
    }
    __syncthreads();
    const long long rows_total = (long long)p.B * p.Hq * p.Sq;
    for (int i = tid; i < rows * D; i += GW * 32) {
        const int r = i / D, ch = i % D, gr = r0 + r;
        float M = -INFINITY, L = 0.f, A = 0.f;
#pragma unroll
        for (int w = 0; w < GW; ++w) M = fmaxf(M, sm[w][r]);
        const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
        for (int w = 0; w < GW; ++w) {
            const float wt = ex2_approx(sm[w][r] - ref);
            A += wt * sacc[(w * RB + r) * D + ch];
            L += wt * sl[w][r];
        }
        const int hq = kvh * G + gr / p.Sq, qi = gr % p.Sq;
        const long long grow = ((long long)b * p.Hq + hq) * p.Sq + qi;
        if (p.splits == 1) {
            static_cast<T *>(p.o)[o_at(p, b, hq, qi) + ch] = from_f32<T>(L > 0.f || L != L ? A / L : 0.f);
            if (p.lse && ch == 0) p.lse[grow] = L > 0.f ? (M + __log2f(L)) * kLn2 : L != L ? L : -INFINITY;
        } else {
            p.part_acc[((size_t)blockIdx.y * rows_total + grow) * D + ch] = A;
            if (ch == 0) {
                p.part_m[(size_t)blockIdx.y * rows_total + grow] = M;
                p.part_l[(size_t)blockIdx.y * rows_total + grow] = L;
            }
        }
    }
}


// ============================================================================ tensor-core kernel
// bfloat16 queries, D up to 128 (the template's D is 64 or 128: rows of 32 and 96 channels are filled up with zeros on their
// way into shared memory).  The codes go from memory to the tensor cores as they are: TMA copies pages into shared
// memory, and tcgen05.mma (kind::f8f6f4) takes both products' large operands from there,
//   S^T[128 tokens x columns]   = K[128 x D] . Q parts^T,      O^T[D x columns] += V^T[D x 128] . P parts[128 x columns],
// so no thread touches a code but at a sequence's edges.  The small operands are sums of e4m3 parts, one column of the
// product each, the k-th part in units of 16^-k: a bfloat16 query has 8 bits, which are two parts exactly (its row scaled by
// a power of two to a largest entry in 128 .. 256; entries below 2^-14 of that lose low bits, 2^-22 of it at most).
// A token's V scale is not applied to its codes but to its weight.  Scales can lie far apart, so what goes into the
// product is 2^x with x = y + e - m', y the base-2 score, e the exponent of the scale and m' a reference of the sums y + e.  The
// denominator has its own reference m of the y.  Both references are whole numbers and move only when a value passes
// them, to 3 .. 4 above the largest.
// One reference serves all tokens and channels, but a channel's sum can be due to tokens far below it (behind a heavy key
// whose V is zero there, or a page with one large channel), so every weight keeps its 11 bits: it is rounded to float16 at one
// of four levels, level l for x in (-28 (l + 1), -28 l] (the last one: all below) in units of 2^(-15 - 28 l), and split into
// three e5m2 parts of 3 bits, which have float16's exponents (part_unit).  That is float16's rounding, 2^-11 of the weight, down
// to 2^-112 of the reference.  Each level has columns of its own, which are zeros but for warps that have weights there.
//
// A CTA takes up to NR query rows of one (b, kv head) against a run of tiles of 128 tokens.  Two warps load, two issue the
// products, and NG teams take the tiles in turn, each with its own S^T, O^T and references, one token's scores per thread;
// their states meet at the end of the run.  A team is four warps, or with 16 rows two groups of four that take 8 rows each.  A
// group's next scores are computed while it works on these: S^T is free as soon as the group has read it.  Runs are cut flat over
// all sequences (see FlatCut), and a second kernel joins the pieces of a sequence that several CTAs share.
// Up to 8 rows of D = 128 are bound by DRAM: 8 sequences of 32768 tokens, 8 kv heads of 4 rows, 537 MB: 90.5 us with launches and
// join, 5.9 TB/s (16 rows 105 us: what the groups issue for their weights; D = 64, 268 MB, 62 us: the same).  The levels
// cost these 0 to 1.5 %, filled or not, and calls of short items 1 to 2 us (128 items of 17 tiles of 16 rows 27.0 to 28.8).
constexpr int TT = 128;                   // tokens per tile
constexpr float kRowFloor = -3.4028235e38f;   // reference of a row that has seen nothing
constexpr int kMaxRing = 12;
constexpr float kHeadroom = 3.f;              // a new reference is this, and up to 1 more, above the largest
constexpr int kLevels = 4;                    // levels of weights, and the binades of one
constexpr float kLevelBits = 28.f, kLevelUnit = 0x1p-28f;

template <int D, int NR>
struct Tc8 {
    // Teams: as many as their registers allow (a thread holds the scores of RT rows).
    static constexpr int NG = NR == 4 ? 4 : NR == 8 ? 3 : 2;
    static constexpr int RT = NR == 16 ? 8 : NR, HS = NR / RT, GROUPS = NG * HS;   // rows of a thread, groups of a team
    static constexpr int W_LOAD = 4 * GROUPS, W_MMA = W_LOAD + 2, THREADS = (W_MMA + 2) * 32;
    static constexpr uint32_t TILE = TT * D;                        // K or V of a tile
    static constexpr int NQ = 2 * NR < 16 ? 16 : 2 * NR;            // columns of Q parts: part p of row r at p * NR + r
    // columns of P parts, in planes of 16: part k of row r at level l at (3 l + k) * NR + r
    static constexpr int NP = 3 * kLevels * NR, PLANES = NP / 16;
    static constexpr uint32_t Q_BYTES = 4096, P_BYTES = PLANES * TT * 16;
    static constexpr uint32_t O_BYTES = NG * NR * D * 4;
    static constexpr uint32_t Q_OFF = 0, P_OFF = Q_BYTES, O_OFF = P_OFF + NG * P_BYTES;
    static constexpr uint32_t RING_OFF = (O_OFF + O_BYTES + 1023) / 1024 * 1024;
    static constexpr int FIT = (int)((232448u - 1024u - 4096u - RING_OFF) / (2 * TILE));   // 4 KB for the static part
    static constexpr int STAGES = FIT < kMaxRing ? FIT : kMaxRing;
    static constexpr uint32_t SMEM = RING_OFF + STAGES * 2 * TILE + 1024;
    static constexpr uint32_t SWZ = D == 128 ? 2 : 4, GROUP8 = 8 * D;   // swizzle type, bytes of eight rows
    static constexpr uint32_t IDESC_S = idesc_f8_f32(TT, NQ, 0, 0, kE4M3, kE4M3);
    static constexpr uint32_t IDESC_O = idesc_f8_f32(D, NP, 1, 1, kE4M3, kE5M2);
    static constexpr uint32_t O_COL = NG * NQ, COLS = O_COL + NG * NP;   // S^T of team g at column NQ g, O^T at O_COL + NP g
    static constexpr uint32_t TMEM = COLS <= 256 ? 256 : 512;
    static_assert(COLS <= 512, "TMEM");
};

// Work is cut flat: an item is one block of query rows of one (batch, kv head), worth its tiles and `cost` more for what it
// costs besides them; the items lie one after another (batch, kv head, row block), and CTA c of nc takes the c-th part of the
// whole, whatever items it spans.  So every CTA gets the same work, in one wave, for any mix of lengths.  An item whose tiles
// all lie in one part is finished there; of the others a CTA holds at most two pieces, the end of one that began before (slot
// 2 c of the partial states) and the start of one that goes on (slot 2 c + 1).
// What an item costs: 10 tiles where a CTA has several (64 sequences of 1 to 16384 tokens, 8 kv heads of D = 128: 265 us with 0, 214
// with 3, 182 with 6, 179 with 10 and 16; 56 of up to 600 tokens and 8 of up to 16384: 132, 71, 58, 51, 58; 64 of 16384 with 16 rows,
// D = 64: 363, 285, 232, 197, 184), 3 where it has a part of one (8 items of 32 tiles: 17 us; with 10, which idles CTAs at the items'
// starts, 20).
constexpr int kMinTiles = 4;   // tiles worth a CTA (1, 2, 3, 4, 6: 8 items of 32 tiles 18, 18, 19, 17, 21 us)
struct FlatCut {
    long long total, base;   // units of all items, and of the batches before b
    int nc;                  // CTAs that take part
};
__device__ __forceinline__ KeyStream stream_of(const Kv8AttnProblem &kp, int b, int &n) {
    n = kv8_length(kp.lens, b, kp.a.Sk, kp.a.status);
    KeyStream ks = kv8_stream(kp, max(n, 1), TT);
    if (n == 0) ks.n = 0;
    return ks;
}
__device__ __forceinline__ int item_units(const Kv8AttnProblem &kp, int cost, int b) {
    int n;
    return max(1, stream_of(kp, b, n).n) + cost;
}
// Called by a whole warp.
__device__ __forceinline__ FlatCut flat_cut(const Kv8AttnProblem &kp, int cost, int items_per_b, int b, int grid) {
    const int lane = threadIdx.x & 31;
    long long all = 0, before = 0;
    for (int i = lane; i < kp.a.B; i += 32) {
        const long long n = item_units(kp, cost, i);
        all += n;
        before += i < b ? n : 0;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        all += __shfl_xor_sync(0xffffffffu, all, o);
        before += __shfl_xor_sync(0xffffffffu, before, o);
    }
    FlatCut f;
    f.total = all * items_per_b;
    f.base = before * items_per_b;
    f.nc = (int)max(1LL, min((long long)grid, f.total / (kMinTiles + cost)));
    return f;
}
// The CTA that has unit x: the last one whose part begins at or before it.
__device__ __forceinline__ int cta_of(const FlatCut &w, long long x) { return (int)(((x + 1) * w.nc - 1) / w.total); }

// A CTA's pieces, one after another.  Every warp walks them for itself.
struct Walk {
    long long rest;                              // what is left
    int b, item, unit0;
    int kvh, r0, rows, n, tile0, tiles, whole;   // the piece: tiles [tile0, tile0 + tiles) of the sequence's stream
    KeyStream ks;
};
// False when this CTA has no work.  Called by a whole warp.
__device__ __forceinline__ bool walk_begin(const Kv8AttnProblem &kp, int items_per_b, int cost, Walk &w) {
    const int lane = threadIdx.x & 31;
    w.unit0 = 0;
    if (cost == 0) {   // whole items, a CTA each
        w.b = blockIdx.x / items_per_b;
        w.item = blockIdx.x % items_per_b;
        w.rest = 1;
        return true;
    }
    const FlatCut f = flat_cut(kp, cost, items_per_b, 0, gridDim.x);
    if ((int)blockIdx.x >= f.nc) return false;
    const long long pos = f.total * blockIdx.x / f.nc;
    w.rest = f.total * (blockIdx.x + 1) / f.nc - pos;
    long long at = 0;   // units before batch b: 32 batches at a time, a lane each
    for (int b0 = 0;; b0 += 32) {
        const int bi = b0 + lane;
        const long long ub = bi < kp.a.B ? (long long)item_units(kp, cost, bi) * items_per_b : 0;
        long long upto = ub;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, pos < at + upto);
        if (past) {
            const int first = __ffs(past) - 1;
            w.b = b0 + first;
            at += __shfl_sync(0xffffffffu, upto - ub, first);
            break;
        }
        at += __shfl_sync(0xffffffffu, upto, 31);
    }
    const int ui = item_units(kp, cost, w.b);
    w.item = (int)((pos - at) / ui);
    w.unit0 = (int)((pos - at) % ui);
    return true;
}
// The next piece; false behind the last one.
template <int NR>
__device__ __forceinline__ bool walk_next(const Kv8AttnProblem &kp, int row_blocks, int cost, Walk &w) {
    if (w.rest <= 0) return false;
    const AttnProblem &p = kp.a;
    w.ks = stream_of(kp, w.b, w.n);
    const int all = max(1, w.ks.n), units = all + cost;   // the item's first cost units hold no tiles
    const int take = cost ? (int)min((long long)(units - w.unit0), w.rest) : units;
    w.tile0 = max(0, w.unit0 - cost);
    const int tile1 = w.unit0 + take - cost;
    if (tile1 <= w.tile0) {   // the part ends before the item's first tile
        w.rest = 0;
        return false;
    }
    w.whole = tile1 - w.tile0 == all;
    w.tiles = min(tile1, w.ks.n) - w.tile0;   // (an empty sequence has a tile's unit, and no tile)
    w.kvh = w.item / row_blocks;
    w.r0 = w.item % row_blocks * NR;
    w.rows = min(NR, p.Hq / p.Hkv * p.Sq - w.r0);
    w.rest = cost ? w.rest - take : 0;
    w.unit0 = 0;
    return true;
}
__device__ __forceinline__ void walk_step(const Kv8AttnProblem &kp, int row_blocks, Walk &w) {
    if (++w.item == kp.a.Hkv * row_blocks) {
        w.item = 0;
        ++w.b;
    }
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

struct Tc8Bars {
    uint64_t full[kMaxRing], empty[kMaxRing], s_full[4], s_free[4], p_full[4], pv_done[4], q_full, drain[2];
};

// x * 2^d for a whole d in -254 .. 254.
__device__ __forceinline__ float scale_by(float x, int d) { return x * pow2_of(d / 2) * pow2_of(d - d / 2); }

// The maxima over a warp of each of N values (N a power of two up to 32): v[0] becomes the maximum of the value whose index
// is returned.  Every step halves the values that a lane still follows.
template <int N>
__device__ __forceinline__ int warp_max_each(float (&v)[N]) {
    const int lane = threadIdx.x & 31;
    int at = 0;
#pragma unroll
    for (int s = 16, n = N; s > 0; s >>= 1) {
        if (n > 1) {
            n >>= 1;
            const bool hi = lane & s;
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                if (i >= n) break;
                const float keep = hi ? v[i + n] : v[i], send = hi ? v[i] : v[i + n];
                v[i] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, send, s));
            }
            at = 2 * at + hi;
        } else {
            v[0] = fmaxf(v[0], __shfl_xor_sync(0xffffffffu, v[0], s));
        }
    }
    return at;
}

template <int N>
__device__ __forceinline__ void tmem_ld_n(uint32_t addr, uint32_t (&r)[N]) {
    if constexpr (N == 8) tmem_ld8(addr, r);
    else if constexpr (N == 16) tmem_ld16(addr, r);
    else tmem_ld32(addr, r);
}

// Units of the e5m2 parts of a float16 weight.  The first has 3 of its 11 bits; what is left is at most 2^-3 of its binade, and
// after the second part at most 2^-7, a whole number of the float16's last places up to 8: so in these units the parts lie in
// e5m2's range, and the third is exact, for weights of 2^-13 and more.
__device__ __forceinline__ constexpr float part_unit(int k) { return k == 0 ? 1.f : k == 1 ? 0x1p-3f : 0x1p-8f; }
// A token's weights of RT rows at level lv, split into parts, to its row of P.
template <int NR, int RT>
__device__ __forceinline__ void store_parts(uint32_t p_row, int lv, const uint32_t (&w)[RT / 2]) {
    uint32_t part[3][RT / 4];   // words of four rows
#pragma unroll
    for (int r = 0; r < RT / 2; ++r) {
        uint32_t h = w[r];
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const uint32_t x = f16x2_to_e5m2x2(h);
            if (r % 2 == 0) part[k][r / 2] = x;
            else part[k][r / 2] |= x << 16;
            if (k < 2) h = f16x2_rest(h, e5m2x2_to_f16x2(x), k == 0 ? 0x48004800u : 0x50005000u);   // times 2^3, 2^5
        }
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        // (16 rows: a plane to a part, and p_row says which half)
        const int word = NR == RT ? (3 * lv + k) * (RT / 4) : 4 * (3 * lv + k);
        const uint32_t at = p_row + (word >> 2) * (TT * 16) + (word & 3) * 4;
        if constexpr (RT == 4) asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(part[k][0]) : "memory");
        else asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at), "r"(part[k][0]), "r"(part[k][1]) : "memory");
    }
}

// FLAT: cut flat, or whole items (one kernel for both: 128 items of 128 tiles of 16 rows, D = 64, 95 us against 87).
template <int D, int NR, bool FLAT>
__global__ void __launch_bounds__((Tc8<D, NR>::THREADS), 1)
attn_kv8_tc_kernel(const __grid_constant__ CUtensorMap mpages, const Kv8AttnProblem kp, int q_vec, int row_blocks, int item_cost) {
    const int cost = FLAT ? item_cost : 0;   // 0: whole items, a CTA each
    using C = Tc8<D, NR>;
    constexpr int NG = C::NG, RT = C::RT, HS = C::HS, SOFT = 128 * C::GROUPS;
    const AttnProblem &p = kp.a;
    const Kv8Cache &c = kp.c;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Tc8Bars bars;
    __shared__ uint32_t tmem_sh;
    __shared__ volatile int abort_flag;
    __shared__ __align__(16) float q_back[NR];             // raw score times K scale to base-2 score
    __shared__ int row_pos[NR];                            // positions of the rows
    __shared__ float red[C::GROUPS][4][2 * RT];                  // maxima of a group's warps: of y, then of y + e
    __shared__ __align__(16) float ref[C::GROUPS][2 * RT], fac[C::GROUPS][2 * RT];   // references m, m', and what moves to them
    __shared__ float sum_l[C::GROUPS][4][RT];
    __shared__ uint32_t poison[NR][D / 32];   // channels that a NaN value reaches
    __shared__ volatile int below[C::GROUPS];  // whether a group has had weights behind the first level in this piece
    griddep_launch();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint8_t *sgen = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = smem_u32(sgen);
    const uint32_t sQ = sbase + C::Q_OFF, sP = sbase + C::P_OFF, sRing = sbase + C::RING_OFF;
    const int G = p.Hq / p.Hkv, items_per_b = p.Hkv * row_blocks;

    if (warp == 0) tmem_alloc(smem_u32(&tmem_sh), C::TMEM);
    if (tid == 32) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(smem_u32(&bars.full[s]), 2);   // the K and the V loads
            mbar_init(smem_u32(&bars.empty[s]), 1);
        }
        for (int g = 0; g < NG; ++g) {
            mbar_init(smem_u32(&bars.s_full[g]), 1);
            mbar_init(smem_u32(&bars.s_free[g]), 4 * HS);
            mbar_init(smem_u32(&bars.p_full[g]), 4 * HS);
            mbar_init(smem_u32(&bars.pv_done[g]), 1);
        }
        mbar_init(smem_u32(&bars.q_full), 4 * C::GROUPS);
        mbar_init(smem_u32(&bars.drain[0]), 1);
        mbar_init(smem_u32(&bars.drain[1]), 1);
        abort_flag = 0;
        mbar_init_fence();
    }
    // unused columns of Q, and the levels of P that no weight is at
    for (int i = tid; i < (int)C::O_OFF / 16; i += C::THREADS) st_shared_v4(sQ + 16 * i, 0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_sh;
    Walk w;
    bool live = walk_begin(kp, items_per_b, cost, w);

    if (warp >= C::W_LOAD && warp < C::W_MMA) {
        // ================================================================ loads: K and V, a lane per page of the tile
        // (one warp for both: 820 cycles a tile, more than its bytes take at D = 64)
        const int half = warp - C::W_LOAD, per_tile = TT >> c.log2_p;
        const int rows_total = c.n_pages * 2 * c.Hkv * c.P;
        tma_prefetch_desc(&mpages);
        bool ok = true;
        int st = 0;
        uint32_t par = 1;
        while (ok && live && walk_next<NR>(kp, row_blocks, cost, w)) {
            // whether some row sees this lane's page of the piece's tile i, and the table's entry for it
            const int near = p.window ? w.n - p.Sq - p.window : -c.P;   // the window of the first row begins behind it
            const int *entries = c.table + (long long)w.b * c.per_seq;
            auto token_of = [&](int i) { return w.ks.tile(w.tile0 + i) * TT + (lane << c.log2_p); };
            auto wanted = [&](int i, int tok) {
                return i < w.tiles && lane < per_tile && tok < w.n && (tok + c.P - 1 > near || tok < p.sinks);
            };
            auto entry_of = [&](int i, int tok) { return wanted(i, tok) ? entries[tok >> c.log2_p] : 0; };
            int tok = token_of(0), tok1 = token_of(1), next = entry_of(0, tok), next1 = entry_of(1, tok1);
            for (int i = 0; i < w.tiles; ++i) {
                const int entry = next, tok2 = token_of(i + 2);
                const bool want = wanted(i, tok);
                next = next1;
                next1 = entry_of(i + 2, tok2);
                tok = tok1;
                tok1 = tok2;
                const int page = want ? kv8_checked(c, entry, p.status) : -1;
                // first row of the page; past the end (zeros) where there is none
                const int row = page < 0 ? rows_total : ((page * 2 + half) * c.Hkv + w.kvh) << c.log2_p;
                ok = mbar_wait(smem_u32(&bars.empty[st]), par, &abort_flag);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                const uint32_t bar = smem_u32(&bars.full[st]);
                if (lane == 0) mbar_expect_tx(bar, C::TILE);
                __syncwarp();
                if (lane < per_tile)
                    tma_load_2d(sRing + (2 * st + half) * C::TILE + (lane << c.log2_p) * D, &mpages, bar, 0, row);
                if (++st == C::STAGES) {
                    st = 0;
                    par ^= 1;
                }
            }
            walk_step(kp, row_blocks, w);
        }
        if (!ok) {
            abort_flag = 1;
            if (lane == 0) atomicExch(p.status, kStatusTimeout);
            const uint64_t t0 = globaltimer_ns();   // copies in flight land
            while (globaltimer_ns() - t0 < 50000ull) {
            }
        }
    } else if (warp >= C::W_MMA) {
        // ================================================================ products
        // Two issuers, the scores' and the values': a product takes 66 cycles whatever its layout (128 bytes x 32 of its large
        // operand from shared memory), so what one thread does around them is as much as they take (one issuer for both:
        // 1300 cycles a tile, of which the products 400 at D = 64).
        const bool is_s = warp == C::W_MMA;
        bool ok = true;
        int st = 0, g = 0;                           // stage and group of the next tile,
        uint32_t st_par = 0, g_par = 0, q_par = 0;   // and the parities of their barriers
        bool again = false;                          // the groups have had a tile each
        while (ok && live && walk_next<NR>(kp, row_blocks, cost, w)) {
            if (lane == 0 && w.tiles > 0) {
                if (is_s) ok = mbar_wait(smem_u32(&bars.q_full), q_par, &abort_flag);
                q_par ^= 1;
                const uint64_t qd = sdesc_any(sQ, 16, C::GROUP8, C::SWZ), pd0 = sdesc_any(sP, 128, TT * 16, 0);
                const uint64_t kd0 = sdesc_any(sRing, 16, C::GROUP8, C::SWZ);
                for (int i = 0; i < w.tiles && ok; ++i) {
                    const uint64_t kd = kd0 + st * (2 * C::TILE / 16);
                    if (is_s) {   // S^T, once its group has read the one before
                        if (again) ok = mbar_wait_spin(smem_u32(&bars.s_free[g]), g_par ^ 1, &abort_flag);
                        ok = ok && mbar_wait_spin(smem_u32(&bars.full[st]), st_par, &abort_flag);
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll
                        for (int k = 0; k < D / 32; ++k) mma_ss_f8(tmem + C::NQ * g, kd + 2 * k, qd + 2 * k, C::IDESC_S, k > 0);
                        mma_commit(smem_u32(&bars.s_full[g]));
                    } else {      // O^T, once its group has its weights; the stage is free when it is done
                        ok = mbar_wait_spin(smem_u32(&bars.p_full[g]), g_par, &abort_flag);
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t vd = kd + C::TILE / 16, pd = pd0 + g * (C::P_BYTES / 16);
#pragma unroll
                        for (int k = 0; k < TT / 32; ++k)
                            mma_ss_f8(tmem + C::O_COL + C::NP * g, vd + k * (4 * C::GROUP8 / 16), pd + k * (512 / 16), C::IDESC_O,
                                      i >= NG || k > 0);
                        mma_commit(smem_u32(&bars.pv_done[g]));
                        mma_commit(smem_u32(&bars.empty[st]));
                    }
                    if (++st == C::STAGES) {
                        st = 0;
                        st_par ^= 1;
                    }
                    if (++g == NG) {
                        g = 0;
                        g_par ^= 1;
                        again = true;
                    }
                }
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
            walk_step(kp, row_blocks, w);
        }
        if (lane == 0) {
            if (!ok) {
                abort_flag = 1;
                atomicExch(p.status, kStatusTimeout);
            }
            const uint32_t dr = smem_u32(&bars.drain[is_s ? 0 : 1]);
            mma_commit(dr);
            mbar_wait(dr, 0, nullptr, 20000000ull);
        }
        __syncwarp();
    } else {
        // ================================================================ scores to weights
        const int gi = warp >> 2, g = gi / HS, rh = gi % HS * RT;   // group, team, and the group's first row
        const int w4 = warp & 3, r128 = tid & 127;
        const uint32_t lane_off = (uint32_t)(w4 * 32) << 16;
        const uint32_t s_addr = tmem + C::NQ * g + rh + lane_off, o_addr = tmem + C::O_COL + C::NP * g + rh + lane_off;
        const uint32_t p_row = sP + g * C::P_BYTES + r128 * 16 + rh;
        // a wait that ran out is told to the whole group at its next vote, so that all leave together
        bool failed = false;
        bool deep = false;   // whether this warp's rows of P hold weights behind the first level
        int gt = 0;   // tiles of the CTA so far; tile t is its team's t / NG-th
        while (live && walk_next<NR>(kp, row_blocks, cost, w)) {
            // ------------------------------------------------------------ Q parts: a warp per row
            for (int r = warp; r < NR; r += 4 * C::GROUPS) {
                constexpr int E = D / 32;   // channels E * lane .., zeros from p.D on
                const int gr = w.r0 + r;
                float x[E], mx = 0.f;
                bool bad = false;
#pragma unroll
                for (int e = 0; e < E; ++e) x[e] = 0.f;
                if (r < w.rows && E * lane < p.D) {
                    const __nv_bfloat16 *Q = static_cast<const __nv_bfloat16 *>(p.q) +
                                             q_at(p, w.b, w.kvh * G + gr / p.Sq, gr % p.Sq) + E * lane;
                    if (q_vec) {
#pragma unroll
                        for (int e = 0; e < E; e += 2) {
                            const uint32_t v = *reinterpret_cast<const uint32_t *>(Q + e);
                            x[e] = __uint_as_float(v << 16);
                            x[e + 1] = __uint_as_float(v & 0xffff0000u);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < E; ++e) x[e] = __bfloat162float(Q[e]);
                    }
                }
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    mx = fmaxf(mx, fabsf(x[e]));
                    bad |= !(fabsf(x[e]) <= 3.4028235e38f);
                }
                mx = warp_max(mx);
                bad = __any_sync(0xffffffffu, bad);
                const int ex = min(119, 7 - ((int)(__float_as_uint(mx) >> 23) - 127));   // -120 at least (larger is not finite)
                const float up = pow2_of(ex);
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    const int col = part * NR + r;
                    uint32_t word = 0;
#pragma unroll
                    for (int e = 0; e < E; e += 2) {
                        const float a = x[e] * (part ? 16.f : up), b2 = x[e + 1] * (part ? 16.f : up);
                        const uint32_t k = bad ? 0x7f7fu : f32_to_e4m3x2(a, b2);
                        const float2 f = e4m3x2_to_f32(k);
                        x[e] = a - f.x;          // what is left, for the next part
                        x[e + 1] = b2 - f.y;
                        word |= k << (8 * e);
                    }
                    const uint32_t byte = E * lane, piece = byte >> 4;
                    const uint32_t at = sQ - sbase + col * D + ((D == 128 ? piece ^ (col & 7) : piece ^ (col >> 1 & 3)) << 4) + (byte & 15);
                    if (E == 4) *reinterpret_cast<uint32_t *>(sgen + at) = word;
                    else *reinterpret_cast<uint16_t *>(sgen + at) = (uint16_t)word;
                }
                if (lane == 0) {
                    q_back[r] = pow2_of(-ex) * p.scale_log2;
                    row_pos[r] = w.n - p.Sq + gr % p.Sq;
                }
            }
            for (int i = tid; i < NR * (D / 32); i += SOFT) poison[i / (D / 32)][i % (D / 32)] = 0;
            if (r128 < 2 * RT) ref[gi][r128] = kRowFloor;
            if (r128 == 0) below[gi] = 0;
            fence_proxy_async_smem();
            named_barrier(1, SOFT);
            // (a piece without tiles waits for no product, so several could pass while the issuer sleeps: they are not counted)
            if (lane == 0 && w.tiles > 0) mbar_arrive(smem_u32(&bars.q_full));

            float m[RT], mp[RT], l[RT];   // -m, -m' and this thread's part of the denominator
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                m[r] = mp[r] = -kRowFloor;
                l[r] = 0.f;
            }
            // whether some row sees this thread's token of the piece's tile i, and the table's entry for it; its page's scales
            const int near = p.window ? w.n - p.Sq - p.window : -1;   // the window of the first row begins behind it
            const int *entries = c.table + (long long)w.b * c.per_seq;
            auto token_of = [&](int i) { return w.ks.tile(w.tile0 + i) * TT + r128; };
            auto wanted = [&](int i) {
                const int key = token_of(i);
                return i < w.tiles && key < w.n && (key > near || key < p.sinks);
            };
            auto entry_of = [&](int i) { return wanted(i) ? entries[token_of(i) >> c.log2_p] : 0; };
            auto scales_of = [&](int page, float &a, float &b) {
                a = b = 1.f;
                if (page < 0) return;
                const float *s = c.scales + (long long)page * 2 * c.Hkv + w.kvh;
                a = s[0];
                b = s[c.Hkv];
            };
            // this team's tiles of the piece, the pages of the next two and the scales of the next in flight
            int i = (g + NG - gt % NG) % NG, done = (gt + i) / NG, taken = 0;   // done: this team's tiles before it
            int entry1 = entry_of(i + NG), page = entry_of(i);
            page = wanted(i) ? kv8_checked(c, page, p.status) : -1;
            float ks, vs;
            scales_of(page, ks, vs);
            for (; i < w.tiles; i += NG) {
                const int entry2 = entry_of(i + 2 * NG), page1 = wanted(i + NG) ? kv8_checked(c, entry1, p.status) : -1;
                float ks1, vs1;
                scales_of(page1, ks1, vs1);
                const int tile = w.ks.tile(w.tile0 + i), key0 = tile * TT, key = key0 + r128;
                const int st = (gt + i) % C::STAGES;
                bool ok = !failed && mbar_wait(smem_u32(&bars.s_full[g]), done & 1, &abort_flag);
                failed = !__all_sync(0xffffffffu, ok);
                tc_fence_after();
                uint32_t raw[2 * RT];   // the first parts' scores, then the second's
                if constexpr (HS == 1) {
                    tmem_ld_n(s_addr, raw);
                } else {
                    tmem_ld8(s_addr, raw);
                    tmem_ld8(s_addr + NR, raw + RT);
                }
                tmem_ld_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bars.s_free[g]));
                const float kscale = pow2_of(kv8_exponent(ks)), ev = (float)kv8_exponent(vs), ev15 = ev + 15.f;
                float y[RT];
#pragma unroll
                for (int r = 0; r < RT; r += 4) {
                    const float4 back = *reinterpret_cast<const float4 *>(q_back + rh + r);
                    const float qb[4] = {back.x, back.y, back.z, back.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        y[r + e] = fmaf(__uint_as_float(raw[RT + r + e]), 0.0625f, __uint_as_float(raw[r + e])) * (qb[e] * kscale);
                }
                // a tile that some row does not see the whole of
                const bool edge = key0 + TT - 1 > w.n - p.Sq || (p.window && key0 <= w.n - 1 - p.window && key0 + TT > p.sinks);
                if (edge) {
                    auto sees = [&](int pos) {
                        return page >= 0 && key <= pos && (!p.window || key > pos - p.window || key < p.sinks);
                    };
#pragma unroll
                    for (int r = 0; r < RT; ++r) y[r] = sees(row_pos[rh + r]) ? y[r] : -INFINITY;
                    // Values of tokens that no row sees, or not all, must not reach the others as 0 * NaN: the former are
                    // cleared, the latter's NaN codes too, and remembered for the rows that do see them.
                    bool all = true;
                    if (rh == 0)
                        for (int r = 0; r < w.rows; ++r) all = all && sees(row_pos[r]);
                    if (!all && !failed) {
                        const uint32_t vrow = sRing + st * 2 * C::TILE + C::TILE + r128 * D;
                        if (mbar_wait(smem_u32(&bars.full[st]), ((gt + i) / C::STAGES) & 1, &abort_flag)) {
#pragma unroll 1
                            for (int q = 0; q < D / 16; ++q) {
                                const uint32_t at = vrow + 16 * q;
                                if (page < 0) {
                                    st_shared_v4(at, 0u, 0u, 0u, 0u);
                                    continue;
                                }
                                const uint4 v = ld_shared_v4(at);
                                uint32_t x[4] = {v.x, v.y, v.z, v.w}, nan_any = 0, bits = 0;
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    // top bit of each byte whose other seven are all set
                                    const uint32_t nan = ((x[e] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                                    nan_any |= nan;
                                    bits |= ((nan >> 7 & 1u) | (nan >> 14 & 2u) | (nan >> 21 & 4u) | (nan >> 28 & 8u)) << (4 * e);
                                    x[e] &= ~((nan >> 7) * 0xffu);
                                }
                                if (!nan_any) continue;
                                st_shared_v4(at, x[0], x[1], x[2], x[3]);
                                const int ch = 16 * (D == 128 ? q ^ (r128 & 7) : q ^ (r128 >> 1 & 3));
                                for (int r = 0; r < w.rows; ++r)
                                    if (sees(row_pos[r])) atomicOr(&poison[r][ch / 32], bits << (ch & 31));
                            }
                        }
                    }
                } else if (page < 0) {   // the table holds no page for it: its codes are zeros
#pragma unroll
                    for (int r = 0; r < RT; ++r) y[r] = -INFINITY;
                }
                float top = -INFINITY;
#pragma unroll
                for (int r = 0; r < RT; ++r) top = fmax3(top, y[r] + m[r], y[r] + (mp[r] + ev));
                if (named_barrier_or(2 + gi, 128, failed || top > 0.f)) {
                    // some reference has to move
                    float v[2 * RT];
#pragma unroll
                    for (int r = 0; r < RT; ++r) {
                        v[r] = y[r];
                        v[RT + r] = y[r] + ev;
                    }
                    const int at = warp_max_each(v);
                    if ((lane & (32 / (2 * RT) - 1)) == 0) red[gi][w4][at] = v[0];
                    if (named_barrier_or(2 + gi, 128, failed)) {
                        failed = true;
                        break;
                    }
                    if (r128 < 2 * RT) {
                        const float a = fmaxf(fmaxf(red[gi][0][r128], red[gi][1][r128]), fmaxf(red[gi][2][r128], red[gi][3][r128]));
                        const float old = ref[gi][r128], now = a > old ? ceilf(a) + kHeadroom : old;
                        fac[gi][r128] = ex2_approx(old - now);
                        ref[gi][r128] = now;
                    }
                    named_barrier(2 + gi, 128);
                    float f[RT];
#pragma unroll
                    for (int r = 0; r < RT; ++r) {
                        l[r] *= fac[gi][r];
                        f[r] = fac[gi][RT + r];
                        m[r] = -ref[gi][r];
                        mp[r] = -ref[gi][RT + r];
                    }
                    if (taken > 0) {   // (every product of the group so far is waited for first)
                        ok = mbar_wait(smem_u32(&bars.pv_done[g]), (done - 1) & 1, &abort_flag);
                        failed = !__all_sync(0xffffffffu, ok);
                        tc_fence_after();
                        const int levels = below[gi] ? kLevels : 1;   // (of earlier tiles: seen since the barrier)
                        if constexpr (HS == 1) {
#pragma unroll 1
                            for (int pl = 0; pl < (levels * 3 * NR + 15) / 16; ++pl) {
                                uint32_t o[16];
                                tmem_ld16(o_addr + 16 * pl, o);
                                tmem_ld_wait();
#pragma unroll
                                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f[e % NR]);
                                tmem_st16(o_addr + 16 * pl, o[0], o[1], o[2], o[3], o[4], o[5], o[6], o[7], o[8], o[9], o[10],
                                          o[11], o[12], o[13], o[14], o[15]);
                            }
                        } else {
#pragma unroll 1
                            for (int k = 0; k < 3 * levels; ++k) {
                                uint32_t o[8];
                                tmem_ld8(o_addr + NR * k, o);
                                tmem_ld_wait();
#pragma unroll
                                for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f[e % RT]);
                                tmem_st8(o_addr + NR * k, o);
                            }
                        }
                        tmem_st_wait();
                    }
                }
                // weights in float16, and the smallest of them
                uint32_t h[RT / 2], low = 0x7bff7bffu;
#pragma unroll
                for (int r = 0; r < RT; r += 2) {
                    l[r] += ex2_approx(y[r] + m[r]);
                    l[r + 1] += ex2_approx(y[r + 1] + m[r + 1]);
                    h[r / 2] = f32_to_f16x2(ex2_approx(y[r] + (mp[r] + ev15)), ex2_approx(y[r + 1] + (mp[r + 1] + ev15)));
                    low = f16x2_min(low, h[r / 2]);
                }
                // the product that read the last weights is done
                if (done > 0) {
                    ok = !failed && mbar_wait(smem_u32(&bars.pv_done[g]), (done - 1) & 1, &abort_flag);
                    failed = !__all_sync(0xffffffffu, ok);
                }
                // weights below the first level (hidden ones look like those at first)
                constexpr uint32_t kLowest = 0x0800u;   // float16 2^(15 - kLevelBits)
                if (__any_sync(0xffffffffu, deep || (low & 0xffffu) < kLowest || low >> 16 < kLowest)) {
                    bool any = false;
#pragma unroll
                    for (int r = 0; r < RT; ++r) {
                        const float x = y[r] + (mp[r] + ev);
                        any |= x <= -kLevelBits && x > -125.f;   // (2^-125 of the reference is nothing at the last level either)
                    }
                    any = __any_sync(0xffffffffu, any);
                    if (any || deep) {
#pragma unroll 1
                        for (int lv = 0; lv < kLevels; ++lv) {
                            const float from = -kLevelBits * lv, to = lv == kLevels - 1 ? -INFINITY : from - kLevelBits;
                            uint32_t w[RT / 2];
#pragma unroll
                            for (int r = 0; r < RT; r += 2) {
                                float v[2];
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    const float x = y[r + e] + (mp[r + e] + ev);
                                    // (a NaN is at the first level)
                                    const bool here = (lv == 0 || x <= from) && !(x <= to);
                                    v[e] = here ? ex2_approx(x - from + 15.f) : 0.f;
                                }
                                w[r / 2] = f32_to_f16x2(v[0], v[1]);
                            }
                            if (lv == 0) {
#pragma unroll
                                for (int r = 0; r < RT / 2; ++r) h[r] = w[r];
                            } else {
                                store_parts<NR, RT>(p_row, lv, w);
                            }
                        }
                    }
                    deep = any;
                    if (any && lane == 0) below[gi] = 1;
                }
                store_parts<NR, RT>(p_row, 0, h);
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bars.p_full[g]));
                ++done;
                ++taken;
                page = page1; entry1 = entry2;
                ks = ks1; vs = vs1;
            }
            // ------------------------------------------------------------ the groups' states meet
            float *so = reinterpret_cast<float *>(sgen + C::O_OFF);   // [NG][NR][D]
            if (taken > 0 && !failed) {
                const bool ok = mbar_wait(smem_u32(&bars.pv_done[g]), (done - 1) & 1, &abort_flag);
                failed = !__all_sync(0xffffffffu, ok);
            }
            tc_fence_after();
            // the sums of the levels that are not zero, each three parts: in units of 2^(m' - 15)
            named_barrier(2 + gi, 128);
            const int top_level = below[gi] ? kLevels - 1 : 0;
            float sum_o[RT];
#pragma unroll
            for (int r = 0; r < RT; ++r) sum_o[r] = 0.f;
#pragma unroll 1
            for (int lv = top_level; lv >= 0; --lv) {
                uint32_t o[3 * RT];   // part k of row r at k * RT + r
                if constexpr (NR == 4) {
                    tmem_ld8(o_addr + 3 * NR * lv, o);
                    tmem_ld4(o_addr + 3 * NR * lv + 8, o + 8);
                } else if constexpr (NR == 8) {
                    tmem_ld16(o_addr + 3 * NR * lv, o);
                    tmem_ld8(o_addr + 3 * NR * lv + 16, o + 16);
                } else {
#pragma unroll
                    for (int k = 0; k < 3; ++k) tmem_ld8(o_addr + NR * (3 * lv + k), o + RT * k);
                }
                tmem_ld_wait();
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const float v = fmaf(__uint_as_float(o[2 * RT + r]), part_unit(2),
                                         fmaf(__uint_as_float(o[RT + r]), part_unit(1), __uint_as_float(o[r])));
                    sum_o[r] = fmaf(sum_o[r], kLevelUnit, v);
                }
            }
            tc_fence_before();
            const int ch = D == 128 ? r128 : w4 * 16 + lane;   // M = 64: 16 lanes of each warp's 32
            const bool mine = D == 128 || lane < 16;
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const float sum = warp_sum(l[r]);
                if (lane == 0) sum_l[gi][w4][r] = sum;
                // relative to m
                const float v = taken > 0 ? scale_by(sum_o[r] * 0x1p-15f, (int)fmaxf(-250.f, fminf(250.f, m[r] - mp[r]))) : 0.f;
                if (mine) so[(g * NR + rh + r) * D + ch] = v;
            }
            named_barrier(1, SOFT);
            const size_t slot = 2 * (size_t)blockIdx.x + (w.tile0 == 0 ? 1 : 0);
            for (int x = tid; x < w.rows * (D / 4); x += SOFT) {
                const int r = x / (D / 4), c4 = x % (D / 4) * 4, gr = w.r0 + r;
                float M = -INFINITY, L = 0.f, mg[NG], lg[NG];
                float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int e = 0; e < NG; ++e) {
                    const int ge = e * HS + r / RT, re = r % RT;
                    lg[e] = (sum_l[ge][0][re] + sum_l[ge][1][re]) + (sum_l[ge][2][re] + sum_l[ge][3][re]);
                    mg[e] = lg[e] > 0.f || lg[e] != lg[e] ? ref[ge][re] : -INFINITY;
                    M = fmaxf(M, mg[e]);
                }
                const float base = M == -INFINITY ? 0.f : M;
#pragma unroll
                for (int e = 0; e < NG; ++e) {
                    const float wt = ex2_approx(mg[e] - base);
                    const float4 v = *reinterpret_cast<const float4 *>(so + (e * NR + r) * D + c4);
                    A.x = fmaf(wt, v.x, A.x); A.y = fmaf(wt, v.y, A.y);
                    A.z = fmaf(wt, v.z, A.z); A.w = fmaf(wt, v.w, A.w);
                    L = fmaf(wt, lg[e], L);
                }
                const uint32_t nan = poison[r][c4 / 32] >> (c4 & 31);
                if (nan & 15u) {
                    if (nan & 1u) A.x = NAN;
                    if (nan & 2u) A.y = NAN;
                    if (nan & 4u) A.z = NAN;
                    if (nan & 8u) A.w = NAN;
                }
                if (w.whole) {
                    if (c4 < p.D) write_row(p, w.b, w.kvh * G + gr / p.Sq, gr % p.Sq, c4, A, M, L);
                } else {
                    *reinterpret_cast<float4 *>(kp.part + (slot * NR + r) * D + c4) = A;
                    if (c4 == 0) kp.part_ml[slot * NR + r] = make_float2(M, L);
                }
            }
            gt += w.tiles;
            walk_step(kp, row_blocks, w);
            if (named_barrier_or(1, SOFT, failed)) {   // (and the buffers are free again)
                failed = true;
                break;
            }
        }
        if (failed) {
            abort_flag = 1;
            if (lane == 0) atomicExch(p.status, kStatusTimeout);
        }
    }
    tc_fence_before();
    __syncwarp();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM);
    }
}

// Rows of the items that several CTAs shared, joined; the same cut of the work as above.  gridDim = (items, parts of their
// rows): a block takes `rpb` rows of an item, four channels to a thread, and the groups of threads that are left take the pieces
// in turn, KG at a time (one sequence of 100000 tokens in 152 pieces: 43 us with the pieces one round after another).
template <int D, int NR>
__global__ void __launch_bounds__(256) kv8_combine_kernel(const Kv8AttnProblem kp, int row_blocks, int grid, int cost, int rpb) {
    __shared__ float4 sA[256];
    __shared__ float2 sML[256];
    const AttnProblem &p = kp.a;
    const int G = p.Hq / p.Hkv, R = G * p.Sq, items_per_b = p.Hkv * row_blocks;
    const int b = blockIdx.x / items_per_b, item = blockIdx.x % items_per_b;
    const FlatCut w = flat_cut(kp, cost, items_per_b, b, grid);
    const int ui = item_units(kp, cost, b);
    const long long p0 = w.base + (long long)item * ui;
    const int c0 = cta_of(w, p0 + cost), c1 = cta_of(w, p0 + ui - 1);   // CTAs of the first and the last tile
    griddep_wait();
    if (c0 == c1) return;
    const int r0 = item % row_blocks * NR, rows = min(NR, R - r0);
    constexpr int KG = 8;   // pieces whose states are loaded together
    const int per = rpb * (D / 4), groups = per < 256 ? 256 / per : 1, g = threadIdx.x / per;   // (rpb, D: powers of two)
    for (int x = threadIdx.x % per; x < per; x += 256) {
        const int r = blockIdx.y * rpb + x / (D / 4), c = x % (D / 4) * 4, gr = r0 + r;
        const bool mine = r < rows && c < p.D;
        float M = -INFINITY, L = 0.f;
        float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k0 = c0 + g * KG; mine && k0 <= c1; k0 += groups * KG) {
            float2 ml[KG];
            float4 v[KG];
            float mx = M;
#pragma unroll
            for (int e = 0; e < KG; ++e) {
                const size_t slot = 2 * (size_t)min(k0 + e, c1) + (k0 + e == c0 ? 1 : 0);
                ml[e] = k0 + e <= c1 ? kp.part_ml[slot * NR + r] : make_float2(-INFINITY, 0.f);
                v[e] = k0 + e <= c1 ? *reinterpret_cast<const float4 *>(kp.part + (slot * NR + r) * D + c)
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
        if (groups > 1 && c1 - c0 + 1 > KG) {   // the groups' sums, in their order
            sA[threadIdx.x] = A;
            sML[threadIdx.x] = make_float2(M, L);
            __syncthreads();
            if (g > 0) return;
            for (int e = 1; e < groups; ++e) M = fmaxf(M, sML[e * per + x].x);
            const float ref = M == -INFINITY ? 0.f : M;
            A = make_float4(0.f, 0.f, 0.f, 0.f);
            L = 0.f;
            for (int e = 0; e < groups; ++e) {
                const float wt = ex2_approx(sML[e * per + x].x - ref);
                const float4 v = sA[e * per + x];
                A.x = fmaf(wt, v.x, A.x); A.y = fmaf(wt, v.y, A.y);
                A.z = fmaf(wt, v.z, A.z); A.w = fmaf(wt, v.w, A.w);
                L = fmaf(wt, sML[e * per + x].y, L);
            }
        } else if (g > 0) {
            return;
        }
        if (mine) write_row(p, b, item / row_blocks * G + gr / p.Sq, gr % p.Sq, c, A, M, L);
    }
}

int general_splits(const AttnProblem &p, int sm_count) {
    const int R = p.Hq / p.Hkv * p.Sq;
    const long long items = (long long)p.B * p.Hkv * ((R + RB - 1) / RB);
    const long long units = key_stream_max(p.Sq, p.Sk, p.window ? p.window : p.Sk, p.sinks, 32);
    long long s = (8LL * sm_count + items - 1) / items;
    const long long most = (units + GW - 1) / GW;   // at least one step of every warp per part
    s = s < most ? s : most;
    return (int)(s < 1 ? 1 : s > 1024 ? 1024 : s);
}

size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace

static bool use_tc(const AttnProblem &p) {
    return p.dtype == OSF_BF16 && p.D <= 128 && p.Sk > 0 && tensor_map_encoder() != nullptr;
}

// Launch shape of the tensor-core kernel.  Whole items, a CTA each, need one launch and no join; cut, all tiles are shared by
// one wave of CTAs.  A cut costs what kCutCost tiles take (a second piece in most CTAs, the join), so it is made where the
// waves of whole items would take that much longer.  (Hkv=8 D=128, whole against cut, us: 1 row x 4 heads, 8 items of 16
// tiles 17.0 against 17.0, of 32 23.2 against 17.0, of 64 37.5 against 21.1; 64 of 32 25.2 against 27.3, of 64 37.5 against
// 35.5; 128 of 64 47.7 against 53.9; 256 of 64 88.7 against 90.8; 512 of 16 62.1 against 58.0, of 32 101 against 94.  16 rows:
// 8 of 16 23.3 against 23.2, of 32 33.4 against 23.2; 64 of 32 33.5 against 37.5, of 64 55.9 against 47.7; 128 of 64 58.0
// against 68.2; 512 of 32 136 against 127.)
constexpr int kCutCost = 20, kCutCost16 = 28;
struct TcPlan {
    int nr, row_blocks, flat, grid, item_cost;
};
static TcPlan tc_plan(const AttnProblem &p, int sm_count) {
    TcPlan t;
    const int R = p.Hq / p.Hkv * p.Sq;
    t.nr = R <= 4 ? 4 : R <= 8 ? 8 : 16;
    t.row_blocks = (R + t.nr - 1) / t.nr;
    const long long items = (long long)p.B * p.Hkv * t.row_blocks;
    const long long per = key_stream_max(p.Sq, p.Sk, p.window ? p.window : p.Sk, p.sinks, TT);
    const long long waves = (items + sm_count - 1) / sm_count;
    t.flat = waves * per - items * per / sm_count > (t.nr == 16 ? kCutCost16 : kCutCost);
    const long long worth = items * per / kMinTiles;
    t.item_cost = items < sm_count ? 3 : 10;
    t.grid = (int)(!t.flat ? items : worth < sm_count ? (worth < 1 ? 1 : worth) : sm_count);
    return t;
}

size_t kv8_attn_partial_bytes(const Kv8AttnProblem &kp, int sm_count) {
    const AttnProblem &p = kp.a;
    if (use_tc(p)) {
        const TcPlan t = tc_plan(p, sm_count);
        const size_t rows = 2 * (size_t)t.grid * t.nr;
        return t.flat ? round256(rows * (p.D <= 64 ? 64 : 128) * sizeof(float)) + round256(rows * sizeof(float2)) : 0;
    }
    const int splits = general_splits(p, sm_count);
    const size_t rows = (size_t)splits * p.B * p.Hq * p.Sq;
    return splits > 1 ? round256(rows * p.D * sizeof(float)) + 2 * round256(rows * sizeof(float)) : 0;
}

template <int D, int NR>
static cudaError_t launch_tc_t(Kv8AttnProblem kp, const TcPlan &t, char *partials, cudaStream_t s) {
    using C = Tc8<D, NR>;
    const AttnProblem &p = kp.a;
    auto kernel = t.flat ? attn_kv8_tc_kernel<D, NR, true> : attn_kv8_tc_kernel<D, NR, false>;
    cudaError_t e = set_max_dynamic_smem((const void *)kernel, (int)C::SMEM);
    if (e != cudaSuccess) return e;
    CUtensorMap m;
    const long long rows = (long long)kp.c.n_pages * 2 * kp.c.Hkv * kp.c.P;
    if (!make_u8_rows_map(&m, kp.c.pages, p.D, D, rows, (uint32_t)kp.c.P)) return cudaErrorInvalidValue;
    kp.part = reinterpret_cast<float *>(partials);
    kp.part_ml = reinterpret_cast<float2 *>(partials + round256(2 * (size_t)t.grid * NR * D * sizeof(float)));
    const int q_vec = (reinterpret_cast<uintptr_t>(p.q) & 3u) == 0 && ((p.q_sb | p.q_sh | p.q_ss) & 1) == 0;
    kernel<<<t.grid, C::THREADS, C::SMEM, s>>>(m, kp, q_vec, t.row_blocks, t.flat ? t.item_cost : 0);
    count_launches(1);
    e = cudaGetLastError();
    if (e != cudaSuccess || !t.flat) return e;
    count_launches(1);
    // a block per row where an item has more than one round of pieces (64 items of 16 rows in 152 CTAs: 91 us; a block per row 95)
    const int items = p.B * p.Hkv * t.row_blocks, rpb = t.grid > 8LL * items ? 1 : NR;
    return launch_dependent(kv8_combine_kernel<D, NR>, dim3((unsigned)items, (unsigned)(NR / rpb)), dim3(256), 0, s, kp, t.row_blocks,
                            t.grid, t.item_cost, rpb);
}

cudaError_t launch_attn_kv8(const Kv8AttnProblem &kp0, void *partials, int sm_count, cudaStream_t s) {
    Kv8AttnProblem kp = kp0;
    AttnProblem &p = kp.a;
    const int R = p.Hq / p.Hkv * p.Sq;
    char *at = static_cast<char *>(partials);
    if (use_tc(p)) {
        const TcPlan t = tc_plan(p, sm_count);
        if (p.D <= 64)
            return t.nr == 4 ? launch_tc_t<64, 4>(kp, t, at, s) : t.nr == 8 ? launch_tc_t<64, 8>(kp, t, at, s) : launch_tc_t<64, 16>(kp, t, at, s);
        return t.nr == 4 ? launch_tc_t<128, 4>(kp, t, at, s) : t.nr == 8 ? launch_tc_t<128, 8>(kp, t, at, s) : launch_tc_t<128, 16>(kp, t, at, s);
    }
    p.splits = general_splits(p, sm_count);
    p.keep_nan = 1;
    const size_t rows = (size_t)p.splits * p.B * p.Hq * p.Sq;
    p.part_acc = reinterpret_cast<float *>(at);
    p.part_m = reinterpret_cast<float *>(at + round256(rows * p.D * sizeof(float)));
    p.part_l = reinterpret_cast<float *>(at + round256(rows * p.D * sizeof(float)) + round256(rows * sizeof(float)));
    const dim3 grid((unsigned)(p.B * p.Hkv), (unsigned)p.splits, (unsigned)((R + RB - 1) / RB));
    const int smem = general_smem(p.D);
    auto kernel = p.dtype == OSF_F32 ? attn_kv8_kernel<float> : attn_kv8_kernel<__nv_bfloat16>;
    cudaError_t e = set_max_dynamic_smem((const void *)kernel, smem);
    if (e != cudaSuccess) return e;
    kernel<<<grid, GW * 32, smem, s>>>(kp);
    count_launches(1);
    e = cudaGetLastError();
    if (e == cudaSuccess && p.splits > 1) e = launch_attn_combine(p, s);
    return e;
}

}  // namespace osf
