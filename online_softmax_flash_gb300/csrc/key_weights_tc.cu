// Weights of keys on the tensor cores, bf16 with D 64 or 128 (the operation: key_weights.cu).
//
// Few query rows per kv head (G * Sq <= 16: a decode step): key_weights_rows_kernel, at the end of this
// file, bound by reading K once.
//
// Otherwise key_weights_tc_kernel.  The score tile is taken transposed, S^T = K Q^T: a TMEM lane is then a
// key and a thread owns one, so its sum over the rows stays in one register and no cross-thread reduction
// or exchange is needed until the end.  One tcgen05 product of 128 x 128 scores costs the tensor pipe
// D / 128 * 512 cycles; its 16384 exponentials cost the special-function unit 1024, so a share of them is
// computed by a polynomial on the FMA pipe instead (kPolyPairs).
//
// A CTA holds 256 keys (two A tiles, so that a query tile from L2 feeds two products) and walks the query
// tiles that see them, for the G heads of the group.  Warp roles (384 threads): warp 0 issues the TMA
// loads, warp 1 the MMAs, warp 2 fills a ring of row offsets (-lse * log2 e, -inf for rows past the end);
// warps 4-7 sum key tile 0, warps 8-11 key tile 1, each a TMEM lane quarter.  Score buffers are double
// (TMEM: 2 key tiles x 2 buffers x 128 columns), so the products of a step run under the sums of the last.
//
// Work is cut flat: an item is 256 keys of one (batch, kv head), of (heads x query tiles that see them)
// steps; CTA c takes the c-th part of all steps.  Causal items shrink along the keys, yet every CTA gets
// the same number of steps.  Items inside one part are written directly; a piece of a shared one goes to the
// workspace (at most two per CTA: the end of an item, slot 2c, and the start of one, slot 2c + 1), and
// key_weights_join_kernel adds the pieces in order.
// Every wait is bounded (2 s): on expiry the CTA records OSF_ERR_TIMEOUT, drains, frees TMEM.
#include "key_weights.cuh"
#include "sm100_ptx.cuh"
#include "tma_host.cuh"

namespace osf {
namespace {

using namespace ptx;

constexpr int TB = 128;                  // keys per A tile, query rows per B tile
constexpr int NTHREADS = 384;
constexpr int NCW = 8;                   // summing warps
constexpr int TSTAGES = 4;               // row-offset tables
constexpr uint32_t TMEM_COLS = 512;
constexpr int MAX_RING = 8;

template <int D>
struct KwCfg {
    static constexpr int RING = D == 64 ? 8 : 4;
    static constexpr uint32_t TILE = TB * D * 2;
    static constexpr uint32_t DBLK = TB * 128;                  // bytes between 64-column blocks
    static constexpr uint32_t RING_OFF = 2 * TILE;              // K tiles first
    static constexpr uint32_t TAB_OFF = RING_OFF + RING * TILE;
    static constexpr uint32_t SMEM_BYTES = TAB_OFF + TSTAGES * TB * 4 + 1024;
    static constexpr uint32_t IDESC = idesc_bf16_f32(TB, TB, 0, 0);
};

// Steps of the items: key block kb of 256 keys is seen by query tiles from max(0, 2 kb - shift) on.
struct KwPlan {
    int nkb, nqt, G, causal;
    long long shift;        // causal: ceil(causal_off / 128)
    long long per_bh;       // steps of one (batch, kv head)
    long long total;
    int nc;                 // CTAs
    __host__ __device__ long long first_tile(int kb) const {
        const long long q = causal ? 2LL * kb - shift : 0;
        return q < 0 ? 0 : q > nqt ? nqt : q;
    }
    // steps of the blocks before kb
    __host__ __device__ long long before(int kb) const {
        if (!causal) return (long long)kb * nqt * G;
        const long long all = shift < 0 ? 0 : shift / 2 + 1;                 // blocks that every tile sees
        const long long a = kb < all ? kb : all;
        const long long none = (nqt + shift + 1) / 2;                        // blocks from here on see none
        long long z = kb < none ? kb : none;
        const long long m = z > a ? z - a : 0;
        return (a * nqt + m * (nqt + shift) - m * (2 * a + m - 1)) * G;
    }
};

struct KwBars {
    uint64_t k_full, k_empty;
    uint64_t full[MAX_RING], empty[MAX_RING];
    uint64_t t_full[TSTAGES], t_empty[TSTAGES];
    uint64_t s_full[2][2], s_empty[2][2];   // [key tile][buffer]
    uint64_t drain;
};

// One piece: steps [u0, u1) of the item (bh, kb).
struct Piece {
    int bh, kb;
    long long u0, u1, units;
};
// Piece that begins at flat position `pos` of a part that ends at `end`.
__device__ __forceinline__ Piece piece_at(const KwPlan &w, long long pos, long long end) {
    Piece c;
    c.bh = (int)(pos / w.per_bh);
    const long long in = pos - (long long)c.bh * w.per_bh;
    int lo = 0, hi = w.nkb - 1;   // the last block that begins at or before `in`, and is not empty
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (w.before(mid) <= in) lo = mid; else hi = mid - 1;
    }
    while (lo > 0 && w.before(lo + 1) == w.before(lo)) --lo;
    c.kb = lo;
    const long long b0 = w.before(lo);
    c.units = w.before(lo + 1) - b0;
    c.u0 = in - b0;
    c.u1 = c.u0 + (end - pos);
    if (c.u1 > c.units) c.u1 = c.units;
    return c;
}

__device__ __forceinline__ void kw_timeout(volatile int *abort, int *status) {
    *abort = 1;
    atomicExch(status, kStatusTimeout);
}

// 2^x of a pair on the FMA pipe: x = n + f with |f| <= 1/2, a degree-5 minimax polynomial (relative error
// 7.5e-8 before rounding, fitted by the Remez exchange) for 2^f, n added to the exponent.  x below -126
// gives 2^-126.
__device__ __forceinline__ uint64_t ex2_poly(uint64_t x) {
    float a, b;
    f2_unpack(x, a, b);
    const uint64_t xc = f2_pack(fmaxf(a, -126.f), fmaxf(b, -126.f));
    const uint64_t magic = f2_pack(12582912.f, 12582912.f), nmagic = f2_pack(-12582912.f, -12582912.f);
    const uint64_t t = f2_add(xc, magic);
    const uint64_t f = f2_fma(f2_add(t, nmagic), f2_pack(-1.f, -1.f), xc);
    uint64_t p = f2_fma(f2_pack(1.3276472454890609e-3f, 1.3276472454890609e-3f), f,
                        f2_pack(9.675540961325169e-3f, 9.675540961325169e-3f));
    p = f2_fma(p, f, f2_pack(5.550713092088699e-2f, 5.550713092088699e-2f));
    p = f2_fma(p, f, f2_pack(2.4022120237350464e-1f, 2.4022120237350464e-1f));
    p = f2_fma(p, f, f2_pack(6.931469440460205e-1f, 6.931469440460205e-1f));
    p = f2_fma(p, f, f2_pack(1.0000001192092896f, 1.0000001192092896f));
    float ta, tb, pa, pb;
    f2_unpack(t, ta, tb);
    f2_unpack(p, pa, pb);
    return f2_pack(__uint_as_float(__float_as_uint(ta) * 8388608u + __float_as_uint(pa)),
                   __uint_as_float(__float_as_uint(tb) * 8388608u + __float_as_uint(pb)));
}
__device__ __forceinline__ uint64_t ex2_mufu(uint64_t x) {
    float a, b;
    f2_unpack(x, a, b);
    return f2_pack(ex2_approx(a), ex2_approx(b));
}

template <int D>
__global__ void __launch_bounds__(NTHREADS, 1)
key_weights_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk, const KeyWeightsProblem p,
                      const KwPlan w) {
    using C = KwCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ KwBars bars;
    __shared__ uint32_t tmem_sh;
    __shared__ volatile int abort_flag;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t sK = sbase, sRing = sbase + C::RING_OFF;
    float *tab = reinterpret_cast<float *>(smem_raw + (sbase - smem_u32(smem_raw)) + C::TAB_OFF);
    if (warp == 0) tmem_alloc(smem_u32(&tmem_sh), TMEM_COLS);
    if (tid == 32) {
        mbar_init(smem_u32(&bars.k_full), 1);
        mbar_init(smem_u32(&bars.k_empty), 1);
        for (int s = 0; s < C::RING; ++s) {
            mbar_init(smem_u32(&bars.full[s]), 1);
            mbar_init(smem_u32(&bars.empty[s]), 1);
        }
        for (int s = 0; s < TSTAGES; ++s) {
            mbar_init(smem_u32(&bars.t_full[s]), 32);
            mbar_init(smem_u32(&bars.t_empty[s]), NCW);
        }
        for (int k = 0; k < 2; ++k)
            for (int s = 0; s < 2; ++s) {
                mbar_init(smem_u32(&bars.s_full[k][s]), 1);
                mbar_init(smem_u32(&bars.s_empty[k][s]), NCW / 2);
            }
        mbar_init(smem_u32(&bars.drain), 1);
        abort_flag = 0;
        mbar_init_fence();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_sh;
    const long long pos0 = w.total * blockIdx.x / w.nc, pos1 = w.total * (blockIdx.x + 1) / w.nc;
    // the second key tile of a block is past the first query tile that sees the first
    auto sees = [&](const Piece &c, long long qt, int kt) {
        const long long key0 = (long long)c.kb * 2 * TB + kt * TB;
        return key0 < p.Sk && (!w.causal || qt * TB + TB - 1 + p.causal_off >= key0);
    };

    if (warp == 0) {
        if (lane == 0) {
            // ------------------------------------------------------------ TMA: K tiles, Q tiles
            tma_prefetch_desc(&mq);
            tma_prefetch_desc(&mk);
            bool ok = true;
            int n = 0, items = 0;
            for (long long pos = pos0; pos < pos1 && ok;) {
                const Piece c = piece_at(w, pos, pos1);
                const int b = c.bh / p.Hkv, kvh = c.bh % p.Hkv;
                // Q tiles may run ahead of the K tiles' release, by the ring's length
                ok = mbar_wait(smem_u32(&bars.k_empty), (items & 1) ^ 1, &abort_flag);
                if (!ok) break;
                mbar_expect_tx(smem_u32(&bars.k_full), 2 * C::TILE);
                tma_load_5d(sK, &mk, smem_u32(&bars.k_full), 0, c.kb * 2 * TB, 0, kvh, b);
                tma_load_5d(sK + C::TILE, &mk, smem_u32(&bars.k_full), 0, c.kb * 2 * TB + TB, 0, kvh, b);
                const long long q0 = w.first_tile(c.kb);
                for (long long u = c.u0; u < c.u1; ++u, ++n) {
                    const int st = n % C::RING;
                    ok = mbar_wait(smem_u32(&bars.empty[st]), ((n / C::RING) & 1) ^ 1, &abort_flag);
                    if (!ok) break;
                    const int qt = (int)(q0 + u / w.G), hq = kvh * w.G + (int)(u % w.G);
                    mbar_expect_tx(smem_u32(&bars.full[st]), C::TILE);
                    tma_load_5d_hint(sRing + st * C::TILE, &mq, smem_u32(&bars.full[st]), 0, qt * TB, 0, hq, b,
                                     l2_policy_evict_last());
                }
                pos += c.u1 - c.u0;
                ++items;
            }
            if (!ok) {
                kw_timeout(&abort_flag, p.status);
                const uint64_t t0 = globaltimer_ns();   // let copies in flight land
                while (globaltimer_ns() - t0 < 50000ull) {
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            // ------------------------------------------------------------ MMA: S^T = K Q^T
            bool ok = true;
            int n = 0, items = 0, done[2] = {0, 0};
            for (long long pos = pos0; pos < pos1 && ok;) {
                const Piece c = piece_at(w, pos, pos1);
                const long long q0 = w.first_tile(c.kb);
                ok = mbar_wait_spin(smem_u32(&bars.k_full), items & 1, &abort_flag);
                for (long long u = c.u0; u < c.u1 && ok; ++u, ++n) {
                    const int st = n % C::RING;
                    ok = mbar_wait_spin(smem_u32(&bars.full[st]), (n / C::RING) & 1, &abort_flag);
                    for (int kt = 0; kt < 2 && ok; ++kt) {
                        if (!sees(c, q0 + u / w.G, kt)) continue;
                        const int buf = done[kt] & 1;
                        ok = mbar_wait_spin(smem_u32(&bars.s_empty[kt][buf]), ((done[kt] >> 1) & 1) ^ 1, &abort_flag);
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t ad = sdesc_sw128(sK + kt * C::TILE, 16, 1024);
                        const uint64_t bd = sdesc_sw128(sRing + st * C::TILE, 16, 1024);
#pragma unroll
                        for (int k = 0; k < D / 16; ++k) {
                            const uint32_t off = ((k >> 2) * C::DBLK + (k & 3) * 32) >> 4;
                            mma_ss(tmem + (uint32_t)(kt * 2 + buf) * TB, ad + off, bd + off, C::IDESC, k > 0);
                        }
                        mma_commit(smem_u32(&bars.s_full[kt][buf]));
                        ++done[kt];
                    }
                    if (ok) mma_commit(smem_u32(&bars.empty[st]));
                }
                if (ok) mma_commit(smem_u32(&bars.k_empty));
                pos += c.u1 - c.u0;
                ++items;
            }
            if (!ok) kw_timeout(&abort_flag, p.status);
            mma_commit(smem_u32(&bars.drain));
            mbar_wait(smem_u32(&bars.drain), 0, nullptr, 20000000ull);
        }
    } else if (warp == 2) {
        // ------------------------------------------------------------ row offsets of each step
        bool ok = true;
        int n = 0;
        for (long long pos = pos0; pos < pos1 && ok;) {
            const Piece c = piece_at(w, pos, pos1);
            const int b = c.bh / p.Hkv, kvh = c.bh % p.Hkv;
            const long long q0 = w.first_tile(c.kb);
            for (long long u = c.u0; u < c.u1; ++u, ++n) {
                const int st = n % TSTAGES;
                ok = mbar_wait(smem_u32(&bars.t_empty[st]), ((n / TSTAGES) & 1) ^ 1, &abort_flag);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                const int qt = (int)(q0 + u / w.G);
                const float *lse = p.lse + ((long long)b * p.Hq + kvh * w.G + u % w.G) * p.Sq;
#pragma unroll
                for (int i = 0; i < TB / 32; ++i) {
                    const int r = lane + 32 * i, q = qt * TB + r;
                    tab[st * TB + r] = q < p.Sq ? row_offset(lse[q]) : -INFINITY;
                }
                mbar_arrive(smem_u32(&bars.t_full[st]));
            }
            pos += c.u1 - c.u0;
        }
        if (!ok) kw_timeout(&abort_flag, p.status);
    } else if (warp >= 4) {
        // ------------------------------------------------------------ sums, one key per thread
        const int kt = (warp - 4) >> 2, q4 = warp & 3;
        const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
        const uint64_t c2 = f2_pack(p.scale_log2, p.scale_log2);
        bool ok = true;
        int n = 0, done = 0;
        for (long long pos = pos0; pos < pos1 && ok;) {
            const Piece c = piece_at(w, pos, pos1);
            const long long q0 = w.first_tile(c.kb);
            const int key = c.kb * 2 * TB + kt * TB + q4 * 32 + lane;
            float total = 0.f;
            for (long long u = c.u0; u < c.u1; ++u, ++n) {
                const int st = n % TSTAGES;
                ok = mbar_wait(smem_u32(&bars.t_full[st]), (n / TSTAGES) & 1, &abort_flag);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                const long long qt = q0 + u / w.G;
                if (sees(c, qt, kt)) {
                    const int buf = done & 1;
                    ok = mbar_wait(smem_u32(&bars.s_full[kt][buf]), (done >> 1) & 1, &abort_flag);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    tc_fence_after();
                    // columns below qmin are rows that do not see this key, those from qmax on rows past the last (a
                    // NaN key would get through their offset of -inf); a warp without either skips the test
                    const long long first = (long long)key - p.causal_off - qt * TB;
                    const int qmin = w.causal ? (int)max(0LL, min((long long)TB, first)) : 0;
                    const int qmax = (int)min((long long)TB, p.Sq - qt * TB);
                    const bool some = __any_sync(0xffffffffu, qmin > 0) || qmax < TB;
                    uint64_t acc[2] = {0, 0};
                    const uint32_t taddr = tmem + (uint32_t)(kt * 2 + buf) * TB + lane_off;
                    const float4 *off4 = reinterpret_cast<const float4 *>(tab + st * TB);
#pragma unroll
                    for (int ch = 0; ch < 4; ++ch) {
                        uint32_t s[32];
                        tmem_ld32(taddr + 32 * ch, s);
                        tmem_ld_wait();
                        if (ch == 3) {   // the scores are in registers: the buffer may take the step after next
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(smem_u32(&bars.s_empty[kt][buf]));
                        }
#pragma unroll
                        for (int k4 = 0; k4 < 8; ++k4) {
                            const float4 o = off4[8 * ch + k4];
#pragma unroll
                            for (int e = 0; e < 4; e += 2) {
                                const int k = 4 * k4 + e;
                                const uint64_t x = f2_fma(f2_pack(__uint_as_float(s[k]), __uint_as_float(s[k + 1])), c2,
                                                          e ? f2_pack(o.z, o.w) : f2_pack(o.x, o.y));
                                uint64_t v = ex2_mufu(x);
                                if (some) {
                                    float a, bb;
                                    f2_unpack(v, a, bb);
                                    v = f2_pack(32 * ch + k >= qmin && 32 * ch + k < qmax ? a : 0.f,
                                                32 * ch + k + 1 >= qmin && 32 * ch + k + 1 < qmax ? bb : 0.f);
                                }
                                acc[(k >> 1) & 1] = f2_add(acc[(k >> 1) & 1], v);
                            }
                        }
                    }
                    ++done;
                    float a, bb;
                    f2_unpack(f2_add(acc[0], acc[1]), a, bb);
                    total += a + bb;   // 128 terms among themselves, then one addition to the long sum
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bars.t_empty[st]));
            }
            if (!ok) break;
            if (c.u1 - c.u0 == c.units) {
                if (key < p.Sk) {
                    float *out = p.w + (long long)c.bh * p.Sk + key;
                    *out = p.accumulate ? *out + total : total;
                }
            } else {
                const long long slot = 2LL * blockIdx.x + (c.u0 == 0 ? 1 : 0);
                p.part[slot * 2 * TB + kt * TB + q4 * 32 + lane] = total;
            }
            pos += c.u1 - c.u0;
        }
        if (!ok) kw_timeout(&abort_flag, p.status);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, TMEM_COLS);
}

// Items that several CTAs shared, and items that no row sees: a block per item.
__global__ void __launch_bounds__(2 * TB) key_weights_join_kernel(const KeyWeightsProblem p, const KwPlan w) {
    griddep_wait();
    const int bh = blockIdx.y, kb = blockIdx.x, key = kb * 2 * TB + threadIdx.x;
    if (key >= p.Sk) return;
    float *out = p.w + (long long)bh * p.Sk + key;
    const long long p0 = (long long)bh * w.per_bh + w.before(kb), p1 = (long long)bh * w.per_bh + w.before(kb + 1);
    if (p0 == p1) {
        if (!p.accumulate) *out = 0.f;
        return;
    }
    // CTA of step x: the last one whose part begins at or before it
    const int c0 = (int)(((p0 + 1) * w.nc - 1) / w.total), c1 = (int)((p1 * w.nc - 1) / w.total);
    if (c0 == c1) return;
    float v = 0.f;
    for (int c = c0; c <= c1; ++c) v += p.part[(2LL * c + (c == c0 ? 1 : 0)) * 2 * TB + threadIdx.x];
    *out = p.accumulate ? *out + v : v;
}

KwPlan make_plan(const KeyWeightsProblem &p, int sm_count) {
    KwPlan w;
    w.nkb = (p.Sk + 2 * TB - 1) / (2 * TB);
    w.nqt = (p.Sq + TB - 1) / TB;
    w.G = p.Hq / p.Hkv;
    w.causal = p.causal;
    // ceil(causal_off / 128), for negative offsets too
    w.shift = p.causal_off >= 0 ? (p.causal_off + TB - 1) / TB : -(long long)(-(long long)p.causal_off / TB);
    w.per_bh = w.before(w.nkb);
    w.total = w.per_bh * p.B * p.Hkv;
    const long long worth = w.total / 4;   // at least four steps for a CTA
    w.nc = (int)(worth < 1 ? 1 : worth < sm_count ? worth : sm_count);
    return w;
}

template <int D>
cudaError_t launch_tc_t(const KeyWeightsProblem &p, const KwPlan &w, cudaStream_t s) {
    using C = KwCfg<D>;
    cudaError_t e = set_max_dynamic_smem((const void *)key_weights_tc_kernel<D>, (int)C::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    CUtensorMap mq, mk;
    if (!make_bf16_tile_map_strided(&mq, p.q, D, p.Sq, p.Hq, p.B, p.q_ss, p.q_sh, p.q_sb, TB) ||
        !make_bf16_tile_map_strided(&mk, p.k, D, p.Sk, p.Hkv, p.B, p.k_ss, p.k_sh, p.k_sb, TB))
        return cudaErrorInvalidValue;
    key_weights_tc_kernel<D><<<w.nc, NTHREADS, C::SMEM_BYTES, s>>>(mq, mk, p, w);
    count_launches(1);
    return cudaGetLastError();
}

// ============================================================================ few rows (decode)
// One warp takes 16 keys at a time as the M rows of m16n8k16 products, the query rows as N columns.  Lane
// (g, t) reads channels 8t .. 8t+7 of every group of 32 of keys g and g + 8 with 16-byte loads: any order of
// the channels does for a contraction, so these are its A operands as they come, without shared memory.
// The next tile's loads are in flight while this one is computed; a key's sum over the rows is two shuffles.
constexpr int RW = 8;   // warps per CTA

template <int D>
struct KeyTile {
    uint4 x[D / 32][2];
};

template <int D, int NT>
__global__ void __launch_bounds__(RW * 32, D == 64 ? 3 : 2)
key_weights_rows_kernel(const KeyWeightsProblem p, int q_vec) {
    constexpr int NG = D / 32;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int G = p.Hq / p.Hkv, R = G * p.Sq;
    const int kvbh = blockIdx.x, b = kvbh / p.Hkv, kvh = kvbh % p.Hkv;
    const int tiles = (p.Sk + 15) / 16;
    const int t0 = (int)((long long)tiles * blockIdx.y / gridDim.y), t1 = (int)((long long)tiles * (blockIdx.y + 1) / gridDim.y);
    const __nv_bfloat16 *K = static_cast<const __nv_bfloat16 *>(p.k) + b * p.k_sb + kvh * p.k_sh + 8 * t;
    auto load = [&](int tile, KeyTile<D> &kt) {
        // rows past the last key repeat it: read, never written
        const uint4 *r0 = reinterpret_cast<const uint4 *>(K + min(tile * 16 + g, p.Sk - 1) * p.k_ss);
        const uint4 *r1 = reinterpret_cast<const uint4 *>(K + min(tile * 16 + g + 8, p.Sk - 1) * p.k_ss);
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            kt.x[i][0] = __ldcs(r0 + 4 * i);
            kt.x[i][1] = __ldcs(r1 + 4 * i);
        }
    };
    int tile = t0 + warp;
    KeyTile<D> cur;
    if (tile < t1) load(tile, cur);
    uint32_t qb[NT][NG][4];
    float off[NT][2];
    int lim[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int r = nt * 8 + g;
        const __nv_bfloat16 *Q = static_cast<const __nv_bfloat16 *>(p.q);
        if (r < R) Q += b * p.q_sb + (long long)(kvh * G + r / p.Sq) * p.q_sh + r % p.Sq * p.q_ss;
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (r < R) {
                const __nv_bfloat16 *q = Q + 32 * i + 8 * t;
                if (q_vec) {
                    v = *reinterpret_cast<const uint4 *>(q);
                } else {
                    const unsigned short *h = reinterpret_cast<const unsigned short *>(q);
                    v.x = h[0] | (uint32_t)h[1] << 16; v.y = h[2] | (uint32_t)h[3] << 16;
                    v.z = h[4] | (uint32_t)h[5] << 16; v.w = h[6] | (uint32_t)h[7] << 16;
                }
            }
            qb[nt][i][0] = v.x; qb[nt][i][1] = v.y; qb[nt][i][2] = v.z; qb[nt][i][3] = v.w;
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int col = nt * 8 + 2 * t + c;
            off[nt][c] = col < R ? row_offset(p.lse[((long long)b * p.Hq + kvh * G + col / p.Sq) * p.Sq + col % p.Sq]) : -INFINITY;
            lim[nt][c] = col >= R ? 0 : p.causal ? max(0, min(p.Sk, col % p.Sq + p.causal_off + 1)) : p.Sk;
        }
    }
    float *W = p.w + (long long)kvbh * p.Sk;
    while (tile < t1) {
        const int next = tile + RW;
        KeyTile<D> ahead;
        if (next < t1) load(next, ahead);
        float sum[2] = {0.f, 0.f};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                const uint4 a = cur.x[i][0], c = cur.x[i][1];
                const uint32_t lo[4] = {a.x, c.x, a.y, c.y}, hi[4] = {a.z, c.z, a.w, c.w};
                mma_m16n8k16_bf16(y, lo, qb[nt][i][0], qb[nt][i][1]);
                mma_m16n8k16_bf16(y, hi, qb[nt][i][2], qb[nt][i][3]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float v = ex2_approx(fmaf(y[e], p.scale_log2, off[nt][e & 1]));
                sum[e >> 1] += tile * 16 + g + (e >> 1) * 8 < lim[nt][e & 1] ? v : 0.f;
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 1);
            sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 2);
        }
        const int key = tile * 16 + g + 8 * (t & 1);
        if (t < 2 && key < p.Sk) {
            const float v = t ? sum[1] : sum[0];
            W[key] = p.accumulate ? W[key] + v : v;
        }
        cur = ahead;
        tile = next;
    }
}

template <int D, int NT>
cudaError_t launch_rows_t(const KeyWeightsProblem &p, int sm_count, cudaStream_t s) {
    const long long items = (long long)p.B * p.Hkv, tiles = ((long long)p.Sk + 15) / 16;
    // about four waves, so the last wave's imbalance stays small; two tiles for every warp at least
    long long parts = (4LL * sm_count * (D == 64 ? 3 : 2) + items / 2) / items;
    const long long most = tiles / (2 * RW);
    parts = parts < most ? parts : most;
    parts = parts < 1 ? 1 : parts > 65535 ? 65535 : parts;
    const int q_vec = aligned16(p.q) && ((p.q_sb | p.q_sh | p.q_ss) & 7) == 0;
    key_weights_rows_kernel<D, NT><<<dim3((unsigned)items, (unsigned)parts), RW * 32, 0, s>>>(p, q_vec);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace

bool key_weights_rows_supported(const KeyWeightsProblem &p) {
    return p.dtype == OSF_BF16 && (p.D == 64 || p.D == 128) && (long long)(p.Hq / p.Hkv) * p.Sq <= 16 && aligned16(p.k) &&
           ((p.k_sb | p.k_sh | p.k_ss) & 7) == 0;
}

bool key_weights_tc_supported(const KeyWeightsProblem &p) {
    return p.dtype == OSF_BF16 && (p.D == 64 || p.D == 128) && tensor_map_encoder() != nullptr &&
           tile_map_addressable(p.q, p.D, p.Sq, p.Hq, p.B, p.q_ss, p.q_sh, p.q_sb) &&
           tile_map_addressable(p.k, p.D, p.Sk, p.Hkv, p.B, p.k_ss, p.k_sh, p.k_sb);
}

size_t key_weights_tc_floats(int sm_count) { return (size_t)2 * sm_count * 2 * TB; }

cudaError_t launch_key_weights_rows(const KeyWeightsProblem &p, int sm_count, cudaStream_t s) {
    const bool few = (p.Hq / p.Hkv) * p.Sq <= 8;
    return p.D == 64 ? (few ? launch_rows_t<64, 1>(p, sm_count, s) : launch_rows_t<64, 2>(p, sm_count, s))
                     : (few ? launch_rows_t<128, 1>(p, sm_count, s) : launch_rows_t<128, 2>(p, sm_count, s));
}

cudaError_t launch_key_weights_tc(const KeyWeightsProblem &p, int sm_count, cudaStream_t s) {
    const KwPlan w = make_plan(p, sm_count);
    cudaError_t e = cudaSuccess;
    if (w.total > 0) e = p.D == 64 ? launch_tc_t<64>(p, w, s) : launch_tc_t<128>(p, w, s);
    if (e != cudaSuccess) return e;
    count_launches(1);
    return launch_dependent(key_weights_join_kernel, dim3((unsigned)w.nkb, (unsigned)(p.B * p.Hkv)), dim3(2 * TB), 0, s, p, w);
}

}  // namespace osf
