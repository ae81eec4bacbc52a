// Weights of keys on the tensor cores, bf16 (the operation: key_weights.cu).
//
// Few query rows per kv head (G * Sq <= 16: a decode step), D 32, 64, 96 or 128: key_weights_rows_kernel, at the end
// of this file, bound by reading K once.
//
// Otherwise, with D 64 or 128, key_weights_tc_kernel.  The score tile is taken transposed, S^T = K Q^T: a TMEM lane is then a
// key and a thread owns one, so its sum over the rows stays in one register and no cross-thread reduction
// or exchange is needed until the end.  One tcgen05 product of 128 x 128 scores costs the tensor pipe
// D / 128 * 512 cycles, its 16384 exponentials the special-function units about as much.  (A share of the
// exponentials as a polynomial on the FMA pipe was measured and is slower: 3 of 16 pairs 153 us against
// 143 us for the B=2 Hq=32 S=4096 D=128 causal prompt, 8 of 16 199 us.)
//
// A CTA holds 256 keys (two A tiles, so that a query tile from L2 feeds two products) and walks the query
// tiles that see them, for the G heads of the group.  Warp roles (640 threads): warp 0 issues the TMA
// loads, warps 1 and 3 the MMAs of key tile 0 and 1 (one issuer for both: 140 us against 120 us for that prompt,
// since it waits for the slower of the two), warp 2 fills a ring of row offsets (-lse * log2 e, -inf for rows past
// the end); warps 4-11 sum key tile 0, warps 12-19 key tile 1: a warp has a TMEM lane quarter and every other step.
// Score buffers are double (TMEM: 2 key tiles x 2 buffers x 128 columns), one to a parity, so the products of a
// step run under the sums of the last.
//
// That prompt: 117 us for the whole call, where its products take 60 us of the tensor pipe at 1.9 GHz and its 5.5e8
// exponentials as long of the special-function units; both are busy 59 % of the time.  A score buffer goes round from
// product to sum to product, with some 700 cycles of hand-off on the way even where there is nothing to compute, and
// TMEM holds no more than these four.  (Without the exponentials the call takes 113 us, with half the products 109 us,
// without the loads of Q 115 us.  The other way round, S = Q K^T, a row to a lane and 64 keys' sums to a thread, with
// products of 256 columns in two buffers, needs no table of offsets and less of shared memory's bandwidth, but has only
// two buffers to hide the hand-off: 128 us.  Eight warps that take a whole tile into registers: 141 us.)
//
// Work is cut flat: an item is 256 keys of one (batch, kv head), of (heads x query tiles that see them)
// steps; CTA c takes the c-th part of all steps.  Causal items shrink along the keys, yet every CTA gets
// the same number of steps.  Items inside one part are written directly; a piece of a shared one goes to the
// workspace (at most two per CTA: the end of an item, slot 2c, and the start of one, slot 2c + 1), and
// key_weights_join_kernel adds the pieces in order.  (Short items that are all alike get a CTA each: make_plan.)
// Every wait is bounded (2 s): on expiry the CTA records OSF_ERR_TIMEOUT, drains, frees TMEM.
#include <climits>

#include "key_weights.cuh"
#include "sm100_ptx.cuh"
#include "tma_host.cuh"

namespace osf {
namespace {

using namespace ptx;

constexpr int TB = 128;                  // keys per A tile, query rows per B tile
constexpr int NCW = 16;                  // summing warps: 2 key tiles x 2 step parities x 4 lane quarters
constexpr int NTHREADS = (4 + NCW) * 32;
constexpr int TSTAGES = 4;               // row-offset tables
constexpr uint32_t TMEM_COLS = 512;
constexpr int MAX_RING = 8;
// Most steps of an item that is left to one CTA without the join (B=13 Hq=16 Hkv=8 Sq=49 Sk=129, 2 steps: 8.0 us against
// 9.1 us; B=5 Hq=40 Hkv=8 Sq=64, 5 steps: 8.7 us against 9.6 us; B=1 Hq=32 Hkv=8 Sq=256, 8 steps: 12.0 us against 8.6 us).
constexpr int kWholeSteps = 5;

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
    int whole;              // every CTA has one item
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
    uint64_t drain[2];
};

// One piece: steps [u0, u1) of the item (bh, kb).
struct Piece {
    int bh, kb, u0, u1, units;
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
    c.units = (int)(w.before(lo + 1) - b0);
    c.u0 = (int)(in - b0);
    c.u1 = (int)min((long long)c.units, c.u0 + (end - pos));
    return c;
}
// Query tile and head (of the group) of the steps of a piece, heads innermost.
struct Step {
    int qt, h, G;
    __device__ __forceinline__ Step(const KwPlan &w, const Piece &c) : G(w.G) {
        qt = (int)w.first_tile(c.kb) + c.u0 / G;
        h = c.u0 % G;
    }
    __device__ __forceinline__ void next() {
        if (++h == G) {
            h = 0;
            ++qt;
        }
    }
};

// Number of query tiles, from tile `first` on, that begin before row x.
__device__ __forceinline__ int tiles_before(long long x, int first) {
    const long long t = x > 0 ? (x + TB - 1) / TB : 0;   // tiles qt with qt * 128 < x
    return (int)max(0LL, t - first);
}

__device__ __forceinline__ void kw_timeout(volatile int *abort, int *status) {
    *abort = 1;
    atomicExch(status, kStatusTimeout);
}

__device__ __forceinline__ uint64_t ex2_pair(uint64_t x) {
    float a, b;
    f2_unpack(x, a, b);
    return f2_pack(ex2_approx(a), ex2_approx(b));
}

__device__ __forceinline__ void lds_pairs(uint32_t addr, uint64_t &a, uint64_t &b) {
    asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "r"(addr));
}

// One key's terms of a score tile: 128 TMEM columns against the offsets of their rows; `sempty` is told once the
// last are in registers.  (The SM quarter's four warps cover each other's TMEM loads: loads of the next 32
// columns under the sums of these, 117.9 us against 116.8 us; 64 columns at once 121.5 us.)  The 128 terms are
// added among themselves, so the long sum gets one rounding per tile.
// MASK: columns below qmin, and those whose offset is -inf, add nothing whatever their score (a NaN as well).
template <bool MASK>
__device__ __forceinline__ float sum_tile(uint32_t taddr, uint32_t toff, uint64_t c2, int qmin, uint32_t sempty, int lane) {
    uint64_t acc[2] = {0, 0};
#pragma unroll
    for (int ch = 0; ch < 4; ++ch) {
        uint32_t s[32];
        tmem_ld32(taddr + 32 * ch, s);
        tmem_ld_wait();
        if (ch == 3) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(sempty);
        }
#pragma unroll
        for (int k = 0; k < 32; k += 4) {
            uint64_t o[2];
            lds_pairs(toff + (32 * ch + k) * 4, o[0], o[1]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = k + 2 * e;
                uint64_t v = ex2_pair(f2_fma(f2_pack(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), c2, o[e]));
                if (MASK) {
                    float a, b, oa, ob;
                    f2_unpack(v, a, b);
                    f2_unpack(o[e], oa, ob);
                    v = f2_pack(32 * ch + i >= qmin && oa != -INFINITY ? a : 0.f,
                                32 * ch + i + 1 >= qmin && ob != -INFINITY ? b : 0.f);
                }
                acc[e] = f2_add(acc[e], v);
            }
        }
    }
    float a, b;
    f2_unpack(f2_add(acc[0], acc[1]), a, b);
    return a + b;
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
    __shared__ float other[2][TB];        // sums of the odd steps
    __shared__ int holes[TSTAGES];        // an offset of the table is -inf
    __shared__ volatile int failed[2];    // a summing warp of the key tile gave up
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t sK = sbase, sRing = sbase + C::RING_OFF;
    float *tab = reinterpret_cast<float *>(smem_raw + (sbase - smem_u32(smem_raw)) + C::TAB_OFF);
    if (warp == 0) tmem_alloc(smem_u32(&tmem_sh), TMEM_COLS);
    if (tid == 32) {
        mbar_init(smem_u32(&bars.k_full), 1);
        mbar_init(smem_u32(&bars.k_empty), 2);   // one release from each issuer
        for (int s = 0; s < C::RING; ++s) {
            mbar_init(smem_u32(&bars.full[s]), 1);
            mbar_init(smem_u32(&bars.empty[s]), 2);
        }
        for (int s = 0; s < TSTAGES; ++s) {
            mbar_init(smem_u32(&bars.t_full[s]), 32);
            mbar_init(smem_u32(&bars.t_empty[s]), NCW / 2);
        }
        for (int k = 0; k < 2; ++k)
            for (int s = 0; s < 2; ++s) {
                mbar_init(smem_u32(&bars.s_full[k][s]), 1);
                mbar_init(smem_u32(&bars.s_empty[k][s]), NCW / 4);
            }
        mbar_init(smem_u32(&bars.drain[0]), 1);
        mbar_init(smem_u32(&bars.drain[1]), 1);
        abort_flag = failed[0] = failed[1] = 0;
        mbar_init_fence();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_sh;
    const long long pos0 = w.total * blockIdx.x / w.nc, pos1 = w.total * (blockIdx.x + 1) / w.nc;
    // step of a piece's item from which on a query tile sees key tile kt (INT_MAX: it is past the last key)
    auto first_step = [&](const Piece &c, int kt) {
        const long long key0 = (long long)c.kb * 2 * TB + kt * TB;
        if (key0 >= p.Sk) return INT_MAX;
        return w.causal ? tiles_before(key0 - p.causal_off - (TB - 1), (int)w.first_tile(c.kb)) * w.G : 0;
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
                Step at(w, c);
                for (int u = c.u0; u < c.u1; ++u, ++n, at.next()) {
                    const int st = n % C::RING;
                    ok = mbar_wait(smem_u32(&bars.empty[st]), ((n / C::RING) & 1) ^ 1, &abort_flag);
                    if (!ok) break;
                    mbar_expect_tx(smem_u32(&bars.full[st]), C::TILE);
                    tma_load_5d_hint(sRing + st * C::TILE, &mq, smem_u32(&bars.full[st]), 0, at.qt * TB, 0, kvh * w.G + at.h,
                                     b, l2_policy_evict_last());
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
    } else if (warp == 1 || warp == 3) {
        if (lane == 0) {
            // ------------------------------------------------------------ MMA: S^T = K Q^T, an issuer per key tile
            const int kt = warp >> 1;
            bool ok = true;
            int n = 0, items = 0;
            int phase = 3;   // bit b: parity of the next wait for buffer b to be free
            const uint64_t ad = sdesc_sw128(sK + kt * C::TILE, 16, 1024);
            for (long long pos = pos0; pos < pos1 && ok;) {
                const Piece c = piece_at(w, pos, pos1);
                const int u_see = first_step(c, kt);
                ok = mbar_wait_spin(smem_u32(&bars.k_full), items & 1, &abort_flag);
                for (int u = c.u0; u < c.u1 && ok; ++u, ++n) {
                    const int st = n % C::RING, buf = n & 1;
                    ok = mbar_wait_spin(smem_u32(&bars.full[st]), (n / C::RING) & 1, &abort_flag);
                    if (ok && u >= u_see) {
                        ok = mbar_wait_spin(smem_u32(&bars.s_empty[kt][buf]), (phase >> buf) & 1, &abort_flag);
                        if (!ok) break;
                        phase ^= 1 << buf;
                        tc_fence_after();
                        const uint64_t bd = sdesc_sw128(sRing + st * C::TILE, 16, 1024);
#pragma unroll
                        for (int k = 0; k < D / 16; ++k) {
                            const uint32_t off = ((k >> 2) * C::DBLK + (k & 3) * 32) >> 4;
                            mma_ss(tmem + (uint32_t)(kt * 2 + buf) * TB, ad + off, bd + off, C::IDESC, k > 0);
                        }
                        mma_commit(smem_u32(&bars.s_full[kt][buf]));
                    }
                    if (ok) mma_commit(smem_u32(&bars.empty[st]));
                }
                if (ok) mma_commit(smem_u32(&bars.k_empty));
                pos += c.u1 - c.u0;
                ++items;
            }
            if (!ok) kw_timeout(&abort_flag, p.status);
            mma_commit(smem_u32(&bars.drain[kt]));
            mbar_wait(smem_u32(&bars.drain[kt]), 0, nullptr, 20000000ull);
        }
    } else if (warp == 2) {
        // ------------------------------------------------------------ row offsets of each step
        bool ok = true;
        int n = 0;
        for (long long pos = pos0; pos < pos1 && ok;) {
            const Piece c = piece_at(w, pos, pos1);
            const int b = c.bh / p.Hkv, kvh = c.bh % p.Hkv;
            Step at(w, c);
            for (int u = c.u0; u < c.u1; ++u, ++n, at.next()) {
                const int st = n % TSTAGES;
                ok = mbar_wait(smem_u32(&bars.t_empty[st]), ((n / TSTAGES) & 1) ^ 1, &abort_flag);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                const float *lse = p.lse + ((long long)b * p.Hq + kvh * w.G + at.h) * p.Sq;
                bool hole = false;
#pragma unroll
                for (int i = 0; i < TB / 32; ++i) {
                    const int r = lane + 32 * i, q = at.qt * TB + r;
                    const float o = q < p.Sq ? row_offset(lse[q]) : -INFINITY;
                    tab[st * TB + r] = o;
                    hole |= o == -INFINITY;
                }
                hole = __any_sync(0xffffffffu, hole);
                if (lane == 0) holes[st] = hole;
                mbar_arrive(smem_u32(&bars.t_full[st]));
            }
            pos += c.u1 - c.u0;
        }
        if (!ok) kw_timeout(&abort_flag, p.status);
    } else if (warp >= 4) {
        // ------------------------------------------------------------ sums, a key per thread
        // steps of parity `odd` only, whose scores are in buffer `odd`: two warps of a lane quarter take turns
        const int kt = (warp - 4) >> 3, odd = ((warp - 4) >> 2) & 1, q4 = warp & 3;
        const uint32_t taddr = tmem + (uint32_t)(kt * 2 + odd) * TB + ((uint32_t)(q4 * 32) << 16);
        const uint32_t toff0 = smem_u32(tab), sfull = smem_u32(&bars.s_full[kt][odd]), sempty = smem_u32(&bars.s_empty[kt][odd]);
        const uint64_t c2 = f2_pack(p.scale_log2, p.scale_log2);
        bool ok = true;
        int n0 = 0, phase = 0;   // steps before the piece; parity of the next wait for scores
        for (long long pos = pos0; pos < pos1 && ok;) {
            const Piece c = piece_at(w, pos, pos1);
            const int key0 = c.kb * 2 * TB + kt * TB, key = key0 + q4 * 32 + lane;
            const int q_first = (int)w.first_tile(c.kb);
            // steps of the item from which on: the key tile is seen; every row of a tile sees all keys of this warp
            const int u_see = first_step(c, kt);
            const int u_full = w.causal ? tiles_before((long long)key0 + q4 * 32 + 31 - p.causal_off, q_first) * w.G : 0;
            float total = 0.f;
            int n = n0 + ((n0 ^ odd) & 1);
            for (int u = c.u0 + (n - n0); u < c.u1; u += 2, n += 2) {
                const int st = n % TSTAGES;
                ok = mbar_wait(smem_u32(&bars.t_full[st]), (n / TSTAGES) & 1, &abort_flag);
                if (u >= u_see) {
                    ok = ok && mbar_wait(sfull, phase, &abort_flag);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    phase ^= 1;
                    tc_fence_after();
                    if (u >= u_full && !holes[st]) {
                        total += sum_tile<false>(taddr, toff0 + st * (TB * 4), c2, 0, sempty, lane);
                    } else {
                        // columns below qmin are rows that do not see this key
                        const int q0 = (q_first + u / w.G) * TB;
                        const int qmin = w.causal ? (int)max(0LL, min((long long)TB, (long long)key - p.causal_off - q0)) : 0;
                        total += sum_tile<true>(taddr, toff0 + st * (TB * 4), c2, qmin, sempty, lane);
                    }
                } else {
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bars.t_empty[st]));
            }
            n0 += c.u1 - c.u0;
            // the two parities of a key meet; a warp that gave up still comes here, so that none waits at the
            // barriers alone, and all then stop together
            if (!ok) abort_flag = failed[kt] = 1;
            if (odd) other[kt][q4 * 32 + lane] = total;
            named_barrier(1 + kt, NCW / 2 * 32);
            const bool stop = failed[kt] != 0;
            if (!odd) total += other[kt][q4 * 32 + lane];
            named_barrier(1 + kt, NCW / 2 * 32);
            if (stop) ok = false;
            if (!ok) break;
            if (!odd) {
                if (c.u1 - c.u0 != c.units) {
                    const long long slot = 2LL * blockIdx.x + (c.u0 == 0 ? 1 : 0);
                    p.part[slot * 2 * TB + kt * TB + q4 * 32 + lane] = total;
                } else if (key < p.Sk) {
                    float *out = p.w + (long long)c.bh * p.Sk + key;
                    *out = p.accumulate ? *out + total : total;
                }
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

// Items that several CTAs shared, and items that no row sees: a block per item.  Latency: 3 us after the kernel above.
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
    // at least two steps for a CTA (B=1 Hq=32 Hkv=8 Sq=256: 8.6 us; four 10.6 us, eight 13.1 us; one 8.0 us, but 11.7 us
    // against 10.2 us for B=3 Hq=40 Hkv=8 Sq=201)
    const long long worth = w.total / 2;
    w.nc = (int)(worth < 1 ? 1 : worth < sm_count ? worth : sm_count);
    // Short items that are all alike, one to a CTA: no piece is shared, and nothing to join.
    const long long items = (long long)w.nkb * p.B * p.Hkv, steps = w.total / items;
    w.whole = items <= sm_count && steps >= 1 && steps <= kWholeSteps && (w.nkb == 1 || !w.causal);
    if (w.whole) w.nc = (int)items;
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
// Bound by reading K: B=8 Hq=32 Hkv=8 Sk=32768 D=128, 545 MB in 83 us, 0.97 of the copy's rate; on the CUDA cores
// 2223 us.
constexpr int RW = 8;   // warps per CTA

template <int D>
struct KeyTile {
    uint4 x[D / 32][2];
};

template <int D, int NT>
__global__ void __launch_bounds__(RW * 32, D <= 64 ? 3 : 2)
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
            lim[nt][c] = col >= R || off[nt][c] == -INFINITY ? 0 : p.causal ? max(0, min(p.Sk, col % p.Sq + p.causal_off + 1)) : p.Sk;
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
    long long parts = (4LL * sm_count * (D <= 64 ? 3 : 2) + items / 2) / items;
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
    return p.dtype == OSF_BF16 && p.D % 32 == 0 && p.D <= 128 && (long long)(p.Hq / p.Hkv) * p.Sq <= 16 && aligned16(p.k) &&
           ((p.k_sb | p.k_sh | p.k_ss) & 7) == 0;
}

bool key_weights_tc_supported(const KeyWeightsProblem &p) {
    return p.dtype == OSF_BF16 && (p.D == 64 || p.D == 128) && tensor_map_encoder() != nullptr &&
           tile_map_addressable(p.q, p.D, p.Sq, p.Hq, p.B, p.q_ss, p.q_sh, p.q_sb) &&
           tile_map_addressable(p.k, p.D, p.Sk, p.Hkv, p.B, p.k_ss, p.k_sh, p.k_sb);
}

size_t key_weights_tc_floats(int sm_count) { return (size_t)2 * sm_count * 2 * TB; }

template <int D>
static cudaError_t launch_rows_d(const KeyWeightsProblem &p, int sm_count, cudaStream_t s) {
    return (p.Hq / p.Hkv) * p.Sq <= 8 ? launch_rows_t<D, 1>(p, sm_count, s) : launch_rows_t<D, 2>(p, sm_count, s);
}

cudaError_t launch_key_weights_rows(const KeyWeightsProblem &p, int sm_count, cudaStream_t s) {
    return p.D == 32   ? launch_rows_d<32>(p, sm_count, s)
           : p.D == 64 ? launch_rows_d<64>(p, sm_count, s)
           : p.D == 96 ? launch_rows_d<96>(p, sm_count, s)
                       : launch_rows_d<128>(p, sm_count, s);
}

cudaError_t launch_key_weights_tc(const KeyWeightsProblem &p, int sm_count, cudaStream_t s) {
    const KwPlan w = make_plan(p, sm_count);
    cudaError_t e = cudaSuccess;
    if (w.total > 0) e = p.D == 64 ? launch_tc_t<64>(p, w, s) : launch_tc_t<128>(p, w, s);
    if (e != cudaSuccess || w.whole) return e;
    count_launches(1);
    return launch_dependent(key_weights_join_kernel, dim3((unsigned)w.nkb, (unsigned)(p.B * p.Hkv)), dim3(2 * TB), 0, s, p, w);
}

}  // namespace osf
