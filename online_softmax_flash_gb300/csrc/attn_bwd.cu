// Attention backward: dQ, dK, dV of O = softmax(mask(Q K^T * scale)) V for a loss whose gradient
// with respect to O is dO.  The pages describe only the forward pass (the single-pass attention
// of "softmax_attention", section "实现思路", with the GQA mapping and causal mask of
// "从零开始写Qwen3（五-其一）使用Triton实现自注意力", "自注意力原理" and "GQA"); the backward pass is
// the chain rule through that definition:
//     P = softmax(S),  dV = P^T dO,  dP = dO V^T,  dS = P * (dP - D),  D_i = rowsum(dO_i * O_i),
//     dQ = scale * dS K,  dK = scale * dS^T Q,
// with P rebuilt from the forward's log-sum-exp (P_ij = 2^(S_ij * scale * log2 e - lse_i log2 e)),
// so no [Sq, Sk] matrix is stored.  A kv head's dK and dV sum its G query heads.
//
// Kernels: (1) D_i, one warp per row; (2) dK/dV: one CTA per (b, kv head, 64 keys) walks every
// query head of the group and every query block that sees those keys, so each CTA owns its
// output rows and needs no atomics; (3) dQ: one CTA per (b, q head, 64 rows) walks the key
// blocks its rows see.  bf16 with D in {64, 128} runs (2) and (3) on warp-level tensor cores
// (mma.sync m16n8k16, bf16 in, fp32 accumulate): each warp owns 16 rows, the score
// accumulators are reused in registers as the A operand of the next product (as in the decode
// kernel); other problems run a CUDA-core version with one warp per output row.  bf16 with D in
// {64, 128} and aligned pointers normally takes the tcgen05 kernels of attn_bwd_tc.cu instead;
// the warp-level kernels remain for pointers TMA cannot address.
#include <mutex>
#include <type_traits>

#include "attn_bwd.cuh"
#include "attn_bwd_tc.cuh"
#include "sm100_ptx.cuh"

namespace osf {
namespace {

using namespace ptx;

__device__ __forceinline__ float ldf(const float *p) { return *p; }
__device__ __forceinline__ float ldf(const __nv_bfloat16 *p) { return __bfloat162float(*p); }

__device__ __forceinline__ bool visible(const BwdProblem &p, int i, int j) {
    return i < p.Sq && j < p.Sk && (!p.causal || j <= i + p.causal_off);
}

// ------------------------------------------------------------------ D_i = rowsum(dO_i * O_i)
template <typename T>
__global__ void __launch_bounds__(256) bwd_rowdot_kernel(BwdProblem p) {
    const long long rows = (long long)p.B * p.Hq * p.Sq;
    const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= rows) return;
    const T *o = static_cast<const T *>(p.o) + row * p.D;
    const T *g = static_cast<const T *>(p.dout) + row * p.D;
    float acc = 0.f;
    for (int d = lane; d < p.D; d += 32) acc += ldf(o + d) * ldf(g + d);
    acc = warp_sum(acc);
    if (lane == 0) p.dvec[row] = acc;
}

// bf16 with D = 32 * VW (VW = 2 or 4 elements per lane) and rows starting on VW * 2-byte
// boundaries: one warp per four rows, every load of the four rows issued before any arithmetic.
template <int VW>
__global__ void __launch_bounds__(256) bwd_rowdot_vec_kernel(BwdProblem p) {
    using V = typename std::conditional<VW == 4, uint2, uint32_t>::type;
    constexpr int R = 4;
    const long long rows = (long long)p.B * p.Hq * p.Sq;
    const long long row0 = ((long long)blockIdx.x * 8 + (threadIdx.x >> 5)) * R;
    const int lane = threadIdx.x & 31;
    V o[R], g[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const long long row = row0 + r;
        if (row < rows) {
            o[r] = reinterpret_cast<const V *>(static_cast<const __nv_bfloat16 *>(p.o) + row * p.D)[lane];
            g[r] = reinterpret_cast<const V *>(static_cast<const __nv_bfloat16 *>(p.dout) + row * p.D)[lane];
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        float acc = 0.f;
        if (row0 + r < rows) {
            const uint32_t *ow = reinterpret_cast<const uint32_t *>(&o[r]);
            const uint32_t *gw = reinterpret_cast<const uint32_t *>(&g[r]);
#pragma unroll
            for (int w = 0; w < VW / 2; ++w)
                acc += __uint_as_float(ow[w] << 16) * __uint_as_float(gw[w] << 16) +
                       __uint_as_float(ow[w] & 0xffff0000u) * __uint_as_float(gw[w] & 0xffff0000u);
        }
        acc = warp_sum(acc);
        if (lane == r && row0 + r < rows) p.dvec[row0 + r] = acc;
    }
}

// bf16 with D = 8 * LPR and 16-byte aligned rows: LPR lanes per row, one 16-byte load of O and
// of dO per lane and row, four rounds of 32 / LPR rows per warp, every load issued before any
// arithmetic; the partial sums meet within each group of LPR lanes.
template <int LPR>
__global__ void __launch_bounds__(256) bwd_rowdot_v16_kernel(BwdProblem p) {
    constexpr int RPI = 32 / LPR, IT = 4, RPW = RPI * IT;
    const long long rows = (long long)p.B * p.Hq * p.Sq;
    const int lane = threadIdx.x & 31, sub = lane / LPR, c = lane % LPR;
    const long long wrow = ((long long)blockIdx.x * 8 + (threadIdx.x >> 5)) * RPW;
    uint4 o[IT], g[IT];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const long long row = wrow + i * RPI + sub;
        if (row < rows) {
            o[i] = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.o) + row * p.D)[c];
            g[i] = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.dout) + row * p.D)[c];
        }
    }
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const long long row = wrow + i * RPI + sub;
        float acc = 0.f;
        if (row < rows) {
            const uint32_t ow[4] = {o[i].x, o[i].y, o[i].z, o[i].w}, gw[4] = {g[i].x, g[i].y, g[i].z, g[i].w};
#pragma unroll
            for (int w = 0; w < 4; ++w)
                acc += __uint_as_float(ow[w] << 16) * __uint_as_float(gw[w] << 16) +
                       __uint_as_float(ow[w] & 0xffff0000u) * __uint_as_float(gw[w] & 0xffff0000u);
        }
#pragma unroll
        for (int off = LPR / 2; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
        if (c == 0 && row < rows) p.dvec[row] = acc;
    }
}

// ------------------------------------------------------------------ CUDA-core version
// One warp per query row: dQ_i = scale * sum_j dS_ij K_j.
template <typename T>
__global__ void __launch_bounds__(256) bwd_dq_simt_kernel(BwdProblem p) {
    const long long rows = (long long)p.B * p.Hq * p.Sq;
    const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= rows) return;
    const int i = (int)(row % p.Sq);
    const long long bh = row / p.Sq;
    const int b = (int)(bh / p.Hq), hq = (int)(bh % p.Hq);
    const int kvh = hq / (p.Hq / p.Hkv);
    const int D = p.D;
    const T *q = static_cast<const T *>(p.q) + row * D;
    const T *go = static_cast<const T *>(p.dout) + row * D;
    const T *K = static_cast<const T *>(p.k) + ((long long)b * p.Hkv + kvh) * p.Sk * D;
    const T *V = static_cast<const T *>(p.v) + ((long long)b * p.Hkv + kvh) * p.Sk * D;
    float qr[8], gr[8], acc[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        const int d = lane + 32 * c;
        qr[c] = d < D ? ldf(q + d) : 0.f;
        gr[c] = d < D ? ldf(go + d) : 0.f;
        acc[c] = 0.f;
    }
    const float lse2 = p.lse[row] * kLog2e, dv = p.dvec[row];
    const int j_end = p.causal ? min(p.Sk, max(0, i + p.causal_off + 1)) : p.Sk;
    for (int j = 0; j < j_end; ++j) {
        float s = 0.f, dp = 0.f;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const int d = lane + 32 * c;
            if (d < D) {
                s += qr[c] * ldf(K + (long long)j * D + d);
                dp += gr[c] * ldf(V + (long long)j * D + d);
            }
        }
        s = warp_sum(s);
        dp = warp_sum(dp);
        const float pr = ex2_approx(s * p.scale_log2 - lse2);
        const float ds = pr * (dp - dv);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const int d = lane + 32 * c;
            if (d < D) acc[c] += ds * ldf(K + (long long)j * D + d);
        }
    }
    T *dq = static_cast<T *>(p.dq) + row * D;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        const int d = lane + 32 * c;
        if (d < D) dq[d] = from_f32<T>(acc[c] * p.scale);
    }
}

// One warp per key row of a kv head: dV_j = sum_i P_ij dO_i, dK_j = scale * sum_i dS_ij Q_i over
// the G query heads of the group.
template <typename T>
__global__ void __launch_bounds__(256) bwd_dkdv_simt_kernel(BwdProblem p) {
    const long long rows = (long long)p.B * p.Hkv * p.Sk;
    const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= rows) return;
    const int j = (int)(row % p.Sk);
    const long long bk = row / p.Sk;
    const int b = (int)(bk / p.Hkv), kvh = (int)(bk % p.Hkv);
    const int G = p.Hq / p.Hkv, D = p.D;
    const T *k = static_cast<const T *>(p.k) + row * D;
    const T *v = static_cast<const T *>(p.v) + row * D;
    float kr[8], vr[8], dk[8], dv[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        const int d = lane + 32 * c;
        kr[c] = d < D ? ldf(k + d) : 0.f;
        vr[c] = d < D ? ldf(v + d) : 0.f;
        dk[c] = dv[c] = 0.f;
    }
    const int i_begin = p.causal ? max(0, j - p.causal_off) : 0;
    for (int g = 0; g < G; ++g) {
        const long long bh = (long long)b * p.Hq + kvh * G + g;
        const T *Q = static_cast<const T *>(p.q) + bh * p.Sq * D;
        const T *GO = static_cast<const T *>(p.dout) + bh * p.Sq * D;
        for (int i = i_begin; i < p.Sq; ++i) {
            float s = 0.f, dp = 0.f;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const int d = lane + 32 * c;
                if (d < D) {
                    s += kr[c] * ldf(Q + (long long)i * D + d);
                    dp += vr[c] * ldf(GO + (long long)i * D + d);
                }
            }
            s = warp_sum(s);
            dp = warp_sum(dp);
            const float pr = ex2_approx(s * p.scale_log2 - p.lse[bh * p.Sq + i] * kLog2e);
            const float ds = pr * (dp - p.dvec[bh * p.Sq + i]);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const int d = lane + 32 * c;
                if (d < D) {
                    dv[c] += pr * ldf(GO + (long long)i * D + d);
                    dk[c] += ds * ldf(Q + (long long)i * D + d);
                }
            }
        }
    }
    T *gk = static_cast<T *>(p.dk) + row * D;
    T *gv = static_cast<T *>(p.dv) + row * D;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        const int d = lane + 32 * c;
        if (d < D) {
            gk[d] = from_f32<T>(dk[c] * p.scale);
            gv[d] = from_f32<T>(dv[c]);
        }
    }
}

// ------------------------------------------------------------------ a window, on the CUDA cores
// dK, dV (DKV) of KPW keys per warp, or dQ of KPW query rows per warp, of a problem with a window (BwdProblem::window); any D up
// to 256, float32 or bfloat16.  A block's eight warps own neighbouring keys (rows), whose rows (keys) overlap for the most part:
// chunks of 32 of those are staged in shared memory for all of them.  For a chunk a lane first takes one of its rows (keys)
// and both dot products with each of the warp's vectors (16-byte reads, KPW products to each), which gives P and dS; then a
// channel of each 32, and adds up dS . b1 and P . b2 over the chunk.  Sums have one order.
// Keys of tiles with sinks are seen by every later row: their chunks of rows are shared out over p.parts blocks, whose sums meet
// in a second kernel.  (float32, B=1 Hq=8 Hkv=2, 2000 tokens of D=64, window 65, 3 sinks: 627 us with a block for all of them,
// 106 shared out.)
// This form, of many vectors, is bound by its reads of shared memory: KPW vectors to a warp divide them.  float32, B=4 Hq=32
// Hkv=8, 512 tokens of D=64, window 65: 300 us; the multiplications of the pairs seen alone take 39.
constexpr int RW_WARPS = 8, RW_CHUNK = 32;

template <int C, int KPW>
struct RowsCfg {
    static constexpr int DP = 32 * C, PITCH = DP + 4;   // an odd number of 16-byte pieces: reads of 32 rows do not clash
    static constexpr int B_FLOATS = RW_CHUNK * PITCH, A_FLOATS = RW_WARPS * KPW * 2 * DP, P_FLOATS = RW_WARPS * RW_CHUNK * 2 * KPW;
    static constexpr size_t SMEM = sizeof(float) * (2 * B_FLOATS + A_FLOATS + P_FLOATS);
};

// Four channels from d on, zeros from D on.  vec: rows start on 16-byte (bfloat16: 8-byte) boundaries and D % 4 == 0.
__device__ __forceinline__ float4 ld_four(const float *p, int d, int D, bool vec) {
    if (vec) return d < D ? *reinterpret_cast<const float4 *>(p + d) : make_float4(0.f, 0.f, 0.f, 0.f);
    return make_float4(d < D ? p[d] : 0.f, d + 1 < D ? p[d + 1] : 0.f, d + 2 < D ? p[d + 2] : 0.f, d + 3 < D ? p[d + 3] : 0.f);
}
__device__ __forceinline__ float4 ld_four(const __nv_bfloat16 *p, int d, int D, bool vec) {
    if (vec) {
        const uint2 v = d < D ? *reinterpret_cast<const uint2 *>(p + d) : make_uint2(0u, 0u);
        return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u), __uint_as_float(v.y << 16),
                           __uint_as_float(v.y & 0xffff0000u));
    }
    return make_float4(d < D ? ldf(p + d) : 0.f, d + 1 < D ? ldf(p + d + 1) : 0.f, d + 2 < D ? ldf(p + d + 2) : 0.f,
                       d + 3 < D ? ldf(p + d + 3) : 0.f);
}

// Which tile of `bid`'s head a block has (the shared ones come first, a block for each part), and its part.
__device__ __forceinline__ int part_tile(const BwdProblem &p, bool dkv, int t, int &part) {
    part = 0;
    if (!dkv) return t;
    if (t >= p.shared_tiles * p.parts) return t - p.shared_tiles * (p.parts - 1);
    part = t % p.parts;
    return t / p.parts;
}
// Sums of a part: [key][D] of dK (h = 0) or dV (1).
__device__ __forceinline__ float *part_sums(const BwdProblem &p, int tile, int part, int head, int h) {
    return p.part_acc + ((((size_t)tile * p.parts + part) * p.B * p.Hkv + head) * 2 + h) * p.part_keys * p.D;
}

template <typename T, int C, int KPW, bool DKV>
__device__ __forceinline__ void window_rows(const BwdProblem &p, int bid, int tiles, bool vec) {
    using R = RowsCfg<C, KPW>;
    constexpr int PITCH = R::PITCH, DP = R::DP;
    extern __shared__ __align__(16) float rw_smem[];
    __shared__ float s_lse[RW_CHUNK], s_dvec[RW_CHUNK];
    float *b1 = rw_smem, *b2 = b1 + R::B_FLOATS, *av = b2 + R::B_FLOATS, *spd = av + R::A_FLOATS;
    const int D = p.D, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int part;
    const int tile = part_tile(p, DKV, bid % tiles, part), head = bid / tiles, G = p.Hq / p.Hkv;
    const int b = DKV ? head / p.Hkv : head / p.Hq, kvh = DKV ? head % p.Hkv : head % p.Hq / G;
    const int n_outer = DKV ? p.Sk : p.Sq, o0 = tile * RW_WARPS * KPW, o1 = min(o0 + RW_WARPS * KPW, n_outer);
    const T *A1 = static_cast<const T *>(DKV ? p.k : p.q) + (long long)head * n_outer * D;
    const T *A2 = static_cast<const T *>(DKV ? p.v : p.dout) + (long long)head * n_outer * D;
#pragma unroll
    for (int i = tid; i < RW_WARPS * KPW * DP / 4; i += RW_WARPS * 32) {
        const int o = i / (DP / 4), d = i % (DP / 4) * 4;
        const bool ok = o0 + o < o1;
        const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
        *reinterpret_cast<float4 *>(av + (o * 2) * DP + d) = ok ? ld_four(A1 + (long long)(o0 + o) * D, d, D, vec) : z;
        *reinterpret_cast<float4 *>(av + (o * 2 + 1) * DP + d) = ok ? ld_four(A2 + (long long)(o0 + o) * D, d, D, vec) : z;
    }
    // what the block's vectors meet: rows [i0, i1) of each of the group's heads, or the keys of a stream of chunks
    int i0 = 0, i1 = 0, steps;
    KeyStream ks{};
    if (DKV) {
        i0 = max(0, o0 - p.causal_off);
        i1 = o0 < p.sinks ? p.Sq : min(p.Sq, max(0, o1 - 1 - p.causal_off + p.window));
        steps = i1 > i0 ? G * ((i1 - i0 + RW_CHUNK - 1) / RW_CHUNK) : 0;
    } else {
        ks = key_stream(o0 + p.causal_off, o1 - 1 + p.causal_off, p.Sk, p.window, p.sinks, RW_CHUNK);
        steps = ks.n;
    }
    const int per_head = DKV && steps ? steps / G : 1;
    const bool partial = DKV && p.parts > 1 && tile < p.shared_tiles;   // this block has steps st0 .. steps - 1 alone
    int st0 = 0;
    if (partial) {
        st0 = (int)((long long)steps * part / p.parts);
        steps = (int)((long long)steps * (part + 1) / p.parts);
    }
    // chunk st: rows c0 .. c0 + cnt - 1 of head bh of the two arrays
    auto chunk = [&](int st, long long &bh, int &c0, int &cnt) {
        const int g = st / per_head;
        bh = DKV ? (long long)b * p.Hq + kvh * G + g : (long long)b * p.Hkv + kvh;
        c0 = DKV ? i0 + (st - g * per_head) * RW_CHUNK : ks.tile(st) * RW_CHUNK;
        cnt = min(RW_CHUNK, (DKV ? i1 : p.Sk) - c0);
    };
    float4 n1[C], n2[C];   // the next chunk, on its way
    float n_lse = 0.f;
    auto fetch = [&](int st) {
        long long bh;
        int c0, cnt;
        chunk(st, bh, c0, cnt);
        const int n_inner = DKV ? p.Sq : p.Sk;
        const T *B1 = static_cast<const T *>(DKV ? p.q : p.k) + (bh * n_inner + c0) * D;
        const T *B2 = static_cast<const T *>(DKV ? p.dout : p.v) + (bh * n_inner + c0) * D;
        auto rows = [&](auto v) {   // (a test of `vec` at each load keeps them from being in flight together)
#pragma unroll
            for (int e = 0; e < C; ++e) {
                const int f = tid + 256 * e, r = f / (DP / 4), d = f % (DP / 4) * 4;
                n1[e] = ld_four(B1 + (long long)min(r, cnt - 1) * D, r < cnt ? d : D, D, decltype(v)::value);
                n2[e] = ld_four(B2 + (long long)min(r, cnt - 1) * D, r < cnt ? d : D, D, decltype(v)::value);
            }
        };
        if (vec) rows(std::true_type{});
        else rows(std::false_type{});
        if (DKV && tid < 2 * RW_CHUNK) {
            const int r = tid & (RW_CHUNK - 1);
            n_lse = r >= cnt ? 0.f : tid < RW_CHUNK ? p.lse[bh * p.Sq + c0 + r] * kLog2e : p.dvec[bh * p.Sq + c0 + r];
        }
    };
    float acc1[KPW][C], acc2[KPW][C], lse_o[KPW], dvec_o[KPW];
#pragma unroll
    for (int k = 0; k < KPW; ++k) {
        const int o = o0 + warp * KPW + k;
        lse_o[k] = !DKV && o < o1 ? p.lse[(long long)head * p.Sq + o] * kLog2e : 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c) acc1[k][c] = acc2[k][c] = 0.f;
    }
    griddep_wait();   // launched as a dependent of the kernel that writes the row sums
#pragma unroll
    for (int k = 0; k < KPW; ++k) {
        const int o = o0 + warp * KPW + k;
        dvec_o[k] = !DKV && o < o1 ? p.dvec[(long long)head * p.Sq + o] : 0.f;
    }
    if (steps > st0) fetch(st0);
    const float *mine = av + warp * KPW * 2 * DP;
    float *mp = spd + warp * RW_CHUNK * 2 * KPW;
    const int d_end = (D + 3) / 4 * 4;
    for (int st = st0; st < steps; ++st) {
        long long bh;
        int c0, cnt;
        chunk(st, bh, c0, cnt);
        __syncthreads();   // the previous chunk is done with (and the vectors are there, first time)
#pragma unroll
        for (int e = 0; e < C; ++e) {
            const int f = tid + 256 * e, r = f / (DP / 4), d = f % (DP / 4) * 4;
            *reinterpret_cast<float4 *>(b1 + r * PITCH + d) = n1[e];
            *reinterpret_cast<float4 *>(b2 + r * PITCH + d) = n2[e];
        }
        if (DKV && tid < 2 * RW_CHUNK) (tid < RW_CHUNK ? s_lse : s_dvec)[tid & (RW_CHUNK - 1)] = n_lse;
        __syncthreads();
        if (st + 1 < steps) fetch(st + 1);
        float s[KPW], t[KPW];
#pragma unroll
        for (int k = 0; k < KPW; ++k) s[k] = t[k] = 0.f;
#pragma unroll 4
        for (int d = 0; d < d_end; d += 4) {
            const float4 x = *reinterpret_cast<const float4 *>(b1 + lane * PITCH + d);
            const float4 y = *reinterpret_cast<const float4 *>(b2 + lane * PITCH + d);
#pragma unroll
            for (int k = 0; k < KPW; ++k) {
                const float4 u = *reinterpret_cast<const float4 *>(mine + 2 * k * DP + d);
                const float4 v = *reinterpret_cast<const float4 *>(mine + (2 * k + 1) * DP + d);
                s[k] = fmaf(x.x, u.x, s[k]); s[k] = fmaf(x.y, u.y, s[k]); s[k] = fmaf(x.z, u.z, s[k]); s[k] = fmaf(x.w, u.w, s[k]);
                t[k] = fmaf(y.x, v.x, t[k]); t[k] = fmaf(y.y, v.y, t[k]); t[k] = fmaf(y.z, v.z, t[k]); t[k] = fmaf(y.w, v.w, t[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < KPW; ++k) {
            const int o = o0 + warp * KPW + k, key = DKV ? o : c0 + lane, pos = (DKV ? c0 + lane : o) + p.causal_off;
            const bool sees = o < o1 && lane < cnt && key <= pos && (key > pos - p.window || key < p.sinks);
            const float pr = sees ? ex2_approx(s[k] * p.scale_log2 - (DKV ? s_lse[lane] : lse_o[k])) : 0.f;
            mp[lane * 2 * KPW + k] = sees ? pr * (t[k] - (DKV ? s_dvec[lane] : dvec_o[k])) : 0.f;
            if (DKV) mp[lane * 2 * KPW + KPW + k] = pr;
        }
        __syncwarp();
#pragma unroll 8
        for (int r = 0; r < RW_CHUNK; ++r) {
            float ds[KPW], pr[KPW];
            if constexpr (KPW == 4) {
                const float4 a = *reinterpret_cast<const float4 *>(mp + 8 * r);
                ds[0] = a.x; ds[1] = a.y; ds[2] = a.z; ds[3] = a.w;
                if (DKV) {
                    const float4 q = *reinterpret_cast<const float4 *>(mp + 8 * r + 4);
                    pr[0] = q.x; pr[1] = q.y; pr[2] = q.z; pr[3] = q.w;
                }
            } else {
                ds[0] = mp[2 * r];
                pr[0] = DKV ? mp[2 * r + 1] : 0.f;
            }
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const float x = b1[r * PITCH + lane + 32 * c];
#pragma unroll
                for (int k = 0; k < KPW; ++k) acc1[k][c] = fmaf(ds[k], x, acc1[k][c]);
                if (DKV) {
                    const float y = b2[r * PITCH + lane + 32 * c];
#pragma unroll
                    for (int k = 0; k < KPW; ++k) acc2[k][c] = fmaf(pr[k], y, acc2[k][c]);
                }
            }
        }
    }
    T *O1 = static_cast<T *>(DKV ? p.dk : p.dq) + (long long)head * n_outer * D;
    T *O2 = static_cast<T *>(p.dv) + (long long)head * n_outer * D;
#pragma unroll
    for (int k = 0; k < KPW; ++k) {
        const int o = o0 + warp * KPW + k;
        if (o >= o1) break;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int d = lane + 32 * c;
            if (d >= D) continue;
            if (partial) {
                part_sums(p, tile, part, head, 0)[(o - o0) * D + d] = acc1[k][c];
                part_sums(p, tile, part, head, 1)[(o - o0) * D + d] = acc2[k][c];
            } else {
                O1[(long long)o * D + d] = from_f32<T>(acc1[k][c] * p.scale);
                if (DKV) O2[(long long)o * D + d] = from_f32<T>(acc2[k][c]);
            }
        }
    }
}

// The same where there are few vectors, D up to 128: all warps of a block take its eight vectors, each against every NW-th
// chunk, which it stages for itself, and their sums meet in the order of the warps: a block's walk is NW times shorter, and no
// warp waits for another's chunk.  Bound by what a block does one after another (loads, two products, sums, the join).
// float32, B=1 Hq=4 Hkv=2, 301 tokens of D=64, window 65, 3 sinks: 20 us with the row sums and the join of the parts, of which
// launches 10 (52 with a key to a warp and chunks shared by the block, 264 with a reduction over the lanes for every pair).
template <int C>
struct FewCfg {
    static constexpr int V = 8, NW = C == 2 ? 8 : 4, DP = 32 * C, PITCH = DP + 4, SP = 2 * V + 4;
    static constexpr int B_FLOATS = RW_CHUNK * PITCH, WARP_FLOATS = 2 * B_FLOATS + RW_CHUNK * SP;
    static constexpr size_t SMEM = sizeof(float) * (V * 2 * DP + NW * WARP_FLOATS);
    static_assert(2 * V * DP <= WARP_FLOATS, "a warp's sums take its chunk's place");
};
template <typename T, int C, bool DKV>
__device__ __forceinline__ void window_few(const BwdProblem &p, int bid, int tiles, bool vec) {
    using F = FewCfg<C>;
    constexpr int V = F::V, NW = F::NW, DP = F::DP, PITCH = F::PITCH;
    extern __shared__ __align__(16) float rw_smem[];
    const int D = p.D, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    float *av = rw_smem, *b1 = av + V * 2 * DP + warp * F::WARP_FLOATS, *b2 = b1 + F::B_FLOATS, *sp = b2 + F::B_FLOATS;
    int part;
    const int tile = part_tile(p, DKV, bid % tiles, part), head = bid / tiles, G = p.Hq / p.Hkv;
    const int b = DKV ? head / p.Hkv : head / p.Hq, kvh = DKV ? head % p.Hkv : head % p.Hq / G;
    const int n_outer = DKV ? p.Sk : p.Sq, n_inner = DKV ? p.Sq : p.Sk, o0 = tile * V, o1 = min(o0 + V, n_outer);
    const T *A1 = static_cast<const T *>(DKV ? p.k : p.q) + (long long)head * n_outer * D;
    const T *A2 = static_cast<const T *>(DKV ? p.v : p.dout) + (long long)head * n_outer * D;
    const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = tid; i < V * DP / 4; i += NW * 32) {
        const int o = i / (DP / 4), d = i % (DP / 4) * 4;
        const bool ok = o0 + o < o1;
        *reinterpret_cast<float4 *>(av + (o * 2) * DP + d) = ok ? ld_four(A1 + (long long)(o0 + o) * D, d, D, vec) : z;
        *reinterpret_cast<float4 *>(av + (o * 2 + 1) * DP + d) = ok ? ld_four(A2 + (long long)(o0 + o) * D, d, D, vec) : z;
    }
    int i0 = 0, i1 = 0, steps;
    KeyStream ks{};
    if (DKV) {
        i0 = max(0, o0 - p.causal_off);
        i1 = o0 < p.sinks ? p.Sq : min(p.Sq, max(0, o1 - 1 - p.causal_off + p.window));
        steps = i1 > i0 ? G * ((i1 - i0 + RW_CHUNK - 1) / RW_CHUNK) : 0;
    } else {
        ks = key_stream(o0 + p.causal_off, o1 - 1 + p.causal_off, p.Sk, p.window, p.sinks, RW_CHUNK);
        steps = ks.n;
    }
    const int per_head = DKV && steps ? steps / G : 1, d_end = (D + 3) / 4 * 4;
    const bool partial = DKV && p.parts > 1 && tile < p.shared_tiles;   // this block has steps st0 .. steps - 1 alone
    int st0 = 0;
    if (partial) {
        st0 = (int)((long long)steps * part / p.parts);
        steps = (int)((long long)steps * (part + 1) / p.parts);
    }
    float acc1[V][C], acc2[V][C];
#pragma unroll
    for (int k = 0; k < V; ++k)
#pragma unroll
        for (int c = 0; c < C; ++c) acc1[k][c] = acc2[k][c] = 0.f;
    griddep_wait();   // launched as a dependent of the kernel that writes the row sums
    __syncthreads();
    for (int st = st0 + warp; st < steps; st += NW) {
        const int g = st / per_head;
        const long long bh = DKV ? (long long)b * p.Hq + kvh * G + g : (long long)b * p.Hkv + kvh;
        const int c0 = DKV ? i0 + (st - g * per_head) * RW_CHUNK : ks.tile(st) * RW_CHUNK;
        const int cnt = min(RW_CHUNK, (DKV ? i1 : p.Sk) - c0);
        const T *B1 = static_cast<const T *>(DKV ? p.q : p.k) + (bh * n_inner + c0) * D;
        const T *B2 = static_cast<const T *>(DKV ? p.dout : p.v) + (bh * n_inner + c0) * D;
        float lse = 0.f, dvec = 0.f;
        if (DKV && lane < cnt) {
            lse = p.lse[bh * p.Sq + c0 + lane] * kLog2e;
            dvec = p.dvec[bh * p.Sq + c0 + lane];
        }
        constexpr int ROUND = 8;   // loads of each array that are in flight together
        auto stage = [&](auto v) {   // (see above)
#pragma unroll 1
            for (int f0 = 0; f0 < RW_CHUNK * DP / 4; f0 += 32 * ROUND) {
                float4 n1[ROUND], n2[ROUND];
#pragma unroll
                for (int e = 0; e < ROUND; ++e) {
                    const int f = f0 + 32 * e + lane, r = f / (DP / 4), d = f % (DP / 4) * 4;
                    n1[e] = ld_four(B1 + (long long)min(r, cnt - 1) * D, r < cnt ? d : D, D, decltype(v)::value);
                    n2[e] = ld_four(B2 + (long long)min(r, cnt - 1) * D, r < cnt ? d : D, D, decltype(v)::value);
                }
#pragma unroll
                for (int e = 0; e < ROUND; ++e) {
                    const int f = f0 + 32 * e + lane, r = f / (DP / 4), d = f % (DP / 4) * 4;
                    *reinterpret_cast<float4 *>(b1 + r * PITCH + d) = n1[e];
                    *reinterpret_cast<float4 *>(b2 + r * PITCH + d) = n2[e];
                }
            }
        };
        if (vec) stage(std::true_type{});
        else stage(std::false_type{});
        __syncwarp();
        float s[V], t[V];
#pragma unroll
        for (int k = 0; k < V; ++k) s[k] = t[k] = 0.f;
#pragma unroll 2
        for (int d = 0; d < d_end; d += 4) {
            const float4 x = *reinterpret_cast<const float4 *>(b1 + lane * PITCH + d);
            const float4 y = *reinterpret_cast<const float4 *>(b2 + lane * PITCH + d);
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const float4 u = *reinterpret_cast<const float4 *>(av + 2 * k * DP + d);
                const float4 v = *reinterpret_cast<const float4 *>(av + (2 * k + 1) * DP + d);
                s[k] = fmaf(x.x, u.x, s[k]); s[k] = fmaf(x.y, u.y, s[k]); s[k] = fmaf(x.z, u.z, s[k]); s[k] = fmaf(x.w, u.w, s[k]);
                t[k] = fmaf(y.x, v.x, t[k]); t[k] = fmaf(y.y, v.y, t[k]); t[k] = fmaf(y.z, v.z, t[k]); t[k] = fmaf(y.w, v.w, t[k]);
            }
        }
        float pr[V];
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int o = o0 + k, key = DKV ? o : c0 + lane, pos = (DKV ? c0 + lane : o) + p.causal_off;
            const bool sees = o < o1 && lane < cnt && key <= pos && (key > pos - p.window || key < p.sinks);
            if (!DKV) {
                lse = sees ? p.lse[(long long)head * p.Sq + o] * kLog2e : 0.f;
                dvec = sees ? p.dvec[(long long)head * p.Sq + o] : 0.f;
            }
            pr[k] = sees ? ex2_approx(s[k] * p.scale_log2 - lse) : 0.f;
            t[k] = sees ? pr[k] * (t[k] - dvec) : 0.f;
        }
#pragma unroll
        for (int k = 0; k < V; k += 4) {
            *reinterpret_cast<float4 *>(sp + lane * F::SP + k) = make_float4(t[k], t[k + 1], t[k + 2], t[k + 3]);
            if (DKV) *reinterpret_cast<float4 *>(sp + lane * F::SP + V + k) = make_float4(pr[k], pr[k + 1], pr[k + 2], pr[k + 3]);
        }
        __syncwarp();
#pragma unroll 4
        for (int r = 0; r < RW_CHUNK; ++r) {
            float ds[V], q[V];
#pragma unroll
            for (int k = 0; k < V; k += 4) {
                const float4 a = *reinterpret_cast<const float4 *>(sp + r * F::SP + k);
                ds[k] = a.x; ds[k + 1] = a.y; ds[k + 2] = a.z; ds[k + 3] = a.w;
                if (DKV) {
                    const float4 e = *reinterpret_cast<const float4 *>(sp + r * F::SP + V + k);
                    q[k] = e.x; q[k + 1] = e.y; q[k + 2] = e.z; q[k + 3] = e.w;
                }
            }
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const float x = b1[r * PITCH + lane + 32 * c];
#pragma unroll
                for (int k = 0; k < V; ++k) acc1[k][c] = fmaf(ds[k], x, acc1[k][c]);
                if (DKV) {
                    const float y = b2[r * PITCH + lane + 32 * c];
#pragma unroll
                    for (int k = 0; k < V; ++k) acc2[k][c] = fmaf(q[k], y, acc2[k][c]);
                }
            }
        }
        __syncwarp();
    }
#pragma unroll
    for (int k = 0; k < V; ++k)
#pragma unroll
        for (int c = 0; c < C; ++c) {
            b1[(2 * k) * DP + lane + 32 * c] = acc1[k][c];
            if (DKV) b1[(2 * k + 1) * DP + lane + 32 * c] = acc2[k][c];
        }
    __syncthreads();
    const float *sums = av + V * 2 * DP;
    T *O1 = static_cast<T *>(DKV ? p.dk : p.dq) + ((long long)head * n_outer + o0) * D;
    T *O2 = static_cast<T *>(p.dv) + ((long long)head * n_outer + o0) * D;
    const int used = min(NW, steps - st0);
    for (int i = tid; i < (o1 - o0) * DP; i += NW * 32) {
        const int o = i / DP, d = i % DP;
        if (d >= D) continue;
        float a = 0.f, e = 0.f;
        for (int w = 0; w < used; ++w) {
            a += sums[w * F::WARP_FLOATS + 2 * o * DP + d];
            if (DKV) e += sums[w * F::WARP_FLOATS + (2 * o + 1) * DP + d];
        }
        if (partial) {
            part_sums(p, tile, part, head, 0)[o * D + d] = a;
            part_sums(p, tile, part, head, 1)[o * D + d] = e;
            continue;
        }
        O1[(long long)o * D + d] = from_f32<T>(a * p.scale);
        if (DKV) O2[(long long)o * D + d] = from_f32<T>(e);
    }
}
template <typename T, int C>
__global__ void __launch_bounds__(FewCfg<C>::NW * 32)
bwd_window_few_kernel(BwdProblem p, unsigned kv_blocks, int kv_tiles, int q_tiles, int vec) {
    if (blockIdx.x < kv_blocks) window_few<T, C, true>(p, blockIdx.x, kv_tiles, vec);
    else window_few<T, C, false>(p, blockIdx.x - kv_blocks, q_tiles, vec);
}

// One grid: the blocks of dK and dV, then those of dQ.
template <typename T, int C, int KPW>
__global__ void __launch_bounds__(RW_WARPS * 32)
bwd_window_rows_kernel(BwdProblem p, unsigned kv_blocks, int kv_tiles, int q_tiles, int vec) {
    if (blockIdx.x < kv_blocks) window_rows<T, C, KPW, true>(p, blockIdx.x, kv_tiles, vec);
    else window_rows<T, C, KPW, false>(p, blockIdx.x - kv_blocks, q_tiles, vec);
}

// dK and dV of the keys in shared tiles: the parts' sums, added in the order of the parts.  gridDim = (values of the tiles / 256,
// b * kv head, dK | dV).
template <typename T>
__global__ void __launch_bounds__(256) bwd_rows_sum_kernel(const BwdProblem p) {
    griddep_wait();
    const int i = blockIdx.x * 256 + threadIdx.x, key = i / p.D, d = i % p.D, head = blockIdx.y, h = blockIdx.z;
    if (key >= min(p.shared_tiles * p.part_keys, p.Sk)) return;
    const size_t part = (size_t)p.B * p.Hkv * 2 * p.part_keys * p.D;
    const float *src = part_sums(p, key / p.part_keys, 0, head, h) + key % p.part_keys * p.D + d;
    float a = 0.f;
#pragma unroll 8
    for (int s = 0; s < p.parts; ++s) a += src[s * part];
    static_cast<T *>(h ? p.dv : p.dk)[((long long)head * p.Sk + key) * p.D + d] = from_f32<T>(h ? a : a * p.scale);
}

using RowsKernel = void (*)(BwdProblem, unsigned, int, int, int);
template <typename T>
cudaError_t launch_rows_k(BwdProblem p, RowsKernel kernel, int per, int threads, size_t smem, cudaStream_t s) {
    cudaError_t e = set_max_dynamic_smem((const void *)kernel, (int)smem);
    if (e != cudaSuccess) return e;
    // (nothing to share out, or the plan is the tensor-core path's, whose tensors TMA did not address)
    if (p.part_keys != per || p.shared_tiles == 0 || p.parts <= 1) {
        p.shared_tiles = 0;
        p.parts = 1;
    }
    const int kv_tiles = (p.Sk + per - 1) / per + p.shared_tiles * (p.parts - 1), q_tiles = (p.Sq + per - 1) / per;
    const long long kv = (long long)kv_tiles * p.B * p.Hkv, all = kv + (long long)q_tiles * p.B * p.Hq;
    if (all >= (1LL << 31)) return cudaErrorInvalidValue;
    const uintptr_t at = reinterpret_cast<uintptr_t>(p.q) | reinterpret_cast<uintptr_t>(p.k) | reinterpret_cast<uintptr_t>(p.v) |
                         reinterpret_cast<uintptr_t>(p.dout);
    const int vec = p.D % 4 == 0 && at % (4 * sizeof(T)) == 0;
    count_launches(1);
    e = launch_dependent(kernel, dim3((unsigned)all), dim3(threads), smem, s, p, (unsigned)kv, kv_tiles, q_tiles, vec);
    if (e != cudaSuccess || p.parts == 1) return e;
    count_launches(1);
    const dim3 g((unsigned)(((long long)p.shared_tiles * per * p.D + 255) / 256), (unsigned)(p.B * p.Hkv), 2);
    return launch_dependent(bwd_rows_sum_kernel<T>, g, dim3(256), 0, s, p);
}
template <typename T, int C, int KPW>
cudaError_t launch_rows(const BwdProblem &p, cudaStream_t s) {
    return launch_rows_k<T>(p, bwd_window_rows_kernel<T, C, KPW>, RW_WARPS * KPW, RW_WARPS * 32, RowsCfg<C, KPW>::SMEM, s);
}
template <typename T, int C>
cudaError_t launch_few(const BwdProblem &p, cudaStream_t s) {
    return launch_rows_k<T>(p, bwd_window_few_kernel<T, C>, FewCfg<C>::V, FewCfg<C>::NW * 32, FewCfg<C>::SMEM, s);
}
// Vectors to a block: 8 (the form for few vectors, or a vector to a warp where D > 128), or 32 where there are many: a block
// then runs long, and reads less.  (us, 8 against 32, window 600: float32 D = 64, 1806 vectors 27 against 78, 12000 158, 316, 20480
// 228, 406, 40960 439, 408, 81920 861, 678; D = 128, 1806 48, 126, 12000 318, 443, 20480 465, 377, 40960 904, 674; window 65, D = 64,
// 12000 75, 78, 40960 227, 161.)
int rows_per_block(long long B, int Hq, int Hkv, int Sq, int Sk, int D, int sm_count) {
    const long long vectors = B * ((long long)Hkv * Sk + (long long)Hq * Sq);
    return vectors >= (D > 128 ? 64LL : D > 64 ? 108LL : 216LL) * sm_count ? 32 : 8;
}
template <typename T>
cudaError_t launch_window_rows(const BwdProblem &p, cudaStream_t s) {
    int sms = 0;
    if (device_sm_count(&sms) != OSF_OK) return cudaErrorInvalidValue;
    const bool wide = rows_per_block(p.B, p.Hq, p.Hkv, p.Sq, p.Sk, p.D, sms) == 32;
    if (p.D <= 64) return wide ? launch_rows<T, 2, 4>(p, s) : launch_few<T, 2>(p, s);
    if (p.D <= 128) return wide ? launch_rows<T, 4, 4>(p, s) : launch_few<T, 4>(p, s);
    return wide ? launch_rows<T, 8, 4>(p, s) : launch_rows<T, 8, 1>(p, s);
}

// ------------------------------------------------------------------ tensor-core version (bf16)
// Shared-memory tiles are row-major with rows padded to D + 8 elements, so the 16-byte rows that
// ldmatrix reads for one 8x8 matrix fall in different banks.
template <int D> struct BwdCfg {
    static constexpr int LD = D + 8;
    static constexpr int BQ = D == 64 ? 64 : 32;   // query rows per step of the dK/dV kernel
    static constexpr int BK = D == 64 ? 64 : 32;   // keys per step of the dQ kernel
    static constexpr int NT = D / 8;               // n8 tiles across D
};

// Copy rows [r0, r0 + n) of a [rows_total, D] bf16 matrix into a padded tile (zero past the end).
template <int D>
__device__ __forceinline__ void load_tile(__nv_bfloat16 *dst, const __nv_bfloat16 *src, int r0, int n,
                                          int rows_total) {
    constexpr int LD = D + 8, VPR = D / 8;   // 16-byte vectors per row
    for (int idx = threadIdx.x; idx < n * VPR; idx += blockDim.x) {
        const int r = idx / VPR, c = idx % VPR;
        uint4 val = make_uint4(0u, 0u, 0u, 0u);
        if (r0 + r < rows_total) val = *reinterpret_cast<const uint4 *>(src + (long long)(r0 + r) * D + c * 8);
        *reinterpret_cast<uint4 *>(dst + r * LD + c * 8) = val;
    }
}

// A fragment (16 x 16) of rows r0.., cols c0.. of a padded tile.
__device__ __forceinline__ void ld_a(const __nv_bfloat16 *tile, int ld, int r0, int c0, uint32_t (&a)[4]) {
    const int lane = threadIdx.x & 31;
    const int r = r0 + (lane & 7) + ((lane >> 3) & 1) * 8, c = c0 + (lane >> 4) * 8;
    ldmatrix_x4(smem_u32(tile + r * ld + c), a[0], a[1], a[2], a[3]);
}
// B fragments of two n8 tiles where B[k][n] = tile[n][k] (n rows n0..n0+15, k cols k0..k0+15).
__device__ __forceinline__ void ld_b_nt(const __nv_bfloat16 *tile, int ld, int n0, int k0, uint32_t &b0, uint32_t &b1,
                                        uint32_t &b2, uint32_t &b3) {
    const int lane = threadIdx.x & 31, mi = lane >> 3, rr = lane & 7;
    const int r = n0 + ((mi >> 1) << 3) + rr, c = k0 + ((mi & 1) << 3);
    ldmatrix_x4(smem_u32(tile + r * ld + c), b0, b1, b2, b3);
}
// B fragments of two n8 tiles where B[k][n] = tile[k][n] (k rows k0..k0+15, n cols n0..n0+15).
__device__ __forceinline__ void ld_b_t(const __nv_bfloat16 *tile, int ld, int k0, int n0, uint32_t &b0, uint32_t &b1,
                                       uint32_t &b2, uint32_t &b3) {
    const int lane = threadIdx.x & 31, mi = lane >> 3, rr = lane & 7;
    const int r = k0 + ((mi & 1) << 3) + rr, c = n0 + ((mi >> 1) << 3);
    ldmatrix_x4_trans(smem_u32(tile + r * ld + c), b0, b1, b2, b3);
}
// A fragment (16 x 16) from the fp32 accumulators of two n8 tiles (cols 0-7 and 8-15).
__device__ __forceinline__ void acc_to_a(const float (&x)[4], const float (&y)[4], uint32_t (&a)[4]) {
    a[0] = pack_bf16x2(x[0], x[1]);
    a[1] = pack_bf16x2(x[2], x[3]);
    a[2] = pack_bf16x2(y[0], y[1]);
    a[3] = pack_bf16x2(y[2], y[3]);
}

// dK, dV for 64 keys (4 warps x 16) of one (b, kv head).
template <int D>
__global__ void __launch_bounds__(128) bwd_dkdv_mma_kernel(BwdProblem p) {
    using C = BwdCfg<D>;
    constexpr int KB = 64, LD = C::LD, BQ = C::BQ, NT = C::NT;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    __nv_bfloat16 *sK = reinterpret_cast<__nv_bfloat16 *>(smem_raw);
    __nv_bfloat16 *sV = sK + KB * LD, *sQ = sV + KB * LD, *sG = sQ + BQ * LD;
    float *sL = reinterpret_cast<float *>(sG + BQ * LD), *sDv = sL + BQ;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int key0 = blockIdx.x * KB;
    const int bk = blockIdx.y, b = bk / p.Hkv, kvh = bk % p.Hkv;
    const int G = p.Hq / p.Hkv;
    const __nv_bfloat16 *Kg = static_cast<const __nv_bfloat16 *>(p.k) + (long long)bk * p.Sk * D;
    const __nv_bfloat16 *Vg = static_cast<const __nv_bfloat16 *>(p.v) + (long long)bk * p.Sk * D;
    load_tile<D>(sK, Kg, key0, KB, p.Sk);
    load_tile<D>(sV, Vg, key0, KB, p.Sk);
    float dk[NT][4], dv[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) dk[t][e] = dv[t][e] = 0.f;
    const int kw = warp * 16;                           // this warp's keys within the block
    const int krow = key0 + kw + (lane >> 2);           // key of accumulator elements 0, 1 (+8: 2, 3)
    // first query row that sees a key of this block
    int q_first = p.causal ? max(0, key0 - p.causal_off) : 0;
    q_first = (q_first / BQ) * BQ;
    for (int g = 0; g < G; ++g) {
        const long long bh = (long long)b * p.Hq + kvh * G + g;
        const __nv_bfloat16 *Qg = static_cast<const __nv_bfloat16 *>(p.q) + bh * p.Sq * D;
        const __nv_bfloat16 *Gg = static_cast<const __nv_bfloat16 *>(p.dout) + bh * p.Sq * D;
        for (int q0 = q_first; q0 < p.Sq; q0 += BQ) {
            __syncthreads();   // previous step's Q, dO done (and K, V stored, first time)
            load_tile<D>(sQ, Qg, q0, BQ, p.Sq);
            load_tile<D>(sG, Gg, q0, BQ, p.Sq);
            for (int r = threadIdx.x; r < BQ; r += blockDim.x) {
                const bool ok = q0 + r < p.Sq;
                sL[r] = ok ? p.lse[bh * p.Sq + q0 + r] * kLog2e : INFINITY;   // P = 0 past Sq
                sDv[r] = ok ? p.dvec[bh * p.Sq + q0 + r] : 0.f;
            }
            __syncthreads();
            // S^T = K_w Q^T  [16 keys x BQ queries]
            float st[BQ / 8][4];
#pragma unroll
            for (int t = 0; t < BQ / 8; ++t) st[t][0] = st[t][1] = st[t][2] = st[t][3] = 0.f;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                uint32_t a[4];
                ld_a(sK, LD, kw, kk * 16, a);
#pragma unroll
                for (int j = 0; j < BQ / 16; ++j) {
                    uint32_t b0, b1, b2, b3;
                    ld_b_nt(sQ, LD, j * 16, kk * 16, b0, b1, b2, b3);
                    mma_m16n8k16_bf16(st[2 * j], a, b0, b1);
                    mma_m16n8k16_bf16(st[2 * j + 1], a, b2, b3);
                }
            }
            // P^T (masked), in place
#pragma unroll
            for (int t = 0; t < BQ / 8; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int qi = t * 8 + 2 * (lane & 3) + (e & 1);
                    const int kj = krow + (e >> 1) * 8;
                    st[t][e] = visible(p, q0 + qi, kj) ? ex2_approx(st[t][e] * p.scale_log2 - sL[qi]) : 0.f;
                }
            // dV += P^T dO
#pragma unroll
            for (int j = 0; j < BQ / 16; ++j) {
                uint32_t a[4];
                acc_to_a(st[2 * j], st[2 * j + 1], a);
#pragma unroll
                for (int dt = 0; dt < D / 16; ++dt) {
                    uint32_t b0, b1, b2, b3;
                    ld_b_t(sG, LD, j * 16, dt * 16, b0, b1, b2, b3);
                    mma_m16n8k16_bf16(dv[2 * dt], a, b0, b1);
                    mma_m16n8k16_bf16(dv[2 * dt + 1], a, b2, b3);
                }
            }
            // dP^T = V_w dO^T, then dS^T = P^T * (dP^T - D) in place
            float dpt[BQ / 8][4];
#pragma unroll
            for (int t = 0; t < BQ / 8; ++t) dpt[t][0] = dpt[t][1] = dpt[t][2] = dpt[t][3] = 0.f;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                uint32_t a[4];
                ld_a(sV, LD, kw, kk * 16, a);
#pragma unroll
                for (int j = 0; j < BQ / 16; ++j) {
                    uint32_t b0, b1, b2, b3;
                    ld_b_nt(sG, LD, j * 16, kk * 16, b0, b1, b2, b3);
                    mma_m16n8k16_bf16(dpt[2 * j], a, b0, b1);
                    mma_m16n8k16_bf16(dpt[2 * j + 1], a, b2, b3);
                }
            }
#pragma unroll
            for (int t = 0; t < BQ / 8; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int qi = t * 8 + 2 * (lane & 3) + (e & 1);
                    dpt[t][e] = st[t][e] * (dpt[t][e] - sDv[qi]);
                }
            // dK += dS^T Q
#pragma unroll
            for (int j = 0; j < BQ / 16; ++j) {
                uint32_t a[4];
                acc_to_a(dpt[2 * j], dpt[2 * j + 1], a);
#pragma unroll
                for (int dt = 0; dt < D / 16; ++dt) {
                    uint32_t b0, b1, b2, b3;
                    ld_b_t(sQ, LD, j * 16, dt * 16, b0, b1, b2, b3);
                    mma_m16n8k16_bf16(dk[2 * dt], a, b0, b1);
                    mma_m16n8k16_bf16(dk[2 * dt + 1], a, b2, b3);
                }
            }
        }
    }
    // write this warp's 16 keys
    __nv_bfloat16 *dKg = static_cast<__nv_bfloat16 *>(p.dk) + (long long)bk * p.Sk * D;
    __nv_bfloat16 *dVg = static_cast<__nv_bfloat16 *>(p.dv) + (long long)bk * p.Sk * D;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int kj = krow + h * 8;
            if (kj < p.Sk) {
                const int d = t * 8 + 2 * (lane & 3);
                *reinterpret_cast<uint32_t *>(dKg + (long long)kj * D + d) =
                    pack_bf16x2(dk[t][2 * h] * p.scale, dk[t][2 * h + 1] * p.scale);
                *reinterpret_cast<uint32_t *>(dVg + (long long)kj * D + d) = pack_bf16x2(dv[t][2 * h], dv[t][2 * h + 1]);
            }
        }
}

// dQ for 64 query rows (4 warps x 16) of one (b, q head).
template <int D>
__global__ void __launch_bounds__(128) bwd_dq_mma_kernel(BwdProblem p) {
    using C = BwdCfg<D>;
    constexpr int QB = 64, LD = C::LD, BK = C::BK, NT = C::NT;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    __nv_bfloat16 *sQ = reinterpret_cast<__nv_bfloat16 *>(smem_raw);
    __nv_bfloat16 *sG = sQ + QB * LD, *sK = sG + QB * LD, *sV = sK + BK * LD;
    float *sL = reinterpret_cast<float *>(sV + BK * LD), *sDv = sL + QB;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int q0 = blockIdx.x * QB;
    const long long bh = blockIdx.y;
    const int b = (int)(bh / p.Hq), hq = (int)(bh % p.Hq);
    const int kvh = hq / (p.Hq / p.Hkv);
    const __nv_bfloat16 *Kg = static_cast<const __nv_bfloat16 *>(p.k) + ((long long)b * p.Hkv + kvh) * p.Sk * D;
    const __nv_bfloat16 *Vg = static_cast<const __nv_bfloat16 *>(p.v) + ((long long)b * p.Hkv + kvh) * p.Sk * D;
    load_tile<D>(sQ, static_cast<const __nv_bfloat16 *>(p.q) + bh * p.Sq * D, q0, QB, p.Sq);
    load_tile<D>(sG, static_cast<const __nv_bfloat16 *>(p.dout) + bh * p.Sq * D, q0, QB, p.Sq);
    for (int r = threadIdx.x; r < QB; r += blockDim.x) {
        const bool ok = q0 + r < p.Sq;
        sL[r] = ok ? p.lse[bh * p.Sq + q0 + r] * kLog2e : INFINITY;
        sDv[r] = ok ? p.dvec[bh * p.Sq + q0 + r] : 0.f;
    }
    float dq[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) dq[t][0] = dq[t][1] = dq[t][2] = dq[t][3] = 0.f;
    const int qw = warp * 16;
    const int qrow = q0 + qw + (lane >> 2);   // query row of accumulator elements 0, 1 (+8: 2, 3)
    // last key any row of this block sees
    int k_end = p.Sk;
    if (p.causal) k_end = min(k_end, max(0, min(q0 + QB, p.Sq) - 1 + p.causal_off + 1));
    for (int k0 = 0; k0 < k_end; k0 += BK) {
        __syncthreads();
        load_tile<D>(sK, Kg, k0, BK, p.Sk);
        load_tile<D>(sV, Vg, k0, BK, p.Sk);
        __syncthreads();
        // S = Q_w K^T, dP = dO_w V^T  [16 rows x BK keys]
        float s[BK / 8][4], dp[BK / 8][4];
#pragma unroll
        for (int t = 0; t < BK / 8; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[t][e] = dp[t][e] = 0.f;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            uint32_t a[4], g[4];
            ld_a(sQ, LD, qw, kk * 16, a);
            ld_a(sG, LD, qw, kk * 16, g);
#pragma unroll
            for (int j = 0; j < BK / 16; ++j) {
                uint32_t b0, b1, b2, b3;
                ld_b_nt(sK, LD, j * 16, kk * 16, b0, b1, b2, b3);
                mma_m16n8k16_bf16(s[2 * j], a, b0, b1);
                mma_m16n8k16_bf16(s[2 * j + 1], a, b2, b3);
                ld_b_nt(sV, LD, j * 16, kk * 16, b0, b1, b2, b3);
                mma_m16n8k16_bf16(dp[2 * j], g, b0, b1);
                mma_m16n8k16_bf16(dp[2 * j + 1], g, b2, b3);
            }
        }
        // dS = P * (dP - D), P rebuilt from lse
#pragma unroll
        for (int t = 0; t < BK / 8; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int ri = qw + (lane >> 2) + (e >> 1) * 8;
                const int kj = k0 + t * 8 + 2 * (lane & 3) + (e & 1);
                const float pr = visible(p, q0 + ri, kj) ? ex2_approx(s[t][e] * p.scale_log2 - sL[ri]) : 0.f;
                s[t][e] = pr * (dp[t][e] - sDv[ri]);
            }
        // dQ += dS K
#pragma unroll
        for (int j = 0; j < BK / 16; ++j) {
            uint32_t a[4];
            acc_to_a(s[2 * j], s[2 * j + 1], a);
#pragma unroll
            for (int dt = 0; dt < D / 16; ++dt) {
                uint32_t b0, b1, b2, b3;
                ld_b_t(sK, LD, j * 16, dt * 16, b0, b1, b2, b3);
                mma_m16n8k16_bf16(dq[2 * dt], a, b0, b1);
                mma_m16n8k16_bf16(dq[2 * dt + 1], a, b2, b3);
            }
        }
    }
    __nv_bfloat16 *dQg = static_cast<__nv_bfloat16 *>(p.dq) + bh * p.Sq * D;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int qi = qrow + h * 8;
            if (qi < p.Sq)
                *reinterpret_cast<uint32_t *>(dQg + (long long)qi * D + t * 8 + 2 * (lane & 3)) =
                    pack_bf16x2(dq[t][2 * h] * p.scale, dq[t][2 * h + 1] * p.scale);
        }
}

template <int D>
cudaError_t launch_mma(const BwdProblem &p, cudaStream_t s) {
    using C = BwdCfg<D>;
    constexpr int LD = C::LD;
    const size_t smem_kv = (size_t)(2 * 64 + 2 * C::BQ) * LD * 2 + 2 * C::BQ * 4;
    const size_t smem_q = (size_t)(2 * 64 + 2 * C::BK) * LD * 2 + 2 * 64 * 4;
    cudaError_t attr_err = set_max_dynamic_smem((const void *)bwd_dkdv_mma_kernel<D>, (int)smem_kv);
    if (attr_err == cudaSuccess) attr_err = set_max_dynamic_smem((const void *)bwd_dq_mma_kernel<D>, (int)smem_q);
    if (attr_err != cudaSuccess) return attr_err;
    bwd_dkdv_mma_kernel<D><<<dim3((p.Sk + 63) / 64, p.B * p.Hkv), 128, smem_kv, s>>>(p);
    bwd_dq_mma_kernel<D><<<dim3((p.Sq + 63) / 64, p.B * p.Hq), 128, smem_q, s>>>(p);
    count_launches(2);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_simt(const BwdProblem &p, cudaStream_t s) {
    const long long rq = (long long)p.B * p.Hq * p.Sq, rk = (long long)p.B * p.Hkv * p.Sk;
    bwd_dkdv_simt_kernel<T><<<(unsigned)((rk + 7) / 8), 256, 0, s>>>(p);
    bwd_dq_simt_kernel<T><<<(unsigned)((rq + 7) / 8), 256, 0, s>>>(p);
    count_launches(2);
    return cudaGetLastError();
}

}  // namespace

bool attn_bwd_mma_supported(const BwdProblem &p) {
    if (p.dtype != OSF_BF16 || (p.D != 64 && p.D != 128)) return false;
    const uintptr_t a = reinterpret_cast<uintptr_t>(p.q) | reinterpret_cast<uintptr_t>(p.k) |
                        reinterpret_cast<uintptr_t>(p.v) | reinterpret_cast<uintptr_t>(p.dout) |
                        reinterpret_cast<uintptr_t>(p.dq) | reinterpret_cast<uintptr_t>(p.dk) |
                        reinterpret_cast<uintptr_t>(p.dv);
    return (a & 15u) == 0 && (p.Sk + 63) / 64 < 65536 && (long long)p.B * p.Hq < 65536;
}

BwdWindowPlan bwd_rows_plan(int B, int Hq, int Hkv, int Sq, int Sk, int D, int window, int sinks, int sm_count) {
    BwdWindowPlan w{};
    w.part_keys = rows_per_block(B, Hq, Hkv, Sq, Sk, D, sm_count);
    w.parts = 1;
    w.shared_tiles = (int)(((long long)sinks + w.part_keys - 1) / w.part_keys);
    const int tiles = (Sk - 1) / w.part_keys + 1;
    if (w.shared_tiles > tiles) w.shared_tiles = tiles;
    if (w.shared_tiles == 0) return w;
    // Keys of tiles with sinks are seen by every later row: their chunks of rows are shared out in parts as long as the others'
    // walks, or than a step of all warps, as long as the parts are within four blocks to an SM
    const long long chunks = ((long long)Sq + RW_CHUNK - 1) / RW_CHUNK, group = Hq / Hkv;
    long long walk = group * ((window + w.part_keys - 1) / RW_CHUNK + 1);
    if (walk < RW_WARPS) walk = RW_WARPS;
    const long long tiles_all = (long long)w.shared_tiles * B * Hkv;
    const long long parts = (group * chunks + walk - 1) / walk, most = (4LL * sm_count + tiles_all - 1) / tiles_all;
    w.parts = (int)(parts < most ? parts : most);
    return w;
}

cudaError_t launch_attn_bwd(const BwdProblem &p, cudaStream_t s) {
    const long long rows = (long long)p.B * p.Hq * p.Sq;
    const unsigned g = (unsigned)((rows + 7) / 8);
    const bool vec_ok = p.dtype == OSF_BF16 && (p.D == 64 || p.D == 128) &&
                        ((reinterpret_cast<uintptr_t>(p.o) | reinterpret_cast<uintptr_t>(p.dout)) & 7u) == 0;
    const bool v16_ok = vec_ok && ((reinterpret_cast<uintptr_t>(p.o) | reinterpret_cast<uintptr_t>(p.dout)) & 15u) == 0;
    if (v16_ok) {
        // 8 warps x (4 rounds of 32 / LPR rows) per CTA
        if (p.D == 128) bwd_rowdot_v16_kernel<16><<<(unsigned)((rows + 63) / 64), 256, 0, s>>>(p);
        else bwd_rowdot_v16_kernel<8><<<(unsigned)((rows + 127) / 128), 256, 0, s>>>(p);
    } else if (vec_ok) {
        const unsigned g4 = (unsigned)((rows + 31) / 32);   // 8 warps x 4 rows per CTA
        if (p.D == 128) bwd_rowdot_vec_kernel<4><<<g4, 256, 0, s>>>(p);
        else bwd_rowdot_vec_kernel<2><<<g4, 256, 0, s>>>(p);
    } else if (p.dtype == OSF_BF16) {
        bwd_rowdot_kernel<__nv_bfloat16><<<g, 256, 0, s>>>(p);
    } else {
        bwd_rowdot_kernel<float><<<g, 256, 0, s>>>(p);
    }
    count_launches(1);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if (attn_bwd_tc_supported(p)) return launch_attn_bwd_tc(p, s);
    if (p.window) return p.dtype == OSF_BF16 ? launch_window_rows<__nv_bfloat16>(p, s) : launch_window_rows<float>(p, s);
    if (attn_bwd_mma_supported(p)) return p.D == 64 ? launch_mma<64>(p, s) : launch_mma<128>(p, s);
    return p.dtype == OSF_BF16 ? launch_simt<__nv_bfloat16>(p, s) : launch_simt<float>(p, s);
}

}  // namespace osf
