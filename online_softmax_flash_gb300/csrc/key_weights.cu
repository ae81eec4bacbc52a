// Attention weight that every key has received:
//     w[b, g, j] (+)= sum over the G query heads of kv head g and the rows i that see key j of
//                     exp(scale * q_i . k_j - lse_i)
// the column sums of the softmax matrix that the forward pass never writes.  With the forward's
// log-sum-exp known, every term stands alone: no running maximum, and the sums of any parts of the rows
// simply add.  Terms are computed in base 2, 2^(s * scale * log2 e - lse * log2 e), sums kept in float32.
//
// This file: the CUDA-core kernel for every type, head dimension and stride, and the sum over row
// splits.  A CTA holds 64 keys of one kv head in shared memory and walks the kv head's G * Sq query rows in
// tiles of 64 (of 16 where there are no more: a decode step); a thread computes 4 (1) rows x 4 keys.  The next 32
// channels of the rows are in flight while these are multiplied.  Rows that see none of the keys are left out, and
// the others cut into parts of `tiles_per_part` tiles, so that the key blocks of a causal problem, whose row counts
// differ, give even parts.
// Bound by instruction issue (two 16-byte shared loads to 16 FMAs) and the latency of a part's first loads: B=1 Hq=8
// Hkv=2 S=1001 D=64 float32, causal, 0.51 GFLOP, 25 us with the sum of the parts.  Packed pairs of FMAs, with the
// rows' values doubled in shared memory, are bound by that memory's bandwidth: the kernel alone 32 us against 26 us.
#include "key_weights.cuh"

namespace osf {
namespace {

constexpr int TK = 64, TC = 32;     // keys of a CTA; channels of the rows in shared memory at a time
constexpr int KPAD = TK + 4;         // channel-major tiles: the pad spreads the transposing writes over the banks

// Rows of a head that see any of the keys from key0 on: the last `visible_rows` of Sq.
__host__ __device__ __forceinline__ int visible_rows(const KeyWeightsProblem &p, int key0) {
    if (!p.causal) return p.Sq;
    const long long first = (long long)key0 - p.causal_off;
    return first <= 0 ? p.Sq : first >= p.Sq ? 0 : p.Sq - (int)first;
}
// Parts that the rows of the key block from key0 on are cut into (one, possibly empty, at least).
__host__ __device__ __forceinline__ int parts_of(const KeyWeightsProblem &p, int key0, int tile_rows) {
    const long long tiles = ((long long)(p.Hq / p.Hkv) * visible_rows(p, key0) + tile_rows - 1) / tile_rows;
    const long long parts = (tiles + p.tiles_per_part - 1) / p.tiles_per_part;
    return parts < 1 ? 1 : (int)parts;
}

// Eight channels c0 .. c0+7 of a row of D; those past the end are 0.
__device__ __forceinline__ void row8(const float *p, int c0, int D, bool vec, float (&x)[8]) {
    if (vec && c0 + 8 <= D) {
        const float4 a = *reinterpret_cast<const float4 *>(p + c0), b = *reinterpret_cast<const float4 *>(p + c0 + 4);
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = c0 + e < D ? p[c0 + e] : 0.f;
    }
}
__device__ __forceinline__ void row8(const __nv_bfloat16 *p, int c0, int D, bool vec, float (&x)[8]) {
    if (vec && c0 + 8 <= D) {
        const uint4 a = *reinterpret_cast<const uint4 *>(p + c0);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[2 * e] = __uint_as_float(w[e] << 16);
            x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = c0 + e < D ? __bfloat162float(p[c0 + e]) : 0.f;
    }
}

// TR: rows of a tile, 64 or 16.
template <typename T, int TR>
__global__ void __launch_bounds__(256, TR == 64 ? 4 : 5)
key_weights_simt_kernel(const KeyWeightsProblem p, int q_vec, int k_vec) {
    constexpr int RPT = TR / 16, QPAD = TR + 4;
    extern __shared__ __align__(16) float sk[];        // [D rounded up to 32][KPAD]
    __shared__ __align__(16) float sq[TC][QPAD];
    __shared__ float off[TR];
    __shared__ int lim[TR];       // keys below this are visible to the row
    __shared__ float red[16][TK];
    griddep_launch();
    const int tid = threadIdx.x, tk = tid & 15, tr = tid >> 4;
    const int kvbh = blockIdx.y, b = kvbh / p.Hkv, kvh = kvbh % p.Hkv;
    const int key0 = blockIdx.x * TK;
    if ((int)blockIdx.z >= parts_of(p, key0, TR)) return;
    const int G = p.Hq / p.Hkv;
    // rows of a head that see these keys, and its first one; tiles run over the G heads' visible rows
    const int V = visible_rows(p, key0), v0 = p.Sq - V;
    const long long tiles = ((long long)G * V + TR - 1) / TR, t0 = (long long)blockIdx.z * p.tiles_per_part;
    const long long t1 = min(tiles, t0 + p.tiles_per_part);
    const T *K = static_cast<const T *>(p.k) + b * p.k_sb + kvh * p.k_sh;
    const T *Q = static_cast<const T *>(p.q) + b * p.q_sb + (long long)kvh * G * p.q_sh;
    const int chunks = (p.D + TC - 1) / TC;
    // loads: four threads share a row, eight channels each
    const int lr = tid >> 2, lc = (tid & 3) * 8;
    for (int c = 0; c < chunks; ++c) {
        float x[8];
        row8(K + min(key0 + lr, p.Sk - 1) * p.k_ss, c * TC + lc, p.D, k_vec, x);   // keys past the end are not stored
#pragma unroll
        for (int e = 0; e < 8; ++e) sk[(c * TC + lc + e) * KPAD + lr] = x[e];
    }
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    // head (of the group) and visible row of the tile's first row; rows of a tile follow with 32-bit divisions
    const unsigned Vu = V > 0 ? (unsigned)V : 1u;
    int h0 = (int)(t0 * TR / Vu);
    unsigned i0 = (unsigned)(t0 * TR - (long long)h0 * Vu);
    for (long long t = t0; t < t1; ++t, h0 += (int)((i0 + TR) / Vu), i0 = (i0 + TR) % Vu) {
        __syncthreads();   // the last tile's off and lim have been read
        if (tid < TR) {    // offset and limit of a row
            const unsigned x = i0 + tid;
            const int h = h0 + (int)(x / Vu), i = v0 + (int)(x % Vu);
            off[tid] = h < G ? row_offset(p.lse[((long long)b * p.Hq + kvh * G + h) * p.Sq + i]) : -INFINITY;
            lim[tid] = off[tid] == -INFINITY ? 0 : p.causal ? (int)min((long long)p.Sk, (long long)i + p.causal_off + 1) : p.Sk;
        }
        const bool loads = lr < TR;
        const unsigned y = i0 + lr;
        int qh = h0 + (int)(y / Vu), qi = v0 + (int)(y % Vu);
        if (qh >= G) {   // rows past the end repeat the last: their limit of 0 takes them out
            qh = G - 1;
            qi = p.Sq - 1;
        }
        const T *row = Q + qh * p.q_sh + qi * p.q_ss;
        float acc[RPT][4] = {}, x[8];
        if (loads) row8(row, lc, p.D, q_vec, x);
        for (int c = 0; c < chunks; ++c) {
            if (loads) {
#pragma unroll
                for (int e = 0; e < 8; ++e) sq[lc + e][lr] = x[e];
            }
            __syncthreads();
            if (loads && c + 1 < chunks) row8(row, (c + 1) * TC + lc, p.D, q_vec, x);
            const float *kc = sk + c * TC * KPAD + 4 * tk;
#pragma unroll
            for (int d = 0; d < TC; ++d) {
                const float4 k = *reinterpret_cast<const float4 *>(kc + d * KPAD);
                float a[RPT];
                if (RPT == 4) {
                    const float4 v = *reinterpret_cast<const float4 *>(&sq[d][4 * tr]);
                    a[0] = v.x; a[RPT > 1 ? 1 : 0] = v.y; a[RPT > 2 ? 2 : 0] = v.z; a[RPT > 3 ? 3 : 0] = v.w;
                } else {
                    a[0] = sq[d][tr];
                }
#pragma unroll
                for (int i = 0; i < RPT; ++i) {
                    acc[i][0] = fmaf(a[i], k.x, acc[i][0]);
                    acc[i][1] = fmaf(a[i], k.y, acc[i][1]);
                    acc[i][2] = fmaf(a[i], k.z, acc[i][2]);
                    acc[i][3] = fmaf(a[i], k.w, acc[i][3]);
                }
            }
            __syncthreads();
        }
        // a tile's terms are added among themselves first: the long sum then has one rounding per tile
        float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const float o = off[RPT * tr + i];
            const int l = lim[RPT * tr + i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float e = ex2_approx(fmaf(acc[i][j], p.scale_log2, o));
                part[j] += key0 + 4 * tk + j < l ? e : 0.f;
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[j] += part[j];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) red[tr][4 * tk + j] = sum[j];
    __syncthreads();
    if (tid < TK && key0 + tid < p.Sk) {
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) v += red[i][tid];
        const long long at = (long long)kvbh * p.Sk + key0 + tid;
        if (p.splits > 1) p.part[(long long)blockIdx.z * p.B * p.Hkv * p.Sk + at] = v;
        else p.w[at] = p.accumulate ? p.w[at] + v : v;
    }
}

// The parts of every key: eight threads of a block share a key, each takes every eighth part, and their sums are
// added in order.  (A thread per key: 14 us under ncu for the 63 parts of the problem above, its loads one after another.)
constexpr int RK = 32, RT = 8;   // keys of a block, threads of a key
__global__ void __launch_bounds__(RK * RT) key_weights_reduce_kernel(const KeyWeightsProblem p, int tile_rows) {
    __shared__ float sums[RT][RK];
    const long long n = (long long)p.B * p.Hkv * p.Sk;
    const int k = threadIdx.x % RK, t = threadIdx.x / RK;
    const long long i = (long long)blockIdx.x * RK + k;
    const int parts = i < n ? parts_of(p, (int)(i % p.Sk) / TK * TK, tile_rows) : 0;
    griddep_wait();
    float v = 0.f;
#pragma unroll 8
    for (int s = t; s < parts; s += RT) v += p.part[s * n + i];
    sums[t][k] = v;
    __syncthreads();
    if (t != 0 || i >= n) return;
#pragma unroll
    for (int e = 1; e < RT; ++e) v += sums[e][k];
    p.w[i] = p.accumulate ? p.w[i] + v : v;
}

}  // namespace

static int tile_rows(const KeyWeightsProblem &p) { return (long long)(p.Hq / p.Hkv) * p.Sq <= 16 ? 16 : 64; }

void key_weights_simt_plan(KeyWeightsProblem &p, int sm_count) {
    // at most four CTAs to an SM over all key blocks, one wave, of equal numbers of tiles (the problem above: 27 us, now
    // 25; a little more than a wave then 29 us, three to an SM 33 us); at most 64 parts of a block
    const int tr = tile_rows(p);
    const long long blocks = (p.Sk + TK - 1) / TK;
    auto tiles = [&](long long kb) {
        return ((long long)(p.Hq / p.Hkv) * visible_rows(p, (int)(kb * TK)) + tr - 1) / tr;
    };
    // the first blocks are seen by every row, then each by 64 rows of a head fewer
    long long all_see = !p.causal ? blocks : p.causal_off < 0 ? 0 : (long long)p.causal_off / TK + 1;
    all_see = all_see < blocks ? all_see : blocks;
    const long long most = tiles(0);
    long long all = all_see * most;
    for (long long kb = all_see; kb < blocks; ++kb) {
        const long long t = tiles(kb);
        if (t == 0) break;
        all += t;
    }
    all *= (long long)p.B * p.Hkv;
    long long per = (all + 4LL * sm_count - 1) / (4LL * sm_count);
    const long long least = (most + 63) / 64;
    per = per < least ? least : per;
    p.tiles_per_part = per < 1 ? 1 : per;
    p.splits = (int)((most + p.tiles_per_part - 1) / p.tiles_per_part);
    if (p.splits < 1) p.splits = 1;
}

template <typename T, int TR>
static cudaError_t launch_simt_t(const KeyWeightsProblem &p, cudaStream_t s) {
    const int smem = (p.D + TC - 1) / TC * TC * KPAD * (int)sizeof(float);
    const cudaError_t e = set_max_dynamic_smem((const void *)key_weights_simt_kernel<T, TR>, smem);
    if (e != cudaSuccess) return e;
    // eight channels at once where rows keep 16-byte alignment
    const int unit = 16 / (int)sizeof(T);
    const int q_vec = (reinterpret_cast<uintptr_t>(p.q) & 15u) == 0 && ((p.q_sb | p.q_sh | p.q_ss) % unit) == 0;
    const int k_vec = (reinterpret_cast<uintptr_t>(p.k) & 15u) == 0 && ((p.k_sb | p.k_sh | p.k_ss) % unit) == 0;
    const dim3 grid((unsigned)((p.Sk + TK - 1) / TK), (unsigned)(p.B * p.Hkv), (unsigned)p.splits);
    key_weights_simt_kernel<T, TR><<<grid, 256, smem, s>>>(p, q_vec, k_vec);
    count_launches(1);
    return cudaGetLastError();
}

cudaError_t launch_key_weights_simt(const KeyWeightsProblem &p, cudaStream_t s) {
    const bool few = tile_rows(p) == 16;
    if (p.dtype == OSF_F32) return few ? launch_simt_t<float, 16>(p, s) : launch_simt_t<float, 64>(p, s);
    return few ? launch_simt_t<__nv_bfloat16, 16>(p, s) : launch_simt_t<__nv_bfloat16, 64>(p, s);
}

cudaError_t launch_key_weights_reduce(const KeyWeightsProblem &p, cudaStream_t s) {
    const long long n = (long long)p.B * p.Hkv * p.Sk;
    count_launches(1);
    return launch_dependent(key_weights_reduce_kernel, dim3((unsigned)((n + RK - 1) / RK)), dim3(RK * RT), 0, s, p, tile_rows(p));
}

}  // namespace osf
