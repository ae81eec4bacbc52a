// Attention weight that every key has received:
//     w[b, g, j] (+)= sum over the G query heads of kv head g and the rows i that see key j of
//                     exp(scale * q_i . k_j - lse_i)
// the column sums of the softmax matrix that the forward pass never writes.  With the forward's
// log-sum-exp known, every term stands alone: no running maximum, and the sums of any parts of the rows
// simply add.  Terms are computed in base 2, 2^(s * scale * log2 e - lse * log2 e), sums kept in float32.
//
// This file: the CUDA-core kernel for every type, head dimension and stride, and the sum over row
// splits.  A CTA owns 64 keys of one kv head and walks the kv head's G * Sq query rows in tiles of 64;
// a thread computes 4 rows x 4 keys, so a pair of shared-memory float4 reads feeds 16 FMAs.  It is
// bound by FMA issue.  Row tiles that see none of the keys are skipped.
#include "key_weights.cuh"

namespace osf {
namespace {

constexpr int TK = 64, TR = 64, TC = 32;   // keys, rows and channels per tile

template <typename T>
__global__ void __launch_bounds__(256)
key_weights_simt_kernel(const KeyWeightsProblem p) {
    // channel-major tiles; the pad keeps the transposing writes off one bank
    __shared__ __align__(16) float sk[TC][TK + 4], sq[TC][TR + 4];
    __shared__ float off[TR];
    __shared__ int lim[TR];       // keys below this are visible to the row
    __shared__ float red[16][TK];
    const int tid = threadIdx.x, tk = tid & 15, tr = tid >> 4;
    const int kvbh = blockIdx.y, b = kvbh / p.Hkv, kvh = kvbh % p.Hkv;
    const int key0 = blockIdx.x * TK;
    const int G = p.Hq / p.Hkv;
    const long long R = (long long)G * p.Sq;
    const long long tiles = (R + TR - 1) / TR;
    const long long t0 = tiles * blockIdx.z / p.splits, t1 = tiles * (blockIdx.z + 1) / p.splits;
    const T *K = static_cast<const T *>(p.k) + b * p.k_sb + kvh * p.k_sh;
    const T *Q = static_cast<const T *>(p.q) + b * p.q_sb;
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    for (long long t = t0; t < t1; ++t) {
        const long long r0 = t * TR;
        int mine = 0;
        if (tid < TR) {
            const long long r = r0 + tid;
            int l = 0;
            float o = -INFINITY;
            if (r < R) {
                const int h = (int)(r / p.Sq), i = (int)(r - (long long)h * p.Sq);
                l = p.causal ? (int)min((long long)p.Sk, max(0LL, (long long)i + p.causal_off + 1)) : p.Sk;
                o = row_offset(p.lse[((long long)b * p.Hq + kvh * G + h) * p.Sq + i]);
            }
            off[tid] = o;
            lim[tid] = l;
            mine = l > key0;
        }
        if (!__syncthreads_or(mine)) continue;
        float acc[4][4] = {};
        for (int c0 = 0; c0 < p.D; c0 += TC) {
            // 32 channels of the 64 keys and rows: a warp reads 32 channels of one row at a time
            for (int e = tid; e < TK * TC; e += 256) {
                const int c = e & (TC - 1), r = e / TC;
                const int key = key0 + r;
                sk[c][r] = (key < p.Sk && c0 + c < p.D) ? to_f32(K[key * p.k_ss + c0 + c]) : 0.f;
                const long long gr = r0 + r;
                float x = 0.f;
                if (gr < R && c0 + c < p.D) {
                    const int h = (int)(gr / p.Sq), i = (int)(gr - (long long)h * p.Sq);
                    x = to_f32(Q[(kvh * G + h) * p.q_sh + i * p.q_ss + c0 + c]);
                }
                sq[c][r] = x;
            }
            __syncthreads();
#pragma unroll 8
            for (int c = 0; c < TC; ++c) {
                const float4 a = *reinterpret_cast<const float4 *>(&sq[c][4 * tr]);
                const float4 k = *reinterpret_cast<const float4 *>(&sk[c][4 * tk]);
                const float av[4] = {a.x, a.y, a.z, a.w}, kv[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(av[i], kv[j], acc[i][j]);
            }
            __syncthreads();
        }
        // a tile's terms are added among themselves first: the long sum then has one rounding per tile
        float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float o = off[4 * tr + i];
            const int l = lim[4 * tr + i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float e = ex2_approx(fmaf(acc[i][j], p.scale_log2, o));
                part[j] += key0 + 4 * tk + j < l ? e : 0.f;
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[j] += part[j];
        __syncthreads();   // off and lim are rewritten by the next tile
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

__global__ void __launch_bounds__(256) key_weights_reduce_kernel(const KeyWeightsProblem p) {
    griddep_wait();
    const long long n = (long long)p.B * p.Hkv * p.Sk;
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    float v = 0.f;
    for (int s = 0; s < p.splits; ++s) v += p.part[s * n + i];
    p.w[i] = p.accumulate ? p.w[i] + v : v;
}

}  // namespace

int key_weights_simt_splits(const KeyWeightsProblem &p, int sm_count) {
    const long long ctas = (long long)((p.Sk + TK - 1) / TK) * p.B * p.Hkv;
    const long long tiles = ((long long)(p.Hq / p.Hkv) * p.Sq + TR - 1) / TR;
    long long s = (3LL * sm_count + ctas - 1) / ctas;
    s = s < tiles ? s : tiles;
    return (int)(s < 1 ? 1 : s > 64 ? 64 : s);
}

cudaError_t launch_key_weights_simt(const KeyWeightsProblem &p, cudaStream_t s) {
    const dim3 grid((unsigned)((p.Sk + TK - 1) / TK), (unsigned)(p.B * p.Hkv), (unsigned)p.splits);
    if (p.dtype == OSF_F32) key_weights_simt_kernel<float><<<grid, 256, 0, s>>>(p);
    else key_weights_simt_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(p);
    count_launches(1);
    return cudaGetLastError();
}

cudaError_t launch_key_weights_reduce(const KeyWeightsProblem &p, cudaStream_t s) {
    const long long n = (long long)p.B * p.Hkv * p.Sk;
    count_launches(1);
    return launch_dependent(key_weights_reduce_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, p);
}

}  // namespace osf
