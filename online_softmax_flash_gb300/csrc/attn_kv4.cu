// Attention over the 4-bit K/V cache (record format: kv4.cuh): a few query rows per sequence against
// a long cache, the decode step.  Like the bf16 decode kernel, one CTA takes the query rows of one
// (batch, kv head) against one part of its keys, so a record leaves HBM once; every part yields a partial
// online-softmax state (m, l, acc), and the log-sum-exp combine merges them.  The parts are cut from each
// sequence's own length, on the device, so a ragged batch splits every sequence evenly.
//
// This kernel is the general one: any D that is a multiple of 32, float32 or bfloat16 queries.  A warp takes 32 keys
// at a time: first a key per lane (its whole dot product with up to 4 query rows held in shared memory),
// then a channel of each group per lane (the weights come from the other lanes by shuffle).
#include "kv4.cuh"

namespace osf {
namespace {

constexpr int GW = 4;        // warps per CTA
constexpr int RB = 4;        // query rows per CTA
constexpr int MAXG = 8;      // groups of 32 channels: D <= 256
constexpr int WS_D = 256;

__device__ __forceinline__ float lo_bf16(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// Keys [begin, end) that part `split` of `splits` has of a sequence of n keys, in steps of `unit`.
__device__ __forceinline__ void part_of(int n, int unit, int split, int splits, int &begin, int &end) {
    const long long units = ((long long)n + unit - 1) / unit;
    begin = (int)(units * split / splits) * unit;
    end = min(n, (int)(units * (split + 1) / splits) * unit);
}

template <typename T>
__global__ void __launch_bounds__(GW * 32)
attn_kv4_kernel(const Kv4AttnProblem kp) {
    const AttnProblem &p = kp.a;
    __shared__ float sq[RB][WS_D];
    __shared__ float sacc[GW][RB][WS_D];
    __shared__ float sm[GW][RB], sl[GW][RB];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = p.Hq / p.Hkv, R = G * p.Sq;
    const int kvbh = blockIdx.x, b = kvbh / p.Hkv, kvh = kvbh % p.Hkv;
    const int r0 = blockIdx.z * RB, rows = min(RB, R - r0);
    const int n = kv4_length(kp.lens, b, p.Sk, p.status);
    const int NG = p.D / kKv4Group, rec = kv4_record_bytes(p.D);
    for (int i = tid; i < RB * p.D; i += GW * 32) {
        const int r = i / p.D, c = i % p.D;
        float x = 0.f;
        if (r < rows) {
            const int gr = r0 + r;
            x = to_f32(static_cast<const T *>(p.q)[q_at(p, b, kvh * G + gr / p.Sq, gr % p.Sq) + c]);
        }
        sq[r][c] = x;
    }
    __syncthreads();
    int lim[RB];
#pragma unroll
    for (int r = 0; r < RB; ++r) {
        const int i = (r0 + min(r, rows - 1)) % p.Sq;
        lim[r] = r >= rows ? 0 : p.causal ? min(n, max(0, n - p.Sq + i + 1)) : n;
    }
    int begin, end;
    part_of(n, 32, blockIdx.y, p.splits, begin, end);
    const unsigned char *head = kp.cache + (long long)kvbh * p.Sk * rec;
    float m[RB], l[RB], acc[RB][MAXG];
#pragma unroll
    for (int r = 0; r < RB; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.f;
#pragma unroll
        for (int g = 0; g < MAXG; ++g) acc[r][g] = 0.f;
    }
    for (int k0 = begin + warp * 32; k0 < end; k0 += GW * 32) {
        const int key = k0 + lane;
        float s[RB] = {0.f, 0.f, 0.f, 0.f};
        if (key < end) {
            const unsigned char *row = head + (long long)key * rec;
            const uint32_t *codes = reinterpret_cast<const uint32_t *>(row);
            const uint32_t *pairs = reinterpret_cast<const uint32_t *>(row + p.D);
            for (int g = 0; g < NG; ++g) {
                const uint32_t sp = pairs[g];
                const float sc = lo_bf16(sp), mn = hi_bf16(sp);
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const uint32_t w = codes[t * NG + g];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float x = fmaf((float)((w >> (4 * e)) & 15u), sc, mn);
#pragma unroll
                        for (int r = 0; r < RB; ++r) s[r] = fmaf(x, sq[r][g * 32 + t * 8 + e], s[r]);
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
            for (int g = 0; g < MAXG; ++g) acc[r][g] *= a;
        }
        const int cnt = min(32, end - k0);
        for (int kk = 0; kk < cnt; ++kk) {
            float pk[RB];
            float any = 0.f;
#pragma unroll
            for (int r = 0; r < RB; ++r) {
                pk[r] = __shfl_sync(0xffffffffu, pr[r], kk);
                any = fmaxf(any, pk[r]);
            }
            if (any == 0.f) continue;   // no row of this CTA sees the key
            const unsigned char *row = head + (long long)(k0 + kk) * rec;
            const uint32_t *codes = reinterpret_cast<const uint32_t *>(row + p.D / 2);
            const uint32_t *pairs = reinterpret_cast<const uint32_t *>(row + p.D + p.D / 8);
#pragma unroll
            for (int g = 0; g < MAXG; ++g) {
                if (g < NG) {
                    const uint32_t sp = pairs[g], w = codes[(lane >> 3) * NG + g];
                    const float x = fmaf((float)((w >> (4 * (lane & 7))) & 15u), lo_bf16(sp), hi_bf16(sp));
#pragma unroll
                    for (int r = 0; r < RB; ++r)
                        acc[r][g] = pk[r] != 0.f ? fmaf(pk[r], x, acc[r][g]) : acc[r][g];
                }
            }
        }
    }
#pragma unroll
    for (int r = 0; r < RB; ++r) {
        if (lane == 0) {
            sm[warp][r] = m[r];
            sl[warp][r] = l[r];
        }
#pragma unroll
        for (int g = 0; g < MAXG; ++g)
            if (g < NG) sacc[warp][r][g * 32 + lane] = acc[r][g];
    }
    __syncthreads();
    const long long rows_total = (long long)p.B * p.Hq * p.Sq;
    for (int i = tid; i < rows * p.D; i += GW * 32) {
        const int r = i / p.D, c = i % p.D, gr = r0 + r;
        float M = -INFINITY, L = 0.f, A = 0.f;
#pragma unroll
        for (int w = 0; w < GW; ++w) M = fmaxf(M, sm[w][r]);
        const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
        for (int w = 0; w < GW; ++w) {
            const float wt = ex2_approx(sm[w][r] - ref);
            A += wt * sacc[w][r][c];
            L += wt * sl[w][r];
        }
        const int hq = kvh * G + gr / p.Sq, qi = gr % p.Sq;
        const long long grow = ((long long)b * p.Hq + hq) * p.Sq + qi;
        if (p.splits == 1) {
            static_cast<T *>(p.o)[o_at(p, b, hq, qi) + c] = from_f32<T>(L > 0.f || L != L ? A / L : 0.f);
            if (p.lse && c == 0) p.lse[grow] = L > 0.f ? (M + __log2f(L)) * kLn2 : L != L ? L : -INFINITY;
        } else {
            p.part_acc[((size_t)blockIdx.y * rows_total + grow) * p.D + c] = A;
            if (c == 0) {
                p.part_m[(size_t)blockIdx.y * rows_total + grow] = M;
                p.part_l[(size_t)blockIdx.y * rows_total + grow] = L;
            }
        }
    }
}

// Weights from the stored scores, once every row's log-sum-exp is known.
__global__ void __launch_bounds__(256) kv4_weights_kernel(const Kv4AttnProblem kp) {
    griddep_wait();
    const AttnProblem &p = kp.a;
    const int G = p.Hq / p.Hkv, R = G * p.Sq;
    const int kvbh = blockIdx.y, b = kvbh / p.Hkv, kvh = kvbh % p.Hkv;
    const int n = kv4_length(kp.lens, b, p.Sk, p.status);
    const int key = blockIdx.x * 256 + threadIdx.x;
    if (key >= p.Sk) return;
    float *w = kp.weights + (long long)kvbh * p.Sk + key;
    if (key >= n) {
        if (!kp.accumulate) *w = 0.f;
        return;
    }
    const float *lse = p.lse + ((long long)b * p.Hq + kvh * G) * p.Sq;   // the R rows of a kv head are consecutive
    const float *sc = kp.scores + (long long)kvbh * R * p.Sk + key;
    float v = 0.f;
    for (int r = 0; r < R; ++r) {
        const float z = lse[r];
        v += ex2_approx(sc[(long long)r * p.Sk] - (z == -INFINITY ? INFINITY : z * kLog2e));
    }
    *w = kp.accumulate ? *w + v : v;
}

}  // namespace

bool kv4_attn_fast(int, int) { return false; }

int kv4_attn_pick_splits(const Kv4AttnProblem &kp, int sm_count) {
    const AttnProblem &p = kp.a;
    const int R = p.Hq / p.Hkv * p.Sq;
    const long long items = (long long)p.B * p.Hkv * ((R + RB - 1) / RB);
    const long long units = ((long long)p.Sk + 31) / 32;
    long long s = (8LL * sm_count + items - 1) / items;
    const long long most = (units + GW - 1) / GW;   // at least one step of every warp per part
    s = s < most ? s : most;
    return (int)(s < 1 ? 1 : s > 1024 ? 1024 : s);
}

cudaError_t launch_attn_kv4(const Kv4AttnProblem &kp, cudaStream_t s) {
    const AttnProblem &p = kp.a;
    const int R = p.Hq / p.Hkv * p.Sq;
    const dim3 grid((unsigned)(p.B * p.Hkv), (unsigned)p.splits, (unsigned)((R + RB - 1) / RB));
    if (p.dtype == OSF_F32) attn_kv4_kernel<float><<<grid, GW * 32, 0, s>>>(kp);
    else attn_kv4_kernel<__nv_bfloat16><<<grid, GW * 32, 0, s>>>(kp);
    count_launches(1);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess && p.splits > 1) e = launch_attn_combine(p, s);
    if (e == cudaSuccess && kp.weights && p.Sk > 0) {
        count_launches(1);
        e = launch_dependent(kv4_weights_kernel, dim3((unsigned)((p.Sk + 255) / 256), (unsigned)(p.B * p.Hkv)), dim3(256), 0,
                             s, kp);
    }
    return e;
}

}  // namespace osf
