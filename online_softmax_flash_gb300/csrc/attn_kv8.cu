// Attention over the paged 8-bit K/V cache (format: kv8.cuh): the last Sq tokens of each sequence against it, with or
// without a window and sinks.
//
// General kernel (any D that is a multiple of 32, float32 or bfloat16 queries): a CTA takes up to 4 query rows of one (b, kv
// head) and a part of the keys that they see; a warp copies the rows of 32 keys to shared memory, takes a key per lane
// (its whole dot product with the rows), then a channel of every 32 per lane.
#include "kv8.cuh"
#include "sm100_ptx.cuh"

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
            at = (s * c.P + key % c.P) * D;
        }
        const long long v_off = (long long)c.Hkv * c.P * D;
        const int per = 2 * D / 16;   // 16-byte pieces of a key: K's, then V's
        for (int i0 = 0; i0 < 32 * per; i0 += 32 * 8) {
            uint4 v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int i = i0 + 32 * e + lane, k = i / per % 32, w = i % per;
                const long long from = __shfl_sync(0xffffffffu, at, k);
                const int have = __shfl_sync(0xffffffffu, page, k);
                v[e] = make_uint4(0, 0, 0, 0);
                if (i < 32 * per && have >= 0)
                    v[e] = *reinterpret_cast<const uint4 *>(c.pages + from + (w < per / 2 ? w * 16 : v_off + (w - per / 2) * 16));
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int i = i0 + 32 * e + lane, k = i / per, w = i % per;
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
        const int cnt = min(32, n - k0);
        for (int k = 0; k < cnt; ++k) {
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

size_t kv8_attn_partial_bytes(const Kv8AttnProblem &kp, int sm_count) {
    const AttnProblem &p = kp.a;
    const int splits = general_splits(p, sm_count);
    const size_t rows = (size_t)splits * p.B * p.Hq * p.Sq;
    return splits > 1 ? round256(rows * p.D * sizeof(float)) + 2 * round256(rows * sizeof(float)) : 0;
}

cudaError_t launch_attn_kv8(const Kv8AttnProblem &kp0, void *partials, int sm_count, cudaStream_t s) {
    Kv8AttnProblem kp = kp0;
    AttnProblem &p = kp.a;
    const int R = p.Hq / p.Hkv * p.Sq;
    p.splits = general_splits(p, sm_count);
    p.keep_nan = 1;
    const size_t rows = (size_t)p.splits * p.B * p.Hq * p.Sq;
    char *at = static_cast<char *>(partials);
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
