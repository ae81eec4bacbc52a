// Eviction from a K/V cache: of the n valid keys of each (batch, kv head), keep the first `sinks`, the
// last `recent` and, of those between, the `budget - sinks - recent` with the largest accumulated
// weight (ties: the lowest index), in their old order, and move their rows together.
//
// Choice: the k-th largest of up to a few hundred thousand floats, by radix selection.  Floats map to
// unsigned integers of the same order (NaN below everything, -0 equal to 0); three passes over the
// key's bits, 11 + 11 + 10 from the top, each count the keys of every digit among those that match the
// digits chosen so far, and take the digit in which the k-th largest lies.  A fourth pass writes the
// indices of the keys above the threshold and the lowest-indexed of the equal ones.  Counts are
// integers, so the result does not depend on the order of the atomics.
// One (batch, kv head) is a cluster of up to 8 CTAs, each holding a slice of the keys; the digit
// counts are summed, and the output offsets of the slices found, through distributed shared memory.
//
// Move: rows are copied through registers in 16-byte pieces where their size and address allow.  Into
// another buffer, every piece is independent.  In place, row r is overwritten by row idx[r] >= r, so
// one CTA walks a slice of the columns of one (batch, kv head) in blocks of ascending rows: it reads a
// whole block before it writes it, and a later block's sources are never behind its own first row.
#include "kv_evict.cuh"
#include "sm100_ptx.cuh"

namespace osf {
namespace {

using namespace ptx;

constexpr int kSelThreads = 512;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr int kSelItems = 4;                             // keys per thread and block step
constexpr int kSliceStep = kSelThreads * kSelItems;

__device__ __forceinline__ int valid_length(const EvictProblem &p, int b) {
    if (!p.lens) return p.S;
    const int n = p.lens[b];
    return min(max(n, 0), p.S);
}

// Order-preserving integer of a weight: NaN is 0, -0 equals +0.
__device__ __forceinline__ uint32_t order_key(float w) {
    if (w != w) return 0u;
    const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);
    return (u >> 31) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// Exclusive prefix sum over the block, and the block's total (two barriers).
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t *warp_sums, uint32_t &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    uint32_t before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < kSelThreads / 32; ++i) {
        const uint32_t s = warp_sums[i];
        before += i < warp ? s : 0u;
        all += s;
    }
    __syncthreads();
    total = all;
    return before + x - v;
}

__global__ void __launch_bounds__(kSelThreads)
kv_select_kernel(const EvictProblem p, int cluster) {
    __shared__ uint32_t hist[kBins];
    __shared__ uint32_t warp_sums[kSelThreads / 32];
    __shared__ uint32_t sh_bin, sh_above, sh_count;
    __shared__ uint32_t slice_counts[2];   // keys above the threshold, keys equal to it, in this slice
    const int tid = threadIdx.x;
    const int row = blockIdx.x / cluster, rank = blockIdx.x % cluster;
    const int b = row / p.Hkv;
    const int n = valid_length(p, b);
    int *idx = p.idx + (long long)row * p.budget;
    if (rank == 0 && tid == 0 && p.lens && (p.lens[b] < 0 || p.lens[b] > p.S)) atomicExch(p.status, (int)OSF_ERR_INVALID);
    if (n <= p.budget) {   // everything stays (uniform over the cluster)
        for (int i = rank * kSelThreads + tid; i < p.budget; i += cluster * kSelThreads) idx[i] = i < n ? i : -1;
        return;
    }
    const float *w = p.w + (long long)row * p.S;
    const int lo = p.sinks, hi = n - p.recent;           // candidates: n > budget >= sinks + recent
    const int k = p.budget - p.sinks - p.recent;         // of which k are kept, k < hi - lo
    for (int i = rank * kSelThreads + tid; i < p.sinks; i += cluster * kSelThreads) idx[i] = i;
    for (int i = rank * kSelThreads + tid; i < p.recent; i += cluster * kSelThreads) idx[p.budget - p.recent + i] = hi + i;
    if (k == 0) return;
    // this CTA's slice of the candidates
    const int per = (hi - lo + cluster - 1) / cluster;
    const int s0 = lo + rank * per, s1 = min(hi, s0 + per);

    uint32_t prefix = 0, mask = 0, left = (uint32_t)k;   // left: still to take among keys matching prefix
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const uint32_t digits = pass == 2 ? 1024u : 2048u;
        for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
        __syncthreads();
        for (int i = s0 + tid; i < s1; i += kSelThreads) {
            const uint32_t key = order_key(w[i]);
            if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & (digits - 1)], 1u);
        }
        if (cluster > 1) cluster_sync();
        else __syncthreads();
        // thread t owns digits 4t' .. 4t'+3 counted from the top, so a prefix sum gives the keys above
        uint32_t c[4], sum = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t bin = kBins - 1 - (4 * tid + e);
            c[e] = 0;
            if (cluster > 1) {
                for (int r = 0; r < cluster; ++r) c[e] += ld_cluster_u32(mapa_shared(smem_u32(&hist[bin]), r));
            } else {
                c[e] = hist[bin];
            }
            sum += c[e];
        }
        uint32_t total;
        uint32_t above = block_scan(sum, warp_sums, total);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (above < left && left <= above + c[e]) {
                sh_bin = kBins - 1 - (4 * tid + e);
                sh_above = above;
                sh_count = c[e];
            }
            above += c[e];
        }
        if (cluster > 1) cluster_sync();   // also: every CTA has read this one's counts
        else __syncthreads();
        prefix |= sh_bin << shift;
        mask |= (digits - 1) << shift;
        left -= sh_above;
        if (left == sh_count) break;   // every key with this prefix is taken (uniform over the cluster)
    }
    // kept: (key & mask) > prefix, and the first `left` of those equal to it
    uint32_t gt = 0, eq = 0;
    for (int i = s0 + tid; i < s1; i += kSelThreads) {
        const uint32_t key = order_key(w[i]) & mask;
        gt += key > prefix;
        eq += key == prefix;
    }
    uint32_t gt_all, eq_all;
    block_scan(gt, warp_sums, gt_all);
    block_scan(eq, warp_sums, eq_all);
    uint32_t out = (uint32_t)p.sinks, eq_before = 0;
    if (cluster > 1) {
        if (tid == 0) {
            slice_counts[0] = gt_all;
            slice_counts[1] = eq_all;
        }
        cluster_sync();
        for (int r = 0; r < rank; ++r) {
            const uint32_t g = ld_cluster_u32(mapa_shared(smem_u32(&slice_counts[0]), r));
            const uint32_t q = ld_cluster_u32(mapa_shared(smem_u32(&slice_counts[1]), r));
            out += g + min(q, left - min(left, eq_before));
            eq_before += q;
        }
        cluster_sync();   // nobody leaves while its shared memory may still be read
    }
    for (int i0 = s0; i0 < s1; i0 += kSliceStep) {
        uint32_t flag[kSelItems];   // 1: above, 0x10000: equal
        uint32_t sum = 0;
#pragma unroll
        for (int e = 0; e < kSelItems; ++e) {
            const int i = i0 + tid * kSelItems + e;
            const uint32_t key = i < s1 ? (order_key(w[i]) & mask) : 0u;
            flag[e] = i >= s1 ? 0u : key > prefix ? 1u : key == prefix ? 0x10000u : 0u;
            sum += flag[e];
        }
        uint32_t total;
        uint32_t before = block_scan(sum, warp_sums, total);
#pragma unroll
        for (int e = 0; e < kSelItems; ++e) {
            const uint32_t g = before & 0xffffu, q = eq_before + (before >> 16);
            if (flag[e] == 1u || (flag[e] == 0x10000u && q < left)) {
                // equal keys before this one that were taken: those of the whole row, less those of earlier steps
                const uint32_t taken = min(q, left) - min(eq_before, left);
                idx[out + g + taken] = i0 + tid * kSelItems + e;
            }
            before += flag[e];
        }
        const uint32_t q_after = eq_before + (total >> 16);
        out += (total & 0xffffu) + min(q_after, left) - min(eq_before, left);
        eq_before = q_after;
    }
}

template <typename U>
__device__ __forceinline__ U ld_stream(const U *p) { return __ldcs(p); }

// Rows to another buffer: piece u of the row block is unit u % upr of kept row u / upr.
template <typename U>
__global__ void __launch_bounds__(256)
kv_move_kernel(const EvictProblem p, int t, int upr) {
    griddep_wait();
    const int row = blockIdx.y, b = row / p.Hkv;
    const int keep = min(valid_length(p, b), p.budget);
    const int *idx = p.idx + (long long)row * p.budget;
    const U *src = reinterpret_cast<const U *>(p.src[t] + (long long)row * p.S * p.row_bytes[t]);
    U *dst = reinterpret_cast<U *>(p.dst[t] + (long long)row * p.S_out * p.row_bytes[t]);
    constexpr int IL = 4;   // independent pieces per thread
    const long long total = (long long)keep * upr;
    for (long long u0 = (long long)blockIdx.x * (256 * IL) + threadIdx.x; u0 < total; u0 += (long long)gridDim.x * (256 * IL)) {
        U v[IL];
#pragma unroll
        for (int e = 0; e < IL; ++e) {
            const long long u = u0 + e * 256;
            if (u < total) {
                const int r = (int)(u / upr), c = (int)(u - (long long)r * upr);
                v[e] = ld_stream(src + (long long)idx[r] * upr + c);
            }
        }
#pragma unroll
        for (int e = 0; e < IL; ++e) {
            const long long u = u0 + e * 256;
            if (u < total) dst[u] = v[e];
        }
    }
}

// Rows within one buffer (see the top): `cols` neighbouring pieces of every row per CTA.
template <typename U>
__global__ void __launch_bounds__(256)
kv_move_in_place_kernel(const EvictProblem p, int t, int upr, int cols) {
    griddep_wait();
    const int row = blockIdx.y, b = row / p.Hkv;
    const int keep = min(valid_length(p, b), p.budget);
    const int *idx = p.idx + (long long)row * p.budget;
    U *buf = reinterpret_cast<U *>(p.dst[t] + (long long)row * p.S * p.row_bytes[t]);
    const int c = blockIdx.x * cols + threadIdx.x % cols;
    const int rows_per = 256 / cols, r_in = threadIdx.x / cols;
    const bool on = r_in < rows_per && c < upr;
    constexpr int IL = 4;
    for (int r0 = 0; r0 < keep; r0 += rows_per * IL) {
        U v[IL];
        int from[IL];
#pragma unroll
        for (int e = 0; e < IL; ++e) {
            const int r = r0 + e * rows_per + r_in;
            from[e] = on && r < keep ? idx[r] : -1;
            if (from[e] > r) v[e] = buf[(long long)from[e] * upr + c];
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < IL; ++e) {
            const int r = r0 + e * rows_per + r_in;
            if (from[e] > r) buf[(long long)r * upr + c] = v[e];
        }
        __syncthreads();
    }
}

// Weights of the kept rows, zeros behind them, and the new length.  In place like the rows.
__global__ void __launch_bounds__(1024)
kv_move_weights_kernel(const EvictProblem p) {
    griddep_wait();
    const int row = blockIdx.x, b = row / p.Hkv;
    const int keep = min(valid_length(p, b), p.budget);
    const int *idx = p.idx + (long long)row * p.budget;
    const float *src = p.w + (long long)row * p.S;
    float *dst = p.w_out + (long long)row * p.S_out;
    constexpr int IL = 4;
    for (int r0 = 0; r0 < keep; r0 += 1024 * IL) {
        float v[IL];
#pragma unroll
        for (int e = 0; e < IL; ++e) {
            const int r = r0 + e * 1024 + threadIdx.x;
            if (r < keep) v[e] = src[idx[r]];
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < IL; ++e) {
            const int r = r0 + e * 1024 + threadIdx.x;
            if (r < keep) dst[r] = v[e];
        }
        __syncthreads();
    }
    for (int r = keep + threadIdx.x; r < p.S_out; r += 1024) dst[r] = 0.f;
    // a length that is written over the old one gives the same `keep` to a block that reads it late
    if (p.lens_out && row % p.Hkv == 0 && threadIdx.x == 0) p.lens_out[b] = keep;
}

template <typename U>
cudaError_t launch_move_t(const EvictProblem &p, int t, int sm_count, cudaStream_t s) {
    const int rows = p.B * p.Hkv;
    const long long upr = p.row_bytes[t] / (long long)sizeof(U);
    if (p.src[t] == p.dst[t]) {
        // 64 bytes of every row per CTA: two whole sectors
        const int cols = (int)(upr < 64 / (int)sizeof(U) ? upr : 64 / (int)sizeof(U));
        return launch_dependent(kv_move_in_place_kernel<U>, dim3((unsigned)((upr + cols - 1) / cols), rows), dim3(256), 0, s,
                                p, t, (int)upr, cols);
    }
    const long long work = ((long long)p.budget * upr + 1023) / 1024;
    long long blocks = ((long long)sm_count * 16 + rows - 1) / rows;
    blocks = blocks < work ? blocks : work;
    return launch_dependent(kv_move_kernel<U>, dim3((unsigned)(blocks < 1 ? 1 : blocks), rows), dim3(256), 0, s, p, t, (int)upr);
}

cudaError_t launch_move(const EvictProblem &p, int t, int sm_count, cudaStream_t s) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p.src[t]) | reinterpret_cast<uintptr_t>(p.dst[t]) | (uintptr_t)p.row_bytes[t];
    if ((a & 15) == 0) return launch_move_t<uint4>(p, t, sm_count, s);
    if ((a & 3) == 0) return launch_move_t<uint32_t>(p, t, sm_count, s);
    return launch_move_t<unsigned char>(p, t, sm_count, s);
}

}  // namespace

cudaError_t launch_kv_evict(const EvictProblem &p, int sm_count, cudaStream_t s) {
    const int rows = p.B * p.Hkv;
    // a CTA takes up to 8192 keys before the row is spread over more of them
    int cluster = 1;
    while (cluster < kMaxCluster && (long long)cluster * 8192 < p.S) cluster *= 2;
    cudaError_t e = launch_clustered(kv_select_kernel, dim3((unsigned)rows * cluster), dim3(kSelThreads), 0, s,
                                     dim3(cluster, 1, 1), false, p, cluster);
    if (e != cudaSuccess) return e;
    int launches = 2;
    for (int t = 0; t < 2 && e == cudaSuccess; ++t)
        if (p.src[t]) {
            e = launch_move(p, t, sm_count, s);
            ++launches;
        }
    if (e == cudaSuccess) e = launch_dependent(kv_move_weights_kernel, dim3((unsigned)rows), dim3(1024), 0, s, p);
    count_launches(launches);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace osf
