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
// One (batch, kv head) is a cluster of up to 8 CTAs, each holding a slice of the keys, in shared memory while a
// slice has at most 49152 (longer ones are read again in every pass).  (In registers, with every pass unrolled over
// them, the code is too long for one walk through it: a whole call of 16 rows of 131072 keys 59 us against 50 us.)
// The digit counts are summed, and the output offsets of the slices found, through distributed shared memory.
// 64 rows of 32768 keys: 20 us, 16 rows of 131072: 29 us, both bound by the barriers between the passes and the integer
// instructions of the scans (137 per 32 keys over all passes), not by the 8 MB read.
//
// Move: one launch for the cache arrays and the weights.  64 rows of 8192 keys of K and V in bf16, D=128, to another
// buffer: 537 MB in 82 us, 0.96 of the copy's rate.  Rows are copied through registers in 16-byte pieces
// where their size and address allow.  Into another buffer, every piece is independent.  In place, row r is
// overwritten by row idx[r] >= r, so one CTA walks a slice of the columns of one (batch, kv head) in blocks of
// ascending rows: it reads a whole block before it writes it, and a later block's sources are never behind its
// own first row.
#include "kv_evict.cuh"
#include "sm100_ptx.cuh"

namespace osf {
namespace {

using namespace ptx;

constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;

__device__ __forceinline__ int valid_length(const EvictProblem &p, int b) {
    if (!p.lens) return p.S;
    const int n = p.lens[b];
    return min(max(n, 0), p.S);
}

// Order-preserving integer of a weight: NaN is 1, below every number, -0 equals +0; 0 stands for no key.
__device__ __forceinline__ uint32_t order_key(float w) {
    const uint32_t u = __float_as_uint(__fadd_rn(w, 0.f));   // -0 + 0 = +0
    return w != w ? 1u : u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// 8 bytes of shared memory of this CTA or another of the cluster.
__device__ __forceinline__ uint2 ld_cluster_v2(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
    return v;
}

// Exclusive prefix sum over a block of THREADS (two barriers).
template <int THREADS>
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t *warp_sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    constexpr int WARPS = THREADS / 32;
    uint32_t s = lane < WARPS ? warp_sums[lane] : 0u;   // every warp scans the warps' sums
#pragma unroll
    for (int o = 1; o < WARPS; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
    }
    const uint32_t before = warp ? __shfl_sync(0xffffffffu, s, warp - 1) : 0u;
    __syncthreads();
    return before + x - v;
}

// A warp owns a run of neighbouring keys of its CTA's slice, 32 at a time, so that positions within it come from
// ballots.  HELD: the slice's keys stay in shared memory; else they are read again in every pass.  Places behind
// the slice hold 0, below every key: fewer keys are kept than there are, so none of them is ever chosen.
template <bool HELD, int THREADS>
__global__ void __launch_bounds__(THREADS)
kv_select_kernel(const EvictProblem p, int cluster) {
    constexpr int WARPS = THREADS / 32;
    extern __shared__ uint32_t held[];   // [groups][THREADS]
    __shared__ __align__(16) uint32_t hist[kBins];
    __shared__ uint32_t digit_sums[WARPS];
    __shared__ uint32_t warp_above[WARPS], warp_equal[WARPS];
    __shared__ uint32_t sh_bin, sh_above, sh_count;
    __shared__ uint32_t slice_counts[2];   // of this slice: keys above the threshold, keys equal to it
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row = blockIdx.x / cluster, rank = blockIdx.x % cluster;
    const int b = row / p.Hkv;
    const int n = valid_length(p, b);
    int *idx = p.idx + (long long)row * p.budget;
    if (rank == 0 && tid == 0 && p.lens && (p.lens[b] < 0 || p.lens[b] > p.S)) atomicExch(p.status, (int)OSF_ERR_INVALID);
    if (n <= p.budget) {   // everything stays (uniform over the cluster)
        for (int i = rank * THREADS + tid; i < p.budget; i += cluster * THREADS) idx[i] = i < n ? i : -1;
        return;
    }
    const int lo = p.sinks, hi = n - p.recent;           // candidates: n > budget >= sinks + recent
    const int k = p.budget - p.sinks - p.recent;         // of which k are kept, k < hi - lo
    // this CTA's slice of the candidates, this warp's run of it
    const int per = (hi - lo + cluster - 1) / cluster;
    const int s1 = min(hi, lo + (rank + 1) * per);
    const int groups = (per + THREADS - 1) / THREADS;   // of 32 keys
    const int first = lo + rank * per + warp * groups * 32 + lane;
    const float *w = p.w + (long long)row * p.S;
    auto key_of = [&](int i) {   // the load is unconditional, so that several are in flight
        const float v = w[max(0, min(first + i * 32, s1 - 1))];
        return first + i * 32 < s1 ? order_key(v) : 0u;
    };
    if (HELD) {
#pragma unroll 8
        for (int i = 0; i < groups; ++i) held[i * THREADS + tid] = key_of(i);
    }
    for (int i = rank * THREADS + tid; i < p.sinks; i += cluster * THREADS) idx[i] = i;
    for (int i = rank * THREADS + tid; i < p.recent; i += cluster * THREADS) idx[p.budget - p.recent + i] = hi + i;
    if (k == 0) return;
    // apply f to every group's key of this lane, in order
    auto each = [&](auto f) {
#pragma unroll 4
        for (int i = 0; i < groups; ++i) f(i, HELD ? held[i * THREADS + tid] : key_of(i));
    };

    uint32_t prefix = 0, mask = 0, left = (uint32_t)k;   // left: still to take among keys matching prefix
    for (int i = tid; i < kBins; i += THREADS) hist[i] = 0;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const uint32_t digits = pass == 2 ? 1024u : 2048u;
        __syncthreads();
        each([&](int, uint32_t x) {
            if ((x & mask) == prefix && x) atomicAdd(&hist[(x >> shift) & (digits - 1)], 1u);
        });
        if (cluster > 1) cluster_sync();
        else __syncthreads();
        // thread t owns OWN digits, counted from the top, so a prefix sum gives the keys above; the counts of all
        // ranks are read before any is used
        constexpr int OWN = kBins / THREADS;
        const uint32_t mine_at = smem_u32(&hist[kBins - OWN * (tid + 1)]);
        uint2 part[kMaxCluster][OWN / 2];
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r)
#pragma unroll
            for (int e = 0; e < OWN / 2; ++e)
                part[r][e] = r < cluster ? ld_cluster_v2((cluster > 1 ? mapa_shared(mine_at, r) : mine_at) + 8 * e) : make_uint2(0, 0);
        uint32_t c[OWN], sum = 0;
#pragma unroll
        for (int e = 0; e < OWN; ++e) {   // digit kBins - 1 - (OWN tid + e)
            c[e] = 0;
#pragma unroll
            for (int r = 0; r < kMaxCluster; ++r) {
                const uint2 v = part[r][(OWN - 1 - e) / 2];
                c[e] += (OWN - 1 - e) & 1 ? v.y : v.x;
            }
            sum += c[e];
        }
        uint32_t above = block_scan<THREADS>(sum, digit_sums);
#pragma unroll
        for (int e = 0; e < OWN; ++e) {
            if (above < left && left <= above + c[e]) {
                sh_bin = kBins - 1 - (OWN * tid + e);
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
        for (int i = tid; i < kBins; i += THREADS) hist[i] = 0;
    }
    // kept: (key & mask) > prefix, and the first `left` of those equal to it.  Of both, the number before each warp:
    uint32_t above = 0, equal = 0;
    each([&](int, uint32_t x) {
        above += __popc(__ballot_sync(0xffffffffu, (x & mask) > prefix));
        equal += __popc(__ballot_sync(0xffffffffu, (x & mask) == prefix && x));
    });
    if (lane == 0) {
        warp_above[warp] = above;
        warp_equal[warp] = equal;
    }
    __syncthreads();
    uint32_t all_above = 0, all_equal = 0;
    above = equal = 0;
#pragma unroll
    for (int i = 0; i < WARPS; ++i) {
        above += i < warp ? warp_above[i] : 0u;
        equal += i < warp ? warp_equal[i] : 0u;
        all_above += warp_above[i];
        all_equal += warp_equal[i];
    }
    if (cluster > 1) {
        if (tid == 0) {
            slice_counts[0] = all_above;
            slice_counts[1] = all_equal;
        }
        cluster_sync();
        for (int r = 0; r < rank; ++r) {
            const uint32_t at = mapa_shared(smem_u32(slice_counts), r);
            above += ld_cluster_u32(at);
            equal += ld_cluster_u32(at + 4);
        }
        cluster_sync();   // nobody leaves while its shared memory may still be read
    }
    griddep_launch();
    // Positions in index order; of the equal keys the first `left` take one.
    uint32_t out = (uint32_t)p.sinks + above + min(equal, left);
    const uint32_t lower = (1u << lane) - 1u;
    each([&](int i, uint32_t x) {
        const bool gt = (x & mask) > prefix, eq = (x & mask) == prefix && x;
        const uint32_t g = __ballot_sync(0xffffffffu, gt), q = __ballot_sync(0xffffffffu, eq);
        const uint32_t taken = min(equal, left), mine = min(equal + __popc(q & lower), left);
        if (gt || (eq && equal + __popc(q & lower) < left)) idx[out + __popc(g & lower) + mine - taken] = first + i * 32;
        equal += __popc(q);
        out += __popc(g) + min(equal, left) - taken;
    });
}

constexpr int kMoveThreads = 256;
constexpr int IL = 4;   // independent pieces per thread

// One cache array of the call (0 or 1).
struct Array {
    const unsigned char *src;
    unsigned char *dst;
    long long row_bytes;
};

// Rows to another buffer, pieces of type U: piece u of the kept rows is unit u % upr of row u / upr.
template <typename U>
__device__ __forceinline__ void move_out(const EvictProblem &p, const Array &t, int row, int keep) {
    const int *idx = p.idx + (long long)row * p.budget;
    const U *src = reinterpret_cast<const U *>(t.src + (long long)row * p.S * t.row_bytes);
    U *dst = reinterpret_cast<U *>(t.dst + (long long)row * p.S_out * t.row_bytes);
    const unsigned upr = (unsigned)(t.row_bytes / sizeof(U)), total = keep * upr;   // budget * row_bytes < 2^31
    const unsigned step = gridDim.x * (kMoveThreads * IL);
    for (unsigned u0 = blockIdx.x * (kMoveThreads * IL) + threadIdx.x; u0 < total; u0 += step) {
        U v[IL];
#pragma unroll
        for (int e = 0; e < IL; ++e) {
            const unsigned u = u0 + e * kMoveThreads;
            if (u < total) {
                const unsigned r = u / upr;
                v[e] = __ldcs(src + (long long)idx[r] * upr + (u - r * upr));
            }
        }
#pragma unroll
        for (int e = 0; e < IL; ++e)
            if (u0 + e * kMoveThreads < total) __stcs(dst + u0 + e * kMoveThreads, v[e]);
    }
}

// Rows within one buffer (see the top): 64 bytes, two whole sectors, of every row per CTA.
template <typename U>
__device__ __forceinline__ void move_in_place(const EvictProblem &p, const Array &t, int row, int keep) {
    const int *idx = p.idx + (long long)row * p.budget;
    U *buf = reinterpret_cast<U *>(t.dst + (long long)row * p.S * t.row_bytes);
    const int upr = (int)(t.row_bytes / sizeof(U)), cols = min(upr, (int)(64 / sizeof(U)));
    const int c = blockIdx.x * cols + threadIdx.x % cols;
    const int rows_per = kMoveThreads / cols, r_in = threadIdx.x / cols;
    const bool on = r_in < rows_per && c < upr;
    if ((int)blockIdx.x * cols >= upr) return;
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

// Weights of the kept rows, zeros behind them, and the new length.  One CTA per row when in place.
__device__ __forceinline__ void move_weights(const EvictProblem &p, int row, int b, int keep) {
    const int *idx = p.idx + (long long)row * p.budget;
    const float *src = p.w + (long long)row * p.S;
    float *dst = p.w_out + (long long)row * p.S_out;
    // a length that is written over the old one gives the same `keep` to a block that reads it late
    if (blockIdx.x == 0 && p.lens_out && row % p.Hkv == 0 && threadIdx.x == 0) p.lens_out[b] = keep;
    if (p.w != p.w_out) {
        for (unsigned r = blockIdx.x * kMoveThreads + threadIdx.x; r < (unsigned)p.S_out; r += gridDim.x * kMoveThreads)
            dst[r] = r < (unsigned)keep ? src[idx[r]] : 0.f;
        return;
    }
    if (blockIdx.x != 0) return;
    constexpr int WL = 16;
    for (int r0 = 0; r0 < keep; r0 += kMoveThreads * WL) {
        float v[WL];
#pragma unroll
        for (int e = 0; e < WL; ++e) {
            const int r = r0 + e * kMoveThreads + threadIdx.x;
            if (r < keep) v[e] = src[idx[r]];
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < WL; ++e) {
            const int r = r0 + e * kMoveThreads + threadIdx.x;
            if (r < keep) dst[r] = v[e];
        }
        __syncthreads();
    }
    for (int r = keep + threadIdx.x; r < p.S_out; r += kMoveThreads) dst[r] = 0.f;
}

// blockIdx.z: 0 the weights, 1 and 2 the cache arrays.
__global__ void __launch_bounds__(kMoveThreads) kv_move_kernel(const EvictProblem p) {
    griddep_wait();   // the indices
    const int row = blockIdx.y, b = row / p.Hkv;
    const int keep = min(valid_length(p, b), p.budget);
    if (blockIdx.z == 0) {
        move_weights(p, row, b, keep);
        return;
    }
    const Array t = blockIdx.z == 1 ? Array{p.src[0], p.dst[0], p.row_bytes[0]} : Array{p.src[1], p.dst[1], p.row_bytes[1]};
    if (!t.src) return;
    const uintptr_t a = reinterpret_cast<uintptr_t>(t.src) | reinterpret_cast<uintptr_t>(t.dst) | (uintptr_t)t.row_bytes;
    if (t.src == t.dst) {
        if ((a & 15) == 0) move_in_place<uint4>(p, t, row, keep);
        else if ((a & 3) == 0) move_in_place<uint32_t>(p, t, row, keep);
        else move_in_place<unsigned char>(p, t, row, keep);
    } else {
        if ((a & 15) == 0) move_out<uint4>(p, t, row, keep);
        else if ((a & 3) == 0) move_out<uint32_t>(p, t, row, keep);
        else move_out<unsigned char>(p, t, row, keep);
    }
}

}  // namespace

cudaError_t launch_kv_evict(const EvictProblem &p, int sm_count, cudaStream_t s) {
    const int rows = p.B * p.Hkv;
    // CTAs of a row: what its keys need of shared memory, and up to four while the GPU has room for them and each
    // gets 2048 keys.  (16 rows of 131072 keys: 35 us with eight, clusters of which the GPU cannot place all at
    // once, 29 us with four.)  Up to 4096 keys for a CTA, half the threads meet at its barriers: 7.5 us against
    // 8.6 us for 8 rows of 1237.
    constexpr int kHeldKeys = 48 * 1024;
    int cluster = 1;
    while (cluster < kMaxCluster && ((long long)cluster * kHeldKeys < p.S ||
                                     (cluster < 4 && rows * cluster * 2 <= sm_count && cluster * 4096 <= p.S)))
        cluster *= 2;
    const long long per = ((long long)p.S + cluster - 1) / cluster;
    const int threads = per <= 4096 ? 512 : 1024;
    const long long keys = (per + threads - 1) / threads * threads;
    const bool held = keys <= kHeldKeys;
    auto select = threads == 512 ? kv_select_kernel<true, 512> : held ? kv_select_kernel<true, 1024> : kv_select_kernel<false, 1024>;
    const size_t smem = held ? (size_t)keys * sizeof(uint32_t) : 0;
    cudaError_t e = set_max_dynamic_smem((const void *)select, (int)smem);
    if (e != cudaSuccess) return e;
    e = launch_clustered(select, dim3((unsigned)rows * cluster), dim3((unsigned)threads), smem, s, dim3(cluster, 1, 1), false, p,
                         cluster);
    if (e != cudaSuccess) return e;
    // blocks along a row's pieces: all that the work can use, about sixteen to an SM over the grid; in place, a
    // block per 64 bytes of the row
    long long want = ((long long)sm_count * 16 + 2 * rows - 1) / (2 * rows), blocks = 1;
    for (int t = 0; t < 2; ++t) {
        if (!p.src[t]) continue;
        const long long work = p.src[t] == p.dst[t] ? (p.row_bytes[t] + 63) / 64
                                                    : (p.budget * p.row_bytes[t] / 16 + kMoveThreads * IL - 1) / (kMoveThreads * IL);
        const long long need = p.src[t] == p.dst[t] ? work : work < want ? work : want;
        blocks = need > blocks ? need : blocks;
    }
    count_launches(2);
    e = launch_dependent(kv_move_kernel, dim3((unsigned)blocks, (unsigned)rows, p.src[1] ? 3 : p.src[0] ? 2 : 1), dim3(kMoveThreads), 0,
                         s, p);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace osf
