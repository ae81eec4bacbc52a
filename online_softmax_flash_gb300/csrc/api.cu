// C ABI of libosf (declared in include/osf.h): argument checks, kernel choice, workspace
// sizing and the device status word.  Every entry point validates on the host, then enqueues
// kernels on the caller's stream and returns; nothing here allocates device memory.
#include <limits.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <atomic>
#include <mutex>
#include <map>
#include <utility>

#include "osf_internal.cuh"
#include "softmax_ex.cuh"
#include "attn_bwd.cuh"
#include "selftest.cuh"
#include "attn_tc.cuh"
#include "decode.cuh"
#include "kv4.cuh"
#include "kv8.cuh"
#include "key_weights.cuh"
#include "kv_evict.cuh"

namespace osf {

static std::atomic<unsigned long long> g_launches{0};
void count_launches(int n) { g_launches.fetch_add((unsigned long long)n, std::memory_order_relaxed); }

cudaError_t set_max_dynamic_smem(const void *kernel, int bytes) {
    static std::mutex mu;
    static std::map<std::pair<int, const void *>, int> done;   // (device, kernel) -> limit set
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    const auto key = std::make_pair(dev, kernel);
    auto it = done.find(key);
    if (it != done.end() && it->second >= bytes) return cudaSuccess;   // the limit is only raised
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done[key] = bytes;
    return e;
}

namespace {

constexpr int kMaxDevices = 64;

// One status word per device; kernels with bounded waits write kStatusTimeout here.
__device__ int g_status_word;

struct DeviceInfo {
    int sm_count = 0;
    int *status = nullptr;   // device address of g_status_word
    std::atomic<bool> ready{false};   // set (release) after the fields above
};
DeviceInfo g_dev[kMaxDevices];

int current_device(int *dev) {
    if (cudaGetDevice(dev) != cudaSuccess || *dev < 0 || *dev >= kMaxDevices) return OSF_ERR_CUDA;
    return OSF_OK;
}

// Per-device set-up (SM count, status word address), once per device under a lock; later
// calls see the published fields through the acquire load of `ready`.
int device_info(DeviceInfo **out) {
    static std::mutex mu;
    int dev;
    if (current_device(&dev) != OSF_OK) return OSF_ERR_CUDA;
    DeviceInfo &d = g_dev[dev];
    if (!d.ready.load(std::memory_order_acquire)) {
        std::lock_guard<std::mutex> lock(mu);
        if (!d.ready.load(std::memory_order_relaxed)) {
            int sms = 0;
            if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
                return OSF_ERR_CUDA;
            void *addr = nullptr;
            if (cudaGetSymbolAddress(&addr, g_status_word) != cudaSuccess) return OSF_ERR_CUDA;
            d.sm_count = sms;
            d.status = static_cast<int *>(addr);
            d.ready.store(true, std::memory_order_release);
        }
    }
    *out = &d;
    return OSF_OK;
}

}  // namespace

int device_sm_count(int *sms) {
    DeviceInfo *d;
    const int st = device_info(&d);
    if (st != OSF_OK) return st;
    *sms = d->sm_count;
    return OSF_OK;
}

namespace {

bool overlaps(const void *a, size_t na, const void *b, size_t nb) {
    if (!a || !b || na == 0 || nb == 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a0 < b0 + nb && b0 < a0 + na;
}

size_t elem_size(int dtype) { return dtype == OSF_F32 ? 4 : 2; }

int launch_status(cudaError_t e) { return e == cudaSuccess ? OSF_OK : OSF_ERR_CUDA; }

// Bytes spanned by a strided [n0, n1, n2, D] tensor (strides s0..s2 in elements, d contiguous).
size_t span_bytes(long long n0, long long n1, long long n2, long long D, long long s0, long long s1,
                  long long s2, size_t es) {
    return (size_t)((n0 - 1) * s0 + (n1 - 1) * s1 + (n2 - 1) * s2 + D) * es;
}

// True when no two rows of a [n0, n1, n2, D] tensor with these strides share an element: the
// dimensions, sorted by stride, each step over the whole block of the smaller ones.
bool rows_disjoint(long long n0, long long n1, long long n2, long long D, long long s0, long long s1,
                   long long s2) {
    long long st[3] = {s0, s1, s2}, n[3] = {n0, n1, n2};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (st[j] < st[i]) {
                long long t = st[i]; st[i] = st[j]; st[j] = t;
                t = n[i]; n[i] = n[j]; n[j] = t;
            }
    long long block = D;
    for (int i = 0; i < 3; ++i) {
        if (n[i] <= 1) continue;
        if (st[i] < block) return false;
        block = st[i] * (n[i] - 1) + block;
    }
    return true;
}

// Shared validation of the GQA problem; fills `p` (without workspace pointers).  `strides`:
// NULL (contiguous [B, H, S, D]) or Q, K, V, O x (b, h, s) element strides.  `mask`: an
// osf_mask; the original entry point passes TOP_LEFT for causal and keeps its Sq == Sk rule.
int check_gqa_ex(const void *Q, const void *K, const void *V, void *O, int dtype, int B, int Hq,
                 int Hkv, int Sq, int Sk, int D, const long long *strides, int mask, float scale,
                 float *lse, AttnProblem &p, bool &empty) {
    empty = false;
    if (dtype != OSF_F32 && dtype != OSF_BF16) return OSF_ERR_INVALID;
    if (B < 0 || Hq < 0 || Hkv < 0 || Sq < 0 || Sk < 0 || D <= 0) return OSF_ERR_INVALID;
    if (Hq == 0 || Hkv == 0 || Hq % Hkv != 0) return OSF_ERR_INVALID;
    if (!(scale == scale)) return OSF_ERR_INVALID;  // NaN
    if (mask != OSF_MASK_NONE && mask != OSF_MASK_TOP_LEFT && mask != OSF_MASK_BOTTOM_RIGHT)
        return OSF_ERR_INVALID;
    long long st[12];
    if (strides) {
        for (int i = 0; i < 12; ++i) {
            if (strides[i] < 0) return OSF_ERR_INVALID;
            st[i] = strides[i];
        }
    } else {
        const long long q[3] = {(long long)Hq * Sq * D, (long long)Sq * D, D};
        const long long kv[3] = {(long long)Hkv * Sk * D, (long long)Sk * D, D};
        for (int i = 0; i < 3; ++i) {
            st[i] = q[i];
            st[3 + i] = kv[i];
            st[6 + i] = kv[i];
            st[9 + i] = q[i];
        }
    }
    if (D > 256) return OSF_ERR_UNSUPPORTED;
    if (B == 0 || Sq == 0 || Sk == 0) { empty = true; return OSF_OK; }
    // per-head element counts index with 32-bit row numbers inside kernels
    if ((long long)Sq * D >= (1LL << 31) || (long long)Sk * D >= (1LL << 31) ||
        (long long)B * Hq >= (1LL << 31) || (long long)B * Hq * Sq >= (1LL << 40))
        return OSF_ERR_UNSUPPORTED;
    for (int i = 0; i < 12; ++i)
        if (st[i] >= (1LL << 40)) return OSF_ERR_UNSUPPORTED;
    if (!Q || !K || !V || !O) return OSF_ERR_INVALID;
    const size_t es = elem_size(dtype);
    const size_t nq = span_bytes(B, Hq, Sq, D, st[0], st[1], st[2], es);
    const size_t nk = span_bytes(B, Hkv, Sk, D, st[3], st[4], st[5], es);
    const size_t nv = span_bytes(B, Hkv, Sk, D, st[6], st[7], st[8], es);
    const size_t no = span_bytes(B, Hq, Sq, D, st[9], st[10], st[11], es);
    if (!rows_disjoint(B, Hq, Sq, D, st[9], st[10], st[11])) return OSF_ERR_INVALID;
    if (overlaps(O, no, Q, nq) || overlaps(O, no, K, nk) || overlaps(O, no, V, nv))
        return OSF_ERR_INVALID;
    if (lse) {
        const size_t nl = (size_t)B * Hq * Sq * sizeof(float);
        if (overlaps(lse, nl, O, no) || overlaps(lse, nl, Q, nq) || overlaps(lse, nl, K, nk) ||
            overlaps(lse, nl, V, nv))
            return OSF_ERR_INVALID;
    }
    p = AttnProblem{};
    p.q = Q; p.k = K; p.v = V; p.o = O; p.lse = lse;
    p.dtype = dtype;
    p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.Sq = Sq; p.Sk = Sk; p.D = D;
    p.q_sb = st[0]; p.q_sh = st[1]; p.q_ss = st[2];
    p.k_sb = st[3]; p.k_sh = st[4]; p.k_ss = st[5];
    p.v_sb = st[6]; p.v_sh = st[7]; p.v_ss = st[8];
    p.o_sb = st[9]; p.o_sh = st[10]; p.o_ss = st[11];
    // key j is visible to row i iff j <= i + off; a mask that hides nothing is dropped
    const long long off = mask == OSF_MASK_BOTTOM_RIGHT ? (long long)Sk - Sq : 0;
    const bool masks = (mask == OSF_MASK_TOP_LEFT && Sq > 1) || mask == OSF_MASK_BOTTOM_RIGHT;
    p.causal = (masks && off < (long long)Sk - 1) ? 1 : 0;
    p.causal_off = p.causal ? (int)off : 0;
    const float sc = scale > 0.f ? scale : 1.0f / sqrtf((float)D);
    p.scale_log2 = sc * kLog2e;
    p.splits = 1;
    return OSF_OK;
}

int check_gqa(const void *Q, const void *K, const void *V, void *O, int dtype, int B, int Hq,
              int Hkv, int Sq, int Sk, int D, int causal, float scale, float *lse,
              AttnProblem &p, bool &empty) {
    // the original entry point: contiguous tensors, causal only with Sq == Sk (or Sq == 1)
    if (causal && Sq > 1 && Sq != Sk) return OSF_ERR_INVALID;
    return check_gqa_ex(Q, K, V, O, dtype, B, Hq, Hkv, Sq, Sk, D, nullptr,
                        causal ? OSF_MASK_TOP_LEFT : OSF_MASK_NONE, scale, lse, p, empty);
}

// Workspace layout for split partial states: acc | m | l (floats), 256-byte aligned pieces.
size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

size_t partial_bytes(int splits, long long rows, int D) {
    if (splits <= 1) return 0;
    return align256((size_t)splits * rows * D * 4) + 2 * align256((size_t)splits * rows * 4);
}

void carve_partials(AttnProblem &p, void *ws, long long rows) {
    char *base = static_cast<char *>(ws);
    p.part_acc = reinterpret_cast<float *>(base);
    base += align256((size_t)p.splits * rows * p.D * 4);
    p.part_m = reinterpret_cast<float *>(base);
    base += align256((size_t)p.splits * rows * 4);
    p.part_l = reinterpret_cast<float *>(base);
}

// Which kernel runs a (validated, non-empty) problem.
enum class Path { Simt, TensorCore, Decode };

// float32 rows of 64 channels under a window, where the call is short: the tensor cores first split what is seen of K and V into
// bfloat16 parts, in a launch of its own, and take 256 rows to a CTA; the CUDA cores take 64 at a sixth of the rate, which is less while
// their tiles of 64 keys number no more than the SMs and none has many in a row.  (us, CUDA cores against tensor cores, rows x
// heads / window: 20 x 2 / 200 15, 17; 200 x 2 / 1000 17, 22; 500 x 2 / 200 17, 20; 2 x 8 / 1000 17, 19; 77 x 8 / 200 17, 17; with more
// tiles 1000 x 2 / 200 21, 19; 200 x 8 / 200 21, 19; 77 x 8 / 1000 21, 19; 1000 x 8 / 200 53, 25; 77 x 128 / 1000 194, 57; 4000 x 32 / 1000
// 1307, 255; in a row: 20 x 2 / 4000 27, 20.)
bool f32_window_small(const AttnProblem &p) {
    int sms = 0;
    if (!p.window || p.dtype != OSF_F32 || device_sm_count(&sms) != OSF_OK) return false;
    const long long tiles = key_stream_max(64, p.Sk, p.window, p.sinks, 64), blocks = (p.Sq + 63LL) / 64 * p.B * p.Hq;
    return tiles <= 32 && blocks * tiles <= sms;
}

Path choose_path(const AttnProblem &p, const void *Q, const void *K, const void *V, const void *O) {
    // one or a few query rows per head (G * Sq <= 16): the HBM-bound decode kernel, which reads
    // each K/V byte once for all the query heads of its kv head
    if (p.dtype == OSF_BF16 && decode_supported(p, Q, K, V, O)) return Path::Decode;
    // bf16, and fp32 with D = 64 (as bf16 high / low parts)
    if (p.Sq > 1 && !f32_window_small(p) && attn_tc_supported(p, Q, K, V, O)) return Path::TensorCore;
    return Path::Simt;
}

int plan_splits(const AttnProblem &p, Path path, int sm_count, int requested) {
    if (path == Path::TensorCore) return attn_tc_pick_splits(p, sm_count);
    if (path == Path::Decode) return decode_pick_splits(p, sm_count, requested);
    if (requested > 0 && (long long)p.B * p.Hq <= 65535) {
        const int n_kt = (p.Sk + 63) / 64;
        return requested < n_kt ? requested : n_kt;
    }
    return attn_simt_pick_splits(p, sm_count);
}

size_t path_workspace(const AttnProblem &p, Path path, int splits) {
    // every path keeps split partial states in the same layout; the tensor-core path keeps the
    // fp32 operands' bf16 parts after them
    const size_t part = partial_bytes(splits, (long long)p.B * p.Hq * p.Sq, p.D);
    return path == Path::TensorCore ? part + align256(attn_tc_extra_bytes(p)) : part;
}

int run_gqa(AttnProblem &p, Path path, void *workspace, size_t workspace_bytes, int splits,
            DeviceInfo *dev, cudaStream_t s) {
    p.splits = splits;
    p.status = dev->status;
    const size_t need = path_workspace(p, path, splits);
    if (need > 0 && (!workspace || workspace_bytes < need)) return OSF_ERR_WORKSPACE;
    const long long rows = (long long)p.B * p.Hq * p.Sq;
    switch (path) {
        case Path::TensorCore:
            if (splits > 1) carve_partials(p, workspace, rows);
            p.x3_ws = attn_tc_extra_bytes(p) > 0
                          ? static_cast<void *>(static_cast<char *>(workspace) + partial_bytes(splits, rows, p.D))
                          : nullptr;
            return launch_status(launch_attn_tc(p, dev->sm_count, s));
        case Path::Decode:
            if (splits > 1) carve_partials(p, workspace, rows);
            return launch_status(launch_decode(p, s));
        case Path::Simt:
        default: {
            if (splits > 1) carve_partials(p, workspace, rows);
            cudaError_t e = launch_attn_simt(p, s);
            if (e == cudaSuccess && splits > 1) e = launch_attn_combine(p, s);
            return launch_status(e);
        }
    }
}

// ------------------------------------------------------------- host buffers in and out
// osf_attn_fwd_gqa_host splits the problem into chunks of whole (batch, kv head) units: unit u =
// b * Hkv + g owns the G query heads g*G .. g*G+G-1 of batch b and kv head g, so a run of
// consecutive units is one contiguous range of Q, K, V and O, and a chunk of n units is itself a
// GQA problem with B = n, Hq = G, Hkv = 1.  Each chunk's copies in, attention and copy out are
// enqueued on three streams (copy-in, the caller's, copy-out) linked by events, so the copies of
// one chunk overlap the attention of another and the two copy directions overlap each other.
constexpr int kHostChunks = 8;

struct HostUnits {
    long long units = 0;      // B * Hkv
    int chunks = 0;           // number of chunks
    long long per = 0;        // units per chunk (the last may have fewer)
    size_t q_unit = 0, kv_unit = 0;   // bytes of one unit's Q (and O) and of its K (and V)
};

HostUnits host_units(int dtype, int B, int Hq, int Hkv, int Sq, int Sk, int D) {
    HostUnits h;
    const int G = Hq / Hkv;
    h.units = (long long)B * Hkv;
    h.chunks = (int)std::min<long long>(h.units, kHostChunks);
    h.per = (h.units + h.chunks - 1) / h.chunks;
    h.chunks = (int)((h.units + h.per - 1) / h.per);
    h.q_unit = (size_t)G * Sq * D * elem_size(dtype);
    h.kv_unit = (size_t)Sk * D * elem_size(dtype);
    return h;
}

// Device-buffer layout: Q | K | V | O | chunk workspace, each piece 256-byte aligned.
struct HostLayout {
    size_t q = 0, k = 0, v = 0, o = 0, ws = 0, ws_bytes = 0, total = 0;
};

int host_layout(int dtype, int B, int Hq, int Hkv, int Sq, int Sk, int D, HostLayout &L) {
    const HostUnits h = host_units(dtype, B, Hq, Hkv, Sq, Sk, D);
    const size_t qb = h.q_unit * h.units, kvb = h.kv_unit * h.units;
    // workspace: the larger need of a full chunk and of the last (smaller) one
    size_t ws = 0;
    const long long sizes[2] = {h.per, h.units - (long long)(h.chunks - 1) * h.per};
    for (long long n : sizes) {
        size_t w = 0;
        const int st = osf_attn_workspace_bytes(dtype, (int)n, Hq / Hkv, 1, Sq, Sk, D, &w);
        if (st != OSF_OK) return st;
        ws = std::max(ws, w);
    }
    L.q = 0;
    L.k = align256(qb);
    L.v = L.k + align256(kvb);
    L.o = L.v + align256(kvb);
    L.ws = L.o + align256(qb);
    L.ws_bytes = ws;
    L.total = L.ws + align256(ws);
    return OSF_OK;
}

// Per-device copy streams and events, created on the first host-buffer call on the device.
struct HostStreams {
    cudaStream_t in = nullptr, out = nullptr;
    cudaEvent_t start = nullptr, done = nullptr;
    cudaEvent_t landed[kHostChunks] = {}, computed[kHostChunks] = {};
    bool ready = false;
};
HostStreams g_host[kMaxDevices];
std::mutex g_host_mutex;   // held while a call enqueues its work (the events are shared)

int host_streams(HostStreams **out) {
    int dev;
    if (current_device(&dev) != OSF_OK) return OSF_ERR_CUDA;
    HostStreams &h = g_host[dev];
    if (!h.ready) {
        bool ok = cudaStreamCreateWithFlags(&h.in, cudaStreamNonBlocking) == cudaSuccess &&
                  cudaStreamCreateWithFlags(&h.out, cudaStreamNonBlocking) == cudaSuccess &&
                  cudaEventCreateWithFlags(&h.start, cudaEventDisableTiming) == cudaSuccess &&
                  cudaEventCreateWithFlags(&h.done, cudaEventDisableTiming) == cudaSuccess;
        for (int i = 0; ok && i < kHostChunks; ++i)
            ok = cudaEventCreateWithFlags(&h.landed[i], cudaEventDisableTiming) == cudaSuccess &&
                 cudaEventCreateWithFlags(&h.computed[i], cudaEventDisableTiming) == cudaSuccess;
        if (!ok) {
            // release what was created, so a later call starts over cleanly
            if (h.in) cudaStreamDestroy(h.in);
            if (h.out) cudaStreamDestroy(h.out);
            cudaEvent_t *evs[] = {&h.start, &h.done};
            for (cudaEvent_t *e : evs)
                if (*e) cudaEventDestroy(*e);
            for (int i = 0; i < kHostChunks; ++i) {
                if (h.landed[i]) cudaEventDestroy(h.landed[i]);
                if (h.computed[i]) cudaEventDestroy(h.computed[i]);
            }
            h = HostStreams();
            return OSF_ERR_CUDA;
        }
        h.ready = true;
    }
    *out = &h;
    return OSF_OK;
}

}  // namespace
}  // namespace osf

using namespace osf;

extern "C" {

const char *osf_status_string(int status) {
    switch (status) {
        case OSF_OK: return "OSF_OK";
        case OSF_ERR_INVALID: return "OSF_ERR_INVALID: invalid argument";
        case OSF_ERR_UNSUPPORTED: return "OSF_ERR_UNSUPPORTED: unsupported size or type";
        case OSF_ERR_CUDA: return "OSF_ERR_CUDA: CUDA runtime error";
        case OSF_ERR_TIMEOUT: return "OSF_ERR_TIMEOUT: a bounded device wait expired";
        case OSF_ERR_WORKSPACE: return "OSF_ERR_WORKSPACE: workspace missing or too small";
        default: return "unknown osf status";
    }
}

int osf_version(void) { return 100; }

unsigned long long osf_launch_count(void) { return g_launches.load(std::memory_order_relaxed); }

int osf_sm_count(void) {
    DeviceInfo *d;
    return device_info(&d) == OSF_OK ? d->sm_count : 0;
}

int osf_attn_fwd(const float *Q, const float *K, const float *V, float *out, int M, int N, int d,
                 osf_stream stream) {
    if (M < 0 || N < 0 || d <= 0) return OSF_ERR_INVALID;
    if (M == 0 || N == 0) return OSF_OK;
    AttnProblem p;
    bool empty;
    int st = check_gqa(Q, K, V, out, OSF_F32, 1, 1, 1, M, N, d, 0, 0.f, nullptr, p, empty);
    if (st != OSF_OK || empty) return st;
    DeviceInfo *dev;
    if (device_info(&dev) != OSF_OK) return OSF_ERR_CUDA;
    // no workspace in this signature: run unsplit
    return run_gqa(p, Path::Simt, nullptr, 0, 1, dev, (cudaStream_t)stream);
}

int osf_attn_workspace_bytes(int dtype, int B, int Hq, int Hkv, int Sq, int Sk, int D,
                             size_t *bytes) {
    if (!bytes) return OSF_ERR_INVALID;
    *bytes = 0;
    AttnProblem p;
    bool empty;
    // pointers are not known here: validate sizes with placeholder addresses
    const void *ph = reinterpret_cast<const void *>(uintptr_t(1) << 40);
    int st = check_gqa(ph, ph, ph, reinterpret_cast<void *>(uintptr_t(1) << 44), dtype, B, Hq, Hkv,
                       Sq, Sk, D, 0, 0.f, nullptr, p, empty);
    if (st != OSF_OK || empty) return st;
    DeviceInfo *dev;
    if (device_info(&dev) != OSF_OK) return OSF_ERR_CUDA;
    // the larger of the possible paths' needs (alignment decides the path at call time)
    size_t need = partial_bytes(attn_simt_pick_splits(p, dev->sm_count), (long long)B * Hq * Sq, D);
    if (Sq > 1 && ((dtype == OSF_BF16 && (D == 64 || D == 128)) || (dtype == OSF_F32 && D == 64))) {
        const size_t tc = path_workspace(p, Path::TensorCore, attn_tc_pick_splits(p, dev->sm_count));
        if (tc > need) need = tc;
    }
    if (dtype == OSF_BF16 && (long long)(Hq / Hkv) * Sq <= 16) {
        const size_t dn = partial_bytes(decode_pick_splits(p, dev->sm_count, 0), (long long)B * Hq * Sq, D);
        if (dn > need) need = dn;
    }
    *bytes = need;
    return OSF_OK;
}

int osf_attn_fwd_gqa(const void *Q, const void *K, const void *V, void *O, int dtype, int B,
                     int Hq, int Hkv, int Sq, int Sk, int D, int causal, float scale, float *lse,
                     void *workspace, size_t workspace_bytes, osf_stream stream) {
    AttnProblem p;
    bool empty;
    int st = check_gqa(Q, K, V, O, dtype, B, Hq, Hkv, Sq, Sk, D, causal, scale, lse, p, empty);
    if (st != OSF_OK || empty) return st;
    DeviceInfo *dev;
    if (device_info(&dev) != OSF_OK) return OSF_ERR_CUDA;
    const Path path = choose_path(p, Q, K, V, O);
    const int splits = plan_splits(p, path, dev->sm_count, 0);
    return run_gqa(p, path, workspace, workspace_bytes, splits, dev, (cudaStream_t)stream);
}

int osf_attn_fwd_gqa_ex(const void *Q, const void *K, const void *V, void *O, int dtype, int B,
                        int Hq, int Hkv, int Sq, int Sk, int D, const long long *strides, int mask,
                        float scale, float *lse, void *workspace, size_t workspace_bytes,
                        osf_stream stream) {
    AttnProblem p;
    bool empty;
    int st = check_gqa_ex(Q, K, V, O, dtype, B, Hq, Hkv, Sq, Sk, D, strides, mask, scale, lse, p, empty);
    if (st != OSF_OK || empty) return st;
    DeviceInfo *dev;
    if (device_info(&dev) != OSF_OK) return OSF_ERR_CUDA;
    const Path path = choose_path(p, Q, K, V, O);
    const int splits = plan_splits(p, path, dev->sm_count, 0);
    return run_gqa(p, path, workspace, workspace_bytes, splits, dev, (cudaStream_t)stream);
}

int osf_attn_host_buffer_bytes(int dtype, int B, int Hq, int Hkv, int Sq, int Sk, int D, int causal,
                               size_t *bytes) {
    if (!bytes) return OSF_ERR_INVALID;
    *bytes = 0;
    AttnProblem p;
    bool empty;
    const void *ph = reinterpret_cast<const void *>(uintptr_t(1) << 40);
    int st = check_gqa(ph, ph, ph, reinterpret_cast<void *>(uintptr_t(1) << 44), dtype, B, Hq, Hkv,
                       Sq, Sk, D, causal, 0.f, nullptr, p, empty);
    if (st != OSF_OK || empty) return st;
    HostLayout L;
    st = host_layout(dtype, B, Hq, Hkv, Sq, Sk, D, L);
    if (st != OSF_OK) return st;
    *bytes = L.total;
    return OSF_OK;
}

int osf_attn_fwd_gqa_host(const void *Q, const void *K, const void *V, void *O, int dtype, int B,
                          int Hq, int Hkv, int Sq, int Sk, int D, int causal, float scale,
                          void *device_buffer, size_t device_buffer_bytes, osf_stream stream) {
    AttnProblem p;
    bool empty;
    // validate the sizes and the host pointers as a whole problem
    int st = check_gqa(Q, K, V, O, dtype, B, Hq, Hkv, Sq, Sk, D, causal, scale, nullptr, p, empty);
    if (st != OSF_OK || empty) return st;
    if (!device_buffer) return OSF_ERR_WORKSPACE;
    HostLayout L;
    st = host_layout(dtype, B, Hq, Hkv, Sq, Sk, D, L);
    if (st != OSF_OK) return st;
    if (device_buffer_bytes < L.total) return OSF_ERR_WORKSPACE;
    DeviceInfo *dev;
    if (device_info(&dev) != OSF_OK) return OSF_ERR_CUDA;
    HostStreams *hs;
    std::lock_guard<std::mutex> lock(g_host_mutex);
    if (host_streams(&hs) != OSF_OK) return OSF_ERR_CUDA;
    const cudaStream_t s = (cudaStream_t)stream;
    const HostUnits h = host_units(dtype, B, Hq, Hkv, Sq, Sk, D);
    char *base = static_cast<char *>(device_buffer);
    char *dq = base + L.q, *dk = base + L.k, *dv = base + L.v, *dout = base + L.o;
    void *ws = L.ws_bytes > 0 ? base + L.ws : nullptr;
    const char *hq = static_cast<const char *>(Q), *hk = static_cast<const char *>(K),
               *hv = static_cast<const char *>(V);
    char *ho = static_cast<char *>(O);
    const int G = Hq / Hkv;
    // everything earlier on the caller's stream (a previous call using this buffer) comes first
    if (cudaEventRecord(hs->start, s) != cudaSuccess || cudaStreamWaitEvent(hs->in, hs->start, 0) != cudaSuccess)
        return OSF_ERR_CUDA;
    // On an error after this point some chunks may already be queued on the copy streams: the
    // caller's stream is made to wait for both of them (best effort) so that work it enqueues
    // next still runs after them, and the error is returned.  O is then undefined.
    auto fail = [&](int code) {
        if (cudaEventRecord(hs->start, hs->in) == cudaSuccess) cudaStreamWaitEvent(s, hs->start, 0);
        if (cudaEventRecord(hs->done, hs->out) == cudaSuccess) cudaStreamWaitEvent(s, hs->done, 0);
        cudaGetLastError();
        return code;
    };
    for (int c = 0; c < h.chunks; ++c) {
        const long long u0 = (long long)c * h.per;
        const long long n = std::min<long long>(h.per, h.units - u0);
        const size_t qo = (size_t)u0 * h.q_unit, ko = (size_t)u0 * h.kv_unit;
        const size_t qn = (size_t)n * h.q_unit, kn = (size_t)n * h.kv_unit;
        if (cudaMemcpyAsync(dq + qo, hq + qo, qn, cudaMemcpyHostToDevice, hs->in) != cudaSuccess ||
            cudaMemcpyAsync(dk + ko, hk + ko, kn, cudaMemcpyHostToDevice, hs->in) != cudaSuccess ||
            cudaMemcpyAsync(dv + ko, hv + ko, kn, cudaMemcpyHostToDevice, hs->in) != cudaSuccess ||
            cudaEventRecord(hs->landed[c], hs->in) != cudaSuccess || cudaStreamWaitEvent(s, hs->landed[c], 0) != cudaSuccess)
            return fail(OSF_ERR_CUDA);
        // the chunk as its own problem: B = n units, Hq = G, Hkv = 1
        AttnProblem pc;
        bool ec;
        st = check_gqa(dq + qo, dk + ko, dv + ko, dout + qo, dtype, (int)n, G, 1, Sq, Sk, D, causal, scale, nullptr,
                       pc, ec);
        if (st != OSF_OK) return fail(st);
        const Path path = choose_path(pc, dq + qo, dk + ko, dv + ko, dout + qo);
        st = run_gqa(pc, path, ws, L.ws_bytes, plan_splits(pc, path, dev->sm_count, 0), dev, s);
        if (st != OSF_OK) return fail(st);
        if (cudaEventRecord(hs->computed[c], s) != cudaSuccess || cudaStreamWaitEvent(hs->out, hs->computed[c], 0) != cudaSuccess ||
            cudaMemcpyAsync(ho + qo, dout + qo, qn, cudaMemcpyDeviceToHost, hs->out) != cudaSuccess)
            return fail(OSF_ERR_CUDA);
    }
    // the caller's stream continues once O has reached the host
    if (cudaEventRecord(hs->done, hs->out) != cudaSuccess || cudaStreamWaitEvent(s, hs->done, 0) != cudaSuccess)
        return fail(OSF_ERR_CUDA);
    return OSF_OK;
}

int osf_attn_decode_workspace_bytes(int dtype, int B, int Hq, int Hkv, int Sk, int D,
                                    int num_splits, size_t *bytes) {
    if (!bytes) return OSF_ERR_INVALID;
    *bytes = 0;
    AttnProblem p;
    bool empty;
    const void *ph = reinterpret_cast<const void *>(uintptr_t(1) << 40);
    int st = check_gqa(ph, ph, ph, reinterpret_cast<void *>(uintptr_t(1) << 44), dtype, B, Hq, Hkv,
                       1, Sk, D, 0, 0.f, nullptr, p, empty);
    if (st != OSF_OK || empty) return st;
    DeviceInfo *dev;
    if (device_info(&dev) != OSF_OK) return OSF_ERR_CUDA;
    size_t need = partial_bytes(plan_splits(p, Path::Simt, dev->sm_count, num_splits), (long long)B * Hq, D);
    if (dtype == OSF_BF16) {
        const size_t dn = partial_bytes(decode_pick_splits(p, dev->sm_count, num_splits), (long long)B * Hq, D);
        if (dn > need) need = dn;
    }
    *bytes = need;
    return OSF_OK;
}

int osf_attn_decode_gqa(const void *Q, const void *K, const void *V, void *O, int dtype, int B,
                        int Hq, int Hkv, int Sk, int D, float scale, float *lse, int num_splits,
                        void *workspace, size_t workspace_bytes, osf_stream stream) {
    AttnProblem p;
    bool empty;
    int st = check_gqa(Q, K, V, O, dtype, B, Hq, Hkv, 1, Sk, D, 0, scale, lse, p, empty);
    if (st != OSF_OK || empty) return st;
    DeviceInfo *dev;
    if (device_info(&dev) != OSF_OK) return OSF_ERR_CUDA;
    const Path path = (dtype == OSF_BF16 && decode_supported(p, Q, K, V, O)) ? Path::Decode : Path::Simt;
    const int splits = plan_splits(p, path, dev->sm_count, num_splits);
    return run_gqa(p, path, workspace, workspace_bytes, splits, dev, (cudaStream_t)stream);
}

int osf_softmax_workspace_bytes(long long rows, long long T, size_t *bytes) {
    if (!bytes) return OSF_ERR_INVALID;
    *bytes = 0;
    if (rows < 0 || T < 0) return OSF_ERR_INVALID;
    if (rows == 0 || T == 0) return OSF_OK;
    if (rows > 65535 && T > 32768) return OSF_ERR_UNSUPPORTED;
    DeviceInfo *dev;
    if (device_info(&dev) != OSF_OK) return OSF_ERR_CUDA;
    *bytes = softmax_workspace_floats(rows, T, dev->sm_count) * sizeof(float);
    return OSF_OK;
}

int osf_softmax_rows(const float *x, float *z, long long rows, long long T, void *workspace,
                     size_t workspace_bytes, osf_stream stream) {
    if (rows < 0 || T < 0) return OSF_ERR_INVALID;
    if (rows == 0 || T == 0) return OSF_OK;
    if (!x || !z) return OSF_ERR_INVALID;
    if (rows > (1LL << 31) - 1 || (rows > 65535 && T > 32768)) return OSF_ERR_UNSUPPORTED;
    const size_t n = (size_t)rows * (size_t)T * sizeof(float);
    if ((const void *)x != (const void *)z && overlaps(x, n, z, n)) return OSF_ERR_INVALID;
    DeviceInfo *dev;
    if (device_info(&dev) != OSF_OK) return OSF_ERR_CUDA;
    const size_t need = softmax_workspace_floats(rows, T, dev->sm_count) * sizeof(float);
    if (need > 0 && (!workspace || workspace_bytes < need)) return OSF_ERR_WORKSPACE;
    return launch_status(launch_softmax_rows(x, z, rows, T, static_cast<float *>(workspace),
                                             dev->sm_count, (cudaStream_t)stream));
}

// Bytes of bf16 dS^T the tensor-core backward keeps for its separate dQ product ([128 x 128]
// tiles covering [B * Hq][Sk rounded up to 128][Sq rounded up to 128]); 0 where that path does not
// apply or the buffer would pass 16 GiB (dQ then recomputes S and dP instead).
static size_t bwd_ds_bytes(int dtype, int B, int Hq, int Sq, int Sk, int D) {
    if (dtype != OSF_BF16 || (D != 64 && D != 128) || B <= 0 || Hq <= 0 || Sq <= 0 || Sk <= 0) return 0;
    const size_t cap = (size_t)16 << 30;
    const size_t tile = ((size_t)Sk + 127) / 128 * 128 * (((size_t)Sq + 127) / 128 * 128) * 2;
    if (tile > cap / ((size_t)B * (size_t)Hq)) return 0;
    return align256(tile * (size_t)B * (size_t)Hq);
}

int osf_attn_bwd_workspace_bytes(int dtype, int B, int Hq, int Hkv, int Sq, int Sk, int D, size_t *bytes) {
    if (!bytes) return OSF_ERR_INVALID;
    *bytes = 0;
    AttnProblem p;
    bool empty;
    const void *ph = reinterpret_cast<const void *>(uintptr_t(1) << 40);
    int st = check_gqa_ex(ph, ph, ph, reinterpret_cast<void *>(uintptr_t(1) << 44), dtype, B, Hq, Hkv, Sq, Sk, D,
                          nullptr, OSF_MASK_NONE, 0.f, nullptr, p, empty);
    if (st != OSF_OK || empty) return st;
    *bytes = align256((size_t)B * Hq * Sq * sizeof(float)) + bwd_ds_bytes(dtype, B, Hq, Sq, Sk, D);
    return OSF_OK;
}

// The backward problem of a checked forward one (p, whose output is dQ): its buffers' checks, and its fields but for the
// workspace.
static int check_bwd(const AttnProblem &p, const void *O, const void *dO, const float *lse, void *dK, void *dV, BwdProblem &b) {
    if (!O || !dO || !lse || !dK || !dV) return OSF_ERR_INVALID;
    const size_t es = elem_size(p.dtype);
    const size_t nq = (size_t)p.B * p.Hq * p.Sq * p.D * es, nkv = (size_t)p.B * p.Hkv * p.Sk * p.D * es;
    const size_t nl = (size_t)p.B * p.Hq * p.Sq * sizeof(float);
    const void *ins[6] = {p.q, p.k, p.v, O, dO, lse};
    const size_t in_n[6] = {nq, nkv, nkv, nq, nq, nl};
    void *outs[3] = {p.o, dK, dV};
    const size_t out_n[3] = {nq, nkv, nkv};
    for (int o = 0; o < 3; ++o) {
        for (int i = 0; i < 6; ++i)
            if (overlaps(outs[o], out_n[o], ins[i], in_n[i])) return OSF_ERR_INVALID;
        for (int o2 = o + 1; o2 < 3; ++o2)
            if (overlaps(outs[o], out_n[o], outs[o2], out_n[o2])) return OSF_ERR_INVALID;
    }
    b = BwdProblem{};
    b.q = p.q; b.k = p.k; b.v = p.v; b.o = O; b.dout = dO; b.lse = lse;
    b.dq = p.o; b.dk = dK; b.dv = dV;
    b.dtype = p.dtype;
    b.B = p.B; b.Hq = p.Hq; b.Hkv = p.Hkv; b.Sq = p.Sq; b.Sk = p.Sk; b.D = p.D;
    b.causal = p.causal; b.causal_off = p.causal_off;
    b.scale_log2 = p.scale_log2;
    b.scale = p.scale_log2 / kLog2e;
    return OSF_OK;
}

int osf_attn_bwd_gqa(const void *Q, const void *K, const void *V, const void *O, const void *dO,
                     const float *lse, void *dQ, void *dK, void *dV, int dtype, int B, int Hq, int Hkv,
                     int Sq, int Sk, int D, int mask, float scale, void *workspace, size_t workspace_bytes,
                     osf_stream stream) {
    AttnProblem p;
    bool empty;
    // the forward problem's checks (sizes, mask, scale; dQ plays the output's part)
    int st = check_gqa_ex(Q, K, V, dQ, dtype, B, Hq, Hkv, Sq, Sk, D, nullptr, mask, scale, nullptr, p, empty);
    if (st != OSF_OK) return st;
    if (empty) {
        // no keys or no rows: gradients are zero (written when there is anything to write)
        return OSF_OK;
    }
    BwdProblem b;
    st = check_bwd(p, O, dO, lse, dK, dV, b);
    if (st != OSF_OK) return st;
    const size_t need = align256((size_t)B * Hq * Sq * sizeof(float));
    if (!workspace || workspace_bytes < need) return OSF_ERR_WORKSPACE;
    DeviceInfo *dev;
    if (device_info(&dev) != OSF_OK) return OSF_ERR_CUDA;
    b.dvec = static_cast<float *>(workspace);
    // a workspace that also holds dS^T selects the tensor-core path's separate dQ product
    const size_t ds_bytes = bwd_ds_bytes(dtype, B, Hq, Sq, Sk, D);
    if (ds_bytes > 0 && workspace_bytes >= need + ds_bytes &&
        ((reinterpret_cast<uintptr_t>(workspace) + need) & 31u) == 0) {
        b.ds = static_cast<char *>(workspace) + need;
        b.ds_rows = ((long long)Sk + 127) / 128 * 128;
        b.ds_ld = ((long long)Sq + 127) / 128 * 128;
    }
    b.status = dev->status;
    return launch_status(launch_attn_bwd(b, (cudaStream_t)stream));
}

// A workspace of `need` bytes: large enough, and aligned for the 16-byte accesses that the kernels make to it.
static int check_workspace(const void *workspace, size_t bytes, size_t need) {
    if (need == 0) return OSF_OK;
    if (!workspace || bytes < need) return OSF_ERR_WORKSPACE;
    return (reinterpret_cast<uintptr_t>(workspace) & 15u) ? OSF_ERR_INVALID : OSF_OK;
}

// Whether a pointer is not on a boundary of its elements (a kernel's access to it would be a fault).
static bool misaligned(const void *q, size_t es) { return reinterpret_cast<uintptr_t>(q) % es != 0; }

// ------------------------------------------------------------------ a window with sinks
// The checks of a windowed problem: those of a bottom-right one, then the window.  One that hides nothing is dropped, but where
// the windowed kernels are the faster ones: `keep` (the window then is the whole sequence).
static int check_window(const void *Q, const void *K, const void *V, void *O, int dtype, int B, int Hq, int Hkv, int Sq,
                        int Sk, int D, const long long *strides, int window, int sinks, float scale, float *lse, bool keep,
                        AttnProblem &p, bool &empty) {
    empty = false;
    if (window < 1 || sinks < 0) return OSF_ERR_INVALID;
    const int st = check_gqa_ex(Q, K, V, O, dtype, B, Hq, Hkv, Sq, Sk, D, strides, OSF_MASK_BOTTOM_RIGHT, scale, lse, p, empty);
    if (st != OSF_OK || empty) return st;
    const size_t es = elem_size(dtype);
    if (misaligned(Q, es) || misaligned(K, es) || misaligned(V, es) || misaligned(O, es) || misaligned(lse, 4)) return OSF_ERR_INVALID;
    // kernels add lengths and the window in ints
    if (Sq >= (1 << 29) || Sk >= (1 << 29)) return OSF_ERR_UNSUPPORTED;
    // the last row sees the most hidden keys: those between the sinks and its window
    const bool hides = (long long)window + sinks < Sk;
    if (hides || keep) {
        p.causal = 1;
        p.causal_off = Sk - Sq;
        p.window = hides ? window : Sk;
        p.sinks = hides ? sinks : 0;
    }
    return OSF_OK;
}
// bfloat16 rows of 32 and 96 channels run on the tensor cores with a window, and on the CUDA cores without one.
static bool keep_fwd_window(int dtype, int D) { return dtype == OSF_BF16 && (D == 32 || D == 96); }
// The backward pass on the CUDA cores: chunks of 32 with a window, a warp per row without one.
static bool keep_bwd_window(int dtype, int D) { return !(dtype == OSF_BF16 && (D == 64 || D == 128)); }
static bool window_tc(int dtype, int D) { return dtype == OSF_BF16 && (D == 32 || D == 64 || D == 96 || D == 128); }

int osf_attn_window_workspace_bytes(int dtype, int B, int Hq, int Hkv, int Sq, int Sk, int D, int window, int sinks,
                                    size_t *bytes) {
    if (!bytes) return OSF_ERR_INVALID;
    *bytes = 0;
    AttnProblem p;
    bool empty;
    const void *ph = reinterpret_cast<const void *>(uintptr_t(1) << 40);
    const int st = check_window(ph, ph, ph, reinterpret_cast<void *>(uintptr_t(1) << 44), dtype, B, Hq, Hkv, Sq, Sk, D,
                                nullptr, window, sinks, 0.f, nullptr, keep_fwd_window(dtype, D), p, empty);
    if (st != OSF_OK || empty) return st;
    DeviceInfo *dev;
    if (device_info(&dev) != OSF_OK) return OSF_ERR_CUDA;
    // the largest of the possible paths' needs (alignment decides the path at call time)
    size_t need = path_workspace(p, Path::Simt, plan_splits(p, Path::Simt, dev->sm_count, 0));
    if (Sq > 1 && (window_tc(dtype, D) || (dtype == OSF_F32 && D == 64 && !f32_window_small(p))))
        need = std::max(need, path_workspace(p, Path::TensorCore, plan_splits(p, Path::TensorCore, dev->sm_count, 0)));
    if (dtype == OSF_BF16 && (long long)(Hq / Hkv) * Sq <= 16)
        need = std::max(need, path_workspace(p, Path::Decode, plan_splits(p, Path::Decode, dev->sm_count, 0)));
    *bytes = need;
    return OSF_OK;
}

int osf_attn_fwd_gqa_window(const void *Q, const void *K, const void *V, void *O, int dtype, int B, int Hq, int Hkv, int Sq,
                            int Sk, int D, const long long *strides, int window, int sinks, float scale, float *lse,
                            void *workspace, size_t workspace_bytes, osf_stream stream) {
    AttnProblem p;
    bool empty;
    int st = check_window(Q, K, V, O, dtype, B, Hq, Hkv, Sq, Sk, D, strides, window, sinks, scale, lse, keep_fwd_window(dtype, D),
                          p, empty);
    if (st != OSF_OK || B == 0 || Sq == 0) return st;
    DeviceInfo *dev;
    if (device_info(&dev) != OSF_OK) return OSF_ERR_CUDA;
    if (empty) {
        // no keys: every row sees nothing.  The problem of one key, whose place nothing reads, without it
        long long sd[12] = {};   // (K and V: strides of no extent)
        for (int i = 0; strides && i < 3; ++i) {
            sd[i] = strides[i];
            sd[9 + i] = strides[9 + i];
        }
        st = check_window(Q, Q, Q, O, dtype, B, Hq, Hkv, Sq, 1, D, strides ? sd : nullptr, window, sinks, scale, lse, false,
                          p, empty);
        if (st != OSF_OK) return st;
        p.Sk = p.causal = p.window = 0;
        return run_gqa(p, Path::Simt, nullptr, 0, 1, dev, (cudaStream_t)stream);
    }
    const Path path = choose_path(p, Q, K, V, O);
    const int splits = plan_splits(p, path, dev->sm_count, 0);
    const int ws = check_workspace(workspace, workspace_bytes, path_workspace(p, path, splits));
    if (ws != OSF_OK) return ws;
    return run_gqa(p, path, workspace, workspace_bytes, splits, dev, (cudaStream_t)stream);
}

// Workspace of the windowed backward: row sums | sums of the key tiles that several CTAs share | dS^T tiles that some row sees,
// where the plan stores them and they stay within 16 GiB; they may be left out by the caller (dQ then recomputes S and dP).
struct BwdWindowLayout {
    size_t rows = 0, ds = 0, parts = 0;
    BwdWindowPlan plan{};
};
static BwdWindowLayout bwd_window_layout(const AttnProblem &p, int sm_count) {
    BwdWindowLayout L;
    L.rows = align256((size_t)p.B * p.Hq * p.Sq * sizeof(float));
    if (!window_tc(p.dtype, p.D)) {
        L.plan = bwd_rows_plan(p.B, p.Hq, p.Hkv, p.Sq, p.Sk, p.D, p.window, p.sinks, sm_count);
        if (L.plan.parts > 1)
            L.parts = (size_t)L.plan.shared_tiles * L.plan.parts * p.B * p.Hkv * 2 * L.plan.part_keys * p.D * sizeof(float);
        return L;
    }
    L.plan = bwd_window_plan(p.B, p.Hq, p.Hkv, p.Sq, p.Sk, p.window, p.sinks, sm_count);
    const size_t tile = (size_t)128 * 128 * 2, per_head = (size_t)L.plan.slots * (((size_t)p.Sq + 127) / 128) * tile;
    const size_t cap = (size_t)16 << 30, heads = (size_t)p.B * p.Hq;
    if (L.plan.store_ds && per_head <= cap / heads) L.ds = per_head * heads;
    if (L.plan.parts > 1)
        L.parts = (size_t)L.plan.shared_tiles * L.plan.parts * p.B * p.Hkv * 2 * 128 * (p.D <= 64 ? 64 : 128) * sizeof(float);
    return L;
}
// A problem whose window hides nothing runs on the causal kernels, but a small one: those share no key tile out.
static void keep_small(AttnProblem &p, int sm_count) {
    if (p.window || 2LL * p.B * p.Hkv * ((p.Sk + 127) / 128) > sm_count) return;
    p.causal = 1;
    p.causal_off = p.Sk - p.Sq;
    p.window = p.Sk;
}

int osf_attn_bwd_window_workspace_bytes(int dtype, int B, int Hq, int Hkv, int Sq, int Sk, int D, int window, int sinks,
                                        size_t *bytes) {
    if (!bytes) return OSF_ERR_INVALID;
    *bytes = 0;
    AttnProblem p;
    bool empty;
    const void *ph = reinterpret_cast<const void *>(uintptr_t(1) << 40);
    const int st = check_window(ph, ph, ph, reinterpret_cast<void *>(uintptr_t(1) << 44), dtype, B, Hq, Hkv, Sq, Sk, D,
                                nullptr, window, sinks, 0.f, nullptr, keep_bwd_window(dtype, D), p, empty);
    if (st != OSF_OK || empty) return st;
    DeviceInfo *dev;
    if (device_info(&dev) != OSF_OK) return OSF_ERR_CUDA;
    keep_small(p, dev->sm_count);
    if (!p.window) return osf_attn_bwd_workspace_bytes(dtype, B, Hq, Hkv, Sq, Sk, D, bytes);
    const BwdWindowLayout L = bwd_window_layout(p, dev->sm_count);
    *bytes = L.rows + L.ds + L.parts;
    return OSF_OK;
}

int osf_attn_bwd_gqa_window(const void *Q, const void *K, const void *V, const void *O, const void *dO, const float *lse,
                            void *dQ, void *dK, void *dV, int dtype, int B, int Hq, int Hkv, int Sq, int Sk, int D,
                            int window, int sinks, float scale, void *workspace, size_t workspace_bytes, osf_stream stream) {
    AttnProblem p;
    bool empty;
    const int st = check_window(Q, K, V, dQ, dtype, B, Hq, Hkv, Sq, Sk, D, nullptr, window, sinks, scale, nullptr,
                                keep_bwd_window(dtype, D), p, empty);
    if (st != OSF_OK) return st;
    if (empty) {   // no rows, or no keys: what gradients there are are zero
        const size_t es = elem_size(dtype), nq = (size_t)B * Hq * Sq * D * es, nk = (size_t)B * Hkv * Sk * D * es;
        if ((nq && !dQ) || (nk && (!dK || !dV)) || overlaps(dK, nk, dV, nk)) return OSF_ERR_INVALID;
        if (nq && cudaMemsetAsync(dQ, 0, nq, (cudaStream_t)stream) != cudaSuccess) return OSF_ERR_CUDA;
        if (nk && (cudaMemsetAsync(dK, 0, nk, (cudaStream_t)stream) != cudaSuccess ||
                   cudaMemsetAsync(dV, 0, nk, (cudaStream_t)stream) != cudaSuccess))
            return OSF_ERR_CUDA;
        return OSF_OK;
    }
    BwdProblem b;
    const int sb = check_bwd(p, O, dO, lse, dK, dV, b);
    if (sb != OSF_OK) return sb;
    const size_t es = elem_size(dtype);
    if (misaligned(O, es) || misaligned(dO, es) || misaligned(lse, 4) || misaligned(dK, es) || misaligned(dV, es)) return OSF_ERR_INVALID;
    DeviceInfo *dev;
    if (device_info(&dev) != OSF_OK) return OSF_ERR_CUDA;
    keep_small(p, dev->sm_count);
    if (!p.window)
        return osf_attn_bwd_gqa(Q, K, V, O, dO, lse, dQ, dK, dV, dtype, B, Hq, Hkv, Sq, Sk, D, OSF_MASK_BOTTOM_RIGHT, scale,
                                workspace, workspace_bytes, stream);
    b.causal = p.causal;
    b.causal_off = p.causal_off;
    const BwdWindowLayout L = bwd_window_layout(p, dev->sm_count);
    const size_t need = L.rows + L.parts;
    if (!workspace || workspace_bytes < need) return OSF_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(workspace) & (L.ds + L.parts ? 127u : 3u)) != 0) return OSF_ERR_INVALID;
    char *at = static_cast<char *>(workspace);
    b.window = p.window;
    b.sinks = p.sinks;
    b.dvec = reinterpret_cast<float *>(at);
    b.shared_tiles = L.plan.shared_tiles;
    b.parts = L.plan.parts;
    b.part_keys = L.plan.part_keys;
    b.ds_slots = L.plan.slots;
    b.ds_ld = ((long long)Sq + 127) / 128 * 128;
    if (L.parts) b.part_acc = reinterpret_cast<float *>(at + L.rows);
    if (L.ds && workspace_bytes >= need + L.ds) b.ds = at + need;
    b.status = dev->status;
    return launch_status(launch_attn_bwd(b, (cudaStream_t)stream));
}

int osf_softmax_ex_workspace_bytes(long long rows, long long T, size_t *bytes) {
    if (!bytes) return OSF_ERR_INVALID;
    *bytes = 0;
    if (rows < 0 || T < 0) return OSF_ERR_INVALID;
    if (rows == 0 || T == 0) return OSF_OK;
    if (rows > 65535 && T > 32768) return OSF_ERR_UNSUPPORTED;
    DeviceInfo *dev;
    if (device_info(&dev) != OSF_OK) return OSF_ERR_CUDA;
    // the larger of the float32 path's and the general path's needs
    const size_t a = softmax_workspace_floats(rows, T, dev->sm_count);
    const size_t b = softmax_ex_workspace_floats(rows, T, dev->sm_count);
    *bytes = (a > b ? a : b) * sizeof(float);
    return OSF_OK;
}

int osf_softmax_rows_ex(const void *x, void *z, int x_dtype, int z_dtype, long long rows, long long T,
                        long long x_row_stride, long long z_row_stride, float scale, long long causal_period,
                        void *workspace, size_t workspace_bytes, osf_stream stream) {
    if ((x_dtype != OSF_F32 && x_dtype != OSF_BF16) || (z_dtype != OSF_F32 && z_dtype != OSF_BF16))
        return OSF_ERR_INVALID;
    if (rows < 0 || T < 0 || causal_period < 0 || x_row_stride < 0 || z_row_stride < 0) return OSF_ERR_INVALID;
    if (!(scale == scale) || scale == INFINITY || scale == -INFINITY) return OSF_ERR_INVALID;
    if (rows == 0 || T == 0) return OSF_OK;
    const long long xs = x_row_stride ? x_row_stride : T, zs = z_row_stride ? z_row_stride : T;
    if (xs < T || zs < T) return OSF_ERR_INVALID;   // rows may not overlap one another
    if (!x || !z) return OSF_ERR_INVALID;
    if (rows > (1LL << 31) - 1 || (rows > 65535 && T > 32768) || xs >= (1LL << 40) || zs >= (1LL << 40))
        return OSF_ERR_UNSUPPORTED;
    const size_t nx = (size_t)((rows - 1) * xs + T) * elem_size(x_dtype);
    const size_t nz = (size_t)((rows - 1) * zs + T) * elem_size(z_dtype);
    const bool in_place = x == (const void *)z && x_dtype == z_dtype && xs == zs;
    if (!in_place && overlaps(x, nx, z, nz)) return OSF_ERR_INVALID;
    const float sc = scale == 0.f ? 1.f : scale;
    DeviceInfo *dev;
    if (device_info(&dev) != OSF_OK) return OSF_ERR_CUDA;
    if (x_dtype == OSF_F32 && z_dtype == OSF_F32 && sc == 1.f && causal_period == 0 && xs == T && zs == T)
        return osf_softmax_rows(static_cast<const float *>(x), static_cast<float *>(z), rows, T, workspace,
                                workspace_bytes, stream);
    const size_t need = softmax_ex_workspace_floats(rows, T, dev->sm_count) * sizeof(float);
    if (need > 0 && (!workspace || workspace_bytes < need)) return OSF_ERR_WORKSPACE;
    SoftmaxExProblem q{x, z, x_dtype, z_dtype, rows, T, xs, zs, sc * kLog2e, causal_period, dev->sm_count,
                       dev->status};
    return launch_status(launch_softmax_ex(q, static_cast<float *>(workspace), (cudaStream_t)stream));
}

// ------------------------------------------------------------------ weights of keys
// Shared validation of osf_attn_key_weights; `strides`: NULL (contiguous) or Q, K x (b, h, s).
static int check_key_weights(const void *Q, const void *K, const float *lse, float *weights, int dtype, int B, int Hq,
                             int Hkv, int Sq, int Sk, int D, const long long *strides, int mask, float scale,
                             KeyWeightsProblem &w, bool &empty) {
    // the forward problem's checks, with V = K and an output that overlaps nothing
    AttnProblem p;
    long long st[12];
    if (strides) {
        for (int i = 0; i < 6; ++i) st[i] = strides[i];
        for (int i = 0; i < 3; ++i) st[6 + i] = strides[3 + i];
        st[9] = (long long)Hq * Sq * D;
        st[10] = (long long)Sq * D;
        st[11] = D;
    }
    empty = false;
    if (Sq == 0 && Sk > 0 && B > 0) {   // no rows: the weights are zero, so the sizes alone matter
        const int st0 = check_gqa_ex(K, K, K, reinterpret_cast<void *>(~uintptr_t(0) >> 8), dtype, B, Hq, Hkv, 1, Sk, D,
                                     nullptr, mask, scale, nullptr, p, empty);
        if (st0 != OSF_OK) return st0;
    } else {
        // the placeholder output lies above every address in use
        const int st0 = check_gqa_ex(Q, K, K, reinterpret_cast<void *>(~uintptr_t(0) >> 8), dtype, B, Hq, Hkv, Sq, Sk, D,
                                     strides ? st : nullptr, mask, scale, nullptr, p, empty);
        if (st0 != OSF_OK || empty) return st0;
        if (!lse) return OSF_ERR_INVALID;
    }
    if (!weights) return OSF_ERR_INVALID;
    // (kernels count keys in ints, up to the end of the last block of 64)
    if ((long long)B * Hkv > 65535 || Sk > INT_MAX - 63) return OSF_ERR_UNSUPPORTED;
    w = KeyWeightsProblem{};
    w.q = Q; w.k = K; w.lse = lse; w.w = weights;
    w.dtype = dtype; w.B = B; w.Hq = Hq; w.Hkv = Hkv; w.Sq = Sq; w.Sk = Sk; w.D = D;
    if (Sq == 0) return OSF_OK;
    w.causal = p.causal; w.causal_off = p.causal_off; w.scale_log2 = p.scale_log2;
    w.q_sb = p.q_sb; w.q_sh = p.q_sh; w.q_ss = p.q_ss;
    w.k_sb = p.k_sb; w.k_sh = p.k_sh; w.k_ss = p.k_ss;
    const size_t es = elem_size(dtype), nw = (size_t)B * Hkv * Sk * sizeof(float);
    if (overlaps(weights, nw, Q, span_bytes(B, Hq, Sq, D, w.q_sb, w.q_sh, w.q_ss, es)) ||
        overlaps(weights, nw, K, span_bytes(B, Hkv, Sk, D, w.k_sb, w.k_sh, w.k_ss, es)) ||
        overlaps(weights, nw, lse, (size_t)B * Hq * Sq * sizeof(float)))
        return OSF_ERR_INVALID;
    return OSF_OK;
}

// Which kernel runs a validated problem, and the bytes of partial sums it keeps in the workspace.
enum class WeightsPath { Rows, TensorCore, Simt };

static WeightsPath key_weights_path(const KeyWeightsProblem &w) {
    if (key_weights_rows_supported(w)) return WeightsPath::Rows;
    return key_weights_tc_supported(w) ? WeightsPath::TensorCore : WeightsPath::Simt;
}

static size_t key_weights_partial_bytes(KeyWeightsProblem w, WeightsPath path, int sm_count) {
    if (path == WeightsPath::Rows) return 0;
    if (path == WeightsPath::TensorCore) return align256(key_weights_tc_floats(sm_count) * sizeof(float));
    key_weights_simt_plan(w, sm_count);
    return w.splits > 1 ? align256((size_t)w.splits * w.B * w.Hkv * w.Sk * sizeof(float)) : 0;
}

int osf_attn_key_weights_workspace_bytes(int dtype, int B, int Hq, int Hkv, int Sq, int Sk, int D, size_t *bytes) {
    if (!bytes) return OSF_ERR_INVALID;
    *bytes = 0;
    KeyWeightsProblem w;
    bool empty;
    const void *ph = reinterpret_cast<const void *>(uintptr_t(1) << 40);
    // the larger of the possible paths' needs, over the masks (the call's mask and alignment decide then)
    size_t need = 0;
    for (int mask : {OSF_MASK_NONE, OSF_MASK_TOP_LEFT, OSF_MASK_BOTTOM_RIGHT}) {
        const int st = check_key_weights(ph, ph, static_cast<const float *>(ph), reinterpret_cast<float *>(uintptr_t(1) << 44),
                                         dtype, B, Hq, Hkv, Sq, Sk, D, nullptr, mask, 0.f, w, empty);
        if (st != OSF_OK || empty || Sq == 0) return st;
        DeviceInfo *dev;
        if (device_info(&dev) != OSF_OK) return OSF_ERR_CUDA;
        need = std::max(need, key_weights_partial_bytes(w, WeightsPath::Simt, dev->sm_count));
        if (dtype == OSF_BF16 && (D == 64 || D == 128))
            need = std::max(need, key_weights_partial_bytes(w, WeightsPath::TensorCore, dev->sm_count));
    }
    *bytes = need;
    return OSF_OK;
}

int osf_attn_key_weights(const void *Q, const void *K, const float *lse, float *weights, int dtype, int B, int Hq, int Hkv,
                         int Sq, int Sk, int D, const long long *strides, int mask, float scale, int accumulate,
                         void *workspace, size_t workspace_bytes, osf_stream stream) {
    KeyWeightsProblem w;
    bool empty;
    const int st = check_key_weights(Q, K, lse, weights, dtype, B, Hq, Hkv, Sq, Sk, D, strides, mask, scale, w, empty);
    if (st != OSF_OK || empty) return st;
    const cudaStream_t s = (cudaStream_t)stream;
    if (Sq == 0)
        return accumulate ? OSF_OK
                          : launch_status(cudaMemsetAsync(weights, 0, (size_t)B * Hkv * Sk * sizeof(float), s));
    DeviceInfo *dev;
    if (device_info(&dev) != OSF_OK) return OSF_ERR_CUDA;
    w.accumulate = accumulate != 0;
    w.status = dev->status;
    const WeightsPath path = key_weights_path(w);
    const size_t need = key_weights_partial_bytes(w, path, dev->sm_count);
    const int ws = check_workspace(workspace, workspace_bytes, need);
    if (ws != OSF_OK) return ws;
    w.part = static_cast<float *>(workspace);
    if (path == WeightsPath::Rows) return launch_status(launch_key_weights_rows(w, dev->sm_count, s));
    if (path == WeightsPath::TensorCore) return launch_status(launch_key_weights_tc(w, dev->sm_count, s));
    key_weights_simt_plan(w, dev->sm_count);
    cudaError_t e = launch_key_weights_simt(w, s);
    if (e == cudaSuccess && w.splits > 1) e = launch_key_weights_reduce(w, s);
    return launch_status(e);
}

// ------------------------------------------------------------------ 4-bit cache
int osf_kv4_record_bytes(int D, size_t *bytes) {
    if (!bytes) return OSF_ERR_INVALID;
    *bytes = 0;
    if (D <= 0) return OSF_ERR_INVALID;
    if (D > 256 || D % kKv4Group != 0) return OSF_ERR_UNSUPPORTED;
    *bytes = (size_t)kv4_record_bytes(D);
    return OSF_OK;
}

// Sizes shared by the calls on a cache [B, Hkv, S, record].
static int check_kv4(int dtype, int B, int Hkv, long long n, int S, int D) {
    if (dtype != OSF_F32 && dtype != OSF_BF16) return OSF_ERR_INVALID;
    if (B < 0 || Hkv <= 0 || n < 0 || S < 0) return OSF_ERR_INVALID;
    size_t rec;
    const int st = osf_kv4_record_bytes(D, &rec);
    if (st != OSF_OK) return st;
    if ((long long)B * Hkv > 65535 || (long long)n * D >= (1LL << 31) || (long long)S * D >= (1LL << 31))
        return OSF_ERR_UNSUPPORTED;
    return OSF_OK;
}

int osf_kv4_append(const void *K, const void *V, int dtype, int B, int Hkv, int n, int D, const long long *strides, void *cache,
                   int S, const int *lens, const int *counts, osf_stream stream) {
    const int st = check_kv4(dtype, B, Hkv, n, S, D);
    if (st != OSF_OK) return st;
    Kv4StoreProblem p{};
    long long sd[6] = {(long long)Hkv * n * D, (long long)n * D, D, (long long)Hkv * n * D, (long long)n * D, D};
    if (strides)
        for (int i = 0; i < 6; ++i) {
            if (strides[i] < 0) return OSF_ERR_INVALID;
            if (strides[i] >= (1LL << 40)) return OSF_ERR_UNSUPPORTED;
            sd[i] = strides[i];
        }
    if (B == 0 || n == 0) return OSF_OK;
    if (n > S && !counts) return OSF_ERR_INVALID;
    if (!K || !V || !cache || (reinterpret_cast<uintptr_t>(cache) & 15u) != 0) return OSF_ERR_INVALID;
    const size_t es = elem_size(dtype), nc = (size_t)B * Hkv * S * kv4_record_bytes(D);
    if (overlaps(cache, nc, K, span_bytes(B, Hkv, n, D, sd[0], sd[1], sd[2], es)) ||
        overlaps(cache, nc, V, span_bytes(B, Hkv, n, D, sd[3], sd[4], sd[5], es)) ||
        overlaps(cache, nc, lens, (size_t)B * 4) || overlaps(cache, nc, counts, (size_t)B * 4))
        return OSF_ERR_INVALID;
    DeviceInfo *dev;
    if (device_info(&dev) != OSF_OK) return OSF_ERR_CUDA;
    p.k = K; p.v = V; p.cache = static_cast<unsigned char *>(cache); p.lens = lens; p.counts = counts;
    p.dtype = dtype; p.B = B; p.Hkv = Hkv; p.n = n; p.S = S; p.D = D;
    p.k_sb = sd[0]; p.k_sh = sd[1]; p.k_ss = sd[2]; p.v_sb = sd[3]; p.v_sh = sd[4]; p.v_ss = sd[5];
    p.status = dev->status;
    return launch_status(launch_kv4_append(p, dev->sm_count, (cudaStream_t)stream));
}

int osf_kv4_read(const void *cache, void *K, void *V, int dtype, int B, int Hkv, int n, int D, int S, const int *starts,
                 const int *lens, osf_stream stream) {
    const int st = check_kv4(dtype, B, Hkv, n, S, D);
    if (st != OSF_OK) return st;
    if (B == 0 || n == 0) return OSF_OK;
    if (!K || !V || (!cache && S > 0) || (reinterpret_cast<uintptr_t>(cache) & 15u) != 0) return OSF_ERR_INVALID;
    const size_t no = (size_t)B * Hkv * n * D * elem_size(dtype), nc = (size_t)B * Hkv * S * kv4_record_bytes(D);
    if (overlaps(K, no, V, no) || overlaps(K, no, cache, nc) || overlaps(V, no, cache, nc) ||
        overlaps(K, no, lens, (size_t)B * 4) || overlaps(V, no, lens, (size_t)B * 4) ||
        overlaps(K, no, starts, (size_t)B * 4) || overlaps(V, no, starts, (size_t)B * 4))
        return OSF_ERR_INVALID;
    DeviceInfo *dev;
    if (device_info(&dev) != OSF_OK) return OSF_ERR_CUDA;
    Kv4StoreProblem p{};
    p.ko = K; p.vo = V; p.cache = static_cast<unsigned char *>(const_cast<void *>(cache)); p.lens = lens; p.starts = starts;
    p.dtype = dtype; p.B = B; p.Hkv = Hkv; p.n = n; p.S = S; p.D = D;
    p.status = dev->status;
    return launch_status(launch_kv4_read(p, dev->sm_count, (cudaStream_t)stream));
}

// Sizes and layout of an attention call over records; fills kp (without workspace pointers).
static int check_attn_kv4(const void *Q, const void *cache, void *O, int dtype, int B, int Hq, int Hkv, int Sq, int S, int D,
                          const long long *strides, const int *lens, int mask, float scale, float *lse, float *weights,
                          Kv4AttnProblem &kp, bool &empty) {
    empty = false;
    const int st = check_kv4(dtype, B, Hkv, 0, S, D);
    if (st != OSF_OK) return st;
    if (Hq <= 0 || Hq % Hkv != 0 || Sq < 0) return OSF_ERR_INVALID;
    if (mask != OSF_MASK_NONE && mask != OSF_MASK_BOTTOM_RIGHT) return OSF_ERR_INVALID;
    if (!(scale == scale)) return OSF_ERR_INVALID;
    long long sd[6] = {(long long)Hq * Sq * D, (long long)Sq * D, D, (long long)Hq * Sq * D, (long long)Sq * D, D};
    if (strides)
        for (int i = 0; i < 6; ++i) {
            if (strides[i] < 0) return OSF_ERR_INVALID;
            if (strides[i] >= (1LL << 40)) return OSF_ERR_UNSUPPORTED;
            sd[i] = strides[i];
        }
    // the query rows of one kv head number at most 2^15: one CTA column per few of them
    if ((long long)(Hq / Hkv) * Sq > (1LL << 15)) return OSF_ERR_UNSUPPORTED;
    if (B == 0 || Sq == 0) { empty = true; return OSF_OK; }
    if (!Q || !O || (!cache && S > 0) || (reinterpret_cast<uintptr_t>(cache) & 15u) != 0) return OSF_ERR_INVALID;
    if (!rows_disjoint(B, Hq, Sq, D, sd[3], sd[4], sd[5])) return OSF_ERR_INVALID;
    const size_t es = elem_size(dtype);
    const void *bufs[6] = {O, lse, weights, Q, cache, lens};
    const size_t size[6] = {span_bytes(B, Hq, Sq, D, sd[3], sd[4], sd[5], es), (size_t)B * Hq * Sq * sizeof(float),
                            (size_t)B * Hkv * S * sizeof(float), span_bytes(B, Hq, Sq, D, sd[0], sd[1], sd[2], es),
                            (size_t)B * Hkv * S * kv4_record_bytes(D), (size_t)B * sizeof(int)};
    for (int i = 0; i < 3; ++i)   // no output overlaps another buffer
        for (int j = i + 1; j < 6; ++j)
            if (overlaps(bufs[i], size[i], bufs[j], size[j])) return OSF_ERR_INVALID;
    kp = Kv4AttnProblem{};
    AttnProblem &p = kp.a;
    p.q = Q; p.o = O; p.lse = lse;
    p.dtype = dtype; p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.Sq = Sq; p.Sk = S; p.D = D;
    p.causal = mask == OSF_MASK_BOTTOM_RIGHT && Sq > 1;   // one row sees every valid key
    p.q_sb = sd[0]; p.q_sh = sd[1]; p.q_ss = sd[2]; p.o_sb = sd[3]; p.o_sh = sd[4]; p.o_ss = sd[5];
    p.scale_log2 = (scale > 0.f ? scale : 1.0f / sqrtf((float)D)) * kLog2e;
    p.splits = 1;
    kp.cache = static_cast<const unsigned char *>(cache);
    kp.lens = lens;
    kp.weights = weights;
    return OSF_OK;
}

// Workspace: split partial states | scores and the log-sum-exp, with weights.
static size_t kv4_lse_bytes(const Kv4AttnProblem &kp) { return align256((size_t)kp.a.B * kp.a.Hq * kp.a.Sq * sizeof(float)); }
static size_t kv4_scores_bytes(const Kv4AttnProblem &kp) {
    return align256((size_t)kp.a.B * kp.a.Hq * kp.a.Sq * kp.a.Sk * sizeof(float));
}
static size_t kv4_workspace(const Kv4AttnProblem &kp, int sm_count, bool weights) {
    return kv4_attn_partial_bytes(kp, sm_count) + (weights ? kv4_lse_bytes(kp) + kv4_scores_bytes(kp) : 0);
}

int osf_attn_kv4_workspace_bytes(int dtype, int B, int Hq, int Hkv, int Sq, int S, int D, int with_weights, size_t *bytes) {
    if (!bytes) return OSF_ERR_INVALID;
    *bytes = 0;
    Kv4AttnProblem kp;
    bool empty;
    const int st = check_attn_kv4(reinterpret_cast<const void *>(uintptr_t(1) << 40), reinterpret_cast<const void *>(uintptr_t(1) << 50),
                                  reinterpret_cast<void *>(uintptr_t(1) << 44), dtype, B, Hq, Hkv, Sq, S, D, nullptr, nullptr,
                                  OSF_MASK_NONE, 0.f, nullptr, nullptr, kp, empty);
    if (st != OSF_OK || empty) return st;
    DeviceInfo *dev;
    if (device_info(&dev) != OSF_OK) return OSF_ERR_CUDA;
    *bytes = kv4_workspace(kp, dev->sm_count, with_weights != 0);
    return OSF_OK;
}

int osf_attn_kv4(const void *Q, const void *cache, void *O, int dtype, int B, int Hq, int Hkv, int Sq, int S, int D,
                 const long long *strides, const int *lens, int mask, float scale, float *lse, float *weights, int accumulate,
                 void *workspace, size_t workspace_bytes, osf_stream stream) {
    Kv4AttnProblem kp;
    bool empty;
    const int st = check_attn_kv4(Q, cache, O, dtype, B, Hq, Hkv, Sq, S, D, strides, lens, mask, scale, lse, weights, kp, empty);
    if (st != OSF_OK || empty) return st;
    DeviceInfo *dev;
    if (device_info(&dev) != OSF_OK) return OSF_ERR_CUDA;
    AttnProblem &p = kp.a;
    p.status = dev->status;
    kp.accumulate = accumulate != 0;
    const size_t need = kv4_workspace(kp, dev->sm_count, weights != nullptr);
    const int ws = check_workspace(workspace, workspace_bytes, need);
    if (ws != OSF_OK) return ws;
    if (weights) {
        char *at = static_cast<char *>(workspace) + kv4_attn_partial_bytes(kp, dev->sm_count);
        if (!p.lse) p.lse = reinterpret_cast<float *>(at);
        kp.scores = reinterpret_cast<float *>(at + kv4_lse_bytes(kp));
    }
    return launch_status(launch_attn_kv4(kp, workspace, dev->sm_count, (cudaStream_t)stream));
}

// ------------------------------------------------------------------ paged 8-bit cache
// Sizes and buffers shared by the calls on a paged cache.
static int check_kv8(const void *pages, const float *scales, int n_pages, int page_tokens, const int *table, int per_seq,
                     int dtype, int B, int Hkv, long long n, int D, Kv8Cache &c) {
    if (dtype != OSF_F32 && dtype != OSF_BF16) return OSF_ERR_INVALID;
    if (B < 0 || Hkv <= 0 || n < 0 || D <= 0 || n_pages < 0 || per_seq < 0 || page_tokens <= 0) return OSF_ERR_INVALID;
    if (D > 256 || D % 32 != 0) return OSF_ERR_UNSUPPORTED;
    if (page_tokens != 16 && page_tokens != 32 && page_tokens != 64 && page_tokens != 128) return OSF_ERR_UNSUPPORTED;
    if ((long long)B * Hkv > 65535 || n * D >= (1LL << 31) || (long long)per_seq * page_tokens >= (1LL << 29))
        return OSF_ERR_UNSUPPORTED;
    if ((long long)n_pages * 2 * Hkv * page_tokens >= (1LL << 31)) return OSF_ERR_UNSUPPORTED;   // rows of the pages
    c.pages = static_cast<unsigned char *>(const_cast<void *>(pages));
    c.scales = const_cast<float *>(scales);
    c.table = table;
    c.n_pages = n_pages; c.P = page_tokens; c.log2_p = 31 - __builtin_clz(page_tokens); c.per_seq = per_seq; c.Hkv = Hkv; c.D = D;
    return OSF_OK;
}
static int check_kv8_buffers(const Kv8Cache &c, int B) {
    if ((c.n_pages > 0 && (!c.pages || !c.scales)) || (B > 0 && c.per_seq > 0 && !c.table)) return OSF_ERR_INVALID;
    if (misaligned(c.scales, 4) || misaligned(c.table, 4)) return OSF_ERR_INVALID;
    return (reinterpret_cast<uintptr_t>(c.pages) & 15u) != 0 ? OSF_ERR_INVALID : OSF_OK;
}
// The cache's three buffers, for the checks of overlaps.
struct Kv8Buffers {
    const void *at[3];
    size_t size[3];
};
static Kv8Buffers kv8_buffers(const Kv8Cache &c, int B) {
    const size_t heads = (size_t)c.n_pages * 2 * c.Hkv;
    return {{c.pages, c.scales, c.table}, {heads * c.P * c.D, heads * sizeof(float), (size_t)B * c.per_seq * sizeof(int)}};
}
// `count` element strides into st, or the contiguous ones of [B, H, n, D] for each three.
static int take_strides(const long long *strides, int count, const int *H, long long n, int D, long long *st) {
    for (int i = 0; i < count; ++i) {
        const long long h = H[i / 3];
        st[i] = strides ? strides[i] : i % 3 == 0 ? h * n * D : i % 3 == 1 ? n * D : D;
        if (st[i] < 0) return OSF_ERR_INVALID;
        if (st[i] >= (1LL << 40)) return OSF_ERR_UNSUPPORTED;
    }
    return OSF_OK;
}

int osf_kv8_append(const void *K, const void *V, int dtype, int B, int Hkv, int n, int D, const long long *strides, void *pages,
                   float *scales, int n_pages, int page_tokens, const int *table, int table_len, const int *lens,
                   const int *counts, const float *cos_table, const float *sin_table, int max_positions, int rotary_dim,
                   int interleaved, const void *Q, void *Q_out, int Hq, osf_stream stream) {
    Kv8StoreProblem p{};
    Kv8Cache &c = p.c;
    int st = check_kv8(pages, scales, n_pages, page_tokens, table, table_len, dtype, B, Hkv, n, D, c);
    if (st != OSF_OK) return st;
    if (rotary_dim < 0 || rotary_dim > D || max_positions < 0) return OSF_ERR_INVALID;
    if (rotary_dim % 8 != 0) return OSF_ERR_UNSUPPORTED;
    if ((Q == nullptr) != (Q_out == nullptr)) return OSF_ERR_INVALID;
    if (Q && (Hq <= 0 || Hq % Hkv != 0)) return OSF_ERR_INVALID;
    if (Q && (long long)B * Hq > 65535) return OSF_ERR_UNSUPPORTED;
    const int heads[4] = {Hkv, Hkv, Hq, Hq};
    long long sd[12];
    st = take_strides(strides, Q ? 12 : 6, heads, n, D, sd);
    if (st != OSF_OK) return st;
    if (B == 0 || n == 0) return OSF_OK;
    if (!K || !V || (rotary_dim > 0 && (!cos_table || !sin_table || max_positions == 0))) return OSF_ERR_INVALID;
    st = check_kv8_buffers(c, B);
    if (st != OSF_OK) return st;
    if ((long long)table_len * page_tokens < n && !counts) return OSF_ERR_INVALID;
    const size_t es = elem_size(dtype);
    if (misaligned(K, es) || misaligned(V, es) || misaligned(Q, es) || misaligned(Q_out, es) || misaligned(lens, 4) ||
        misaligned(counts, 4) || misaligned(cos_table, 4) || misaligned(sin_table, 4))
        return OSF_ERR_INVALID;
    const size_t nt = (size_t)max_positions * (rotary_dim / 2) * sizeof(float);
    const size_t nk = span_bytes(B, Hkv, n, D, sd[0], sd[1], sd[2], es), nv = span_bytes(B, Hkv, n, D, sd[3], sd[4], sd[5], es);
    const size_t nq = Q ? span_bytes(B, Hq, n, D, sd[6], sd[7], sd[8], es) : 0;
    const size_t no = Q ? span_bytes(B, Hq, n, D, sd[9], sd[10], sd[11], es) : 0;
    const Kv8Buffers cb = kv8_buffers(c, B);
    // written: pages, scales, Q_out; read: the others
    const void *in[8] = {K, V, lens, counts, rotary_dim ? cos_table : nullptr, rotary_dim ? sin_table : nullptr, table, Q};
    const size_t in_n[8] = {nk, nv, (size_t)B * 4, (size_t)B * 4, nt, nt, cb.size[2], nq};
    const void *out[3] = {pages, scales, Q_out};
    const size_t out_n[3] = {cb.size[0], cb.size[1], no};
    const bool in_place = Q && Q == Q_out && sd[6] == sd[9] && sd[7] == sd[10] && sd[8] == sd[11];
    for (int o = 0; o < 3; ++o) {
        for (int i = 0; i < 8; ++i)
            if (!(o == 2 && i == 7 && in_place) && overlaps(out[o], out_n[o], in[i], in_n[i])) return OSF_ERR_INVALID;
        for (int o2 = o + 1; o2 < 3; ++o2)
            if (overlaps(out[o], out_n[o], out[o2], out_n[o2])) return OSF_ERR_INVALID;
    }
    if (Q && !rows_disjoint(B, Hq, n, D, sd[9], sd[10], sd[11])) return OSF_ERR_INVALID;
    if (n_pages == 0 || table_len == 0) return OSF_ERR_INVALID;   // nowhere to put the tokens
    DeviceInfo *dev;
    if (device_info(&dev) != OSF_OK) return OSF_ERR_CUDA;
    p.k = K; p.v = V; p.q = Q; p.qo = Q_out; p.lens = lens; p.counts = counts;
    p.cos = cos_table; p.sin = sin_table; p.max_pos = rotary_dim ? max_positions : INT_MAX; p.R = rotary_dim;
    p.interleaved = interleaved != 0;
    p.dtype = dtype; p.B = B; p.Hq = Hq; p.n = n;
    p.k_sb = sd[0]; p.k_sh = sd[1]; p.k_ss = sd[2]; p.v_sb = sd[3]; p.v_sh = sd[4]; p.v_ss = sd[5];
    if (Q) {
        p.q_sb = sd[6]; p.q_sh = sd[7]; p.q_ss = sd[8]; p.o_sb = sd[9]; p.o_sh = sd[10]; p.o_ss = sd[11];
    }
    p.status = dev->status;
    return launch_status(launch_kv8_append(p, dev->sm_count, (cudaStream_t)stream));
}

int osf_kv8_read(const void *pages, const float *scales, int n_pages, int page_tokens, const int *table, int table_len, void *K,
                 void *V, int dtype, int B, int Hkv, int n, int D, const int *starts, const int *lens, osf_stream stream) {
    Kv8StoreProblem p{};
    int st = check_kv8(pages, scales, n_pages, page_tokens, table, table_len, dtype, B, Hkv, n, D, p.c);
    if (st != OSF_OK) return st;
    if (B == 0 || n == 0) return OSF_OK;
    if (!K || !V) return OSF_ERR_INVALID;
    st = check_kv8_buffers(p.c, B);
    if (st != OSF_OK) return st;
    const size_t es = elem_size(dtype), no = (size_t)B * Hkv * n * D * es;
    if (misaligned(K, es) || misaligned(V, es) || misaligned(starts, 4) || misaligned(lens, 4)) return OSF_ERR_INVALID;
    const Kv8Buffers cb = kv8_buffers(p.c, B);
    const void *in[5] = {cb.at[0], cb.at[1], cb.at[2], starts, lens};
    const size_t in_n[5] = {cb.size[0], cb.size[1], cb.size[2], (size_t)B * 4, (size_t)B * 4};
    if (overlaps(K, no, V, no)) return OSF_ERR_INVALID;
    for (int i = 0; i < 5; ++i)
        if (overlaps(K, no, in[i], in_n[i]) || overlaps(V, no, in[i], in_n[i])) return OSF_ERR_INVALID;
    DeviceInfo *dev;
    if (device_info(&dev) != OSF_OK) return OSF_ERR_CUDA;
    p.ko = K; p.vo = V; p.lens = lens; p.starts = starts;
    p.dtype = dtype; p.B = B; p.n = n;
    p.status = dev->status;
    return launch_status(launch_kv8_read(p, dev->sm_count, (cudaStream_t)stream));
}

// Sizes and layout of an attention call over pages; fills kp (without workspace pointers).
static int check_attn_kv8(const void *Q, const void *pages, const float *scales, void *O, int dtype, int B, int Hq, int Hkv,
                          int Sq, int n_pages, int page_tokens, int D, const long long *strides, const int *table, int table_len,
                          const int *lens, int window, int sinks, float scale, float *lse, Kv8AttnProblem &kp, bool &empty) {
    empty = false;
    kp = Kv8AttnProblem{};
    int st = check_kv8(pages, scales, n_pages, page_tokens, table, table_len, dtype, B, Hkv, Sq, D, kp.c);
    if (st != OSF_OK) return st;
    if (Hq <= 0 || Hq % Hkv != 0 || window < 0 || sinks < 0 || !(scale == scale)) return OSF_ERR_INVALID;
    const int heads[2] = {Hq, Hq};
    long long sd[6];
    st = take_strides(strides, 6, heads, Sq, D, sd);
    if (st != OSF_OK) return st;
    // the query rows of one kv head number at most 2^15: one CTA column per few of them
    if ((long long)(Hq / Hkv) * Sq > (1LL << 15)) return OSF_ERR_UNSUPPORTED;
    if (B == 0 || Sq == 0) { empty = true; return OSF_OK; }
    if (!Q || !O) return OSF_ERR_INVALID;
    st = check_kv8_buffers(kp.c, B);
    if (st != OSF_OK) return st;
    if (!rows_disjoint(B, Hq, Sq, D, sd[3], sd[4], sd[5])) return OSF_ERR_INVALID;
    const size_t es = elem_size(dtype);
    if (misaligned(Q, es) || misaligned(O, es) || misaligned(lse, 4) || misaligned(lens, 4)) return OSF_ERR_INVALID;
    const Kv8Buffers cb = kv8_buffers(kp.c, B);
    const void *bufs[7] = {O, lse, Q, cb.at[0], cb.at[1], cb.at[2], lens};
    const size_t size[7] = {span_bytes(B, Hq, Sq, D, sd[3], sd[4], sd[5], es), (size_t)B * Hq * Sq * sizeof(float),
                            span_bytes(B, Hq, Sq, D, sd[0], sd[1], sd[2], es), cb.size[0], cb.size[1], cb.size[2],
                            (size_t)B * sizeof(int)};
    for (int i = 0; i < 2; ++i)   // no output overlaps another buffer
        for (int j = i + 1; j < 7; ++j)
            if (overlaps(bufs[i], size[i], bufs[j], size[j])) return OSF_ERR_INVALID;
    AttnProblem &p = kp.a;
    p.q = Q; p.o = O; p.lse = lse;
    p.dtype = dtype; p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.Sq = Sq; p.Sk = n_pages > 0 ? table_len * page_tokens : 0; p.D = D;
    p.causal = 1;
    // a window that hides nothing of the longest sequence is none
    if (window > 0 && (long long)window + sinks < p.Sk) {
        p.window = window;
        p.sinks = sinks;
    }
    p.q_sb = sd[0]; p.q_sh = sd[1]; p.q_ss = sd[2]; p.o_sb = sd[3]; p.o_sh = sd[4]; p.o_ss = sd[5];
    p.scale_log2 = (scale > 0.f ? scale : 1.0f / sqrtf((float)D)) * kLog2e;
    p.splits = 1;
    kp.lens = lens;
    return OSF_OK;
}

int osf_attn_kv8_workspace_bytes(int dtype, int B, int Hq, int Hkv, int Sq, int D, int page_tokens, int table_len, int window,
                                 int sinks, size_t *bytes) {
    if (!bytes) return OSF_ERR_INVALID;
    *bytes = 0;
    Kv8AttnProblem kp;
    bool empty;
    // (placeholder addresses, far from one another)
    auto at = [](int i) { return reinterpret_cast<char *>(uintptr_t(i) << 44); };
    const int st = check_attn_kv8(at(1), at(2), reinterpret_cast<const float *>(at(3)), at(4), dtype, B, Hq, Hkv, Sq, 1, page_tokens,
                                  D, nullptr, reinterpret_cast<const int *>(at(5)), table_len, nullptr, window, sinks, 0.f, nullptr,
                                  kp, empty);
    if (st != OSF_OK || empty) return st;
    DeviceInfo *dev;
    if (device_info(&dev) != OSF_OK) return OSF_ERR_CUDA;
    *bytes = kv8_attn_partial_bytes(kp, dev->sm_count);
    return OSF_OK;
}

int osf_attn_kv8(const void *Q, const void *pages, const float *scales, void *O, int dtype, int B, int Hq, int Hkv, int Sq,
                 int n_pages, int page_tokens, int D, const long long *strides, const int *table, int table_len, const int *lens,
                 int window, int sinks, float scale, float *lse, void *workspace, size_t workspace_bytes, osf_stream stream) {
    Kv8AttnProblem kp;
    bool empty;
    const int st = check_attn_kv8(Q, pages, scales, O, dtype, B, Hq, Hkv, Sq, n_pages, page_tokens, D, strides, table, table_len,
                                  lens, window, sinks, scale, lse, kp, empty);
    if (st != OSF_OK || empty) return st;
    DeviceInfo *dev;
    if (device_info(&dev) != OSF_OK) return OSF_ERR_CUDA;
    kp.a.status = dev->status;
    const int ws = check_workspace(workspace, workspace_bytes, kv8_attn_partial_bytes(kp, dev->sm_count));
    if (ws != OSF_OK) return ws;
    return launch_status(launch_attn_kv8(kp, workspace, dev->sm_count, (cudaStream_t)stream));
}

// ------------------------------------------------------------------ eviction
int osf_kv_evict(const void *src0, void *dst0, long long row_bytes0, const void *src1, void *dst1, long long row_bytes1,
                 const float *weights, float *weights_out, const int *lens, int *lens_out, int *idx, int B, int Hkv, int S,
                 int S_out, int budget, int sinks, int recent, osf_stream stream) {
    if (B < 0 || Hkv <= 0 || S < 0 || budget < 1 || sinks < 0 || recent < 0 || S_out < budget) return OSF_ERR_INVALID;
    if ((long long)sinks + recent > budget) return OSF_ERR_INVALID;
    if ((src0 && row_bytes0 < 1) || (src1 && row_bytes1 < 1)) return OSF_ERR_INVALID;
    // (an array of no keys may have no address)
    if ((src0 && !dst0) || (!src0 && dst0 && S > 0) || (src1 && !dst1) || (!src1 && dst1 && S > 0)) return OSF_ERR_INVALID;
    if ((long long)B * Hkv > 65535 || S >= (1 << 30) || S_out >= (1 << 30)) return OSF_ERR_UNSUPPORTED;
    if ((src0 && row_bytes0 * budget >= (1LL << 31)) || (src1 && row_bytes1 * budget >= (1LL << 31))) return OSF_ERR_UNSUPPORTED;
    if (B == 0) return OSF_OK;
    if ((!weights && S > 0) || !weights_out || !idx) return OSF_ERR_INVALID;
    const size_t heads = (size_t)B * Hkv;
    // buffers read | buffers written; a pair that is the same buffer with the same row count is moved in place
    const void *in[4] = {src0, src1, weights, lens};
    const size_t in_n[4] = {heads * S * (src0 ? row_bytes0 : 0), heads * S * (src1 ? row_bytes1 : 0), heads * S * 4, (size_t)B * 4};
    void *out[5] = {dst0, dst1, weights_out, lens_out, idx};
    const size_t out_n[5] = {heads * S_out * (dst0 ? row_bytes0 : 0), heads * S_out * (dst1 ? row_bytes1 : 0), heads * S_out * 4,
                             (size_t)B * 4, heads * budget * 4};
    for (int o = 0; o < 5; ++o) {
        for (int i = 0; i < 4; ++i) {
            const bool in_place = o == i && in[i] == out[o] && (o == 3 || S == S_out);
            if (!in_place && overlaps(out[o], out_n[o], in[i], in_n[i])) return OSF_ERR_INVALID;
        }
        for (int o2 = o + 1; o2 < 5; ++o2)
            if (overlaps(out[o], out_n[o], out[o2], out_n[o2])) return OSF_ERR_INVALID;
    }
    DeviceInfo *dev;
    if (device_info(&dev) != OSF_OK) return OSF_ERR_CUDA;
    EvictProblem p{};
    p.w = weights; p.w_out = weights_out; p.lens = lens; p.lens_out = lens_out; p.idx = idx;
    p.src[0] = static_cast<const unsigned char *>(src0); p.dst[0] = static_cast<unsigned char *>(dst0); p.row_bytes[0] = row_bytes0;
    p.src[1] = static_cast<const unsigned char *>(src1); p.dst[1] = static_cast<unsigned char *>(dst1); p.row_bytes[1] = row_bytes1;
    p.B = B; p.Hkv = Hkv; p.S = S; p.S_out = S_out; p.budget = budget; p.sinks = sinks; p.recent = recent;
    p.status = dev->status;
    return launch_status(launch_kv_evict(p, dev->sm_count, (cudaStream_t)stream));
}

int osf_selftest_bounded_wait(unsigned long long limit_ns, osf_stream stream) {
    if (limit_ns == 0 || limit_ns > 2000000000ull) return OSF_ERR_INVALID;
    DeviceInfo *dev;
    if (device_info(&dev) != OSF_OK) return OSF_ERR_CUDA;
    return launch_status(launch_bounded_wait_selftest(limit_ns, dev->status, (cudaStream_t)stream));
}

int osf_device_status(osf_stream stream) {
    DeviceInfo *dev;
    if (device_info(&dev) != OSF_OK) return OSF_ERR_CUDA;
    if (cudaStreamSynchronize((cudaStream_t)stream) != cudaSuccess) return OSF_ERR_CUDA;
    int word = 0;
    if (cudaMemcpyFromSymbol(&word, g_status_word, sizeof(int)) != cudaSuccess) return OSF_ERR_CUDA;
    if (word != 0) {
        const int zero = 0;
        if (cudaMemcpyToSymbol(g_status_word, &zero, sizeof(int)) != cudaSuccess) return OSF_ERR_CUDA;
    }
    return word;
}

}  // extern "C"
