// Attention backward (dQ, dK, dV from Q, K, V, O, dO and the saved log-sum-exp).
#pragma once
#include "osf_internal.cuh"

namespace osf {
struct BwdProblem {
    const void *q, *k, *v, *o, *dout;
    const float *lse;      // [B, Hq, Sq] natural-log log-sum-exp of the forward pass
    void *dq, *dk, *dv;
    int dtype;             // OSF_F32 / OSF_BF16
    int B, Hq, Hkv, Sq, Sk, D;
    int causal, causal_off;  // key j visible to row i iff !causal || j <= i + causal_off
    // 0, or (with causal = 1, causal_off = Sk - Sq): of those keys only j > i + causal_off - window or j < sinks
    int window, sinks;
    float scale, scale_log2;
    float *dvec;           // workspace [B, Hq, Sq]: rowsum(dO * O)
    // optional workspace (tensor-core path): dS^T as bf16 [128 x 128] tiles, tile (bh, key tile,
    // query tile) at ((bh * ds_rows / 128 + key tile) * ds_ld / 128 + query tile) * 32 KB, each
    // [128 keys][128 queries]; ds_rows and ds_ld the key and query counts rounded up to 128.
    // null: dQ recomputes S and dP instead
    // With a window only the tiles that some row sees: that of query tile t and place s of its key_stream at
    // (bh * (ds_ld / 128) + t) * ds_slots + s
    void *ds;
    long long ds_rows, ds_ld;
    int ds_slots;
    // with a window: the steps (query head, query tile) of each of the first shared_tiles tiles of part_keys keys are shared out
    // over `parts` CTAs, whose sums of dK and dV (float32 [part_keys][D] each) meet in part_acc [tile][part][b, kv head][2]
    int shared_tiles, parts, part_keys;
    float *part_acc;
    int *status;
};
// True when the bf16 tensor-core (mma.sync) kernels handle the problem.
bool attn_bwd_mma_supported(const BwdProblem &p);
cudaError_t launch_attn_bwd(const BwdProblem &p, cudaStream_t s);

// How a windowed problem runs on the tensor-core path, and on the CUDA cores.
struct BwdWindowPlan {
    int shared_tiles, parts, part_keys;
    int slots;                 // tensor cores: tiles of the longest key stream,
    bool store_ds;             // and dQ as a product over stored dS^T tiles
};
BwdWindowPlan bwd_window_plan(int B, int Hq, int Hkv, int Sq, int Sk, int window, int sinks, int sm_count);
BwdWindowPlan bwd_rows_plan(int B, int Hq, int Hkv, int Sq, int Sk, int D, int window, int sinks, int sm_count);
}  // namespace osf
