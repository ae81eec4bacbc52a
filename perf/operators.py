"""Cases and plain forms of the cache operators: the 4-bit K/V cache (store and read back, attention over
it), the attention weight that every key has accumulated, and eviction by that weight.

``listed()`` and ``draw()`` give cases, ``prepare()`` the tensors a program holds before the call, ``run()``
one call: elementary torch operations while ``own`` is false, the library's entry points while it is true.

A 4-bit record holds K and V of one token of one kv head in 1.25 D bytes: K codes (D/2 bytes), V codes (D/2),
then the (scale, minimum) bfloat16 pairs of K's groups of 32 channels and of V's.  The eight codes of channels
8w .. 8w+7 fill a 32-bit word (channel 8w+i in bits 4i .. 4i+3), and word w is the row's word number
(w % 4) * (D / 32) + w // 4.  A code c stands for minimum + scale * c.
"""
import math

import numpy as np
import torch

own = False

GROUP = 32


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # the weights that a prompt's own queries leave on its keys: the causal prefill of the benchmark
        dict(name="weights_prefill_4096", op="weights", dtype="bf16", B=2, Hq=32, Hkv=8, Sq=4096, Sk=4096, D=128,
             mask="top_left"),
        # a ragged chunk of new rows behind a cache
        dict(name="weights_chunk_ragged", op="weights", dtype="bf16", B=3, Hq=12, Hkv=4, Sq=333, Sk=1999, D=64,
             mask="bottom_right"),
        # one decode step over the benchmark's bf16 cache
        dict(name="weights_decode_32k", op="weights", dtype="bf16", B=8, Hq=32, Hkv=8, Sq=1, Sk=32768, D=128,
             mask="none"),
        # float32 attention, an odd length
        dict(name="weights_f32_1001", op="weights", dtype="f32", B=1, Hq=8, Hkv=2, Sq=1001, Sk=1001, D=64,
             mask="top_left"),
        # a batch of long prompts cut to a quarter of its keys before decoding starts
        dict(name="evict_32k_to_8k", op="evict", rows="bf16", B=8, Hkv=8, S=32768, D=128, budget=8192, sinks=4,
             recent=1024, ragged=False),
        # one short sequence: what the call costs at least
        dict(name="evict_1237_to_600", op="evict", rows="bf16", B=1, Hkv=8, S=1237, D=64, budget=600, sinks=4,
             recent=64, ragged=False),
        # 4-bit records of long contexts of different lengths
        dict(name="evict_records_128k", op="evict", rows="kv4", B=2, Hkv=8, S=131072, D=128, budget=16384, sinks=16,
             recent=2048, ragged=True),
        # the new token of every sequence of a decode batch
        dict(name="store_token_b32", op="store", dtype="bf16", B=32, Hkv=8, n=1, S=1024, D=128, ragged=True),
        # a batch of whole prompts
        dict(name="store_prompt_4096", op="store", dtype="bf16", B=8, Hkv=8, n=4096, S=4096, D=128, ragged=False),
        # the benchmark's decode step, over 4-bit records
        dict(name="attn_decode_32k", op="attn", dtype="bf16", B=8, Hq=32, Hkv=8, Sq=1, S=32768, D=128, ragged=False,
             mask="none", weights=False),
        # one short sequence: latency
        dict(name="attn_decode_500", op="attn", dtype="bf16", B=1, Hq=16, Hkv=8, Sq=1, S=500, D=128, ragged=False,
             mask="none", weights=False),
        # four draft tokens over sequences of different lengths, with the weights for a later eviction
        dict(name="attn_draft_ragged_8k", op="attn", dtype="bf16", B=16, Hq=32, Hkv=8, Sq=4, S=8192, D=64, ragged=True,
             mask="bottom_right", weights=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["weights", "weights", "evict", "store", "attn", "attn"])
    D = rng.choice([64, 128, 128, 96])
    Hkv, G = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 3, 4, 5, 8])
    while True:
        B = rng.choice([1, 2, 3, 5, 8, 13])
        if op == "weights":
            kind = rng.choice(["prompt", "chunk", "decode"])
            dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
            Sk = _log(rng, 64, 32768 if kind == "decode" else 4096)
            Sq = Sk if kind == "prompt" else rng.randint(1, 4) if kind == "decode" else max(1, _log(rng, 8, 1024) % Sk)
            mask = "top_left" if kind == "prompt" else "bottom_right"
            # the CUDA-core path (float32, or a head dimension other than 64 and 128) gets less work
            slow = dtype == "f32" or D == 96
            if B * Hkv * G * Sq * Sk * D > (2e9 if slow else 1.3e11) or B * Hkv * Sk * D > (1 << 27 if slow else 1 << 28):
                continue
            return dict(op=op, dtype=dtype, B=B, Hq=Hkv * G, Hkv=Hkv, Sq=Sq, Sk=Sk, D=D, mask=mask)
        if op == "evict":
            rows = rng.choice(["bf16", "kv4"])
            S = _log(rng, 300, 131072)
            budget = max(32, int(S * rng.uniform(0.1, 0.8)))
            recent, sinks = int(budget * rng.uniform(0, 0.5)), rng.choice([0, 1, 4, 16])
            if B * Hkv * S * D > 1 << 28:
                continue
            return dict(op=op, rows=rows, B=B, Hkv=Hkv, S=S, D=D, budget=budget, sinks=sinks, recent=recent,
                        ragged=rng.random() < 0.5)
        if op == "store":
            n = 1 if rng.random() < 0.4 else _log(rng, 2, 8192)
            S = n + rng.randint(0, 1000)
            if B * Hkv * S * D > 1 << 25:
                continue
            return dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), B=B, Hkv=Hkv, n=n, S=S, D=D, ragged=True)
        Sq, dtype = rng.choice([1, 1, 1, 2, 4, 5]), rng.choice(["bf16", "bf16", "bf16", "f32"])
        S = _log(rng, 48, 32768)
        slow = dtype == "f32" or D == 96
        if B * Hkv * S * D > (1 << 24 if slow else 1 << 28):
            continue
        return dict(op=op, dtype=dtype, B=B, Hq=Hkv * G, Hkv=Hkv, Sq=Sq, S=S, D=D, ragged=rng.random() < 0.6,
                    mask="bottom_right", weights=rng.random() < 0.4)


# ------------------------------------------------------------------------------------------ inputs
def _dtype(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _rows(gen, B, H, S, D):
    """K or V rows [B, H, S, D]: normal values around an offset, with a width, of each channel."""
    wide = torch.rand(1, H, 1, D, generator=gen, device="cuda") + 0.5
    off = torch.randn(1, H, 1, D, generator=gen, device="cuda") * 0.5
    return torch.randn(B, H, S, D, generator=gen, device="cuda") * wide + off


def _lens(gen, B, S, ragged, least):
    if not ragged:
        return torch.full((B,), S, dtype=torch.int32, device="cuda")
    lens = torch.randint(least, S + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
    lens[0] = S
    return lens


def _quantise(x):
    """(codes, scale, minimum) of float64 x [..., D]: groups of 32 channels, codes 0 .. 15 in float64."""
    g = x.unflatten(-1, (-1, GROUP))
    lo, hi = g.amin(-1), g.amax(-1)
    # the nearest bfloat16 at or below the minimum
    m = lo.to(torch.bfloat16)
    m = torch.where(m.double() > lo, torch.nextafter(m, torch.full_like(m, -math.inf)), m)
    # the nearest bfloat16 at or above a fifteenth of the range
    r = (hi - m.double()) / 15
    s = r.to(torch.bfloat16)
    s = torch.where(15 * s.double() < hi - m.double(), torch.nextafter(s, torch.full_like(s, math.inf)), s)
    step = torch.where(s == 0, torch.ones_like(s), s).double()
    codes = torch.round((g - m.double().unsqueeze(-1)) / step.unsqueeze(-1))
    return codes, s, m


def _words(codes, D):
    """Codes [..., D/32, 32] as the D/8 int32 words of a record's half, in record order."""
    c = codes.to(torch.int64).flatten(-2).unflatten(-1, (-1, 8))
    w = (c << (4 * torch.arange(8, device=c.device))).sum(-1)
    w = torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)
    return w.unflatten(-1, (D // 32, 4)).transpose(-1, -2).flatten(-2).contiguous()


def _records(k, v):
    """The 4-bit records, uint8 [B, H, S, 1.25 D], of K and V rows."""
    parts, D = [], k.shape[-1]
    quantised = [_quantise(t.double()) for t in (k, v)]
    for codes, _, _ in quantised:
        parts.append(_words(codes, D).view(torch.uint8))
    for _, s, m in quantised:
        parts.append(torch.stack([s, m], -1).flatten(-2).contiguous().view(torch.uint8))
    return torch.cat(parts, -1).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, B, Hkv, D = case["op"], case["B"], case["Hkv"], case["D"]
    st = dict(case)
    if op == "weights":
        dt = _dtype(case["dtype"])
        Hq, Sq, Sk = case["Hq"], case["Sq"], case["Sk"]
        st["q"] = torch.randn(B, Hq, Sq, D, generator=gen, device="cuda").to(dt)
        st["k"] = _rows(gen, B, Hkv, Sk, D).to(dt)
        st["scale"] = D ** -0.5
        # the forward pass's log-sum-exp of each row
        st["lse"] = torch.logsumexp(_scores(st["q"].float(), st["k"].float(), case["mask"], st["scale"]), -1).contiguous()
        st["w"] = torch.empty(B, Hkv, Sk, device="cuda")
    elif op == "evict":
        S, budget = case["S"], case["budget"]
        st["lens"] = _lens(gen, B, S, case["ragged"], min(S, budget // 2))
        # accumulated weights: heavy-tailed, with many keys that never got any
        w = torch.rand(B, Hkv, S, generator=gen, device="cuda").pow(6) * 8
        st["w"] = torch.where(torch.rand(B, Hkv, S, generator=gen, device="cuda") < 0.2, torch.zeros_like(w), w)
        if case["rows"] == "bf16":
            make = lambda s: torch.randn(B, Hkv, s, D, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
            st["k"], st["v"] = make(S), make(S)
            st["k_out"], st["v_out"] = torch.zeros_like(st["k"][:, :, :budget]), torch.zeros_like(st["v"][:, :, :budget])
            st["k_out"], st["v_out"] = st["k_out"].contiguous(), st["v_out"].contiguous()
        else:
            R = D + D // 4
            st["k"] = torch.randint(0, 256, (B, Hkv, S, R), generator=gen, device="cuda", dtype=torch.uint8)
            st["k_out"] = torch.zeros(B, Hkv, budget, R, dtype=torch.uint8, device="cuda")
            st["v"] = st["v_out"] = None
        st["w_out"] = torch.empty(B, Hkv, budget, device="cuda")
        st["lens_out"] = torch.empty(B, dtype=torch.int32, device="cuda")
        st["idx"] = torch.empty(B, Hkv, budget, dtype=torch.int32, device="cuda")
    elif op == "store":
        dt, n, S = _dtype(case["dtype"]), case["n"], case["S"]
        st["k"], st["v"] = _rows(gen, B, Hkv, n, D).to(dt), _rows(gen, B, Hkv, n, D).to(dt)
        st["cache"] = torch.zeros(B, Hkv, S, D + D // 4, dtype=torch.uint8, device="cuda")
        # the lengths before the call, and after it
        st["lens"] = torch.randint(0, S - n + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
        st["lens_after"] = st["lens"] + n
        st["k_out"], st["v_out"] = torch.empty_like(st["k"]), torch.empty_like(st["v"])
    else:
        dt, Hq, Sq, S = _dtype(case["dtype"]), case["Hq"], case["Sq"], case["S"]
        st["q"] = torch.randn(B, Hq, Sq, D, generator=gen, device="cuda").to(dt)
        st["cache"] = torch.cat([_records(_rows(gen, 1, Hkv, S, D), _rows(gen, 1, Hkv, S, D)) for _ in range(B)])
        st["lens"] = _lens(gen, B, S, case["ragged"], Sq)
        st["scale"] = D ** -0.5
        st["out"], st["lse"] = torch.empty_like(st["q"]), torch.empty(B, Hq, Sq, device="cuda")
        st["w"] = torch.empty(B, Hkv, S, device="cuda") if case["weights"] else None
    return st


# ------------------------------------------------------------------------------------------ plain forms
def _scores(q, k, mask, scale, lens=None):
    """Scaled, masked scores [B, Hkv, G * Sq, Sk] -> [B, Hq, Sq, Sk]; -inf where a row does not see a key."""
    B, Hq, Sq, D = q.shape
    Hkv, Sk = k.shape[1], k.shape[2]
    s = (q.reshape(B, Hkv, -1, D) @ k.transpose(-1, -2)).view(B, Hq, Sq, Sk) * scale
    j = torch.arange(Sk, device=q.device)
    i = torch.arange(Sq, device=q.device)[:, None]
    if lens is not None:
        n = lens.view(B, 1, 1, 1)
        last = n - Sq + i if mask == "bottom_right" else n - 1
        s.masked_fill_((j > last) | (j >= n), -math.inf)
    elif mask != "none":
        s.masked_fill_(j > i + (Sk - Sq if mask == "bottom_right" else 0), -math.inf)
    return s


def _values(cache, D, half):
    """The float32 values [B, H, S, D] that one half (0: K, 1: V) of the records stands for."""
    w = cache[..., half * D // 2:(half + 1) * D // 2].contiguous().view(torch.int32)
    w = w.unflatten(-1, (4, D // 32)).transpose(-1, -2).flatten(-2)
    codes = (w.unsqueeze(-1) >> (4 * torch.arange(8, device=w.device, dtype=torch.int32))) & 15
    at = D + half * (D // 8)
    sm = cache[..., at:at + D // 8].contiguous().view(torch.bfloat16).float().unflatten(-1, (-1, 2))
    codes = codes.flatten(-2).unflatten(-1, (-1, GROUP)).float()
    return (codes * sm[..., 0:1] + sm[..., 1:2]).flatten(-2)


def _plain_weights(st):
    s = _scores(st["q"].float(), st["k"].float(), st["mask"], st["scale"])
    p = torch.exp(s - st["lse"].unsqueeze(-1))
    return p.view(st["B"], st["Hkv"], -1, st["Sk"]).sum(2)


def _plain_evict(st):
    B, Hkv, S, budget, sinks, recent = (st[x] for x in ("B", "Hkv", "S", "budget", "sinks", "recent"))
    lens = st["lens"].view(B, 1, 1)
    j = torch.arange(S, device="cuda")
    kept_anyway = (j < sinks) | (j >= lens - recent) | (lens <= budget)
    rank = torch.where(kept_anyway, math.inf, st["w"])
    rank = torch.where(j < lens, rank, -math.inf)
    order = torch.sort(rank, dim=-1, descending=True, stable=True)[1][..., :budget]
    new = torch.minimum(lens, torch.full_like(lens, budget))
    slot = torch.arange(budget, device="cuda")
    idx = torch.sort(torch.where(slot < new, order, S), -1)[0]
    live = slot < new
    at = torch.where(live, idx, 0)
    take = lambda x: torch.where(live.unsqueeze(-1), x.gather(2, at.unsqueeze(-1).expand(-1, -1, -1, x.shape[-1])), torch.zeros((), dtype=x.dtype, device="cuda"))  # noqa: E731
    k, v = take(st["k"]), None if st["v"] is None else take(st["v"])
    w = torch.where(live, st["w"].gather(2, at), 0.0)
    return k, v, w, new.view(B).to(torch.int32), torch.where(live, idx, -1).to(torch.int32)


def _stored(x):
    codes, s, m = _quantise(x.double())
    return (m.double().unsqueeze(-1) + s.double().unsqueeze(-1) * codes).flatten(-2).to(x.dtype)


def _plain_attn(st):
    B, Hq, Hkv, Sq, D = st["B"], st["Hq"], st["Hkv"], st["Sq"], st["D"]
    s = _scores(st["q"].float(), _values(st["cache"], D, 0), st["mask"], st["scale"], st["lens"])
    top = s.amax(-1, keepdim=True).clamp_min(-3e38)
    e = torch.exp(s - top)
    total = e.sum(-1, keepdim=True)
    p = torch.where(total > 0, e / total, 0.0)
    lse = (top + torch.log(total)).squeeze(-1)
    o = (p.view(B, Hkv, -1, st["S"]) @ _values(st["cache"], D, 1)).view(B, Hq, Sq, D)
    # every slot of a sequence is valid: a slot behind its end would meet a weight of zero
    w = p.view(B, Hkv, -1, st["S"]).sum(2) if st["weights"] else None
    return o.to(st["q"].dtype), lse, w


def _some(**outs):
    return {k: v for k, v in outs.items() if v is not None}


def run(st):
    op = st["op"]
    if not own:
        if op == "weights":
            return _some(weights=_plain_weights(st))
        if op == "evict":
            k, v, w, lens, idx = _plain_evict(st)
            return _some(k=k, v=v, weights=w, lens=lens, idx=idx)
        if op == "store":
            return _some(k=_stored(st["k"]), v=_stored(st["v"]))
        o, lse, w = _plain_attn(st)
        return _some(out=o, lse=lse, weights=w)
    import online_softmax_flash_gb300 as osf
    if op == "weights":
        if "ws" not in st:   # a program keeps its workspace
            n = osf.osf_attn_key_weights_workspace_bytes(osf.OSF_F32 if st["dtype"] == "f32" else osf.OSF_BF16, st["B"],
                                                         st["Hq"], st["Hkv"], st["Sq"], st["Sk"], st["D"])
            st["ws"] = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
        w = osf.osf_attn_key_weights(st["q"], st["k"], st["lse"], weights=st["w"], mask=st["mask"], scale=st["scale"],
                                     workspace=st["ws"])
        return _some(weights=w)
    if op == "evict":
        k, v, w, lens, idx = osf.osf_kv_evict(st["k"], st["v"], st["w"], st["budget"], lens=st["lens"], sinks=st["sinks"],
                                              recent=st["recent"], k_out=st["k_out"], v_out=st["v_out"],
                                              weights_out=st["w_out"], lens_out=st["lens_out"], idx=st["idx"])
        return _some(k=k, v=v, weights=w, lens=lens, idx=idx)
    if op == "store":
        osf.osf_kv4_append(st["k"], st["v"], st["cache"], lens=st["lens"])
        k, v = osf.osf_kv4_read(st["cache"], st["D"], st["n"], starts=st["lens"], lens=st["lens_after"], k=st["k_out"],
                                v=st["v_out"])
        return _some(k=k, v=v)
    if "ws" not in st:
        n = osf.osf_attn_kv4_workspace_bytes(osf.OSF_F32 if st["dtype"] == "f32" else osf.OSF_BF16, st["B"], st["Hq"],
                                             st["Hkv"], st["Sq"], st["S"], st["D"], st["weights"])
        st["ws"] = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
    o = osf.osf_attn_kv4(st["q"], st["cache"], lens=st["lens"], out=st["out"], mask=st["mask"], scale=st["scale"],
                         lse=st["lse"], weights=st["w"], workspace=st["ws"])
    return _some(out=o, lse=st["lse"], weights=st["w"])


# ------------------------------------------------------------------------------------------ work
def _pairs(Sq, Sk, mask):
    """Visible (row, key) pairs of one head."""
    if mask == "none":
        return Sq * Sk
    off = Sk - Sq if mask == "bottom_right" else 0
    lo, hi = min(max(off + 1, 0), Sk), min(max(off + Sq, 0), Sk)   # keys the first and the last row see
    first = max(0, -off)                                           # rows before it see nothing
    rows = Sq - first
    grow = min(rows, hi - max(lo, 1) + 1) if rows > 0 else 0       # rows until the count stops growing
    a = max(lo, 1)
    return grow * a + grow * (grow - 1) // 2 + (rows - grow) * hi if rows > 0 else 0


def work(case):
    op, B, Hkv, D = case["op"], case["B"], case["Hkv"], case["D"]
    es = 4 if case.get("dtype") == "f32" else 2
    if op == "weights":
        Hq, Sq, Sk = case["Hq"], case["Sq"], case["Sk"]
        return dict(bytes=es * D * (B * Hq * Sq + B * Hkv * Sk) + 4 * B * (Hq * Sq + Hkv * Sk),
                    flops=2 * B * Hq * _pairs(Sq, Sk, case["mask"]) * D)
    if op == "evict":
        row = 2 * 2 * D if case["rows"] == "bf16" else D + D // 4
        # ragged lengths run evenly from half the budget to S
        live = case["S"] if not case["ragged"] else (case["S"] + case["budget"] // 2) / 2
        kept = min(case["budget"], live)
        return dict(bytes=int(B * Hkv * (4 * live + kept * (2 * row + 4 + 4))), flops=0)
    if op == "store":
        return dict(bytes=int(B * Hkv * case["n"] * D * (2 * 2 * es + 2 * 1.25)), flops=0)
    Hq, Sq, S = case["Hq"], case["Sq"], case["S"]
    live = (S + 1) / 2 if case["ragged"] and B > 1 else S
    out = 2 * es * B * Hq * Sq * D + 4 * B * Hq * Sq + (4 * B * Hkv * S if case["weights"] else 0)
    return dict(bytes=int(B * Hkv * live * 1.25 * D) + out, flops=int(4 * B * Hq * Sq * live * D))


# ------------------------------------------------------------------------------------------ exact
def exact(case, seed):
    st = prepare(case, seed)
    op, B, Hkv, D = case["op"], case["B"], case["Hkv"], case["D"]
    if op == "store":
        outs = {}
        for name in ("k", "v"):
            x = st[name].double().cpu().numpy().reshape(-1, GROUP)
            lo, hi = x.min(1), x.max(1)
            m = _to_bf16(lo, down=True)
            s = _to_bf16((hi - m) / 15, down=False)
            code = np.rint((x - m[:, None]) / np.where(s > 0, s, 1)[:, None])
            outs[name] = torch.from_numpy((m[:, None] + s[:, None] * code).reshape(st[name].shape))
        return outs
    if op == "evict":
        w, lens = st["w"].cpu().numpy(), st["lens"].cpu().numpy()
        S, budget, sinks, recent = case["S"], case["budget"], case["sinks"], case["recent"]
        idx = np.full((B, Hkv, budget), -1, np.int32)
        for b in range(B):
            n = int(lens[b])
            for h in range(Hkv):
                if n <= budget:
                    idx[b, h, :n] = np.arange(n)
                    continue
                mid = np.arange(sinks, n - recent)
                order = np.lexsort((mid, -w[b, h, mid].astype(np.float64)))[:budget - sinks - recent]
                idx[b, h] = np.concatenate([np.arange(sinks), np.sort(mid[order]), np.arange(n - recent, n)])
        at = torch.from_numpy(idx).cuda().long()
        live = at >= 0
        at = at.clamp_min(0)
        rows = lambda x: (x.gather(2, at[..., None].expand(-1, -1, -1, x.shape[-1])) * live[..., None].to(x.dtype))  # noqa: E731
        outs = dict(k=rows(st["k"]), weights=st["w"].gather(2, at).double() * live, idx=torch.from_numpy(idx),
                    lens=torch.from_numpy(np.minimum(lens, budget).astype(np.int32)))
        outs["k"] = outs["k"].double() if case["rows"] == "bf16" else outs["k"]
        if st["v"] is not None:
            outs["v"] = rows(st["v"]).double()
        return {k: outs[k] for k in ("k", "v", "weights", "lens", "idx") if k in outs}
    Hq, Sq = case["Hq"], case["Sq"]
    G, scale = Hq // Hkv, st["scale"]
    if op == "weights":
        Sk = case["Sk"]
        out = torch.zeros(B, Hkv, Sk, dtype=torch.float64, device="cuda")
        row, key = torch.arange(Sq, device="cuda")[:, None], torch.arange(Sk, device="cuda")[None, :]
        seen = torch.ones(Sq, Sk, dtype=torch.bool, device="cuda")
        if case["mask"] != "none":
            seen = key <= row + (Sk - Sq if case["mask"] == "bottom_right" else 0)
        for b in range(B):
            for h in range(Hq):
                s = torch.einsum("id,jd->ij", st["q"][b, h].double(), st["k"][b, h // G].double()) * scale
                out[b, h // G] += (torch.exp(s - st["lse"][b, h].double()[:, None]) * seen).sum(0)
        return dict(weights=out)
    o = torch.zeros(B, Hq, Sq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq, Sq), -math.inf, dtype=torch.float64, device="cuda")
    w = torch.zeros(B, Hkv, case["S"], dtype=torch.float64, device="cuda")
    for b in range(B):
        n = int(st["lens"][b])
        kv = _decode64(st["cache"][b, :, :n].cpu().numpy(), D)
        k, v = (torch.from_numpy(x).cuda() for x in kv)
        q = st["q"][b].double().view(Hkv, G, Sq, D)
        s = torch.einsum("hgid,hjd->hgij", q, k) * scale
        if case["mask"] == "bottom_right":
            row, key = torch.arange(Sq, device="cuda")[:, None], torch.arange(n, device="cuda")[None, :]
            s = torch.where(key <= row + n - Sq, s, -math.inf)
        z = torch.logsumexp(s, -1)
        p = torch.nan_to_num(torch.exp(s - z[..., None]), nan=0.0)
        o[b] = torch.einsum("hgij,hjd->hgid", p, v).reshape(Hq, Sq, D)
        lse[b] = z.reshape(Hq, Sq)
        w[b, :, :n] = p.sum((1, 2))
    outs = dict(out=o, lse=lse)
    if case["weights"]:
        outs["weights"] = w
    return outs


def _to_bf16(x, down):
    """The bfloat16 value (as float64) nearest to x on the lower or the upper side."""
    f = x.astype(np.float32)
    b = (f.view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32).astype(np.float64)   # towards zero
    out = ((b > x) if down else (b < x))
    step = (b.astype(np.float32).view(np.uint32) + np.uint32(0x10000)).view(np.float32).astype(np.float64)   # away from zero
    back = np.where(np.abs(b) > 0, (b.astype(np.float32).view(np.uint32) - np.uint32(0x10000)).view(np.float32).astype(np.float64), 0.0)
    away = (x < 0) if down else (x > 0)
    return np.where(out, np.where(away, step, back), b)


def _decode64(rec, D):
    """float64 K and V [H, n, D] of records uint8 [H, n, 1.25 D]."""
    halves = []
    for half in range(2):
        c = np.arange(D)
        byte = half * (D // 2) + 4 * ((c // 8 % 4) * (D // 32) + c // 32) + c % 8 // 2
        code = (rec[..., byte] >> (4 * (c % 2)).astype(np.uint8)) & 15
        at = D + half * (D // 8)
        pair = np.ascontiguousarray(rec[..., at:at + D // 8]).view(np.uint16).astype(np.uint32) << 16
        pair = pair.view(np.float32).astype(np.float64)
        halves.append(pair[..., 1::2][..., c // 32] + pair[..., 0::2][..., c // 32] * code)
    return halves
