"""Cases and plain forms of sliding-window attention with sinks (forward and backward) and of the paged 8-bit K/V
cache (appending with the position rotation, attention over it).

``listed()`` and ``draw()`` give cases, ``prepare()`` the tensors a program holds before the call, ``run()`` one
call: elementary torch operations while ``own`` is false, the library's entry points while it is true.

Window and sinks: the Sq rows are the last of Sk tokens, row i stands at position p = i + Sk - Sq and sees key j where
j <= p and (p - j < window or j < sinks).

The 8-bit cache: ``pages`` [n_pages, 2, Hkv, P, D] holds e4m3 codes (K, then V) of P tokens a page, ``scales``
[n_pages, 2, Hkv] a power of two for each page and head, ``table`` [B, pages of a sequence] the pages of a sequence in
order.  A value is code * scale.  The scale of a page is 2^e with the least e >= -110 for which its largest finite
magnitude is at most 448 * 2^e; it grows when a token that comes later needs it, and the codes that are there are
rounded again to the new one.  K is rotated before it is stored: channels i and i + R/2 (or 2i and 2i + 1) by the
angle whose cosine and sine the tables [positions, R/2] hold, rounded once to float32.
"""
import math

import numpy as np
import torch

own = False


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # a training step's (and a prompt's) attention with a window of 1024: the shape of the benchmark's prefill
        dict(name="window_prefill_4096", op="fwd", dtype="bf16", B=2, Hq=32, Hkv=8, Sq=4096, Sk=4096, D=128, window=1024,
             sinks=4),
        # one long document
        dict(name="window_prefill_16k", op="fwd", dtype="bf16", B=1, Hq=8, Hkv=2, Sq=16384, Sk=16384, D=64, window=2047,
             sinks=16),
        # a decode step that looks back 4096 tokens in the benchmark's bf16 cache
        dict(name="window_decode_32k", op="fwd", dtype="bf16", B=8, Hq=32, Hkv=8, Sq=1, Sk=32768, D=128, window=4096,
             sinks=4),
        # float32, a short chunk behind an odd length: the CUDA cores
        dict(name="window_f32_chunk", op="fwd", dtype="f32", B=1, Hq=8, Hkv=2, Sq=77, Sk=1001, D=96, window=200, sinks=1),
        # the gradients of the first case
        dict(name="window_grad_4096", op="bwd", dtype="bf16", B=2, Hq=32, Hkv=8, Sq=4096, Sk=4096, D=128, window=1024,
             sinks=4),
        # gradients of an odd length in float32
        dict(name="window_grad_f32_301", op="bwd", dtype="f32", B=1, Hq=4, Hkv=2, Sq=301, Sk=301, D=64, window=65, sinks=3),
        # the new token of every sequence of a decode batch, with its queries
        dict(name="append_token_b32", op="append", dtype="bf16", B=32, Hq=32, Hkv=8, n=1, S=2048, D=128, P=64, rot=128,
             interleaved=False, ragged=True),
        # a batch of whole prompts
        dict(name="append_prompt_4096", op="append", dtype="bf16", B=8, Hq=32, Hkv=8, n=4096, S=4096, D=128, P=64, rot=128,
             interleaved=False, ragged=False),
        # the benchmark's decode step, over the 8-bit cache
        dict(name="cache8_decode_32k", op="attn", dtype="bf16", B=8, Hq=32, Hkv=8, Sq=1, S=32768, D=128, P=64, window=0,
             sinks=0, ragged=False),
        # one short sequence: latency
        dict(name="cache8_decode_500", op="attn", dtype="bf16", B=1, Hq=16, Hkv=8, Sq=1, S=500, D=128, P=64, window=0,
             sinks=0, ragged=False),
        # four draft tokens over sequences of different lengths, within a window
        dict(name="cache8_draft_window", op="attn", dtype="bf16", B=16, Hq=32, Hkv=8, Sq=4, S=16384, D=64, P=16,
             window=2048, sinks=4, ragged=True),
        # float32 queries, another head dimension
        dict(name="cache8_f32_777", op="attn", dtype="f32", B=2, Hq=12, Hkv=4, Sq=2, S=777, D=96, P=32, window=0, sinks=0,
             ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "append", "attn", "attn"])
    D = rng.choice([64, 128, 128, 96])
    Hkv, G = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 3, 4, 5, 8])
    P = rng.choice([16, 32, 64, 64, 128])
    while True:
        B = rng.choice([1, 2, 3, 5, 8, 13])
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        # the CUDA-core path (float32, or a head dimension other than 64 and 128) gets less work
        slow = dtype == "f32" or D == 96
        if op in ("fwd", "bwd"):
            kind = rng.choice(["prompt", "chunk", "decode"]) if op == "fwd" else rng.choice(["prompt", "prompt", "chunk"])
            Sk = _log(rng, 64, 32768 if kind == "decode" else 8192)
            Sq = Sk if kind == "prompt" else rng.randint(1, 4) if kind == "decode" else max(1, _log(rng, 8, 1024) % Sk)
            window, sinks = _log(rng, 16, 4096), rng.choice([0, 1, 4, 17, 130])
            scores = B * Hkv * G * Sq * Sk
            if scores > (2e7 if slow else 1e9) or B * Hkv * Sk * D > (1 << 26 if slow else 1 << 28):
                continue
            return dict(op=op, dtype=dtype, B=B, Hq=Hkv * G, Hkv=Hkv, Sq=Sq, Sk=Sk, D=D, window=window, sinks=sinks)
        if op == "append":
            n = 1 if rng.random() < 0.4 else _log(rng, 2, 8192)
            S = n + rng.randint(0, 1000)
            if B * Hkv * S * D > 1 << 25:
                continue
            rot = rng.choice([D, D, D // 2, 0])
            return dict(op=op, dtype=dtype, B=B, Hq=Hkv * G, Hkv=Hkv, n=n, S=S, D=D, P=P, rot=rot,
                        interleaved=rng.random() < 0.3, ragged=True)
        Sq, S = rng.choice([1, 1, 1, 2, 4, 5]), _log(rng, 48, 32768)
        if B * Hkv * S * D > (1 << 24 if slow else 1 << 28):
            continue
        window = 0 if rng.random() < 0.5 else _log(rng, 16, 8192)
        return dict(op=op, dtype=dtype, B=B, Hq=Hkv * G, Hkv=Hkv, Sq=Sq, S=S, D=D, P=P, window=window,
                    sinks=rng.choice([0, 1, 4, 17, 130]) if window else 0, ragged=rng.random() < 0.6)


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


def _exponent(amax):
    """The least e >= -110 with amax <= 448 * 2^e, of float64 amax."""
    mant, e = torch.frexp(amax)   # amax = mant * 2^e, mant in [0.5, 1); 448 = 0.875 * 2^9
    e = e - 9 + (mant > 0.875)
    return torch.where(amax > 0, e, -110).clamp_min(-110)


def _to_e4m3(x):
    """float64 x, |x| <= 448, to the nearest e4m3 value, ties to even; NaN stays."""
    e = torch.frexp(x)[1].clamp_min(-5) - 4
    return torch.ldexp(torch.round(torch.ldexp(x, -e)), e)


def _table(gen, B, S, P):
    """Pages of B sequences of up to S tokens, in no order, among a few that nobody has."""
    per = (S + P - 1) // P
    n_pages = B * per + 3
    order = torch.randperm(n_pages, generator=gen, device="cuda")[:B * per]
    return n_pages, order.view(B, per).to(torch.int32).contiguous()


def _fill(pages, scales, table, rows, half, P):
    """Put rows [B, Hkv, S, D] into the K (0) or V (1) half of the pages of a table, each page with its own scale."""
    B, Hkv, S, D = rows.shape
    per = table.shape[1]
    x = torch.zeros(B, Hkv, per * P, D, device="cuda")
    x[:, :, :S] = rows
    x = x.view(B, Hkv, per, P, D).transpose(1, 2).double()
    e = _exponent(x.abs().amax((-1, -2)))
    codes = _to_e4m3(torch.ldexp(x, -e[..., None, None])).float().to(torch.float8_e4m3fn).view(torch.uint8)
    pages[table.long().flatten(), half] = codes.flatten(0, 1)
    scales[table.long().flatten(), half] = torch.ldexp(torch.ones_like(e, dtype=torch.float32), e).flatten(0, 1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, B, Hq, Hkv, D = case["op"], case["B"], case["Hq"], case["Hkv"], case["D"]
    dt = _dtype(case["dtype"])
    st = dict(case)
    if op in ("fwd", "bwd"):
        Sq, Sk = case["Sq"], case["Sk"]
        st["scale"] = D ** -0.5
        st["q"] = torch.randn(B, Hq, Sq, D, generator=gen, device="cuda").to(dt)
        st["k"], st["v"] = _rows(gen, B, Hkv, Sk, D).to(dt), _rows(gen, B, Hkv, Sk, D).to(dt)
        if op == "bwd":
            # what the forward pass left
            st["dout"] = torch.randn(B, Hq, Sq, D, generator=gen, device="cuda").to(dt)
            st["o"], st["lse"] = _plain_fwd(st)
            st["grads"] = [torch.empty_like(st[x]) for x in ("q", "k", "v")]
        else:
            st["out"], st["lse"] = torch.empty_like(st["q"]), torch.empty(B, Hq, Sq, device="cuda")
        return st
    P, S = case["P"], case["S"]
    n_pages, st["table"] = _table(gen, B, S, P)
    st["pages"] = torch.randint(0, 120, (n_pages, 2, Hkv, P, D), generator=gen, device="cuda", dtype=torch.uint8)
    st["scales"] = torch.ones(n_pages, 2, Hkv, device="cuda")
    if op == "append":
        n, R = case["n"], case["rot"]
        st["k"], st["v"] = _rows(gen, B, Hkv, n, D).to(dt), _rows(gen, B, Hkv, n, D).to(dt)
        st["q"] = torch.randn(B, Hq, n, D, generator=gen, device="cuda").to(dt)
        # the lengths before the call, and after it
        st["lens"] = torch.randint(0, S - n + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
        st["lens_after"] = st["lens"] + n
        # what is there already: tokens before the new ones, smaller now and then
        old = _rows(gen, B, Hkv, S, D) * torch.rand(B, 1, 1, 1, generator=gen, device="cuda")
        _fill(st["pages"], st["scales"], st["table"], old, 0, P)
        _fill(st["pages"], st["scales"], st["table"], old.flip(-1), 1, P)
        st["cos"] = st["sin"] = None
        if R:
            turn = torch.arange(S, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (
                -torch.arange(R // 2, device="cuda", dtype=torch.float64) * 2 / R)
            st["cos"], st["sin"] = torch.cos(turn).float().contiguous(), torch.sin(turn).float().contiguous()
        # read back from the start of the page that the first new token falls into
        st["starts"] = st["lens"] // P * P
        st["n_read"] = n + P - 1
        st["q_out"] = torch.empty_like(st["q"])
        st["k_out"], st["v_out"] = (torch.empty(B, Hkv, st["n_read"], D, dtype=dt, device="cuda") for _ in range(2))
        return st
    Sq = case["Sq"]
    for b in range(B):
        for half in range(2):
            _fill(st["pages"], st["scales"], st["table"][b:b + 1], _rows(gen, 1, Hkv, S, D), half, P)
    st["lens"] = _lens(gen, B, S, case["ragged"], min(S, Sq))
    st["scale"] = D ** -0.5
    st["q"] = torch.randn(B, Hq, Sq, D, generator=gen, device="cuda").to(dt)
    st["out"], st["lse"] = torch.empty_like(st["q"]), torch.empty(B, Hq, Sq, device="cuda")
    return st


# ------------------------------------------------------------------------------------------ plain forms
def _hidden(Sq, Sk, window, sinks, lens=None):
    """True where a row does not see a key, [Sq, Sk] or [B, 1, Sq, Sk]; lens: the tokens of each sequence, in place of Sk."""
    j = torch.arange(Sk, device="cuda")
    n = Sk if lens is None else lens.view(-1, 1, 1, 1)
    pos = torch.arange(Sq, device="cuda")[:, None] + (n - Sq)
    hidden = j > pos
    return hidden | ((pos - j >= window) & (j >= sinks)) if window else hidden


def _plain_softmax(s):
    """Softmax over the last dimension and its log-sum-exp; rows that are all -inf give 0 and -inf."""
    top = s.amax(-1, keepdim=True).clamp_min(-3e38)
    e = torch.exp(s - top)
    total = e.sum(-1, keepdim=True)
    return torch.where(total > 0, e / total, 0.0), (top + torch.log(total)).squeeze(-1)


def _plain_fwd(st):
    B, Hq, Hkv, Sq, Sk, D = (st[x] for x in ("B", "Hq", "Hkv", "Sq", "Sk", "D"))
    q, k, v = st["q"].float(), st["k"].float(), st["v"].float()
    s = (q.view(B, Hkv, -1, D) @ k.transpose(-1, -2)).view(B, Hq, Sq, Sk) * st["scale"]
    s.masked_fill_(_hidden(Sq, Sk, st["window"], st["sinks"]), -math.inf)
    p, lse = _plain_softmax(s)
    o = (p.view(B, Hkv, -1, Sk) @ v).view(B, Hq, Sq, D)
    return o.to(st["q"].dtype), lse


def _plain_bwd(st):
    B, Hq, Hkv, Sq, Sk, D = (st[x] for x in ("B", "Hq", "Hkv", "Sq", "Sk", "D"))
    q, k, v, o, do = (st[x].float() for x in ("q", "k", "v", "o", "dout"))
    s = (q.view(B, Hkv, -1, D) @ k.transpose(-1, -2)).view(B, Hq, Sq, Sk) * st["scale"]
    s.masked_fill_(_hidden(Sq, Sk, st["window"], st["sinks"]), -math.inf)
    p = torch.exp(s - st["lse"].clamp_min(-3e38).unsqueeze(-1)).view(B, Hkv, -1, Sk)
    dog, qg = do.view(B, Hkv, -1, D), q.view(B, Hkv, -1, D)
    dv = p.transpose(-1, -2) @ dog
    ds = p * (dog @ v.transpose(-1, -2) - (do * o).sum(-1).view(B, Hkv, -1, 1))
    dq = (ds @ k).view(B, Hq, Sq, D) * st["scale"]
    dk = ds.transpose(-1, -2) @ qg * st["scale"]
    return [g.to(st["q"].dtype) for g in (dq, dk, dv)]


def _rotated(x, st):
    """float32 rows [B, H, n, D] at positions lens .. lens + n - 1, rotated."""
    R = st["rot"]
    if not R:
        return x.float()
    at = st["lens"].long()[:, None] + torch.arange(x.shape[2], device="cuda")
    c, s = st["cos"][at].double().unsqueeze(1), st["sin"][at].double().unsqueeze(1)
    x = x.double()
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if st["interleaved"] else (x[..., :R // 2], x[..., R // 2:R])
    ra, rb = a * c - b * s, b * c + a * s
    turned = torch.stack([ra, rb], -1).flatten(-2) if st["interleaved"] else torch.cat([ra, rb], -1)
    return torch.cat([turned, x[..., R:]], -1).float()


def _plain_append(st):
    B, Hkv, n, P, D = (st[x] for x in ("B", "Hkv", "n", "P", "D"))
    at, per = st["lens"].long() % P, (n + 2 * P - 2) // P
    page = (st["lens"].long() // P)[:, None] + torch.arange(per, device="cuda")
    there = page < st["table"].shape[1]
    page = torch.where(there, page, 0)
    ids = st["table"].long().gather(1, page)                                     # pages that a token may fall into
    slot = torch.arange(per * P, device="cuda")
    is_old, is_new = slot < at[:, None], (slot >= at[:, None]) & (slot < at[:, None] + n)
    is_old, is_new = (m.view(B, 1, per, P, 1) for m in (is_old, is_new))
    src = (slot - at[:, None]).clamp(0, n - 1).view(B, 1, -1, 1).expand(-1, Hkv, -1, D)
    outs = []
    for half, rows in ((0, _rotated(st["k"], st)), (1, st["v"].float())):
        new = rows.gather(2, src).view(B, Hkv, per, P, D).double()
        old_scale = st["scales"][ids, half].transpose(1, 2)                      # [B, Hkv, per]
        codes = st["pages"][ids, half].transpose(1, 2)                           # [B, Hkv, per, P, D]
        old = codes.view(torch.float8_e4m3fn).double() * old_scale[..., None, None]
        e = _exponent(torch.where(is_new, new.abs(), 0.0).amax((-1, -2)))
        e = torch.where(is_old.any(3).squeeze(-1), torch.maximum(e, torch.frexp(old_scale)[1] - 1), e)
        value = torch.where(is_new, new, torch.where(is_old, old, 0.0))
        kept = _to_e4m3(torch.ldexp(value, -e[..., None, None]))
        # written back where a new token falls into the page
        touch = (is_new.any(3).view(B, 1, per) & there.view(B, 1, per)).expand(-1, Hkv, -1).transpose(1, 2)
        bytes_ = kept.float().to(torch.float8_e4m3fn).view(torch.uint8).transpose(1, 2)
        keep = (is_old | is_new).transpose(1, 2)
        hit = torch.where(keep, bytes_, codes.transpose(1, 2))
        b_i, p_i, h_i = touch.nonzero(as_tuple=True)
        st["pages"][ids[b_i, p_i], half, h_i] = hit[b_i, p_i, h_i]
        st["scales"][ids[b_i, p_i], half, h_i] = torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)[b_i, h_i, p_i]
        back = torch.ldexp(torch.where(is_old | is_new, kept, 0.0), e[..., None, None])
        outs.append(back.view(B, Hkv, -1, D)[:, :, :st["n_read"]].to(st["k"].dtype))
    return outs[0], outs[1], _rotated(st["q"], st).to(st["q"].dtype)


def _values(st, half):
    """The float32 values [B, Hkv, S, D] that one half of the pages of the sequences stands for."""
    ids = st["table"].long()
    x = st["pages"][ids, half].view(torch.float8_e4m3fn).float() * st["scales"][ids, half][..., None, None]
    return x.transpose(1, 2).flatten(2, 3)[:, :, :st["S"]]


def _plain_attn(st):
    B, Hq, Hkv, Sq, S, D = (st[x] for x in ("B", "Hq", "Hkv", "Sq", "S", "D"))
    s = (st["q"].float().view(B, Hkv, -1, D) @ _values(st, 0).transpose(-1, -2)).view(B, Hq, Sq, S) * st["scale"]
    s.masked_fill_(_hidden(Sq, S, st["window"], st["sinks"], st["lens"]), -math.inf)
    p, lse = _plain_softmax(s)
    o = (p.view(B, Hkv, -1, S) @ _values(st, 1)).view(B, Hq, Sq, D)
    return o.to(st["q"].dtype), lse


def run(st):
    op = st["op"]
    if not own:
        if op == "fwd":
            o, lse = _plain_fwd(st)
            return dict(out=o, lse=lse)
        if op == "bwd":
            dq, dk, dv = _plain_bwd(st)
            return dict(dq=dq, dk=dk, dv=dv)
        if op == "append":
            k, v, q = _plain_append(st)
            return dict(k=k, v=v, q=q)
        o, lse = _plain_attn(st)
        return dict(out=o, lse=lse)
    import online_softmax_flash_gb300 as osf
    code = osf.OSF_F32 if st["dtype"] == "f32" else osf.OSF_BF16
    sizes = [st[x] for x in ("B", "Hq", "Hkv")]
    if op in ("fwd", "bwd"):
        if "ws" not in st:   # a program keeps its workspace
            need = osf.osf_attn_window_workspace_bytes if op == "fwd" else osf.osf_attn_bwd_window_workspace_bytes
            n = need(code, *sizes, st["Sq"], st["Sk"], st["D"], st["window"], st["sinks"])
            st["ws"] = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
        if op == "fwd":
            o = osf.osf_attn_fwd_gqa_window(st["q"], st["k"], st["v"], st["window"], sinks=st["sinks"], out=st["out"],
                                            scale=st["scale"], lse=st["lse"], workspace=st["ws"])
            return dict(out=o, lse=st["lse"])
        dq, dk, dv = osf.osf_attn_bwd_gqa_window(st["q"], st["k"], st["v"], st["o"], st["dout"], st["lse"], st["window"],
                                                 sinks=st["sinks"], dq=st["grads"][0], dk=st["grads"][1],
                                                 dv=st["grads"][2], scale=st["scale"], workspace=st["ws"])
        return dict(dq=dq, dk=dk, dv=dv)
    if op == "append":
        osf.osf_kv8_append(st["k"], st["v"], st["pages"], st["scales"], st["table"], lens=st["lens"], cos=st["cos"],
                           sin=st["sin"], interleaved=st["interleaved"], q=st["q"], q_out=st["q_out"])
        k, v = osf.osf_kv8_read(st["pages"], st["scales"], st["table"], st["n_read"], starts=st["starts"],
                                lens=st["lens_after"], k=st["k_out"], v=st["v_out"])
        return dict(k=k, v=v, q=st["q_out"])
    if "ws" not in st:
        n = osf.osf_attn_kv8_workspace_bytes(code, *sizes, st["Sq"], st["D"], st["P"], st["table"].shape[1], st["window"],
                                             st["sinks"])
        st["ws"] = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
    o = osf.osf_attn_kv8(st["q"], st["pages"], st["scales"], st["table"], lens=st["lens"], out=st["out"],
                         window=st["window"], sinks=st["sinks"], scale=st["scale"], lse=st["lse"], workspace=st["ws"])
    return dict(out=o, lse=st["lse"])


# ------------------------------------------------------------------------------------------ work
def _seen(Sq, n, window, sinks):
    """Visible (row, key) pairs of one head, and the keys that some row sees, of Sq rows that end a sequence of n tokens."""
    pos = np.arange(n - Sq, n, dtype=np.int64)
    pos = pos[pos >= 0]
    if not len(pos):
        return 0, 0
    if not window:
        return int((pos + 1).sum()), int(n)
    first = np.maximum(pos - window + 1, 0)
    return int((pos + 1 - first + np.minimum(first, sinks)).sum()), int(n - first[0] + min(first[0], sinks))


def work(case):
    op, B, Hq, Hkv, D = (case[x] for x in ("op", "B", "Hq", "Hkv", "D"))
    es = 4 if case["dtype"] == "f32" else 2
    if op in ("fwd", "bwd"):
        Sq, Sk = case["Sq"], case["Sk"]
        pairs, keys = _seen(Sq, Sk, case["window"], case["sinks"])
        q, kv = B * Hq * Sq * D * es, B * Hkv * keys * D * es
        if op == "fwd":
            return dict(bytes=2 * q + 2 * kv + 4 * B * Hq * Sq, flops=4 * B * Hq * pairs * D)
        return dict(bytes=4 * q + 2 * kv + 2 * B * Hkv * Sk * D * es + 4 * B * Hq * Sq, flops=10 * B * Hq * pairs * D)
    P = case["P"]
    if op == "append":
        n = case["n"]
        # K, V and Q in, codes and rotated Q out, the codes read again and their values out
        return dict(bytes=int(B * n * D * (Hkv * (2 * es + 2 + 2 + 2 * es) + Hq * 2 * es)) + 2 * 4 * case["rot"] // 2 * B * n,
                    flops=0)
    Sq, S = case["Sq"], case["S"]
    # ragged lengths run evenly up to S: eight lengths stand for them
    lens = [S] if not case["ragged"] or B == 1 else [S] + [min(S, Sq) + (S - min(S, Sq)) * (2 * i + 1) // 16 for i in range(8)]
    seen = [_seen(Sq, n, case["window"], case["sinks"]) for n in lens]
    if len(seen) > 1:
        mean = [sum(x[i] for x in seen[1:]) / 8 for i in range(2)]
        pairs, keys = (seen[0][i] + (B - 1) * mean[i] for i in range(2))
    else:
        pairs, keys = (B * x for x in seen[0])
    return dict(bytes=int(Hkv * keys * 2 * D * (1 + 4 / (P * D))) + 2 * es * B * Hq * Sq * D + 4 * B * Hq * Sq,
                flops=int(4 * Hq * pairs * D))


# ------------------------------------------------------------------------------------------ exact
def _e4m3_table():
    """What each of the 256 e4m3 codes stands for."""
    c = np.arange(256)
    e, m = c >> 3 & 15, c & 7
    mag = np.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e - 7.0))
    return np.where(c & 127 == 127, np.nan, np.where(c & 128, -mag, mag))


def _sees(pos, n, window, sinks):
    """[len(pos), n]: whether a row at each position sees each key."""
    j, p = torch.arange(n, device="cuda")[None, :], pos[:, None]
    near = (p - j) < window if window else torch.ones_like(p - j, dtype=torch.bool)
    return (j <= p) & (near | (j < sinks))


def _exact_rows(q, k, v, pos, window, sinks, scale):
    """One head in 64 bits: outputs and log-sum-exp of rows q at positions pos over keys k and values v."""
    s = torch.where(_sees(pos, k.shape[0], window, sinks), q @ k.T * scale, -math.inf)
    z = torch.logsumexp(s, -1)
    return torch.nan_to_num(torch.exp(s - z[:, None]), nan=0.0) @ v, z


def exact(case, seed):
    op, B, Hq, Hkv, D = (case[x] for x in ("op", "B", "Hq", "Hkv", "D"))
    G = Hq // Hkv
    st = prepare(case, seed)
    if op in ("fwd", "bwd"):
        Sq, Sk, scale = case["Sq"], case["Sk"], st["scale"]
        pos = torch.arange(Sk - Sq, Sk, device="cuda")
        if op == "fwd":
            o = torch.empty(B, Hq, Sq, D, dtype=torch.float64, device="cuda")
            lse = torch.empty(B, Hq, Sq, dtype=torch.float64, device="cuda")
            for b in range(B):
                for h in range(Hq):
                    o[b, h], lse[b, h] = _exact_rows(st["q"][b, h].double(), st["k"][b, h // G].double(),
                                                     st["v"][b, h // G].double(), pos, case["window"], case["sinks"], scale)
            return dict(out=o, lse=lse)
        dq = torch.zeros(B, Hq, Sq, D, dtype=torch.float64, device="cuda")
        dk, dv = (torch.zeros(B, Hkv, Sk, D, dtype=torch.float64, device="cuda") for _ in range(2))
        see = _sees(pos, Sk, case["window"], case["sinks"])
        for b in range(B):
            for h in range(Hq):
                q, do, o = (st[x][b, h].double() for x in ("q", "dout", "o"))
                k, v = (st[x][b, h // G].double() for x in ("k", "v"))
                p = torch.where(see, torch.exp(q @ k.T * scale - st["lse"][b, h].double()[:, None]), 0.0)
                ds = p * (do @ v.T - (do * o).sum(-1)[:, None]) * scale
                dq[b, h] = ds @ k
                dk[b, h // G] += ds.T @ q
                dv[b, h // G] += p.T @ do
        return dict(dq=dq, dk=dk, dv=dv)
    if op == "append":
        # stored values are rounded to codes: they have no other value.  The queries are rotated alone.
        q, R = st["q"].double(), case["rot"]
        if R:
            i = torch.arange(R // 2, device="cuda")
            i, j = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + R // 2)
            for b in range(B):
                at = int(st["lens"][b])
                z = torch.complex(st["cos"][at:at + case["n"]].double(), st["sin"][at:at + case["n"]].double())
                z = torch.complex(q[b, :, :, i], q[b, :, :, j]) * z
                q[b, :, :, i], q[b, :, :, j] = z.real, z.imag
        return dict(k=None, v=None, q=q)
    codes = torch.from_numpy(_e4m3_table()).cuda()
    Sq, P, scale = case["Sq"], case["P"], st["scale"]
    o = torch.zeros(B, Hq, Sq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq, Sq), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(B):
        n = int(st["lens"][b])
        ids = st["table"][b, :(n + P - 1) // P].long()
        kv = codes[st["pages"][ids].long()] * st["scales"][ids].double()[..., None, None]      # [pages, 2, Hkv, P, D]
        kv = kv.permute(1, 2, 0, 3, 4).flatten(2, 3)[:, :, :n]
        pos = torch.arange(n - Sq, n, device="cuda")
        for h in range(Hq):
            o[b, h], lse[b, h] = _exact_rows(st["q"][b, h].double(), kv[0, h // G], kv[1, h // G], pos, case["window"],
                                             case["sinks"], scale)
    return dict(out=o, lse=lse)
