"""Operators over 4-bit caches and windowed attention: the cases that are timed,
their plain forms and their values in 64 bits.

Four operators of one attention block over a paged low-rank cache (exact Keys
K of width d, Value latents z of width r_v, Key residuals e of width r_k, one
row per token and KV head):

* ``cache4``: rows of k, z and e are rounded to 4 bits as they are written
  into pages, and the same tokens are read back as the values they stand for;
* ``route4``: page scores over a 4-bit cache, the maximum over a page's live
  tokens and a KV group's query heads of q . (z P_K + e U_K^T);
* ``attend4``: attention of one query token per sequence over the selected
  pages of a 4-bit cache, the softmax weights combining the latents;
* ``window``: attention of the last n tokens of every sequence over a sliding
  window and a few first tokens that stay visible (sinks), for single tokens
  and prompt chunks, over bf16, E4M3 and 4-bit caches.

The 4-bit format: blocks of 16 columns share one scale byte, 5 exponent bits
(bias 15) above 3 mantissa bits, the upper bits of an IEEE half without its
sign; the codes are E2M1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives).
scale = amax / 6 rounded to nearest even, at most 10240; code = x / scale
rounded to nearest even, at most 6.  One (page, KV head) tile holds the codes
[S][w / 2] (column 2i in the low nibble of byte i), then the scales
[S][w / 16].

With ``own`` false everything here is elementary torch arithmetic; with it
true ``run`` makes the library's calls.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases
def _llama(**kw):
    # Llama-8B attention layer: 32 query heads on 8 KV heads, pages of 16
    return dict(dict(Hq=32, Hkv=8, d=128, r_v=64, r_k=32, page=16), **kw)


def _qwen(**kw):
    # Qwen3-32B attention layer: 64 query heads on 8 KV heads, pages of 32
    return dict(dict(Hq=64, Hkv=8, d=128, r_v=96, r_k=64, page=32), **kw)


def listed():
    return [
        # one decode step's token of each of 16 sequences: a latency
        _llama(name="cache4_token_b16", op="cache4", B=16, T=32769, n=1),
        # a short ragged tail of a small layer, read back by an inspection tool
        dict(name="cache4_small", op="cache4", B=3, Hq=4, Hkv=1, d=64, r_v=32, r_k=16, page=16,
             T=512, n=37),
        # a 4096-token prompt chunk of eight sequences (the prefill workload)
        _qwen(name="cache4_prompt", op="cache4", B=8, T=9001, n=4096),
        # page scores of one sequence at a short context
        _llama(name="route4_b1_t4k", op="route4", B=1, T=4096, r_v=96),
        # page scores of the serving batch at 32K tokens (the headline decode)
        _llama(name="route4_b16_t32k", op="route4", B=16, T=32768, equal=True),
        # selected attention, one sequence, 64 pages
        _llama(name="attend4_b1_t4k", op="attend4", B=1, T=4096, r_v=96, top_k=64),
        # selected attention of the headline decode: 128 of 2048 pages
        _llama(name="attend4_b16_t32k", op="attend4", B=16, T=32768, top_k=128, equal=True),
        # a sliding-window layer's decode step, bf16 cache
        _llama(name="window_token_bf16", op="window", fmt="bf16", B=16, T=32768, n=1,
               window=4096, sink=4, equal=True),
        # a full-attention layer's decode step over a 4-bit cache
        _llama(name="window_token_4bit_full", op="window", fmt="4bit", B=16, T=32768, n=1,
               window=0, sink=0, equal=True),
        # five draft tokens verified in one call, ragged lengths, E4M3 cache
        _llama(name="window_draft_e4m3", op="window", fmt="e4m3", B=7, T=20001, n=5, window=8192,
               sink=16),
        # a prompt chunk of 4096 tokens in the middle of a long prompt
        _llama(name="window_prompt_bf16", op="window", fmt="bf16", B=1, T=16384, n=4096,
               window=4096, sink=4),
        # ragged prompts over a 4-bit cache, wide groups, odd chunk
        _qwen(name="window_prompt_4bit", op="window", fmt="4bit", B=3, T=5003, n=1023,
              window=2000, sink=5, r_k=32),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    most = [work(c) for c in listed()]
    max_bytes = max(w["bytes"] for w in most)
    max_flops = max(w["flops"] for w in most)
    while True:
        op = rng.choice(["cache4", "route4", "attend4", "window", "window"])
        c = dict(op=op, B=_log_int(rng, 1, 32), Hkv=rng.choice([1, 2, 3, 4, 8]),
                 d=rng.choice([64, 128, 128]), r_v=rng.choice([32, 64, 64, 96, 128]),
                 r_k=rng.choice([16, 32, 64]), page=rng.choice([16, 32]))
        G = rng.choice([1, 2, 4, 4, 8])
        c["T"] = _log_int(rng, 1, 65536)
        if op == "cache4":
            c["n"] = min(c["T"], _log_int(rng, 1, 8192))
        elif op == "attend4":
            c["top_k"] = _log_int(rng, 2, 512)
        elif op == "window":
            c["fmt"] = rng.choice(["bf16", "e4m3", "4bit"])
            if c["fmt"] == "bf16":
                c["page"] = rng.choice([8, 16, 32])
            if c["fmt"] == "e4m3":
                G = rng.choice([4, 8])
                c["r_k"] = 32
                c["r_v"] = rng.choice([64, 96, 128])
            c["n"] = min(c["T"], rng.choice([1, 1, _log_int(rng, 2, 16), _log_int(rng, 16, 4096)]))
            c["window"] = rng.choice([0, _log_int(rng, 1, c["T"]), _log_int(rng, 64, 8192)])
            c["sink"] = rng.choice([0, 1, 4, _log_int(rng, 1, 64)])
        c["Hq"] = c["Hkv"] * G
        c["equal"] = rng.random() < 0.3
        if c["Hq"] * c["r_v"] % 64:
            continue
        w = work(c)
        if w["bytes"] <= max_bytes and w["flops"] <= max_flops and \
                c["B"] * c["T"] * c["Hkv"] * c["d"] <= 16 * 32768 * 8 * 128:
            return c


def _lengths(c):
    """Lengths of the batch: the first sequence has all T tokens, the others
    fall short of it by odd amounts, or have as many (`equal`)."""
    T, B = c["T"], c["B"]
    if c.get("equal"):
        return [T] * B
    return [T - (b * 2741) % (T // 3 + 1) for b in range(B)]


def _visible(p, window, sink):
    """How many tokens the query at position p sees."""
    if p < 0:
        return 0
    lo = 0 if window == 0 else max(0, p - window + 1)
    return p + 1 - lo + min(sink, lo)


def _sum_visible(L, n, window, sink):
    return sum(_visible(p, window, sink) for p in range(L - n, L))


def _union(L, n, window, sink):
    p0, p1 = max(L - n, 0), L - 1
    if p1 < 0:
        return 0
    lo = 0 if window == 0 else max(0, p0 - window + 1)
    return p1 + 1 - lo + min(sink, lo)


def work(case):
    c = case
    B, Hq, Hkv, d, rv, rk, S = (c[k] for k in ("B", "Hq", "Hkv", "d", "r_v", "r_k", "page"))
    L = _lengths(c)
    q4 = 9.0 / 16.0  # bytes of a 4-bit column with its share of the scale
    if c["op"] == "cache4":
        rows = B * c["n"] * Hkv * (d + rv + rk)
        return {"bytes": rows * (2 + 2 * q4 + 2) + 8 * B, "flops": rows * 4}
    if c["op"] == "route4":
        toks = sum(L) * Hkv
        pages = sum(-(-x // S) for x in L) * Hkv
        fac = Hkv * d * (rv + rk) * 2
        return {"bytes": toks * (rv + rk) * q4 + pages * 4 + B * Hq * d * 2 + fac,
                "flops": 2 * toks * (rv + rk) * (Hq // Hkv) + 2 * B * Hq * d * (rv + rk)}
    if c["op"] == "attend4":
        toks = sum(min(x, c["top_k"] * S) for x in L) * Hkv
        return {"bytes": toks * (d + rv) * q4 + B * Hq * (d + rv) * 2,
                "flops": 2 * toks * (d + rv) * (Hq // Hkv)}
    per = {"bf16": 2.0, "e4m3": 1.0, "4bit": q4}[c["fmt"]]
    toks = sum(_union(x, c["n"], c["window"], c["sink"]) for x in L) * Hkv
    pairs = sum(_sum_visible(x, c["n"], c["window"], c["sink"]) for x in L) * Hq
    return {"bytes": toks * (d + rv) * per + B * c["n"] * Hq * (d + rv) * 2,
            "flops": 2 * pairs * (d + rv)}


# ------------------------------------------------------------- 4-bit format
def _quantise(x):
    """fp32 [..., w] -> (codes uint8 [..., w], scale bytes uint8 [..., w/16])."""
    w = x.shape[-1]
    blk = x.reshape(*x.shape[:-1], w // 16, 16)
    s = (blk.abs().amax(-1) / 6.0).clamp(max=10240.0)
    u = s.view(torch.int32)
    norm = ((u + 0x7FFFF + ((u >> 20) & 1)) >> 20) - 896
    sub = torch.round(s * 131072.0).to(torch.int32)  # steps of 2^-17 below 2^-14
    byte = torch.where(s < 2.0 ** -14, sub, norm)
    a = (blk / _scale_value(byte).clamp(min=2.0 ** -17)[..., None]).abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
            + (a >= 3.5) + (a > 5.0)).to(torch.uint8)
    code = torch.where((byte == 0)[..., None], torch.zeros_like(code), code)
    code = code | (torch.signbit(blk).to(torch.uint8) << 3)
    return code.reshape(x.shape), byte.to(torch.uint8)


def _scale_value(byte):
    """Scale bytes (integers) -> fp32: the byte is the top of a half."""
    h = (byte.to(torch.int32) << 7).to(torch.int16)
    return h.view(torch.float16).to(torch.float32)


def _values(codes, scales):
    """codes [..., w], scale bytes [..., w/16] -> fp32 [..., w] (exact)."""
    lut = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6],
                       device=codes.device)
    v = lut[codes.to(torch.int64)]
    return v * _scale_value(scales).repeat_interleave(16, dim=-1)


def _pack_tiles(x, S):
    """fp32 [pages][Hkv][S][w] -> 4-bit tiles, uint8 [pages][Hkv][S * w * 9 / 16]."""
    codes, scales = _quantise(x)
    by = codes[..., 0::2] | (codes[..., 1::2] << 4)
    return torch.cat([by.flatten(-2), scales.flatten(-2)], -1).contiguous()


def _unpack_tiles(t, S, w):
    """4-bit tiles uint8 [..., S * w * 9 / 16] -> fp32 [..., S][w]."""
    by = t[..., :S * w // 2].reshape(*t.shape[:-1], S, w // 2)
    sc = t[..., S * w // 2:].reshape(*t.shape[:-1], S, w // 16)
    codes = torch.stack([by & 15, by >> 4], -1).flatten(-2)
    return _values(codes, sc)


def _tiles(cache, fmt, S, w):
    """Cache tiles of any format -> fp32 [..., S][w]."""
    if fmt == "4bit":
        return _unpack_tiles(cache, S, w)
    if fmt == "e4m3":
        return cache.view(torch.float8_e4m3fn).to(torch.float32)
    return cache.to(torch.float32)


# ----------------------------------------------------------------- prepare
def _gen(seed, salt):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1000003 + salt)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def prepare(case, seed):
    c = case
    op, B, Hq, Hkv, d, rv, rk, S, T = (c[k] for k in ("op", "B", "Hq", "Hkv", "d", "r_v", "r_k",
                                                      "page", "T"))
    G = Hq // Hkv
    fmt = c.get("fmt", "4bit")
    mp = -(-T // S) + 1                     # block-table row: the context and one spare page
    phys = B * mp
    g = _gen(seed, 1)
    st = {"case": dict(c), "fmt": fmt, "mp": mp, "phys": phys}
    lens = _lengths(c)
    st["table"] = torch.randperm(phys, generator=g, device=DEV).to(torch.int32).reshape(B, mp)
    P_K = (_randn(g, Hkv, rv, d) / math.sqrt(rv)).to(torch.bfloat16)
    U_K = torch.linalg.qr(_randn(g, Hkv, d, rk))[0].to(torch.bfloat16).contiguous()
    if op == "cache4":
        n = c["n"]
        # per-row and per-head magnitudes differ, a few rows are zero
        mag = torch.exp(0.7 * _randn(g, B, n, Hkv, 1))
        mag = mag * (torch.rand(B, n, Hkv, 1, generator=g, device=DEV) > 0.002)
        st["k"] = (_randn(g, B, n, Hkv, d) * mag).to(torch.bfloat16)
        st["z"] = (_randn(g, B, n, Hkv, rv) * mag).to(torch.bfloat16)
        st["e"] = (_randn(g, B, n, Hkv, rk) * mag * 0.3).to(torch.bfloat16)
        st["lens"] = torch.tensor([x - n if x > n else 0 for x in lens], dtype=torch.int32,
                                  device=DEV)
        st["first"] = st["lens"].clone()
        st["new_lens"] = torch.zeros_like(st["lens"])
        for name, w in (("K", d), ("Z", rv), ("E", rk)):
            st[name] = torch.zeros(phys, Hkv, S * w * 9 // 16, dtype=torch.uint8, device=DEV)
        for name, w in (("k_out", d), ("z_out", rv), ("e_out", rk)):
            st[name] = torch.zeros(B, n, Hkv, w, dtype=torch.bfloat16, device=DEV)
        return _with_plan(st)
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    # latents and residuals are normal, Keys follow from them with some noise
    # (made page by page, so the pages' slots past a length hold values too)
    K = torch.empty(phys, Hkv, S, d, dtype=torch.bfloat16, device=DEV)
    Z = torch.empty(phys, Hkv, S, rv, dtype=torch.bfloat16, device=DEV)
    E = torch.empty(phys, Hkv, S, rk, dtype=torch.bfloat16, device=DEV)
    step = max(1, (1 << 26) // (Hkv * S * d))
    for i in range(0, phys, step):
        m = min(step, phys - i)
        z, e = _randn(g, m, Hkv, S, rv), _randn(g, m, Hkv, S, rk)
        Z[i:i + m] = z
        E[i:i + m] = e
        if op != "route4":
            K[i:i + m] = (torch.matmul(z, P_K.float()) + torch.matmul(e, U_K.float().mT)
                          + 0.1 * _randn(g, m, Hkv, S, d))
    n = c.get("n", 1)
    # each query is drawn towards one live token's Key
    q = _randn(g, B, n, Hkv, G, d)
    u = torch.rand(B, n, Hkv, G, generator=g, device=DEV)
    pos = (st["lens"][:, None] - n + torch.arange(n, device=DEV)).clamp(min=0)
    w_eff = c.get("window", 0) or T
    tok = (pos[..., None, None] - (u * torch.minimum(pos + 1, torch.tensor(w_eff, device=DEV))
                                   [..., None, None]).long()).clamp(min=0)
    page = st["table"].long().gather(1, (tok // S).reshape(B, -1)).reshape(tok.shape)
    head = torch.arange(Hkv, device=DEV)[None, None, :, None].expand_as(tok)
    if op == "route4":
        zt, et = Z[page, head, tok % S].float(), E[page, head, tok % S].float()
        q = q + (torch.einsum("bngcr,grd->bngcd", zt, P_K.float())
                 + torch.einsum("bngcr,gdr->bngcd", et, U_K.float())) * 0.5
    else:
        q = q + 0.6 * K[page, head, tok % S].float()
    q = q.to(torch.bfloat16).reshape(B, n, Hq, d)
    st["q"] = q if op == "window" else q.reshape(B, Hq, d).contiguous()
    if op == "route4":
        st["P_K"], st["U_K"] = P_K, U_K
        st["scores"] = torch.zeros(B, Hkv, mp, dtype=torch.float32, device=DEV)
        st["Z"], st["E"] = _packed(Z, S), _packed(E, S)
        return _with_plan(st)
    if op == "attend4":
        k = c["top_k"]
        sel = torch.full((B, Hkv, k), -1, dtype=torch.int32)
        cg = torch.Generator().manual_seed(seed * 7 + 3)
        for b in range(B):
            P = -(-lens[b] // S)
            for h in range(Hkv):
                if k >= P:
                    p = torch.arange(P)
                else:
                    p = torch.randperm(P, generator=cg)[:k]
                    p[0] = P - 1
                    p = torch.unique(p)
                sel[b, h, :len(p)] = p.to(torch.int32)
        st["sel"] = sel.to(DEV)
        st["out"] = torch.zeros(B, Hq, rv, dtype=torch.bfloat16, device=DEV)
    else:
        st["out"] = torch.zeros(B, n, Hq, rv, dtype=torch.bfloat16, device=DEV)
    if fmt == "4bit":
        st["K"], st["Z"] = _packed(K, S), _packed(Z, S)
    elif fmt == "e4m3":
        st["K"] = K.float().clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        st["Z"] = Z.float().clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        st["K"], st["Z"] = K, Z
    return _with_plan(st)


def _packed(x, S):
    """_pack_tiles of a bf16 cache, some pages at a time."""
    step = max(1, (1 << 25) // x[0].numel())
    return torch.cat([_pack_tiles(x[i:i + step].float(), S) for i in range(0, x.shape[0], step)])


def _with_plan(st):
    """The dims and the workspace that a program keeps beside its caches."""
    if not own:
        return st
    import sparse_decode_attention_basiskv_b200 as bkv
    c = st["case"]
    st["dims"] = dims = bkv.Dims(
        B=c["B"], Hq=c["Hq"], Hkv=c["Hkv"], d=c["d"], hidden=128, r_v=c["r_v"], r_k=c["r_k"],
        page_size=c["page"], max_pages_per_seq=st["mp"], num_phys_pages=st["phys"],
        cache_fp8=1 if st["fmt"] == "e4m3" else 0)
    st["msl"] = c["T"]
    if c["op"] == "window":
        need = bkv.window_workspace_size(dims, c["n"], c["T"], c["sink"], c["window"])
    elif c["op"] == "cache4":
        need = 0
    else:
        need = bkv.workspace_size(dims, c.get("top_k", 2), c["T"])
    st["ws"] = torch.empty(max(need, 256), dtype=torch.uint8, device=DEV)
    return st


# --------------------------------------------------------------------- run
def run(state):
    st, c = state, state["case"]
    if own:
        return _run_own(st, c)
    if c["op"] == "cache4":
        out = [_values(*_quantise(st[x].float())).to(torch.bfloat16) for x in ("k", "z", "e")]
        return {"k": out[0], "z": out[1], "e": out[2], "lens": st["lens"] + c["n"]}
    if c["op"] == "route4":
        return _plain_route(st, c)
    if c["op"] == "attend4":
        return _plain_selected(st, c)
    return _plain_window(st, c)


def _run_own(st, c):
    import sparse_decode_attention_basiskv_b200 as bkv
    if c["op"] == "cache4":
        bkv.basiskv_cache4_write(st["dims"], st["k"], st["z"], st["e"], c["n"], st["lens"],
                                 st["new_lens"], st["table"], st["K"], st["Z"], st["E"])
        bkv.basiskv_cache4_read(st["dims"], st["first"], c["n"], st["new_lens"], st["table"],
                                st["K"], st["Z"], st["E"], st["k_out"], st["z_out"],
                                st["e_out"])
        return {"k": st["k_out"], "z": st["z_out"], "e": st["e_out"], "lens": st["new_lens"]}
    if c["op"] == "route4":
        bkv.basiskv_cache4_route(st["dims"], st["q"], st["lens"], st["msl"], st["table"],
                                 st["P_K"], st["U_K"], st["Z"], st["E"], 2, st["scores"], None,
                                 st["ws"])
        return st["scores"]
    if c["op"] == "attend4":
        bkv.basiskv_cache4_attend(st["dims"], st["q"], st["lens"], st["msl"], st["table"],
                                  st["K"], st["Z"], st["sel"], c["top_k"], st["out"], st["ws"])
        return st["out"]
    bkv.basiskv_attend_window(st["dims"], st["q"], c["n"], st["lens"], st["msl"], st["table"],
                              st["K"], st["Z"], c["sink"], c["window"], st["out"], st["ws"],
                              cache4=st["fmt"] == "4bit")
    return st["out"]


def _plain_route(st, c):
    B, Hkv, S, rv, rk = c["B"], c["Hkv"], c["page"], c["r_v"], c["r_k"]
    G = c["Hq"] // Hkv
    qg = st["q"].float().reshape(B, Hkv, G, c["d"])
    qz = torch.einsum("bgcd,grd->bgcr", qg, st["P_K"].float())
    qe = torch.einsum("bgcd,gdr->bgcr", qg, st["U_K"].float())
    out = torch.zeros_like(st["scores"])
    for b, L in enumerate(_lengths(c)):
        P = -(-L // S)
        pages = st["table"][b, :P].long()
        z = _unpack_tiles(st["Z"][pages], S, rv).transpose(0, 1).reshape(Hkv, P * S, rv)
        e = _unpack_tiles(st["E"][pages], S, rk).transpose(0, 1).reshape(Hkv, P * S, rk)
        s = torch.matmul(z, qz[b].mT) + torch.matmul(e, qe[b].mT)  # [Hkv][tokens][G]
        s = s.amax(-1)
        s[:, L:] = -math.inf
        out[b, :, :P] = s.reshape(Hkv, P, S).amax(-1)
    return out


def _softmax_mix(s, z):
    """softmax over the last axis of s (-inf: masked; rows of nothing give
    zeros) times z, fp32."""
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
    return torch.matmul(p, z) / p.sum(-1, keepdim=True).clamp(min=1e-30)


def _plain_selected(st, c):
    B, Hkv, S, d, rv = c["B"], c["Hkv"], c["page"], c["d"], c["r_v"]
    G = c["Hq"] // Hkv
    sel = st["sel"].long()
    out = []
    heads = torch.arange(Hkv, device=DEV)[:, None]
    for b, L in enumerate(_lengths(c)):
        pages = st["table"][b].long()[sel[b].clamp(min=0)]  # [Hkv][k]
        K = _unpack_tiles(st["K"][pages, heads], S, d).reshape(Hkv, -1, d)
        Z = _unpack_tiles(st["Z"][pages, heads], S, rv).reshape(Hkv, -1, rv)
        tok = (sel[b][..., None] * S + torch.arange(S, device=DEV)).reshape(Hkv, -1)
        live = (tok >= 0) & (tok < L)
        qb = st["q"][b].float().reshape(Hkv, G, d)
        s = torch.matmul(qb, K.mT) / math.sqrt(d)
        s = torch.where(live[:, None, :], s, torch.full_like(s, -math.inf))
        out.append(_softmax_mix(s, Z).reshape(c["Hq"], rv))
    return torch.stack(out).to(torch.bfloat16)


def _plain_window(st, c):
    B, Hkv, S, d, rv, n = c["B"], c["Hkv"], c["page"], c["d"], c["r_v"], c["n"]
    G, W, sink = c["Hq"] // Hkv, c["window"], c["sink"]
    out = torch.zeros_like(st["out"])
    for b, L in enumerate(_lengths(c)):
        rows = max(1, min(n, (1 << 28) // (max(1, L) * c["Hq"])))
        for j0 in range(0, n, rows):
            j1 = min(n, j0 + rows)
            p0, p1 = L - n + j0, L - n + j1 - 1
            if p1 < 0:
                continue
            lo = 0 if W == 0 else max(0, max(p0, 0) - W + 1)
            first = min(-(-sink // S), lo // S)  # whole pages of sinks before the window's
            pg = torch.cat([torch.arange(first, device=DEV),
                            torch.arange(lo // S, p1 // S + 1, device=DEV)])
            tok = (pg[:, None] * S + torch.arange(S, device=DEV)).reshape(-1)
            pages = st["table"][b].long()[pg]
            K = _tiles(st["K"][pages], st["fmt"], S, d).transpose(0, 1).reshape(Hkv, -1, d)
            Z = _tiles(st["Z"][pages], st["fmt"], S, rv).transpose(0, 1).reshape(Hkv, -1, rv)
            Z = torch.where((tok <= p1)[:, None], Z, torch.zeros_like(Z))
            qb = st["q"][b, j0:j1].float().reshape(j1 - j0, Hkv, G, d).permute(1, 2, 0, 3)
            s = torch.matmul(qb.reshape(Hkv, -1, d), K.mT) / math.sqrt(d)
            s = s.reshape(Hkv, G, j1 - j0, -1)
            p = torch.arange(p0, p1 + 1, device=DEV)[:, None]
            see = tok <= p
            if W:
                see &= (tok > p - W) | (tok < sink)
            s = torch.where(see, s, torch.full_like(s, -math.inf))
            a = _softmax_mix(s.reshape(Hkv, -1, s.shape[-1]), Z)
            a = a.reshape(Hkv, G, j1 - j0, rv).permute(2, 0, 1, 3).reshape(j1 - j0, c["Hq"], rv)
            out[b, j0:j1] = a.to(torch.bfloat16)
    return out


# ------------------------------------------------------------------- exact
_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _exact_scale(byte):
    e, m = (byte.long() >> 3).double(), (byte.long() & 7).double()
    return torch.where(e > 0, (1 + m / 8) * torch.exp2(e - 15), m / 8 * 2.0 ** -14)


def _exact_round4(x):
    """The format's definition on float64 [..., w]: the nearest scale byte to
    amax / 6 (ties to the even byte), then the nearest code (ties to the even
    code)."""
    blk = x.reshape(*x.shape[:-1], -1, 16)
    table = _exact_scale(torch.arange(227, device=x.device))  # 0 .. 10240
    target = blk.abs().amax(-1) / 6
    hi = torch.searchsorted(table, target.contiguous()).clamp(max=226)
    lo = (hi - 1).clamp(min=0)
    dl, dh = (target - table[lo]).abs(), (table[hi] - target).abs()
    byte = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    s = table[byte][..., None]
    grid = torch.tensor(_E2M1, dtype=torch.float64, device=x.device)
    a = torch.where(s > 0, blk.abs() / torch.where(s > 0, s, torch.ones_like(s)),
                    torch.zeros_like(blk))
    hi = torch.searchsorted(grid, a.contiguous()).clamp(max=7)
    lo = (hi - 1).clamp(min=0)
    dl, dh = (a - grid[lo]).abs(), (grid[hi] - a).abs()
    code = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    v = grid[code] * s
    return torch.where(blk < 0, -v, v).reshape(x.shape)


def _exact_rows(st, name, b, tokens, w):
    """float64 [Hkv][tokens][w]: cache rows of sequence b by token number."""
    S, fmt = st["case"]["page"], st["fmt"]
    pages, r = st["table"][b].long()[tokens // S], tokens % S
    t = st[name]
    if fmt == "bf16":
        return t[pages, :, r].double().transpose(0, 1)
    if fmt == "e4m3":
        return t.view(torch.float8_e4m3fn)[pages, :, r].double().transpose(0, 1)
    half, col = w // 2, torch.arange(w, device=t.device)
    cb = (r * half)[:, None] + torch.arange(half, device=t.device)
    heads = torch.arange(t.shape[1], device=t.device)[:, None, None]
    by = t[pages[None, :, None], heads, cb[None]].long()
    codes = (by[..., col // 2] >> (4 * (col % 2))) & 15
    sb = (S * half + r * (w // 16))[:, None] + torch.arange(w // 16, device=t.device)
    sc = _exact_scale(t[pages[None, :, None], heads, sb[None]])
    grid = torch.tensor(_E2M1, dtype=torch.float64, device=t.device)
    v = grid[codes & 7] * sc[..., col // 16]
    return torch.where(codes >= 8, -v, v)


def _exact_mix(q, K, Z, see, d):
    """softmax(q K^T / sqrt(d)) Z over the tokens that `see` allows, float64."""
    s = torch.einsum("gqd,gtd->gqt", q, K) / math.sqrt(d)
    s = s.masked_fill(~see, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.where(see, (s - top.nan_to_num(neginf=0.0)).exp(), torch.zeros_like(s))
    tot = p.sum(-1, keepdim=True)
    return torch.einsum("gqt,gtr->gqr", p, Z) / torch.where(tot > 0, tot, torch.ones_like(tot))


def exact(case, seed):
    c = case
    st = prepare(case, seed)
    B, Hq, Hkv, d, rv = c["B"], c["Hq"], c["Hkv"], c["d"], c["r_v"]
    G, lens = Hq // Hkv, _lengths(c)
    if c["op"] == "cache4":
        out = {}
        for x in ("k", "z", "e"):
            out[x] = torch.cat([_exact_round4(st[x][:, i:i + 512].double())
                                for i in range(0, c["n"], 512)], 1)
        out["lens"] = (st["lens"] + c["n"]).double()
        return out
    if c["op"] == "route4":
        out = torch.zeros(B, Hkv, st["mp"], dtype=torch.float64, device=DEV)
        for b, L in enumerate(lens):
            t = torch.arange(L, device=DEV)
            z = _exact_rows(st, "Z", b, t, rv)
            k = torch.einsum("gtr,grd->gtd", z, st["P_K"].double())
            k += torch.einsum("gtr,gdr->gtd", _exact_rows(st, "E", b, t, c["r_k"]),
                              st["U_K"].double())
            qb = st["q"][b].double().reshape(Hkv, G, d)
            s = torch.einsum("gcd,gtd->gct", qb, k).amax(1)
            P = -(-L // c["page"])
            full = torch.full((Hkv, P * c["page"]), -math.inf, dtype=torch.float64, device=DEV)
            full[:, :L] = s
            out[b, :, :P] = full.reshape(Hkv, P, -1).amax(-1)
        return out
    if c["op"] == "attend4":
        out = torch.zeros(B, Hq, rv, dtype=torch.float64, device=DEV)
        for b, L in enumerate(lens):
            for g in range(Hkv):
                p = st["sel"][b, g]
                p = p[p >= 0].long()
                t = (p[:, None] * c["page"] + torch.arange(c["page"], device=DEV)).reshape(-1)
                t = t[t < L]
                qb = st["q"][b].double().reshape(Hkv, G, d)[g:g + 1]
                a = _exact_mix(qb, _exact_rows(st, "K", b, t, d)[g:g + 1],
                               _exact_rows(st, "Z", b, t, rv)[g:g + 1],
                               torch.ones(1, 1, len(t), dtype=torch.bool, device=DEV), d)
                out[b, g * G:(g + 1) * G] = a[0]
        return out
    n, W, sink = c["n"], c["window"], c["sink"]
    out = torch.zeros(B, n, Hq, rv, dtype=torch.float64, device=DEV)
    for b, L in enumerate(lens):
        t_all = torch.arange(L, device=DEV)
        Kb, Zb = _exact_rows(st, "K", b, t_all, d), _exact_rows(st, "Z", b, t_all, rv)
        rows = max(1, min(n, (1 << 26) // (L * G)))
        for g in range(Hkv):
            for j0 in range(0, n, rows):
                j = torch.arange(j0, min(n, j0 + rows), device=DEV)
                p = (L - n + j)[:, None]
                see = (t_all[None] <= p) & ((t_all[None] < sink) | (p - t_all[None] < (W or L + 1)))
                see = see[:, None].expand(-1, G, -1).reshape(1, -1, L)
                qb = st["q"][b, j].double()[:, g * G:(g + 1) * G].reshape(1, -1, d)
                a = _exact_mix(qb, Kb[g:g + 1], Zb[g:g + 1], see, d)
                out[b, j, g * G:(g + 1) * G] = a.reshape(len(j), G, rv)
    return out
