"""Cases and plain forms of the cache-compression operators.

Four operators that shrink a decode-time key/value cache and read it:

  block    attention over a cache held in 8 bits (E4M3 or int8) with one scale
           per block of T tokens and kv head, contiguous or in pages:
               k_t = k_scale[b,h,t // T] * decode(k_code[b,h,t]),  v_t likewise,
               out = softmax(scale * q k^T) v,  lse = log sum exp(scale * q k^T)
  append   writes new bf16 tokens into such a cache. Per touched block with new
           tokens' largest magnitude a:  s = a / R rounded up to 8 significant
           bits (R = 448 or 127); a block that already holds tokens keeps
           max(old scale, s) and, when that grew, its older codes become
           round(decode(code) * old / new); new codes are round(x / s), half
           to even.
  weights  decode attention that also adds each cached token's attention
           weight, summed over the query heads of its kv head and over the
           queries, to a running total:  w_out[t] = w_in[t] + sum_i p_i[t].
  evict    keeps, per (sequence, kv head), the last `recent` tokens and the
           keep - recent others with the largest totals (ties to the lowest
           index), in order, and gathers their keys, values and totals.

`run` computes them with elementary torch operations in fp32 (own = False) or
through the package's entry points (own = True); `exact` gives the definition
in 64 bits.
"""
import math
import random

import torch

own = False

RANGE = {"e4m3": 448.0, "int8": 127.0}


# -------------------------------------------------------------------- cases --

def listed():
    return [
        # the smallest call: one short sequence, a launch's worth of work
        dict(name="block tiny d64", op="block", B=1, q_len=1, Hq=4, Hkv=4, D=64, Lmax=1024, T=16, kv="e4m3", page=0,
             layout="HND", ragged=False),
        # one sequence over a long context, one query head per kv head
        dict(name="block mha 16k", op="block", B=1, q_len=1, Hq=32, Hkv=32, D=128, Lmax=16384, T=64, kv="e4m3", page=0,
             layout="HND", ragged=False),
        # a very long context, eight query heads per kv head
        dict(name="block gqa 128k", op="block", B=1, q_len=1, Hq=64, Hkv=8, D=128, Lmax=131072, T=32, kv="int8",
             page=0, layout="HND", ragged=False),
        # a serving batch of uneven sequences in shuffled pages
        dict(name="block paged batch", op="block", B=32, q_len=1, Hq=32, Hkv=8, D=128, Lmax=8000, T=64, kv="e4m3",
             page=64, layout="HND", ragged=True),
        # one new token for each sequence of a serving batch
        dict(name="append token", op="append", B=64, n=1, Hkv=8, D=128, Lmax=4096, T=64, kv="e4m3", page=0,
             layout="HND", ragged=True),
        # a whole prompt into an empty cache
        dict(name="append prompt", op="append", B=1, n=16384, Hkv=32, D=128, Lmax=16384, T=32, kv="int8", page=0,
             layout="HND", ragged=False),
        # chunks of prompts, uneven, on top of cached tokens, in pages
        dict(name="append paged chunk", op="append", B=16, n=1000, Hkv=8, D=128, Lmax=8192, T=16, kv="e4m3", page=32,
             layout="NHD", ragged=True),
        # scored decoding over the long single sequences
        dict(name="weights mha 16k", op="weights", B=1, q_len=1, Hq=32, Hkv=32, D=128, Lmax=16384, ragged=False),
        dict(name="weights gqa 128k", op="weights", B=1, q_len=1, Hq=64, Hkv=8, D=128, Lmax=131072, ragged=False),
        # a window of the last queries scores uneven prompts
        dict(name="weights window", op="weights", B=8, q_len=4, Hq=16, Hkv=4, D=64, Lmax=9001, ragged=True),
        # a very long cache cut to a quarter
        dict(name="evict 128k", op="evict", B=1, Hkv=8, D=128, Lmax=131072, keep=32768, recent=1024, ragged=False),
        # a batch of uneven sequences cut to a budget (some are shorter than it)
        dict(name="evict batch", op="evict", B=64, Hkv=8, D=128, Lmax=4096, keep=1000, recent=100, ragged=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["block", "append", "weights", "evict"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8, 8, 32])
    B = _log_int(rng, 1, 64)
    # cached K elements: at most the largest listed case's bytes (an append or an eviction also writes them)
    most = max(64, (1 << (27 if op in ("block", "weights") else 26)) // (B * Hkv * D))
    Lmax = _log_int(rng, 64, min(131072, most))
    c = dict(op=op, B=B, Hkv=Hkv, D=D, Lmax=Lmax, ragged=rng.random() < 0.6)
    if op in ("block", "weights"):
        g = rng.choice([1, 1, 2, 3, 4, 8, 16])
        c.update(Hq=g * Hkv, q_len=rng.choice([q for q in (1, 1, 1, 2, 3, 5) if q * g <= 16]))
    if op in ("block", "append"):
        c.update(T=rng.choice([16, 32, 64, 128]), kv=rng.choice(["e4m3", "int8"]), layout=rng.choice(["HND", "NHD"]))
        c["page"] = rng.choice([0, max(c["T"], rng.choice([16, 64, 256]))])
    if op == "append":
        c["n"] = _log_int(rng, 1, Lmax)
    if op == "evict":
        c["keep"] = _log_int(rng, 1, Lmax)
        c["recent"] = rng.randint(0, min(c["keep"], 256))
    return c


# ------------------------------------------------------------------- inputs --

def _lengths(case):
    """Cached tokens of each sequence: all Lmax, or spread over [1, Lmax]
    (the golden ratio's multiples), the same set for every seed."""
    B, L = case["B"], case["Lmax"]
    if not case["ragged"]:
        return [L] * B
    return [1 + int((L - 1) * (((i + 1) * 0.6180339887498949) % 1.0)) for i in range(B)]


def _news(case, lens):
    """New tokens of each sequence (append)."""
    n = case["n"]
    if not case["ragged"]:
        return [min(n, L) for L in lens]
    return [min(L, max(1, n - (i * n) // (2 * case["B"]))) for i, L in enumerate(lens)]


def _block_scale(a, kv):
    """Largest magnitudes a to scales: a / R rounded up to 8 significant bits.
    (R as a tensor: torch multiplies by the reciprocal of a number.)"""
    x = a / torch.full((), RANGE[kv], device="cuda")
    return ((x.view(torch.int32) + 0xFFFF) & -0x10000).view(torch.float32)


def _to_codes(x, kv):
    """fp32 values inside the code range to code bytes, half to even."""
    if kv == "e4m3":
        return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.round(x).clamp(-127.0, 127.0).to(torch.int8).view(torch.uint8)


def _from_codes(c, kv):
    return c.view(torch.float8_e4m3fn if kv == "e4m3" else torch.int8).float()


def _paged(case, codes, scales, lens, gen):
    """Codes [B,Hkv,Lmax,D] and scales [B,Hkv,nblk] scattered into shuffled
    pages; returns the pools, their scales and the block table."""
    B, Hkv, D, T, ps = case["B"], case["Hkv"], case["D"], case["T"], case["page"]
    L = case["Lmax"]
    per = -(-L // ps)
    need = sum(-(-n // ps) for n in lens)
    pages = need + 2
    order = torch.randperm(pages, generator=gen, device="cuda")[:need].to(torch.int32)
    table = torch.full((B, (per + 3) // 4 * 4), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(lens):
        m = -(-n // ps)
        table[b, :m] = order[at:at + m]
        at += m
    pad = per * ps
    out = []
    for c in codes:
        full = torch.zeros((B, Hkv, pad, D), dtype=torch.uint8, device="cuda")
        full[:, :, :L] = c
        full = full.view(B, Hkv, per, ps, D)
        full = full.permute(0, 2, 1, 3, 4) if case["layout"] == "HND" else full.permute(0, 2, 3, 1, 4)
        pool = torch.full((pages,) + tuple(full.shape[2:]), 0x7F if case["op"] == "block" else 0x21, dtype=torch.uint8,
                          device="cuda")
        used = table[:, :per] >= 0
        pool[table[:, :per][used].long()] = full[used]
        out.append(pool)
    for s in scales:
        full = torch.zeros((B, Hkv, pad // T), device="cuda")
        full[:, :, :s.shape[2]] = s
        full = full.view(B, Hkv, per, ps // T).permute(0, 2, 1, 3)
        pool = torch.full((pages, Hkv, ps // T), float("nan") if case["op"] == "block" else 5.0, device="cuda")
        used = table[:, :per] >= 0
        pool[table[:, :per][used].long()] = full[used]
        out.append(pool)
    return out, table


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    rng = random.Random(int(seed))
    op, B, Hkv, D, L = case["op"], case["B"], case["Hkv"], case["D"], case["Lmax"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    lens = _lengths(case)
    news = _news(case, lens) if op == "append" else [0] * B
    both = list(zip(lens, news))
    rng.shuffle(both)
    lens, news = [x for x, _ in both], [x for _, x in both]
    s = dict(case=case, scale=1.0 / math.sqrt(D), seqlens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    inside = torch.arange(L, device="cuda")[None, :] < s["seqlens"][:, None]

    if op in ("block", "append"):
        # a cache as appends leave it: per block of T tokens the largest magnitude sets the scale
        T, kv = case["T"], case["kv"]
        nblk = -(-L // T)
        held = inside if op == "block" else \
            torch.arange(L, device="cuda")[None, :] < (s["seqlens"] - torch.tensor(news, device="cuda"))[:, None]
        codes, scales = [], []
        for _ in range(2):
            c = torch.empty((B, Hkv, L, D), dtype=torch.uint8, device="cuda")
            sc = torch.empty((B, Hkv, nblk), device="cuda")
            for b in range(B):
                x = torch.zeros((Hkv, nblk * T, D), device="cuda")
                x[:, :L] = normal(Hkv, L, D)
                # magnitudes drift along the sequence and differ by head
                x.view(Hkv, nblk, T * D).mul_(torch.exp2(torch.rand((Hkv, nblk, 1), generator=g, device="cuda") * 2 - 1))
                x = x.to(torch.bfloat16).float()
                x[:, :L] *= held[b][None, :, None]
                sc[b] = _block_scale(x.view(Hkv, nblk, T * D).abs().amax(2), kv)
                y = x.view(Hkv, nblk, T, D) / sc[b].clamp_min(1e-30)[:, :, None, None]
                c[b] = _to_codes(y, kv).view(Hkv, nblk * T, D)[:, :L]
            # what lies past the cached tokens is never used (NaN where only a read could show it)
            codes.append(torch.where(held[:, None, :, None], c, torch.full_like(c, 0x7F if op == "block" else 0x21)))
            used = held.new_zeros((B, nblk * T))
            used[:, :L] = held
            used = used.view(B, nblk, T).any(2)
            scales.append(torch.where(used[:, None, :], sc, torch.full_like(sc, float("nan") if op == "block" else 5.0)))
        if case["page"]:
            (kc, vc, ks, vs), s["table"] = _paged(case, codes, scales, lens, g)
        else:
            (kc, vc), (ks, vs) = codes, scales
        s.update(k=kc, v=vc, ks=ks, vs=vs)
        if op == "append":
            s["new_lens"] = torch.tensor(news, dtype=torch.int32, device="cuda")
            s["k_new"] = normal(B, case["n"], Hkv, D).to(torch.bfloat16)
            s["v_new"] = normal(B, case["n"], Hkv, D).to(torch.bfloat16)
            return s
    else:
        k = normal(B, Hkv, L, D).to(torch.bfloat16)
        v = normal(B, Hkv, L, D).to(torch.bfloat16)
        pad = ~inside[:, None, :, None]
        s.update(k=k.masked_fill_(pad, float("nan")), v=v.masked_fill_(pad, float("nan")))
        # totals so far: uneven, many tokens equal and many never looked at
        w = torch.exp(2.0 * normal(B, Hkv, L)).to(torch.bfloat16).float()
        w = torch.where(torch.rand((B, Hkv, L), generator=g, device="cuda") < 0.3, torch.zeros_like(w), w)
        s["w"] = w.masked_fill_(~inside[:, None, :], float("nan"))
    if op == "evict":
        s.update(k_out=torch.zeros((B, Hkv, case["keep"], D), dtype=torch.bfloat16, device="cuda"),
                 v_out=torch.zeros((B, Hkv, case["keep"], D), dtype=torch.bfloat16, device="cuda"),
                 w_out=torch.zeros((B, Hkv, case["keep"]), device="cuda"),
                 kept=torch.zeros((B, Hkv, case["keep"]), dtype=torch.int32, device="cuda"),
                 new_seqlens=torch.zeros((B,), dtype=torch.int32, device="cuda"))
        return s
    s["q"] = normal(B, case["q_len"], case["Hq"], D).to(torch.bfloat16)
    s["out"] = torch.zeros((B, case["q_len"], case["Hq"], D), device="cuda")
    s["lse"] = torch.zeros((B, case["q_len"], case["Hq"]), device="cuda")
    if op == "weights":
        s["w_out"] = torch.zeros((B, Hkv, L), device="cuda")
    return s


# -------------------------------------------------------------- plain forms --

def _attention(case, q, k, v, seqlens, scale):
    """out, lse and the probabilities [B,Hkv,q_len*g,L] of fp32 k, v; query j
    sees the first seqlens - (q_len - 1 - j) tokens."""
    B, q_len, Hq, D = q.shape
    Hkv, L = k.shape[1], k.shape[2]
    g = Hq // Hkv
    x = q.float().view(B, q_len, Hkv, g, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, q_len * g, D)
    z = torch.matmul(x, k.transpose(2, 3)) * scale
    sees = seqlens[:, None] - (q_len - 1 - torch.arange(q_len, device="cuda"))[None, :]
    mask = torch.arange(L, device="cuda")[None, None, :] < sees[:, :, None]
    mask = mask[:, None, :, None, :].expand(B, Hkv, q_len, g, L).reshape(B, Hkv, q_len * g, L)
    z = torch.where(mask, z, torch.full_like(z, -math.inf))
    m = z.amax(3, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    e = torch.exp(z - m)
    total = e.sum(3, keepdim=True)
    p = torch.where(total > 0, e / total, torch.zeros_like(e))
    lse = (m + torch.log(total))[..., 0]
    o = torch.matmul(p, v)
    o = o.view(B, Hkv, q_len, g, D).permute(0, 2, 1, 3, 4).reshape(B, q_len, Hq, D)
    return o, lse.view(B, Hkv, q_len, g).permute(0, 2, 1, 3).reshape(B, q_len, Hq), p


def _slots(s, pos):
    """Index of token positions pos [B, n] in the cache arrays, and of their
    blocks in the scale arrays."""
    c = s["case"]
    if c["page"]:
        per = s["table"].shape[1]
        page = torch.gather(s["table"].long(), 1, (pos // c["page"]).clamp(0, per - 1)).clamp_min(0)
        off = pos % c["page"]
        at = (page, slice(None), off) if c["layout"] == "HND" else (page, off)
        return at, (page, slice(None), off // c["T"])
    seq = torch.arange(pos.shape[0], device="cuda")[:, None].expand_as(pos)
    pos = pos.clamp(0, c["Lmax"] - 1)
    return (seq, slice(None), pos), (seq, slice(None), pos // c["T"])


def _plain_block(s):
    c = s["case"]
    pos = torch.arange(c["Lmax"], device="cuda")[None, :].expand(c["B"], -1)
    at, blk = _slots(s, pos)
    inside = (pos < s["seqlens"][:, None])[:, :, None, None]
    kv = []
    for codes, scale in ((s["k"], s["ks"]), (s["v"], s["vs"])):
        x = _from_codes(codes[at], c["kv"]) * scale[blk][..., None]          # [B, L, Hkv, D]
        kv.append(torch.where(inside, x, torch.zeros_like(x)).transpose(1, 2))
    o, lse, _ = _attention(c, s["q"], kv[0], kv[1], s["seqlens"], s["scale"])
    return dict(out=o, lse=lse)


def _plain_append(s):
    c = s["case"]
    B, n, Hkv, D, T, kv = c["B"], c["n"], c["Hkv"], c["D"], c["T"], c["kv"]
    end = s["seqlens"].long()
    start = end - s["new_lens"].long()
    first = start.clamp_min(0) // T
    blocks = (n + T - 2) // T + 1                                            # a run of n tokens touches this many at most
    pos = first[:, None] * T + torch.arange(blocks * T, device="cuda")[None, :]
    old = pos < start[:, None]
    new = ~old & (pos < end[:, None].clamp_max(c["Lmax"]))
    at, blk = _slots(s, pos)
    row = (pos - start[:, None]).clamp(0, n - 1)[:, :, None, None].expand(-1, -1, Hkv, D)
    write = (old | new)
    wat = tuple(x if isinstance(x, slice) else x[write] for x in at)
    has = write.view(B, blocks, T).any(2)
    bat = tuple(x if isinstance(x, slice) else x.view(B, blocks, T)[:, :, 0][has] for x in blk)
    fresh = ~old.view(B, blocks, T).any(2)[:, :, None]                       # blocks without older tokens
    for x_new, codes, scale in ((s["k_new"], s["k"], s["ks"]), (s["v_new"], s["v"], s["vs"])):
        x = torch.gather(x_new.float(), 1, row)                              # [B, blocks*T, Hkv, D]
        x = torch.where(new[:, :, None, None], x, torch.zeros_like(x))
        a = x.view(B, blocks, T, Hkv, D).abs().amax(dim=(2, 4))              # [B, blocks, Hkv]
        sc = _block_scale(a, kv)
        before = scale[blk].view(B, blocks, T, Hkv)[:, :, 0]
        sc = torch.where(fresh, sc, torch.maximum(sc, before))
        per = sc[:, :, None, :].expand(B, blocks, T, Hkv).reshape(B, blocks * T, Hkv, 1)
        was = before[:, :, None, :].expand(B, blocks, T, Hkv).reshape(B, blocks * T, Hkv, 1)
        x = torch.where(old[:, :, None, None], _from_codes(codes[at], kv) * was, x)
        y = torch.where(per > 0, x / per, torch.zeros_like(x))
        codes[wat] = _to_codes(y, kv)[write]
        scale[bat] = sc[has]
    return _append_outputs(s)


def _append_outputs(s):
    kind = torch.float8_e4m3fn if s["case"]["kv"] == "e4m3" else torch.int8
    return dict(k=s["k"].view(kind), v=s["v"].view(kind), k_scale=s["ks"], v_scale=s["vs"])


def _plain_weights(s):
    c = s["case"]
    inside = torch.arange(c["Lmax"], device="cuda")[None, :] < s["seqlens"][:, None]
    m = inside[:, None, :, None]
    k = torch.where(m, s["k"].float(), torch.zeros((), device="cuda"))
    v = torch.where(m, s["v"].float(), torch.zeros((), device="cuda"))
    o, lse, p = _attention(c, s["q"], k, v, s["seqlens"], s["scale"])
    s["w_out"].copy_(torch.where(inside[:, None, :], s["w"] + p.sum(2), s["w_out"]))
    return dict(out=o, lse=lse, weights=s["w_out"])


def _plain_evict(s):
    c = s["case"]
    B, Hkv, L, D, keep = c["B"], c["Hkv"], c["Lmax"], c["D"], c["keep"]
    lens = s["seqlens"].long()[:, None, None]
    t = torch.arange(L, device="cuda")[None, None, :]
    w = torch.where(t >= lens, -math.inf, torch.where(t >= lens - c["recent"], math.inf, s["w"]))
    w = torch.where((lens <= keep) & (t < lens), math.inf, w)
    order = torch.sort(w, dim=2, descending=True, stable=True).indices
    n = lens.clamp_max(keep)
    slot = torch.arange(keep, device="cuda")[None, None, :]
    idx = order[:, :, :keep]
    if idx.shape[2] < keep:
        idx = torch.cat([idx, idx.new_zeros((B, Hkv, keep - idx.shape[2]))], 2)
    idx = torch.sort(torch.where(slot < n, idx, idx.new_full((), 1 << 40)), dim=2).values
    live = slot < n
    idx = torch.where(live, idx, torch.zeros_like(idx))
    wide = idx[..., None].expand(-1, -1, -1, D)
    s["k_out"].copy_(torch.where(live[..., None], torch.gather(s["k"], 2, wide), s["k_out"]))
    s["v_out"].copy_(torch.where(live[..., None], torch.gather(s["v"], 2, wide), s["v_out"]))
    s["w_out"].copy_(torch.where(live, torch.gather(s["w"], 2, idx), torch.zeros((), device="cuda")))
    s["kept"].copy_(torch.where(live, idx, idx.new_full((), -1)))
    s["new_seqlens"].copy_(n[:, 0, 0])
    return _evict_outputs(s)


def _evict_outputs(s):
    return dict(k=s["k_out"], v=s["v_out"], weights=s["w_out"], kept=s["kept"], seqlens=s["new_seqlens"])


# ------------------------------------------------------- the framework's calls --

def _own_call(s):
    """The prepared call that a decode loop keeps for its buffers: arguments
    checked and marshalled once, workspace allocated and zeroed once."""
    import decode_attention_07_b200 as fd
    c = s["case"]

    def zeroed(nbytes):
        return torch.zeros(nbytes, dtype=torch.uint8, device="cuda") if nbytes else None

    if c["op"] == "block":
        S = fd.fd_plan(c["B"], c["Hq"], c["Hkv"], c["D"],
                       s["table"].shape[1] * c["page"] if c["page"] else c["Lmax"])
        ws = zeroed(fd.fd_workspace_bytes(c["B"], c["Hq"] * c["q_len"], c["Hkv"], c["D"], c["Lmax"], S))
        if c["page"]:
            return fd.prepare_decode_quant_block_paged(s["q"], s["k"], s["v"], s["ks"], s["vs"], c["kv"], c["T"],
                                                       s["table"], s["seqlens"], s["scale"], s["out"], s["lse"], ws,
                                                       c["layout"], S)
        return fd.prepare_decode_quant_block(s["q"], s["k"], s["v"], s["ks"], s["vs"], c["kv"], c["T"], s["seqlens"],
                                             s["scale"], s["out"], s["lse"], ws, S)
    if c["op"] == "append":
        if c["page"]:
            return fd.prepare_quant_append_paged(s["k_new"], s["v_new"], s["k"], s["v"], s["ks"], s["vs"], c["kv"],
                                                 c["T"], s["table"], s["seqlens"], s["new_lens"], c["layout"])
        return fd.prepare_quant_append(s["k_new"], s["v_new"], s["k"], s["v"], s["ks"], s["vs"], c["kv"], c["T"],
                                       s["seqlens"], s["new_lens"])
    if c["op"] == "weights":
        S = fd.fd_plan(c["B"], c["Hq"], c["Hkv"], c["D"], c["Lmax"])
        ws = zeroed(fd.fd_weights_workspace_bytes(c["B"], c["q_len"], c["Hq"], c["Hkv"], c["D"], c["Lmax"], S))
        return fd.prepare_decode_weights(s["q"], s["k"], s["v"], s["seqlens"], s["scale"], s["out"], s["lse"], s["w"],
                                         s["w_out"], ws, S)
    return fd.prepare_evict(s["k"], s["v"], s["w"], s["seqlens"], c["keep"], c["recent"], s["k_out"], s["v_out"],
                            s["w_out"], s["kept"], s["new_seqlens"])


def run(state):
    op = state["case"]["op"]
    if own:
        call = state.get("call")
        if call is None:
            call = state["call"] = _own_call(state)
        call()
        if op == "append":
            return _append_outputs(state)
        if op == "evict":
            return _evict_outputs(state)
        r = dict(out=state["out"], lse=state["lse"])
        if op == "weights":
            r["weights"] = state["w_out"]
        return r
    return {"block": _plain_block, "append": _plain_append, "weights": _plain_weights, "evict": _plain_evict}[op](state)


# --------------------------------------------------------------------- work --

def work(case):
    lens = _lengths(case)
    B, Hkv, D = case["B"], case["Hkv"], case["D"]
    tokens = sum(lens) * Hkv                                  # cached (token, kv head) pairs
    if case["op"] in ("block", "weights"):
        rows = B * case["q_len"] * case["Hq"]
        moved = rows * D * 2 + rows * D * 4 + rows * 4 + B * 4
        flops = 4 * sum(lens) * case["q_len"] * case["Hq"] * D
        if case["op"] == "weights":
            return dict(bytes=moved + tokens * (2 * D * 2 + 8), flops=flops)
        blocks = sum(-(-n // case["T"]) for n in lens) * Hkv
        return dict(bytes=moved + tokens * 2 * D + blocks * 8, flops=flops)
    if case["op"] == "append":
        T = case["T"]
        new = sum(_news(case, lens)) * Hkv
        blocks = sum(-(-n // T) - (n - m) // T for n, m in zip(lens, _news(case, lens))) * Hkv
        return dict(bytes=new * 2 * D * 3 + blocks * 8, flops=new * 2 * D * 3)
    kept = sum(min(n, case["keep"]) for n in lens) * Hkv
    return dict(bytes=tokens * 4 + kept * (2 * 2 * D * 2 + 8) + B * 4, flops=tokens * 4)


# -------------------------------------------------- the definition in 64 bits --

def _e4m3_values():
    v = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = math.nan if (c & 127) == 127 else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        v.append(-x if c & 128 else x)
    return torch.tensor(v, dtype=torch.float64, device="cuda")


def _values64(codes, kv):
    if kv == "e4m3":
        return _e4m3_values()[codes.long()]
    return torch.where(codes > 127, codes.double() - 256.0, codes.double())


def _round64(y, kv):
    """Values to the nearest representable ones, half to even."""
    if kv == "int8":
        return torch.round(y).clamp(-127, 127)
    e = torch.frexp(y).exponent.double() - 1                  # 2^e <= |y| < 2^(e+1)
    step = torch.exp2(e.clamp_min(-6) - 3)
    return (torch.round(y / step) * step).clamp(-448, 448)


def _scale64(a, kv):
    m, e = torch.frexp(a / RANGE[kv])
    return torch.ldexp(torch.ceil(m * 256) / 256, e)


def _row(s, name, b, h, n):
    """First n tokens of one (sequence, kv head) from array `name`: [n, ...]."""
    c = s["case"]
    if not c.get("page"):
        return s[name][b, h, :n]
    ps, t = c["page"], torch.arange(n, device="cuda")
    page = s["table"][b, t // ps].long()
    return s[name][page, h, t % ps] if c["layout"] == "HND" else s[name][page, t % ps, h]


def _row_scale(s, name, b, h, n):
    c = s["case"]
    t = torch.arange(n, device="cuda")
    if not c["page"]:
        return s[name][b, h, t // c["T"]].double()
    ps = c["page"]
    return s[name][s["table"][b, t // ps].long(), h, (t % ps) // c["T"]].double()


def exact(case, seed):
    s = prepare(case, seed)
    op, B, Hkv, D = case["op"], case["B"], case["Hkv"], case["D"]
    lens = s["seqlens"].tolist()
    if op == "evict":
        keep, recent = case["keep"], case["recent"]
        r = {a: torch.zeros((B, Hkv, keep, D), dtype=torch.float64, device="cuda") for a in ("k", "v")}
        r["weights"] = torch.zeros((B, Hkv, keep), dtype=torch.float64, device="cuda")
        r["kept"] = torch.full((B, Hkv, keep), -1, dtype=torch.int64, device="cuda")
        r["seqlens"] = torch.tensor([min(n, keep) for n in lens], device="cuda")
        for b, n in enumerate(lens):
            for h in range(Hkv):
                take = torch.arange(n, device="cuda")
                if n > keep:
                    older = s["w"][b, h, :n - recent].double()
                    heaviest = torch.argsort(-older, stable=True)[:keep - recent]
                    take = torch.cat([heaviest.sort().values, take[n - recent:]])
                m = take.numel()
                r["kept"][b, h, :m] = take
                r["weights"][b, h, :m] = s["w"][b, h][take].double()
                for a in ("k", "v"):
                    r[a][b, h, :m] = s[a][b, h][take].double()
        return r
    if op == "append":
        T, kv = case["T"], case["kv"]
        news = s["new_lens"].tolist()
        kind = torch.float64 if kv == "e4m3" else torch.int64
        r = {}
        for name in ("k", "v"):
            codes = _values64(s[name], kv)
            scale = s[name + "s"].double()
            for b in range(B):
                start = lens[b] - news[b]
                lo, hi = start // T * T, -(-lens[b] // T) * T
                x = torch.zeros((Hkv, hi - lo, D), dtype=torch.float64, device="cuda")
                x[:, start - lo:lens[b] - lo] = s[name + "_new"][b, :news[b]].double().transpose(0, 1)
                sc = _scale64(x.view(Hkv, -1, T * D).abs().amax(2), kv)
                if start > lo:
                    was = torch.stack([_row_scale(s, name + "s", b, h, lo + 1)[lo] for h in range(Hkv)])
                    sc[:, 0] = torch.maximum(sc[:, 0], was)
                    older = torch.stack([_values64(_row(s, name, b, h, start)[lo:], kv) for h in range(Hkv)])
                    x[:, :start - lo] = older * was[:, None, None]
                y = _round64(x / sc.clamp_min(1e-300).repeat_interleave(T, 1)[:, :, None], kv)
                for h in range(Hkv):
                    if not case["page"]:
                        codes[b, h, lo:lens[b]] = y[h, :lens[b] - lo]
                        scale[b, h, lo // T:hi // T] = sc[h]
                        continue
                    t = torch.arange(lo, lens[b], device="cuda")
                    page, off = s["table"][b, t // case["page"]].long(), t % case["page"]
                    if case["layout"] == "HND":
                        codes[page, h, off] = y[h, :lens[b] - lo]
                    else:
                        codes[page, off, h] = y[h, :lens[b] - lo]
                    t = torch.arange(lo, hi, T, device="cuda")
                    scale[s["table"][b, t // case["page"]].long(), h, t % case["page"] // T] = sc[h]
            r[name], r[name + "_scale"] = codes.to(kind), scale
        return r
    q_len, Hq = case["q_len"], case["Hq"]
    g = Hq // Hkv
    out = torch.zeros((B, q_len, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, q_len, Hq), -math.inf, dtype=torch.float64, device="cuda")
    total = torch.zeros((B, Hkv, case["Lmax"]), dtype=torch.float64, device="cuda") if op == "weights" else None
    for b in range(B):
        for h in range(Hkv):
            n = lens[b]
            if op == "block":
                k, v = (_values64(_row(s, a, b, h, n), case["kv"]) * _row_scale(s, a + "s", b, h, n)[:, None]
                        for a in ("k", "v"))
            else:
                k, v = s["k"][b, h, :n].double(), s["v"][b, h, :n].double()
                total[b, h, :n] = s["w"][b, h, :n].double()
            for j in range(q_len):
                m = n - (q_len - 1 - j)
                if m < 1:
                    continue
                z = (k[:m] @ s["q"][b, j, h * g:(h + 1) * g].double().T) / math.sqrt(D)      # [m, g]
                e = torch.logsumexp(z, 0)
                p = torch.exp(z - e)
                lse[b, j, h * g:(h + 1) * g] = e
                out[b, j, h * g:(h + 1) * g] = p.T @ v[:m]
                if op == "weights":
                    total[b, h, :m] += p.sum(1)
    r = dict(out=out, lse=lse)
    if op == "weights":
        r["weights"] = total
    return r
