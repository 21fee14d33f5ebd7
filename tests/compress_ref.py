"""Plain 64-bit definitions of the cache-compression operators, for their
tests: block-scaled 8-bit attention, the append that writes such a cache,
attention weights per token, eviction. Straight loops over sequences and
heads; no code shared with the library or the package."""
import math

import torch

RANGE = {"e4m3": 448.0, "int8": 127.0}


def e4m3_values(device):
    v = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = math.nan if (c & 127) == 127 else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        v.append(-x if c & 128 else x)
    return torch.tensor(v, dtype=torch.float64, device=device)


def values(codes, kv):
    """Code bytes (uint8) to the numbers they stand for."""
    if kv == "e4m3":
        return e4m3_values(codes.device)[codes.long()]
    return torch.where(codes > 127, codes.double() - 256.0, codes.double())


def nearest(y, kv):
    """Numbers to the nearest representable ones, half to even."""
    if kv == "int8":
        return torch.round(y).clamp(-127, 127)
    e = torch.frexp(y).exponent.double() - 1
    step = torch.exp2(e.clamp_min(-6) - 3)
    return (torch.round(y / step) * step).clamp(-448, 448)


def codes_of(v, kv):
    """Representable numbers to code bytes (the positive zero for zeros)."""
    if kv == "int8":
        return v.to(torch.int8).view(torch.uint8)
    table = e4m3_values(v.device)[:127]                         # 0 .. 448, ascending
    mag = torch.searchsorted(table, v.abs().contiguous())
    return torch.where(v < 0, mag + 128, mag).to(torch.uint8)


def block_scale(a, kv):
    """a / R rounded up to 8 significant bits."""
    m, e = torch.frexp(a.double() / RANGE[kv])
    return torch.ldexp(torch.ceil(m * 256) / 256, e).double()


def append(codes, scale, new, seqlens, news, T, kv):
    """In place on float64 values `codes` [B,Hkv,L,D] (not bytes) and float64
    scales [B,Hkv,nblk]; new [B,n,Hkv,D]."""
    B, Hkv, L, D = codes.shape
    for b in range(B):
        n, end = int(news[b]), int(seqlens[b])
        start = end - n
        for h in range(Hkv):
            lo, hi = max(start, 0), min(end, L)
            for blk in range(lo // T, -(-hi // T) if hi > lo else lo // T):
                t0, t1 = max(blk * T, lo), min(blk * T + T, hi)
                x = new[b, t0 - start:t1 - start, h].double()
                s = block_scale(x.abs().max(), kv)
                if blk * T < lo:
                    was = scale[b, h, blk].clone()
                    s = torch.maximum(s, was)
                    if s > was:
                        codes[b, h, blk * T:lo] = nearest(codes[b, h, blk * T:lo] * was / s, kv)
                scale[b, h, blk] = s
                codes[b, h, t0:t1] = nearest(x / s, kv) if s > 0 else 0.0


def attention(q, k, v, seqlens, scale):
    """q [B,q_len,Hq,D], k, v [B,Hkv,L,D] float64, seqlens ints. Returns out,
    lse, token weights [B,Hkv,L], and per (b, j, head) the error unit of the
    logits: max_t sum_d |q k| * scale."""
    B, q_len, Hq, D = q.shape
    Hkv, L = k.shape[1], k.shape[2]
    g = Hq // Hkv
    dev = q.device
    out = torch.zeros((B, q_len, Hq, D), dtype=torch.float64, device=dev)
    lse = torch.full((B, q_len, Hq), -math.inf, dtype=torch.float64, device=dev)
    wts = torch.zeros((B, Hkv, L), dtype=torch.float64, device=dev)
    unit = torch.zeros((B, q_len, Hq), dtype=torch.float64, device=dev)
    for b in range(B):
        n = min(max(int(seqlens[b]), 0), L)
        for j in range(q_len):
            m = n - (q_len - 1 - j)
            if m < 1:
                continue
            for h in range(Hkv):
                hs = slice(h * g, (h + 1) * g)
                qq, kk = q[b, j, hs].double(), k[b, h, :m].double()
                z = kk @ qq.T * scale
                e = torch.logsumexp(z, 0)
                p = torch.exp(z - e)
                lse[b, j, hs] = e
                out[b, j, hs] = p.T @ v[b, h, :m].double()
                wts[b, h, :m] += p.sum(1)
                unit[b, j, hs] = (kk.abs() @ qq.abs().T * abs(scale)).max(0).values
    return out, lse, wts, unit


def close(out, lse, ref, v, D, p_eps, what):
    """Hold kernel outputs to the 64-bit ones. A logit is a sum of D exact
    products accumulated in fp32, scaled by a few fp32 factors: off by at most
    dz = (D + 8) 2^-24 unit, plus 2^-22 of its own size for the base-2
    exponential's argument. p_eps: the relative rounding of P and of the
    hardware exponential. Each weight is then off by (2 dz + p_eps) relative
    (once for itself, once through the log-sum-exp), and out, a convex
    combination of value rows, by twice that times the largest |v|."""
    r_out, r_lse, _, unit = ref
    out, lse = out.double().view(r_out.shape), lse.double().view(r_lse.shape)
    dz = (D + 8) * 2.0 ** -24 * unit + 2.0 ** -22 * unit
    vmax = v.double().abs().nan_to_num(0.0).amax(dim=(1, 2, 3))[:, None, None]
    tol = vmax * 2 * (2 * dz + p_eps)
    assert torch.isfinite(out).all(), what
    err = (out - r_out).abs().amax(3)
    assert (err <= tol).all(), f"{what}: out error {err.max():.3e}, {(err / tol.clamp_min(1e-300)).max():.2f} of the bound"
    empty = torch.isneginf(r_lse)
    assert torch.equal(torch.isneginf(lse), empty), what
    ltol = dz + 2.0 ** -20 * r_lse.abs().clamp_min(1.0)
    lerr = torch.where(empty, torch.zeros_like(lse), lse - r_lse).abs()
    assert (lerr <= ltol).all(), f"{what}: lse error {lerr.max():.3e}"
    return dz


def evict(w, n, keep, recent):
    """Kept positions of one row of n tokens with totals w (a list of floats)."""
    if n <= keep:
        return list(range(n))
    m = n - recent
    order = sorted(range(m), key=lambda t: (math.isnan(w[t]), -w[t] if not math.isnan(w[t]) else 0.0, t))
    return sorted(order[:keep - recent]) + list(range(m, n))
