"""fd_evict against the definition: kept positions, keys, values and totals
equal it exactly. And the operators together: score, evict, hold in 8 bits,
go on decoding."""
import math
import os
import subprocess
import sys

import pytest
import torch

import compress_ref as ref
import decode_attention_07_b200 as fd

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    torch.cuda.set_device(0)
    yield
    assert fd.fd_device_status() == 0


def bits(t):
    return t.contiguous().view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


def check(w, seqlens, keep, recent, D=64, out_len=None, seed=0):
    """w [B,Hkv,L] totals; keys and values random bits (NaN patterns too)."""
    B, Hkv, L = w.shape
    g = torch.Generator(device="cuda").manual_seed(seed)
    k, v = (torch.randint(-2 ** 15, 2 ** 15, (B, Hkv, L, D), generator=g, device="cuda", dtype=torch.int16)
            .view(torch.bfloat16) for _ in "kv")
    n_out = keep if out_len is None else out_len
    ko, vo = (torch.full((B, Hkv, n_out, D), 9.0, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    wo = torch.full((B, Hkv, n_out), 9.0, device="cuda")
    kept = torch.full((B, Hkv, keep), 77, dtype=torch.int32, device="cuda")
    so = torch.full((B,), 77, dtype=torch.int32, device="cuda")
    lens = torch.tensor(seqlens, dtype=torch.int32, device="cuda")
    fd.fd_evict(k, v, w, lens, keep, recent, ko, vo, wo, kept, so)
    torch.cuda.synchronize()
    for b in range(B):
        n = min(max(seqlens[b], 0), L)
        m = min(n, keep)
        assert so[b] == m
        for h in range(Hkv):
            want = ref.evict(w[b, h, :n].tolist(), n, keep, recent)
            got = kept[b, h].tolist()
            assert got == want + [-1] * (keep - m), f"b={b} h={h} n={n} keep={keep} recent={recent}"
            idx = torch.tensor(want, dtype=torch.int64, device="cuda")
            for src, dst in ((k, ko), (v, vo)):
                assert torch.equal(bits(dst[b, h, :m]), bits(src[b, h][idx]))
                assert torch.all(dst[b, h, m:] == 9.0)
            assert torch.equal(bits(wo[b, h, :m]), bits(w[b, h][idx]))
            assert torch.all(wo[b, h, m:] == 0)


def totals(B, Hkv, L, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.exp(2 * torch.randn((B, Hkv, L), generator=g, device="cuda"))


@pytest.mark.parametrize("L,keep,recent", [(1, 1, 0), (1, 1, 1), (2, 1, 0), (2, 1, 1), (100, 99, 0), (100, 1, 0),
                                           (513, 256, 100), (1000, 64, 64), (4097, 1000, 17), (9000, 8999, 3),
                                           (9001, 4500, 0)])
@pytest.mark.parametrize("D", [64, 128])
def test_sizes(L, keep, recent, D):
    w = totals(3, 2, L, L)
    check(w, [L, L // 2, max(L - 1, 0)], keep, recent, D)


@pytest.mark.parametrize("B,Hkv", [(1, 1), (1, 8), (2, 32)])
def test_clusters_of_blocks(B, Hkv):
    """Few long rows: several blocks share a row (slices kept in registers,
    and, at 140001 tokens, read again)."""
    L = 140001 if B * Hkv == 1 else 20011
    check(totals(B, Hkv, L, 3), [L - 7] * B, L // 4, 999)


def test_a_long_row_in_one_block():
    """Many rows, so one block each, with slices longer than its registers hold."""
    w = totals(1, 200, 9999, 4)
    check(w, [9999], 2500, 13)


@pytest.mark.parametrize("kind", ["equal", "two", "bf16", "dense bits", "negative", "special"])
@pytest.mark.parametrize("L", [700, 20000])
def test_ties_and_special_totals(kind, L):
    B, Hkv = 2, 2
    g = torch.Generator(device="cuda").manual_seed(5)
    if kind == "equal":
        w = torch.zeros((B, Hkv, L), device="cuda")
    elif kind == "two":
        w = (torch.rand((B, Hkv, L), generator=g, device="cuda") < 0.3).float()
    elif kind == "bf16":
        w = totals(B, Hkv, L, 6).to(torch.bfloat16).float()
    elif kind == "dense bits":                       # totals that differ in their last bits only
        w = (torch.randint(0, 3000, (B, Hkv, L), generator=g, device="cuda", dtype=torch.int32) + 0x3F800000).view(
            torch.float32)
    elif kind == "negative":
        w = torch.randn((B, Hkv, L), generator=g, device="cuda")
    else:
        pick = torch.tensor([0.0, -0.0, math.nan, math.inf, -math.inf, 1e-42, -1e-42, 3.4e38, -3.4e38], device="cuda")
        w = pick[torch.randint(0, 9, (B, Hkv, L), generator=g, device="cuda")]
    for keep, recent in ((L // 3, 0), (L // 2, 50), (L - 1, 0), (5, 5)):
        check(w, [L, L - 100], keep, recent, seed=keep)


def test_short_empty_and_clamped_rows():
    w = totals(6, 2, 300, 7)
    check(w, [0, 100, 101, 300, 900, -4], 100, 20, out_len=150)
    check(w, [0, 100, 101, 300, 900, -4], 400, 20, out_len=401)      # a budget beyond the cache


def test_offsets_past_32_bits():
    """A cache of more than 2^32 elements: only the last sequence is long."""
    B, Hkv, L, D = 33, 8, 131072, 128
    k = torch.zeros((B, Hkv, L, D), dtype=torch.bfloat16, device="cuda")
    k[-1] = torch.randn((Hkv, L, D), device="cuda").to(torch.bfloat16)
    v = torch.zeros_like(k)
    v[-1] = k[-1] + 1
    w = totals(B, Hkv, L, 8)
    lens = torch.full((B,), 3, dtype=torch.int32, device="cuda")
    lens[-1] = L
    ko, vo, wo, kept, so = fd.evict(k, v, w, lens, 5000, 100)
    torch.cuda.synchronize()
    assert so.tolist() == [3] * (B - 1) + [5000]
    for h in (0, Hkv - 1):
        idx = torch.tensor(ref.evict(w[-1, h].tolist(), L, 5000, 100), device="cuda")
        assert torch.equal(kept[-1, h].long(), idx)
        assert torch.equal(ko[-1, h], k[-1, h][idx]) and torch.equal(vo[-1, h], v[-1, h][idx])
        assert torch.equal(wo[-1, h], w[-1, h][idx])


def test_in_a_graph_and_refusals():
    w = totals(2, 2, 1000, 9)
    k = torch.randn((2, 2, 1000, 64), device="cuda").to(torch.bfloat16)
    lens = torch.tensor([1000, 500], dtype=torch.int32, device="cuda")
    outs = fd.evict(k, k, w, lens, 300, 10)
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    side = torch.cuda.Stream()
    call = fd.prepare_evict(k, k, w, lens, 300, 10, *outs, stream=side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    for t in outs:
        t.zero_()
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    for bad in (dict(keep=0), dict(recent=301), dict(out_len=299)):
        a = dict(keep=300, recent=10)
        a.update(bad)
        with pytest.raises((ValueError, fd.FdError)):
            fd.evict(k, k, w, lens, **a)
    with pytest.raises(fd.FdError):                  # in place
        fd.fd_evict(k, k, w, lens, 1000, 10, k, torch.empty_like(k), torch.empty_like(w),
                    torch.empty((2, 2, 1000), dtype=torch.int32, device="cuda"), torch.empty_like(lens))
    torch.cuda.synchronize()


def test_caches_without_room():
    """max_len = 0: rows without tokens, nothing written past the outputs."""
    dev = dict(device="cuda")
    k = torch.zeros((2, 2, 0, 64), dtype=torch.bfloat16, **dev)
    w = torch.zeros((2, 2, 0), **dev)
    lens = torch.tensor([0, 5], dtype=torch.int32, **dev)
    q = torch.ones((2, 4, 64), dtype=torch.bfloat16, **dev)
    ko, vo, wo, kept, so = fd.evict(k, k, w, lens, 3, 1)
    out, lse, total = fd.decode_weights(q, k, k, lens, 0.1)
    k8, v8, ks, vs = fd.empty_quant_block_cache(2, 2, 0, 64, 16)
    fd.fd_quant_append(q.view(2, 1, 4, 64)[:, :, :2].contiguous(), q.view(2, 1, 4, 64)[:, :, :2].contiguous(), k8, v8, ks,
                       vs, "int8", 16, lens)
    out8, lse8 = fd.decode_quant_block(q, k8, v8, ks, vs, "int8", 16, lens, 0.1)
    torch.cuda.synchronize()
    assert so.tolist() == [0, 0] and torch.all(kept == -1) and torch.all(wo == 0) and total.numel() == 0
    for o, l in ((out, lse), (out8, lse8)):
        assert torch.all(o == 0) and torch.isneginf(l).all()


def test_failed_launches_are_reported():
    """With the library's host-side injection every entry point returns
    FD_ERR_LAUNCH, writes nothing and leaves the device status clean."""
    code = """
import torch, decode_attention_07_b200 as fd
dev = dict(device="cuda")
q = torch.ones((1, 4, 64), dtype=torch.bfloat16, **dev)
k = torch.ones((1, 2, 100, 64), dtype=torch.bfloat16, **dev)
lens = torch.tensor([100], dtype=torch.int32, **dev)
w = torch.full((1, 2, 100), 7.0, **dev)
k8, v8, ks, vs = fd.empty_quant_block_cache(1, 2, 100, 64, 16)
outs = [torch.full(s, 7.0, **dev) for s in ((1, 4, 64), (1, 4))]
ko, vo, wo = torch.full_like(k, 7.0), torch.full_like(k, 7.0), torch.full_like(w, 7.0)
kept, so = torch.full((1, 2, 10), 7, dtype=torch.int32, **dev), torch.full((1,), 7, dtype=torch.int32, **dev)
ws = torch.zeros(fd.fd_weights_workspace_bytes(1, 1, 4, 2, 64, 100, 1), dtype=torch.uint8, **dev)
calls = [lambda: fd.fd_decode_quant_block(q, k8, v8, ks, vs, "int8", 16, lens, 0.1, *outs, None, 1),
         lambda: fd.fd_quant_append(k.transpose(1, 2), k.transpose(1, 2), k8, v8, ks, vs, "int8", 16, lens),
         lambda: fd.fd_decode_weights(q, k, k, lens, 0.1, *outs, None, w, ws, 1),
         lambda: fd.fd_evict(k, k, w, lens, 10, 2, ko, vo, wo, kept, so)]
for call in calls:
    try:
        call()
    except fd.FdError as e:
        assert e.code == -9, e
    else:
        raise AssertionError("no error")
torch.cuda.synchronize()
assert fd.fd_device_status() == 0
assert all(torch.all(t == 7) for t in (*outs, w, ko, vo, wo, kept, so)) and torch.all(k8 == 0) and torch.all(ks == 0)
"""
    env = dict(os.environ, FD_TEST_FAIL_LAUNCH="1")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("kv", ["e4m3", "int8"])
def test_score_evict_quantise_decode(kv):
    """The operators as they are used together: a prompt's last queries score
    its tokens, the cache is cut to a budget, what is kept moves into an 8-bit
    block-scaled cache, and decoding goes on there one token at a time."""
    B, Hkv, g, D, L, T, q_len = 3, 2, 4, 128, 700, 32, 4
    keep, recent, steps, scale = 200, 32, 5, D ** -0.5
    seqlens = [700, 150, 433]
    gen = torch.Generator(device="cuda").manual_seed(10)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)

    k, v, q = normal(B, Hkv, L, D), normal(B, Hkv, L, D), normal(B, q_len, g * Hkv, D)
    lens = torch.tensor(seqlens, dtype=torch.int32, device="cuda")
    _, _, w = fd.decode_weights(q, k, v, lens, scale)
    r = ref.attention(q, k, v, seqlens, scale)
    ko, vo, wo, kept, so = fd.evict(k, v, w, lens, keep, recent)
    k8, v8, ks, vs = fd.empty_quant_block_cache(B, Hkv, keep + steps, D, T)
    fd.fd_quant_append(ko.transpose(1, 2), vo.transpose(1, 2), k8, v8, ks, vs, kv, T, so, so)
    torch.cuda.synchronize()
    k64, v64 = (torch.zeros((B, Hkv, keep + steps, D), dtype=torch.float64, device="cuda") for _ in "kv")
    sk, sv = (torch.zeros(ks.shape, dtype=torch.float64, device="cuda") for _ in "kv")
    now = [min(n, keep) for n in seqlens]
    kk, vv = (torch.zeros((B, keep, Hkv, D), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    for b, n in enumerate(seqlens):
        for h in range(Hkv):
            # the library's own totals decide; they are the definition's to 2^-10
            assert torch.allclose(w[b, h, :n].double(), r[2][b, h, :n], rtol=2.0 ** -10, atol=0)
            idx = torch.tensor(ref.evict(w[b, h, :n].tolist(), n, keep, recent), device="cuda")
            kk[b, :now[b], h], vv[b, :now[b], h] = k[b, h][idx], v[b, h][idx]
    ref.append(k64, sk, kk, now, now, T, kv)
    ref.append(v64, sv, vv, now, now, T, kv)
    lens = so.clone()
    for i in range(steps):
        kn, vn, qn = normal(B, 1, Hkv, D) * (1 + i), normal(B, 1, Hkv, D) * (1 + i), normal(B, g * Hkv, D)
        lens += 1
        now = [n + 1 for n in now]
        fd.fd_quant_append(kn, vn, k8, v8, ks, vs, kv, T, lens)
        out, lse = fd.decode_quant_block(qn, k8, v8, ks, vs, kv, T, lens, scale)
        torch.cuda.synchronize()
        ref.append(k64, sk, kn, now, [1] * B, T, kv)
        ref.append(v64, sv, vn, now, [1] * B, T, kv)
        assert torch.equal(ref.values(k8, kv), k64) and torch.equal(ref.values(v8, kv), v64)
        K, V = (c * s.repeat_interleave(T, 2)[:, :, :keep + steps, None] for c, s in ((k64, sk), (v64, sv)))
        rr = ref.attention(qn.view(B, 1, g * Hkv, D), K, V, now, scale)
        ref.close(out, lse, rr, V, D, 2.0 ** -18, f"step {i}")
