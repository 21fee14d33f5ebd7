"""The cache-compression entry points on the host (no GPU): argument checks
run before any CUDA call and return their own codes; workspace sizes."""
import ctypes

import pytest
import torch

import decode_attention_07_b200 as fd

HAS_GPU = torch.cuda.is_available()


@pytest.fixture(scope="module")
def mem():
    buf = (ctypes.c_uint8 * (1 << 16))()
    base = (ctypes.addressof(buf) + 255) // 256 * 256
    return buf, base


def test_block_attention_refusals(mem):
    L, p = fd.lib(), ctypes.c_void_p(mem[1])
    odd = ctypes.c_void_p(mem[1] + 2)

    def c(B=1, q_len=1, Hq=4, Hkv=2, D=64, n=64, T=16, kv=1, q=p, k=p, v=p, ks=p, vs=p, s=p, out=p, lse=p, ws=p, wsb=4096,
          S=1):
        return L.fd_decode_quant_block(B, q_len, Hq, Hkv, D, n, T, kv, q, k, v, ks, vs, s, 0.1, out, lse, ws, wsb, S, None)
    for T in (0, 8, 24, 256, -16):
        assert c(T=T) == -2
    assert c(kv=0) == -2 and c(kv=3) == -2 and c(q_len=0) == -2 and c(q_len=17) == -2 and c(B=0) == -2
    assert c(Hq=5) == -3 and c(Hq=34) == -3 and c(Hq=8, q_len=5) == -3
    assert c(D=96) == -4
    assert c(ks=None) == -1 and c(vs=None) == -1 and c(q=None) == -1 and c(out=None) == -1
    assert c(ks=odd) == -5 and c(k=ctypes.c_void_p(mem[1] + 8)) == -5
    assert c(S=-1) == -7 and c(S=2, ws=None) == -6
    if not HAS_GPU:
        assert c() == -8

    def paged(T=16, ps=16, pages=8, per=4, layout=0, bt=p, ks=p, kv=1):
        return L.fd_decode_quant_block_paged(1, 1, 4, 2, 64, ps, pages, per, layout, T, kv, p, p, p, ks, p, bt, p, 0.1, p, p,
                                             p, 4096, 1, None)
    assert paged(T=32) == -2 and paged(ps=8) == -2 and paged(ps=24) == -2 and paged(per=3) == -2 and paged(layout=2) == -2
    assert paged(bt=None) == -1 and paged(ks=None) == -1 and paged(bt=odd) == -5 and paged(kv=9) == -2
    assert paged(ps=4096, pages=1 << 20) == -2          # flattened coordinate past int32
    if not HAS_GPU:
        assert paged() == -8


def test_append_refusals(mem):
    L, p = fd.lib(), ctypes.c_void_p(mem[1])

    def c(B=1, n=1, Hkv=2, D=64, len_=64, T=16, kv=1, k=p, v=p, sb=128, st=128, sh=64, nl=None, s=p, kc=p, ks=p):
        return L.fd_quant_append(B, n, Hkv, D, len_, T, kv, k, v, sb, st, sh, nl, s, kc, p, ks, p, None)
    assert c(n=-1) == -2 and c(T=8) == -2 and c(kv=0) == -2 and c(B=0) == -2 and c(len_=-1) == -2 and c(D=32) == -4
    assert c(k=None) == -1 and c(s=None) == -1 and c(kc=None) == -1 and c(ks=None) == -1
    assert c(st=4) == -5 and c(sb=3) == -5 and c(sh=1) == -5
    assert c(k=ctypes.c_void_p(mem[1] + 8)) == -5 and c(nl=ctypes.c_void_p(mem[1] + 1)) == -5
    assert c(n=0, k=None, v=None) == 0 and c(len_=0, k=None) == 0      # nothing to do
    if not HAS_GPU:
        assert c() == -8

    def paged(T=16, ps=16, bt=p):
        return L.fd_quant_append_paged(1, 1, 2, 64, ps, 8, 4, 0, T, 1, p, p, 128, 128, 64, None, bt, p, p, p, p, p, None)
    assert paged(T=32) == -2 and paged(ps=20) == -2 and paged(bt=None) == -1
    if not HAS_GPU:
        assert paged() == -8


def test_weights_refusals_and_workspace(mem):
    L, p = fd.lib(), ctypes.c_void_p(mem[1])
    big = 1 << 15
    other = ctypes.c_void_p(mem[1] + 64)

    def c(B=1, q_len=1, Hq=4, Hkv=2, D=64, n=64, q=p, wi=None, wo=p, ws=p, wsb=big, S=1):
        return L.fd_decode_weights(B, q_len, Hq, Hkv, D, n, q, p, p, p, 0.1, p, p, wi, wo, ws, wsb, S, None)
    assert c(q_len=0) == -2 and c(Hq=34) == -3 and c(Hq=16, q_len=3) == -3 and c(D=65) == -4 and c(n=-1) == -2
    assert c(wo=None) == -1 and c(q=None) == -1 and c(wo=ctypes.c_void_p(mem[1] + 1)) == -5
    assert c(ws=None) == -6 and c(wsb=100) == -6 and c(S=-1) == -7
    assert c(wi=other) == -14                               # totals that overlap in part
    if not HAS_GPU:
        assert c() == -8 and c(wi=p) == -8
    # logits [B, Hkv, Lmax, columns (even above one)], 256-byte aligned, then fd_decode_multi's workspace
    for B, q_len, Hq, Hkv, D, n, S, cols in ((1, 1, 4, 4, 64, 100, 7, 1), (3, 2, 12, 4, 128, 33, 1, 6),
                                             (2, 1, 6, 2, 128, 1000, 20, 4)):
        want = (B * Hkv * n * cols * 4 + 255) // 256 * 256 + fd.fd_workspace_bytes(B, Hq * q_len, Hkv, D, n, S)
        assert fd.fd_weights_workspace_bytes(B, q_len, Hq, Hkv, D, n, S) == want
    assert fd.fd_weights_workspace_bytes(1, 0, 4, 4, 64, 10, 1) == 0


def test_evict_refusals(mem):
    L, base = fd.lib(), mem[1]
    at = [ctypes.c_void_p(base + i * 4096) for i in range(10)]

    def c(B=1, Hkv=1, D=64, n=16, keep=8, recent=2, out=8, k=at[0], v=at[1], w=at[2], s=at[3], ko=at[4], vo=at[5],
          wo=at[6], kept=at[7], so=at[8]):
        return L.fd_evict(B, Hkv, D, n, keep, recent, out, k, v, w, s, ko, vo, wo, kept, so, None)
    assert c(keep=0) == -2 and c(recent=9) == -2 and c(recent=-1) == -2 and c(out=7) == -2 and c(B=0) == -2
    assert c(D=32) == -4 and c(k=None) == -1 and c(w=None) == -1 and c(kept=None) == -1 and c(so=None) == -1
    assert c(ko=ctypes.c_void_p(base + 4 * 4096 + 8)) == -5
    assert c(ko=at[0]) == -14 and c(vo=ctypes.c_void_p(base + 16)) == -14      # in place: refused
    assert c(wo=at[2]) == -14 and c(kept=at[6]) == -14 and c(so=at[3]) == -14 and c(vo=at[4]) == -14
    if not HAS_GPU:
        assert c() == -8 and c(n=0, k=None, v=None, w=None) == -8


def test_bindings_refuse_host_tensors():
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    k8 = torch.zeros(1, 2, 64, 64, dtype=torch.uint8)
    sc = torch.zeros(1, 2, 4)
    lens = torch.zeros(1, dtype=torch.int32)
    k = torch.zeros(1, 2, 64, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fd.fd_decode_quant_block(q, k8, k8, sc, sc, "e4m3", 16, lens, 0.1, q.float(), sc[0, :, 0])
    with pytest.raises(ValueError):
        fd.fd_quant_append(k.transpose(1, 2), k.transpose(1, 2), k8, k8, sc, sc, "e4m3", 16, lens)
    with pytest.raises(ValueError):
        fd.fd_decode_weights(q, k, k, lens, 0.1, q.float(), sc[0, :, 0], None, torch.zeros(1, 2, 64), None)
    with pytest.raises(ValueError):
        fd.fd_evict(k, k, torch.zeros(1, 2, 64), lens, 8, 2, k, k, torch.zeros(1, 2, 64), torch.zeros(1, 2, 8).int(), lens)
