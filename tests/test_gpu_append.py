"""fd_quant_append and fd_quant_append_paged against the 64-bit definition:
codes and scales equal it exactly (scales that the append sets have 8
significant bits, so every quotient rounds as the real number does)."""
import pytest
import torch

import compress_ref as ref
import decode_attention_07_b200 as fd
from test_gpu_block import to_pages

pytestmark = pytest.mark.gpu
KV = ["e4m3", "int8"]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    torch.cuda.set_device(0)
    yield
    assert fd.fd_device_status() == 0


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def tokens(B, n, Hkv, D, seed, sigma=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn((B, n, Hkv, D), generator=g, device="cuda") * sigma).to(torch.bfloat16) for _ in range(2)]


class Model:
    """A cache and its 64-bit twin; both start with garbage, which stays
    wherever no token goes."""

    def __init__(self, B, Hkv, L, D, T, kv, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.T, self.kv, self.L = T, kv, L
        nblk = -(-L // T)
        self.codes = [torch.randint(0, 127, (B, Hkv, L, D), generator=g, device="cuda", dtype=torch.uint8) for _ in "kv"]
        self.scales = [torch.full((B, Hkv, nblk), 3.7, device="cuda") for _ in "kv"]
        self.vals = [ref.values(c, kv) for c in self.codes]
        self.s64 = [s.double() for s in self.scales]

    def append(self, new, seqlens, new_lens=None, run=True):
        n = new[0].shape[1]
        news = [min(max(x, 0), n) for x in new_lens] if new_lens is not None else [n] * len(seqlens)
        if run:
            fd.fd_quant_append(new[0], new[1], self.codes[0], self.codes[1], self.scales[0], self.scales[1], self.kv,
                               self.T, ints(seqlens), None if new_lens is None else ints(new_lens))
        for v, s, x in zip(self.vals, self.s64, new):
            ref.append(v, s, x, seqlens, news, self.T, self.kv)

    def check(self, what=""):
        torch.cuda.synchronize()
        for a, c, v, s, t in zip("kv", self.codes, self.vals, self.scales, self.s64):
            assert torch.equal(s.double(), t), f"{what}: {a} scales, {(s.double() != t).sum()} differ"
            got = ref.values(c, self.kv)
            assert torch.equal(got, v), f"{what}: {a} codes, {(got != v).sum()} of {v.numel()} differ"


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("T", [16, 32, 64, 128])
@pytest.mark.parametrize("D", [64, 128])
def test_a_prompt_a_chunk_then_single_tokens(kv, T, D):
    B, Hkv, L = 3, 2, 400
    m = Model(B, Hkv, L, D, T, kv)
    prompt = [200, 1, T + 3]
    m.append(tokens(B, 200, Hkv, D, 1), prompt, prompt)
    m.check("prompt")
    lens = [x + 37 for x in prompt]
    m.append(tokens(B, 37, Hkv, D, 2, 0.7), lens)
    m.check("chunk")
    for i in range(6):     # growing tokens: the open block's scale grows, its older codes follow
        lens = [x + 1 for x in lens]
        m.append(tokens(B, 1, Hkv, D, 10 + i, 1.5 ** i), lens)
        m.check(f"token {i}")


@pytest.mark.parametrize("kv", KV)
def test_ties_and_extremes(kv):
    """Values on rounding ties of the block's scale (largest magnitude a power
    of two, halves and quarters of steps), the top of the range, zeros, and
    bf16's smallest and largest numbers."""
    D, T, Hkv = 64, 16, 1
    base = torch.arange(-128, 128, device="cuda").double() / 128          # every 8-bit fraction
    x = base.repeat(4).view(1, 16, 1, 64).to(torch.bfloat16)
    for i, f in enumerate((1.0, 7.0 / 8, 127.0 / 128, 3e38, 1e-38, 2.0 ** -133, 2.0 ** -100, 0.0)):
        y = (x.double() * f).to(torch.bfloat16).contiguous()
        m = Model(1, Hkv, 48, D, T, kv, i)
        m.append([y, y.flip(3).contiguous()], [16])
        m.check(f"factor {f}")


@pytest.mark.parametrize("kv", KV)
def test_positions_outside_the_cache_are_dropped(kv):
    B, Hkv, L, D, T = 6, 2, 100, 64, 32
    m = Model(B, Hkv, L, D, T, kv, 3)
    #        before 0, across 0, across the end, past it, nothing new, more new tokens than given
    lens, news = [0, 5, 104, 130, 50, 20], [20, 20, 20, 20, 0, 99]
    m.append(tokens(B, 20, Hkv, D, 4), lens, news)
    m.check("clipped")
    m.append(tokens(B, 20, Hkv, D, 5), [2 ** 31 - 1, -2 ** 31, -5, 1, 100, 19], [20, 20, -3, 20, 20, 1])
    m.check("far out")


@pytest.mark.parametrize("kv", KV)
def test_strided_tokens(kv):
    """Views: heads of a fused projection, and a head-major bf16 cache."""
    B, n, Hkv, D, T = 2, 50, 3, 128, 16
    g = torch.Generator(device="cuda").manual_seed(6)
    fused = torch.randn((B, n, 4 * Hkv, D), generator=g, device="cuda").to(torch.bfloat16)
    m = Model(B, Hkv, 64, D, T, kv, 7)
    m.append([fused[:, :, Hkv:2 * Hkv], fused[:, :, 2 * Hkv:3 * Hkv]], [50, 60])
    m.check("fused")
    hnd = torch.randn((2, B, Hkv, 64, D), generator=g, device="cuda").to(torch.bfloat16)
    m = Model(B, Hkv, 64, D, T, kv, 8)
    m.append([hnd[0].transpose(1, 2), hnd[1].transpose(1, 2)], [64, 61], [64, 61])
    m.check("head-major")
    step = hnd[0][:, :, 5:6].transpose(1, 2)          # one token: its token stride says nothing
    m.append([step, step], [64, 62])
    m.check("one token of a view")


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("ps,T,layout", [(16, 16, "HND"), (64, 16, "NHD"), (128, 64, "HND"), (256, 128, "NHD")])
def test_pages_equal_contiguous(kv, ps, T, layout):
    B, Hkv, L, D = 3, 2, 512, 64
    m = Model(B, Hkv, L, D, T, kv, 9)
    lens = [300, 17, 129]
    first = tokens(B, 300, Hkv, D, 10)
    m.append(first, lens, lens)
    m.check("prompt")
    (kp, vp), (ks, vs), table = to_pages(m.codes, m.scales, [L] * B, ps, T, layout, 11, kv)
    before = [kp.clone(), vp.clone(), ks.clone(), vs.clone()]
    lens2 = [x + 40 for x in lens]
    more = tokens(B, 40, Hkv, D, 12, 3.0)
    bad = table.clone()
    bad[1] = -1                                        # sequence 1 has no pages: dropped
    bad[1, 1] = kp.shape[0]
    fd.fd_quant_append_paged(more[0], more[1], kp, vp, ks, vs, kv, T, bad, ints(lens2), None, layout)
    m.append(more, lens2, [40, 0, 40])                 # the same in the contiguous twin
    m.check("chunk")
    (kw, vw), (ksw, vsw), _ = to_pages(m.codes, m.scales, [L] * B, ps, T, layout, 11, kv)
    torch.cuda.synchronize()
    for got, want, was in zip((kp, vp, ks, vs), (kw, vw, ksw, vsw), before):
        same = (got == want) | (torch.isnan(got.float()) & torch.isnan(want.float()))
        assert same.all(), f"{(~same).sum()} differ"
        assert not torch.equal(got, was)


def test_tokens_in_a_graph():
    """One captured step (append, then attention over the longer cache),
    replayed: the lengths advance on the device between replays."""
    B, Hkv, L, D, T, kv = 2, 2, 128, 64, 32, "e4m3"
    m = Model(B, Hkv, L, D, T, kv, 13)
    start = [40, 3]
    m.append(tokens(B, 40, Hkv, D, 14), start, start)
    lens = ints(start)
    new = [torch.zeros((B, 1, Hkv, D), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    q = torch.zeros((B, 4, D), dtype=torch.bfloat16, device="cuda")
    out, lse = torch.empty((B, 4, D), device="cuda"), torch.empty((B, 4), device="cuda")
    side = torch.cuda.Stream()
    S = 3
    ws = torch.zeros(fd.quant_workspace_bytes(q, m.codes[0], S), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        push = fd.prepare_quant_append(new[0], new[1], *m.codes, *m.scales, kv, T, lens)
        look = fd.prepare_decode_quant_block(q, m.codes[0], m.codes[1], m.scales[0], m.scales[1], kv, T, lens, 0.125, out,
                                             lse, ws, S)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        lens.add_(1)
        push()
        look()
    for i in range(30):
        x = tokens(B, 1, Hkv, D, 20 + i, 1.0 + i)
        new[0].copy_(x[0])
        new[1].copy_(x[1])
        q.copy_(tokens(1, B, 4, D, 50 + i)[0][0])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        now = [n + i + 1 for n in start]
        assert lens.tolist() == now
        m.append(x, now, run=False)
        m.check(f"replay {i}")
        k, v = (c * s.repeat_interleave(T, 2)[..., None] for c, s in zip(m.vals, m.s64))
        r = ref.attention(q.view(B, 1, 4, D), k, v, now, 0.125)
        vs = v.clone()
        for b in range(B):
            vs[b, :, now[b]:] = 0
        ref.close(out, lse, r, vs, D, 2.0 ** -18, f"replay {i}")


def test_binding_refusals():
    m = Model(2, 2, 64, 64, 16, "int8")
    x = tokens(2, 5, 2, 64, 1)
    ok = dict(k_new=x[0], v_new=x[1], k_codes=m.codes[0], v_codes=m.codes[1], k_scale=m.scales[0], v_scale=m.scales[1],
              kv_type="int8", block_tokens=16, seqlens=ints([5, 5]))
    fd.fd_quant_append(**ok)
    for bad in (dict(k_new=x[0].float()), dict(k_new=x[0][:, :, :1]), dict(k_new=x[0].transpose(2, 3)),
                dict(v_new=x[1].transpose(0, 1).contiguous().transpose(0, 1)), dict(new_lens=ints([1])),
                dict(seqlens=ints([5, 5]).cpu()), dict(block_tokens=8), dict(k_scale=m.scales[0].half())):
        with pytest.raises(ValueError):
            fd.fd_quant_append(**{**ok, **bad})
    with pytest.raises(fd.FdError):                    # an odd base address
        y = torch.zeros(2 * 5 * 2 * 64 + 8, dtype=torch.bfloat16, device="cuda")[1:1281].view(2, 5, 2, 64)
        fd.fd_quant_append(**{**ok, "k_new": y})
    torch.cuda.synchronize()
