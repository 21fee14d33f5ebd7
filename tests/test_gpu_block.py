"""Attention over an 8-bit cache with one scale per block of tokens
(fd_decode_quant_block, fd_decode_quant_block_paged) against the 64-bit
definition over the same codes and scales."""
import numpy as np
import pytest
import torch

import compress_ref as ref
import decode_attention_07_b200 as fd

pytestmark = pytest.mark.gpu
KV = ["e4m3", "int8"]
# P as f16 high part + remainder: 2^-22 relative, and f16's smallest step,
# 2^-25 under a largest weight of 2^7 (a lazy reference may put it at 2^-1):
# 2^-24; two hardware exponentials, each 2^-22 relative; a log2 of the value
# scale, |log2 s| <= 32 here, 2^-22 + 32 * 2^-24 absolute; the running sum
P_EPS = 2.0 ** -18


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    torch.cuda.set_device(0)
    yield
    assert fd.fd_device_status() == 0


def make(B, Hkv, L, D, T, kv, seqlens, seed, spread=1.0):
    """Codes and scales of a cache; positions and blocks past seqlens hold
    NaN codes (E4M3) and NaN scales. spread: log2 range of the scales."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    nblk = -(-L // T)
    cache = []
    for _ in range(2):
        x = torch.randn((B, Hkv, L, D), generator=g, device="cuda", dtype=torch.float64)
        vals = ref.nearest(x * (ref.RANGE[kv] / 4.0), kv)
        codes = ref.codes_of(vals, kv)
        scale = torch.exp2((torch.rand((B, Hkv, nblk), generator=g, device="cuda") - 0.5) * 2 * spread) * (
            4.0 / ref.RANGE[kv])
        for b in range(B):
            n = min(max(seqlens[b], 0), L)
            codes[b, :, n:] = 0x7F
            scale[b, :, -(-n // T):] = float("nan")
        cache += [codes.contiguous(), scale.contiguous()]
    return cache[0], cache[2], cache[1], cache[3]


def dense(codes, scale, T, kv, seqlens):
    v = ref.values(codes, kv) * scale.double().repeat_interleave(T, 2)[:, :, :codes.shape[2], None]
    for b in range(v.shape[0]):
        v[b, :, min(max(seqlens[b], 0), v.shape[2]):] = 0.0
    return v


def query(B, q_len, Hq, D, seed, sigma=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = (torch.randn((B, q_len, Hq, D), generator=g, device="cuda") * sigma).to(torch.bfloat16)
    return q[:, 0].contiguous() if q_len == 1 else q


def check(kv, T, g, D, q_len, L, seqlens, seed=0, spread=1.0, sigma=1.0, splits=(1, None, 13), Hkv=2, edit=None):
    B = len(seqlens)
    k8, v8, ks, vs = make(B, Hkv, L, D, T, kv, seqlens, seed, spread)
    if edit:
        edit(k8, v8, ks, vs)
    q = query(B, q_len, g * Hkv, D, seed + 1, sigma)
    lens = torch.tensor(seqlens, dtype=torch.int32, device="cuda")
    k, v = dense(k8, ks, T, kv, seqlens), dense(v8, vs, T, kv, seqlens)
    scale = D ** -0.5
    r = ref.attention(q.view(B, q_len, g * Hkv, D), k, v, seqlens, scale)
    for S in splits:
        out, lse = fd.decode_quant_block(q, k8, v8, ks, vs, kv, T, lens, scale, num_splits=S)
        torch.cuda.synchronize()
        ref.close(out, lse, r, v, D, P_EPS, f"{kv} T={T} g={g} D={D} q_len={q_len} S={S}")
    return q, k8, v8, ks, vs, lens, r, v


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("T", [16, 32, 64, 128])
@pytest.mark.parametrize("g,D,q_len", [(1, 128, 1), (8, 128, 1), (16, 64, 1), (3, 64, 2)])
def test_against_the_definition(kv, T, g, D, q_len):
    check(kv, T, g, D, q_len, 1000, [1000, 0, 1, 2, 577, 65], splits=(1, None, 13))


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("D,q_len,g", [(128, 4, 4), (128, 16, 1), (64, 5, 3)])
def test_several_queries(kv, D, q_len, g):
    # sequences shorter than the window: queries that see nothing
    check(kv, 32, g, D, q_len, 300, [300, q_len - 1, 1, 128, 0])


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("L", [1, 15, 16, 17, 63, 64, 65, 129])
def test_short_caches(kv, L):
    check(kv, 16, 4, 128, 1, L, [L, max(L - 1, 0), 1])


@pytest.mark.parametrize("kv", KV)
def test_scales_of_very_different_sizes(kv):
    """Block scales spread over 2^-15 .. 2^15: values of the heavy blocks and
    of the light ones keep their precision relative to the row's output."""
    check(kv, 16, 4, 128, 1, 700, [700, 333], spread=15.0, sigma=1e-4)


@pytest.mark.parametrize("kv", KV)
def test_an_outlier_block_of_values_with_no_weight(kv):
    """One block has values 2^20 times the others', and keys that give it no
    weight: the output is the other blocks', at their own precision."""
    T, D = 16, 128

    def edit(k8, v8, ks, vs):
        big = torch.full_like(k8[:, :, :T], 0x7E if kv == "e4m3" else 127)
        k8[:, :, 2 * T:3 * T] = big            # all keys of the block at the top code
        vs[:, :, 2] *= 2.0 ** 20
        ks[:, :, 2] *= 8.0
    B, Hkv, L = 2, 2, 400
    k8, v8, ks, vs = make(B, Hkv, L, D, T, kv, [L, 399], 3)
    edit(k8, v8, ks, vs)
    q = -torch.ones((B, 4, D), device="cuda").to(torch.bfloat16)     # strongly negative logits for the big keys
    lens = torch.tensor([L, 399], dtype=torch.int32, device="cuda")
    k, v = dense(k8, ks, T, kv, [L, 399]), dense(v8, vs, T, kv, [L, 399])
    r = ref.attention(q.view(B, 1, 4, D), k, v, [L, 399], D ** -0.5)
    assert r[0].abs().max() < 8.0                                      # the outlier block does not show
    others = torch.cat([v[:, :, :2 * T], v[:, :, 3 * T:]], 2)          # the values that carry the weight
    for S in (1, 3):
        out, lse = fd.decode_quant_block(q, k8, v8, ks, vs, kv, T, lens, D ** -0.5, num_splits=S)
        torch.cuda.synchronize()
        # the heavy keys' logits are the largest unit by far, and weigh nothing: take the others' unit
        kk = torch.cat([k[:, :, :2 * T], k[:, :, 3 * T:]], 2)
        rr = ref.attention(q.view(B, 1, 4, D), kk, others, [L - T, 399 - T], D ** -0.5)
        ref.close(out, lse, (r[0], r[1], r[2], rr[3]), others, D, P_EPS, f"{kv} outlier block S={S}")


@pytest.mark.parametrize("kv", KV)
def test_zero_scales_and_a_whole_row_of_zeros(kv):
    def edit(k8, v8, ks, vs):
        ks[0, :, 1] = 0.0                      # a block of zero keys
        vs[0, :, 2] = 0.0                      # a block of zero values
        vs[1] = torch.where(torch.isnan(vs[1]), vs[1], torch.zeros_like(vs[1]))   # a sequence of zero values
    check(kv, 32, 4, 64, 1, 500, [500, 200], edit=edit)


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("rising", [True, False])
def test_rising_and_falling_logits(kv, rising):
    """Key scales that grow along the sequence move the reference maximum on
    many tiles; falling ones put it in the first tile. Value scales run the
    other way, so the two references part."""
    def edit(k8, v8, ks, vs):
        ramp = torch.linspace(0.2, 6.0, ks.shape[2], device="cuda")
        ks.mul_(ramp if rising else ramp.flip(0))
        vs.mul_(torch.exp2(-4 * (ramp if rising else ramp.flip(0))))
    check(kv, 64, 4, 128, 1, 3001, [3001, 2999], edit=edit, splits=(1, 9, 61))


def test_more_splits_than_tiles_and_determinism():
    q, k8, v8, ks, vs, lens, r, v = check("e4m3", 32, 4, 128, 1, 700, [700, 13, 350], splits=(200, 7))
    a = fd.decode_quant_block(q, k8, v8, ks, vs, "e4m3", 32, lens, 128 ** -0.5, num_splits=7)
    b = fd.decode_quant_block(q, k8, v8, ks, vs, "e4m3", 32, lens, 128 ** -0.5, num_splits=7)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("kv", KV)
def test_one_scale_everywhere_equals_the_per_head_form(kv):
    """With the same scale in every block of a head, within rounding of
    fd_decode_quant over the same codes."""
    B, Hkv, L, D, T = 2, 2, 900, 128, 64
    k8, v8, ks, vs = make(B, Hkv, L, D, T, kv, [L, 450], 5)
    hk = torch.tensor([0.01, 0.02], device="cuda")
    hv = torch.tensor([0.5, 0.003], device="cuda")
    ks[:] = hk[None, :, None]
    vs[:] = hv[None, :, None]
    q = query(B, 1, 8, D, 6)
    lens = torch.tensor([L, 450], dtype=torch.int32, device="cuda")
    a, la = fd.decode_quant_block(q, k8, v8, ks, vs, kv, T, lens, 0.1)
    b, lb = fd.decode_quant(q, k8, v8, hk, hv, kv, lens, 0.1)
    torch.cuda.synchronize()
    vmax = float((ref.values(v8[:, :, :450], kv).abs().amax() * hv.max()))
    assert (a - b).abs().max() <= 4 * P_EPS * vmax and (la - lb).abs().max() <= 1e-5 * lb.abs().max()


# ------------------------------------------------------------------- pages --

def to_pages(codes, scales, seqlens, ps, T, layout, seed, kv, inorder=False):
    """Scatter [B,Hkv,L,D] codes and [B,Hkv,nblk] scales into shuffled pages
    (inorder: a sequence's pages follow one another in the pool)."""
    B, Hkv, L, D = codes[0].shape
    per = (-(-L // ps) + 3) // 4 * 4
    need = [-(-min(max(n, 0), L) // ps) for n in seqlens]
    pages = sum(need) + 3
    order = np.arange(pages) if inorder else np.random.RandomState(seed).permutation(pages)
    table = np.full((B, per), 10 ** 6, np.int32)
    shape = (pages, Hkv, ps, D) if layout == "HND" else (pages, ps, Hkv, D)
    pools = [torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda") for _ in codes]
    spools = [torch.full((pages, Hkv, ps // T), float("nan"), device="cuda") for _ in scales]
    at = 0
    for b in range(B):
        for i in range(need[b]):
            page = int(order[at])
            at += 1
            table[b, i] = page
            t0, t1 = i * ps, min(i * ps + ps, L)
            for c, pool in zip(codes, pools):
                part = c[b, :, t0:t1]
                if layout == "HND":
                    pool[page, :, :t1 - t0] = part
                else:
                    pool[page, :t1 - t0] = part.transpose(0, 1)
            for s, pool in zip(scales, spools):
                part = s[b, :, t0 // T:-(-t1 // T)]
                pool[page, :, :part.shape[1]] = part
    return pools, spools, torch.from_numpy(table).cuda()


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("ps,T,layout,g,D,q_len", [(16, 16, "HND", 4, 128, 1), (32, 16, "NHD", 1, 128, 1),
                                                   (64, 64, "HND", 8, 128, 1), (256, 128, "NHD", 16, 64, 1),
                                                   (128, 32, "HND", 2, 64, 3), (16, 16, "NHD", 16, 128, 1)])
def test_pages_equal_contiguous(kv, ps, T, layout, g, D, q_len):
    seqlens = [1100, 0, 17, 530, 16]
    B, Hkv, L = len(seqlens), 2, 1100
    k8, v8, ks, vs = make(B, Hkv, L, D, T, kv, seqlens, 7)
    q = query(B, q_len, g * Hkv, D, 8)
    lens = torch.tensor(seqlens, dtype=torch.int32, device="cuda")
    (kp, vp), (ksp, vsp), table = to_pages([k8, v8], [ks, vs], seqlens, ps, T, layout, 9, kv)
    v = dense(v8, vs, T, kv, seqlens)
    r = ref.attention(q.view(B, q_len, g * Hkv, D), dense(k8, ks, T, kv, seqlens), v, seqlens, 0.1)
    for S in (1, 23):
        a = fd.decode_quant_block_paged(q, kp, vp, ksp, vsp, kv, T, table, lens, 0.1, layout, num_splits=S)
        b = fd.decode_quant_block(q, k8, v8, ks, vs, kv, T, lens, 0.1, num_splits=S)
        torch.cuda.synchronize()
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]), f"S={S}"
        ref.close(a[0], a[1], r, v, D, P_EPS, f"{kv} pages of {ps}, S={S}")


@pytest.mark.parametrize("ps,T,layout,D", [(16, 16, "HND", 128), (32, 32, "NHD", 64), (64, 16, "NHD", 128)])
def test_pages_in_pool_order(ps, T, layout, D):
    """Small pages that follow one another in the pool come with one copy per tile."""
    kv, seqlens = "int8", [900, 77, 512]
    k8, v8, ks, vs = make(3, 2, 900, D, T, kv, seqlens, 20)
    q = query(3, 1, 8, D, 21)
    lens = torch.tensor(seqlens, dtype=torch.int32, device="cuda")
    (kp, vp), (ksp, vsp), table = to_pages([k8, v8], [ks, vs], seqlens, ps, T, layout, 22, kv, inorder=True)
    a = fd.decode_quant_block_paged(q, kp, vp, ksp, vsp, kv, T, table, lens, 0.1, layout, num_splits=11)
    b = fd.decode_quant_block(q, k8, v8, ks, vs, kv, T, lens, 0.1, num_splits=11)
    torch.cuda.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_two_calls_at_once():
    """Two streams, two workspaces, overlapping on the device."""
    calls = []
    for i in range(2):
        seqlens = [4000, 17, 3999, 2500]
        k8, v8, ks, vs = make(4, 2, 4000, 128, 64, "e4m3", seqlens, 30 + i)
        q = query(4, 1, 8, 128, 40 + i)
        lens = torch.tensor(seqlens, dtype=torch.int32, device="cuda")
        want = fd.decode_quant_block(q, k8, v8, ks, vs, "e4m3", 64, lens, 0.1, num_splits=37)
        ws = torch.zeros(fd.quant_workspace_bytes(q, k8, 37), dtype=torch.uint8, device="cuda")
        out, lse = torch.empty(q.shape, device="cuda"), torch.empty(q.shape[:-1], device="cuda")
        side = torch.cuda.Stream()
        calls.append((fd.prepare_decode_quant_block(q, k8, v8, ks, vs, "e4m3", 64, lens, 0.1, out, lse, ws, 37,
                                                    stream=side), out, lse, want))
    torch.cuda.synchronize()
    for rep in range(20):
        for call, *_ in calls:
            call()
    torch.cuda.synchronize()
    for _, out, lse, want in calls:
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_a_bad_page_reads_as_zeros():
    kv, T, D, ps = "e4m3", 16, 128, 16
    seqlens = [300, 128]
    k8, v8, ks, vs = make(2, 2, 300, D, T, kv, seqlens, 11)
    (kp, vp), (ksp, vsp), table = to_pages([k8, v8], [ks, vs], seqlens, ps, T, "HND", 12, kv)
    table[0, 3] = -1
    table[1, 5] = kp.shape[0]
    for c in (k8, v8):
        c[0, :, 3 * ps:4 * ps] = 0
        c[1, :, 5 * ps:6 * ps] = 0
    q = query(2, 1, 4, D, 13)
    lens = torch.tensor(seqlens, dtype=torch.int32, device="cuda")
    v = dense(v8, vs, T, kv, seqlens)
    r = ref.attention(q.view(2, 1, 4, D), dense(k8, ks, T, kv, seqlens), v, seqlens, 0.1)
    out, lse = fd.decode_quant_block_paged(q, kp, vp, ksp, vsp, kv, T, table, lens, 0.1, "HND")
    torch.cuda.synchronize()
    ref.close(out, lse, r, v, D, P_EPS, "bad pages")


# ------------------------------------------------------- streams and graphs --

def test_on_a_side_stream_and_in_a_graph():
    kv, T, D = "int8", 32, 128
    seqlens = [900, 450]
    k8, v8, ks, vs = make(2, 2, 900, D, T, kv, seqlens, 14)
    q = query(2, 1, 8, D, 15)
    lens = torch.tensor(seqlens, dtype=torch.int32, device="cuda")
    S = 9
    ws = torch.zeros(fd.quant_workspace_bytes(q, k8, S), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty(q.shape, device="cuda"), torch.empty(q.shape[:-1], device="cuda")
    want = fd.decode_quant_block(q, k8, v8, ks, vs, kv, T, lens, 0.1, num_splits=S)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    call = fd.prepare_decode_quant_block(q, k8, v8, ks, vs, kv, T, lens, 0.1, out, lse, ws, S, stream=side)
    call()
    side.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
        call()
    for n in ([900, 450], [17, 0], [640, 900]):
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        for b in range(2):   # positions that become visible hold valid codes and scales
            k8[b, :, seqlens[b]:] = 1
            v8[b, :, seqlens[b]:] = 1
        ks.nan_to_num_(0.01)
        vs.nan_to_num_(0.01)
        want = fd.decode_quant_block(q, k8, v8, ks, vs, kv, T, lens, 0.1, num_splits=S)
        out.fill_(9.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1]), n


def test_offsets_past_32_bits():
    """A cache of more than 2^32 codes: the last sequence against the definition."""
    B, Hkv, L, D, T, kv = 33, 8, 131072, 128, 128, "int8"
    g = torch.Generator(device="cuda").manual_seed(16)
    k8 = torch.randint(0, 256, (B, Hkv, L, D), generator=g, device="cuda", dtype=torch.uint8)
    v8 = torch.randint(0, 256, (B, Hkv, L, D), generator=g, device="cuda", dtype=torch.uint8)
    ks = torch.rand((B, Hkv, L // T), generator=g, device="cuda") * 0.01
    vs = torch.rand((B, Hkv, L // T), generator=g, device="cuda") * 0.01
    q = query(B, 1, Hkv, D, 17)
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    lens[-1] = L - 5
    out, lse = fd.decode_quant_block(q, k8, v8, ks, vs, kv, T, lens, 0.1)
    torch.cuda.synchronize()
    v = ref.values(v8[-1:], kv) * vs[-1:].double().repeat_interleave(T, 2)[..., None]
    k = ref.values(k8[-1:], kv) * ks[-1:].double().repeat_interleave(T, 2)[..., None]
    r = ref.attention(q[-1:].view(1, 1, Hkv, D), k, v, [L - 5], 0.1)
    ref.close(out[-1:], lse[-1:], r, v, D, P_EPS, "last sequence")
    assert torch.all(out[:-1] == 0) and torch.isneginf(lse[:-1]).all()


def test_binding_refusals():
    k8, v8, ks, vs = make(1, 2, 100, 64, 32, "e4m3", [100], 18)
    q = query(1, 1, 4, 64, 19)
    lens = torch.tensor([100], dtype=torch.int32, device="cuda")

    def call(**kw):
        a = dict(q=q, k_codes=k8, v_codes=v8, k_scale=ks, v_scale=vs, kv_type="e4m3", block_tokens=32, seqlens=lens,
                 scale=0.1)
        a.update(kw)
        return fd.decode_quant_block(**a)
    call()
    for bad in (dict(block_tokens=48), dict(block_tokens=64), dict(kv_type="e5m2"), dict(k_scale=ks[:, :, :1]),
                dict(k_codes=k8.transpose(1, 2)), dict(q=q.float()), dict(v_scale=vs.double()), dict(q=q.cpu()),
                dict(seqlens=lens.long())):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(fd.FdError):
        call(num_splits=-1)
    torch.cuda.synchronize()
