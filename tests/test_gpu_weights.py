"""fd_decode_weights against the 64-bit definition: outputs, and each cached
token's attention weight added to a running total."""
import pytest
import torch

import compress_ref as ref
import decode_attention_07_b200 as fd

pytestmark = pytest.mark.gpu
# P as bf16 high part + remainder (2^-17 relative), the hardware exponential
# (2^-22) and the running sums
P_EPS = 2.0 ** -16


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    torch.cuda.set_device(0)
    yield
    assert fd.fd_device_status() == 0


def make(B, q_len, Hq, Hkv, L, D, seqlens, seed=0, sigma_k=1.0):
    """NaN keys and values past seqlens; totals NaN there too."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randn((B, q_len, Hq, D), generator=g, device="cuda").to(torch.bfloat16)
    k = (torch.randn((B, Hkv, L, D), generator=g, device="cuda") * sigma_k).to(torch.bfloat16)
    v = torch.randn((B, Hkv, L, D), generator=g, device="cuda").to(torch.bfloat16)
    w = torch.rand((B, Hkv, L), generator=g, device="cuda") * 3
    for b, n in enumerate(seqlens):
        n = min(max(n, 0), L)
        k[b, :, n:] = v[b, :, n:] = w[b, :, n:] = float("nan")
    lens = torch.tensor(seqlens, dtype=torch.int32, device="cuda")
    return (q[:, 0].contiguous() if q_len == 1 else q), k, v, w, lens


def hold(out, lse, w_out, w_in, before, r, v, D, g, seqlens, what):
    """w_out against the definition for t < seqlens, untouched after. A weight
    is off by 2 dz + 2^-20 relative (its own logit, the log-sum-exp, the
    exponential and their fp32 arguments of up to 64), their sum and the
    total by another 2^-23 each per addition."""
    dz = ref.close(out, lse, r, v.nan_to_num(0.0), D, P_EPS, what)
    B, Hkv, L = w_out.shape
    for b, n in enumerate(seqlens):
        n = min(max(n, 0), L)
        assert torch.equal(w_out[b, :, n:].nan_to_num(-1.0), before[b, :, n:].nan_to_num(-1.0)), what
        base = w_in[b, :, :n].double() if w_in is not None else 0.0
        want = base + r[2][b, :, :n]
        rel = 2 * dz[b].amax() + 2.0 ** -18
        tol = r[2][b, :, :n] * rel + want * 18 * 2.0 ** -24 + 1e-30
        err = (w_out[b, :, :n].double() - want).abs()
        assert (err <= tol).all(), f"{what}: weights of sequence {b} off by {(err / tol).max():.2f} of the bound"


@pytest.mark.parametrize("g,D,q_len", [(1, 128, 1), (1, 64, 1), (2, 128, 1), (3, 64, 1), (8, 128, 1), (16, 64, 1),
                                       (1, 128, 2), (5, 128, 3), (4, 64, 4), (1, 64, 16)])
def test_against_the_definition(g, D, q_len):
    seqlens = [1000, 0, 1, 17, 640, 64]
    Hkv, L = 2, 1000
    q, k, v, w, lens = make(len(seqlens), q_len, g * Hkv, Hkv, L, D, seqlens, g + q_len)
    scale = D ** -0.5
    r = ref.attention(q.view(len(seqlens), q_len, g * Hkv, D), k, v, seqlens, scale)
    for S in (1, 13, None):
        total = torch.full_like(w, 7.0)
        S_ = fd.fd_plan(len(seqlens), g * Hkv, Hkv, D, L) if S is None else S
        ws = torch.zeros(fd.fd_weights_workspace_bytes(len(seqlens), q_len, g * Hkv, Hkv, D, L, S_), dtype=torch.uint8,
                         device="cuda")
        out, lse = torch.empty(q.shape, device="cuda"), torch.empty(q.shape[:-1], device="cuda")
        fd.fd_decode_weights(q, k, v, lens, scale, out, lse, w, total, ws, S_)
        torch.cuda.synchronize()
        hold(out, lse, total, w, torch.full_like(w, 7.0), r, v, D, g, seqlens, f"g={g} D={D} q_len={q_len} S={S}")
        # in place, and once more on the same workspace: the second call adds the same weights
        acc = w.clone()
        fd.fd_decode_weights(q, k, v, lens, scale, out, lse, acc, acc, ws, S_)
        torch.cuda.synchronize()
        assert torch.equal(acc.nan_to_num(-1.0)[lens.argmax()], total.nan_to_num(-1.0)[lens.argmax()])
        hold(out, lse, acc, w, w, r, v, D, g, seqlens, f"in place g={g} S={S}")


def test_no_totals_in_and_the_mass():
    """From zeros: each row's weights sum to its columns that saw a token."""
    seqlens, Hkv, g, D, L, q_len = [777, 3, 0, 2], 2, 2, 128, 800, 4
    q, k, v, w, lens = make(4, q_len, g * Hkv, Hkv, L, D, seqlens, 3, sigma_k=3.0)
    out, lse, total = fd.decode_weights(q, k, v, lens, 0.1)
    torch.cuda.synchronize()
    for b, n in enumerate(seqlens):
        seen = sum(1 for j in range(q_len) if n - (q_len - 1 - j) > 0) * g
        assert torch.all((total[b].double().sum(1) - seen).abs() <= seen * 2.0 ** -14)
        assert torch.all(total[b, :, max(n, 0):] == 0)


def test_outputs_equal_fd_decode():
    """The logits are stored beside the arithmetic, which stays fd_decode's."""
    for g, D in ((1, 128), (4, 128), (16, 128), (1, 64), (8, 64)):
        q, k, v, w, lens = make(3, 1, 2 * g, 2, 900, D, [900, 31, 0], g)
        a = fd.decode_weights(q, k, v, lens, 0.1, num_splits=7)
        b = fd.decode(q, k, v, lens, 0.1, num_splits=7)
        torch.cuda.synchronize()
        if g == 1 and D == 64:
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        assert (a[0] - b[0]).abs().max() <= 2.0 ** -15 and torch.equal(torch.isneginf(a[1]), torch.isneginf(b[1]))


def test_peaked_rows_and_infinite_keys_outside():
    """One token holds all the weight; keys and values past the end infinite."""
    seqlens, D, L = [500, 100], 64, 512
    q, k, v, w, lens = make(2, 1, 4, 2, L, D, seqlens, 5)
    k[0, :, 123] = q[0, :2] * 20
    for b, n in enumerate(seqlens):
        k[b, :, n:] = float("inf")
        v[b, :, n:] = float("-inf")
    r = ref.attention(q.view(2, 1, 4, D), k, v.masked_fill(torch.isinf(v), 0.0), seqlens, 0.125)
    out, lse, total = fd.decode_weights(q, k, v, lens, 0.125)
    torch.cuda.synchronize()
    hold(out, lse, total, None, torch.zeros_like(w), r, v.masked_fill(torch.isinf(v), 0.0), D, 2, seqlens, "peaked")


def test_two_graphs_with_their_own_workspaces():
    """Two captured calls replayed on two streams at once."""
    calls = []
    for seed in (1, 2):
        q, k, v, w, lens = make(4, 1, 8, 2, 2000, 128, [2000, 1999, 5, 1000], seed)
        S = 31
        ws = torch.zeros(fd.fd_weights_workspace_bytes(4, 1, 8, 2, 128, 2000, S), dtype=torch.uint8, device="cuda")
        out, lse, acc = torch.empty(q.shape, device="cuda"), torch.empty(q.shape[:-1], device="cuda"), torch.zeros_like(w)
        side = torch.cuda.Stream()
        call = fd.prepare_decode_weights(q, k, v, lens, 0.1, out, lse, None, acc, ws, S, stream=side)
        want = fd.decode_weights(q, k, v, lens, 0.1, num_splits=S)
        torch.cuda.synchronize()
        call()                                        # warm: the kernels are loaded before the capture
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call()
        calls.append((graph, side, out, lse, acc, want, (q, k, v, w, lens, ws)))
    for rep in range(5):
        for _, _, out, lse, acc, *_ in calls:
            out.zero_()
            acc.zero_()
        torch.cuda.synchronize()
        for graph, side, *_ in calls:
            with torch.cuda.stream(side):
                graph.replay()
        torch.cuda.synchronize()
        for _, _, out, lse, acc, want, _ in calls:
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1]) and torch.equal(acc, want[2])


def test_a_prepared_call_keeps_its_tensors():
    q, k, v, w, lens = make(1, 1, 4, 2, 500, 64, [500], 7)
    ws = torch.zeros(fd.fd_weights_workspace_bytes(1, 1, 4, 2, 64, 500, 5), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty(q.shape, device="cuda"), torch.empty(q.shape[:-1], device="cuda")
    call = fd.prepare_decode_weights(q, k, v, lens, 0.1, out, lse, None, w, ws, 5)
    assert any(t is ws for t in call.tensors) and any(t is k for t in call.tensors)
    want = fd.decode_weights(q, k, v, lens, 0.1, num_splits=5)
    del ws, k, v
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    call()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_binding_refusals():
    q, k, v, w, lens = make(1, 1, 4, 2, 100, 64, [100], 6)
    with pytest.raises(ValueError):
        fd.decode_weights(q, k, v, lens, 0.1, weights=w[:, :, :50])
    with pytest.raises(ValueError):
        fd.decode_weights(q, k.transpose(2, 3), v, lens, 0.1)
    with pytest.raises(fd.FdError):
        fd.fd_decode_weights(q, k, v, lens, 0.1, torch.empty(q.shape, device="cuda"), torch.empty((1, 4), device="cuda"),
                             None, w, None)
    torch.cuda.synchronize()
