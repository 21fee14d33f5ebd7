"""Block-scaled attention where value scales are zero, dominated by a block of
zeros, or far from 1: a column that has met only zero value scales holds no
output yet, and what follows must neither spoil it nor lose precision."""
import pytest
import torch

import compress_ref as ref
import decode_attention_07_b200 as fd
from test_gpu_block import KV, P_EPS, check, dense, make, query, to_pages

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    torch.cuda.set_device(0)
    yield
    assert fd.fd_device_status() == 0


def zero_values(*blocks):
    def edit(k8, v8, ks, vs):
        for b in blocks:
            vs[:, :, b] = 0.0
    return edit


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("g,D", [(1, 128), (4, 64), (8, 128)])
def test_zero_values_then_tokens_only_later_queries_see(kv, g, D):
    """Block 0 is zeros; the one token after it is masked for the first query."""
    check(kv, 16, g, D, 2, 17, [17, 17], splits=(1, 2), edit=zero_values(0))
    check(kv, 16, g, D, 2, 33, [33, 32], splits=(1, 2), edit=zero_values(0, 1))


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("g,D", [(1, 128), (4, 64), (16, 128), (16, 64)])
@pytest.mark.parametrize("blocks", [(3,), (0, 1, 2, 3), tuple(range(10))])
def test_zero_values_then_only_tokens_past_the_row(kv, g, D, blocks):
    """The warps that own the zero blocks meet nothing but tokens past the
    row's end afterwards (the last token's scale is not zero)."""
    check(kv, 32, g, D, 1, 330, [330, 321], splits=(1, 2, 5), edit=zero_values(*blocks))


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("g", [4, 16])
@pytest.mark.parametrize("ps,T", [(16, 16), (64, 16), (64, 32)])
def test_a_first_page_outside_the_pool(kv, g, ps, T):
    D, seqlens = 128, [ps + 1, ps + 2, 5 * 64 + 10]
    B, L, q_len = len(seqlens), 330, 1 if g == 16 else 2
    k8, v8, ks, vs = make(B, 2, L, D, T, kv, seqlens, 50)
    (kp, vp), (ksp, vsp), table = to_pages([k8, v8], [ks, vs], seqlens, ps, T, "HND", 51, kv)
    table[:, 0] = -1
    for c in (k8, v8):
        c[:, :, :ps] = 0
    lens = torch.tensor(seqlens, dtype=torch.int32, device="cuda")
    q = query(B, q_len, 2 * g, D, 52)
    v = dense(v8, vs, T, kv, seqlens)
    r = ref.attention(q.view(B, q_len, 2 * g, D), dense(k8, ks, T, kv, seqlens), v, seqlens, 0.1)
    for S in (1, 2):
        out, lse = fd.decode_quant_block_paged(q, kp, vp, ksp, vsp, kv, T, table, lens, 0.1, "HND", num_splits=S)
        torch.cuda.synchronize()
        ref.close(out, lse, r, v, D, P_EPS, f"{kv} pages of {ps}, T={T}, S={S}")


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("g", [2, 16])
@pytest.mark.parametrize("gap", [20.0, 60.0, 200.0, 2000.0])
def test_a_block_of_zero_values_that_takes_the_weight(kv, g, gap):
    """Logits of about `gap` (natural) in a block of zero values, about 0 in
    the others: their outputs are good relative to what they contribute, and
    exactly absent once their weights leave float's range (e^-200)."""
    D, T, L, Hkv = 64, 32, 400, 2
    k8, v8, ks, vs = make(2, Hkv, L, D, T, kv, [L, 390], 53)
    top = 0x7E if kv == "e4m3" else 127
    q = query(2, 1, g * Hkv, D, 54, 0.05).abs()
    for block in (0, 5):
        k8[:, :, block * T:(block + 1) * T] = top
        ks[:, :, block] = gap / ref.RANGE[kv] / float(q.float().sum(-1).mean()) / 0.125
        vs[:, :, block] = 0.0
    lens = torch.tensor([L, 390], dtype=torch.int32, device="cuda")
    k, v = dense(k8, ks, T, kv, [L, 390]), dense(v8, vs, T, kv, [L, 390])
    r = ref.attention(q.view(2, 1, g * Hkv, D), k, v, [L, 390], 0.125)
    # the weight that is not on zeros, per (sequence, head)
    live = (vs.repeat_interleave(T, 2)[:, :, :L] > 0) & (torch.arange(L, device="cuda") < lens[:, None])[:, None]
    z = torch.einsum("bhgd,bhtd->bhgt", q.double().view(2, Hkv, g, D), k) * 0.125
    mass = (torch.exp(z - r[1].view(2, Hkv, g, 1)) * live[:, :, None]).sum(3).view(2, 1, g * Hkv)
    dz = (D + 8) * 2.0 ** -24 * r[3] + 2.0 ** -22 * r[3]
    tol = float(v.abs().max()) * (mass * 2 * (2 * dz + P_EPS) + 2.0 ** -126)
    for S in (1, 3):
        out, lse = fd.decode_quant_block(q, k8, v8, ks, vs, kv, T, lens, 0.125, num_splits=S)
        torch.cuda.synchronize()
        assert torch.isfinite(out).all(), f"S={S}"
        err = (out.double().view(r[0].shape) - r[0]).abs().amax(3)
        assert (err <= tol).all(), f"S={S}: {(err / tol).max():.2f} of the bound"
        assert (lse.double().view(r[1].shape) - r[1]).abs().max() <= float(dz.max()) + 2.0 ** -20 * gap * 2


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("g", [4, 16])
@pytest.mark.parametrize("power", [-100, -31, 60])
def test_values_scaled_by_a_power_of_two(kv, g, power):
    """Value scales times 2^power give outputs times 2^power. The weights are
    the same in both; the reference that P's f16 pair is held against may land
    one power of two apart, a rounding of 2^-22 in each."""
    B, Hkv, L, D, T = 16, 2, 16, 64, 16
    k8, v8, ks, vs = make(B, Hkv, L, D, T, kv, [L] * B, 55, spread=0.5)
    v8[:] = 0x7E if kv == "e4m3" else 127      # one value per block: an error of its scale does not average out
    q = query(B, 1, g * Hkv, D, 56)
    lens = torch.full((B,), L, dtype=torch.int32, device="cuda")
    a, la = fd.decode_quant_block(q, k8, v8, ks, vs, kv, T, lens, 0.125, num_splits=1)
    b, lb = fd.decode_quant_block(q, k8, v8, ks, vs * 2.0 ** power, kv, T, lens, 0.125, num_splits=1)
    torch.cuda.synchronize()
    want = a.double() * 2.0 ** power
    assert torch.equal(la, lb)
    err = ((b.double() - want).abs() / want.abs()).max()
    assert err <= 2 * 2.0 ** -22 + 2.0 ** -24, f"relative difference {err:.3e}"


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("g", [4, 16])
def test_the_log_sum_exp_of_one_token_is_its_logit(kv, g):
    """One-hot queries, so the products are exact. What is left: four roundings
    of the logit and its base-2 form, the argument of the exponential (below 8
    in size, 2^-21), the exponential (2^-22 of it) and the logarithm of a number
    within a factor of 2 of 1 (2^-22), in base 2: below 2^-20 ln 2, and 2^-22 of
    the logit."""
    B, Hkv, D, T = 64, 2, 64, 16
    k8, v8, ks, vs = make(B, Hkv, 1, D, T, kv, [1] * B, 57)
    q = torch.zeros((B, g * Hkv, D), dtype=torch.bfloat16, device="cuda")
    q[:, :, 5] = query(B, 1, g * Hkv, 1, 58)[..., 0]
    lens = torch.ones(B, dtype=torch.int32, device="cuda")
    out, lse = fd.decode_quant_block(q, k8, v8, ks, vs, kv, T, lens, 0.125, num_splits=1)
    torch.cuda.synchronize()
    k = dense(k8, ks, T, kv, [1] * B)
    z = torch.einsum("bhgd,bhd->bhg", q.double().view(B, Hkv, g, D), k[:, :, 0]).reshape(B, g * Hkv) * 0.125
    err = (lse.double() - z).abs()
    assert (err <= 0.7 * 2.0 ** -20 + 2.0 ** -22 * z.abs()).all(), f"off by {float(err.max()):.2e}"
