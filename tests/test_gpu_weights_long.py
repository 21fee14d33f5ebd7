"""fd_decode_weights on rows that the second kernel takes in several blocks,
its precision, and logits past 2^32 elements."""
import math

import pytest
import torch

import compress_ref as ref
import decode_attention_07_b200 as fd
from test_gpu_weights import make

pytestmark = pytest.mark.gpu
# P in three bf16 parts holds all 24 bits of the fp32 p; the hardware
# exponential, 2^-22, once in the weight and once in the sum; a few tens of
# fp32 additions (merges, splits) of 2^-25 to 2^-24 each
P_EPS = 2.0 ** -19


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    torch.cuda.set_device(0)
    yield
    assert fd.fd_device_status() == 0


def run(q, k, v, lens, scale, total_in, S, Hq, Hkv, L, D, q_len):
    total = torch.full((k.shape[0], Hkv, L), 7.0, device="cuda")
    ws = torch.zeros(fd.fd_weights_workspace_bytes(k.shape[0], q_len, Hq, Hkv, D, L, S), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty(q.shape, device="cuda"), torch.empty(q.shape[:-1], device="cuda")
    fd.fd_decode_weights(q, k, v, lens, scale, out, lse, total_in, total, ws, S)
    torch.cuda.synchronize()
    return out, lse, total


def hold(total, total_in, r, dz, seqlens, what):
    """Totals inside a row: each weight off by 2 dz + 2^-20 relative (its logit
    and the log-sum-exp, the exponential and their fp32 arguments of up to 64),
    16 of them and the total added in fp32. Past the row: untouched."""
    for b, n in enumerate(seqlens):
        want = total_in[b, :, :n].double() + r[2][b, :, :n]
        tol = r[2][b, :, :n] * (2 * dz[b].amax() + 2.0 ** -18) + want * 18 * 2.0 ** -24 + 1e-30
        err = (total[b, :, :n].double() - want).abs()
        assert (err <= tol).all(), f"{what}: sequence {b}, {(err / tol).max():.2f} of the bound at {int((err / tol).argmax())}"
        assert torch.all(total[b, :, n:] == 7.0), what


# columns a token's logits take: 1, 2, 4, 6, 8 (1024 tokens a block of the second kernel), 10 .. 16 (512)
@pytest.mark.parametrize("g,q_len,D", [(1, 1, 128), (1, 1, 64), (2, 1, 128), (1, 3, 64), (4, 1, 128), (5, 1, 64), (3, 2, 128),
                                       (8, 1, 128), (7, 1, 64), (5, 2, 128), (4, 3, 64), (7, 2, 128), (16, 1, 64),
                                       (15, 1, 128)])
@pytest.mark.parametrize("L", [2500, 2049])
def test_rows_of_several_blocks(g, q_len, D, L):
    """Row ends around the blocks' ends, in one segment and in many."""
    step = 512 if g * q_len > 8 else 1024
    seqlens = [L, step, step - 1, step + 1, 2 * step, 2 * step + 1, 2 * step - 31, 0, 3]
    Hkv, B = 2, len(seqlens)
    q, k, v, w, lens = make(B, q_len, g * Hkv, Hkv, L, D, seqlens, L + g)
    r = ref.attention(q.view(B, q_len, g * Hkv, D), k, v, seqlens, D ** -0.5)
    for S in (1, 29, fd.fd_plan(B, g * Hkv, Hkv, D, L)):
        out, lse, total = run(q, k, v, lens, D ** -0.5, w, S, g * Hkv, Hkv, L, D, q_len)
        what = f"g={g} q_len={q_len} D={D} L={L} S={S}"
        dz = ref.close(out, lse, r, v.nan_to_num(0.0), D, P_EPS, what)
        hold(total, w, r, dz, seqlens, what)


@pytest.mark.parametrize("g,D", [(4, 128), (4, 64), (16, 128), (16, 64)])
def test_the_weights_keep_all_their_bits(g, D):
    """All values 1, so the output is 1 whatever the logits. One token of each
    warp's 16 has logit 0 and the others one whose p = e^-kappa leaves the most
    behind two bf16 parts (1.4 * 2^-18 of it): with two parts the output would
    be low by about that much (fd_decode's is, by 5.0e-6). With all bits: one tile, at most three truncations
    of 2^-23 in its products, 5 additions of 2^-25 in each sum, and the merge of
    four warps, 8 steps of 2^-24, together below 2^-19."""
    def left(x):
        p = torch.tensor(math.exp(-x), dtype=torch.float32)
        hi = p.to(torch.bfloat16).float()
        return float((p - hi - (p - hi).to(torch.bfloat16).float()) / p)
    kappa = max((float(torch.tensor(0.02 + i * 2.0 ** -9).to(torch.bfloat16)) for i in range(300)), key=left)
    assert left(kappa) > 0.8 * 2.0 ** -18
    q = torch.zeros((1, g, D), dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = 1.0
    k = torch.zeros((1, 1, 64, D), dtype=torch.bfloat16, device="cuda")
    k[:, :, :, 0] = -kappa
    k[:, :, ::16, 0] = 0.0
    lens = torch.tensor([64], dtype=torch.int32, device="cuda")
    out, lse, total = fd.decode_weights(q, k, torch.ones_like(k), lens, 1.0, num_splits=1)
    torch.cuda.synchronize()
    assert (out.double() - 1).abs().max() <= 2.0 ** -19, f"off by {float((out.double() - 1).abs().max()):.2e}"


@pytest.mark.parametrize("g,D", [(8, 128), (16, 64)])
def test_a_long_run_keeps_its_sum(g, D):
    """131072 tokens in one segment, all values 1: each warp adds 1024 tiles to
    its running sums. Rounded to nearest these additions err by 2^-23.5 / sqrt(12)
    of the sum so far each, independently: 4.5e-7 of the sum a warp, 1.6e-7 over
    8 warps, in the outputs and less in the sum of p; six times both, and 2^-22
    for a tile's own products, is below 2^-18. Added by the tensor cores instead,
    which cut bits off, 2048 steps of 2^-25 lose some 2^-15 (fd_decode: 2.8e-5)."""
    L = 131072
    gen = torch.Generator(device="cuda").manual_seed(7)
    q = torch.randn((1, g, D), generator=gen, device="cuda").to(torch.bfloat16)
    k = torch.randn((1, 1, L, D), generator=gen, device="cuda").to(torch.bfloat16)
    lens = torch.tensor([L], dtype=torch.int32, device="cuda")
    out, lse, total = fd.decode_weights(q, k, torch.ones_like(k), lens, D ** -0.5, num_splits=1)
    torch.cuda.synchronize()
    assert (out.double() - 1).abs().max() <= 2.0 ** -18, f"off by {float((out.double() - 1).abs().max()):.2e}"
    z = (k[0, 0].double() @ q[0].double().T) * D ** -0.5
    assert (lse[0].double() - torch.logsumexp(z, 0)).abs().max() <= 2.0 ** -18 + 24 * 2.0 ** -24
    want = torch.softmax(z, 0).sum(1)
    assert ((total[0, 0].double() - want).abs() <= want * 2.0 ** -15).all()


def test_logits_past_32_bits():
    """136 rows of 2^21 tokens and 16 columns: the last sequence's logits start
    at element 2^32. Only that sequence is long."""
    B, Hkv, g, L, D = 17, 8, 16, 1 << 21, 64
    gen = torch.Generator(device="cuda").manual_seed(8)
    k = torch.zeros((B, Hkv, L, D), dtype=torch.bfloat16, device="cuda")
    for h in range(Hkv):
        k[-1, h] = torch.randn((L, D), generator=gen, device="cuda").to(torch.bfloat16)
    q = torch.randn((B, g * Hkv, D), generator=gen, device="cuda").to(torch.bfloat16)
    seqlens = [3] * (B - 1) + [L - 5]
    lens = torch.tensor(seqlens, dtype=torch.int32, device="cuda")
    out, lse, total = fd.decode_weights(q, k, k, lens, 0.1)
    torch.cuda.synchronize()
    assert ((total[:-1, :, :3].double() - g / 3).abs() <= 1e-5 * g).all()        # keys of 0: each token a third
    assert torch.all(total[:-1, :, 3:] == 0) and torch.all(total[-1, :, L - 5:] == 0)
    for h in (0, Hkv - 1):
        r = ref.attention(q[-1:, h * g:(h + 1) * g].view(1, 1, g, D), k[-1:, h:h + 1], k[-1:, h:h + 1], [L - 5], 0.1)
        dz = ref.close(out[-1:, h * g:(h + 1) * g], lse[-1:, h * g:(h + 1) * g], r, k[-1:, h:h + 1], D, P_EPS, f"head {h}")
        want = r[2][0, 0, :L - 5]
        err = (total[-1, h, :L - 5].double() - want).abs()
        assert (err <= want * (2 * dz.amax() + 2.0 ** -17)).all(), f"head {h}"
