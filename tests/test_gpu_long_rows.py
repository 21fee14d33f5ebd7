"""A paged row of nearly 2^31 tokens over a pool of three pages: token
arithmetic at the top of its range, on the row's last tile above all."""
import math

import pytest
import torch

import compress_ref as ref
import decode_attention_07_b200 as fd

pytestmark = pytest.mark.gpu


def test_a_row_of_nearly_2_31_tokens():
    torch.cuda.set_device(0)
    ps, T, D, kv = 64, 16, 64, "int8"
    pages = 2 ** 25 - 4                                   # the widest table: a multiple of 4, 2^31 - 256 tokens
    g = torch.Generator(device="cuda").manual_seed(1)
    kp, vp = (torch.randint(-127, 128, (3, 1, ps, D), generator=g, device="cuda").to(torch.int8).view(torch.uint8)
              for _ in "kv")
    ks, vs = (torch.full((3, 1, ps // T), 1.0 / 127, device="cuda") for _ in "kv")
    q = torch.randn((1, 1, D), generator=g, device="cuda").to(torch.bfloat16)
    # page 2, the row's last one, weighs about as much as all the others: one key along q at ln(2^31) more
    kp[2] = (q.float() / q.float().abs().max() * 127).round().to(torch.int8).view(torch.uint8)
    along = float((ref.values(kp[2, 0, 0], kv) / 127) @ q[0, 0].double())
    ks[2] *= math.log(2.0 ** 31 / ps) / (along * 0.125)
    table = torch.arange(pages, dtype=torch.int32, device="cuda").view(1, pages) % 2
    table[0, -1] = 2
    lens = torch.tensor([2 ** 31 - 1], dtype=torch.int32, device="cuda")     # clamped to the table's end
    out, lse = fd.decode_quant_block_paged(q, kp, vp, ks, vs, kv, T, table, lens, 0.125)
    torch.cuda.synchronize()
    assert fd.fd_device_status() == 0
    k, v = (ref.values(c, kv)[:, 0] * s[:, 0].double().repeat_interleave(T, 1)[..., None] for c, s in ((kp, ks), (vp, vs)))
    times = torch.tensor([pages // 2, pages // 2 - 1, 1], dtype=torch.float64, device="cuda")
    z = k @ q[0, 0].double() * 0.125 + times.log()[:, None]
    e = torch.logsumexp(z.flatten(), 0)
    want = torch.einsum("pt,ptd->d", torch.exp(z - e), v)
    assert 0.1 < float(torch.exp(z[2] - e).sum()) < 0.9
    # a warp sums 2^31 / (148 * 8) tokens, a lane some 2^17 terms: at most 2^17 roundings of 2^-25 in each of l and o
    tol = 2 * 2.0 ** 17 * 2.0 ** -25
    assert abs(float(lse[0, 0]) - float(e)) <= tol + 2.0 ** -18 * float(e)
    assert float((out[0, 0].double() - want).abs().max()) <= tol
