"""fd_decode_weights refuses arrays that overlap (a host check: nothing is
launched), through the C ABI with raw addresses."""
import pytest
import torch

import decode_attention_07_b200 as fd

pytestmark = pytest.mark.gpu
B, HQ, HKV, D, L, S = 2, 4, 2, 64, 300, 3
NEED = fd.fd_weights_workspace_bytes(B, 1, HQ, HKV, D, L, S)
SIZES = dict(q=B * HQ * D * 2, k=B * HKV * L * D * 2, v=B * HKV * L * D * 2, lens=B * 4, out=B * HQ * D * 4,
             lse=B * HQ * 4, w_in=B * HKV * L * 4, w_out=B * HKV * L * 4, ws=NEED)


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    torch.cuda.set_device(0)
    yield
    assert fd.fd_device_status() == 0


@pytest.fixture(scope="module")
def arena():
    """Every array in one allocation, one after the other, 256 bytes apart."""
    at, end = {}, 256
    for name, n in SIZES.items():
        at[name] = end
        end += (n + 511) // 256 * 256
    mem = torch.zeros(end, dtype=torch.uint8, device="cuda")
    lens = mem[at["lens"]:at["lens"] + B * 4].view(torch.int32)
    lens[0], lens[1] = L, 100
    return mem, at


def call(arena, **moved):
    mem, at = arena
    p = {name: mem.data_ptr() + off for name, off in {**at, **moved}.items()}
    return fd.lib().fd_decode_weights(B, 1, HQ, HKV, D, L, p["q"], p["k"], p["v"], p["lens"], 0.1, p["out"], p["lse"],
                                      p["w_in"], p["w_out"], p["ws"], NEED, S,
                                      torch.cuda.current_stream().cuda_stream)


def test_arrays_side_by_side_are_fine(arena):
    assert call(arena) == 0
    assert call(arena, w_in=arena[1]["w_out"]) == 0            # totals in place
    torch.cuda.synchronize()


# (not an array over itself, nor totals in place)
@pytest.mark.parametrize("written,other", [(w, o) for w in ("out", "lse", "w_out", "ws") for o in SIZES
                                           if o != w and (w, o) != ("w_out", "w_in")])
def test_overlaps_are_refused(arena, written, other):
    mem, at = arena
    before = mem.clone()
    last = (SIZES[other] - 1) // 16 * 16                         # its last 16 bytes
    for off in (at[other], at[other] + last):
        assert call(arena, **{written: off}) == -14
    if written != "lse":                                         # the written array's last bytes over the other's first
        start = at[other] + 16 - (SIZES[written] + 15) // 16 * 16
        if start >= 0:
            assert call(arena, **{written: start}) == -14
    torch.cuda.synchronize()
    assert torch.equal(mem, before)                              # nothing ran


def test_totals_that_overlap_in_part(arena):
    at = arena[1]
    assert call(arena, w_in=at["w_out"] + 16) == -14 and call(arena, w_in=at["w_out"] - 16) == -14
