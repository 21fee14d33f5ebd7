"""The calls that allocate (outputs, workspace) on a stream other than the
current one: what they allocate is filled in the call's order, and reused only
after it."""
import pytest
import torch

import decode_attention_07_b200 as fd
from decode_attention_07_b200 import context

pytestmark = pytest.mark.gpu
B, HKV, G, L, D, PS, T, S = 3, 2, 4, 700, 128, 64, 32, 7
DELAY = 40_000_000          # clock cycles, some 20 ms: longer than the host takes to enqueue a test


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    torch.cuda.set_device(0)
    yield
    assert fd.fd_device_status() == 0


def calls():
    g = torch.Generator(device="cuda").manual_seed(1)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)

    def codes(*shape):
        return torch.randint(0, 120, shape, generator=g, device="cuda", dtype=torch.uint8)

    q, qm = normal(B, G * HKV, D), normal(B, 3, G * HKV, D)
    k, v = normal(B, HKV, L, D), normal(B, HKV, L, D)
    lens = torch.tensor([L, 17, 333], dtype=torch.int32, device="cuda")
    per = (-(-L // PS) + 3) // 4 * 4
    table = torch.arange(B * per, dtype=torch.int32, device="cuda").view(B, per)
    kp, vp = normal(B * per, HKV, PS, D), normal(B * per, HKV, PS, D)
    k8, v8, kp8, vp8 = codes(B, HKV, L, D), codes(B, HKV, L, D), codes(B * per, HKV, PS, D), codes(B * per, HKV, PS, D)
    head = torch.rand(HKV, generator=g, device="cuda")
    sc = torch.rand((B, HKV, -(-L // T)), generator=g, device="cuda")
    psc = torch.rand((B * per, HKV, PS // T), generator=g, device="cuda")
    w = torch.rand((B, HKV, L), generator=g, device="cuda")
    z = 0.01
    return {
        "decode": lambda st: fd.decode(q, k, v, lens, z, S, st),
        "decode_multi": lambda st: fd.decode_multi(qm, k, v, lens, z, S, st),
        "decode_paged": lambda st: fd.decode_paged(q, kp, vp, table, lens, z, "HND", S, st),
        "decode_quant": lambda st: fd.decode_quant(q, k8, v8, head, head, "int8", lens, z, S, st),
        "decode_quant_paged": lambda st: fd.decode_quant_paged(q, kp8, vp8, head, head, "int8", table, lens, z, "HND", S, st),
        "decode_quant_block": lambda st: fd.decode_quant_block(q, k8, v8, sc, sc, "int8", T, lens, z, S, st),
        "decode_quant_block_paged": lambda st: fd.decode_quant_block_paged(q, kp8, vp8, psc, psc, "int8", T, table, lens, z,
                                                                          "HND", S, st),
        "decode_weights": lambda st: fd.decode_weights(q, k, v, lens, z, None, S, st),
        "evict": lambda st: fd.evict(k, v, w, lens, 200, 20, 220, st),
        "cp_decode": lambda st: context.cp_decode(q, k, v, lens, 0, z, None, S, st),
    }


def dirty(stream):
    """Memory that both allocations and fills on `stream` would take next, all bits set."""
    with torch.cuda.stream(stream):
        junk = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for n in (1 << 10, 1 << 16, 1 << 18, 1 << 20, 1 << 22)
                for _ in range(4)]
        del junk


def same(got, want):
    return all(torch.equal(a.float(), b.float()) for a, b in zip(got, want))


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("name", ["decode", "decode_multi", "decode_paged", "decode_quant", "decode_quant_paged",
                                  "decode_quant_block", "decode_quant_block_paged", "decode_weights", "evict",
                                  "cp_decode"])
def test_allocations_follow_the_calls_stream(name, handle):
    call = calls()[name]
    want = call(None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    main = torch.cuda.current_stream()
    stream = side.cuda_stream if handle else side
    # the current stream is busy: nothing of the call waits for it, and nothing comes after it
    dirty(main)
    dirty(side)
    torch.cuda.synchronize()
    torch.cuda._sleep(DELAY)
    got = call(stream)
    side.synchronize()
    with torch.cuda.stream(side):
        assert same(got, want)
    torch.cuda.synchronize()
    assert same(got, want)
    # the call's stream is busy: what the call allocated is not given away before it has run
    del got
    with torch.cuda.stream(side):
        torch.cuda._sleep(DELAY)
    got = call(stream)
    dirty(main)
    torch.cuda.synchronize()
    assert same(got, want)
    # results used on the current stream, then dropped: their memory waits for that use
    got = call(stream)
    main.wait_stream(side)
    torch.cuda._sleep(DELAY)
    copies = [t.clone() for t in got]
    del got
    dirty(side)
    torch.cuda.synchronize()
    assert same(copies, want)


def test_the_default_stream_by_its_handle():
    call = calls()["decode_weights"]
    want = call(None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = call(0)
    torch.cuda.synchronize()
    assert same(got, want)
