"""Prepared calls hold the tensors whose addresses they keep, and run on their
tensors' device."""
import gc
import weakref

import pytest
import torch

import decode_attention_07_b200 as fd

pytestmark = pytest.mark.gpu
B, HKV, G, L, D, PS, S = 2, 2, 4, 500, 64, 16, 5


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    torch.cuda.set_device(0)
    yield
    assert fd.fd_device_status() == 0


def arguments(kind):
    g = torch.Generator(device="cuda").manual_seed(3)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)

    def codes(*shape):
        return torch.randint(0, 120, shape, generator=g, device="cuda", dtype=torch.uint8)

    q = normal(B, 2, G * HKV, D) if kind == "multi" else normal(B, G * HKV, D)
    lens = torch.tensor([L, 99], dtype=torch.int32, device="cuda")
    out, lse = torch.empty(q.shape, device="cuda"), torch.empty(q.shape[:-1], device="cuda")
    per = (-(-L // PS) + 3) // 4 * 4
    columns = G * HKV * (2 if kind == "multi" else 1)
    ws = torch.zeros(fd.fd_workspace_bytes(B, columns, HKV, D, per * PS, S), dtype=torch.uint8, device="cuda")
    table = torch.arange(B * per, dtype=torch.int32, device="cuda").view(B, per)
    scales = [torch.rand(HKV, generator=g, device="cuda") for _ in "kv"]
    if kind in ("decode", "multi"):
        return (q, normal(B, HKV, L, D), normal(B, HKV, L, D), lens, 0.1, out, lse, ws), (S,)
    if kind == "paged":
        pool = [normal(B * per, HKV, PS, D) for _ in "kv"]
        return (q, *pool, table, lens, 0.1, out, lse, ws), ("HND", S)
    if kind == "quant":
        return (q, codes(B, HKV, L, D), codes(B, HKV, L, D), *scales, "int8", lens, 0.1, out, lse, ws), (S,)
    pool = [codes(B * per, HKV, PS, D) for _ in "kv"]
    return (q, *pool, *scales, "int8", table, lens, 0.1, out, lse, ws), ("HND", S)


PREPARE = {"decode": fd.prepare_decode, "multi": fd.prepare_decode_multi, "paged": fd.prepare_decode_paged,
           "quant": fd.prepare_decode_quant, "quant_paged": fd.prepare_decode_quant_paged}


@pytest.mark.parametrize("kind", list(PREPARE))
def test_a_prepared_call_holds_its_tensors(kind):
    args, rest = arguments(kind)
    call = PREPARE[kind](*args, *rest)
    refs = [weakref.ref(a) for a in args if isinstance(a, torch.Tensor)]
    out, lse = args[-3], args[-2]
    call()
    torch.cuda.synchronize()
    want = out.clone(), lse.clone()
    assert torch.isfinite(want[0]).all()
    out.zero_()
    del args
    gc.collect()
    assert all(r() is not None for r in refs), "the call keeps an address whose tensor is gone"
    call()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    del call, out, lse
    gc.collect()
    assert not any(r() is not None for r in refs)      # and nothing else does


@pytest.mark.parametrize("kind", ["decode", "multi", "quant"])
def test_the_split_count_is_readable(kind):
    args, _ = arguments(kind)
    planned = PREPARE[kind](*args)
    assert planned.num_splits == fd.fd_plan(B, G * HKV, HKV, D, L)
    assert PREPARE[kind](*args, S).num_splits == S


@pytest.mark.parametrize("kind", list(PREPARE))
def test_errors_are_raised_by_the_call(kind):
    args, rest = arguments(kind)
    call = PREPARE[kind](*args[:-1], None, *rest)       # several splits without a workspace
    with pytest.raises(fd.FdError) as e:
        call()
    assert e.value.code == -6


@pytest.mark.parametrize("kind", list(PREPARE))
def test_lengths_with_gaps_are_refused(kind):
    """A view's lengths are not side by side in memory, where the kernels read them."""
    args, rest = arguments(kind)
    at = next(i for i, a in enumerate(args) if isinstance(a, torch.Tensor) and a.dtype == torch.int32 and a.dim() == 1)
    spaced = torch.tensor([L, 1, 99, 1], dtype=torch.int32, device="cuda")
    for bad in (spaced[::2], args[at][:1].expand(B)):
        with pytest.raises(ValueError):
            PREPARE[kind](*args[:at], bad, *args[at + 1:], *rest)
    PREPARE[kind](*args[:at], spaced[::2].contiguous(), *args[at + 1:], *rest)()
    torch.cuda.synchronize()


def test_lengths_with_gaps_are_refused_by_the_direct_calls():
    (q, k, v, lens, scale, out, lse, ws), _ = arguments("decode")
    bad = torch.tensor([L, 1, 99, 1], dtype=torch.int32, device="cuda")[::2]
    for call in (lambda n: fd.fd_decode(q, k, v, n, scale, out, lse, ws), lambda n: fd.decode(q, k, v, n, scale),
                 lambda n: fd.fd_decode_splits(q, k, v, n, scale, out, lse, ws, S),
                 lambda n: fd.fd_split(q, k, v, n, scale, out, lse, ws, S),
                 lambda n: fd.fd_combine(B, G * HKV, HKV, D, L, n, out, lse, ws, S),
                 lambda n: fd.fd_decode_static(q, k, v, n, scale, out, lse)):
        with pytest.raises(ValueError):
            call(bad)
    torch.cuda.synchronize()
