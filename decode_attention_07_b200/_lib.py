"""ctypes binding over libfdecode.so: the C ABI of include/fd.h with the same
names, taking torch tensors. Argument marshalling only -- every step of the
computation runs in the library's CUDA kernels. There is no fallback: if the
library is missing or a call fails, an exception is raised."""
import contextlib
import ctypes
import os
import warnings

import numpy as np
import torch

PKG = os.path.dirname(os.path.abspath(__file__))
LIBRARY = os.path.join(PKG, "libfdecode.so")
DEBUG_LIBRARY = os.path.join(PKG, "libfdecode_debug.so")   # built with -DFD_DEBUG (device-side bounds checks)

FD_OK = 0
FD_TILE_TOKENS = 64
FD_MAX_SPLITS = 65535
FD_MAX_GROUP = 16
ERRORS = {
    -1: "FD_ERR_NULL_POINTER", -2: "FD_ERR_SHAPE", -3: "FD_ERR_GROUP", -4: "FD_ERR_HEAD_DIM",
    -5: "FD_ERR_ALIGNMENT", -6: "FD_ERR_WORKSPACE", -7: "FD_ERR_SPLITS", -8: "FD_ERR_DEVICE",
    -9: "FD_ERR_LAUNCH", -10: "FD_ERR_TIMEOUT", -11: "FD_ERR_CAPACITY", -12: "FD_ERR_STATIC_LIMIT", -13: "FD_ERR_BOUNDS",
    -14: "FD_ERR_OVERLAP",
}
FD_STATIC_SCRATCH_BYTES = 8 << 20
FD_KV_HND, FD_KV_NHD = 0, 1
LAYOUTS = {"HND": FD_KV_HND, "NHD": FD_KV_NHD}


class FdError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {ERRORS.get(code, code)} ({fd_strerror(code)})")


_lib = None
_i, _p, _sz, _f = ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_float
_ll = ctypes.c_longlong


def _newer_sources(path: str) -> list:
    """Sources of the library (decode_attention_07_b200.build.DEPS) modified
    after the library at `path` was built; those not shipped are skipped."""
    from .build import DEPS
    t = os.path.getmtime(path)
    return sorted(os.path.basename(d) for d in DEPS if os.path.exists(d) and os.path.getmtime(d) > t)


def lib() -> ctypes.CDLL:
    """Load libfdecode.so (built in-tree by decode_attention_07_b200.build);
    with FD_DEBUG=1 in the environment, the debug build libfdecode_debug.so."""
    global _lib
    if _lib is None:
        path = DEBUG_LIBRARY if os.environ.get("FD_DEBUG", "0") not in ("", "0") else LIBRARY
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is not built: run `python -c 'import __graft_entry__ as g; g.build()'`")
        stale = _newer_sources(path)
        if stale:
            warnings.warn(f"{os.path.basename(path)} is older than {', '.join(stale)}: the loaded kernels may not be "
                          "the sources' (rebuild with `python -c 'import __graft_entry__ as g; g.build()'`)",
                          RuntimeWarning, stacklevel=2)
        L = ctypes.CDLL(path)
        L.fd_plan.argtypes = [_i] * 5
        L.fd_plan_for_sms.argtypes = [_i] * 6
        L.fd_workspace_bytes.argtypes = [_i] * 6
        L.fd_workspace_bytes.restype = _sz
        compute = [_i] * 5 + [_p, _p, _p, _p, _f, _p, _p, _p, _sz]
        L.fd_decode.argtypes = compute + [_p]
        L.fd_decode_splits.argtypes = compute + [_i, _p]
        L.fd_split.argtypes = compute + [_i, _p]
        L.fd_combine.argtypes = [_i] * 5 + [_p, _p, _p, _p, _sz, _i, _p]
        L.fd_segments.argtypes = [_i, _i, _i, _p, _i, _p, _p, _p, _p, _i]
        L.fd_device_status.argtypes = [_p]
        L.fd_workspace_init.argtypes = [_p, _sz, _p]
        L.fd_decode_static.argtypes = [_i] * 5 + [_p, _p, _p, _p, _f, _p, _p, _p]
        L.fd_decode_paged.argtypes = [_i] * 8 + [_p, _p, _p, _p, _p, _f, _p, _p, _p, _sz, _i, _p]
        L.fd_decode_multi.argtypes = [_i] * 6 + [_p, _p, _p, _p, _f, _p, _p, _p, _sz, _i, _p]
        L.fd_decode_quant.argtypes = [_i] * 7 + [_p, _p, _p, _p, _p, _p, _f, _p, _p, _p, _sz, _i, _p]
        L.fd_merge_partials.argtypes = [_i, _i, _i, _p, _p, _p, _p, _p]
        L.fd_read_probe.argtypes = [_p, _sz, _p, _p]
        L.fd_decode_quant_paged.argtypes = [_i] * 10 + [_p] * 7 + [_f, _p, _p, _p, _sz, _i, _p]
        L.fd_decode_quant_block.argtypes = [_i] * 8 + [_p] * 6 + [_f, _p, _p, _p, _sz, _i, _p]
        L.fd_decode_quant_block_paged.argtypes = [_i] * 11 + [_p] * 7 + [_f, _p, _p, _p, _sz, _i, _p]
        L.fd_quant_append.argtypes = [_i] * 7 + [_p, _p, _ll, _ll, _ll] + [_p] * 7
        L.fd_quant_append_paged.argtypes = [_i] * 10 + [_p, _p, _ll, _ll, _ll] + [_p] * 8
        L.fd_weights_workspace_bytes.argtypes = [_i] * 7
        L.fd_weights_workspace_bytes.restype = _sz
        L.fd_decode_weights.argtypes = [_i] * 6 + [_p, _p, _p, _p, _f] + [_p] * 5 + [_sz, _i, _p]
        L.fd_evict.argtypes = [_i] * 7 + [_p] * 10
        L.fd_strerror.argtypes = [_i]
        L.fd_strerror.restype = ctypes.c_char_p
        L.fd_version.argtypes = []
        for name in ("fd_plan", "fd_plan_for_sms", "fd_decode", "fd_decode_splits", "fd_split", "fd_combine",
                     "fd_segments", "fd_device_status", "fd_version", "fd_workspace_init", "fd_decode_static",
                     "fd_decode_paged", "fd_decode_multi", "fd_decode_quant", "fd_merge_partials", "fd_read_probe", "fd_decode_quant_paged",
                     "fd_decode_quant_block", "fd_decode_quant_block_paged", "fd_quant_append", "fd_quant_append_paged",
                     "fd_decode_weights", "fd_evict"):
            getattr(L, name).restype = _i
        _lib = L
    return _lib


def _check(rc: int, what: str) -> int:
    if rc < 0:
        raise FdError(rc, what)
    return rc


def _stream(stream, device) -> int:
    if stream is None:
        return torch.cuda.current_stream(device).cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


@contextlib.contextmanager
def _on_stream(stream, device):
    """For calls that allocate: `stream` (a Stream, a raw handle, None: the
    current one) as the current stream, so that what is allocated inside is
    filled in the call's order and, once dropped, only reused after the call.
    Yields a function that passes on its arguments, the call's results, which
    the caller goes on using on the stream that was current outside."""
    if stream is None:
        yield lambda *tensors: tensors
        return
    if not isinstance(stream, torch.cuda.Stream):
        handle = int(stream)
        stream = torch.cuda.ExternalStream(handle, device=device) if handle else torch.cuda.default_stream(device)
    outer = torch.cuda.current_stream(device)

    def hand_over(*tensors):
        if outer != stream:
            for t in tensors:
                t.record_stream(outer)
        return tensors

    with torch.cuda.stream(stream):
        yield hand_over


def _shapes(q, k_cache, v_cache):
    if q.dim() != 3 or k_cache.dim() != 4 or v_cache.shape != k_cache.shape:
        raise ValueError("expected q [B,Hq,D] and k_cache, v_cache [B,Hkv,Lmax,D]")
    B, Hq, D = q.shape
    B2, Hkv, Lmax, D2 = k_cache.shape
    if B2 != B or D2 != D:
        raise ValueError("q and the caches disagree on B or D")
    for t, name in ((q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache")):
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous bf16 CUDA tensor")
    return B, Hq, Hkv, D, Lmax


def _outputs(out, lse, B, Hq, D):
    if out.shape != (B, Hq, D) or lse.shape != (B, Hq):
        raise ValueError("out must be [B,Hq,D] and lse [B,Hq]")
    for t, name in ((out, "out"), (lse, "lse")):
        if t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous fp32 CUDA tensor")


def _seqlens(seqlens, B):
    if seqlens.shape != (B,) or seqlens.dtype != torch.int32 or not seqlens.is_cuda or not seqlens.is_contiguous():
        raise ValueError("seqlens must be a contiguous int32 CUDA tensor of shape [B]")


def _ws(workspace):
    if workspace is None:
        return None, 0
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _one_device(*tensors):
    """Index of the device that holds all of `tensors` (None entries aside)."""
    devices = {t.device.index for t in tensors if t is not None}
    if len(devices) != 1:
        raise ValueError("all tensors must be on one device")
    return devices.pop()


def _prepared(what, tensors, args):
    """A no-argument callable that runs entry point `what` with `args`, with
    the device of `tensors` as the current one. It holds the tensors (None
    entries aside): their memory stays theirs as long as it lives."""
    device = _one_device(*tensors)
    fn = getattr(lib(), what)
    # converted once here, not on every call
    args = tuple(t(a) if a is not None else a for t, a in zip(fn.argtypes, args))

    def call():
        if torch.cuda.current_device() == device:
            rc = fn(*args)
        else:
            with torch.cuda.device(device):
                rc = fn(*args)
        if rc != 0:
            raise FdError(rc, what)

    call.tensors = tensors
    return call


# ---------------------------------------------------------------- the ABI --

def fd_plan(B: int, Hq: int, Hkv: int, D: int, max_len: int) -> int:
    return _check(lib().fd_plan(B, Hq, Hkv, D, max_len), "fd_plan")


def fd_plan_for_sms(B: int, Hq: int, Hkv: int, D: int, max_len: int, num_sms: int) -> int:
    return _check(lib().fd_plan_for_sms(B, Hq, Hkv, D, max_len, num_sms), "fd_plan_for_sms")


def fd_workspace_bytes(B: int, Hq: int, Hkv: int, D: int, max_len: int, num_splits: int) -> int:
    return int(lib().fd_workspace_bytes(B, Hq, Hkv, D, max_len, num_splits))


def fd_decode(q, k_cache, v_cache, seqlens, scale, out, lse, workspace=None, stream=None):
    B, Hq, Hkv, D, Lmax = _shapes(q, k_cache, v_cache)
    _outputs(out, lse, B, Hq, D)
    _seqlens(seqlens, B)
    wp, wb = _ws(workspace)
    _check(lib().fd_decode(B, Hq, Hkv, D, Lmax, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                           seqlens.data_ptr(), float(scale), out.data_ptr(), lse.data_ptr(), wp, wb,
                           _stream(stream, q.device)), "fd_decode")


def fd_decode_splits(q, k_cache, v_cache, seqlens, scale, out, lse, workspace, num_splits, stream=None):
    B, Hq, Hkv, D, Lmax = _shapes(q, k_cache, v_cache)
    _outputs(out, lse, B, Hq, D)
    _seqlens(seqlens, B)
    wp, wb = _ws(workspace)
    _check(lib().fd_decode_splits(B, Hq, Hkv, D, Lmax, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                  seqlens.data_ptr(), float(scale), out.data_ptr(), lse.data_ptr(), wp, wb,
                                  int(num_splits), _stream(stream, q.device)), "fd_decode_splits")


def fd_split(q, k_cache, v_cache, seqlens, scale, out, lse, workspace, num_splits, stream=None):
    B, Hq, Hkv, D, Lmax = _shapes(q, k_cache, v_cache)
    _outputs(out, lse, B, Hq, D)
    _seqlens(seqlens, B)
    wp, wb = _ws(workspace)
    _check(lib().fd_split(B, Hq, Hkv, D, Lmax, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                          seqlens.data_ptr(), float(scale), out.data_ptr(), lse.data_ptr(), wp, wb,
                          int(num_splits), _stream(stream, q.device)), "fd_split")


def fd_combine(B, Hq, Hkv, D, max_len, seqlens, out, lse, workspace, num_splits, stream=None):
    _outputs(out, lse, B, Hq, D)
    _seqlens(seqlens, B)
    wp, wb = _ws(workspace)
    _check(lib().fd_combine(B, Hq, Hkv, D, max_len, seqlens.data_ptr(), out.data_ptr(), lse.data_ptr(), wp, wb,
                            int(num_splits), _stream(stream, out.device)), "fd_combine")


def fd_segments(B: int, Hkv: int, max_len: int, seqlens_host, num_splits: int) -> dict:
    """Where the split stage cuts each row (host computation). Returns numpy
    arrays indexed by workspace slot: row (-1 = unused), begin, end, whole."""
    lens = np.ascontiguousarray(np.asarray(seqlens_host, dtype=np.int32).reshape(B))
    cap = num_splits + B * Hkv - 1
    arrs = [np.zeros(cap, np.int32) for _ in range(4)]
    n = _check(lib().fd_segments(B, Hkv, max_len, lens.ctypes.data, int(num_splits),
                                 *(a.ctypes.data for a in arrs), cap), "fd_segments")
    return dict(row=arrs[0][:n], begin=arrs[1][:n], end=arrs[2][:n], whole=arrs[3][:n])


def fd_decode_static(q, k_cache, v_cache, seqlens, scale, out, lse, stream=None):
    """fd_decode without a workspace argument: the library's fixed device
    scratch buffer is used instead (see include/fd.h)."""
    B, Hq, Hkv, D, Lmax = _shapes(q, k_cache, v_cache)
    _outputs(out, lse, B, Hq, D)
    _seqlens(seqlens, B)
    _check(lib().fd_decode_static(B, Hq, Hkv, D, Lmax, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                  seqlens.data_ptr(), float(scale), out.data_ptr(), lse.data_ptr(),
                                  _stream(stream, q.device)), "fd_decode_static")


def fd_decode_multi(q, k_cache, v_cache, seqlens, scale, out, lse, workspace=None, num_splits=0, stream=None):
    """Several queries per sequence: q [B, q_len, Hq, D], out [B, q_len, Hq, D],
    lse [B, q_len, Hq]; query j sees the first seqlens[b] - (q_len-1-j) tokens.
    num_splits 0 lets the library plan the split count."""
    prepare_decode_multi(q, k_cache, v_cache, seqlens, scale, out, lse, workspace, num_splits, stream)()


def decode_multi(q, k_cache, v_cache, seqlens, scale, num_splits=None, stream=None):
    """Allocate out / lse / workspace with torch and run fd_decode_multi."""
    B, q_len, Hq, D = q.shape
    Hkv, Lmax = k_cache.shape[1], k_cache.shape[2]
    with _on_stream(stream, q.device) as hand_over:
        S = fd_plan(B, Hq, Hkv, D, Lmax) if num_splits is None else int(num_splits)
        nbytes = fd_workspace_bytes(B, Hq * q_len, Hkv, D, Lmax, S)
        ws = torch.zeros(nbytes, dtype=torch.uint8, device=q.device) if nbytes else None
        out = torch.empty((B, q_len, Hq, D), dtype=torch.float32, device=q.device)
        lse = torch.empty((B, q_len, Hq), dtype=torch.float32, device=q.device)
        fd_decode_multi(q, k_cache, v_cache, seqlens, scale, out, lse, ws, S, stream)
        return hand_over(out, lse)


def _paged_shapes(q, k_pages, v_pages, block_table, layout, pool_dtype=torch.bfloat16):
    if layout not in LAYOUTS:
        raise ValueError("layout must be 'HND' ([pages, Hkv, page_size, D]) or 'NHD' ([pages, page_size, Hkv, D])")
    if q.dim() not in (3, 4) or k_pages.dim() != 4 or v_pages.shape != k_pages.shape or block_table.dim() != 2:
        raise ValueError("expected q [B,Hq,D] (or [B,q_len,Hq,D]), k_pages/v_pages 4-D, block_table [B, max_pages]")
    B, Hq, D = q.shape[0], q.shape[-2], q.shape[-1]
    if layout == "HND":
        num_pages, Hkv, page_size, D2 = k_pages.shape
    else:
        num_pages, page_size, Hkv, D2 = k_pages.shape
    if D2 != D or block_table.shape[0] != B:
        raise ValueError("q, pages and block_table disagree on B or D")
    if q.dtype != torch.bfloat16 or not q.is_cuda or not q.is_contiguous():
        raise ValueError("q must be a contiguous bf16 CUDA tensor")
    for t, name in ((k_pages, "k_pages"), (v_pages, "v_pages")):
        if t.dtype != pool_dtype or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {pool_dtype} CUDA tensor")
    if block_table.dtype != torch.int32 or not block_table.is_cuda or not block_table.is_contiguous():
        raise ValueError("block_table must be a contiguous int32 CUDA tensor")
    return B, Hq, Hkv, D, page_size, num_pages, block_table.shape[1]


def fd_decode_paged(q, k_pages, v_pages, block_table, seqlens, scale, out, lse, workspace=None, layout="HND",
                    num_splits=0, stream=None):
    B, Hq, Hkv, D, page_size, num_pages, max_pages = _paged_shapes(q, k_pages, v_pages, block_table, layout)
    _outputs(out, lse, B, Hq, D)
    _seqlens(seqlens, B)
    wp, wb = _ws(workspace)
    _check(lib().fd_decode_paged(B, Hq, Hkv, D, page_size, num_pages, max_pages, LAYOUTS[layout], q.data_ptr(),
                                 k_pages.data_ptr(), v_pages.data_ptr(), block_table.data_ptr(), seqlens.data_ptr(),
                                 float(scale), out.data_ptr(), lse.data_ptr(), wp, wb, int(num_splits),
                                 _stream(stream, q.device)), "fd_decode_paged")


def prepare_decode_paged(q, k_pages, v_pages, block_table, seqlens, scale, out, lse, workspace=None, layout="HND",
                         num_splits=0, stream=None):
    """Check and marshal once; return a no-argument callable that enqueues
    fd_decode_paged with those pointers."""
    B, Hq, Hkv, D, page_size, num_pages, max_pages = _paged_shapes(q, k_pages, v_pages, block_table, layout)
    _outputs(out, lse, B, Hq, D)
    _seqlens(seqlens, B)
    wp, wb = _ws(workspace)
    return _prepared("fd_decode_paged", (q, k_pages, v_pages, block_table, seqlens, out, lse, workspace), (
        B, Hq, Hkv, D, page_size, num_pages, max_pages, LAYOUTS[layout], q.data_ptr(), k_pages.data_ptr(),
        v_pages.data_ptr(), block_table.data_ptr(), seqlens.data_ptr(), float(scale), out.data_ptr(), lse.data_ptr(), wp,
        wb, int(num_splits), _stream(stream, q.device)))


def prepare_decode_quant_paged(q, k_pages, v_pages, k_scale, v_scale, kv_type, block_table, seqlens, scale, out, lse,
                               workspace=None, layout="HND", num_splits=0, stream=None):
    """prepare_decode for fd_decode_quant_paged: 8-bit page pools (uint8,
    layouts as fd_decode_paged), per-kv-head float32 scales, kv_type "e4m3"
    or "int8"; q [B, Hq, D] or [B, q_len, Hq, D], out / lse shaped to match."""
    if kv_type not in KV_CODES:
        raise ValueError("kv_type must be 'e4m3' or 'int8'")
    B, Hq, Hkv, D, page_size, num_pages, max_pages = _paged_shapes(q, k_pages, v_pages, block_table, layout,
                                                                   torch.uint8)
    q_len = 1 if q.dim() == 3 else q.shape[1]
    for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
        if t.shape != (Hkv,) or t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous float32 CUDA tensor of shape [Hkv]")
    if out.shape != q.shape or lse.shape != q.shape[:-1]:
        raise ValueError("out must be shaped like q and lse like q without D")
    for t, name in ((out, "out"), (lse, "lse")):
        if t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous fp32 CUDA tensor")
    _seqlens(seqlens, B)
    wp, wb = _ws(workspace)
    tensors = (q, k_pages, v_pages, k_scale, v_scale, block_table, seqlens, out, lse, workspace)
    return _prepared("fd_decode_quant_paged", tensors, (
        B, q_len, Hq, Hkv, D, page_size, num_pages, max_pages, LAYOUTS[layout], KV_CODES[kv_type], q.data_ptr(),
        k_pages.data_ptr(), v_pages.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), block_table.data_ptr(),
        seqlens.data_ptr(), float(scale), out.data_ptr(), lse.data_ptr(), wp, wb, int(num_splits),
        _stream(stream, q.device)))


def decode_quant_paged(q, k_pages, v_pages, k_scale, v_scale, kv_type, block_table, seqlens, scale, layout="HND",
                       num_splits=None, stream=None):
    """Allocate out / lse / workspace with torch and run fd_decode_quant_paged."""
    B, Hq, Hkv, D, page_size, num_pages, max_pages = _paged_shapes(q, k_pages, v_pages, block_table, layout,
                                                                   torch.uint8)
    q_len = 1 if q.dim() == 3 else q.shape[1]
    Lmax = max_pages * page_size
    with _on_stream(stream, q.device) as hand_over:
        S = fd_plan(B, Hq, Hkv, D, Lmax) if num_splits is None else int(num_splits)
        nbytes = fd_workspace_bytes(B, Hq * q_len, Hkv, D, Lmax, S)
        ws = torch.zeros(nbytes, dtype=torch.uint8, device=q.device) if nbytes else None
        out = torch.empty(q.shape, dtype=torch.float32, device=q.device)
        lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device)
        prepare_decode_quant_paged(q, k_pages, v_pages, k_scale, v_scale, kv_type, block_table, seqlens, scale, out,
                                   lse, ws, layout, S, stream)()
        return hand_over(out, lse)


def decode_paged(q, k_pages, v_pages, block_table, seqlens, scale, layout="HND", num_splits=None, stream=None):
    """Allocate out / lse / workspace with torch and run fd_decode_paged."""
    B, Hq, Hkv, D, page_size, num_pages, max_pages = _paged_shapes(q, k_pages, v_pages, block_table, layout)
    Lmax = max_pages * page_size
    with _on_stream(stream, q.device) as hand_over:
        S = fd_plan(B, Hq, Hkv, D, Lmax) if num_splits is None else int(num_splits)
        nbytes = fd_workspace_bytes(B, Hq, Hkv, D, Lmax, S)
        ws = torch.zeros(nbytes, dtype=torch.uint8, device=q.device) if nbytes else None
        out = torch.empty((B, Hq, D), dtype=torch.float32, device=q.device)
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
        fd_decode_paged(q, k_pages, v_pages, block_table, seqlens, scale, out, lse, ws, layout, S, stream)
        return hand_over(out, lse)


def fd_workspace_init(workspace, stream=None):
    wp, wb = _ws(workspace)
    if wb:
        _check(lib().fd_workspace_init(wp, wb, _stream(stream, workspace.device)), "fd_workspace_init")


def fd_device_status(stream=None, device=None) -> int:
    return lib().fd_device_status(_stream(stream, device))


def fd_strerror(code: int) -> str:
    return lib().fd_strerror(int(code)).decode()


def fd_version() -> int:
    return lib().fd_version()


# ------------------------------------------------------------ convenience --
# Prepared calls, and calls that allocate their outputs and workspace: these
# allocate on the stream they run on, and their results may be used and dropped
# on the stream that was current, once that has waited for the call.

def prepare_decode(q, k_cache, v_cache, seqlens, scale, out, lse, workspace=None, num_splits=None, stream=None):
    """Check and marshal the arguments once; return a no-argument callable
    that enqueues fd_decode_splits with those pointers (for decode loops that
    reuse the same buffers). The planned split count is used by default."""
    B, Hq, Hkv, D, Lmax = _shapes(q, k_cache, v_cache)
    _outputs(out, lse, B, Hq, D)
    _seqlens(seqlens, B)
    S = fd_plan(B, Hq, Hkv, D, Lmax) if num_splits is None else int(num_splits)
    wp, wb = _ws(workspace)
    call = _prepared("fd_decode_splits", (q, k_cache, v_cache, seqlens, out, lse, workspace), (
        B, Hq, Hkv, D, Lmax, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), seqlens.data_ptr(), float(scale),
        out.data_ptr(), lse.data_ptr(), wp, wb, S, _stream(stream, q.device)))
    call.num_splits = S
    return call


def prepare_decode_multi(q, k_cache, v_cache, seqlens, scale, out, lse, workspace=None, num_splits=None,
                         stream=None):
    """prepare_decode for fd_decode_multi: q [B, q_len, Hq, D], out
    [B, q_len, Hq, D], lse [B, q_len, Hq]."""
    if q.dim() != 4 or not q.is_contiguous():
        raise ValueError("q must be a contiguous [B, q_len, Hq, D] tensor")
    B, q_len, Hq, D = q.shape
    _, _, Hkv, _, Lmax = _shapes(q.view(B, q_len * Hq, D), k_cache, v_cache)
    if out.shape != (B, q_len, Hq, D) or lse.shape != (B, q_len, Hq):
        raise ValueError("out must be [B,q_len,Hq,D] and lse [B,q_len,Hq]")
    for t, name in ((out, "out"), (lse, "lse")):
        if t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous fp32 CUDA tensor")
    _seqlens(seqlens, B)
    S = fd_plan(B, Hq, Hkv, D, Lmax) if num_splits is None else int(num_splits)
    wp, wb = _ws(workspace)
    call = _prepared("fd_decode_multi", (q, k_cache, v_cache, seqlens, out, lse, workspace), (
        B, q_len, Hq, Hkv, D, Lmax, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), seqlens.data_ptr(),
        float(scale), out.data_ptr(), lse.data_ptr(), wp, wb, S, _stream(stream, q.device)))
    call.num_splits = S
    return call


FD_KV_E4M3, FD_KV_INT8 = 1, 2
KV_CODES = {"e4m3": FD_KV_E4M3, "int8": FD_KV_INT8}


def prepare_decode_quant(q, k_codes, v_codes, k_scale, v_scale, kv_type, seqlens, scale, out, lse, workspace=None,
                         num_splits=None, stream=None):
    """prepare_decode for fd_decode_quant: an 8-bit cache (k_codes / v_codes
    uint8 [B, Hkv, Lmax, D], k_scale / v_scale float32 [Hkv], kv_type "e4m3"
    or "int8"); q [B, Hq, D] (one query) or [B, q_len, Hq, D], out / lse
    shaped to match."""
    if kv_type not in KV_CODES:
        raise ValueError("kv_type must be 'e4m3' or 'int8'")
    if q.dim() == 3:
        B, Hq, D = q.shape
        q_len = 1
    elif q.dim() == 4:
        B, q_len, Hq, D = q.shape
    else:
        raise ValueError("q must be [B, Hq, D] or [B, q_len, Hq, D]")
    if q.dtype != torch.bfloat16 or not q.is_cuda or not q.is_contiguous():
        raise ValueError("q must be a contiguous bf16 CUDA tensor")
    if k_codes.dim() != 4 or v_codes.shape != k_codes.shape or k_codes.shape[0] != B or k_codes.shape[3] != D:
        raise ValueError("k_codes, v_codes must be [B, Hkv, Lmax, D]")
    _, Hkv, Lmax, _ = k_codes.shape
    for t, name in ((k_codes, "k_codes"), (v_codes, "v_codes")):
        if t.dtype != torch.uint8 or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous uint8 CUDA tensor")
    for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
        if t.shape != (Hkv,) or t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous float32 CUDA tensor of shape [Hkv]")
    oshape = q.shape[:-1]
    if out.shape != q.shape or lse.shape != oshape:
        raise ValueError("out must be shaped like q and lse like q without D")
    for t, name in ((out, "out"), (lse, "lse")):
        if t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous fp32 CUDA tensor")
    _seqlens(seqlens, B)
    S = fd_plan(B, Hq, Hkv, D, Lmax) if num_splits is None else int(num_splits)
    wp, wb = _ws(workspace)
    tensors = (q, k_codes, v_codes, k_scale, v_scale, seqlens, out, lse, workspace)
    call = _prepared("fd_decode_quant", tensors, (
        B, q_len, Hq, Hkv, D, Lmax, KV_CODES[kv_type], q.data_ptr(), k_codes.data_ptr(), v_codes.data_ptr(),
        k_scale.data_ptr(), v_scale.data_ptr(), seqlens.data_ptr(), float(scale), out.data_ptr(), lse.data_ptr(), wp, wb,
        S, _stream(stream, q.device)))
    call.num_splits = S
    return call


def fd_decode_quant(q, k_codes, v_codes, k_scale, v_scale, kv_type, seqlens, scale, out, lse, workspace=None,
                    num_splits=0, stream=None):
    """Attention over an 8-bit key/value cache (see prepare_decode_quant);
    num_splits 0 lets the library plan the split count."""
    prepare_decode_quant(q, k_codes, v_codes, k_scale, v_scale, kv_type, seqlens, scale, out, lse, workspace,
                         num_splits, stream)()


def quant_workspace_bytes(q, k_codes, num_splits):
    """Workspace bytes fd_decode_quant needs for these shapes."""
    q_len = 1 if q.dim() == 3 else q.shape[1]
    B, Hq, D = q.shape[0], q.shape[-2], q.shape[-1]
    return fd_workspace_bytes(B, Hq * q_len, k_codes.shape[1], D, k_codes.shape[2], num_splits)


def decode_quant(q, k_codes, v_codes, k_scale, v_scale, kv_type, seqlens, scale, num_splits=None, stream=None):
    """Allocate out / lse / workspace with torch and run fd_decode_quant."""
    B, Hq, D = q.shape[0], q.shape[-2], q.shape[-1]
    Hkv, Lmax = k_codes.shape[1], k_codes.shape[2]
    with _on_stream(stream, q.device) as hand_over:
        S = fd_plan(B, Hq, Hkv, D, Lmax) if num_splits is None else int(num_splits)
        nbytes = quant_workspace_bytes(q, k_codes, S)
        ws = torch.zeros(nbytes, dtype=torch.uint8, device=q.device) if nbytes else None
        out = torch.empty(q.shape, dtype=torch.float32, device=q.device)
        lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device)
        fd_decode_quant(q, k_codes, v_codes, k_scale, v_scale, kv_type, seqlens, scale, out, lse, ws, S, stream)
        return hand_over(out, lse)


def fd_merge_partials(part_out, part_lse, out, lse, stream=None):
    """Merge R partial results per row: part_out [R, ..., D] and part_lse
    [R, ...] (fp32, contiguous, CUDA) into out [..., D] and lse [...]."""
    if part_out.dim() < 2 or part_lse.shape != part_out.shape[:-1]:
        raise ValueError("part_out must be [R, ..., D] and part_lse [R, ...]")
    R, D = part_out.shape[0], part_out.shape[-1]
    rows = part_lse[0].numel()
    if out.shape != part_out.shape[1:] or lse.shape != part_lse.shape[1:]:
        raise ValueError("out / lse must be shaped like one part")
    for t, name in ((part_out, "part_out"), (part_lse, "part_lse"), (out, "out"), (lse, "lse")):
        if t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous fp32 CUDA tensor")
    _check(lib().fd_merge_partials(R, rows, D, part_out.data_ptr(), part_lse.data_ptr(), out.data_ptr(),
                                   lse.data_ptr(), _stream(stream, out.device)), "fd_merge_partials")


def fd_read_probe(buf, sink, stream=None):
    """Read every byte of the CUDA tensor `buf` once (HBM read-bandwidth
    probe); `sink` is a one-element int64 CUDA tensor."""
    if not buf.is_cuda or not buf.is_contiguous() or sink.dtype != torch.int64 or not sink.is_cuda:
        raise ValueError("buf must be a contiguous CUDA tensor and sink an int64 CUDA tensor")
    nbytes = buf.numel() * buf.element_size()
    _check(lib().fd_read_probe(buf.data_ptr(), nbytes, sink.data_ptr(), _stream(stream, buf.device)),
           "fd_read_probe")


def workspace_layout(B, Hq, Hkv, D, num_splits):
    """(slots, g, byte offset of seg_lse, byte offset of the counters) of the
    documented workspace layout. The counters are B*Hkv row counters followed
    by `slots` chunk counters, all int32."""
    slots = num_splits + B * Hkv - 1
    g = Hq // Hkv
    off = (slots * g * D * 4 + 255) // 256 * 256
    tick = off + (slots * g * 4 + 255) // 256 * 256
    return slots, g, off, tick


def decode(q, k_cache, v_cache, seqlens, scale, num_splits=None, stream=None):
    """Allocate out / lse / workspace with torch and run fd_decode (or
    fd_decode_splits when num_splits is given). Returns (out, lse)."""
    B, Hq, Hkv, D, Lmax = _shapes(q, k_cache, v_cache)
    with _on_stream(stream, q.device) as hand_over:
        S = fd_plan(B, Hq, Hkv, D, Lmax) if num_splits is None else int(num_splits)
        nbytes = fd_workspace_bytes(B, Hq, Hkv, D, Lmax, S)
        ws = torch.zeros(nbytes, dtype=torch.uint8, device=q.device) if nbytes else None
        out = torch.empty((B, Hq, D), dtype=torch.float32, device=q.device)
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
        fd_decode_splits(q, k_cache, v_cache, seqlens, scale, out, lse, ws, S, stream)
        return hand_over(out, lse)


# -------------------------------------------------------- cache compression --
# 8-bit caches with one scale per block of tokens (append and attention),
# attention weights per cached token, eviction by them (see include/fd.h).

FD_BLOCK_TOKENS = (16, 32, 64, 128)


def _tensor(t, name, shape, dtype):
    if t.shape != shape or t.dtype != dtype or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor of shape {list(shape)}")


def _planned(device, B, Hq, Hkv, D, Lmax, num_splits):
    if num_splits is not None:
        return int(num_splits)
    with torch.cuda.device(device):
        return fd_plan(B, Hq, Hkv, D, Lmax)


def _query(q):
    if q.dim() not in (3, 4) or q.dtype != torch.bfloat16 or not q.is_cuda or not q.is_contiguous():
        raise ValueError("q must be a contiguous bf16 CUDA tensor [B, Hq, D] or [B, q_len, Hq, D]")
    return q.shape[0], 1 if q.dim() == 3 else q.shape[1], q.shape[-2], q.shape[-1]


def _block_codes(k_codes, v_codes, k_scale, v_scale, kv_type, block_tokens):
    """(B, Hkv, Lmax, D) of a contiguous block-scaled cache."""
    if kv_type not in KV_CODES:
        raise ValueError("kv_type must be 'e4m3' or 'int8'")
    if block_tokens not in FD_BLOCK_TOKENS:
        raise ValueError(f"block_tokens must be one of {FD_BLOCK_TOKENS}")
    if k_codes.dim() != 4:
        raise ValueError("k_codes, v_codes must be [B, Hkv, Lmax, D]")
    B, Hkv, Lmax, D = k_codes.shape
    for t, name in ((k_codes, "k_codes"), (v_codes, "v_codes")):
        _tensor(t, name, k_codes.shape, torch.uint8)
    for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
        _tensor(t, name, (B, Hkv, -(-Lmax // block_tokens)), torch.float32)
    return B, Hkv, Lmax, D


def _block_pages(k_pages, v_pages, k_scale, v_scale, kv_type, block_tokens, block_table, layout):
    """(Hkv, D, page_size, num_pages, max_pages) of a paged block-scaled cache."""
    if kv_type not in KV_CODES:
        raise ValueError("kv_type must be 'e4m3' or 'int8'")
    if layout not in LAYOUTS:
        raise ValueError("layout must be 'HND' ([pages, Hkv, page_size, D]) or 'NHD' ([pages, page_size, Hkv, D])")
    if k_pages.dim() != 4 or block_table.dim() != 2:
        raise ValueError("expected k_pages, v_pages 4-D and block_table [B, max_pages]")
    for t, name in ((k_pages, "k_pages"), (v_pages, "v_pages")):
        _tensor(t, name, k_pages.shape, torch.uint8)
    num_pages, page_size, D = k_pages.shape[0], k_pages.shape[2 if layout == "HND" else 1], k_pages.shape[3]
    Hkv = k_pages.shape[1 if layout == "HND" else 2]
    if block_tokens not in FD_BLOCK_TOKENS or block_tokens > page_size:
        raise ValueError(f"block_tokens must be one of {FD_BLOCK_TOKENS} and at most the page size")
    for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
        _tensor(t, name, (num_pages, Hkv, page_size // block_tokens), torch.float32)
    _tensor(block_table, "block_table", block_table.shape, torch.int32)
    return Hkv, D, page_size, num_pages, block_table.shape[1]


def _block_outputs(q, out, lse):
    _tensor(out, "out", q.shape, torch.float32)
    _tensor(lse, "lse", q.shape[:-1], torch.float32)


def prepare_decode_quant_block(q, k_codes, v_codes, k_scale, v_scale, kv_type, block_tokens, seqlens, scale, out, lse,
                               workspace=None, num_splits=None, stream=None):
    """Check and marshal once; return a no-argument callable that enqueues
    fd_decode_quant_block with those pointers on `stream` (None: the stream
    current now): attention over uint8 codes [B, Hkv, Lmax, D] with float32
    scales [B, Hkv, ceil(Lmax / block_tokens)]; q [B, Hq, D] or
    [B, q_len, Hq, D], out / lse shaped to match; workspace as for
    fd_decode_quant (quant_workspace_bytes)."""
    B, Hkv, Lmax, D = _block_codes(k_codes, v_codes, k_scale, v_scale, kv_type, block_tokens)
    Bq, q_len, Hq, Dq = _query(q)
    if Bq != B or Dq != D:
        raise ValueError("q and the cache disagree on B or D")
    _block_outputs(q, out, lse)
    _tensor(seqlens, "seqlens", (B,), torch.int32)
    wp, wb = _ws(workspace)
    tensors = (q, k_codes, v_codes, k_scale, v_scale, seqlens, out, lse, workspace)
    S = _planned(q.device.index, B, Hq, Hkv, D, Lmax, num_splits)
    call = _prepared("fd_decode_quant_block", tensors, (
        B, q_len, Hq, Hkv, D, Lmax, block_tokens, KV_CODES[kv_type], q.data_ptr(), k_codes.data_ptr(),
        v_codes.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), seqlens.data_ptr(), float(scale), out.data_ptr(),
        lse.data_ptr(), wp, wb, S, _stream(stream, q.device)))
    call.num_splits = S
    return call


def fd_decode_quant_block(q, k_codes, v_codes, k_scale, v_scale, kv_type, block_tokens, seqlens, scale, out, lse,
                          workspace=None, num_splits=0, stream=None):
    """prepare_decode_quant_block, enqueued once; num_splits 0 lets the library
    plan the split count."""
    prepare_decode_quant_block(q, k_codes, v_codes, k_scale, v_scale, kv_type, block_tokens, seqlens, scale, out, lse,
                               workspace, num_splits, stream)()


def decode_quant_block(q, k_codes, v_codes, k_scale, v_scale, kv_type, block_tokens, seqlens, scale, num_splits=None,
                       stream=None):
    """Allocate out / lse / workspace with torch and run fd_decode_quant_block."""
    _, Hkv, Lmax, _ = _block_codes(k_codes, v_codes, k_scale, v_scale, kv_type, block_tokens)
    B, _, Hq, D = _query(q)
    S = _planned(q.device.index, B, Hq, Hkv, D, Lmax, num_splits)
    nbytes = quant_workspace_bytes(q, k_codes, S)
    with _on_stream(stream, q.device) as hand_over:
        ws = torch.zeros(nbytes, dtype=torch.uint8, device=q.device) if nbytes else None
        out = torch.empty(q.shape, dtype=torch.float32, device=q.device)
        lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device)
        fd_decode_quant_block(q, k_codes, v_codes, k_scale, v_scale, kv_type, block_tokens, seqlens, scale, out, lse, ws,
                              S, stream)
        return hand_over(out, lse)


def prepare_decode_quant_block_paged(q, k_pages, v_pages, k_scale, v_scale, kv_type, block_tokens, block_table, seqlens,
                                     scale, out, lse, workspace=None, layout="HND", num_splits=None, stream=None):
    """prepare_decode_quant_block over page pools: codes as for
    fd_decode_quant_paged, scales [num_pages, Hkv, page_size / block_tokens]."""
    Hkv, D, page_size, num_pages, max_pages = _block_pages(k_pages, v_pages, k_scale, v_scale, kv_type, block_tokens,
                                                           block_table, layout)
    B, q_len, Hq, Dq = _query(q)
    if Dq != D or block_table.shape[0] != B:
        raise ValueError("q, pages and block_table disagree on B or D")
    _block_outputs(q, out, lse)
    _tensor(seqlens, "seqlens", (B,), torch.int32)
    wp, wb = _ws(workspace)
    tensors = (q, k_pages, v_pages, k_scale, v_scale, block_table, seqlens, out, lse, workspace)
    S = _planned(q.device.index, B, Hq, Hkv, D, max_pages * page_size, num_splits)
    call = _prepared("fd_decode_quant_block_paged", tensors, (
        B, q_len, Hq, Hkv, D, page_size, num_pages, max_pages, LAYOUTS[layout], block_tokens, KV_CODES[kv_type],
        q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
        block_table.data_ptr(), seqlens.data_ptr(), float(scale), out.data_ptr(), lse.data_ptr(), wp, wb, S,
        _stream(stream, q.device)))
    call.num_splits = S
    return call


def fd_decode_quant_block_paged(q, k_pages, v_pages, k_scale, v_scale, kv_type, block_tokens, block_table, seqlens,
                                scale, out, lse, workspace=None, layout="HND", num_splits=0, stream=None):
    """prepare_decode_quant_block_paged, enqueued once."""
    prepare_decode_quant_block_paged(q, k_pages, v_pages, k_scale, v_scale, kv_type, block_tokens, block_table, seqlens,
                                     scale, out, lse, workspace, layout, num_splits, stream)()


def decode_quant_block_paged(q, k_pages, v_pages, k_scale, v_scale, kv_type, block_tokens, block_table, seqlens, scale,
                             layout="HND", num_splits=None, stream=None):
    """Allocate out / lse / workspace with torch and run
    fd_decode_quant_block_paged."""
    Hkv, D, page_size, _, max_pages = _block_pages(k_pages, v_pages, k_scale, v_scale, kv_type, block_tokens,
                                                   block_table, layout)
    B, q_len, Hq, _ = _query(q)
    Lmax = max_pages * page_size
    S = _planned(q.device.index, B, Hq, Hkv, D, Lmax, num_splits)
    nbytes = fd_workspace_bytes(B, Hq * q_len, Hkv, D, Lmax, S)
    with _on_stream(stream, q.device) as hand_over:
        ws = torch.zeros(nbytes, dtype=torch.uint8, device=q.device) if nbytes else None
        out = torch.empty(q.shape, dtype=torch.float32, device=q.device)
        lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device)
        fd_decode_quant_block_paged(q, k_pages, v_pages, k_scale, v_scale, kv_type, block_tokens, block_table, seqlens,
                                    scale, out, lse, ws, layout, S, stream)
        return hand_over(out, lse)


def _new_tokens(k_new, v_new, B, Hkv, D):
    """n_new and the element strides of k_new / v_new [B, n_new, Hkv, D] (any
    strides that are multiples of 8, head dim contiguous)."""
    if k_new.dim() != 4 or v_new.shape != k_new.shape or k_new.shape[0] != B or k_new.shape[2:] != (Hkv, D):
        raise ValueError("k_new, v_new must be [B, n_new, Hkv, D]")
    for t, name in ((k_new, "k_new"), (v_new, "v_new")):
        if t.dtype != torch.bfloat16 or not t.is_cuda or t.stride(3) != 1:
            raise ValueError(f"{name} must be a bf16 CUDA tensor with a contiguous head dimension")
    # the stride of a dimension of length 1 says nothing
    strides = [[0 if t.shape[d] == 1 else t.stride(d) for d in range(3)] for t in (k_new, v_new)]
    if strides[0] != strides[1]:
        raise ValueError("k_new and v_new must have the same strides")
    return k_new.shape[1], strides[0]


def _append_lens(new_lens, seqlens, B):
    _tensor(seqlens, "seqlens", (B,), torch.int32)
    if new_lens is None:
        return None
    _tensor(new_lens, "new_lens", (B,), torch.int32)
    return new_lens.data_ptr()


def prepare_quant_append(k_new, v_new, k_codes, v_codes, k_scale, v_scale, kv_type, block_tokens, seqlens, new_lens=None,
                         stream=None):
    """Check and marshal once; return a no-argument callable that enqueues
    fd_quant_append with those pointers: bf16 tokens k_new, v_new
    [B, n_new, Hkv, D] (a view with any strides that are multiples of 8, e.g.
    a transposed [B, Hkv, n_new, D] cache) into a block-scaled cache (see
    prepare_decode_quant_block). seqlens counts the new tokens; new_lens
    [B] int32 gives how many of the n_new each sequence has (None: all)."""
    B, Hkv, Lmax, D = _block_codes(k_codes, v_codes, k_scale, v_scale, kv_type, block_tokens)
    n_new, (sb, st, sh) = _new_tokens(k_new, v_new, B, Hkv, D)
    lens = _append_lens(new_lens, seqlens, B)
    tensors = (k_new, v_new, k_codes, v_codes, k_scale, v_scale, seqlens, new_lens)
    return _prepared("fd_quant_append", tensors, (
        B, n_new, Hkv, D, Lmax, block_tokens, KV_CODES[kv_type], k_new.data_ptr(), v_new.data_ptr(), sb, st, sh, lens,
        seqlens.data_ptr(), k_codes.data_ptr(), v_codes.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
        _stream(stream, k_new.device)))


def fd_quant_append(k_new, v_new, k_codes, v_codes, k_scale, v_scale, kv_type, block_tokens, seqlens, new_lens=None,
                    stream=None):
    """prepare_quant_append, enqueued once."""
    prepare_quant_append(k_new, v_new, k_codes, v_codes, k_scale, v_scale, kv_type, block_tokens, seqlens, new_lens,
                         stream)()


def prepare_quant_append_paged(k_new, v_new, k_pages, v_pages, k_scale, v_scale, kv_type, block_tokens, block_table,
                               seqlens, new_lens=None, layout="HND", stream=None):
    """prepare_quant_append into page pools (see
    prepare_decode_quant_block_paged)."""
    Hkv, D, page_size, num_pages, max_pages = _block_pages(k_pages, v_pages, k_scale, v_scale, kv_type, block_tokens,
                                                           block_table, layout)
    B = block_table.shape[0]
    n_new, (sb, st, sh) = _new_tokens(k_new, v_new, B, Hkv, D)
    lens = _append_lens(new_lens, seqlens, B)
    tensors = (k_new, v_new, k_pages, v_pages, k_scale, v_scale, block_table, seqlens, new_lens)
    return _prepared("fd_quant_append_paged", tensors, (
        B, n_new, Hkv, D, page_size, num_pages, max_pages, LAYOUTS[layout], block_tokens, KV_CODES[kv_type],
        k_new.data_ptr(), v_new.data_ptr(), sb, st, sh, lens, block_table.data_ptr(), seqlens.data_ptr(),
        k_pages.data_ptr(), v_pages.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), _stream(stream, k_new.device)))


def fd_quant_append_paged(k_new, v_new, k_pages, v_pages, k_scale, v_scale, kv_type, block_tokens, block_table, seqlens,
                          new_lens=None, layout="HND", stream=None):
    """prepare_quant_append_paged, enqueued once."""
    prepare_quant_append_paged(k_new, v_new, k_pages, v_pages, k_scale, v_scale, kv_type, block_tokens, block_table,
                               seqlens, new_lens, layout, stream)()


def empty_quant_block_cache(B, Hkv, max_len, D, block_tokens, device="cuda"):
    """Codes and scales of an empty contiguous block-scaled cache, zeroed:
    k_codes, v_codes, k_scale, v_scale, for fd_quant_append to fill."""
    if block_tokens not in FD_BLOCK_TOKENS:
        raise ValueError(f"block_tokens must be one of {FD_BLOCK_TOKENS}")
    blocks = -(-max_len // block_tokens)
    codes = [torch.zeros((B, Hkv, max_len, D), dtype=torch.uint8, device=device) for _ in range(2)]
    scales = [torch.zeros((B, Hkv, blocks), dtype=torch.float32, device=device) for _ in range(2)]
    return codes[0], codes[1], scales[0], scales[1]


def fd_weights_workspace_bytes(B: int, q_len: int, Hq: int, Hkv: int, D: int, max_len: int, num_splits: int) -> int:
    return int(lib().fd_weights_workspace_bytes(B, q_len, Hq, Hkv, D, max_len, num_splits))


def prepare_decode_weights(q, k_cache, v_cache, seqlens, scale, out, lse, weights_in, weights_out, workspace,
                           num_splits=None, stream=None):
    """Check and marshal once; return a no-argument callable that enqueues
    fd_decode_weights with those pointers: decode attention (q [B, Hq, D] or
    [B, q_len, Hq, D]) that also writes weights_out [B, Hkv, Lmax] =
    weights_in (None: zeros; may be weights_out) + each cached token's
    attention weight. workspace: fd_weights_workspace_bytes, zeroed once."""
    B, q_len, Hq, D = _query(q)
    _, _, Hkv, _, Lmax = _shapes(q.view(B, q_len * Hq, D), k_cache, v_cache)
    _block_outputs(q, out, lse)
    _tensor(seqlens, "seqlens", (B,), torch.int32)
    for t, name in ((weights_in, "weights_in"), (weights_out, "weights_out")):
        if t is not None or name == "weights_out":
            _tensor(t, name, (B, Hkv, Lmax), torch.float32)
    wp, wb = _ws(workspace)
    tensors = (q, k_cache, v_cache, seqlens, out, lse, weights_in, weights_out, workspace)
    S = _planned(q.device.index, B, Hq, Hkv, D, Lmax, num_splits)
    call = _prepared("fd_decode_weights", tensors, (
        B, q_len, Hq, Hkv, D, Lmax, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), seqlens.data_ptr(),
        float(scale), out.data_ptr(), lse.data_ptr(), None if weights_in is None else weights_in.data_ptr(),
        weights_out.data_ptr(), wp, wb, S, _stream(stream, q.device)))
    call.num_splits = S
    return call


def fd_decode_weights(q, k_cache, v_cache, seqlens, scale, out, lse, weights_in, weights_out, workspace, num_splits=0,
                      stream=None):
    """prepare_decode_weights, enqueued once; num_splits 0 lets the library
    plan the split count."""
    prepare_decode_weights(q, k_cache, v_cache, seqlens, scale, out, lse, weights_in, weights_out, workspace, num_splits,
                           stream)()


def decode_weights(q, k_cache, v_cache, seqlens, scale, weights=None, num_splits=None, stream=None):
    """Allocate out / lse / workspace with torch and run fd_decode_weights.
    `weights` [B, Hkv, Lmax] is updated in place (None: a new one, from zeros).
    Returns (out, lse, weights)."""
    B, q_len, Hq, D = _query(q)
    _, _, Hkv, _, Lmax = _shapes(q.view(B, q_len * Hq, D), k_cache, v_cache)
    S = _planned(q.device.index, B, Hq, Hkv, D, Lmax, num_splits)
    nbytes = fd_weights_workspace_bytes(B, q_len, Hq, Hkv, D, Lmax, S)
    with _on_stream(stream, q.device) as hand_over:
        ws = torch.zeros(nbytes, dtype=torch.uint8, device=q.device) if nbytes else None
        out = torch.empty(q.shape, dtype=torch.float32, device=q.device)
        lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device)
        if weights is None:
            weights = torch.zeros((B, Hkv, Lmax), dtype=torch.float32, device=q.device)
        fd_decode_weights(q, k_cache, v_cache, seqlens, scale, out, lse, weights, weights, ws, S, stream)
        return hand_over(out, lse, weights)


def prepare_evict(k_cache, v_cache, weights, seqlens, keep, recent, k_out, v_out, weights_out, kept, seqlens_out,
                  stream=None):
    """Check and marshal once; return a no-argument callable that enqueues
    fd_evict with those pointers: caches [B, Hkv, Lmax, D] bf16 and totals
    `weights` [B, Hkv, Lmax] cut to `keep` tokens per (sequence, kv head), the
    last `recent` and the heaviest others, into k_out, v_out
    [B, Hkv, out_len, D], weights_out [B, Hkv, out_len], kept [B, Hkv, keep]
    int32 and seqlens_out [B] int32."""
    if k_cache.dim() != 4 or k_out.dim() != 4:
        raise ValueError("k_cache and k_out must be [B, Hkv, length, D]")
    B, Hkv, Lmax, D = k_cache.shape
    out_len = k_out.shape[2]
    for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _tensor(t, name, k_cache.shape, torch.bfloat16)
    for t, name in ((k_out, "k_out"), (v_out, "v_out")):
        _tensor(t, name, (B, Hkv, out_len, D), torch.bfloat16)
    _tensor(weights, "weights", (B, Hkv, Lmax), torch.float32)
    _tensor(weights_out, "weights_out", (B, Hkv, out_len), torch.float32)
    _tensor(kept, "kept", (B, Hkv, keep), torch.int32)
    for t, name in ((seqlens, "seqlens"), (seqlens_out, "seqlens_out")):
        _tensor(t, name, (B,), torch.int32)
    tensors = (k_cache, v_cache, weights, seqlens, k_out, v_out, weights_out, kept, seqlens_out)
    return _prepared("fd_evict", tensors, (
        B, Hkv, D, Lmax, keep, recent, out_len, k_cache.data_ptr(), v_cache.data_ptr(), weights.data_ptr(),
        seqlens.data_ptr(), k_out.data_ptr(), v_out.data_ptr(), weights_out.data_ptr(), kept.data_ptr(),
        seqlens_out.data_ptr(), _stream(stream, k_cache.device)))


def fd_evict(k_cache, v_cache, weights, seqlens, keep, recent, k_out, v_out, weights_out, kept, seqlens_out,
             stream=None):
    """prepare_evict, enqueued once."""
    prepare_evict(k_cache, v_cache, weights, seqlens, keep, recent, k_out, v_out, weights_out, kept, seqlens_out,
                  stream)()


def evict(k_cache, v_cache, weights, seqlens, keep, recent=0, out_len=None, stream=None):
    """Allocate the outputs with torch and run fd_evict; out_len (default
    keep) tokens are allocated per row, so a decode loop can append to the cut
    cache. Returns (k_out, v_out, weights_out, kept, seqlens_out)."""
    B, Hkv, _, D = k_cache.shape
    n = keep if out_len is None else int(out_len)
    dev = k_cache.device
    with _on_stream(stream, dev) as hand_over:
        k_out = torch.zeros((B, Hkv, n, D), dtype=torch.bfloat16, device=dev)
        v_out = torch.zeros_like(k_out)
        w_out = torch.empty((B, Hkv, n), dtype=torch.float32, device=dev)
        kept = torch.empty((B, Hkv, keep), dtype=torch.int32, device=dev)
        lens = torch.empty((B,), dtype=torch.int32, device=dev)
        fd_evict(k_cache, v_cache, weights, seqlens, keep, recent, k_out, v_out, w_out, kept, lens, stream)
        return hand_over(k_out, v_out, w_out, kept, lens)
