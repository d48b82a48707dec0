"""ctypes binding of libfattn (argument marshalling only).

The functions named like the C entry points (``fattn_fwd``, ``fattn_bwd``, ...)
take torch tensors (or raw integer device addresses) and pass their pointers,
sizes and the current CUDA stream straight to the library; every step of the
computation runs in the library's kernels.  ``forward`` and ``backward``
allocate the outputs with torch and then call those entry points.

The library is loaded on first use.  If ``libfattn.so`` is missing the
binding raises: there is no fallback path.
"""
import contextlib
import ctypes
import os
import struct
import threading
import typing

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfattn.so")

FATTN_OK = 0
STATUS_NAMES = {0: "FATTN_OK", 1: "FATTN_ERR_INVALID_ARG", 2: "FATTN_ERR_UNSUPPORTED",
                3: "FATTN_ERR_CUDA", 4: "FATTN_ERR_WORKSPACE", 5: "FATTN_ERR_TIMEOUT"}

# Every exported symbol of include/fattn.h: name -> (restype, argtypes)
_vp, _i, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_ll = ctypes.c_longlong


# fattn_cache and fattn_cache_batch, packed; a bytes object is passed by its address
_pack_cache = struct.Struct("@4P5i").pack
_pack_batch = struct.Struct("@3P4i").pack
_cp = _bp = ctypes.c_char_p

SIGNATURES = {
    "fattn_fwd": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _vp]),
    "fattn_fwd_ex": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _vp, _vp]),
    "fattn_bwd_workspace_bytes": (_sz, [_i, _i, _i, _i]),
    "fattn_bwd": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _vp,
                       _sz, _vp]),
    "fattn_bwd_ex": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i,
                          _vp, _sz, _vp, _vp]),
    "fattn_bwd_noalloc": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f,
                               _i, _vp]),
    "fattn_tile_sizes": (_i, [_i, _i, ctypes.POINTER(_i), ctypes.POINTER(_i)]),
    "fattn_device_error": (_i, [ctypes.POINTER(ctypes.c_uint), _i]),
    "fattn_softmax_rows": (_i, [_vp, _vp, _vp, ctypes.c_longlong, _i, _vp]),
    "fattn_decode": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _i, _i, _vp, _sz, _vp]),
    "fattn_decode_splits": (_i, [_i, _i, _i, _i, _i, _i]),
    "fattn_decode_workspace_bytes": (_sz, [_i, _i, _i, _i, _i, _i]),
    "fattn_merge_partials": (_i, [_vp, _vp, _i, ctypes.c_longlong, _i, _vp, _vp, _vp]),
    "fattn_fwd_varlen": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _i, _vp]),
    "fattn_bwd_varlen": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i,
                              _i, _f, _i, _vp, _sz, _vp]),
    "fattn_fwd_bwd_host_workspace_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "fattn_fwd_bwd_host": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f,
                                _i, _i, _vp, _sz, _vp]),
    "fattn_cache_append": (_i, [_cp, _bp, _vp, _ll, _ll, _vp, _ll, _ll, _vp]),
    "fattn_cache_read": (_i, [_cp, _bp, _vp, _ll, _ll, _vp, _ll, _ll, _vp]),
    "fattn_cache_fwd": (_i, [_cp, _bp, _vp, _ll, _ll, _vp, _ll, _ll, _vp, _i, _f, _i, _vp, _sz,
                             _vp]),
    "fattn_cache_fwd_workspace_bytes": (_sz, [_cp, _bp, _i]),
    "fattn_cache_weights": (_i, [_cp, _bp, _vp, _ll, _ll, _vp, _i, _f, _i, _vp, _ll, _ll, _vp, _ll,
                                 _ll, _i, _vp]),
    "fattn_cache_evict": (_i, [_cp, _bp, _vp, _ll, _ll, _i, _vp, _i, _i, _i, _vp, _vp, _vp, _ll, _ll,
                               _i, _vp]),
    "fattn_rope_turns": (_i, [_vp, ctypes.POINTER(_f), _i, ctypes.c_double, _i, ctypes.c_double, _i,
                              ctypes.c_double, ctypes.c_double]),
    "fattn_rope": (_i, [_vp, _ll, _ll, _vp, _ll, _ll, _i, _vp, _ll, _ll, _vp, _ll, _ll, _i, _vp, _vp,
                        _f, _i, _i, _i, _i, _i, _vp]),
    "fattn_status_string": (ctypes.c_char_p, [_i]),
}

# The test and measurement hooks of include/fattn_testing.h (exported by the
# same library, not part of the attention interface).
TESTING_SIGNATURES = {
    "fattn_check_wait_timeout": (_i, [_vp]),
    "fattn_ex2_throughput": (_i, [ctypes.POINTER(ctypes.c_double), _vp]),
}

_lock = threading.Lock()
_lib = None


def _raw_stream(dev):
    """The handle of device `dev`'s current stream."""
    return torch.cuda.current_stream(dev).cuda_stream


# the same without the Stream object, which costs as much as a short launch
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)


class FattnError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__("%s returned %s (%d)" % (fn, STATUS_NAMES.get(status, "?"), status))


def load(path=None):
    """Load libfattn.so (once) and declare the C signatures."""
    global _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError("libfattn.so not found at %s: build it with "
                               "`python -c 'import __graft_entry__ as g; g.build()'`" % p)
        lib = ctypes.CDLL(p)
        for name, (res, args) in list(SIGNATURES.items()) + list(TESTING_SIGNATURES.items()):
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        if path is None:
            _lib = lib
        return lib


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(name, status):
    if status != FATTN_OK:
        raise FattnError(name, status)


# ------------------------------------------------------------------ entry points

def fattn_fwd(q, k, v, o, lse, B, H, N, d, scale, causal, stream=None):
    _check("fattn_fwd", load().fattn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, d,
                                         float(scale), int(bool(causal)), _stream(stream)))


def fattn_fwd_ex(q, k, v, o, lse, B, H, N, d, scale, causal, tile_counts, stream=None):
    _check("fattn_fwd_ex", load().fattn_fwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H,
                                               N, d, float(scale), int(bool(causal)),
                                               _ptr(tile_counts), _stream(stream)))


def fattn_bwd_workspace_bytes(B, H, N, d):
    return int(load().fattn_bwd_workspace_bytes(B, H, N, d))


def fattn_bwd(q, k, v, o, lse, do, dq, dk, dv, B, H, N, d, scale, causal, workspace,
              workspace_bytes, stream=None):
    _check("fattn_bwd", load().fattn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do),
                                         _ptr(dq), _ptr(dk), _ptr(dv), B, H, N, d, float(scale),
                                         int(bool(causal)), _ptr(workspace), int(workspace_bytes),
                                         _stream(stream)))


def fattn_bwd_ex(q, k, v, o, lse, do, dq, dk, dv, B, H, N, d, scale, causal, workspace,
                 workspace_bytes, phase_events, stream=None):
    """phase_events: None or 4 torch.cuda.Event(enable_timing=True) objects."""
    arr = None
    if phase_events is not None:
        for ev in phase_events:
            if ev.cuda_event == 0:  # torch creates the handle on first record
                ev.record()
        arr = (ctypes.c_void_p * 4)(*[ev.cuda_event for ev in phase_events])
    _check("fattn_bwd_ex", load().fattn_bwd_ex(
        _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do), _ptr(dq), _ptr(dk), _ptr(dv), B, H,
        N, d, float(scale), int(bool(causal)), _ptr(workspace), int(workspace_bytes),
        ctypes.cast(arr, ctypes.c_void_p) if arr is not None else None, _stream(stream)))


def fattn_bwd_noalloc(q, k, v, o, lse, do, dq, dk, dv, B, H, N, d, scale, causal, stream=None):
    """fattn_bwd with the library's built-in workspace (allocates nothing)."""
    _check("fattn_bwd_noalloc", load().fattn_bwd_noalloc(
        _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do), _ptr(dq), _ptr(dk), _ptr(dv), B, H,
        N, d, float(scale), int(bool(causal)), _stream(stream)))


def fattn_fwd_varlen(q, k, v, o, lse, cu_seqlens, B, H, max_seqlen, total, d, scale, causal,
                     stream=None):
    _check("fattn_fwd_varlen", load().fattn_fwd_varlen(
        _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(cu_seqlens), B, H, int(max_seqlen),
        int(total), d, float(scale), int(bool(causal)), _stream(stream)))


def fattn_bwd_varlen(q, k, v, o, lse, do, dq, dk, dv, cu_seqlens, B, H, max_seqlen, total, d,
                     scale, causal, workspace, workspace_bytes, stream=None):
    _check("fattn_bwd_varlen", load().fattn_bwd_varlen(
        _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do), _ptr(dq), _ptr(dk), _ptr(dv),
        _ptr(cu_seqlens), B, H, int(max_seqlen), int(total), d, float(scale), int(bool(causal)),
        _ptr(workspace), int(workspace_bytes), _stream(stream)))


def fattn_fwd_bwd_host_workspace_bytes(B, H, N, d, heads_per_chunk=0):
    return int(load().fattn_fwd_bwd_host_workspace_bytes(B, H, N, d, int(heads_per_chunk)))


def fattn_fwd_bwd_host(q, k, v, do, o, lse, dq, dk, dv, B, H, N, d, scale, causal,
                       heads_per_chunk, workspace, workspace_bytes, stream=None):
    """q, k, v, do, o, lse, dq, dk, dv: HOST tensors (pinned for overlap) or addresses;
    workspace: a device tensor or address."""
    _check("fattn_fwd_bwd_host", load().fattn_fwd_bwd_host(
        _ptr(q), _ptr(k), _ptr(v), _ptr(do), _ptr(o), _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv), B, H,
        N, d, float(scale), int(bool(causal)), int(heads_per_chunk), _ptr(workspace),
        int(workspace_bytes), _stream(stream)))


def fattn_tile_sizes(d, pass_):
    bq, bk = ctypes.c_int(0), ctypes.c_int(0)
    _check("fattn_tile_sizes", load().fattn_tile_sizes(d, pass_, ctypes.byref(bq), ctypes.byref(bk)))
    return bq.value, bk.value


FATTN_ERR_TIMEOUT = 5


def fattn_device_error(clear=True):
    """The device error word (0: no in-kernel wait ran out); the C call returns
    FATTN_ERR_TIMEOUT while the word is set, which is a successful read here."""
    code = ctypes.c_uint(0)
    st = load().fattn_device_error(ctypes.byref(code), int(bool(clear)))
    if st not in (FATTN_OK, FATTN_ERR_TIMEOUT):
        raise FattnError("fattn_device_error", st)
    return code.value


def check_wait_timeout(stream=None):
    """Launch the library's failure-path check (a bounded wait that must give up
    after about 1 ms) on the current stream; read the outcome with
    fattn_device_error()."""
    import torch
    s = stream if stream is not None else torch.cuda.current_stream().cuda_stream
    _check("fattn_check_wait_timeout", load().fattn_check_wait_timeout(s))


def ex2_throughput(stream=None):
    """Measured ex2 evaluations per second of the current device (synchronises)."""
    rate = ctypes.c_double(0.0)
    _check("fattn_ex2_throughput", load().fattn_ex2_throughput(ctypes.byref(rate), _stream(stream)))
    return rate.value


def fattn_status_string(status):
    return load().fattn_status_string(int(status)).decode()


# ------------------------------------------------------------------ allocating wrappers

def _shape(q):
    if q.dim() != 4:
        raise ValueError("expected [B, H, N, d] tensors")
    return tuple(q.shape)


def forward(q, k, v, scale, causal, tile_counts=None, stream=None):
    """O, LSE of bf16 [B,H,N,d] device tensors q, k, v (contiguous)."""
    B, H, N, d = _shape(q)
    o = torch.empty_like(q)
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    if tile_counts is None:
        fattn_fwd(q, k, v, o, lse, B, H, N, d, scale, causal, stream)
    else:
        fattn_fwd_ex(q, k, v, o, lse, B, H, N, d, scale, causal, tile_counts, stream)
    return o, lse


def backward(q, k, v, o, lse, do, scale, causal, workspace=None, stream=None):
    """dQ, dK, dV for dL/dO = do.  workspace: None (a torch allocation), a
    device tensor, or "stream" (the library's stream-ordered scratch: the C
    call gets a NULL workspace)."""
    B, H, N, d = _shape(q)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    if isinstance(workspace, str):
        if workspace != "stream":
            raise ValueError(workspace)
        fattn_bwd(q, k, v, o, lse, do, dq, dk, dv, B, H, N, d, scale, causal, None, 0, stream)
        return dq, dk, dv
    nbytes = fattn_bwd_workspace_bytes(B, H, N, d)
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    fattn_bwd(q, k, v, o, lse, do, dq, dk, dv, B, H, N, d, scale, causal, workspace,
              workspace.numel() * workspace.element_size(), stream)
    return dq, dk, dv


def forward_backward_host(q, k, v, do, scale, causal, heads_per_chunk=0, workspace=None,
                          device=None, stream=None):
    """Forward and backward of HOST bf16 tensors [B,H,N,d] through the device:
    returns HOST (o, lse, dq, dk, dv), page-locked.  The call is asynchronous on
    the stream; synchronise before reading the results."""
    B, H, N, d = _shape(q)
    device = torch.device("cuda") if device is None else torch.device(device)
    with torch.cuda.device(device):
        if stream is None:
            stream = torch.cuda.current_stream(device)
        nbytes = fattn_fwd_bwd_host_workspace_bytes(B, H, N, d, heads_per_chunk)
        own = workspace is None
        if own:
            workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)
        o, dq, dk, dv = (torch.empty(q.shape, dtype=torch.bfloat16).pin_memory() for _ in range(4))
        lse = torch.empty((B, H, N), dtype=torch.float32).pin_memory()
        fattn_fwd_bwd_host(q, k, v, do, o, lse, dq, dk, dv, B, H, N, d, scale, causal,
                           heads_per_chunk, workspace, workspace.numel() * workspace.element_size(),
                           stream)
        if own and isinstance(stream, torch.cuda.Stream):
            # the workspace is in use until `stream` passes the call: keep the
            # allocator from handing it out before then
            workspace.record_stream(stream)
    return o, lse, dq, dk, dv


def forward_varlen(q, k, v, cu_seqlens, max_seqlen, scale, causal, stream=None):
    """O, LSE of packed bf16 [H, total, d] device tensors; cu_seqlens is a device
    int32 tensor of B + 1 offsets (its last entry, total, is q.shape[1])."""
    H, T, d = q.shape
    B = cu_seqlens.numel() - 1
    o = torch.empty_like(q)
    lse = torch.empty((H, T), dtype=torch.float32, device=q.device)
    fattn_fwd_varlen(q, k, v, o, lse, cu_seqlens, B, H, max_seqlen, T, d, scale, causal, stream)
    return o, lse


def backward_varlen(q, k, v, o, lse, do, cu_seqlens, max_seqlen, scale, causal, workspace=None,
                    stream=None):
    """dQ, dK, dV of forward_varlen for dL/dO = do."""
    H, T, d = q.shape
    B = cu_seqlens.numel() - 1
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    if workspace is None:
        workspace = torch.empty(max(fattn_bwd_workspace_bytes(1, H, max(T, 1), d), 1),
                                dtype=torch.uint8, device=q.device)
    fattn_bwd_varlen(q, k, v, o, lse, do, dq, dk, dv, cu_seqlens, B, H, max_seqlen, T, d, scale,
                     causal, workspace, workspace.numel() * workspace.element_size(), stream)
    return dq, dk, dv


def decode(q, k, v, scale, causal, n_splits=0, workspace=None, stream=None):
    """O, LSE of few queries q [B,H,Nq,d] against k, v [B,H,Nkv,d] (the queries
    are the last Nq positions) by split-KV plus merge."""
    B, H, Nq, d = _shape(q)
    Nkv = k.shape[2]
    lib = load()
    o = torch.empty_like(q)
    lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    nbytes = int(lib.fattn_decode_workspace_bytes(B, H, Nq, Nkv, d, n_splits))
    if workspace is None:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=q.device)
    _check("fattn_decode", lib.fattn_decode(
        _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Nq, Nkv, d, float(scale),
        int(bool(causal)), int(n_splits), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))
    return o, lse


def merge_partials(o_part, lse_part, stream=None):
    """Merge fp32 partials o_part [S, rows, d], lse_part [S, rows] -> bf16 o [rows, d], lse."""
    S, rows, d = o_part.shape
    o = torch.empty((rows, d), dtype=torch.bfloat16, device=o_part.device)
    lse = torch.empty((rows,), dtype=torch.float32, device=o_part.device)
    _check("fattn_merge_partials", load().fattn_merge_partials(
        _ptr(o_part), _ptr(lse_part), S, rows, d, _ptr(o), _ptr(lse), _stream(stream)))
    return o, lse


def softmax_rows(x, with_lse=False, out=None, stream=None):
    """Row-wise softmax of a contiguous fp32 [rows, cols] device tensor."""
    rows, cols = x.shape
    y = torch.empty_like(x) if out is None else out
    lse = torch.empty((rows,), dtype=torch.float32, device=x.device) if with_lse else None
    _check("fattn_softmax_rows", load().fattn_softmax_rows(_ptr(x), _ptr(y), _ptr(lse), rows, cols,
                                                           _stream(stream)))
    return (y, lse) if with_lse else y


# ------------------------------------------------------------------ 8-bit and 4-bit key/value cache

CACHE_FORMATS = {torch.float8_e4m3fn: 0, torch.float8_e5m2: 1, torch.uint8: 4}


class KVCache(typing.NamedTuple):
    """The pool of blocks of fattn_cache, all contiguous on one device.  8 bits: k, v
    float8_e4m3fn or float8_e5m2 [num_blocks, H, block_size, d], k_scale, v_scale fp32
    [num_blocks, H].  4 bits: k, v uint8 [num_blocks, H, block_size, d / 2], two codes a
    byte, k_scale, v_scale float8_e5m2 [num_blocks, H, block_size, d / 16]."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor


class CacheBatch(typing.NamedTuple):
    """The tokens a cache call works on (fattn_cache_batch): the last
    cu_seqlens[b+1] - cu_seqlens[b] tokens of each sequence, packed into `total`
    rows; lens[b] is a sequence's length including them, block_table [B, width]
    names its blocks.  Contiguous device int32 tensors; max_seqlen is an upper
    bound of the tokens of one sequence."""
    block_table: torch.Tensor
    lens: torch.Tensor
    cu_seqlens: torch.Tensor
    total: int
    max_seqlen: int


def new_cache(num_blocks, heads, block_size, d, dtype=torch.float8_e4m3fn, device="cuda"):
    """An empty KVCache, as fattn_cache_append leaves it for zeros.  dtype: float8_e4m3fn
    or float8_e5m2 (codes zero, scales 2^-100), or uint8 for 4 bits (codes 8, scales 0)."""
    if dtype not in CACHE_FORMATS:
        raise ValueError("a cache holds float8_e4m3fn, float8_e5m2 or uint8 (4 bits), not %s" % dtype)
    shape = (num_blocks, heads, block_size, d)
    if dtype is torch.uint8:
        if d % 16:
            raise ValueError("a 4-bit cache has a scale for every 16 channels, not d = %d" % d)
        k, v = (torch.full(shape[:3] + (d // 2,), 0x88, dtype=dtype, device=device)
                for _ in range(2))
        ks, vs = (torch.zeros(shape[:3] + (d // 16,), dtype=dtype, device=device)
                  .view(torch.float8_e5m2) for _ in range(2))
        return KVCache(k, v, ks, vs)
    k, v = (torch.zeros(shape, dtype=torch.uint8, device=device).view(dtype) for _ in range(2))
    ks, vs = (torch.full(shape[:2], 2.0 ** -100, dtype=torch.float32, device=device)
              for _ in range(2))
    return KVCache(k, v, ks, vs)


def _refuse_cache(cache, batch):
    """Say what _cache_args found wrong."""
    k, v, ks, vs = cache
    if k.dtype is torch.uint8 and k.dim() == 4:
        scales = k.shape[:3] + (k.shape[3] // 8,)
        if v.dtype is not k.dtype or ks.dtype is not torch.float8_e5m2 or vs.dtype is not ks.dtype:
            raise ValueError("expected uint8 codes (two a byte) and float8_e5m2 scales")
        if k.shape[3] % 8 or v.shape != k.shape or ks.shape != scales or vs.shape != scales:
            raise ValueError("expected k, v [num_blocks, H, block_size, d / 2] and scales "
                             "[num_blocks, H, block_size, d / 16]")
    elif k.dim() != 4 or v.shape != k.shape or ks.shape != k.shape[:2] or vs.shape != k.shape[:2]:
        raise ValueError("expected k, v [num_blocks, H, block_size, d] and scales [num_blocks, H]")
    if k.dtype is not torch.uint8 and (
            k.dtype not in CACHE_FORMATS or v.dtype != k.dtype or ks.dtype != torch.float32
            or vs.dtype != torch.float32):
        raise ValueError("expected float8 codes of one type and fp32 scales")
    if batch is None:
        raise ValueError("expected contiguous tensors on one CUDA device")
    table, lens, cu = batch[:3]
    if table.dim() != 2 or lens.shape != (table.shape[0],) or cu.shape != (table.shape[0] + 1,):
        raise ValueError("expected block_table [B, width], lens [B], cu_seqlens [B + 1]")
    if table.dtype != torch.int32 or lens.dtype != torch.int32 or cu.dtype != torch.int32:
        raise ValueError("expected int32 block_table, lens and cu_seqlens")
    raise ValueError("expected contiguous tensors on one CUDA device")


def _pool_args(cache, batch=None):
    """The C descriptor of a cache, its tensors checked, with the device index, H and d."""
    k, v, ks, vs = cache
    shape, dtype, dev = k.shape, k.dtype, k.get_device()
    fmt = CACHE_FORMATS.get(dtype)
    if len(shape) != 4 or fmt is None or dev < 0:
        _refuse_cache(cache, batch)
    if fmt == 4:
        scales, kind = shape[:3] + (shape[3] // 8,), torch.float8_e5m2
    else:
        scales, kind = shape[:2], torch.float32
    if not (v.shape == shape and ks.shape == scales and vs.shape == scales
            and v.dtype is dtype and ks.dtype is kind and vs.dtype is kind
            and k.is_contiguous() and v.is_contiguous() and ks.is_contiguous()
            and vs.is_contiguous()
            and v.get_device() == dev and ks.get_device() == dev and vs.get_device() == dev):
        _refuse_cache(cache, batch)
    nb, H, bs, d = shape
    if fmt == 4:
        d *= 2
    return (_pack_cache(k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), nb, H, bs, d, fmt),
            dev, H, d)


def _cache_args(cache, batch):
    """The C descriptors of a cache and a batch, their tensors checked, with the
    device index, H and d.  (A decoding step's calls are as short as the launches
    they make, so the checks take few attribute reads.)"""
    c, dev, H, d = _pool_args(cache, batch)
    table, lens, cu, total, max_seqlen = batch
    if table.dim() != 2:
        _refuse_cache(cache, batch)
    B, width = table.shape
    i32 = torch.int32
    if not (lens.dim() == 1 and lens.numel() == B and cu.dim() == 1 and cu.numel() == B + 1
            and table.dtype is i32 and lens.dtype is i32 and cu.dtype is i32
            and table.is_contiguous() and lens.is_contiguous() and cu.is_contiguous()
            and table.get_device() == dev and lens.get_device() == dev and cu.get_device() == dev):
        _refuse_cache(cache, batch)
    return (c, _pack_batch(table.data_ptr(), lens.data_ptr(), cu.data_ptr(), B, width, total,
                           max_seqlen), dev, H, d)


def _packed(x, total, heads, d, dev):
    """Pointer and token and head strides of a bf16 [total, heads, d] tensor."""
    st = x.stride()
    if len(st) != 3 or x.shape != (total, heads, d) or x.dtype is not torch.bfloat16 or \
            x.get_device() != dev or st[2] != 1:
        raise ValueError("expected a bf16 [%d, %d, %d] tensor on device %d with a contiguous last "
                         "axis" % (total, heads, d, dev))
    return x.data_ptr(), st[0], st[1]


@contextlib.contextmanager
def _on(dev, stream):
    """Work and allocations on `stream` of device `dev` (None: its current stream)."""
    with torch.cuda.device(dev):
        if stream is None:
            yield
            return
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=dev)
        with torch.cuda.stream(stream):
            yield


def _elsewhere(dev, stream):
    """Whether a call has to change the current device or stream first."""
    return stream is not None or torch.cuda.current_device() != dev


def cache_append(k, v, cache, batch, stream=None):
    """Quantise new tokens' k, v (bf16 [total, H, d], any token and head strides)
    into the cache."""
    c, b, dev, H, d = _cache_args(cache, batch)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return cache_append(k, v, cache, batch)
    total = batch[3]
    kp, kt, kh = _packed(k, total, H, d, dev)
    vp, vt, vh = _packed(v, total, H, d, dev)
    st = (_lib or load()).fattn_cache_append(c, b, kp, kt, kh, vp, vt, vh, _raw_stream(dev))
    if st:
        raise FattnError("fattn_cache_append", st)


def cache_read(cache, batch, out=None, stream=None):
    """k, v (bf16 [total, H, d]) of the batch's tokens, read back from the cache;
    out: a pair of tensors to write to."""
    c, b, dev, H, d = _cache_args(cache, batch)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return cache_read(cache, batch, out)
    total = batch[3]
    if out is None:
        shape = (total, H, d)
        k = torch.empty(shape, dtype=torch.bfloat16, device=cache[0].device)
        v = torch.empty_like(k)
    else:
        k, v = out
    kp, kt, kh = _packed(k, total, H, d, dev)
    vp, vt, vh = _packed(v, total, H, d, dev)
    st = (_lib or load()).fattn_cache_read(c, b, kp, kt, kh, vp, vt, vh, _raw_stream(dev))
    if st:
        raise FattnError("fattn_cache_read", st)
    return k, v


_ws_bytes = {}  # fattn_cache_fwd_workspace_bytes by all of its arguments


def cache_forward(q, cache, batch, scale, causal, out=None, workspace=None, stream=None):
    """O (bf16 [total, Hq, d]) and LSE (fp32 [Hq, total]) of the batch's queries q
    (bf16 [total, Hq, d], any token and head strides) over their sequences in the
    cache.  out: a tensor to write O to.  workspace: None (a torch allocation) or a
    device tensor."""
    c, b, dev, H, d = _cache_args(cache, batch)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return cache_forward(q, cache, batch, scale, causal, out, workspace)
    if q.dim() != 3:
        raise ValueError("expected q [total, Hq, d]")
    total, Hq = batch[3], q.shape[1]
    qp, qt, qh = _packed(q, total, Hq, d, dev)
    lib = _lib or load()
    on = q.device
    o = torch.empty((total, Hq, d), dtype=torch.bfloat16, device=on) if out is None else out
    lse = torch.empty((Hq, total), dtype=torch.float32, device=on)
    if workspace is None:
        key = (dev, cache[0].shape, cache[0].dtype, batch[0].shape, total, batch[4], Hq)
        nbytes = _ws_bytes.get(key)
        if nbytes is None:
            nbytes = int(lib.fattn_cache_fwd_workspace_bytes(c, b, Hq))
            if len(_ws_bytes) > 4096:
                _ws_bytes.clear()
            if nbytes:  # (0: a failure, which the call below reports)
                _ws_bytes[key] = nbytes
        workspace = torch.empty((max(nbytes, 256),), dtype=torch.uint8, device=on)
    else:
        if workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError("expected a contiguous workspace on device %d" % dev)
        nbytes = workspace.numel() * workspace.element_size()
    op, ot, oh = _packed(o, total, Hq, d, dev)
    st = lib.fattn_cache_fwd(c, b, qp, qt, qh, op, ot, oh, lse.data_ptr(), Hq, scale,
                             1 if causal else 0, workspace.data_ptr(), nbytes, _raw_stream(dev))
    if st:
        raise FattnError("fattn_cache_fwd", st)
    return o, lse


# ------------------------------------------------------------------ weights of cached keys, eviction

def _weights_of(w, B, H, dev):
    """Pointer, sequence and head strides and width of fp32 weights [B, H, width]."""
    st = w.stride()
    if len(st) != 3 or w.shape[:2] != (B, H) or w.dtype is not torch.float32 or \
            w.get_device() != dev or (st[2] != 1 and w.shape[2] > 1):
        raise ValueError("expected fp32 weights [%d, %d, width] on device %d with a contiguous last "
                         "axis" % (B, H, dev))
    return w.data_ptr(), st[0], st[1], w.shape[2]


def cache_weights(q, lse, cache, batch, scale, causal, weights=None, out=None, stream=None):
    """The attention weight that every key of the batch's sequences gets from its queries q
    (bf16 [total, Hq, d]), whose log-sum-exp lse (fp32 [Hq, total]) cache_forward gave: fp32
    [B, H, width], summed over the queries and the heads of a group.  weights: what the keys
    had before, which is added to (None: nothing); the batch's own tokens start anew.  out: a
    tensor to write to (None: `weights`, in place, or a new one with room for the table).
    Entries behind a sequence's length stay as they are (new: zero), and so do all of a sequence
    without queries: in an `out` apart from `weights`, that is what `out` had, not its weights.
    The rows need room for a sequence's whole length: one that is longer than `width` is left out,
    which only the device error word tells (0x470)."""
    c, b, dev, H, d = _cache_args(cache, batch)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return cache_weights(q, lse, cache, batch, scale, causal, weights, out)
    if q.dim() != 3:
        raise ValueError("expected q [total, Hq, d]")
    total, Hq = batch[3], q.shape[1]
    qp, qt, qh = _packed(q, total, Hq, d, dev)
    if lse.shape != (Hq, total) or lse.dtype is not torch.float32 or not lse.is_contiguous() or \
            lse.get_device() != dev:
        raise ValueError("expected contiguous fp32 lse [%d, %d] on device %d" % (Hq, total, dev))
    B, width = batch[0].shape
    if out is None:
        out = weights if weights is not None else torch.zeros(
            (B, H, width * cache[0].shape[2]), dtype=torch.float32, device=q.device)
    op, ob, oh, width = _weights_of(out, B, H, dev)
    if weights is None:
        wp, wb, wh = None, 0, 0
    else:
        wp, wb, wh, had = _weights_of(weights, B, H, dev)
        width = min(width, had)
    st = (_lib or load()).fattn_cache_weights(c, b, qp, qt, qh, lse.data_ptr(), Hq, scale,
                                              1 if causal else 0, wp, wb, wh, op, ob, oh, width,
                                              _raw_stream(dev))
    if st:
        raise FattnError("fattn_cache_weights", st)
    return out


def cache_evict(cache, weights, block_table, lens, table_out, keep, recent=0, out=None, stream=None):
    """Copies, for every sequence and key/value head, the last `recent` tokens and those of the
    largest weights (fp32 [B, H, width]), `keep` in all and in their order, into the blocks of
    table_out (int32 [B, width]); a sequence of at most `keep` tokens is copied whole.  Returns
    the new lengths (int32 [B]), the positions of the kept tokens (int32 [B, H, keep], -1 behind
    the last) and their weights (fp32 [B, H, keep], or `out`).  The source blocks stay as they
    are.  Weights that cache_weights is to go on with need rows with room for the tokens to come:
    an `out` that is wider than `keep`."""
    c, dev, H, d = _pool_args(cache)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return cache_evict(cache, weights, block_table, lens, table_out, keep, recent, out)
    i32 = torch.int32
    if block_table.dim() != 2 or table_out.dim() != 2 or lens.dim() != 1 or \
            not lens.shape[0] == block_table.shape[0] == table_out.shape[0]:
        raise ValueError("expected block_table and table_out [B, width], lens [B]")
    for x in (block_table, table_out, lens):
        if x.dtype is not i32 or not x.is_contiguous() or x.get_device() != dev:
            raise ValueError("expected contiguous int32 tables and lengths on device %d" % dev)
    if keep < 1:
        raise ValueError("expected keep >= 1")
    B, width = block_table.shape
    wp, wb, wh, w_width = _weights_of(weights, B, H, dev)
    on = weights.device
    if out is None:
        out = torch.zeros((B, H, keep), dtype=torch.float32, device=on)
    op, ob, oh, o_width = _weights_of(out, B, H, dev)
    lens_out = torch.empty((B,), dtype=i32, device=on)
    kept = torch.empty((B, H, keep), dtype=i32, device=on)
    b = _pack_batch(block_table.data_ptr(), lens.data_ptr(), lens.data_ptr(), B, width, 0, 0)
    st = (_lib or load()).fattn_cache_evict(c, b, wp, wb, wh, w_width, table_out.data_ptr(),
                                            table_out.shape[1], keep, recent, lens_out.data_ptr(),
                                            kept.data_ptr(), op, ob, oh, o_width, _raw_stream(dev))
    if st:
        raise FattnError("fattn_cache_evict", st)
    return lens_out, kept, out


# ------------------------------------------------------------------ rotary positions

ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
# how the frequencies are scaled: number, default fast and slow (turns over the original length)
ROPE_SCALINGS = {"none": (0, 0.0, 0.0), "linear": (1, 0.0, 0.0), "base": (2, 0.0, 0.0),
                 "yarn": (3, 32.0, 1.0), "bands": (4, 4.0, 1.0)}


class RopeTable(typing.NamedTuple):
    """What fattn_rope takes its angles from: a device int64 tensor of rot / 2 fractions of a
    turn (2^-64 each), and the magnitude that the turned channels are multiplied by."""
    turns: torch.Tensor
    magnitude: float


def rope_table(rot, base=10000.0, kind="none", factor=1.0, length=0, fast=None, slow=None,
               device="cuda"):
    """The RopeTable of the frequencies base^(-2 i / rot), scaled by `factor` from an original
    length as fattn_rope_scaling says (kind: "none", "linear", "base", "yarn" or "bands")."""
    if kind not in ROPE_SCALINGS:
        raise ValueError("kind is one of %s, not %r" % (", ".join(ROPE_SCALINGS), kind))
    number, f, s = ROPE_SCALINGS[kind]
    turns = torch.empty((max(rot // 2, 1),), dtype=torch.int64)
    m = ctypes.c_float(0.0)
    _check("fattn_rope_turns", load().fattn_rope_turns(
        turns.data_ptr(), ctypes.byref(m), rot, base, number, factor, length,
        f if fast is None else fast, s if slow is None else slow))
    return RopeTable(turns.to(device), m.value)


def _rope(q, k, positions, table, layout, backward, out, stream):
    turns, magnitude = table
    dev = q.get_device()
    if layout not in ROPE_LAYOUTS:
        raise ValueError("layout is 'half' or 'interleaved', not %r" % (layout,))
    if q.dim() != 3 or dev < 0:
        raise ValueError("expected q [total, Hq, d] on a CUDA device")
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return _rope(q, k, positions, table, layout, backward, out, None)
    T, Hq, d = q.shape
    if positions.dtype is not torch.int32 or positions.shape != (T,) or \
            not positions.is_contiguous() or positions.get_device() != dev:
        raise ValueError("expected contiguous int32 positions [%d] on device %d" % (T, dev))
    if turns.dtype is not torch.int64 or turns.dim() != 1 or not turns.is_contiguous() or \
            turns.get_device() != dev:
        raise ValueError("expected the table of rope_table on device %d" % dev)
    if k is not None and k.dim() != 3:
        raise ValueError("expected k [total, Hk, d]")
    Hk = 0 if k is None else k.shape[1]
    qo, ko = (None, None) if out is None else out
    qp = qop = kp = kop = (None, 0, 0)
    if qo is None:
        qo = torch.empty((T, Hq, d), dtype=torch.bfloat16, device=q.device)
    if Hq:
        qp, qop = _packed(q, T, Hq, d, dev), _packed(qo, T, Hq, d, dev)
    if k is None:
        ko = None
    elif ko is None:
        ko = torch.empty((T, Hk, d), dtype=torch.bfloat16, device=q.device)
    if Hk:
        kp, kop = _packed(k, T, Hk, d, dev), _packed(ko, T, Hk, d, dev)
    st = (_lib or load()).fattn_rope(*qp, *qop, Hq, *kp, *kop, Hk, positions.data_ptr(),
                                     turns.data_ptr(), magnitude, T, d, 2 * turns.shape[0],
                                     ROPE_LAYOUTS[layout], 1 if backward else 0, _raw_stream(dev))
    if st:
        raise FattnError("fattn_rope", st)
    return qo, ko


def rope(q, k, positions, table, layout="half", out=None, stream=None):
    """q [total, Hq, d] and k [total, Hk, d] (bf16, any token and head strides; k may be None)
    with their first rot channels turned to `positions` (device int32 [total]) by a RopeTable.
    layout: "half" pairs channels i and rot / 2 + i, "interleaved" 2 i and 2 i + 1.  out: a pair
    of tensors to write to, the inputs themselves for in place."""
    return _rope(q, k, positions, table, layout, False, out, stream)


def rope_backward(dq, dk, positions, table, layout="half", out=None, stream=None):
    """The gradients with respect to rope's q and k, of those with respect to its results."""
    return _rope(dq, dk, positions, table, layout, True, out, stream)
