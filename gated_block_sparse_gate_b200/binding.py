"""Thin ctypes binding over libgbs.so (the C ABI in include/gbs.h).

Argument marshalling only: torch tensors supply device memory and the current
stream; every step of the computation runs in the library's CUDA kernels.
There is no fallback: if the library or a CUDA device is missing, calls raise.
"""
from __future__ import annotations

import ctypes
import functools
import importlib.util
import operator
import os
import struct

import torch

from gated_block_sparse_gate_b200.build import marshal_path

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libgbs.so")

GBS_OK = 0
STATUS_NAMES = {0: "GBS_OK", 1: "GBS_ERR_INVALID_ARG", 2: "GBS_ERR_UNSUPPORTED", 3: "GBS_ERR_CUDA",
                4: "GBS_ERR_TIMEOUT", 5: "GBS_ERR_WORKSPACE", 6: "GBS_ERR_DEVICE_CHECK"}
MODES = {"train": 0, "sparse": 1, "threshold": 2}
DTYPES = {torch.bfloat16: 0, torch.float32: 1}
OP_FWD, OP_BWD, OP_DECODE = 0, 1, 2

EXPORTED = ("gbs_version", "gbs_status_string", "gbs_last_error", "gbs_workspace_bytes",
            "gbs_clear_error", "gbs_check", "gbs_select", "gbs_fwd", "gbs_bwd", "gbs_decode",
            "gbs_set_timer", "gbs_launch_count", "gbs_selftest_wait_timeout",
            "gbs_qkv_rope_workspace_bytes", "gbs_qkv_rope_fwd", "gbs_qkv_rope_bwd", "gbs_kv4_append",
            "gbs_kv4_read", "gbs_kv4_workspace_bytes", "gbs_kv4_decode")


class GbsError(RuntimeError):
    def __init__(self, status, where, detail=""):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)} {detail}".strip())


class Params(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int),
                ("N", ctypes.c_int), ("d", ctypes.c_int), ("block", ctypes.c_int),
                ("topk", ctypes.c_int), ("mode", ctypes.c_int), ("dtype", ctypes.c_int),
                ("scale", ctypes.c_float), ("tau", ctypes.c_float)]


class KvLayout(ctypes.Structure):
    """gbs_kv_layout: paged / variable-length cache and group-shared selection."""
    _fields_ = [("block_table", ctypes.c_void_p), ("max_blocks", ctypes.c_int),
                ("num_pages", ctypes.c_int), ("seq_lens", ctypes.c_void_p),
                ("group_shared", ctypes.c_int)]


class Heads(ctypes.Structure):
    """gbs_heads: a [B, heads, N, d] tensor by pointer and strides."""
    _fields_ = [("ptr", ctypes.c_void_p), ("stride_b", ctypes.c_int64), ("stride_h", ctypes.c_int64),
                ("stride_n", ctypes.c_int64)]


class RopeParams(ctypes.Structure):
    """gbs_rope_params."""
    _fields_ = [("B", ctypes.c_int), ("N", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int),
                ("d", ctypes.c_int), ("rot", ctypes.c_int), ("interleaved", ctypes.c_int),
                ("n_axes", ctypes.c_int), ("axis", ctypes.c_ubyte * 64), ("max_pos", ctypes.c_int),
                ("dtype", ctypes.c_int), ("w_dtype", ctypes.c_int), ("eps", ctypes.c_float)]


class Kv4CacheDesc(ctypes.Structure):
    """gbs_kv4_cache."""
    _fields_ = [("kc", ctypes.c_void_p), ("kp", ctypes.c_void_p), ("vc", ctypes.c_void_p),
                ("vp", ctypes.c_void_p), ("block_table", ctypes.c_void_p), ("max_blocks", ctypes.c_int),
                ("num_pages", ctypes.c_int), ("cap", ctypes.c_int)]


_lib = None


def load_library(path: str = LIB_PATH):
    """Loads libgbs.so and declares the argument types of every entry point."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing; build it with gated_block_sparse_gate_b200.build")
    _load_marshal()
    lib = ctypes.CDLL(path)
    P = ctypes.POINTER(Params)
    vp, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
    sigs = {
        "gbs_version": (i32, []),
        "gbs_status_string": (ctypes.c_char_p, [i32]),
        "gbs_last_error": (ctypes.c_char_p, []),
        "gbs_workspace_bytes": (sz, [P, i32]),
        "gbs_clear_error": (i32, [vp, vp]),
        "gbs_check": (i32, [vp, vp]),
        "gbs_select": (i32, [P, vp, vp, vp, vp, vp, vp]),
        "gbs_fwd": (i32, [P, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
        "gbs_bwd": (i32, [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
        "gbs_decode": (i32, [P, vp, vp, vp, vp, vp, vp, i32, vp, sz, vp]),
        "gbs_decode_ex": (i32, [P, ctypes.POINTER(KvLayout), vp, vp, vp, vp, vp, vp, i32, vp, sz,
                                vp]),
        "gbs_set_timer": (i32, [i32, vp, vp]),
        "gbs_launch_count": (ctypes.c_uint64, []),
        # structures go as bytes (struct.pack) or byref: both are addresses
        "gbs_qkv_rope_workspace_bytes": (sz, [vp]),
        "gbs_qkv_rope_fwd": (i32, [vp] * 14),
        "gbs_qkv_rope_bwd": (i32, [vp] * 17 + [sz, vp]),
        "gbs_kv4_append": (i32, [vp] * 4 + [i32] + [vp] * 4),
        "gbs_kv4_read": (i32, [vp] * 4 + [i32] + [vp] * 4),
        "gbs_kv4_workspace_bytes": (sz, [vp]),
        "gbs_kv4_decode": (i32, [vp] * 3 + [i32] + [vp] * 4 + [i32, vp, sz, vp]),
    }
    for name, (res, args) in sigs.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    lib.native = struct.pack("7P", *(ctypes.cast(getattr(lib, name), vp).value for name in _NATIVE))
    _lib = lib
    return lib


def _check(status, where):
    if status != GBS_OK:
        detail = load_library().gbs_last_error().decode()
        raise GbsError(status, where, detail)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


# Device types whose memory the kernels may be given; only the unit tests of
# the checks below widen it (to "meta", which has shapes but no storage).
_DEVICE_TYPES = ("cuda",)
_F32 = (torch.float32,)
_I32 = (torch.int32,)
_U8 = (torch.uint8,)
_F16 = (torch.float16,)
_WEIGHTS = (torch.float32, torch.bfloat16)


def _fits(t, dtypes, device_index, shape):
    """Whether a tensor plainly is on that device, of one of the dtypes, of that shape
    (None: any) and contiguous; by csrc/marshal.cpp where that is built."""
    return (type(t) is torch.Tensor and t.get_device() == device_index and t.dtype in dtypes
            and (shape is None or t.shape == shape) and t.is_contiguous())


def _heads_of(t, dtypes, device_index, shape, token_major, written):
    """gbs_heads of a tensor as bytes, or None for anything out of the ordinary; by
    csrc/marshal.cpp where that is built."""
    return None


# The entry points that csrc/marshal.cpp calls, in its order.
_NATIVE = ("gbs_qkv_rope_fwd", "gbs_qkv_rope_bwd", "gbs_qkv_rope_workspace_bytes", "gbs_kv4_append", "gbs_kv4_read",
           "gbs_kv4_decode", "gbs_kv4_workspace_bytes")


class _NoCalls:
    """Stands for csrc/marshal.cpp's calls where it is missing: every one is left to this module."""
    qkv_rope = qkv_rope_backward = kv4_append = kv4_read = kv4_decode = staticmethod(lambda *a: None)


# csrc/marshal.cpp as a module, and what takes whole calls: that module or _NoCalls.
_marshal, _native = None, _NoCalls


def _load_marshal():
    """Takes csrc/marshal.cpp's checks and calls where it is built; else the checks below do all of it. Called at
    the import and again when a library is loaded, since build() may have come between the two."""
    global _marshal, _native, _fits, _heads_of
    if _marshal is not None:
        return
    path = marshal_path()
    if not os.path.exists(path):
        return
    spec = importlib.util.spec_from_file_location("gated_block_sparse_gate_b200._marshal", path)
    try:
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
    except ImportError:
        return
    _marshal = module
    _native, _fits, _heads_of = _marshal, _marshal.fits, _marshal.heads


_load_marshal()


def _invalid(where, detail):
    return GbsError(1, where, detail)


def _device(where, name, t):
    """The device of the call's anchor tensor, which must be a CUDA tensor."""
    if type(t) is not torch.Tensor and not isinstance(t, torch.Tensor):
        raise _invalid(where, f"{name} must be a torch.Tensor")
    device = t.device
    if device.type not in _DEVICE_TYPES:
        raise _invalid(where, f"{name} is on {device}; the kernels need CUDA memory")
    return device


def _need(where, name, t, shape, dtypes, device):
    """t is a contiguous tensor on ``device`` with one of ``dtypes`` and, unless
    ``shape`` is None, exactly that shape: the layout the C ABI reads."""
    if _fits(t, dtypes, device.index, shape):
        return
    if not isinstance(t, torch.Tensor):
        raise _invalid(where, f"{name} must be a torch.Tensor")
    if t.device != device:
        raise _invalid(where, f"{name} is on {t.device}; expected {device}")
    if t.dtype not in dtypes:
        raise _invalid(where, f"{name} has dtype {t.dtype}; expected {' or '.join(map(str, dtypes))}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise _invalid(where, f"{name} has shape {tuple(t.shape)}; expected {tuple(shape)}")
    if not t.is_contiguous():
        raise _invalid(where, f"{name} must be contiguous")


def _act_dtype(where, name, t):
    if t.dtype not in DTYPES:
        raise _invalid(where, f"{name} has dtype {t.dtype}; expected torch.bfloat16 or torch.float32")
    return (t.dtype,)


def _check_prefill(where, Q, K, V, S, block, outs=()):
    """Q [B,Hq,N,d], K and V [B,Hkv,N,d] of Q's dtype, S [B,Hq,Nb,Nb] fp32, and
    each (name, tensor, shape, dtypes) of ``outs``; returns (device, shape dict)."""
    dev = _device(where, "Q", Q)
    if Q.dim() != 4 or not isinstance(K, torch.Tensor) or K.dim() != 4:
        raise _invalid(where, "Q and K must be 4-D: [B, H, N, d]")
    B, Hq, N, d = Q.shape
    Hkv = K.shape[1]
    Nb = -(-N // block)
    act = _act_dtype(where, "Q", Q)
    _need(where, "Q", Q, (B, Hq, N, d), act, dev)
    _need(where, "K", K, (B, Hkv, N, d), act, dev)
    _need(where, "V", V, (B, Hkv, N, d), act, dev)
    _need(where, "S", S, (B, Hq, Nb, Nb), _F32, dev)
    for name, t, shape, dtypes in outs:
        _need(where, name, t, shape, dtypes, dev)
    return dev


def _check_decode(where, q, Kc, Vc, S, L, block, block_table=None, seq_lens=None,
                  group_shared=False, outs=()):
    """q [B,Hq,d]; a cache [B,Hkv,L,d] or, with a block table, page pools
    [pages,Hkv,block,d]; S [B,Hq,Nb] (group-shared: [B,Hkv,Nb]) fp32; an int32
    block table [B, max_blocks] and int32 lengths [B]."""
    dev = _device(where, "q", q)
    if q.dim() != 3 or not isinstance(Kc, torch.Tensor) or Kc.dim() != 4:
        raise _invalid(where, "q must be [B, Hq, d] and the cache 4-D")
    B, Hq, d = q.shape
    Hkv = Kc.shape[1]
    Nb = -(-L // block)
    act = _act_dtype(where, "q", q)
    _need(where, "q", q, (B, Hq, d), act, dev)
    cache = (Kc.shape[0], Hkv, block, d) if block_table is not None else (B, Hkv, L, d)
    _need(where, "Kc", Kc, cache, act, dev)
    _need(where, "Vc", Vc, cache, act, dev)
    _need(where, "S", S, (B, Hkv if group_shared else Hq, Nb), _F32, dev)
    if block_table is not None:
        _need(where, "block_table", block_table, None, _I32, dev)
        if block_table.dim() != 2 or block_table.shape[0] != B:
            raise _invalid(where, f"block_table must be [B={B}, max_blocks]")
    if seq_lens is not None:
        _need(where, "seq_lens", seq_lens, (B,), _I32, dev)
    for name, t, shape, dtypes in outs:
        _need(where, name, t, shape, dtypes, dev)
    return dev


def make_params(B, Hq, Hkv, N, d, block=64, topk=0, mode="train", dtype=torch.bfloat16, scale=0.0,
                tau=0.0):
    return Params(B, Hq, Hkv, N, d, block, topk, MODES[mode], DTYPES[dtype], float(scale),
                  float(tau))


def workspace_bytes(params: Params, op: int) -> int:
    return int(load_library().gbs_workspace_bytes(ctypes.byref(params), op))


def alloc_workspace(params: Params, op: int, device) -> torch.Tensor:
    n = workspace_bytes(params, op)
    if n == 0:
        raise GbsError(1, "workspace_bytes", load_library().gbs_last_error().decode())
    ws = torch.zeros(n, dtype=torch.uint8, device=device)
    assert ws.data_ptr() % 256 == 0
    return ws


def _prefill_params(Q, K, S, block, topk, mode, scale, tau=0.0):
    B, Hq, N, d = Q.shape
    return make_params(B, Hq, K.shape[1], N, d, block, topk, mode, Q.dtype, scale, tau)


def select(S, block=64, topk=0, mode="sparse", N=None, tau=0.0, stream=None):
    """K1: (idx, cnt, logg, slse) for S [B, Hq, Nb, Nb]."""
    lib = load_library()
    dev = _device("gbs_select", "S", S)
    if S.dim() != 4:
        raise _invalid("gbs_select", "S must be [B, Hq, Nb, Nb]")
    B, Hq, Nb, _ = S.shape
    _need("gbs_select", "S", S, (B, Hq, Nb, Nb), _F32, dev)
    N = N if N is not None else Nb * block
    p = make_params(B, Hq, Hq, N, 64, block, topk, mode, torch.float32, tau=tau)
    idx = cnt = logg = None
    if mode != "train":
        idx = torch.empty(B, Hq, Nb, topk, dtype=torch.int32, device=dev)
        cnt = torch.empty(B, Hq, Nb, dtype=torch.int32, device=dev)
        logg = torch.empty(B, Hq, Nb, topk, dtype=torch.float32, device=dev)
    slse = torch.empty(B, Hq, Nb, dtype=torch.float32, device=dev)
    _check(lib.gbs_select(ctypes.byref(p), _ptr(S), _ptr(idx), _ptr(cnt), _ptr(logg), _ptr(slse),
                          _stream(stream)), "gbs_select")
    return idx, cnt, logg, slse


def forward(Q, K, V, S, block=64, mode="train", topk=0, scale=0.0, out=None, lse=None, ws=None,
            tau=0.0, stream=None):
    """Gated attention forward: returns (O, LSE)."""
    lib = load_library()
    _check_prefill("gbs_fwd", Q, K, V, S, block)
    p = _prefill_params(Q, K, S, block, topk, mode, scale, tau)
    O = out if out is not None else torch.empty_like(Q)
    LSE = lse if lse is not None else torch.empty(Q.shape[:3], dtype=torch.float32, device=Q.device)
    if ws is None:
        ws = alloc_workspace(p, OP_FWD, Q.device)
    _check_prefill("gbs_fwd", Q, K, V, S, block,
                   outs=(("O", O, Q.shape, (Q.dtype,)), ("LSE", LSE, Q.shape[:3], _F32),
                         ("ws", ws, None, _U8)))
    _check(lib.gbs_fwd(ctypes.byref(p), _ptr(Q), _ptr(K), _ptr(V), _ptr(S), _ptr(O), _ptr(LSE),
                       _ptr(ws), ws.numel(), _stream(stream)), "gbs_fwd")
    return O, LSE


def backward(Q, K, V, S, O, LSE, dO, block=64, scale=0.0, grads=None, ws=None, mode="train",
             topk=0, tau=0.0, stream=None):
    """Backward of ``forward`` with the same mode/topk/tau: returns (dQ, dK, dV, dS)."""
    lib = load_library()
    _check_prefill("gbs_bwd", Q, K, V, S, block)
    p = _prefill_params(Q, K, S, block, topk, mode, scale, tau)
    if grads is None:
        grads = (torch.empty_like(Q), torch.empty_like(K), torch.empty_like(V), torch.empty_like(S))
    dQ, dK, dV, dS = grads
    if ws is None:
        ws = alloc_workspace(p, OP_BWD, Q.device)
    act = (Q.dtype,)
    _check_prefill("gbs_bwd", Q, K, V, S, block,
                   outs=(("O", O, Q.shape, act), ("LSE", LSE, Q.shape[:3], _F32),
                         ("dO", dO, Q.shape, act), ("dQ", dQ, Q.shape, act),
                         ("dK", dK, K.shape, act), ("dV", dV, V.shape, act),
                         ("dS", dS, S.shape, _F32), ("ws", ws, None, _U8)))
    _check(lib.gbs_bwd(ctypes.byref(p), _ptr(Q), _ptr(K), _ptr(V), _ptr(S), _ptr(O), _ptr(LSE),
                       _ptr(dO), _ptr(dQ), _ptr(dK), _ptr(dV), _ptr(dS), _ptr(ws), ws.numel(),
                       _stream(stream)), "gbs_bwd")
    return dQ, dK, dV, dS


def decode(q, Kc, Vc, S, L=None, block=64, topk=32, scale=0.0, num_splits=0, out=None, lse=None,
           ws=None, tau=None, stream=None):
    """Sparse one-token decode: returns (O [B,Hq,d], LSE [B,Hq]).

    ``tau`` set selects threshold mode (blocks whose gate reaches tau, at most topk).
    """
    lib = load_library()
    L = Kc.shape[2] if L is None else L
    _check_decode("gbs_decode", q, Kc, Vc, S, L, block)
    B, Hq, d = q.shape
    mode = "sparse" if tau is None else "threshold"
    p = make_params(B, Hq, Kc.shape[1], L, d, block, topk, mode, q.dtype, scale,
                    0.0 if tau is None else tau)
    O = out if out is not None else torch.empty_like(q)
    LSE = lse if lse is not None else torch.empty(B, Hq, dtype=torch.float32, device=q.device)
    if ws is None:
        ws = alloc_workspace(p, OP_DECODE, q.device)
    _check_decode("gbs_decode", q, Kc, Vc, S, L, block,
                  outs=(("O", O, q.shape, (q.dtype,)), ("LSE", LSE, (B, Hq), _F32),
                        ("ws", ws, None, _U8)))
    _check(lib.gbs_decode(ctypes.byref(p), _ptr(q), _ptr(Kc), _ptr(Vc), _ptr(S), _ptr(O), _ptr(LSE),
                          num_splits, _ptr(ws), ws.numel(), _stream(stream)), "gbs_decode")
    return O, LSE


def decode_ex(q, Kc, Vc, S, L, block=64, topk=32, scale=0.0, num_splits=0, block_table=None,
              seq_lens=None, group_shared=False, out=None, lse=None, ws=None, tau=None,
              stream=None):
    """gbs_decode_ex: decode over a paged and/or variable-length cache, with one
    selection per q-head or per kv group. ``L`` is the maximum length; with
    ``block_table`` (int32 [B, max_blocks]) Kc/Vc are page pools
    [num_pages, Hkv, block, d]; ``seq_lens`` (int32 [B]) gives each length;
    with ``group_shared`` S is [B, Hkv, Nb]. Returns (O, LSE)."""
    lib = load_library()
    _check_decode("gbs_decode_ex", q, Kc, Vc, S, L, block, block_table, seq_lens, group_shared)
    B, Hq, d = q.shape
    mode = "sparse" if tau is None else "threshold"
    p = make_params(B, Hq, Kc.shape[1], L, d, block, topk, mode, q.dtype, scale,
                    0.0 if tau is None else tau)
    kv = KvLayout(None if block_table is None else block_table.data_ptr(),
                  0 if block_table is None else block_table.shape[1],
                  0 if block_table is None else Kc.shape[0],
                  None if seq_lens is None else seq_lens.data_ptr(), 1 if group_shared else 0)
    O = out if out is not None else torch.empty_like(q)
    LSE = lse if lse is not None else torch.empty(B, Hq, dtype=torch.float32, device=q.device)
    if ws is None:
        ws = alloc_workspace(p, OP_DECODE, q.device)
    _check_decode("gbs_decode_ex", q, Kc, Vc, S, L, block, block_table, seq_lens, group_shared,
                  outs=(("O", O, q.shape, (q.dtype,)), ("LSE", LSE, (B, Hq), _F32),
                        ("ws", ws, None, _U8)))
    _check(lib.gbs_decode_ex(ctypes.byref(p), ctypes.byref(kv), _ptr(q), _ptr(Kc), _ptr(Vc), _ptr(S),
                             _ptr(O), _ptr(LSE), num_splits, _ptr(ws), ws.numel(), _stream(stream)),
           "gbs_decode_ex")
    return O, LSE


def set_timer(op: int, start=None, stop=None):
    """Brackets the main kernel of ``op`` with two recorded torch.cuda.Events.

    The events must already exist on the device (record them once first).
    Pass None to clear.
    """
    h0 = None if start is None else ctypes.c_void_p(start.cuda_event)
    h1 = None if stop is None else ctypes.c_void_p(stop.cuda_event)
    _check(load_library().gbs_set_timer(op, h0, h1), "gbs_set_timer")


def launch_count() -> int:
    """Kernels launched by the library so far in this process."""
    return int(load_library().gbs_launch_count())


def check(ws, stream=None):
    """Raises GbsError if a kernel recorded a device-side error in ``ws``."""
    _device("gbs_check", "ws", ws)
    _check(load_library().gbs_check(_ptr(ws), _stream(stream)), "gbs_check")


def clear_error(ws, stream=None):
    """Clears the device error word of ``ws`` (asynchronous)."""
    _device("gbs_clear_error", "ws", ws)
    _check(load_library().gbs_clear_error(_ptr(ws), _stream(stream)), "gbs_clear_error")


def selftest_wait_timeout(ws, limit_us, stream=None):
    """gbs_selftest_wait_timeout: one bounded device wait that nothing releases;
    after ``limit_us`` it records GBS_ERR_TIMEOUT in the error word of ``ws``."""
    lib = load_library()
    f = lib.gbs_selftest_wait_timeout
    f.restype = ctypes.c_int
    f.argtypes = [ctypes.c_void_p, ctypes.c_uint, ctypes.c_void_p]
    _device("gbs_selftest_wait_timeout", "ws", ws)
    _check(f(_ptr(ws), int(limit_us), _stream(stream)), "gbs_selftest_wait_timeout")


def decode_noalloc(q, Kc, Vc, S, L=None, block=64, topk=32, scale=0.0, num_splits=0, out=None,
                   lse=None, tau=None, stream=None):
    """gbs_decode_noalloc: the decode with the library's own static scratch.

    For callers that cannot allocate device memory while decoding; see
    include/gbs.h for the limits and the sharing rules.
    """
    lib = load_library()
    f = lib.gbs_decode_noalloc
    vp = ctypes.c_void_p
    f.restype = ctypes.c_int
    f.argtypes = [ctypes.POINTER(Params), vp, vp, vp, vp, vp, vp, ctypes.c_int, vp]
    L = Kc.shape[2] if L is None else L
    _check_decode("gbs_decode_noalloc", q, Kc, Vc, S, L, block)
    B, Hq, d = q.shape
    mode = "sparse" if tau is None else "threshold"
    p = make_params(B, Hq, Kc.shape[1], L, d, block, topk, mode, q.dtype, scale,
                    0.0 if tau is None else tau)
    O = out if out is not None else torch.empty_like(q)
    LSE = lse if lse is not None else torch.empty(B, Hq, dtype=torch.float32, device=q.device)
    _check_decode("gbs_decode_noalloc", q, Kc, Vc, S, L, block,
                  outs=(("O", O, q.shape, (q.dtype,)), ("LSE", LSE, (B, Hq), _F32)))
    _check(f(ctypes.byref(p), _ptr(q), _ptr(Kc), _ptr(Vc), _ptr(S), _ptr(O), _ptr(LSE), num_splits,
             _stream(stream)), "gbs_decode_noalloc")
    return O, LSE


# ------------------------------------------- projections to attention, 4-bit cache


def _elsewhere(where, device, stream):
    """What a call has to enter before it allocates and launches: ``stream``, so that
    temporaries belong to the stream that uses them, or the tensors' device. None
    where both are current already."""
    if stream is not None:
        if stream.device != device:  # (its kernels would start on another stream, of the tensors' device)
            raise _invalid(where, f"stream is on {stream.device}; expected {device}")
        return torch.cuda.stream(stream)
    if device.type == "cuda" and device.index != torch._C._cuda_getDevice():
        return torch.cuda.device(device)
    return None


def _current(device):
    """The handle of ``device``'s current stream."""
    return torch._C._cuda_getCurrentRawStream(device.index)


def _addr(t):
    return None if t is None else t.data_ptr()


def _in_layout(fmt):
    """pack(where, values...) of a C structure; a value that does not fit is refused in ``where``'s name."""
    pack = struct.Struct(fmt).pack

    def packed(where, *values):
        try:
            return pack(*values)
        except (struct.error, OverflowError) as e:
            raise _invalid(where, f"a size or number cannot be passed: {e}") from None

    return packed


# The structures of include/gbs.h that the calls below pass, in C layout.
_PARAMS = _in_layout("9i2f")
_HEADS = struct.Struct("P3q").pack
_KV4 = struct.Struct("5P3i4x").pack
_ROPE = _in_layout("8i64s3if")
assert struct.calcsize("9i2f") == ctypes.sizeof(Params) and struct.calcsize("P3q") == ctypes.sizeof(Heads)
assert struct.calcsize("5P3i4x") == ctypes.sizeof(Kv4CacheDesc)
assert struct.calcsize("8i64s3if") == ctypes.sizeof(RopeParams)


def _heads(where, name, t, shape, dtypes, device, token_major=False, out=False):
    """A [B, H, N, d] tensor (``token_major``: [B, N, H, d]) with contiguous
    channels as gbs_heads."""
    h = _heads_of(t, dtypes, device.index, shape, token_major, out)
    if h is not None:
        return h
    if not isinstance(t, torch.Tensor):
        raise _invalid(where, f"{name} must be a torch.Tensor")
    if t.device != device:
        raise _invalid(where, f"{name} is on {t.device}; expected {device}")
    if t.dtype not in dtypes:
        raise _invalid(where, f"{name} has dtype {t.dtype}; expected {' or '.join(map(str, dtypes))}")
    if tuple(t.shape) != shape:
        raise _invalid(where, f"{name} has shape {tuple(t.shape)}; expected {shape}")
    b, x, y, c = t.stride()
    if c != 1:
        raise _invalid(where, f"{name} must have contiguous channels")
    if 1 in shape:  # the stride of a dimension of one is never followed
        b, x, y = (0 if n == 1 else step for n, step in zip(shape, (b, x, y)))
    if out and not t.is_contiguous():
        need = shape[3]
        for step, n in sorted(p for p in zip((b, x, y), shape) if p[1] > 1):
            if step < need:
                raise _invalid(where, f"{name} is written and has elements that share memory")
            need = step * n
    if token_major:
        x, y = y, x
    if b < 0 or x < 0 or y < 0:  # (torch has none; pack would take them)
        raise _invalid(where, f"{name} has a negative stride")
    return _HEADS(t.data_ptr(), b, x, y)


def _check_ws(where, ws, device):
    """An optional workspace whose error word is all that is used."""
    if ws is not None:
        _need(where, "ws", ws, None, _U8, device)
        if ws.numel() < 256:
            raise GbsError(5, where, "ws must have at least 256 bytes")


def rope_tables(max_pos, rot, base=10000.0, device="cuda"):
    """(cos, sin) [max_pos, rot / 2] fp32 of the angles pos * base^(-2 i / rot),
    computed in 64 bits (an fp32 angle of a far position is off by whole degrees)."""
    half = rot // 2
    freq = base ** (-torch.arange(half, dtype=torch.float64, device=device) / max(half, 1))
    angle = torch.arange(max_pos, dtype=torch.float64, device=device)[:, None] * freq
    return angle.cos().float(), angle.sin().float()


def rope_axes(sections, interleaved=False):
    """The axis of every rotated pair from the number of pairs per axis: blocks
    (all of axis 0, then axis 1, ...), or dealt out in turn while an axis has
    pairs left."""
    if not interleaved:
        return tuple(a for a, n in enumerate(sections) for _ in range(n))
    left, out = list(sections), []
    while any(left):
        for a in range(len(left)):
            if left[a]:
                left[a] -= 1
                out.append(a)
    return tuple(out)


_ONE_AXIS = (0,) * 64


@functools.lru_cache(maxsize=64)
def _axis_bytes(axes, half, n_axes):
    """The axes of ``half`` pairs as bytes, or the text why they are refused."""
    if len(axes) != half:
        return f"axes has {len(axes)} entries; expected one of each of the {half} pairs"
    if not all(0 <= a < n_axes for a in axes):
        return f"an axis is outside [0, {n_axes})"
    return bytes(axes)


def _rope_call(where, q, k, cos, sin, pos, wq, wk, eps, axes, interleaved, dev):
    """The parameters of a qkv_rope call and (B, N, Hq, Hkv, d), its small tensors checked."""
    if q.dim() != 4 or not isinstance(k, torch.Tensor) or k.dim() != 4:
        raise _invalid(where, "q and k must be 4-D: [B, N, H, d]")
    B, N, Hq, d = q.shape
    Hkv = k.shape[2]
    _act_dtype(where, "q", q)
    if not isinstance(cos, torch.Tensor) or cos.dim() != 2:
        raise _invalid(where, "cos must be [max_pos, rot / 2]")
    table = max_pos, half = cos.shape
    _need(where, "cos", cos, table, _F32, dev)
    _need(where, "sin", sin, table, _F32, dev)
    if not isinstance(pos, torch.Tensor) or pos.dim() not in (2, 3):
        raise _invalid(where, "pos must be [B, N] or [B, N, axes]")
    n_axes = 1 if pos.dim() == 2 else pos.shape[2]
    _need(where, "pos", pos, (B, N) if pos.dim() == 2 else (B, N, n_axes), _I32, dev)
    if half > 64:
        raise _invalid(where, f"cos has {half} columns; at most d / 2 = {d // 2} pairs are rotated")
    try:
        axes = _ONE_AXIS[:half] if axes is None else tuple(map(operator.index, axes))
    except TypeError:
        raise _invalid(where, "axes must be whole numbers, one of each pair") from None
    axis = _axis_bytes(axes, half, n_axes)
    if type(axis) is str:
        raise _invalid(where, axis)
    if (wq is None) != (wk is None):
        raise _invalid(where, "give both weights or neither")
    w_dtype = 1
    if wq is not None:
        _need(where, "wq", wq, (d,), _WEIGHTS, dev)
        _need(where, "wk", wk, (d,), (wq.dtype,), dev)
        w_dtype = DTYPES[wq.dtype]
    return _ROPE(where, B, N, Hq, Hkv, d, 2 * half, 1 if interleaved else 0, n_axes, axis, max_pos, DTYPES[q.dtype],
                 w_dtype, eps), (B, N, Hq, Hkv, d)


def qkv_rope(q, k, v, cos, sin, pos, wq=None, wk=None, eps=1e-6, axes=None, interleaved=False, out=None,
             ws=None, stream=None):
    """Norm of every query and key head (weights ``wq``, ``wk`` [d]; None: no norm)
    and rotary positions, from a projection's q [B, N, Hq, d], k and v
    [B, N, Hkv, d] (any strides with contiguous channels, such as parts of one
    packed tensor; v may be None) to Q [B, Hq, N, d], K and V [B, Hkv, N, d].

    ``cos``, ``sin``: fp32 [max_pos, rot / 2] (``rope_tables``); the first rot
    channels are rotated in pairs of halves or, ``interleaved``, of neighbours.
    ``pos``: int32 [B, N], or [B, N, axes] with ``axes`` the axis of every pair
    (``rope_axes``; without them every pair is on the first). ``out``: (Q, K, V) to write
    to, strided too, in no memory of the inputs. Returns (Q, K, V)."""
    where = "gbs_qkv_rope_fwd"
    if stream is None:
        r = _native.qkv_rope(load_library().native, q, k, v, cos, sin, pos, wq, wk, eps, axes, interleaved, out, ws)
        if r is not None:
            if r[0]:
                _check(r[0], where)
            return r[1:]
    lib = load_library()
    dev = _device(where, "q", q)
    ctx = _elsewhere(where, dev, stream)
    if ctx is not None:
        with ctx:
            return qkv_rope(q, k, v, cos, sin, pos, wq, wk, eps, axes, interleaved, out, ws)
    p, (B, N, Hq, Hkv, d) = _rope_call(where, q, k, cos, sin, pos, wq, wk, eps, axes, interleaved, dev)
    act = (q.dtype,)
    hq = _heads(where, "q", q, (B, N, Hq, d), act, dev, True)
    hk = _heads(where, "k", k, (B, N, Hkv, d), act, dev, True)
    hv = None if v is None else _heads(where, "v", v, (B, N, Hkv, d), act, dev, True)
    if out is not None and (not isinstance(out, (tuple, list)) or len(out) != 3 or (out[2] is None) != (v is None)):
        raise _invalid(where, "out must be (Q, K, V), V None exactly if v is")
    _check_ws(where, ws, dev)
    Q, K, V = out if out is not None else (
        q.new_empty((B, Hq, N, d)), q.new_empty((B, Hkv, N, d)), None if v is None else q.new_empty((B, Hkv, N, d)))
    oq = _heads(where, "Q", Q, (B, Hq, N, d), act, dev, out=True)
    ok = _heads(where, "K", K, (B, Hkv, N, d), act, dev, out=True)
    ov = None if v is None else _heads(where, "V", V, (B, Hkv, N, d), act, dev, out=True)
    s = lib.gbs_qkv_rope_fwd(p, hq, hk, hv, _addr(wq), _addr(wk), cos.data_ptr(), sin.data_ptr(), pos.data_ptr(),
                             oq, ok, ov, _addr(ws), _current(dev))
    if s:
        _check(s, where)
    return Q, K, V


def qkv_rope_backward(q, k, cos, sin, pos, dQ, dK, dV=None, wq=None, wk=None, eps=1e-6, axes=None,
                      interleaved=False, grads=None, ws=None, stream=None):
    """Backward of ``qkv_rope`` with the same arguments: from dQ [B, Hq, N, d], dK and
    dV [B, Hkv, N, d] (what ``backward`` returns; dV may be None) to
    (dq, dk, dv, dwq, dwk): dq [B, N, Hq, d], dk, dv [B, N, Hkv, d] and fp32
    dwq, dwk [d] (None without weights). ``grads``: (dq, dk, dv) to write to,
    such as parts of one packed tensor, in no memory of the inputs."""
    where = "gbs_qkv_rope_bwd"
    if stream is None:
        r = _native.qkv_rope_backward(load_library().native, q, k, cos, sin, pos, dQ, dK, dV, wq, wk, eps, axes,
                                      interleaved, grads, ws)
        if r is not None:
            if r[0]:
                _check(r[0], where)
            return r[1:]
    lib = load_library()
    dev = _device(where, "q", q)
    ctx = _elsewhere(where, dev, stream)
    if ctx is not None:
        with ctx:
            return qkv_rope_backward(q, k, cos, sin, pos, dQ, dK, dV, wq, wk, eps, axes, interleaved, grads, ws)
    p, (B, N, Hq, Hkv, d) = _rope_call(where, q, k, cos, sin, pos, wq, wk, eps, axes, interleaved, dev)
    act = (q.dtype,)
    hq = _heads(where, "q", q, (B, N, Hq, d), act, dev, True)
    hk = _heads(where, "k", k, (B, N, Hkv, d), act, dev, True)
    zq = _heads(where, "dQ", dQ, (B, Hq, N, d), act, dev)
    zk = _heads(where, "dK", dK, (B, Hkv, N, d), act, dev)
    zv = None if dV is None else _heads(where, "dV", dV, (B, Hkv, N, d), act, dev)
    if grads is not None and (not isinstance(grads, (tuple, list)) or len(grads) != 3
                              or (grads[2] is None) != (dV is None)):
        raise _invalid(where, "grads must be (dq, dk, dv), dv None exactly if dV is")
    if ws is not None:
        _need(where, "ws", ws, None, _U8, dev)
    dq, dk, dv = grads if grads is not None else (
        q.new_empty((B, N, Hq, d)), q.new_empty((B, N, Hkv, d)), None if dV is None else q.new_empty((B, N, Hkv, d)))
    oq = _heads(where, "dq", dq, (B, N, Hq, d), act, dev, True, True)
    ok = _heads(where, "dk", dk, (B, N, Hkv, d), act, dev, True, True)
    ov = None if dV is None else _heads(where, "dv", dv, (B, N, Hkv, d), act, dev, True, True)
    dwq, dwk = (None, None) if wq is None else q.new_empty((2, d), dtype=torch.float32).unbind()
    if ws is None:
        ws = q.new_empty(lib.gbs_qkv_rope_workspace_bytes(p) or 256, dtype=torch.uint8)
    s = lib.gbs_qkv_rope_bwd(p, hq, hk, _addr(wq), _addr(wk), cos.data_ptr(), sin.data_ptr(), pos.data_ptr(), zq, zk,
                             zv, oq, ok, ov, _addr(dwq), _addr(dwk), ws.data_ptr(), ws.numel(), _current(dev))
    if s:
        _check(s, where)
    return dq, dk, dv, dwq, dwk


def qkv_rope_workspace_bytes(q, k, rot):
    """Bytes of ``ws`` for ``qkv_rope_backward`` (``qkv_rope`` takes the same one)."""
    B, N, Hq, d = q.shape
    where = "gbs_qkv_rope_workspace_bytes"
    p = _ROPE(where, B, N, Hq, k.shape[2], d, rot, 0, 1, b"", 1, DTYPES[q.dtype], 1, 0.0)
    n = int(load_library().gbs_qkv_rope_workspace_bytes(p))
    if n == 0:
        raise GbsError(1, where, load_library().gbs_last_error().decode())
    return n


def kv4_cache(B, Hkv, d, L=None, num_pages=None, block=64, device="cuda"):
    """A 4-bit cache (codes and parameters of keys, then of values) of zeros:
    contiguous for B sequences of up to L tokens, or ``num_pages`` pages."""
    if (L is None) == (num_pages is None):
        raise _invalid("kv4_cache", "give either L or num_pages")
    rows = (num_pages, Hkv, block) if L is None else (B, Hkv, -(-L // block) * block)
    out = []
    for _ in range(2):
        out += [torch.zeros(*rows, d // 2, dtype=torch.uint8, device=device),
                torch.zeros(*rows, d // 32, 2, dtype=torch.float16, device=device)]
    return tuple(out)


def _check_kv4(where, cache, B, d, device, block, block_table):
    """(gbs_kv4_cache, Hkv, longest length that fits) of a 4-bit cache: four
    tensors, codes [B, Hkv, cap, d / 2] uint8 and parameters [B, Hkv, cap, d / 32, 2]
    fp16 of keys and of values, or pages [num_pages, Hkv, block, ...]."""
    if not isinstance(cache, (tuple, list)) or len(cache) != 4:
        raise _invalid(where, "cache must be (key codes, key parameters, value codes, value parameters)")
    kc, kp, vc, vp = cache
    if not isinstance(kc, torch.Tensor) or kc.dim() != 4:
        raise _invalid(where, "key codes must be 4-D")
    first, Hkv, rows, _ = kc.shape
    if block_table is None:
        if first != B or rows % block:
            raise _invalid(where, f"key codes have shape {tuple(kc.shape)}; expected ({B}, Hkv, a multiple of "
                                  f"{block}, {d // 2})")
    elif rows != block:
        raise _invalid(where, f"a page of the key codes has {rows} rows; expected {block}")
    codes, params = (first, Hkv, rows, d // 2), (first, Hkv, rows, d // 32, 2)
    _need(where, "key codes", kc, codes, _U8, device)
    _need(where, "key parameters", kp, params, _F16, device)
    _need(where, "value codes", vc, codes, _U8, device)
    _need(where, "value parameters", vp, params, _F16, device)
    if block_table is None:
        desc = _KV4(kc.data_ptr(), kp.data_ptr(), vc.data_ptr(), vp.data_ptr(), 0, 0, 0, rows)
        return desc, Hkv, rows
    _need(where, "block_table", block_table, None, _I32, device)
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise _invalid(where, f"block_table must be [B={B}, max_blocks]")
    max_blocks = block_table.shape[1]
    desc = _KV4(kc.data_ptr(), kp.data_ptr(), vc.data_ptr(), vp.data_ptr(), block_table.data_ptr(), max_blocks, first,
                rows)
    return desc, Hkv, min(max_blocks * block, 2**31 - 1)  # (positions are int32)


def _kv4_rows(where, fn, K, V, cache, start, block_table, count, ws, block, out, dev):
    """The checks and the call that ``kv4_append`` and ``kv4_read`` share."""
    if K.dim() != 4:
        raise _invalid(where, "K must be [B, Hkv, T, d]")
    B, _, T, d = K.shape
    act = _act_dtype(where, "K", K)
    desc, Hkv, L = _check_kv4(where, cache, B, d, dev, block, block_table)
    hk = _heads(where, "K", K, (B, Hkv, T, d), act, dev, False, out)
    hv = _heads(where, "V", V, (B, Hkv, T, d), act, dev, False, out)
    _need(where, "start", start, (B,), _I32, dev)
    if count is not None:
        _need(where, "count", count, (B,), _I32, dev)
    _check_ws(where, ws, dev)
    if T == 0:
        return
    s = fn(_PARAMS(where, B, Hkv, Hkv, L, d, block, 0, 0, DTYPES[K.dtype], 0.0, 0.0), desc, hk, hv, T, start.data_ptr(),
           _addr(count), _addr(ws), _current(dev))
    if s:
        _check(s, where)


def kv4_append(K, V, cache, start, block_table=None, count=None, block=64, ws=None, stream=None):
    """Writes K and V [B, Hkv, T, d] (any strides with contiguous channels) into a
    4-bit cache (``kv4_cache``), token t of sequence b at position start[b] + t
    (``start`` int32 [B]); with ``count`` (int32 [B]) only its first count[b]
    tokens. ``block_table`` (int32 [B, max_blocks]) makes the cache page pools."""
    where = "gbs_kv4_append"
    if stream is None:
        r = _native.kv4_append(load_library().native, K, V, cache, start, block_table, count, block, ws)
        if r is not None:
            if r[0]:
                _check(r[0], where)
            return
    fn = load_library().gbs_kv4_append
    dev = _device(where, "K", K)
    ctx = _elsewhere(where, dev, stream)
    if ctx is not None:
        with ctx:
            return kv4_append(K, V, cache, start, block_table, count, block, ws)
    _kv4_rows(where, fn, K, V, cache, start, block_table, count, ws, block, False, dev)


def kv4_read(cache, start, T, block_table=None, count=None, dtype=torch.bfloat16, block=64, out=None, ws=None,
             stream=None):
    """The values of T tokens of every sequence from position ``start`` on:
    (K, V) [B, Hkv, T, d] of ``dtype`` (``out`` to write to, strided too); tokens
    from count[b] on are zeros."""
    where = "gbs_kv4_read"
    if stream is None:
        r = _native.kv4_read(load_library().native, cache, start, T, block_table, count, dtype, block, out, ws)
        if r is not None:
            if r[0]:
                _check(r[0], where)
            return r[1:]
    fn = load_library().gbs_kv4_read
    dev = _device(where, "start", start)
    ctx = _elsewhere(where, dev, stream)
    if ctx is not None:
        with ctx:
            return kv4_read(cache, start, T, block_table, count, dtype, block, out, ws)
    if not isinstance(cache, (tuple, list)) or len(cache) != 4 or not isinstance(cache[0], torch.Tensor) \
            or cache[0].dim() != 4:
        raise _invalid(where, "cache must be (key codes, key parameters, value codes, value parameters)")
    if dtype not in DTYPES:
        raise _invalid(where, f"dtype {dtype}; expected torch.bfloat16 or torch.float32")
    if not isinstance(T, int) or T < 0:
        raise _invalid(where, "T must be a whole number and not negative")
    if start.dim() != 1:
        raise _invalid(where, "start must be [B]")
    if out is None:
        shape = (start.shape[0], cache[0].shape[1], T, 2 * cache[0].shape[3])
        K, V = start.new_empty(shape, dtype=dtype), start.new_empty(shape, dtype=dtype)
    elif not isinstance(out, (tuple, list)) or len(out) != 2:
        raise _invalid(where, "out must be (K, V)")
    else:
        K, V = out
        _device(where, "K", K)
        if K.dim() != 4 or K.shape[2] != T:
            raise _invalid(where, f"out must be (K, V) [B, Hkv, T={T}, d]")
    _kv4_rows(where, fn, K, V, cache, start, block_table, count, ws, block, True, dev)
    return K, V


def kv4_workspace_bytes(params: Params) -> int:
    return int(load_library().gbs_kv4_workspace_bytes(ctypes.byref(params)))


def kv4_decode(q, cache, S, L, block=64, topk=32, scale=0.0, num_splits=0, block_table=None, seq_lens=None,
               group_shared=False, out=None, lse=None, ws=None, tau=None, stream=None):
    """gbs_kv4_decode: ``decode_ex`` over a 4-bit cache (``kv4_cache``). q [B, Hq, d]
    (bf16 or fp32), S [B, Hq, ceil(L / block)] (group-shared: [B, Hkv, ..]) fp32,
    ``L`` the longest length; ``seq_lens`` int32 [B] may hold 0 for an idle slot,
    whose O is 0 and LSE -inf. Returns (O, LSE)."""
    where = "gbs_kv4_decode"
    if stream is None:
        r = _native.kv4_decode(load_library().native, q, cache, S, L, block, topk, scale, num_splits, block_table,
                               seq_lens, group_shared, out, lse, ws, tau)
        if r is not None:
            if r[0]:
                _check(r[0], where)
            return r[1:]
    lib = load_library()
    dev = _device(where, "q", q)
    ctx = _elsewhere(where, dev, stream)
    if ctx is not None:
        with ctx:
            return kv4_decode(q, cache, S, L, block, topk, scale, num_splits, block_table, seq_lens, group_shared,
                              out, lse, ws, tau)
    if q.dim() != 3:
        raise _invalid(where, "q must be [B, Hq, d]")
    B, Hq, d = q.shape
    act = _act_dtype(where, "q", q)
    _need(where, "q", q, (B, Hq, d), act, dev)
    desc, Hkv, most = _check_kv4(where, cache, B, d, dev, block, block_table)
    if not 1 <= L <= most:
        raise _invalid(where, f"L = {L} is outside [1, {most}], what the cache holds")
    _need(where, "S", S, (B, Hkv if group_shared else Hq, -(-L // block)), _F32, dev)
    if seq_lens is not None:
        _need(where, "seq_lens", seq_lens, (B,), _I32, dev)
    if ws is not None:
        _need(where, "ws", ws, None, _U8, dev)
    p = _PARAMS(where, B, Hq, Hkv, L, d, block, topk, 1 if tau is None else 2, DTYPES[q.dtype], scale,
                0.0 if tau is None else tau)
    if out is None:
        out = torch.empty_like(q)
    else:
        _need(where, "O", out, (B, Hq, d), act, dev)
    if lse is None:
        lse = q.new_empty((B, Hq), dtype=torch.float32)
    else:
        _need(where, "LSE", lse, (B, Hq), _F32, dev)
    if ws is None:
        ws = q.new_empty(lib.gbs_kv4_workspace_bytes(p) or 256, dtype=torch.uint8)
    s = lib.gbs_kv4_decode(p, desc, _addr(seq_lens), 1 if group_shared else 0, q.data_ptr(), S.data_ptr(),
                           out.data_ptr(), lse.data_ptr(), num_splits, ws.data_ptr(), ws.numel(), _current(dev))
    if s:
        _check(s, where)
    return out, lse
