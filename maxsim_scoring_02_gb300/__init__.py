"""Late-interaction MaxSim scoring on NVIDIA GB300 (sm_103a).

Thin Python binding over the C ABI of ``libmaxsim.so`` (``include/maxsim.h``).
Every function here only checks and marshals arguments: it takes torch
tensors that already live on the GPU, passes their device pointers and the
current CUDA stream to the library, and allocates outputs with torch when the
caller did not pass them. Every step of the computation runs in the
library's CUDA kernels; there is no CPU or PyTorch fallback, and importing
this package fails loudly if the library has not been built.

Operator (TileMaxSim deep reading §1; FLASH-MAXSIM, Abstract):
    score(Q, D_b) = sum_i max_{j < L_b} <q_i, d_j>
"""
from __future__ import annotations

import array
import contextlib
import ctypes
import functools
import inspect
import math
import operator
import os

import torch

__all__ = [
    "MaxSimError", "library_path", "load_library", "maxsim_score", "maxsim_score_varlen", "maxsim_length_order",
    "maxsim_score_ordered", "maxsim_length_order_workspace_size",
    "maxsim_score_streamed", "maxsim_score_streamed_workspace_size",
    "maxsim_score_pq", "maxsim_score_pq_workspace_size", "maxsim_score_i8", "maxsim_backward",
    "maxsim_backward_workspace_size", "maxsim_backward_dq", "maxsim_backward_dd", "maxsim_device_status",
    "maxsim_version", "allreduce_dq",
    "maxsim_rotary_frequencies", "maxsim_rotary", "maxsim_attention", "maxsim_attention_backward",
    "maxsim_attention_backward_workspace_size", "maxsim_clip_grad_norm", "maxsim_clip_grad_norm_workspace_size",
    "encoder_dropout", "encoder_rms_norm", "encoder_rms_norm_backward", "encoder_rms_norm_backward_workspace_size",
    "encoder_cross_entropy", "encoder_cross_entropy_workspace_size", "encoder_cross_entropy_backward",
    "encoder_cross_entropy_backward_workspace_size",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_NAME = "libmaxsim.so"

BF16, FP16, FP32 = 0, 1, 2
_DTYPE_CODE = {torch.bfloat16: BF16, torch.float16: FP16, torch.float32: FP32}

STATUS_NAMES = {0: "MAXSIM_OK", 1: "MAXSIM_ERR_INVALID_ARG", 2: "MAXSIM_ERR_UNSUPPORTED",
                3: "MAXSIM_ERR_CUDA", 4: "MAXSIM_ERR_TIMEOUT", 5: "MAXSIM_ERR_WORKSPACE"}
DEVERR_TIMEOUT = 0x1
DEVERR_BAD_INPUT = 0x2
DEBUG_STALL_FWD_LOADER = 0x1

# Every symbol the header declares (checked by the tests).
EXPORTS = (
    "maxsim_version", "maxsim_status_string", "maxsim_device_status", "maxsim_debug_set_faults",
    "maxsim_score",
    "maxsim_score_varlen", "maxsim_length_order_workspace_size", "maxsim_length_order", "maxsim_score_ordered",
    "maxsim_score_streamed_workspace_size", "maxsim_score_streamed",
    "maxsim_score_pq_workspace_size", "maxsim_score_pq", "maxsim_score_pq_noalloc",
    "maxsim_score_i8",
    "maxsim_backward_workspace_size", "maxsim_backward", "maxsim_backward_dq", "maxsim_backward_dd",
    "maxsim_rotary_frequencies", "maxsim_rotary", "maxsim_attention",
    "maxsim_attention_backward_workspace_size", "maxsim_attention_backward",
    "maxsim_clip_grad_norm_workspace_size", "maxsim_clip_grad_norm",
    "maxsim_dropout", "maxsim_rms_norm", "maxsim_rms_norm_backward_workspace_size", "maxsim_rms_norm_backward",
    "maxsim_cross_entropy_workspace_size", "maxsim_cross_entropy",
    "maxsim_cross_entropy_backward_workspace_size", "maxsim_cross_entropy_backward",
)

ROTARY_SCALING = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}
MASKS = {"full": 0, "causal": 1, "prefix": 2}
NORM_FORMATS = {None: (0, None), "int8": (1, torch.int8), "e4m3": (2, torch.float8_e4m3fn)}


class _Heads(ctypes.Structure):
    """maxsim_heads: a [T, heads, d] view, strides in elements."""
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class _AttentionSpec(ctypes.Structure):
    """maxsim_attention_spec."""
    _fields_ = [("T", ctypes.c_int64), ("B", ctypes.c_int64), ("heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("d", ctypes.c_int32), ("dtype", ctypes.c_int), ("mask", ctypes.c_int), ("scale", ctypes.c_float),
                ("cap", ctypes.c_float), ("offsets", ctypes.c_void_p), ("key_len", ctypes.c_void_p),
                ("prefix_len", ctypes.c_void_p), ("slopes", ctypes.c_void_p)]


class _Rows(ctypes.Structure):
    """maxsim_rows: a [T, d] view, its stride in elements."""
    _fields_ = [("data", ctypes.c_void_p), ("row_stride", ctypes.c_int64)]


class _NormSpec(ctypes.Structure):
    """maxsim_norm_spec."""
    _fields_ = [("T", ctypes.c_int64), ("d", ctypes.c_int32), ("dtype", ctypes.c_int), ("weight_dtype", ctypes.c_int),
                ("format", ctypes.c_int), ("eps", ctypes.c_float), ("p", ctypes.c_float), ("rng", ctypes.c_void_p),
                ("weight", ctypes.c_void_p)]


class _LossSpec(ctypes.Structure):
    """maxsim_loss_spec."""
    _fields_ = [("T", ctypes.c_int64), ("V", ctypes.c_int64), ("d", ctypes.c_int32), ("dtype", ctypes.c_int),
                ("scale", ctypes.c_float), ("targets", ctypes.c_void_p)]


class MaxSimError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {STATUS_NAMES.get(status, status)}")


def library_path() -> str:
    return os.path.join(_HERE, _LIB_NAME)


_lib = None


def load_library():
    """Load libmaxsim.so (built in-tree by ``__graft_entry__.build()``)."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build the CUDA library first "
                          "(python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(path)
    P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    lib.maxsim_version.restype = I32
    lib.maxsim_status_string.restype = ctypes.c_char_p
    lib.maxsim_status_string.argtypes = [I32]
    lib.maxsim_device_status.restype = I32
    lib.maxsim_device_status.argtypes = [P, ctypes.POINTER(ctypes.c_uint)]
    lib.maxsim_debug_set_faults.restype = I32
    lib.maxsim_debug_set_faults.argtypes = [ctypes.c_uint, ctypes.c_uint64]
    lib.maxsim_score.restype = I32
    lib.maxsim_score.argtypes = [P, I32, I32, I32, P, I64, I32, P, I32, P, P, P]
    lib.maxsim_length_order_workspace_size.restype = SZ
    lib.maxsim_length_order_workspace_size.argtypes = [I64, I32, I32]
    lib.maxsim_length_order.restype = I32
    lib.maxsim_length_order.argtypes = [P, P, I64, I32, P, P, SZ, P]
    lib.maxsim_score_ordered.restype = I32
    lib.maxsim_score_ordered.argtypes = [P, I32, I32, I32, P, I64, I32, P, P, I32, P, P, P]
    lib.maxsim_score_varlen.restype = I32
    lib.maxsim_score_varlen.argtypes = [P, I32, I32, I32, P, P, I64, I64, I32, P, P, P]
    lib.maxsim_score_streamed_workspace_size.restype = SZ
    lib.maxsim_score_streamed_workspace_size.argtypes = [I32, I32, I32, I32, I32, I64]
    lib.maxsim_score_streamed.restype = I32
    lib.maxsim_score_streamed.argtypes = [P, I32, I32, I32, P, I64, I32, P, I32, P, P, P, SZ, I64, P]
    lib.maxsim_score_pq_workspace_size.restype = SZ
    lib.maxsim_score_pq_workspace_size.argtypes = [I32, I32, I32]
    lib.maxsim_score_pq.restype = I32
    lib.maxsim_score_pq.argtypes = [P, I32, I32, P, I32, I32, P, P, I64, I64, P, P, P, SZ, P]
    lib.maxsim_score_pq_noalloc.restype = I32
    lib.maxsim_score_pq_noalloc.argtypes = [P, I32, I32, P, I32, I32, P, P, I64, I64, P, P, P]
    lib.maxsim_score_i8.restype = I32
    lib.maxsim_score_i8.argtypes = [P, P, I32, I32, P, P, P, I64, I64, P, P, P, P, P]
    lib.maxsim_backward_workspace_size.restype = SZ
    lib.maxsim_backward_workspace_size.argtypes = [I32, I32, I32, I64, I32]
    lib.maxsim_backward.restype = I32
    lib.maxsim_backward.argtypes = [P, I32, I32, I32, P, I64, I32, P, I32, P, P, P, P, P, SZ, P]
    lib.maxsim_backward_dq.restype = I32
    lib.maxsim_backward_dq.argtypes = [I32, I32, I32, P, I64, I32, P, I32, P, P, P, P, SZ, P]
    lib.maxsim_backward_dd.restype = I32
    lib.maxsim_backward_dd.argtypes = [P, I32, I32, I32, I64, I32, P, I32, P, P, P, P]
    HP, SP, F32 = ctypes.POINTER(_Heads), ctypes.POINTER(_AttentionSpec), ctypes.c_float
    lib.maxsim_rotary_frequencies.restype = I32
    lib.maxsim_rotary_frequencies.argtypes = [I32, ctypes.c_double, I32, ctypes.c_double, I64, P, ctypes.POINTER(F32)]
    lib.maxsim_rotary.restype = I32
    lib.maxsim_rotary.argtypes = [HP, I64, I32, I32, I32, P, P, I64, P, I32, F32, I32, I32, HP, P]
    lib.maxsim_attention.restype = I32
    lib.maxsim_attention.argtypes = [SP, HP, HP, HP, HP, P, P]
    lib.maxsim_attention_backward_workspace_size.restype = SZ
    lib.maxsim_attention_backward_workspace_size.argtypes = [SP]
    lib.maxsim_attention_backward.restype = I32
    lib.maxsim_attention_backward.argtypes = [SP, HP, HP, HP, HP, HP, P, HP, HP, HP, P, SZ, P]
    lib.maxsim_clip_grad_norm_workspace_size.restype = SZ
    lib.maxsim_clip_grad_norm_workspace_size.argtypes = [I32]
    lib.maxsim_clip_grad_norm.restype = I32
    lib.maxsim_clip_grad_norm.argtypes = [P, P, P, P, I32, F32, P, P, SZ, P]
    RP, NP, LP = ctypes.POINTER(_Rows), ctypes.POINTER(_NormSpec), ctypes.POINTER(_LossSpec)
    lib.maxsim_dropout.restype = I32
    lib.maxsim_dropout.argtypes = [RP, RP, I64, I32, F32, P, I32, RP, P]
    lib.maxsim_rms_norm.restype = I32
    lib.maxsim_rms_norm.argtypes = [NP, RP, RP, RP, RP, P, P]
    lib.maxsim_rms_norm_backward_workspace_size.restype = SZ
    lib.maxsim_rms_norm_backward_workspace_size.argtypes = [NP]
    lib.maxsim_rms_norm_backward.restype = I32
    lib.maxsim_rms_norm_backward.argtypes = [NP, RP, RP, RP, RP, RP, P, P, SZ, P]
    lib.maxsim_cross_entropy_workspace_size.restype = SZ
    lib.maxsim_cross_entropy_workspace_size.argtypes = [LP]
    lib.maxsim_cross_entropy.restype = I32
    lib.maxsim_cross_entropy.argtypes = [LP, RP, RP, P, P, P, SZ, P]
    lib.maxsim_cross_entropy_backward_workspace_size.restype = SZ
    lib.maxsim_cross_entropy_backward_workspace_size.argtypes = [LP]
    lib.maxsim_cross_entropy_backward.restype = I32
    lib.maxsim_cross_entropy_backward.argtypes = [LP, P, RP, RP, P, RP, RP, P, SZ, P]
    _lib = lib
    return lib


# ----------------------------------------------------------------- helpers

def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


# The current stream's handle without a Stream object around it, where torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_on(stream, index):
    """Handle of ``stream``, or of the current stream of device ``index``."""
    if stream is None and _raw_stream is not None:
        return _raw_stream(index)
    return (torch.cuda.current_stream(index) if stream is None else stream).cuda_stream


_devices = None                               # CUDA devices of this process, once asked for
_STAY = contextlib.nullcontext(lambda t: t)   # the current device and stream are the call's


def _several():
    global _devices
    if _devices is None:
        _devices = torch.cuda.device_count()
    return _devices > 1


@contextlib.contextmanager
def _moved(index, stream):
    if stream is None:
        with torch.cuda.device(index):
            yield lambda t: t
    else:
        if stream.device.index != index:
            raise ValueError("stream must be one of the tensors' device")
        outer = torch.cuda.current_stream(index)
        with torch.cuda.stream(stream):
            yield lambda t: t.record_stream(outer)


def _on(index, stream):
    """Makes device ``index`` current for a call, and ``stream`` if one is
    given. The library launches on the current device, where handle 0 is the
    default stream of whichever that is. Memory that the call makes then comes
    from its stream's pool: that of another may have been given up by work that
    has yet to run there, and nothing would order that work and the call's.
    Gives a function that keeps a result's memory from reuse until the caller's
    stream is done with it."""
    if stream is None and (not _several() or index == torch.cuda.current_device()):
        return _STAY
    return _moved(index, stream)


def _elsewhere(fn, names, values):
    """Calls an entry point with its tensors' device and its stream current."""
    index, first = None, None
    for name, t in zip(names, values):
        if isinstance(t, torch.Tensor) and t.is_cuda:
            if index is None:
                index, first = t.get_device(), name
            elif t.get_device() != index:
                raise ValueError(f"{name} must be on the same device as {first}")
    if index is None:
        return fn(*values)  # whose checks say what is wrong
    with _on(index, values[names.index("stream")]) as keep:
        result = fn(*values)
        for t in result if isinstance(result, tuple) else (result,):
            keep(t)
        return result


def _entry(fn):
    """An entry point with a ``stream`` parameter: the call's tensors are on one
    device, which is current for it, and with a stream given its workspace and
    results are made there, too. The common call, on the one device's current
    stream, only passes through a function with fn's own parameters (packing
    and unpacking them cost up to a microsecond)."""
    params = inspect.signature(fn).parameters
    names = tuple(params)
    scope = {"fn": fn, "names": names, "several": _several, "elsewhere": _elsewhere}
    exec(f"def call({', '.join(n if p.default is p.empty else n + '=None' for n, p in params.items())}):\n"
         f"    if stream is None and not several():\n"
         f"        return fn({', '.join(names)})\n"
         f"    return elsewhere(fn, names, ({', '.join(names)},))\n", scope)
    call = functools.wraps(fn)(scope["call"])
    call.__defaults__ = fn.__defaults__
    return call


def _dev(t, name, dtype=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t


def _check(status, what):
    if status != 0:
        raise MaxSimError(status, what)


def maxsim_version() -> int:
    return load_library().maxsim_version()


def maxsim_device_status(stream=None):
    """Synchronise ``stream`` and return (status, flags) of the device status word."""
    flags = ctypes.c_uint(0)
    st = load_library().maxsim_device_status(_stream(stream), ctypes.byref(flags))
    return st, flags.value


# ------------------------------------------------------------- entry points
#
# All CUDA tensors of a call are on one device, which need not be the current
# one. ``stream=None`` is that device's current stream. With a stream given, the call runs on
# it, and so does everything that makes its workspace and results; tensors that
# the caller gives are ordered with that stream by the caller, and the results
# are read elsewhere once that stream has been waited for.

@_entry
def maxsim_score(Q, D, doc_len=None, out=None, argmax_out=None, want_argmax=False, stream=None):
    """Padded layout. Q [nq,d] or [n_queries,nq,d]; D [B,Nd,d] (bf16/fp16/fp32);
    doc_len [B] int32 or None. Returns out [n_queries,B] fp32 (and argmax
    [n_queries,B,nq] int32 when requested)."""
    lib = load_library()
    _dev(Q, "Q")
    _dev(D, "D", Q.dtype)
    Q3 = Q if Q.dim() == 3 else Q.unsqueeze(0)
    nQ, nq, d = Q3.shape
    B, nd, d2 = D.shape
    if d2 != d:
        raise ValueError("Q and D disagree on d")
    if doc_len is not None:
        _dev(doc_len, "doc_len", torch.int32)
    if out is None:
        out = torch.empty((nQ, B), dtype=torch.float32, device=Q.device)
    _dev(out, "out", torch.float32)
    if want_argmax and argmax_out is None:
        argmax_out = torch.empty((nQ, B, nq), dtype=torch.int32, device=Q.device)
    if argmax_out is not None:
        _dev(argmax_out, "argmax_out", torch.int32)
    st = lib.maxsim_score(_ptr(Q3), nQ, nq, d, _ptr(D), B, nd, _ptr(doc_len), _DTYPE_CODE[Q.dtype],
                          _ptr(out), _ptr(argmax_out), _stream(stream))
    _check(st, "maxsim_score")
    return (out, argmax_out) if argmax_out is not None else out


def maxsim_length_order_workspace_size(B, nd, csr=False):
    """Device bytes of the workspace of maxsim_length_order (no GPU needed)."""
    return int(load_library().maxsim_length_order_workspace_size(B, nd, 1 if csr else 0))


@_entry
def maxsim_length_order(doc_len=None, offsets=None, B=None, nd=None, order=None, stream=None):
    """Length-bucketed document order: int32 [B] permutation sorting documents
    by ceil(L_b / 8), ascending and stable. Give doc_len [B] int32 with nd
    (padded layout) or offsets [B+1] int64 (CSR)."""
    lib = load_library()
    if (doc_len is None) == (offsets is None):
        raise ValueError("give exactly one of doc_len and offsets")
    ref = doc_len if doc_len is not None else offsets
    if doc_len is not None:
        _dev(doc_len, "doc_len", torch.int32)
        B = doc_len.numel()
        if nd is None:
            raise ValueError("nd is required with doc_len")
    else:
        _dev(offsets, "offsets", torch.int64)
        B = offsets.numel() - 1
        nd = 0
    if order is None:
        order = torch.empty(B, dtype=torch.int32, device=ref.device)
    _dev(order, "order", torch.int32)
    nb = lib.maxsim_length_order_workspace_size(B, nd, 0 if doc_len is not None else 1)
    ws = torch.empty(max(nb, 16), dtype=torch.uint8, device=ref.device)
    st = lib.maxsim_length_order(_ptr(doc_len), _ptr(offsets), B, nd, _ptr(order), _ptr(ws), ws.numel(),
                                 _stream(stream))
    _check(st, "maxsim_length_order")
    return order


@_entry
def maxsim_score_ordered(Q, D, doc_order, doc_len=None, out=None, argmax_out=None, want_argmax=False, stream=None):
    """maxsim_score with the documents walked in doc_order (int32 [B]
    permutation); results land at the documents' own indices."""
    lib = load_library()
    _dev(Q, "Q")
    _dev(D, "D", Q.dtype)
    _dev(doc_order, "doc_order", torch.int32)
    Q3 = Q if Q.dim() == 3 else Q.unsqueeze(0)
    nQ, nq, d = Q3.shape
    B, nd, d2 = D.shape
    if d2 != d or doc_order.numel() != B:
        raise ValueError("Q, D and doc_order disagree")
    if doc_len is not None:
        _dev(doc_len, "doc_len", torch.int32)
    if out is None:
        out = torch.empty((nQ, B), dtype=torch.float32, device=Q.device)
    _dev(out, "out", torch.float32)
    if want_argmax and argmax_out is None:
        argmax_out = torch.empty((nQ, B, nq), dtype=torch.int32, device=Q.device)
    if argmax_out is not None:
        _dev(argmax_out, "argmax_out", torch.int32)
    st = lib.maxsim_score_ordered(_ptr(Q3), nQ, nq, d, _ptr(D), B, nd, _ptr(doc_len), _ptr(doc_order),
                                  _DTYPE_CODE[Q.dtype], _ptr(out), _ptr(argmax_out), _stream(stream))
    _check(st, "maxsim_score_ordered")
    return (out, argmax_out) if argmax_out is not None else out


def maxsim_score_streamed_workspace_size(n_queries, nq, nd, d, dtype, chunk_docs):
    """Device bytes of the workspace of maxsim_score_streamed (no GPU needed)."""
    return load_library().maxsim_score_streamed_workspace_size(n_queries, nq, nd, d, _DTYPE_CODE[dtype], chunk_docs)


@_entry
def maxsim_score_streamed(Q, D_host, doc_len_host=None, chunk_docs=16384, out=None, argmax_out=None,
                          want_argmax=False, workspace=None, stream=None):
    """Padded layout with the documents in HOST memory: D_host [B,Nd,d] and
    doc_len_host [B] int32 (or None) are CPU tensors (page-locked, e.g.
    ``pin_memory()``, for copies that overlap scoring); Q is on the GPU.
    Chunks of ``chunk_docs`` documents are copied and scored in turn. Returns
    out [n_queries,B] fp32 (and argmax [n_queries,B,nq] int32 when requested).
    The host tensors must stay alive until the stream has completed."""
    lib = load_library()
    _dev(Q, "Q")
    if not isinstance(D_host, torch.Tensor) or D_host.is_cuda or not D_host.is_contiguous() or D_host.dtype != Q.dtype:
        raise ValueError("D_host must be a contiguous CPU tensor of Q's dtype")
    Q3 = Q if Q.dim() == 3 else Q.unsqueeze(0)
    nQ, nq, d = Q3.shape
    B, nd, d2 = D_host.shape
    if d2 != d:
        raise ValueError("Q and D_host disagree on d")
    if doc_len_host is not None and (doc_len_host.is_cuda or doc_len_host.dtype != torch.int32
                                     or not doc_len_host.is_contiguous()):
        raise ValueError("doc_len_host must be a contiguous CPU int32 tensor")
    if out is None:
        out = torch.empty((nQ, B), dtype=torch.float32, device=Q.device)
    _dev(out, "out", torch.float32)
    if want_argmax and argmax_out is None:
        argmax_out = torch.empty((nQ, B, nq), dtype=torch.int32, device=Q.device)
    if argmax_out is not None:
        _dev(argmax_out, "argmax_out", torch.int32)
    nbytes = lib.maxsim_score_streamed_workspace_size(nQ, nq, nd, d, _DTYPE_CODE[Q.dtype], chunk_docs)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=Q.device)
    _dev(workspace, "workspace", torch.uint8)
    st = lib.maxsim_score_streamed(_ptr(Q3), nQ, nq, d, ctypes.c_void_p(D_host.data_ptr()), B, nd,
                                   None if doc_len_host is None else ctypes.c_void_p(doc_len_host.data_ptr()),
                                   _DTYPE_CODE[Q.dtype], _ptr(out), _ptr(argmax_out), _ptr(workspace),
                                   workspace.numel(), chunk_docs, _stream(stream))
    _check(st, "maxsim_score_streamed")
    return (out, argmax_out) if argmax_out is not None else out


@_entry
def maxsim_score_varlen(Q, D_packed, offsets, out=None, argmax_out=None, want_argmax=False, stream=None):
    """CSR layout: document b owns rows offsets[b]..offsets[b+1]-1 of D_packed [T,d]."""
    lib = load_library()
    _dev(Q, "Q")
    _dev(D_packed, "D_packed", Q.dtype)
    _dev(offsets, "offsets", torch.int64)
    Q3 = Q if Q.dim() == 3 else Q.unsqueeze(0)
    nQ, nq, d = Q3.shape
    T, d2 = D_packed.shape
    if d2 != d:
        raise ValueError("Q and D_packed disagree on d")
    B = offsets.numel() - 1
    if out is None:
        out = torch.empty((nQ, B), dtype=torch.float32, device=Q.device)
    if want_argmax and argmax_out is None:
        argmax_out = torch.empty((nQ, B, nq), dtype=torch.int32, device=Q.device)
    st = lib.maxsim_score_varlen(_ptr(Q3), nQ, nq, d, _ptr(D_packed), _ptr(offsets), B, T,
                                 _DTYPE_CODE[Q.dtype], _ptr(out), _ptr(argmax_out), _stream(stream))
    _check(st, "maxsim_score_varlen")
    return (out, argmax_out) if argmax_out is not None else out


def maxsim_score_pq_workspace_size(nq: int, M: int, K: int) -> int:
    return int(load_library().maxsim_score_pq_workspace_size(nq, M, K))


@_entry
def maxsim_score_pq(Q, codebooks, codes, offsets, out=None, argmax_out=None, want_argmax=False,
                    workspace=None, stream=None):
    """PQ scoring: Q [nq,d] fp32, codebooks [M,K,d/M] fp32, codes [T,M] uint8, CSR offsets."""
    lib = load_library()
    _dev(Q, "Q", torch.float32)
    _dev(codebooks, "codebooks", torch.float32)
    _dev(codes, "codes", torch.uint8)
    _dev(offsets, "offsets", torch.int64)
    nq, d = Q.shape
    M, K, _ = codebooks.shape
    T = codes.shape[0]
    B = offsets.numel() - 1
    ws = maxsim_score_pq_workspace_size(nq, M, K)
    if workspace is None:
        workspace = torch.empty(max(ws, 1), dtype=torch.uint8, device=Q.device)
    if out is None:
        out = torch.empty(B, dtype=torch.float32, device=Q.device)
    if want_argmax and argmax_out is None:
        argmax_out = torch.empty((B, nq), dtype=torch.int32, device=Q.device)
    st = lib.maxsim_score_pq(_ptr(Q), nq, d, _ptr(codebooks), M, K, _ptr(codes), _ptr(offsets), B, T,
                             _ptr(out), _ptr(argmax_out), _ptr(workspace), workspace.numel(),
                             _stream(stream))
    _check(st, "maxsim_score_pq")
    return (out, argmax_out) if argmax_out is not None else out


@_entry
def maxsim_score_pq_noalloc(Q, codebooks, codes, offsets, out=None, argmax_out=None, want_argmax=False,
                            stream=None):
    """PQ scoring with the table kept in the library's fixed device array, for
    callers that cannot allocate device memory themselves (see the header)."""
    lib = load_library()
    _dev(Q, "Q", torch.float32)
    _dev(codebooks, "codebooks", torch.float32)
    _dev(codes, "codes", torch.uint8)
    _dev(offsets, "offsets", torch.int64)
    nq, d = Q.shape
    M, K, _ = codebooks.shape
    T = codes.shape[0]
    B = offsets.numel() - 1
    if out is None:
        out = torch.empty(B, dtype=torch.float32, device=Q.device)
    if want_argmax and argmax_out is None:
        argmax_out = torch.empty((B, nq), dtype=torch.int32, device=Q.device)
    st = lib.maxsim_score_pq_noalloc(_ptr(Q), nq, d, _ptr(codebooks), M, K, _ptr(codes), _ptr(offsets), B, T,
                                     _ptr(out), _ptr(argmax_out), _stream(stream))
    _check(st, "maxsim_score_pq_noalloc")
    return (out, argmax_out) if argmax_out is not None else out


@_entry
def maxsim_score_i8(Q, q_scale, D, d_scale, offsets, out=None, maxv_out=None, maxdot_out=None,
                    argmax_out=None, want_details=False, stream=None):
    """INT8 x INT8 scoring with per-token fp32 scales; CSR documents."""
    lib = load_library()
    _dev(Q, "Q", torch.int8)
    _dev(q_scale, "q_scale", torch.float32)
    _dev(D, "D", torch.int8)
    _dev(d_scale, "d_scale", torch.float32)
    _dev(offsets, "offsets", torch.int64)
    nq, d = Q.shape
    T = D.shape[0]
    B = offsets.numel() - 1
    if out is None:
        out = torch.empty(B, dtype=torch.float32, device=Q.device)
    if want_details:
        if maxv_out is None:
            maxv_out = torch.empty((B, nq), dtype=torch.float32, device=Q.device)
        if maxdot_out is None:
            maxdot_out = torch.empty((B, nq), dtype=torch.int32, device=Q.device)
        if argmax_out is None:
            argmax_out = torch.empty((B, nq), dtype=torch.int32, device=Q.device)
    st = lib.maxsim_score_i8(_ptr(Q), _ptr(q_scale), nq, d, _ptr(D), _ptr(d_scale), _ptr(offsets), B, T,
                             _ptr(out), _ptr(maxv_out), _ptr(maxdot_out), _ptr(argmax_out), _stream(stream))
    _check(st, "maxsim_score_i8")
    if want_details:
        return out, maxv_out, maxdot_out, argmax_out
    return out


def maxsim_backward_workspace_size(n_queries, nq, d, B, nd) -> int:
    return int(load_library().maxsim_backward_workspace_size(n_queries, nq, d, B, nd))


@_entry
def maxsim_backward(Q, D, argmax, dS, doc_len=None, dQ=None, dD=None, workspace=None, stream=None):
    """Gradients of sum dS*score through the saved forward argmax (padded layout)."""
    lib = load_library()
    _dev(Q, "Q")
    _dev(D, "D", Q.dtype)
    _dev(argmax, "argmax", torch.int32)
    _dev(dS, "dS", torch.float32)
    Q3 = Q if Q.dim() == 3 else Q.unsqueeze(0)
    nQ, nq, d = Q3.shape
    B, nd, _ = D.shape
    if doc_len is not None:
        _dev(doc_len, "doc_len", torch.int32)
    if dQ is None:
        dQ = torch.empty((nQ, nq, d), dtype=torch.float32, device=Q.device)
    if dD is None:
        dD = torch.empty((B, nd, d), dtype=torch.float32, device=Q.device)
    ws = maxsim_backward_workspace_size(nQ, nq, d, B, nd)
    if workspace is None and ws > 0:
        workspace = torch.empty(ws, dtype=torch.uint8, device=Q.device)
    st = lib.maxsim_backward(_ptr(Q3), nQ, nq, d, _ptr(D), B, nd, _ptr(doc_len), _DTYPE_CODE[Q.dtype],
                             _ptr(argmax), _ptr(dS), _ptr(dQ), _ptr(dD), _ptr(workspace),
                             0 if workspace is None else workspace.numel(), _stream(stream))
    _check(st, "maxsim_backward")
    return dQ.view(Q.shape) if Q.dim() == 2 else dQ, dD


@_entry
def maxsim_backward_dq(D, argmax, dS, nq=None, doc_len=None, dQ=None, workspace=None, stream=None):
    """dQ only (frozen document side). D [B,Nd,d]; argmax [n_queries,B,nq]
    int32; dS [n_queries,B] fp32. Returns dQ [n_queries,nq,d] fp32."""
    lib = load_library()
    _dev(D, "D")
    _dev(argmax, "argmax", torch.int32)
    _dev(dS, "dS", torch.float32)
    nQ, B2, nq_a = argmax.shape
    B, nd, d = D.shape
    if B2 != B or dS.shape != (nQ, B):
        raise ValueError("argmax / dS shapes do not match D")
    if doc_len is not None:
        _dev(doc_len, "doc_len", torch.int32)
    if dQ is None:
        dQ = torch.empty((nQ, nq_a, d), dtype=torch.float32, device=D.device)
    _dev(dQ, "dQ", torch.float32)
    ws = maxsim_backward_workspace_size(nQ, nq_a, d, B, nd)
    if workspace is None and ws > 0:
        workspace = torch.empty(ws, dtype=torch.uint8, device=D.device)
    st = lib.maxsim_backward_dq(nQ, nq_a, d, _ptr(D), B, nd, _ptr(doc_len), _DTYPE_CODE[D.dtype], _ptr(argmax),
                                _ptr(dS), _ptr(dQ), _ptr(workspace), 0 if workspace is None else workspace.numel(),
                                _stream(stream))
    _check(st, "maxsim_backward_dq")
    return dQ


@_entry
def maxsim_backward_dd(Q, argmax, dS, nd, doc_len=None, dD=None, stream=None):
    """dD only (frozen query side). Q [nq,d] or [n_queries,nq,d]; argmax
    [n_queries,B,nq] int32; dS [n_queries,B] fp32. Returns dD [B,nd,d] fp32."""
    lib = load_library()
    _dev(Q, "Q")
    _dev(argmax, "argmax", torch.int32)
    _dev(dS, "dS", torch.float32)
    Q3 = Q if Q.dim() == 3 else Q.unsqueeze(0)
    nQ, nq, d = Q3.shape
    B = argmax.shape[1]
    if argmax.shape != (nQ, B, nq) or dS.shape != (nQ, B):
        raise ValueError("argmax / dS shapes do not match Q")
    if doc_len is not None:
        _dev(doc_len, "doc_len", torch.int32)
    if dD is None:
        dD = torch.empty((B, nd, d), dtype=torch.float32, device=Q.device)
    _dev(dD, "dD", torch.float32)
    st = lib.maxsim_backward_dd(_ptr(Q3), nQ, nq, d, B, nd, _ptr(doc_len), _DTYPE_CODE[Q.dtype], _ptr(argmax),
                                _ptr(dS), _ptr(dD), _stream(stream))
    _check(st, "maxsim_backward_dd")
    return dD


# ------------------------------------------------------------ sharded backward

def allreduce_dq(dQ, group=None):
    """Document-sharded training: every rank runs maxsim_backward on its own
    documents, so its dQ holds only those documents' terms of
    dQ[q,i,:] = sum_b dS[q,b] * D[b, argmax[q,b,i], :]; the sum over ranks is
    the full gradient. One in-place all-reduce (sum) over ``group`` (NCCL for
    CUDA tensors, gloo on CPU); dD rows belong to one rank's documents and
    need no exchange (FLASH-MAXSIM, Abstract: destination-owned reduction).
    A no-op without an initialised process group or with one rank."""
    import torch.distributed as dist
    if not (dist.is_available() and dist.is_initialized()) or dist.get_world_size(group) == 1:
        return dQ
    dist.all_reduce(dQ, op=dist.ReduceOp.SUM, group=group)
    return dQ


# --------------------------------------------------------- the token encoder

def _scratch(nbytes, device):
    """A workspace of the call's own."""
    return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=device)


def _heads(t, name, shape, dtype, index):
    """A [T, heads, d] tensor on CUDA device ``index``, its last dimension
    contiguous, as a maxsim_heads."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.get_device() != index or index < 0:
        raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path) on the first tensor's device")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    token, head, last = t.stride()
    if last != 1 and shape[2] != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    if shape[1] == 1:  # the stride of a dimension of one element says nothing
        head = shape[2]
    if shape[0] == 1:
        token = shape[1] * max(head, shape[2])
    return _Heads(t.data_ptr(), token, head)


def maxsim_rotary_frequencies(rot_dim, base=10000.0, scaling="none", factor=1.0, original_length=0, device="cuda"):
    """Frequency table of maxsim_rotary: (freq [rot_dim/2] int64 on ``device``,
    amplitude). freq is in turns per position times 2^64. ``scaling``: "none",
    "linear", "ntk" or "yarn" (which needs the ``original_length``), by ``factor``."""
    lib = load_library()
    if scaling not in ROTARY_SCALING:
        raise ValueError(f"scaling must be one of {tuple(ROTARY_SCALING)}")
    freq = torch.empty(max(rot_dim // 2, 1), dtype=torch.int64)
    amplitude = ctypes.c_float(0.0)
    st = lib.maxsim_rotary_frequencies(rot_dim, base, ROTARY_SCALING[scaling], factor, original_length, _ptr(freq),
                                       ctypes.byref(amplitude))
    _check(st, "maxsim_rotary_frequencies")
    return freq.to(device), amplitude.value


@_entry
def maxsim_rotary(x, freq, offsets=None, positions=None, interleaved=False, amplitude=1.0, inverse=False, out=None,
                  stream=None):
    """Rotary positions: turns the first 2 * len(freq) dimensions of every head
    of x [T, heads, d] (bf16/fp16/fp32; token and head strides may be any).
    Positions count within the documents of ``offsets`` [B+1] int64, or are
    ``positions`` [T] int32, or the token's index. ``inverse=True`` gives the
    gradient. ``out`` may be x itself; a new tensor is made without it."""
    lib = load_library()
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError("x must be a [T, heads, d] tensor")
    if x.dtype not in _DTYPE_CODE:
        raise TypeError(f"x must be bf16, fp16 or fp32, got {x.dtype}")
    shape, dtype, index = x.shape, x.dtype, x.get_device()
    src = _heads(x, "x", shape, dtype, index)
    _dev(freq, "freq", torch.int64)
    T, heads, d = shape
    B = 0
    if offsets is not None:
        B = _dev(offsets, "offsets", torch.int64).numel() - 1
    if positions is not None and _dev(positions, "positions", torch.int32).numel() != T:
        raise ValueError("positions must have one entry a token")
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=x.device)
    dst = src if out is x else _heads(out, "out", shape, dtype, index)
    st = lib.maxsim_rotary(src, T, heads, d, 2 * freq.numel(), freq.data_ptr(), _ptr(offsets), B, _ptr(positions),
                           1 if interleaved else 0, amplitude, 1 if inverse else 0, _DTYPE_CODE[dtype], dst,
                           _stream_on(stream, index))
    _check(st, "maxsim_rotary")
    return out


def _attention_spec(q, k, offsets, key_len, mask, prefix_len, scale, cap, slopes):
    if not isinstance(q, torch.Tensor) or not isinstance(k, torch.Tensor) or q.dim() != 3 or k.dim() != 3:
        raise ValueError("q and k must be [T, heads, d] tensors")
    if q.dtype not in _DTYPE_CODE:
        raise TypeError(f"q must be bf16 or fp16, got {q.dtype}")
    if mask not in MASKS:
        raise ValueError(f"mask must be one of {tuple(MASKS)}")
    T, heads, d = q.shape
    B = _dev(offsets, "offsets", torch.int64).numel() - 1
    if B < 0:
        raise ValueError("offsets must have at least one entry")
    if key_len is not None and _dev(key_len, "key_len", torch.int32).numel() != B:
        raise ValueError("key_len must have one entry a document")
    if (mask == "prefix") != (prefix_len is not None):
        raise ValueError('prefix_len goes with mask="prefix"')
    if prefix_len is not None and _dev(prefix_len, "prefix_len", torch.int32).numel() != B:
        raise ValueError("prefix_len must have one entry a document")
    if slopes is not None and _dev(slopes, "slopes", torch.float32).numel() != heads:
        raise ValueError("slopes must have one entry a head")
    return _AttentionSpec(T, B, heads, k.shape[1], d, _DTYPE_CODE[q.dtype], MASKS[mask],
                          1.0 / math.sqrt(d) if scale is None else scale, cap, offsets.data_ptr(),
                          None if key_len is None else key_len.data_ptr(),
                          None if prefix_len is None else prefix_len.data_ptr(),
                          None if slopes is None else slopes.data_ptr())


@_entry
def maxsim_attention(q, k, v, offsets, key_len=None, mask="full", prefix_len=None, scale=None, cap=0.0, slopes=None,
                     out=None, lse=None, want_lse=False, stream=None):
    """Softmax attention within each CSR-packed document. q [T, heads, d], k and
    v [T, kv_heads, d] (bf16/fp16; views of one projection's output are fine);
    offsets [B+1] int64; key_len [B] int32 hides the keys from there on (None:
    none); mask "full", "causal" or "prefix" (with prefix_len [B] int32); scale
    None: 1/sqrt(d); cap > 0: scores become cap * tanh(score / cap); slopes
    [heads] fp32: minus slope * distance. Returns out [T, heads, d], and lse
    [heads, T] fp32 when requested."""
    lib = load_library()
    spec = _attention_spec(q, k, offsets, key_len, mask, prefix_len, scale, cap, slopes)
    dtype, index, shape = q.dtype, q.get_device(), q.shape
    kv_shape = (shape[0], spec.kv_heads, shape[2])
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=q.device)
    if lse is None and want_lse:
        lse = torch.empty((shape[1], shape[0]), dtype=torch.float32, device=q.device)
    if lse is not None and _dev(lse, "lse", torch.float32).shape != (shape[1], shape[0]):
        raise ValueError("lse must be [heads, T]")
    st = lib.maxsim_attention(spec, _heads(q, "q", shape, dtype, index), _heads(k, "k", kv_shape, dtype, index),
                              _heads(v, "v", kv_shape, dtype, index), _heads(out, "out", shape, dtype, index),
                              None if lse is None else lse.data_ptr(), _stream_on(stream, index))
    _check(st, "maxsim_attention")
    return (out, lse) if lse is not None else out


def maxsim_attention_backward_workspace_size(q, k, offsets, mask="full", prefix_len=None):
    """Device bytes of the workspace of maxsim_attention_backward."""
    spec = _attention_spec(q, k, offsets, None, mask, prefix_len, None, 0.0, None)
    return int(load_library().maxsim_attention_backward_workspace_size(spec))


@_entry
def maxsim_attention_backward(dO, q, k, v, out, lse, offsets, key_len=None, mask="full", prefix_len=None, scale=None,
                              cap=0.0, slopes=None, dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Gradients of maxsim_attention for the gradient dO of its out, from its
    out and lse; the other arguments as in that call. Returns dq, dk, dv in the
    inputs' dtype (views of one buffer may be given)."""
    lib = load_library()
    spec = _attention_spec(q, k, offsets, key_len, mask, prefix_len, scale, cap, slopes)
    dtype, device, index, shape = q.dtype, q.device, q.get_device(), q.shape
    kv_shape = (shape[0], spec.kv_heads, shape[2])
    if _dev(lse, "lse", torch.float32).shape != (shape[1], shape[0]):
        raise ValueError("lse must be [heads, T]")
    dq = torch.empty(shape, dtype=dtype, device=device) if dq is None else dq
    dk = torch.empty(kv_shape, dtype=dtype, device=device) if dk is None else dk
    dv = torch.empty(kv_shape, dtype=dtype, device=device) if dv is None else dv
    if workspace is None:
        workspace = _scratch(lib.maxsim_attention_backward_workspace_size(spec), device)
    _dev(workspace, "workspace", torch.uint8)
    views = [_heads(t, name, want, dtype, index)
             for t, name, want in ((dO, "dO", shape), (q, "q", shape), (k, "k", kv_shape), (v, "v", kv_shape),
                                   (out, "out", shape), (dq, "dq", shape), (dk, "dk", kv_shape), (dv, "dv", kv_shape))]
    st = lib.maxsim_attention_backward(spec, *views[:5], lse.data_ptr(), *views[5:], workspace.data_ptr(),
                                       workspace.numel(), _stream_on(stream, index))
    _check(st, "maxsim_attention_backward")
    return dq, dk, dv


def maxsim_clip_grad_norm_workspace_size(n_tensors):
    """Device bytes of the workspace of maxsim_clip_grad_norm (no GPU needed)."""
    return int(load_library().maxsim_clip_grad_norm_workspace_size(n_tensors))


def _sizes(tensors):
    return list(map(torch.Tensor.numel, tensors))


def _dtypes(tensors):
    return list(map(operator.attrgetter("dtype"), tensors))


def maxsim_clip_grad_norm(grads, max_norm, out=None, norm=None, workspace=None, stream=None):
    """Global 2-norm of the tensors ``grads`` (contiguous, bf16/fp16/fp32, types
    may be mixed), which are scaled by min(1, max_norm / (norm + 1e-6)): in
    place, or into the tensors ``out`` of the same sizes and types. Returns the
    norm before clipping, [1] fp32 on the device."""
    lib = load_library()
    grads = list(grads)
    outs = grads if out is None else list(out)
    n = len(grads)
    # one pass in C for each attribute: lists have hundreds of tensors
    sizes, dtypes, sides = _sizes(grads), _dtypes(grads), (grads,) if out is None else (grads, outs)
    if out is not None and (_sizes(outs) != sizes or _dtypes(outs) != dtypes):
        raise ValueError("out must have a tensor of the same size and type for each of grads")
    places = set()
    for side in sides:
        places.update(map(torch.Tensor.get_device, side))
        if not all(map(torch.Tensor.is_contiguous, side)):
            raise ValueError("all tensors must be contiguous")
    if norm is not None:
        places.add(_dev(norm, "norm", torch.float32).get_device())
    if workspace is not None:
        places.add(_dev(workspace, "workspace", torch.uint8).get_device())
    if len(places) > 1 or -1 in places:
        raise ValueError("all tensors must be on one CUDA device (the library has no CPU path)")
    try:
        codes = array.array("i", map(_DTYPE_CODE.__getitem__, dtypes))
    except KeyError as e:
        raise TypeError(f"gradients must be bf16, fp16 or fp32, got {e.args[0]}") from None
    if places:
        index = places.pop()
    else:
        index = torch.cuda.current_device() if stream is None else stream.device.index
    pointers = array.array("Q", map(torch.Tensor.data_ptr, grads))
    targets = pointers if out is None else array.array("Q", map(torch.Tensor.data_ptr, outs))
    counts = array.array("q", sizes)
    with _on(index, stream) as keep:
        device = torch.device("cuda", index)
        if norm is None:
            norm = torch.empty(1, dtype=torch.float32, device=device)
        if workspace is None:
            workspace = _scratch(lib.maxsim_clip_grad_norm_workspace_size(n), device)
        st = lib.maxsim_clip_grad_norm(pointers.buffer_info()[0], targets.buffer_info()[0], counts.buffer_info()[0],
                                       codes.buffer_info()[0], n, max_norm, norm.data_ptr(), workspace.data_ptr(),
                                       workspace.numel(), _stream_on(stream, index))
        keep(norm)
    _check(st, "maxsim_clip_grad_norm")
    return norm


# ------------------------------------------------- rows of hidden states, and the loss
#
# The C entry points are maxsim_dropout, maxsim_rms_norm and maxsim_cross_entropy, with
# their gradients.

# Calls on a few rows take as long as their Python: what was just made is not checked.

def _rows(t, name, shape, dtype, index):
    """A [T, d] tensor on CUDA device ``index``, its rows contiguous, as a maxsim_rows."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.get_device() != index or index < 0:
        raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path) on the first tensor's device")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    row, last = t.stride()
    if last != 1 and shape[1] != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    if shape[0] <= 1 or shape[1] == 0:  # the stride of a dimension of one element says nothing
        row = (shape[1] + 7) // 8 * 8
    return _Rows(t.data_ptr(), row)


def _first_rows(x, name, dtypes, said):
    """The call's first tensor: its shape, type, device and view."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError(f"{name} must be a [T, d] tensor")
    dtype, index = x.dtype, x.get_device()
    if dtype not in dtypes:
        raise TypeError(f"{name} must be {said}, got {dtype}")
    if index < 0:
        raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    shape = x.shape
    if shape[1] > 0x7FFFFFFF:  # the library takes a width in 32 bits, of which ctypes would pass on the lower ones
        raise MaxSimError(2, f"{name} of {shape[1]} columns")
    row, last = x.stride()
    if last != 1 and shape[1] != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    if shape[0] <= 1 or shape[1] == 0:
        row = (shape[1] + 7) // 8 * 8
    return shape, dtype, index, _Rows(x.data_ptr(), row)


def _new_rows(t, d):
    """A tensor of the call's own."""
    return _Rows(t.data_ptr(), d if t.shape[0] > 1 else (d + 7) // 8 * 8)


def _rng(p, rng):
    """The device's pointer to a call's seed and number."""
    if rng is None:
        if p:
            raise ValueError("p > 0 needs rng, an int64 tensor of a seed and a call's number")
        return None
    if _dev(rng, "rng", torch.int64).numel() != 2:
        raise ValueError("rng must have two entries: a seed and a call's number")
    return rng.data_ptr()


@_entry
def encoder_dropout(x, p, rng, residual=None, out=None, stream=None):
    """Dropout of x [T, d] (bf16/fp16/fp32; any row stride), plus ``residual``:
    an element is dropped with chance p (a multiple of 2^-16), others are divided by
    1 - p. The mask is made from ``rng``, [2] int64 on the device (a seed, and a
    number that differs between calls), and an element's row and column, and is
    not stored: the same call on the gradient of the result, without a residual,
    gives that of x. ``out`` may be x or residual."""
    lib = load_library()
    shape, dtype, index, src = _first_rows(x, "x", _DTYPE_CODE, "bf16, fp16 or fp32")
    T, d = shape
    res = None if residual is None else _rows(residual, "residual", shape, dtype, index)
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=x.device)
        dst = _new_rows(out, d)
    else:
        dst = _rows(out, "out", shape, dtype, index)
    st = lib.maxsim_dropout(src, res, T, d, p, _rng(p, rng), _DTYPE_CODE[dtype], dst, _stream_on(stream, index))
    if st:
        _check(st, "maxsim_dropout")
    return out


def _norm_spec(x, name, weight, eps, p, rng, fmt):
    shape, dtype, index, view = _first_rows(x, name, _DTYPE_CODE, "bf16, fp16 or fp32")
    T, d = shape
    code, wptr = FP32, None
    if weight is not None:
        wtype = _dev(weight, "weight").dtype
        if wtype != dtype and wtype != torch.float32:
            raise TypeError(f"weight must be fp32 or {dtype}, got {wtype}")
        if weight.numel() != d:
            raise ValueError("weight must have one entry a column")
        code, wptr = _DTYPE_CODE[wtype], weight.data_ptr()
    if fmt not in NORM_FORMATS:
        raise ValueError(f"fmt must be one of {tuple(NORM_FORMATS)}")
    spec = _NormSpec(T, d, _DTYPE_CODE[dtype], code, NORM_FORMATS[fmt][0], eps, p, _rng(p, rng), wptr)
    return spec, shape, dtype, index, view


@_entry
def encoder_rms_norm(x, weight=None, residual=None, eps=1e-6, p=0.0, rng=None, fmt=None, out=None, sum_out=None,
                     want_sum=False, scale=None, stream=None):
    """Root-mean-square norm of the rows h = residual + dropout(x) (p and rng as in
    encoder_dropout; both parts are optional): y = h * weight / sqrt(mean(h^2) +
    eps). x [T, d] and residual bf16/fp16/fp32 with any row stride; weight [d]
    fp32 or of x's type. ``fmt`` None: y in x's type; "int8" or "e4m3": y / scale in
    8 bits, with scale [T] fp32 (int8 rows and scales are what maxsim_score_i8
    takes). Returns out, then scale with a ``fmt``, then h with ``want_sum`` or
    ``sum_out`` (which may be x or residual): one tensor, or a tuple."""
    lib = load_library()
    spec, shape, dtype, index, src = _norm_spec(x, "x", weight, eps, p, rng, fmt)
    device, d = x.device, shape[1]
    res = None if residual is None else _rows(residual, "residual", shape, dtype, index)
    otype = dtype if fmt is None else NORM_FORMATS[fmt][1]
    if out is None:
        out = torch.empty(shape, dtype=otype, device=device)
        dst = _new_rows(out, d)
    else:
        dst = _rows(out, "out", shape, otype, index)
    total = None
    if sum_out is not None:
        total = _rows(sum_out, "sum_out", shape, dtype, index)
    elif want_sum:
        sum_out = torch.empty(shape, dtype=dtype, device=device)
        total = _new_rows(sum_out, d)
    sptr = None
    if fmt is None:
        if scale is not None:
            raise ValueError("scale goes with an 8-bit fmt")
    else:
        if scale is None:
            scale = torch.empty(shape[0], dtype=torch.float32, device=device)
        elif _dev(scale, "scale", torch.float32).numel() != shape[0]:
            raise ValueError("scale must have one entry a row")
        sptr = scale.data_ptr()
    st = lib.maxsim_rms_norm(spec, src, res, total, dst, sptr, _stream_on(stream, index))
    if st:
        _check(st, "maxsim_rms_norm")
    if fmt is None:
        return out if sum_out is None else (out, sum_out)
    return (out, scale) if sum_out is None else (out, scale, sum_out)


def encoder_rms_norm_backward_workspace_size(h, weight=None):
    """Device bytes of the workspace of encoder_rms_norm_backward."""
    spec = _norm_spec(h, "h", weight, 1e-6, 0.0, None, None)[0]
    return int(load_library().maxsim_rms_norm_backward_workspace_size(spec))


@_entry
def encoder_rms_norm_backward(dy, h, weight=None, dsum=None, eps=1e-6, p=0.0, rng=None, dx=None, dresidual=None,
                              dweight=None, workspace=None, stream=None):
    """Gradients of encoder_rms_norm for the gradient dy of its out, from its sum h
    and the same weight, eps, p and rng; ``dsum`` is the gradient that reaches h
    from elsewhere. Returns dx, dresidual and dweight (None without a weight). Without
    dropout dx and dresidual are one tensor, unless both are given."""
    lib = load_library()
    spec, shape, dtype, index, hv = _norm_spec(h, "h", weight, eps, p, rng, None)
    device, d = h.device, shape[1]

    def result(t, name):
        if t is not None:
            return t, _rows(t, name, shape, dtype, index)
        t = torch.empty(shape, dtype=dtype, device=device)
        return t, _new_rows(t, d)

    dyv = _rows(dy, "dy", shape, dtype, index)
    more = None if dsum is None else _rows(dsum, "dsum", shape, dtype, index)
    second = None
    if not p and (dx is None or dresidual is None):
        dx, first = result(dx if dx is not None else dresidual, "dx")
        dresidual = dx
    else:
        dx, first = result(dx, "dx")
        dresidual, second = result(dresidual, "dresidual")
    if weight is not None:
        if dweight is None:
            dweight = torch.empty(d, dtype=weight.dtype, device=device)
        elif _dev(dweight, "dweight", weight.dtype).numel() != d:
            raise ValueError("dweight must have one entry a column")
        if workspace is None:
            workspace = _scratch(lib.maxsim_rms_norm_backward_workspace_size(spec), device)
        else:
            _dev(workspace, "workspace", torch.uint8)
    elif dweight is not None:
        raise ValueError("dweight goes with a weight")
    elif workspace is not None:
        _dev(workspace, "workspace", torch.uint8)
    st = lib.maxsim_rms_norm_backward(spec, dyv, hv, more, first, second,
                                      None if dweight is None else dweight.data_ptr(),
                                      None if workspace is None else workspace.data_ptr(),
                                      0 if workspace is None else workspace.numel(), _stream_on(stream, index))
    if st:
        _check(st, "maxsim_rms_norm_backward")
    return dx, dresidual, dweight


_LOSS_TYPES = {torch.bfloat16: BF16, torch.float16: FP16}


def _loss_spec(x, weight, targets, scale):
    shape, dtype, index, view = _first_rows(x, "x", _LOSS_TYPES, "bf16 or fp16")
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2 or weight.shape[1] != shape[1]:
        raise ValueError("weight must be [V, d], with x's d")
    if _dev(targets, "targets", torch.int64).numel() != shape[0]:
        raise ValueError("targets must have one entry a row")
    spec = _LossSpec(shape[0], weight.shape[0], shape[1], _LOSS_TYPES[dtype], scale, targets.data_ptr())
    return spec, view, _rows(weight, "weight", weight.shape, dtype, index), index


def encoder_cross_entropy_workspace_size(x, weight, targets):
    """Device bytes of the workspace of encoder_cross_entropy."""
    return int(load_library().maxsim_cross_entropy_workspace_size(_loss_spec(x, weight, targets, 1.0)[0]))


def encoder_cross_entropy_backward_workspace_size(x, weight, targets):
    """Device bytes of the workspace of encoder_cross_entropy_backward."""
    return int(load_library().maxsim_cross_entropy_backward_workspace_size(_loss_spec(x, weight, targets, 1.0)[0]))


def _row_values(t, name, n):
    if _dev(t, name, torch.float32).numel() != n:
        raise ValueError(f"{name} must have one entry a row")
    return t


@_entry
def encoder_cross_entropy(x, weight, targets, scale=1.0, loss=None, lse=None, workspace=None, stream=None):
    """Softmax cross entropy of the logits scale * x @ weight.T, which are never
    stored: x [T, d], weight [V, d] (bf16/fp16; d a multiple of 8), targets [T]
    int64, negative where a row has none. Returns loss [T] fp32 (0 without a
    target) and lse [T] fp32, the logarithms of the softmax's denominators, which
    the backward needs."""
    lib = load_library()
    spec, xv, wv, index = _loss_spec(x, weight, targets, scale)
    n, device = spec.T, x.device
    loss = torch.empty(n, dtype=torch.float32, device=device) if loss is None else _row_values(loss, "loss", n)
    lse = torch.empty(n, dtype=torch.float32, device=device) if lse is None else _row_values(lse, "lse", n)
    if workspace is None:
        workspace = _scratch(lib.maxsim_cross_entropy_workspace_size(spec), device)
    else:
        _dev(workspace, "workspace", torch.uint8)
    st = lib.maxsim_cross_entropy(spec, xv, wv, loss.data_ptr(), lse.data_ptr(), workspace.data_ptr(),
                                  workspace.numel(), _stream_on(stream, index))
    if st:
        _check(st, "maxsim_cross_entropy")
    return loss, lse


@_entry
def encoder_cross_entropy_backward(dloss, x, weight, targets, lse, scale=1.0, dx=None, dweight=None, want_dx=True,
                                   want_dweight=True, workspace=None, stream=None):
    """Gradients of encoder_cross_entropy for the gradient dloss [T] fp32 of its
    loss, from its lse; the other arguments as in that call. Returns dx [T, d]
    and dweight [V, d] in the inputs' type; a side that is not wanted, nor given, is
    None, and its product is not made (the workspace has room for both all the same)."""
    lib = load_library()
    spec, xv, wv, index = _loss_spec(x, weight, targets, scale)
    n, dtype, device = spec.T, x.dtype, x.device
    _row_values(dloss, "dloss", n)
    _row_values(lse, "lse", n)
    dxv = dwv = None
    if dx is not None:
        dxv = _rows(dx, "dx", x.shape, dtype, index)
    elif want_dx:
        dx = torch.empty(x.shape, dtype=dtype, device=device)
        dxv = _new_rows(dx, spec.d)
    if dweight is not None:
        dwv = _rows(dweight, "dweight", weight.shape, dtype, index)
    elif want_dweight:
        dweight = torch.empty(weight.shape, dtype=dtype, device=device)
        dwv = _new_rows(dweight, spec.d)
    if workspace is not None:
        _dev(workspace, "workspace", torch.uint8)
    elif dxv is not None or dwv is not None:
        workspace = _scratch(lib.maxsim_cross_entropy_backward_workspace_size(spec), device)
    st = lib.maxsim_cross_entropy_backward(spec, dloss.data_ptr(), xv, wv, lse.data_ptr(), dxv, dwv,
                                           None if workspace is None else workspace.data_ptr(),
                                           0 if workspace is None else workspace.numel(), _stream_on(stream, index))
    if st:
        _check(st, "maxsim_cross_entropy_backward")
    return dx, dweight
