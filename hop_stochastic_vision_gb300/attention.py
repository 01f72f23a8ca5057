"""Softmax cross attention and the learned relative position bias
(C ABI in include/lisa_attention.h), on CUDA tensors.

Argument marshalling only, as in ``lisa``: torch supplies device memory and
streams, every step runs in the library's kernels.
"""
from __future__ import annotations

import ctypes
import functools
import math

import torch

from .lisa import LISA_BF16, LISA_ERR_UNSUPPORTED, LISA_F32, LISA_OK, LisaError, load

LISA_BUCKETS_EXACT = 0
LISA_BUCKETS_LOG = 1
LISA_MAX_OFFSETS = 16384

ATTENTION_EXPORTED = ("lisa_relative_bias", "lisa_relative_bias_backward_workspace_bytes",
                      "lisa_relative_bias_backward", "lisa_cross_attention_workspace_bytes",
                      "lisa_cross_attention", "lisa_cross_attention_backward_workspace_bytes",
                      "lisa_cross_attention_backward")


class lisa_strides(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_longlong), ("head", ctypes.c_longlong), ("token", ctypes.c_longlong)]


class lisa_axis_rule(ctypes.Structure):
    _fields_ = [("rule", ctypes.c_int), ("buckets", ctypes.c_int), ("max_distance", ctypes.c_int)]


class lisa_rel_bias(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p),
                ("q_rows", ctypes.c_int), ("q_cols", ctypes.c_int), ("k_rows", ctypes.c_int),
                ("k_cols", ctypes.c_int), ("key_step_rows", ctypes.c_int), ("key_step_cols", ctypes.c_int),
                ("start_rows", ctypes.c_int), ("start_cols", ctypes.c_int), ("starts", ctypes.c_void_p),
                ("rows", lisa_axis_rule), ("cols", lisa_axis_rule)]


_lib = None


def _library():
    """The loaded library with this module's signatures set."""
    global _lib
    if _lib is None:
        lib = load()
        vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        sp, bp = ctypes.POINTER(lisa_strides), ctypes.POINTER(lisa_rel_bias)
        lib.lisa_relative_bias.argtypes = [bp, i, vp, i, vp]
        lib.lisa_relative_bias.restype = i
        lib.lisa_relative_bias_backward_workspace_bytes.argtypes = [bp, i]
        lib.lisa_relative_bias_backward_workspace_bytes.restype = sz
        lib.lisa_relative_bias_backward.argtypes = [bp, i, vp, i, vp, vp, sz, vp]
        lib.lisa_relative_bias_backward.restype = i
        lib.lisa_cross_attention_workspace_bytes.argtypes = [i] * 6 + [bp, i]
        lib.lisa_cross_attention_workspace_bytes.restype = sz
        lib.lisa_cross_attention.argtypes = [vp, sp, vp, sp, vp, sp, vp, sp, vp, i, i, i, i, i, i, f, vp, bp, i, vp,
                                             sz, vp]
        lib.lisa_cross_attention.restype = i
        lib.lisa_cross_attention_backward_workspace_bytes.argtypes = [i] * 6 + [bp, i]
        lib.lisa_cross_attention_backward_workspace_bytes.restype = sz
        lib.lisa_cross_attention_backward.argtypes = [vp, sp, vp, sp, vp, sp, vp, sp, vp, vp, sp, vp, vp, vp, vp, i, i,
                                                      i, i, i, i, f, vp, bp, i, vp, sz, vp]
        lib.lisa_cross_attention_backward.restype = i
        _lib = lib
    return _lib


# -- the C entry points under their own names ---------------------------------------
# strides: lisa_strides; bias: lisa_rel_bias or None; pointers are ints (device addresses).

def _ref(x):
    return None if x is None else ctypes.byref(x)


def lisa_relative_bias(bias, heads, out, dtype, stream) -> int:
    return int(_library().lisa_relative_bias(_ref(bias), heads, out, dtype, stream))


def lisa_relative_bias_backward_workspace_bytes(bias, heads) -> int:
    return int(_library().lisa_relative_bias_backward_workspace_bytes(_ref(bias), heads))


def lisa_relative_bias_backward(bias, heads, dbias, dtype, dtable, workspace, workspace_bytes, stream) -> int:
    return int(_library().lisa_relative_bias_backward(_ref(bias), heads, dbias, dtype, dtable, workspace,
                                                      workspace_bytes, stream))


def lisa_cross_attention_workspace_bytes(B, heads, kv_heads, n, m, d, bias, dtype) -> int:
    return int(_library().lisa_cross_attention_workspace_bytes(B, heads, kv_heads, n, m, d, _ref(bias), dtype))


def lisa_cross_attention(Q, qs, K, ks, V, vs, O, os, lse, B, heads, kv_heads, n, m, d, scale, kv_lens, bias, dtype,
                         workspace, workspace_bytes, stream) -> int:
    return int(_library().lisa_cross_attention(Q, _ref(qs), K, _ref(ks), V, _ref(vs), O, _ref(os), lse, B, heads,
                                               kv_heads, n, m, d, scale, kv_lens, _ref(bias), dtype, workspace,
                                               workspace_bytes, stream))


def lisa_cross_attention_backward_workspace_bytes(B, heads, kv_heads, n, m, d, bias, dtype) -> int:
    return int(_library().lisa_cross_attention_backward_workspace_bytes(B, heads, kv_heads, n, m, d, _ref(bias),
                                                                        dtype))


def lisa_cross_attention_backward(Q, qs, K, ks, V, vs, O, os, lse, dO, dos, dQ, dK, dV, dtable, B, heads, kv_heads,
                                  n, m, d, scale, kv_lens, bias, dtype, workspace, workspace_bytes, stream) -> int:
    return int(_library().lisa_cross_attention_backward(Q, _ref(qs), K, _ref(ks), V, _ref(vs), O, _ref(os), lse, dO,
                                                        _ref(dos), dQ, dK, dV, dtable, B, heads, kv_heads, n, m, d,
                                                        scale, kv_lens, _ref(bias), dtype, workspace,
                                                        workspace_bytes, stream))


# -- tensor-level convenience ---------------------------------------------------------

_DTYPES = {torch.float32: LISA_F32, torch.bfloat16: LISA_BF16}


def _int32(x) -> int:
    """x as one of the C ABI's 32-bit numbers (ctypes would drop the bits above)."""
    x = int(x)
    if not -(1 << 31) <= x < 1 << 31:
        raise ValueError("%d is beyond 32 bits" % x)
    return x


def exact_buckets(max_distance: int) -> lisa_axis_rule:
    """One bucket for each offset -D .. D of an axis; farther ones share the outermost."""
    return lisa_axis_rule(LISA_BUCKETS_EXACT, _int32(2 * int(max_distance) + 1), _int32(max_distance))


def log_buckets(buckets: int, max_distance: int) -> lisa_axis_rule:
    """``buckets`` of an axis, half to each side: near offsets one by one, farther
    ones in geometrically growing buckets up to ``max_distance``."""
    return lisa_axis_rule(LISA_BUCKETS_LOG, _int32(buckets), _int32(max_distance))


class RelativeBias:
    """A learned relative position bias: the table (fp32 CUDA tensor
    [rows.buckets * cols.buckets, heads]) and the rule that picks its row.

    Queries are the tokens of the grid ``q_grid`` = (rows, columns), keys those
    of ``k_grid``; a sequence is a grid of one row.  Query (r, c) stands at
    ``query_start`` + (r, c), key (r, c) at (key_step[0] r, key_step[1] c).
    ``query_start`` may be an int32 CUDA tensor [B]: each batch entry's own
    start on a sequence (forward only).  The table may be updated between calls,
    and it and ``starts`` replaced by tensors of the same kind; every call checks
    them and the object keeps no copy."""

    def __init__(self, table: torch.Tensor, q_grid, k_grid, rows: lisa_axis_rule = None,
                 cols: lisa_axis_rule = None, key_step=(1, 1), query_start=(0, 0)):
        rows = exact_buckets(0) if rows is None else rows
        if cols is None:
            raise ValueError("RelativeBias needs the columns' bucket rule")
        if not (table.is_cuda and table.dtype == torch.float32 and table.is_contiguous() and table.dim() == 2):
            raise ValueError("the bias table must be a contiguous fp32 CUDA tensor [buckets, heads]")
        if table.shape[0] != rows.buckets * cols.buckets:
            raise ValueError("the bias table has %d rows, the rules give %d buckets"
                             % (table.shape[0], rows.buckets * cols.buckets))
        self.table = table
        self.shape = (int(table.shape[0]), int(table.shape[1]))
        self.heads = self.shape[1]
        self.q_grid = (_int32(q_grid[0]), _int32(q_grid[1]))
        self.k_grid = (_int32(k_grid[0]), _int32(k_grid[1]))
        self.n = self.q_grid[0] * self.q_grid[1]
        self.m = self.k_grid[0] * self.k_grid[1]
        self.starts = None
        start = (0, 0)
        if isinstance(query_start, torch.Tensor):
            self.starts = query_start   # checked with the table, below
        else:
            start = (_int32(query_start[0]), _int32(query_start[1]))
        self.struct = lisa_rel_bias(None, *self.q_grid, *self.k_grid, _int32(key_step[0]), _int32(key_step[1]),
                                    *start, None, rows, cols)
        self.current()

    def current(self) -> lisa_rel_bias:
        """The C struct, with the table and the starts where they are now (an
        optimiser or a module may have moved the storage behind them)."""
        s, table = self.struct, self.table
        if not (table.is_cuda and table.dtype == torch.float32 and table.is_contiguous() and table.shape == self.shape):
            raise ValueError("the bias table must stay a contiguous fp32 CUDA tensor [%d, %d]" % self.shape)
        s.table = table.data_ptr()
        self.index = table.get_device()
        starts = self.starts
        if starts is None:
            s.starts = None
        else:
            if not (starts.get_device() == self.index and starts.dtype == torch.int32 and starts.is_contiguous()
                    and starts.dim() == 1):
                raise ValueError("query_start must be a pair of ints or a contiguous int32 CUDA tensor [B]")
            s.starts = starts.data_ptr()
        return s


def _raw_stream(index: int) -> int:
    return torch.cuda.current_stream(index).cuda_stream


# the same values without the objects and checks around them, where torch offers that
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


class _On:
    """The device and the stream of a call made current, so what the call
    allocates belongs to the stream that uses it."""

    def __init__(self, index, stream):
        self.index = index
        self.device = torch.cuda.device(index)
        self.stream = stream

    def __enter__(self):
        self.device.__enter__()
        self.other = None
        if self.stream is not None:
            of = torch.device("cuda", self.index)
            self.other = torch.cuda.stream(torch.cuda.ExternalStream(int(self.stream), device=of))
            self.other.__enter__()

    def __exit__(self, *exc):
        if self.other is not None:
            self.other.__exit__(*exc)
        self.device.__exit__(*exc)


def _run(index, stream, call, *args):
    """call(raw stream, *args) on the tensors' device and the given or current stream."""
    if stream is None and _current_device() == index:
        return call(_raw_stream(index), *args)
    with _On(index, stream):
        return call(_raw_stream(index), *args)


def _workspace(given, nbytes, device):
    """(tensor to keep, address, bytes) of the call's workspace."""
    if given is None:
        if nbytes == 0:
            return None, None, 0
        given = torch.empty(nbytes, dtype=torch.uint8, device=device)
    elif given.device != device or not given.is_contiguous():
        raise ValueError("the workspace must be a contiguous tensor on the call's device")
    return given, given.data_ptr(), given.numel() * given.element_size()


@functools.lru_cache(maxsize=4096)
def _strides_of(shape, stride) -> lisa_strides:
    if len(shape) != 4:
        raise ValueError("q, k, v, out, dout must be 4-d and share dtype float32 or bfloat16")
    d = shape[3]
    if stride[3] != 1 and d > 1:
        raise ValueError("the elements of a token must be contiguous (last stride 1)")
    # a stride that no step uses may be anything legal
    return lisa_strides(*(stride[x] if shape[x] > 1 else d for x in range(3)))


@functools.lru_cache(maxsize=1024)
def _plain_bytes(B, heads, kv_heads, n, m, d, dtype):
    return lisa_cross_attention_workspace_bytes(B, heads, kv_heads, n, m, d, None, dtype)


@functools.lru_cache(maxsize=64)
def _default_scale(d):
    return 1.0 / math.sqrt(d) if d > 0 else 1.0   # a width of 0 is refused by the call


def _strides(t, shape, dtype, index) -> lisa_strides:
    """Strides of a tensor of the call, which has to match its device and type."""
    if t.dtype != dtype:
        raise ValueError("q, k, v, out, dout must be 4-d and share dtype float32 or bfloat16")
    at = t.get_device()
    if at != index or at < 0:
        raise ValueError("the cross attention runs on CUDA tensors only" if at < 0
                         else "tensors must be on one device")
    return _strides_of(shape, t.stride())


def _prepare(q, k, v, kv_lens, bias, scale):
    """Checks and the call's common arguments."""
    dtype = q.dtype
    dt = _DTYPES.get(dtype)
    if dt is None:
        raise ValueError("q, k, v must share dtype float32 or bfloat16")
    index, shape, kv_shape = q.get_device(), q.shape, k.shape
    qs, ks = _strides(q, shape, dtype, index), _strides(k, kv_shape, dtype, index)
    vs = _strides(v, v.shape, dtype, index)
    B, heads, n, d = shape
    kv_heads, m = kv_shape[1], kv_shape[2]
    if kv_shape[0] != B or kv_shape[3] != d or v.shape != kv_shape:
        raise ValueError("k and v must be [B, kv_heads, m, d] for q [B, heads, n, d]")
    if max(shape) >> 31 or max(kv_shape) >> 31:   # the call itself refuses far less, if it gets to see it
        raise LisaError(LISA_ERR_UNSUPPORTED)
    lens = struct = None
    if kv_lens is not None:
        if not (kv_lens.get_device() == index and kv_lens.dtype == torch.int32 and kv_lens.is_contiguous()
                and kv_lens.shape == (B,)):
            raise ValueError("kv_lens must be a contiguous int32 CUDA tensor [B]")
        lens = kv_lens.data_ptr()
    if bias is not None:
        struct = bias.current()
        if bias.index != index:
            raise ValueError("tensors must be on one device")
        if (bias.heads, bias.n, bias.m) != (heads, n, m):
            raise ValueError("the bias is of %d heads, %d queries and %d keys, the call of %d, %d and %d"
                             % (bias.heads, bias.n, bias.m, heads, n, m))
        if bias.starts is not None and bias.starts.shape[0] != B:
            raise ValueError("query_start must have one entry per batch entry")
    tail = (B, heads, kv_heads, n, m, d, _default_scale(d) if scale is None else float(scale), lens, struct, dt)
    return index, shape, kv_shape, (q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs), tail


def _forward(stream, q, index, shape, head, tail, return_lse, out, workspace):
    device = q.device
    if out is None:
        out = torch.empty(shape, dtype=q.dtype, device=device)
    elif out.shape != shape:
        raise ValueError("out must have q's shape")
    os = _strides(out, shape, q.dtype, index)
    B, heads, kv_heads, n, m, d, _, _, struct, dt = tail
    lse = torch.empty((B, heads, n), dtype=torch.float32, device=device) if return_lse else None
    lib = _library()
    need = _plain_bytes(B, heads, kv_heads, n, m, d, dt) if struct is None else \
        lib.lisa_cross_attention_workspace_bytes(B, heads, kv_heads, n, m, d, struct, dt)
    keep, ws, nbytes = _workspace(workspace, need, device)
    status = lib.lisa_cross_attention(*head, out.data_ptr(), os, lse.data_ptr() if return_lse else None, *tail, ws,
                                      nbytes, stream)
    del keep
    if status != LISA_OK:
        raise LisaError(status)
    return (out, lse) if return_lse else out


def cross_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *, scale=None, kv_lens=None,
                    bias: RelativeBias = None, return_lse: bool = False, out=None, workspace=None, stream=None):
    """Softmax attention of queries [B, heads, n, d] over keys and values
    [B, kv_heads, m, d] (fp32 or bf16; heads a multiple of kv_heads; strided
    views are fine, with d contiguous and strides of 16 bytes).  ``scale``
    defaults to 1 / sqrt(d); ``kv_lens`` (int32 [B]) is the number of valid keys
    of each batch entry; ``bias`` a RelativeBias.  Returns O [B, heads, n, d]
    (a new contiguous tensor unless ``out`` is given), with ``return_lse`` also
    the fp32 log-sum-exp [B, heads, n] that the backward pass reads.
    ``stream`` is a raw stream handle of the tensors' device."""
    index, shape, _, head, tail = _prepare(q, k, v, kv_lens, bias, scale)
    return _run(index, stream, _forward, q, index, shape, head, tail, return_lse, out, workspace)


def _backward(stream, q, shape, kv_shape, head, saved, tail, bias, workspace):
    device, dtype = q.device, q.dtype
    dq = torch.empty(shape, dtype=dtype, device=device)
    dk = torch.empty(kv_shape, dtype=dtype, device=device)
    dv = torch.empty(kv_shape, dtype=dtype, device=device)
    dtable = None if bias is None else torch.empty(bias.shape, dtype=torch.float32, device=device)
    B, heads, kv_heads, n, m, d, _, _, struct, dt = tail
    lib = _library()
    need = lib.lisa_cross_attention_backward_workspace_bytes(B, heads, kv_heads, n, m, d, struct, dt)
    keep, ws, nbytes = _workspace(workspace, need, device)
    status = lib.lisa_cross_attention_backward(*head, *saved, dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                                               None if bias is None else dtable.data_ptr(), *tail, ws, nbytes, stream)
    del keep
    if status != LISA_OK:
        raise LisaError(status)
    return (dq, dk, dv) if bias is None else (dq, dk, dv, dtable)


def cross_attention_backward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor, lse: torch.Tensor,
                             dout: torch.Tensor, *, scale=None, kv_lens=None, bias: RelativeBias = None,
                             workspace=None, stream=None):
    """Gradients of ``cross_attention`` for the upstream gradient ``dout``, given
    the forward's ``out`` and ``lse``: (dq, dk, dv), with ``bias`` also the
    table's gradient dtable (fp32, the table's shape), summed over the batch."""
    index, shape, kv_shape, head, tail = _prepare(q, k, v, kv_lens, bias, scale)
    if out.shape != shape or dout.shape != shape:
        raise ValueError("out and dout must have q's shape")
    if not (lse.get_device() == index and lse.dtype == torch.float32 and lse.is_contiguous()
            and lse.shape == shape[:3]):
        raise ValueError("lse must be the forward's contiguous fp32 tensor [B, heads, n]")
    if bias is not None and bias.starts is not None:
        raise ValueError("a bias with a start for each batch entry has no backward")
    saved = (out.data_ptr(), _strides(out, shape, q.dtype, index), lse.data_ptr(), dout.data_ptr(),
             _strides(dout, shape, q.dtype, index))
    return _run(index, stream, _backward, q, shape, kv_shape, head, saved, tail, bias, workspace)


def _matrix(stream, bias, dtype, out):
    if out is None:
        out = torch.empty((bias.heads, bias.n, bias.m), dtype=dtype, device=bias.table.device)
    status = _library().lisa_relative_bias(bias.struct, bias.heads, out.data_ptr(), _DTYPES[dtype], stream)
    if status != LISA_OK:
        raise LisaError(status)
    return out


def relative_bias(bias: RelativeBias, dtype: torch.dtype = torch.float32, *, out=None, stream=None) -> torch.Tensor:
    """The bias as a matrix [heads, n, m] (fp32 or bf16), for a layer that adds it itself."""
    if dtype not in _DTYPES:
        raise ValueError("dtype must be float32 or bfloat16")
    if bias.starts is not None:
        raise ValueError("a bias with a start for each batch entry has no matrix")
    bias.current()
    if out is not None and not (out.get_device() == bias.index and out.dtype == dtype and out.is_contiguous()
                                and out.shape == (bias.heads, bias.n, bias.m)):
        raise ValueError("out must be a contiguous %s CUDA tensor [heads, n, m]" % (dtype,))
    return _run(bias.index, stream, _matrix, bias, dtype, out)


def _matrix_backward(stream, bias, dbias, workspace):
    dtable = torch.empty(bias.shape, dtype=torch.float32, device=dbias.device)
    lib = _library()
    keep, ws, nbytes = _workspace(workspace, lib.lisa_relative_bias_backward_workspace_bytes(bias.struct, bias.heads),
                                  dbias.device)
    status = lib.lisa_relative_bias_backward(bias.struct, bias.heads, dbias.data_ptr(), _DTYPES[dbias.dtype],
                                             dtable.data_ptr(), ws, nbytes, stream)
    del keep
    if status != LISA_OK:
        raise LisaError(status)
    return dtable


def relative_bias_backward(bias: RelativeBias, dbias: torch.Tensor, *, workspace=None, stream=None) -> torch.Tensor:
    """The table's gradient (fp32, the table's shape): the sums of ``dbias``
    [heads, n, m] (fp32 or bf16) over the pairs of each bucket."""
    if bias.starts is not None:
        raise ValueError("a bias with a start for each batch entry has no matrix")
    bias.current()
    if not (dbias.get_device() == bias.index and dbias.dtype in _DTYPES and dbias.is_contiguous()
            and dbias.shape == (bias.heads, bias.n, bias.m)):
        raise ValueError("dbias must be a contiguous fp32 or bf16 CUDA tensor [heads, n, m]")
    return _run(bias.index, stream, _matrix_backward, bias, dbias, workspace)
