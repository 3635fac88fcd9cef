"""ctypes binding of the cache operators of libkvcopy.so (include/kvcache.h)
for torch tensors: rotary positions, writes into and reads from paged key/value
caches, and attention of new tokens over them.

Every step runs inside the library; this module checks shapes, types and
devices and passes addresses.  Work is enqueued on `stream` (a
torch.cuda.Stream or a raw handle), by default torch's current stream of the
tensors' device.  As with any call on another stream, a tensor used on a stream
other than the one it was made on has to be kept until that work is done
(Tensor.record_stream, or an event).  What a call makes itself (outputs that are
not given, a plan's workspace) is made for the stream it works on.

No call records a gradient: while they are on, tensors that require one are
refused.  That of rope is rope itself, with inverse=True.
"""
from __future__ import annotations

import ctypes
import math
import operator
import struct

import torch

from .kvcopy import EALIGN, EHIP, EINVAL, KvcopyError, OK, lib  # noqa: F401

BF16, FP16, FP32, FP8, INT8 = 0, 1, 2, 3, 4
BAD_PAGE, BAD_SLOT, BAD_LENGTH = 1, 2, 4
ROPE_INTERLEAVED, ROPE_INVERSE = 1, 2
MAX_HEAD_DIM, MAX_ATTENTION_HEAD_DIM = 512, 256
SCALINGS = {"none": 0, "linear": 1, "base": 2, "parts": 3}

EXPORTS = ("kvcache_rope_frequencies", "kvcache_rope", "kvcache_write", "kvcache_read",
           "kvcache_attention_workspace_bytes", "kvcache_attention_check", "kvcache_attention")

_ROW_TYPES = (torch.bfloat16, torch.float16, torch.float32)
_TYPES = {torch.bfloat16: BF16, torch.float16: FP16, torch.float32: FP32,
          torch.float8_e4m3fn: FP8, torch.int8: INT8}


class Rows(ctypes.Structure):
    """kvcache_rows_t."""
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


_S3 = ctypes.c_int64 * 3


class Pages(ctypes.Structure):
    """kvcache_pages_t."""
    _fields_ = [("struct_size", ctypes.c_uint32), ("format", ctypes.c_uint32),
                ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("k_stride", _S3), ("v_stride", _S3), ("ks_stride", _S3), ("vs_stride", _S3),
                ("num_pages", ctypes.c_uint64), ("kv_heads", ctypes.c_uint32),
                ("page_size", ctypes.c_uint32), ("head_dim", ctypes.c_uint32),
                ("reserved", ctypes.c_uint32)]


class Rope(ctypes.Structure):
    """kvcache_rope_t."""
    _fields_ = [("struct_size", ctypes.c_uint32), ("dtype", ctypes.c_uint32),
                ("flags", ctypes.c_uint32), ("factor", ctypes.c_float),
                ("positions", ctypes.c_void_p), ("freq", ctypes.c_void_p),
                ("tokens", ctypes.c_uint64), ("head_dim", ctypes.c_uint32),
                ("rot_dim", ctypes.c_uint32), ("q_heads", ctypes.c_uint32),
                ("k_heads", ctypes.c_uint32), ("q", Rows), ("k", Rows), ("q_out", Rows),
                ("k_out", Rows)]


class AttentionArgs(ctypes.Structure):
    """kvcache_attention_t."""
    _fields_ = [("struct_size", ctypes.c_uint32), ("dtype", ctypes.c_uint32), ("q", Rows),
                ("out", Rows), ("lse", ctypes.c_void_p), ("lse_token_stride", ctypes.c_int64),
                ("lse_head_stride", ctypes.c_int64), ("page_table", ctypes.c_void_p),
                ("table_stride", ctypes.c_int64), ("q_starts", ctypes.c_void_p),
                ("context_lens", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_uint64), ("status", ctypes.c_void_p),
                ("num_seqs", ctypes.c_uint32), ("q_heads", ctypes.c_uint32),
                ("table_columns", ctypes.c_uint32), ("total_q", ctypes.c_uint32),
                ("max_q_len", ctypes.c_uint32), ("max_context", ctypes.c_uint32),
                ("window", ctypes.c_int32), ("scale", ctypes.c_float)]


# kvcache_rope_t in one call: a ctypes structure costs twice the time to fill.
_PACK_ROPE = struct.Struct("@IIIfPPQIIII" + "Pqq" * 4).pack
_ROPE_BYTES, _NO_ROWS = ctypes.sizeof(Rope), (0, 0, 0)


def _declare():
    p, u32, u64 = ctypes.c_void_p, ctypes.c_uint32, ctypes.c_uint64
    pages, rows = ctypes.POINTER(Pages), ctypes.POINTER(Rows)
    lib.kvcache_rope_frequencies.restype = ctypes.c_int
    lib.kvcache_rope_frequencies.argtypes = [p, u32, ctypes.c_double, ctypes.c_int, ctypes.c_double,
                                             u32, ctypes.c_double, ctypes.c_double]
    lib.kvcache_rope.restype = ctypes.c_int
    lib.kvcache_rope.argtypes = [p, p]
    for f in (lib.kvcache_write, lib.kvcache_read):
        f.restype = ctypes.c_int
        f.argtypes = [pages, u32, rows, rows, p, u64, p, p]
    lib.kvcache_attention_workspace_bytes.restype = u64
    lib.kvcache_attention_workspace_bytes.argtypes = [pages, ctypes.POINTER(AttentionArgs)]
    lib.kvcache_attention_check.restype = ctypes.c_int
    lib.kvcache_attention_check.argtypes = [pages, ctypes.POINTER(AttentionArgs)]
    lib.kvcache_attention.restype = ctypes.c_int
    lib.kvcache_attention.argtypes = [pages, ctypes.POINTER(AttentionArgs), p]


_declare()


def _check(rc: int, where: str) -> None:
    if rc != OK:
        raise KvcopyError(rc, where)


def _require(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _whole(x, bits: int, what: str) -> int:
    """x as a whole number of this many bits; ctypes would keep its low ones."""
    x = operator.index(x)
    _require(0 <= x < 1 << bits, f"{what} must be at least 0 and less than 2^{bits}")
    return x


_raw_stream = torch._C._cuda_getCurrentRawStream   # a tenth of the cost of torch.cuda.current_stream


def _handle(stream, index) -> int:
    if stream is None:
        return _raw_stream(index)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """A new tensor that work on `stream` may write at once.  The allocator
    orders the uses of a block only by the stream it was made under: one made
    under another stream may still be written by work that is queued there."""
    if stream is None or _handle(stream, device.index) == _raw_stream(device.index):
        return torch.empty(shape, dtype=dtype, device=device)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device) if int(stream) else \
            torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        out = torch.empty(shape, dtype=dtype, device=device)
    # the caller, who waits for `stream`, goes on with it on the current one
    out.record_stream(torch.cuda.current_stream(device))
    return out


def _call(fn, where: str, device, stream, *args) -> None:
    """fn(*args, stream) with `device` current."""
    index = device.index
    handle = _raw_stream(index) if stream is None else _handle(stream, index)
    if torch.cuda.current_device() == index:
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(index):
            rc = fn(*args, handle)
    if rc != OK:
        raise KvcopyError(rc, where)


# These run on every call: messages are made only when they are raised.

def _no_gradient(t):
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError("a tensor requires a gradient, which this call does not record: detach it, "
                         "or call under torch.no_grad()")



def _status(status, device):
    if status is None:
        return None
    if status.device != device or status.dtype not in (torch.int32, torch.uint32) or status.numel() < 1:
        raise ValueError("status must be an int32 tensor on the same device")
    return status.data_ptr()


def _vector(t, dtype, n, device, what):
    if t.dtype != dtype or t.device != device or t.shape != (n,) or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{what} must be a contiguous {dtype} vector of {n} on {device}")
    return t.data_ptr()


def _rows(t, shape, dtype, device, what):
    st = t.stride()
    if t.dtype != dtype or t.device != device or t.shape != shape or (st[2] != 1 and shape[2] != 1):
        raise ValueError(f"{what} must be {dtype} of shape {tuple(shape)} on {device}, "
                         "its last dimension contiguous")
    if t.requires_grad:
        _no_gradient(t)
    return t.data_ptr(), st[0], st[1]


def rope_frequencies(rot_dim: int, base: float = 10000.0, scaling: str = "none",
                     factor: float = 1.0, original: int = 0, low: float = 1.0,
                     high: float = 4.0, device=None) -> torch.Tensor:
    """Radians per position of each pair, float64 (kvcache_rope_frequencies);
    scaling: "none", "linear", "base" or "parts"."""
    _require(scaling in SCALINGS, f"scaling must be one of {sorted(SCALINGS)}")
    rot_dim, original = _whole(int(rot_dim), 16, "rot_dim"), _whole(int(original), 32, "original")
    out = torch.empty(max(1, rot_dim // 2), dtype=torch.float64)
    _check(lib.kvcache_rope_frequencies(out.data_ptr(), rot_dim, float(base),
                                        SCALINGS[scaling], float(factor), original,
                                        float(low), float(high)), "kvcache_rope_frequencies")
    return out if device is None else out.to(device)


def rope(positions, freqs, q, k=None, *, q_out=None, k_out=None, interleaved: bool = False,
         factor: float = 1.0, inverse: bool = False, stream=None):
    """Turns q (and k), [tokens, heads, head_dim], by rotary positions (see
    kvcache_rope): positions int32 [tokens], freqs float64 [rot_dim / 2].
    q_out and k_out default to new tensors and may be q and k themselves.
    Returns (q_out, k_out)."""
    dev, dt, shape = q.device, q.dtype, q.shape
    if len(shape) != 3 or dev.type != "cuda" or dt not in _ROW_TYPES:
        raise ValueError("q must be a [tokens, heads, head_dim] bfloat16, float16 or float32 GPU tensor")
    tokens, heads, dim = shape
    pairs = freqs.shape[0]
    if q_out is None:
        q_out = _empty(shape, dt, dev, stream)
    k_heads, k_rows, k_out_rows = 0, _NO_ROWS, _NO_ROWS
    if k is not None:
        kshape = k.shape
        if len(kshape) != 3 or kshape[0] != tokens or kshape[2] != dim:
            raise ValueError("k must be [tokens, heads, head_dim], with q's tokens and head_dim")
        if k_out is None:
            k_out = _empty(kshape, dt, dev, stream)
        k_heads = kshape[1]
        k_rows, k_out_rows = _rows(k, kshape, dt, dev, "k"), _rows(k_out, kshape, dt, dev, "k_out")
    elif k_out is not None:
        raise ValueError("k_out without k")
    packed = _PACK_ROPE(_ROPE_BYTES, _TYPES[dt],
                        (ROPE_INTERLEAVED if interleaved else 0) | (ROPE_INVERSE if inverse else 0), factor,
                        _vector(positions, torch.int32, tokens, dev, "positions"),
                        _vector(freqs, torch.float64, pairs, dev, "freqs"),
                        tokens, dim, 2 * pairs, heads, k_heads, *_rows(q, shape, dt, dev, "q"), *k_rows,
                        *_rows(q_out, shape, dt, dev, "q_out"), *k_out_rows)
    _call(lib.kvcache_rope, "kvcache_rope", dev, stream, packed)
    return q_out, k_out


class PagedCache:
    """Keys and values in pages [num_pages, kv_heads, page_size, head_dim]
    (views in any memory order with the last dimension contiguous):
    bfloat16 or float16, or float8_e4m3fn or int8 codes with float32 scales
    [num_pages, kv_heads, page_size].  Holds the tensors; the memory stays the
    caller's."""

    def __init__(self, k, v, k_scales=None, v_scales=None):
        _require(k.dim() == 4 and k.is_cuda and k.dtype in _TYPES and k.dtype != torch.float32,
                 "pages must be 4-dimensional bfloat16, float16, float8_e4m3fn or int8 GPU tensors")
        _require(v.shape == k.shape and v.dtype == k.dtype and v.device == k.device,
                 "k and v must have the same shape, type and device")
        coded = k.dtype in (torch.float8_e4m3fn, torch.int8)
        _require(coded == (k_scales is not None) and coded == (v_scales is not None),
                 "8-bit pages need k_scales and v_scales, others take none")
        ks, vs, dim = k.stride(), v.stride(), k.shape[3]
        _require((ks[3] == 1 and vs[3] == 1) or dim == 1, "head_dim must be contiguous")
        scales = [None, None, (0, 0, 0), (0, 0, 0)]
        if coded:
            for x in (k_scales, v_scales):
                _require(x.shape == k.shape[:3] and x.dtype == torch.float32 and x.device == k.device,
                         "scales must be float32 of shape [num_pages, kv_heads, page_size]")
            scales = [k_scales.data_ptr(), v_scales.data_ptr(), k_scales.stride(), v_scales.stride()]
        for x in (k, v, *((k_scales, v_scales) if coded else ())):
            _no_gradient(x)
        p = Pages(ctypes.sizeof(Pages), _TYPES[k.dtype], k.data_ptr(), v.data_ptr(), scales[0], scales[1],
                  ks[:3], vs[:3], scales[2], scales[3], *k.shape)
        self.k, self.v, self.k_scales, self.v_scales = k, v, k_scales, v_scales
        self.dtype, self.device, self.coded = k.dtype, k.device, coded
        self.num_pages, self.kv_heads, self.page_size, self.head_dim = k.shape
        self.pages, self._ref = p, ctypes.byref(p)


def write(cache: PagedCache, k, v, slots, *, status=None, stream=None) -> None:
    """Writes k and v, [tokens, kv_heads, head_dim], to slots (int64 [tokens];
    negative: left out) of the cache (see kvcache_write).  A slot that is named
    twice ends with a mixture of both tokens."""
    if k.dim() != 3 or k.dtype not in _ROW_TYPES[:2]:
        raise ValueError("k must be a 3-dimensional bfloat16 or float16 tensor")
    dev, shape = cache.device, (k.shape[0], cache.kv_heads, cache.head_dim)
    r, w = Rows(*_rows(k, shape, k.dtype, dev, "k")), Rows(*_rows(v, shape, k.dtype, dev, "v"))
    _call(lib.kvcache_write, "kvcache_write", dev, stream, cache._ref, _TYPES[k.dtype], ctypes.byref(r),
          ctypes.byref(w), _vector(slots, torch.int64, shape[0], dev, "slots"), shape[0], _status(status, dev))


def read(cache: PagedCache, slots, k_out=None, v_out=None, *, dtype=None, status=None, stream=None):
    """The values at slots (int64 [tokens]; negative: zeros) of the cache, in
    k_out and v_out, [tokens, kv_heads, head_dim] (see kvcache_read); new
    tensors of `dtype` (bfloat16, or the pages' own) where not given.
    Returns (k_out, v_out)."""
    dev, shape = cache.device, (slots.shape[0], cache.kv_heads, cache.head_dim)
    if dtype is None:
        given = k_out if k_out is not None else v_out
        dtype = given.dtype if given is not None else torch.bfloat16 if cache.coded else cache.dtype
    if dtype not in _ROW_TYPES:
        raise ValueError("rows are bfloat16, float16 or float32")
    if k_out is None:
        k_out = _empty(shape, dtype, dev, stream)
    if v_out is None:
        v_out = _empty(shape, dtype, dev, stream)
    r, w = Rows(*_rows(k_out, shape, dtype, dev, "k_out")), Rows(*_rows(v_out, shape, dtype, dev, "v_out"))
    _call(lib.kvcache_read, "kvcache_read", dev, stream, cache._ref, _TYPES[dtype], ctypes.byref(r),
          ctypes.byref(w), _vector(slots, torch.int64, shape[0], dev, "slots"), shape[0], _status(status, dev))
    return k_out, v_out


class AttentionPlan:
    """Attention of new tokens over a cache (see kvcache_attention), for
    num_seqs sequences and total_q new tokens: the sizes and the workspace that
    calls of one shape share.  One thread at a time calls a plan.  It keeps a
    workspace for each stream that it was called on, so that calls on several
    streams do not meet; graphs captured from one plan on one stream share it,
    need the plan kept, and must not be replayed at the same time.

    scale defaults to 1 / sqrt(head_dim); window 0 means none.  num_seqs and
    total_q are exact; max_q_len and max_context are bounds.  dtype is the
    queries' and the output's: the pages' own, or over 8-bit pages bfloat16 or
    float16, by default whichever the queries of a call have."""

    def __init__(self, cache: PagedCache, *, q_heads: int, num_seqs: int, total_q: int, max_q_len: int,
                 max_context: int, window: int = 0, scale=None, dtype=None):
        self.cache = cache
        # None: either type, as the queries come (the workspace is the same)
        self.dtype = dtype if dtype is not None else None if cache.coded else cache.dtype
        _require(self.dtype in (None, *_ROW_TYPES[:2]), "rows are bfloat16 or float16")
        a = AttentionArgs(ctypes.sizeof(AttentionArgs), _TYPES[self.dtype or torch.bfloat16])
        for name, value in dict(num_seqs=num_seqs, q_heads=q_heads, total_q=total_q, max_q_len=max_q_len,
                                max_context=max_context, window=window).items():
            setattr(a, name, _whole(value, 31 if name == "window" else 32, name))
        a.scale = 1.0 / math.sqrt(cache.head_dim) if scale is None else scale
        # columns are checked against the table of each call
        a.table_columns = -(-a.max_context // cache.page_size)
        self.columns = a.table_columns
        self.args, self._ref = a, ctypes.byref(a)
        self.shape, self.num_seqs = (a.total_q, a.q_heads, cache.head_dim), a.num_seqs
        _check(lib.kvcache_attention_check(cache._ref, self._ref), "kvcache_attention_check")
        a.workspace_bytes = lib.kvcache_attention_workspace_bytes(cache._ref, ctypes.byref(a))
        # by stream: memory made under one may be handed on while another still uses it
        self._workspaces = {}
        self.workspace = self._workspace(None, cache.device) if a.workspace_bytes else None   # the current stream's

    def _workspace(self, stream, device):
        handle = _handle(stream, device.index)
        if handle not in self._workspaces:
            self._workspaces[handle] = _empty((self.args.workspace_bytes,), torch.uint8, device, stream)
        return self._workspaces[handle]

    def __call__(self, q, page_table, q_starts, context_lens, *, out=None, lse=None, status=None, stream=None):
        """q [total_q, q_heads, head_dim]; page_table int32 [num_seqs, columns];
        q_starts int32 [num_seqs + 1]; context_lens int32 [num_seqs].  lse, if
        given, float32 [total_q, q_heads], receives the log-sums.  Returns out."""
        a, dev, dt = self.args, self.cache.device, self.dtype
        if dt is None:
            dt = q.dtype
            if dt not in _ROW_TYPES[:2]:
                raise ValueError("q must be bfloat16 or float16")
            a.dtype = _TYPES[dt]
        if out is None:
            out = _empty(self.shape, dt, dev, stream)
        a.q = _rows(q, self.shape, dt, dev, "q")       # a tuple fills the structure
        a.out = _rows(out, self.shape, dt, dev, "out")
        ts, st = page_table.shape, page_table.stride()
        if (page_table.dtype != torch.int32 or page_table.device != dev or len(ts) != 2 or ts[0] != self.num_seqs
                or ts[1] < self.columns or (ts[1] > 1 and st[1] != 1)):
            raise ValueError(f"page_table must be int32 [{self.num_seqs}, >= {self.columns}] with contiguous rows "
                             f"on {dev}")
        a.page_table, a.table_stride = page_table.data_ptr(), st[0]
        a.q_starts = _vector(q_starts, torch.int32, self.num_seqs + 1, dev, "q_starts")
        a.context_lens = _vector(context_lens, torch.int32, self.num_seqs, dev, "context_lens")
        if lse is not None:
            if lse.dtype != torch.float32 or lse.device != dev or lse.shape != self.shape[:2]:
                raise ValueError(f"lse must be float32 {self.shape[:2]} on {dev}")
            _no_gradient(lse)
            a.lse_token_stride, a.lse_head_stride = lse.stride()
            a.lse = lse.data_ptr()
        else:
            a.lse = None
        a.status = _status(status, dev)
        if a.workspace_bytes:
            a.workspace = self._workspace(stream, dev).data_ptr()
        _call(lib.kvcache_attention, "kvcache_attention", dev, stream, self.cache._ref, self._ref)
        return out
