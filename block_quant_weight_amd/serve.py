"""Thin Python binding of the calls of include/qmv_serve.h, the operators
between a quantized model's products: the norm, the heads' norm with the
position's rotation, the key/value cache in 8 or 4 bits, attention over it, log
probabilities, and the draw of the next token.  As in qmv.py, arguments are
marshalled from PyTorch tensors and streams and all computation happens in
the HIP library.  Tensors live on the current device."""
from __future__ import annotations

import ctypes
import struct

import torch

from . import qmv as _qmv
from .qmv import QMV_E_ARG, QmvError, _check
from .qmv import _stream as _stream_of

QMV_F32 = 0
QMV_BF16 = 1
QMV_KV_PAGE = 64

# every symbol include/qmv_serve.h declares
EXPORTS = ("qmv_rms_norm", "qmv_kv_write", "qmv_kv_read", "qmv_kv_attend_workspace",
           "qmv_kv_attend", "qmv_logprobs_workspace", "qmv_logprobs", "qmv_qk_rotate",
           "qmv_kv4_write", "qmv_kv4_read", "qmv_kv4_attend_workspace", "qmv_kv4_attend",
           "qmv_sample_workspace", "qmv_sample")


class _Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("pages", ctypes.c_uint32),
                ("kv_heads", ctypes.c_uint32), ("head_dim", ctypes.c_uint32)]


class _Seqs(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("len", ctypes.c_void_p), ("start", ctypes.c_void_p),
                ("seqs", ctypes.c_uint32), ("table_stride", ctypes.c_uint32),
                ("rows", ctypes.c_uint32), ("max_new", ctypes.c_uint32),
                ("max_len", ctypes.c_uint32)]


_lib = None


def lib():
    global _lib
    if _lib is None:
        L = _qmv.lib()
        u32, u64, i32, f32, vp = (ctypes.c_uint32, ctypes.c_uint64, ctypes.c_int, ctypes.c_float,
                                  ctypes.c_void_p)
        pc, ps, pu64 = ctypes.POINTER(_Cache), ctypes.POINTER(_Seqs), ctypes.POINTER(u64)
        sig = {
            "qmv_rms_norm": [vp, vp, vp, f32, u32, u32, vp, vp, vp, vp, vp, vp],
            "qmv_kv_write": [pc, ps, u32, vp, vp, vp],
            "qmv_kv_read": [pc, ps, u32, vp, vp, vp],
            "qmv_kv_attend_workspace": [pc, ps, u32, u32, u32, pu64],
            "qmv_kv_attend": [pc, ps, u32, u32, f32, u32, vp, vp, vp, u64, vp],
            "qmv_logprobs_workspace": [u32, u32, u32, pu64],
            "qmv_logprobs": [vp, u32, u32, vp, u32, u32, vp, vp, vp, vp, vp, u64, vp],
            "qmv_qk_rotate": [vp, vp, u32, u32, u32, u32, f32, vp, vp, u32, u32, f32, vp],
            "qmv_kv4_write": [pc, ps, u32, vp, vp, vp],
            "qmv_kv4_read": [pc, ps, u32, vp, vp, vp],
            "qmv_kv4_attend_workspace": [pc, ps, u32, u32, u32, pu64],
            "qmv_kv4_attend": [pc, ps, u32, u32, f32, u32, vp, vp, vp, u64, vp],
            "qmv_sample_workspace": [u32, u32, pu64],
            "qmv_sample": [vp, u32, u32, vp, vp, vp, vp, vp, vp, vp, vp, u64, vp],
        }
        for name, args in sig.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = i32
        _lib = L
    return _lib


# The current device, and its current stream's handle without a Stream object
# around it (0.1 us, not 3); a torch without them takes the long way.
_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, here):
    """Handle of a call's stream; `here` is the device of its tensors."""
    now = _device()
    if here != now:
        raise ValueError("the tensors are not on the current device")
    if stream is None and _raw_stream is not None:
        return _raw_stream(now)
    return _stream_of(stream)


def _dev(t, dtype, shape, what, here):
    """Address of a contiguous GPU tensor of device `here` of that shape."""
    if t.dtype is dtype and t.get_device() == here >= 0 and t.is_contiguous() and t.shape == shape:
        return t.data_ptr()
    return _refuse(t, dtype, what, None if t.shape == shape else
                   f"{what} must be {list(shape)}, not {list(t.shape)}")


def _first(t, dtype, numel, what, here):
    """Address of a contiguous GPU tensor of device `here` with at least numel
    elements, the first of which are used."""
    if t.dtype is dtype and t.get_device() == here >= 0 and t.is_contiguous() and t.numel() >= numel:
        return t.data_ptr()
    return _refuse(t, dtype, what, None if t.numel() >= numel else
                   f"{what} holds {t.numel()} elements, needs {numel}")


def _refuse(t, dtype, what, size):
    if not t.is_cuda:
        raise ValueError(f"{what} must be a GPU tensor")
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, not {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    raise ValueError(size or f"{what} is not on the call's device")


def _dtype(t, what):
    """QMV_F32 or QMV_BF16 of a tensor."""
    dt = t.dtype
    if dt is torch.float32:
        return QMV_F32
    if dt is torch.bfloat16:
        return QMV_BF16
    raise TypeError(f"{what} must be float32 or bfloat16, not {dt}")


def _u32(n, what):
    """n, which the library takes in 32 bits."""
    if not 0 <= n <= 0xFFFFFFFF:
        raise ValueError(f"{what} must be between 0 and 2^32 - 1")
    return n


def _scratch(nbytes, stream):
    """A workspace that a call allocates itself, in the order of its stream."""
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    with torch.cuda.stream(stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream))):
        return torch.empty(nbytes, dtype=torch.uint8, device="cuda")


def workspace(nbytes, device="cuda"):
    """A scratch tensor of nbytes for the calls that take one (never empty)."""
    return torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=device)


def _kept(name):
    """An attribute that keeps the tensor it is first given: the struct holds its address."""
    at = "_" + name

    def put(self, t):
        if self.__dict__.setdefault(at, t) is not t:
            raise AttributeError(f"{name} can only be changed in place")
    return property(lambda self: self.__dict__[at], put)


class KvCache:
    """The arrays of a cache (qmv_kv_cache): k int8 [pages, kv_heads, 64,
    head_dim], v int8 [pages, kv_heads, head_dim, 64], k_scale and v_scale
    float32 [pages, kv_heads].  KvCache.empty allocates them."""

    k, v, k_scale, v_scale = map(_kept, ("k", "v", "k_scale", "v_scale"))

    def __init__(self, k, v, k_scale, v_scale):
        if k.dim() != 4 or k.shape[2] != QMV_KV_PAGE:
            raise ValueError("k must be [pages, kv_heads, 64, head_dim]")
        self.pages, self.kv_heads, _, self.head_dim = k.shape
        if tuple(v.shape) != (self.pages, self.kv_heads, self.head_dim, QMV_KV_PAGE):
            raise ValueError("v must be [pages, kv_heads, head_dim, 64]")
        if tuple(k_scale.shape) != tuple(k.shape[:2]) or tuple(v_scale.shape) != tuple(k.shape[:2]):
            raise ValueError("the scales must be [pages, kv_heads]")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.device = k.get_device()
        here = self.device
        self.c = _Cache(_dev(k, torch.int8, k.shape, "k", here), _dev(v, torch.int8, v.shape, "v", here),
                        _dev(k_scale, torch.float32, k_scale.shape, "k_scale", here),
                        _dev(v_scale, torch.float32, v_scale.shape, "v_scale", here),
                        self.pages, self.kv_heads, self.head_dim)
        self.ref = ctypes.pointer(self.c)

    @classmethod
    def empty(cls, pages, kv_heads, head_dim, device="cuda"):
        return cls(torch.empty(pages, kv_heads, QMV_KV_PAGE, head_dim, dtype=torch.int8, device=device),
                   torch.empty(pages, kv_heads, head_dim, QMV_KV_PAGE, dtype=torch.int8, device=device),
                   torch.empty(pages, kv_heads, dtype=torch.float32, device=device),
                   torch.empty(pages, kv_heads, dtype=torch.float32, device=device))


class Kv4Cache:
    """The arrays of a cache in 4 bits (qmv_kv4_cache): k and v uint8 [pages,
    kv_heads, 64, head_dim / 2], k_scale and v_scale uint8 [pages, kv_heads, 64,
    head_dim / 32] (the order within a page and head is the library's own).
    Kv4Cache.empty allocates them."""

    k, v, k_scale, v_scale = map(_kept, ("k", "v", "k_scale", "v_scale"))

    def __init__(self, k, v, k_scale, v_scale):
        if k.dim() != 4 or k.shape[2] != QMV_KV_PAGE:
            raise ValueError("k must be [pages, kv_heads, 64, head_dim / 2]")
        self.pages, self.kv_heads, _, half = k.shape
        self.head_dim = 2 * half
        scales = (self.pages, self.kv_heads, QMV_KV_PAGE, self.head_dim // 32)
        if v.shape != k.shape:
            raise ValueError("v must be [pages, kv_heads, 64, head_dim / 2]")
        if tuple(k_scale.shape) != scales or tuple(v_scale.shape) != scales:
            raise ValueError("the scales must be [pages, kv_heads, 64, head_dim / 32]")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.device = k.get_device()
        here, u8 = self.device, torch.uint8
        self.c = _Cache(_dev(k, u8, k.shape, "k", here), _dev(v, u8, v.shape, "v", here),
                        _dev(k_scale, u8, k_scale.shape, "k_scale", here),
                        _dev(v_scale, u8, v_scale.shape, "v_scale", here), self.pages, self.kv_heads, self.head_dim)
        self.ref = ctypes.pointer(self.c)

    @classmethod
    def empty(cls, pages, kv_heads, head_dim, device="cuda"):
        if head_dim % 32 != 0:
            raise ValueError("head_dim must be a multiple of 32")
        def u8(n):
            return torch.empty(pages, kv_heads, QMV_KV_PAGE, n, dtype=torch.uint8, device=device)
        return cls(u8(head_dim // 2), u8(head_dim // 2), u8(head_dim // 32), u8(head_dim // 32))


class KvSeqs:
    """The tokens a call is about (qmv_kv_seqs): table int32 [seqs,
    table_stride], len int32 [seqs], start int32 [seqs + 1] (of longer ones the
    first elements), on the GPU; rows of the call's arrays are given by each
    call's tensors.  max_new and
    max_len, the largest number of rows and of tokens of one sequence, shape
    the launch only.  One object serves all layers of a step, and all steps of
    a graph: its tensors are changed in place."""

    table, len, start = map(_kept, ("table", "len", "start"))

    def __init__(self, table, len, start, max_new, max_len):
        if table.dim() != 2:
            raise ValueError("table must be [seqs, table_stride]")
        if max_new < 0 or max_len < 0:
            raise ValueError("max_new and max_len must not be negative")
        self.seqs = table.shape[0]
        self.table, self.len, self.start = table, len, start
        self.device = table.get_device()
        here = self.device
        self.c = _Seqs(_dev(table, torch.int32, table.shape, "table", here),
                       _first(len, torch.int32, self.seqs, "len", here),
                       _first(start, torch.int32, self.seqs + 1, "start", here),
                       self.seqs, table.shape[1], 0, min(int(max_new), 0xFFFFFFFF), min(int(max_len), 0xFFFFFFFF))
        self.last = (0, ctypes.byref(self.c))

    def with_rows(self, rows):
        """A reference to these sequences' struct for calls of so many rows
        (kept for the next call of as many; the struct never changes)."""
        last = self.last
        if last[0] != rows:
            c = _Seqs.from_buffer_copy(self.c)
            c.rows = rows
            self.last = last = (rows, ctypes.byref(c))
        return last[1]


def _rows(cache, seqs, t, heads, what):
    """seqs with the rows of t [rows, heads, head_dim] for a call, t's
    shape, and the device."""
    here = cache.device
    if seqs.device != here:
        raise ValueError("the sequences are not on the cache's device")
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != cache.head_dim:
        raise ValueError(f"{what} must be [rows, {heads}, {cache.head_dim}]")
    return seqs.with_rows(shape[0]), shape, here


def qmv_rms_norm(x, w, eps, res=None, sum=None, y=None, q=None, d=None, stream=None):
    """x, res, sum: float32 [rows, cols]; w: float32 [cols]; y: float32 or
    bfloat16 [rows, cols]; q int8 [rows, cols] with d float32 [rows, cols/32].
    Outputs that are None are not computed; sum may be res or x."""
    shape = x.shape
    if len(shape) != 2:
        raise ValueError("x must be [rows, cols]")
    rows, cols = shape
    here, f32 = x.get_device(), torch.float32
    y32 = yb = None
    if y is not None:
        if _dtype(y, "y") == QMV_F32:
            y32 = _dev(y, f32, shape, "y", here)
        else:
            yb = _dev(y, torch.bfloat16, shape, "y", here)
    _check(lib().qmv_rms_norm(
        _dev(x, f32, shape, "x", here), None if res is None else _dev(res, f32, shape, "res", here),
        _dev(w, f32, (cols,), "w", here), eps, rows, cols, None if sum is None else _dev(sum, f32, shape, "sum", here),
        y32, yb, None if q is None else _dev(q, torch.int8, shape, "q", here),
        None if d is None else _dev(d, f32, (rows, cols // 32), "d", here), _stream(stream, here)), "qmv_rms_norm")


def _not(cache, other):
    """Refuses a cache of the other kind."""
    if isinstance(cache, other):
        raise TypeError(f"the cache must not be a {other.__name__}")


def qmv_kv_write(cache: KvCache, seqs: KvSeqs, k, v, stream=None):
    """k, v: float32 or bfloat16 [rows, kv_heads, head_dim]: the rows of seqs into the cache."""
    _not(cache, Kv4Cache)
    _write("qmv_kv_write", cache, seqs, k, v, stream)


def _write(name, cache, seqs, k, v, stream):
    dt = _dtype(k, "k")
    ref, shape, here = _rows(cache, seqs, k, cache.kv_heads, "k")
    _check(getattr(lib(), name)(cache.ref, ref, dt, _dev(k, k.dtype, shape, "k", here),
                                _dev(v, k.dtype, shape, "v", here), _stream(stream, here)), name)


def qmv_kv_read(cache: KvCache, seqs: KvSeqs, k=None, v=None, stream=None):
    """k, v (either may be None): float32 or bfloat16 [rows, kv_heads,
    head_dim], receiving the tokens of seqs."""
    _not(cache, Kv4Cache)
    _read("qmv_kv_read", cache, seqs, k, v, stream)


def _read(name, cache, seqs, k, v, stream):
    t = k if k is not None else v
    if t is None:
        raise QmvError(QMV_E_ARG, name)
    dt = _dtype(t, "k or v")
    ref, shape, here = _rows(cache, seqs, t, cache.kv_heads, "k or v")
    _check(getattr(lib(), name)(cache.ref, ref, dt, None if k is None else _dev(k, t.dtype, shape, "k", here),
                                None if v is None else _dev(v, t.dtype, shape, "v", here), _stream(stream, here)), name)


def qmv_kv_attend_workspace(cache: KvCache, seqs: KvSeqs, q, window=0) -> int:
    """Bytes of workspace that qmv_kv_attend needs for q [rows, heads, head_dim]."""
    _not(cache, Kv4Cache)
    return _attend_workspace("qmv_kv_attend_workspace", cache, seqs, q, window)


def _attend_workspace(name, cache, seqs, q, window):
    out = ctypes.c_uint64(0)
    dt = _dtype(q, "q")
    _u32(window, "window")
    shape = q.shape
    heads = shape[1] if len(shape) == 3 else 0
    ref, _, _ = _rows(cache, seqs, q, heads, "q")
    _check(getattr(lib(), name)(cache.ref, ref, dt, heads, window, ctypes.byref(out)), name)
    return out.value


def qmv_kv_attend(cache: KvCache, seqs: KvSeqs, q, out, scale=None, window=0, workspace=None,
                  stream=None):
    """q, out: float32 or bfloat16 [rows, heads, head_dim]; scale defaults to
    head_dim ** -0.5.  workspace: a uint8 GPU tensor of at least
    qmv_kv_attend_workspace bytes; None allocates one in the order of the
    stream."""
    _not(cache, Kv4Cache)
    _attend("qmv_kv_attend", cache, seqs, q, out, scale, window, workspace, stream)


def _attend(name, cache, seqs, q, out, scale, window, workspace, stream):
    dt = _dtype(q, "q")
    _u32(window, "window")
    shape = q.shape
    heads = shape[1] if len(shape) == 3 else 0
    ref, shape, here = _rows(cache, seqs, q, heads, "q")
    if workspace is None:
        nbytes = _attend_workspace(name + "_workspace", cache, seqs, q, window)
        if nbytes:
            workspace = _scratch(nbytes, stream)
    pw, nw = (None, 0) if workspace is None else (_first(workspace, torch.uint8, 0, "workspace", here),
                                                  workspace.numel())
    _check(getattr(lib(), name)(cache.ref, ref, dt, heads,
                                cache.head_dim ** -0.5 if scale is None else scale, window,
                                _dev(q, q.dtype, shape, "q", here), _dev(out, q.dtype, shape, "out", here), pw, nw,
                                _stream(stream, here)), name)


def qmv_logprobs_workspace(rows, vocab, top=0) -> int:
    out = ctypes.c_uint64(0)
    _check(lib().qmv_logprobs_workspace(_u32(rows, "rows"), _u32(vocab, "vocab"), _u32(top, "top"),
                                        ctypes.byref(out)), "qmv_logprobs_workspace")
    return out.value


def qmv_logprobs(logits, ids=None, lp=None, entropy=None, top_ids=None, top_lp=None, workspace=None,
                 stream=None):
    """logits: float32 [rows, vocab]; ids int32 and lp float32 [rows, n];
    entropy float32 [rows]; top_ids int32 and top_lp float32 [rows, top].
    workspace as for qmv_kv_attend."""
    if logits.dim() != 2:
        raise ValueError("logits must be [rows, vocab]")
    rows, vocab = logits.shape
    n = 0
    if ids is not None:
        if ids.dim() != 2 or ids.shape[0] != rows:
            raise ValueError("ids must be [rows, n]")
        n = ids.shape[1]
    top = 0
    if top_ids is not None:
        if top_ids.dim() != 2 or top_ids.shape[0] != rows:
            raise ValueError("top_ids must be [rows, top]")
        top = top_ids.shape[1]
    if workspace is None:
        workspace = _scratch(max(qmv_logprobs_workspace(rows, vocab, top), 16), stream)
    f32, i32, here = torch.float32, torch.int32, logits.get_device()
    _check(lib().qmv_logprobs(
        _dev(logits, f32, (rows, vocab), "logits", here), rows, vocab,
        None if ids is None else _dev(ids, i32, (rows, n), "ids", here), n, top,
        None if lp is None else _dev(lp, f32, lp.shape if ids is None else (rows, n), "lp", here),
        None if entropy is None else _dev(entropy, f32, (rows,), "entropy", here),
        None if top_ids is None else _dev(top_ids, i32, (rows, top), "top_ids", here),
        None if top_lp is None else _dev(top_lp, f32, top_lp.shape if top_ids is None else (rows, top), "top_lp", here),
        _first(workspace, torch.uint8, 0, "workspace", here), workspace.numel(), _stream(stream, here)),
        "qmv_logprobs")


# The fields of qmv_heads, as bytes: they take a fifth of the time of a ctypes
# structure, in calls of which this is most.
_pack_heads = struct.Struct("PPPQQI4x").pack


def _heads(t, out, w, rows, dim, dtype, out_dtype, what, here):
    """One side of qmv_qk_rotate: t and out [rows, heads, dim], their heads
    side by side (rows may be further apart)."""
    if t is None:
        if out is not None or w is not None:
            raise ValueError(f"{what}_out and {what}_w are given with {what}")
        return None
    if out is None:
        raise ValueError(f"{what}_out is missing")
    shape = t.shape
    if len(shape) == 3 and shape == out.shape and t.dtype is dtype and out.dtype is out_dtype and \
            t.get_device() == out.get_device() == here >= 0:
        n, heads, d = shape
        s, z = t.stride(), out.stride()
        if n == rows and d == dim and s[2] == z[2] == 1 and (heads == 1 or s[1] == z[1] == dim):
            least = heads * dim
            return _pack_heads(t.data_ptr(), out.data_ptr(), 0 if w is None else _dev(w, torch.float32, (dim,), what + "_w", here),
                               s[0] if rows > 1 else least, z[0] if rows > 1 else least, heads)
    if len(shape) != 3 or shape[0] != rows or shape[2] != dim or out.shape != shape:
        raise ValueError(f"{what} and {what}_out must be [{rows}, heads, {dim}]")
    for x, dt, name in ((t, dtype, what), (out, out_dtype, what + "_out")):
        if x.get_device() != here or here < 0:
            raise ValueError(f"{name} is not on the call's device")
        if x.dtype is not dt:
            raise TypeError(f"{name} must be {dt}, not {x.dtype}")
    raise ValueError(f"the heads of {what} and {what}_out must lie side by side")


def qmv_qk_rotate(q, k, pos, freq, q_out, k_out, q_w=None, k_w=None, eps=1e-6, neighbours=False, mscale=1.0,
                  stream=None):
    """q, q_out: float32 or bfloat16 [rows, heads, head_dim], k, k_out: [rows,
    kv_heads, head_dim] (k and k_out, or q and q_out, may be None), heads side
    by side, rows at any stride that is a multiple of 8; outputs may be the
    inputs.  q_w, k_w: float32 [head_dim], the norms' weights, None: no norm.
    pos: int32 [rows]; freq: float32 [rot / 2], radians a position, of the
    first rot channels, paired by halves or with neighbours=True side by side."""
    t, o = (q, q_out) if q is not None else (k, k_out)
    if t is None:
        raise QmvError(QMV_E_ARG, "qmv_qk_rotate")
    if o is None:
        raise ValueError("an output is missing")
    if t.dim() != 3:
        raise ValueError("q and k must be [rows, heads, head_dim]")
    rows, _, dim = t.shape
    here, dtype, out_dtype = t.get_device(), t.dtype, o.dtype
    if freq.dim() != 1:
        raise ValueError("freq must be [rot / 2]")
    half = freq.shape[0]
    _check(lib().qmv_qk_rotate(
        _heads(q, q_out, q_w, rows, dim, dtype, out_dtype, "q", here),
        _heads(k, k_out, k_w, rows, dim, dtype, out_dtype, "k", here), rows, dim, _dtype(t, "q or k"),
        _dtype(o, "q_out or k_out"), eps, _dev(pos, torch.int32, (rows,), "pos", here),
        _dev(freq, torch.float32, (half,), "freq", here), 2 * half, 1 if neighbours else 0, mscale, _stream(stream, here)),
        "qmv_qk_rotate")


def qmv_kv4_write(cache: Kv4Cache, seqs: KvSeqs, k, v, stream=None):
    """As qmv_kv_write, into a cache in 4 bits."""
    _not(cache, KvCache)
    _write("qmv_kv4_write", cache, seqs, k, v, stream)


def qmv_kv4_read(cache: Kv4Cache, seqs: KvSeqs, k=None, v=None, stream=None):
    """As qmv_kv_read, from a cache in 4 bits."""
    _not(cache, KvCache)
    _read("qmv_kv4_read", cache, seqs, k, v, stream)


def qmv_kv4_attend_workspace(cache: Kv4Cache, seqs: KvSeqs, q, window=0) -> int:
    """Bytes of workspace that qmv_kv4_attend needs for q [rows, heads, head_dim]."""
    _not(cache, KvCache)
    return _attend_workspace("qmv_kv4_attend_workspace", cache, seqs, q, window)


def qmv_kv4_attend(cache: Kv4Cache, seqs: KvSeqs, q, out, scale=None, window=0, workspace=None, stream=None):
    """As qmv_kv_attend, over a cache in 4 bits."""
    _not(cache, KvCache)
    _attend("qmv_kv4_attend", cache, seqs, q, out, scale, window, workspace, stream)


def qmv_sample_workspace(rows, vocab) -> int:
    out = ctypes.c_uint64(0)
    _check(lib().qmv_sample_workspace(_u32(rows, "rows"), _u32(vocab, "vocab"), ctypes.byref(out)), "qmv_sample_workspace")
    return out.value


def qmv_sample(logits, u, ids, temperature=None, top_k=None, top_p=None, min_p=None, lp=None, workspace=None,
               stream=None):
    """logits: float32 [rows, vocab]; u: float32 [rows], random numbers in [0,
    1); ids: int32 [rows], the tokens drawn; lp: float32 [rows], their log
    probabilities among the tokens that the filters left.  temperature, top_p,
    min_p: float32 [rows], top_k: int32 [rows], None: 1, or no such filter.
    workspace: as for qmv_kv_attend."""
    if logits.dim() != 2:
        raise ValueError("logits must be [rows, vocab]")
    rows, vocab = shape = logits.shape
    f32, i32, here, each = torch.float32, torch.int32, logits.get_device(), (rows,)
    if workspace is None:
        workspace = _scratch(max(qmv_sample_workspace(rows, vocab), 16), stream)
    _check(lib().qmv_sample(
        _dev(logits, f32, shape, "logits", here), rows, vocab, _dev(u, f32, each, "u", here),
        None if temperature is None else _dev(temperature, f32, each, "temperature", here),
        None if top_k is None else _dev(top_k, i32, each, "top_k", here),
        None if top_p is None else _dev(top_p, f32, each, "top_p", here),
        None if min_p is None else _dev(min_p, f32, each, "min_p", here), _dev(ids, i32, each, "ids", here),
        None if lp is None else _dev(lp, f32, each, "lp", here),
        _first(workspace, torch.uint8, 0, "workspace", here), workspace.numel(), _stream(stream, here)), "qmv_sample")
