"""Python binding of the operators of include/kvattend.h (in libkvcodec.so):
argument marshalling only, as in kvcodec.

Every function has the C entry point's name. Rows (queries, keys, values,
outputs) are bf16 GPU tensors [tokens, heads, head_dim] of any strides that are
multiples of 8 with the last dimension contiguous; a paged cache is a uint8
tensor described by (num_pages, num_kv_heads, page_tokens, head_dim, format).
The work is enqueued on `stream`, or on the current stream of the tensors'
device; all tensors of a call are on one device. Errors from the library raise
kvcodec.KvcError. PagedKV holds one paged cache and calls these functions.
"""

import ctypes
import math

import numpy as np
import torch

from . import kvcodec as _kv
from .kvcodec import KVC_ROPE_ADJACENT, KVC_ROPE_HALVES, KvcError, kvc_shape  # noqa: F401

KVC_PAGE_BF16, KVC_PAGE_INT8, KVC_PAGE_FP8 = 0, 1, 2
KVC_DEV_BAD_SLOT, KVC_DEV_BAD_PAGE, KVC_DEV_BAD_LENGTH = 16, 32, 64
EXPORTED = ("kvc_norm_rotate", "kvpage_bytes", "kvpage_write", "kvpage_read", "kvpage_attend_workspace_bytes",
            "kvpage_attend", "kvpool_attend_workspace_bytes", "kvpool_attend")


class kvc_rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_uint64), ("head_stride", ctypes.c_uint64)]


class kvc_pages(ctypes.Structure):
    _fields_ = [("num_pages", ctypes.c_uint32), ("num_kv_heads", ctypes.c_uint32), ("page_tokens", ctypes.c_uint32),
                ("head_dim", ctypes.c_uint32), ("format", ctypes.c_uint32)]


class kvc_tail(ctypes.Structure):
    _fields_ = [("spec", ctypes.POINTER(kvc_pages)), ("pages", ctypes.c_void_p), ("pages_bytes", ctypes.c_size_t),
                ("table", ctypes.c_void_p), ("table_cols", ctypes.c_uint32), ("table_stride", ctypes.c_uint64),
                ("lens", ctypes.c_void_p)]


def _declare(lib):
    sz, i32, u32, u64, f32, p = (ctypes.c_size_t, ctypes.c_int, ctypes.c_uint32, ctypes.c_uint64, ctypes.c_float,
                                 ctypes.c_void_p)
    rows, spec, shape = ctypes.POINTER(kvc_rows), ctypes.POINTER(kvc_pages), ctypes.POINTER(kvc_shape)
    sig = {
        "kvc_norm_rotate": (i32, [u32, u32, u32, u32, rows, rows, p, p, f32, p, p, u32, u32, rows, rows, p]),
        "kvpage_bytes": (sz, [spec]),
        "kvpage_write": (i32, [spec, p, sz, u32, rows, rows, p, p, p]),
        "kvpage_read": (i32, [spec, p, sz, u32, p, rows, rows, p, p]),
        "kvpage_attend_workspace_bytes": (sz, [spec, u32, u32, u32]),
        "kvpage_attend": (i32, [spec, p, sz, u32, u32, rows, p, u32, u64, p, f32, rows, p, p, sz, p, p]),
        "kvpool_attend_workspace_bytes": (sz, [shape, u32, u32, spec, u32]),
        "kvpool_attend": (i32, [shape, p, sz, u32, u32, u32, rows, f32, ctypes.POINTER(kvc_tail), rows, p, p, sz, p, p]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    return lib


_lib = _declare(_kv.library())


def _spec(spec):
    return spec if isinstance(spec, kvc_pages) else kvc_pages(*spec)


_BF16 = torch.bfloat16


def _rows(t, shape, what):
    """bf16 rows of this shape (n, heads, d) of a GPU tensor; strides of dimensions of size 1 are not used."""
    if t.dtype is not _BF16:
        raise ValueError(f"{what}: expected {_BF16}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{what}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    ts, hs, cs = t.stride()
    if cs != 1 and shape[0]:
        raise ValueError(f"{what}: the last dimension must be contiguous")
    return kvc_rows(t.data_ptr(), ts, hs)


def _plain(t, dtype, shape, what):
    """Address of a contiguous GPU tensor of this type and shape."""
    if t.dtype is not dtype:
        raise ValueError(f"{what}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{what}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous tensor")
    return t.data_ptr()


def _bytes(t, what):
    if t.dtype is not torch.uint8 or not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous uint8 tensor")
    return t.data_ptr()


def _status(t):
    return None if t is None else _plain(t, torch.int32, (1,), "dev_status")


def _call(what, function, args, tensors, stream):
    """function(*args, stream) with the tensors' device current (tensors may hold None)."""
    device = tensors[0].get_device()  # -1: not on a GPU
    for t in tensors:
        if t is not None and t.get_device() != device:
            raise ValueError(f"{what}: tensors are on different devices")
    if device < 0:
        raise ValueError("expected a GPU tensor")
    if device == torch._C._cuda_getDevice():
        # the current stream's handle without a Stream object: a call takes a few microseconds in all
        rc = function(*args, torch._C._cuda_getCurrentRawStream(device) if stream is None else _kv._stream(stream))
    else:
        with torch.cuda.device(device):
            rc = function(*args, _kv._stream(stream))
    if rc != 0:
        raise KvcError(rc, what)


def kvc_norm_rotate(q, k, positions, inv_freq, q_out, k_out, q_weight=None, k_weight=None, eps=1e-6,
                    pairing=KVC_ROPE_HALVES, stream=None):
    """q, q_out: rows [n, q_heads, d]; k, k_out: rows [n, kv_heads, d] (either
    pair may be None); the same tensor for in place. positions: int64 [n];
    inv_freq: host floats, one for each pair that is turned (empty: none);
    q_weight, k_weight: bf16 [d] or None (no norm)."""
    first = q if q is not None else k
    if first is None or first.dim() != 3:
        raise ValueError("expected rows [tokens, heads, head_dim]")
    if (q is None) != (q_out is None) or (k is None) != (k_out is None):
        raise ValueError("each input needs its output")
    n, _, d = first.shape
    hq = hk = 0
    qi = qo = ki = ko = qw = kw = at = None
    if q is not None:
        hq = q.shape[1]
        qi, qo = _rows(q, (n, hq, d), "q"), _rows(q_out, (n, hq, d), "q_out")
        if q_weight is not None:
            qw = _plain(q_weight, _BF16, (d,), "q_weight")
    if k is not None:
        hk = k.shape[1]
        ki, ko = _rows(k, (n, hk, d), "k"), _rows(k_out, (n, hk, d), "k_out")
        if k_weight is not None:
            kw = _plain(k_weight, _BF16, (d,), "k_weight")
    f = np.ascontiguousarray(inv_freq, np.float32)
    if not f.flags.writeable:
        f = f.copy()  # only for the cheap way to its address
    if positions is not None:
        at = _plain(positions, torch.int64, (n,), "positions")
    elif f.size:
        raise ValueError("positions: tensor required")
    _call("kvc_norm_rotate", _lib.kvc_norm_rotate,
          (n, hq, hk, d, qi, ki, qw, kw, eps, at, ctypes.addressof(ctypes.c_char.from_buffer(f)) if f.size else None, f.size, pairing, qo, ko),
          (first, q, k, q_out, k_out, positions, q_weight, k_weight), stream)


# ------------------------------------------------------------------ paged cache

def kvpage_bytes(spec):
    return int(_lib.kvpage_bytes(_spec(spec)))


def _page_copy(what, function, write, spec, pages, k, v, slots, dev_status, stream):
    s = _spec(spec)
    n = slots.numel()
    shape = (n, s.num_kv_heads, s.head_dim)
    at, size = _bytes(pages, "pages"), pages.numel()
    kr, vr = _rows(k, shape, "k"), _rows(v, shape, "v")
    sl = _plain(slots, torch.int64, (n,), "slots")
    st = _status(dev_status)
    args = (s, at, size, n, kr, vr, sl, st) if write else (s, at, size, n, sl, kr, vr, st)
    _call(what, function, args, (pages, k, v, slots, dev_status), stream)


def kvpage_write(spec, pages, k, v, slots, dev_status=None, stream=None):
    """k, v: rows [n, num_kv_heads, head_dim]; slots: int64 [n], page *
    page_tokens + offset (negative: skipped); dev_status: int32 [1] or None."""
    _page_copy("kvpage_write", _lib.kvpage_write, True, spec, pages, k, v, slots, dev_status, stream)


def kvpage_read(spec, pages, slots, k_out, v_out, dev_status=None, stream=None):
    """The tokens of `slots` into rows k_out, v_out (rows of negative slots
    are left as they were)."""
    _page_copy("kvpage_read", _lib.kvpage_read, False, spec, pages, k_out, v_out, slots, dev_status, stream)


# ------------------------------------------------------------------ attention

def kvpage_attend_workspace_bytes(spec, n_seqs, q_heads, max_tokens):
    return int(_lib.kvpage_attend_workspace_bytes(_spec(spec), int(n_seqs), int(q_heads), int(max_tokens)))


def _table(table, lens, n):
    if table.dtype is not torch.int32 or table.dim() != 2 or table.shape[0] != n or \
            (n and table.shape[1] > 1 and table.stride(1) != 1):
        raise ValueError(f"table: expected int32 [{n}, columns] with contiguous rows")
    return table.data_ptr(), table.shape[1], table.stride(0), _plain(lens, torch.int32, (n,), "lens")


def _attend_args(q, out, lse, scale, head_dim):
    shape = q.shape
    if len(shape) != 3:
        raise ValueError("q: expected rows [sequences, heads, head_dim]")
    n, hq, d = shape
    if d != head_dim:
        raise ValueError(f"q: expected head_dim {head_dim}, got {d}")
    return (n, hq, _rows(q, shape, "q"), _rows(out, shape, "out"),
            None if lse is None else _plain(lse, torch.float32, (n, hq), "lse"),
            1.0 / math.sqrt(d) if scale is None else scale)


def kvpage_attend(spec, pages, q, table, lens, out, ws, lse=None, scale=None, dev_status=None, stream=None):
    """q, out: rows [n, q_heads, head_dim]; table: int32 [n, columns] page
    numbers; lens: int32 [n]; ws: uint8 workspace
    (kvpage_attend_workspace_bytes of columns * page_tokens); lse: float32
    [n, q_heads] or None; scale: 1 / sqrt(head_dim) if None."""
    s = _spec(spec)
    n, hq, qr, outr, lp, scale = _attend_args(q, out, lse, scale, s.head_dim)
    tab, cols, stride, lens_p = _table(table, lens, n)
    _call("kvpage_attend", _lib.kvpage_attend,
          (s, _bytes(pages, "pages"), pages.numel(), n, hq, qr, tab, cols, stride, lens_p, scale, outr, lp,
           _bytes(ws, "ws"), ws.numel(), _status(dev_status)),
          (pages, q, table, lens, out, ws, lse, dev_status), stream)


def kvpool_attend_workspace_bytes(shape, n_agents, q_heads, tail_spec=None, max_tail_tokens=0):
    return int(_lib.kvpool_attend_workspace_bytes(ctypes.byref(_kv._shape(shape)), int(n_agents), int(q_heads),
                                                  None if tail_spec is None else _spec(tail_spec),
                                                  int(max_tail_tokens)))


def kvpool_attend(shape, pool, layer, q, out, ws, tail=None, lse=None, scale=None, dev_status=None, stream=None):
    """q, out: rows [n_agents, q_heads, head_dim]; pool: uint8 tensor as
    kvpool_encode wrote it; tail: (spec, pages, table, lens) of the agents' own
    pages or None; the rest as for kvpage_attend."""
    sh = shape if isinstance(shape, kvc_shape) else kvc_shape(*shape)
    n, hq, qr, outr, lp, scale = _attend_args(q, out, lse, scale, sh.head_dim)
    tensors, tp = (pool, q, out, ws, lse, dev_status), None
    if tail is not None:
        spec, pages, table, lens = tail
        tab, cols, stride, lens_p = _table(table, lens, n)
        tp = kvc_tail(ctypes.pointer(_spec(spec)), _bytes(pages, "tail pages"), pages.numel(), tab, cols, stride, lens_p)
        tensors += (pages, table, lens)
    _call("kvpool_attend", _lib.kvpool_attend,
          (sh, _bytes(pool, "pool"), pool.numel(), layer, n, hq, qr, scale, tp, outr, lp, _bytes(ws, "ws"), ws.numel(),
           _status(dev_status)), tensors, stream)


# ------------------------------------------------------------------ object wrapper

class PagedKV:
    """The paged cache of one layer (PolyKV 2.A: what an agent adds behind the
    shared document). Holds the pages' bytes and their description; allocates
    outputs and workspaces on the pages' device and calls kvpage_write /
    kvpage_read / kvpage_attend on the current stream."""

    def __init__(self, num_pages, num_kv_heads, page_tokens, head_dim, fmt=KVC_PAGE_INT8, device="cuda"):
        self.spec = kvc_pages(num_pages, num_kv_heads, page_tokens, head_dim, fmt)
        size = kvpage_bytes(self.spec)
        if size == 0:
            raise ValueError("invalid paged cache description")
        self.pages = torch.zeros(size, dtype=torch.uint8, device=device)

    def write(self, k, v, slots, dev_status=None):
        """k, v: rows [n, num_kv_heads, head_dim]; slots: int64 [n]."""
        kvpage_write(self.spec, self.pages, k, v, slots, dev_status)

    def read(self, slots, k_out=None, v_out=None, dev_status=None):
        """Keys and values of `slots` (new tensors laid out by heads,
        [num_kv_heads, n, head_dim] in memory and ready for a pool or a card,
        seen as rows [n, num_kv_heads, head_dim], when k_out / v_out are None)."""
        shape = (self.spec.num_kv_heads, slots.numel(), self.spec.head_dim)
        new = [torch.zeros(shape, dtype=torch.bfloat16, device=self.pages.device).transpose(0, 1) if t is None else t
               for t in (k_out, v_out)]
        kvpage_read(self.spec, self.pages, slots, *new, dev_status=dev_status)
        return tuple(new)

    def attend(self, q, table, lens, out=None, lse=None, scale=None, dev_status=None):
        """One new token per sequence over its pages; returns out."""
        if out is None:
            out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
        need = kvpage_attend_workspace_bytes(self.spec, q.shape[0], q.shape[1], table.shape[1] * self.spec.page_tokens)
        ws = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
        kvpage_attend(self.spec, self.pages, q, table, lens, out, ws, lse, scale, dev_status)
        return out
