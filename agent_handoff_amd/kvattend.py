"""Python binding of the operators of include/kvattend.h (in libkvcodec.so).

Every function has the C entry point's name. Rows (queries, keys, values,
outputs) are bf16 GPU tensors [tokens, heads, head_dim] of any strides that are
multiples of 8 with the last dimension contiguous; a paged cache is a uint8
tensor described by (num_pages, num_kv_heads, page_tokens, head_dim, format).
The work is enqueued on `stream` (a torch.cuda.Stream or a raw hipStream_t
integer), or on the current stream of the tensors' device; all tensors of a
call are on one device. Wrong tensors raise ValueError, errors from the
library kvcodec.KvcError. PagedKV holds one paged cache and calls these
functions.

The calls that enqueue work are marshalled by the module _kvattend (built with
the library; the import fails without it), the size queries through ctypes.
"""

import ctypes

import numpy as np
import torch

from . import _kvattend
from . import kvcodec as _kv
from .kvcodec import KVC_ROPE_ADJACENT, KVC_ROPE_HALVES, KvcError, kvc_shape  # noqa: F401

KVC_PAGE_BF16, KVC_PAGE_INT8, KVC_PAGE_FP8, KVC_PAGE_FP4 = 0, 1, 2, 4
KVC_DEV_BAD_SLOT, KVC_DEV_BAD_PAGE, KVC_DEV_BAD_LENGTH, KVC_DEV_BAD_START = 16, 32, 64, 128
EXPORTED = ("kvc_norm_rotate", "kvpage_bytes", "kvpage_write", "kvpage_read", "kvpage_append",
            "kvpage_attend_workspace_bytes", "kvpage_attend", "kvpage_attend_window_workspace_bytes", "kvpage_attend_window",
            "kvpage_attend_prompt_workspace_bytes", "kvpage_attend_prompt", "kvpool_attend_workspace_bytes", "kvpool_attend")


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
        "kvpage_append": (i32, [spec, p, sz, u32, u32, rows, rows, rows, p, p, f32, p, p, u32, u32, p, rows, p, p]),
        "kvpage_attend_window_workspace_bytes": (sz, [spec, u32, u32, u32, u32, u32]),
        "kvpage_attend_window": (i32, [spec, p, sz, u32, u32, rows, p, u32, u64, p, u32, u32, f32, rows, p, p, sz, p, p]),
        "kvpage_attend_prompt_workspace_bytes": (sz, [spec, u32, u32, u32, u32, u32, u32]),
        "kvpage_attend_prompt": (i32, [spec, p, sz, u32, u32, u32, rows, p, p, u32, u64, p, u32, u32, f32, rows, p, p, sz, p,
                                       p]),
        "kvpool_attend_workspace_bytes": (sz, [shape, u32, u32, spec, u32]),
        "kvpool_attend": (i32, [shape, p, sz, u32, u32, u32, rows, f32, ctypes.POINTER(kvc_tail), rows, p, p, sz, p, p]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    return lib


_lib = _declare(_kv.library())
_kvattend.setup(KvcError, torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice, torch.cuda.device,
                lambda x: np.ascontiguousarray(x, np.float32),
                *(ctypes.cast(getattr(_lib, f), ctypes.c_void_p).value for f in
                  ("kvc_norm_rotate", "kvpage_write", "kvpage_read", "kvpage_attend", "kvpool_attend", "kvpage_append",
                   "kvpage_attend_window", "kvpage_attend_prompt")))
kvc_norm_rotate = _kvattend.kvc_norm_rotate
kvpage_write, kvpage_read = _kvattend.kvpage_write, _kvattend.kvpage_read
kvpage_attend, kvpool_attend = _kvattend.kvpage_attend, _kvattend.kvpool_attend
kvpage_append = _kvattend.kvpage_append
kvpage_attend_window, kvpage_attend_prompt = _kvattend.kvpage_attend_window, _kvattend.kvpage_attend_prompt


def _spec(spec):
    return spec if isinstance(spec, kvc_pages) else kvc_pages(*spec)


def kvpage_bytes(spec):
    return int(_lib.kvpage_bytes(_spec(spec)))


def kvpage_attend_workspace_bytes(spec, n_seqs, q_heads, max_tokens):
    return int(_lib.kvpage_attend_workspace_bytes(_spec(spec), int(n_seqs), int(q_heads), int(max_tokens)))


def kvpage_attend_window_workspace_bytes(spec, n_seqs, q_heads, max_tokens, window, sinks):
    return int(_lib.kvpage_attend_window_workspace_bytes(_spec(spec), int(n_seqs), int(q_heads), int(max_tokens), int(window),
                                                         int(sinks)))


def kvpage_attend_prompt_workspace_bytes(spec, n_seqs, n_tokens, q_heads, max_tokens, window=0, sinks=0):
    return int(_lib.kvpage_attend_prompt_workspace_bytes(_spec(spec), int(n_seqs), int(n_tokens), int(q_heads),
                                                         int(max_tokens), int(window), int(sinks)))


def kvpool_attend_workspace_bytes(shape, n_agents, q_heads, tail_spec=None, max_tail_tokens=0):
    return int(_lib.kvpool_attend_workspace_bytes(ctypes.byref(_kv._shape(shape)), int(n_agents), int(q_heads),
                                                  None if tail_spec is None else _spec(tail_spec),
                                                  int(max_tail_tokens)))


# ------------------------------------------------------------------ object wrapper

class PagedKV:
    """The paged cache of one layer (PolyKV 2.A: what an agent adds behind the
    shared document). Holds the pages' bytes and their description; allocates
    outputs and workspaces on the pages' device and calls the kvpage_ functions
    on the current stream."""

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

    def append(self, q, k, v, positions, inv_freq, slots, q_out=None, q_weight=None, k_weight=None, eps=1e-6,
               pairing=KVC_ROPE_HALVES, dev_status=None):
        """Norms and rotation of q and k, which with v go into their slots; returns the turned queries (q None: None)."""
        if q is not None and q_out is None:
            q_out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
        kvpage_append(self.spec, self.pages, q, k, v, positions, inv_freq, slots, q_out, q_weight, k_weight, eps, pairing,
                      dev_status)
        return q_out

    def attend(self, q, table, lens, out=None, lse=None, scale=None, dev_status=None, window=0, sinks=0):
        """One new token per sequence over its pages, or over the last `window` tokens and the first `sinks`; returns out."""
        if out is None:
            out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
        need = kvpage_attend_window_workspace_bytes(self.spec, q.shape[0], q.shape[1], table.shape[1] * self.spec.page_tokens,
                                                    window, sinks)
        ws = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
        kvpage_attend_window(self.spec, self.pages, q, table, lens, window, sinks, out, ws, lse, scale, dev_status)
        return out

    def attend_prompt(self, q, starts, table, lens, out=None, lse=None, scale=None, dev_status=None, window=0, sinks=0):
        """The new tokens of each sequence (rows starts[b] to starts[b + 1]) over its pages; returns out (new: rows of
        no sequence are zeros)."""
        if out is None:
            out = torch.zeros(q.shape, dtype=torch.bfloat16, device=q.device)
        need = kvpage_attend_prompt_workspace_bytes(self.spec, starts.numel() - 1, q.shape[0], q.shape[1],
                                                    table.shape[1] * self.spec.page_tokens, window, sinks)
        ws = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
        kvpage_attend_prompt(self.spec, self.pages, q, starts, table, lens, out, ws, window, sinks, lse, scale, dev_status)
        return out
