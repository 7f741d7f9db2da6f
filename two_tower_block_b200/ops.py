"""ctypes binding of libtt_block_attn.so (argument marshalling only).

Every entry point here forwards to the C function of the same name in
``include/tt_block_attn.h``.  torch supplies device memory and streams; all
computation happens in the library's CUDA kernels.  If the library is
missing, or a call is made without a CUDA device, the call raises: there is
no CPU fallback.
"""
from __future__ import annotations

import ctypes
import functools
import os
from dataclasses import dataclass

import torch

__all__ = ["TTError", "Plan", "lib", "library_path", "block_attn", "block_attn_block_causal", "confidence_unmask", "MxCache",
           "selftest_wait_timeout", "work_split", "KERNEL_AUTO", "KERNEL_TCGEN05", "KERNEL_MMA_SYNC",
           "TT_OK", "TT_ERR_INVALID_ARG", "TT_ERR_UNSUPPORTED", "TT_ERR_CUDA", "TT_ERR_DEVICE_ARG",
           "TT_ERR_TIMEOUT", "EXPORTED_SYMBOLS"]

TT_OK, TT_ERR_INVALID_ARG, TT_ERR_UNSUPPORTED, TT_ERR_CUDA, TT_ERR_DEVICE_ARG, TT_ERR_TIMEOUT = range(6)
KERNEL_AUTO, KERNEL_TCGEN05, KERNEL_MMA_SYNC = 0, 1, 2
PLAN_HOST_IO = 1
PLAN_OUT_BF16 = 2

_HERE = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_HERE, "libtt_block_attn.so")

# Every symbol the header declares (checked by the CPU test suite).
EXPORTED_SYMBOLS = [
    "tt_block_attn_plan", "tt_block_attn_plan_destroy", "tt_block_attn_plan_get_info", "tt_block_attn",
    "tt_block_attn_block_causal", "tt_block_attn_host", "tt_block_attn_check", "tt_block_attn_profile",
    "tt_block_attn_profile_read", "tt_selftest_wait_timeout", "tt_debug_work_split", "tt_status_string",
    "tt_last_error_detail", "tt_block_attn_noalloc", "tt_selftest_exp2", "tt_kv_append",
    "tt_block_attn_block_causal_backward", "tt_confidence_unmask", "tt_block_attn_paged",
    "tt_debug_causal_split", "tt_block_attn_plan_window", "tt_block_attn_tree", "tt_block_attn_tree_paged",
    "tt_kv_append_mx", "tt_kv_read_mx", "tt_block_attn_mx", "tt_debug_mx_scale_words",
    "tt_debug_decode_split", "tt_debug_causal_split_window",
]


class Desc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int), ("num_q_heads", ctypes.c_int), ("num_kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("block_size", ctypes.c_int), ("ctx_capacity", ctypes.c_int),
                ("seq_len", ctypes.c_int), ("scale", ctypes.c_float), ("kernel", ctypes.c_int),
                ("num_ctas", ctypes.c_int), ("flags", ctypes.c_int), ("wait_timeout_us", ctypes.c_int)]


class PlanInfo(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int), ("num_ctas", ctypes.c_int), ("key_tile", ctypes.c_int),
                ("rows_per_unit", ctypes.c_int), ("workspace_bytes", ctypes.c_size_t),
                ("sm_count", ctypes.c_int), ("variant", ctypes.c_int), ("fused_combine", ctypes.c_int)]


class MxCacheDesc(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("page_table", ctypes.c_void_p), ("num_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("pages_per_seq", ctypes.c_int32)]


_lib = None


def lib() -> ctypes.CDLL:
    """Load the library once; raise (never fall back) if it is absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(library_path):
        raise RuntimeError(f"{library_path} is missing: build it with `python -m two_tower_block_b200.build`")
    L = ctypes.CDLL(library_path)
    vp, ip, i, f = ctypes.c_void_p, ctypes.POINTER(ctypes.c_int), ctypes.c_int, ctypes.c_float
    L.tt_block_attn_plan.argtypes = [ctypes.POINTER(Desc), i, ctypes.POINTER(vp)]
    L.tt_block_attn_plan_destroy.argtypes = [vp]
    L.tt_block_attn_plan_destroy.restype = None
    L.tt_block_attn_plan_get_info.argtypes = [vp, ctypes.POINTER(PlanInfo)]
    L.tt_block_attn.argtypes = [vp] * 10
    L.tt_block_attn_block_causal.argtypes = [vp] * 9
    L.tt_block_attn_paged.argtypes = [vp, vp, vp, vp, vp, i, i, i, vp, vp, vp, vp, vp, vp]
    L.tt_block_attn_block_causal_backward.argtypes = [vp] * 13
    L.tt_kv_append.argtypes = [vp] * 6 + [i, vp]
    L.tt_block_attn_host.argtypes = [vp] * 10
    L.tt_block_attn_check.argtypes = [vp, vp]
    L.tt_block_attn_profile.argtypes = [vp, i]
    L.tt_block_attn_profile_read.argtypes = [vp, i, ip, ctypes.POINTER(ctypes.c_double)]
    L.tt_selftest_wait_timeout.argtypes = [i, i, vp]
    L.tt_debug_work_split.argtypes = [i, ip, i, ctypes.POINTER(ctypes.c_longlong), ip, ip]
    L.tt_block_attn_plan_window.argtypes = [ctypes.POINTER(Desc), i, i, i, ctypes.POINTER(vp)]
    L.tt_block_attn_tree.argtypes = [vp] * 11
    L.tt_block_attn_tree_paged.argtypes = [vp, vp, vp, vp, vp, i, i, i] + [vp] * 7
    cp = ctypes.POINTER(MxCacheDesc)
    L.tt_kv_append_mx.argtypes = [vp, vp, vp, i, vp, cp, vp, i, vp]
    L.tt_kv_read_mx.argtypes = [vp, cp, vp, vp, i, vp, vp, vp]
    L.tt_block_attn_mx.argtypes = [vp, vp, cp, vp, vp, vp, vp, vp, vp, vp]
    L.tt_debug_causal_split.argtypes = [i, i, i, i, i, i, i, ctypes.POINTER(ctypes.c_longlong)]
    L.tt_debug_mx_scale_words.argtypes = [i, i, ip, i, ctypes.POINTER(ctypes.c_longlong), ip, ip]
    L.tt_debug_decode_split.argtypes = [i, ip, i, i, i, i, ctypes.POINTER(ctypes.c_longlong), ip, i, ip, ip, ip]
    L.tt_debug_causal_split_window.argtypes = [i] * 9 + [ctypes.POINTER(ctypes.c_longlong)]
    L.tt_block_attn_noalloc.argtypes = [ctypes.POINTER(Desc)] + [vp] * 10
    L.tt_selftest_exp2.argtypes = [i, vp, vp, i]
    L.tt_status_string.argtypes = [i]
    L.tt_status_string.restype = ctypes.c_char_p
    L.tt_last_error_detail.argtypes = []
    L.tt_last_error_detail.restype = ctypes.c_char_p
    for name in EXPORTED_SYMBOLS:
        if name not in ("tt_block_attn_plan_destroy", "tt_status_string", "tt_last_error_detail"):
            getattr(L, name).restype = ctypes.c_int
    _lib = L
    return L


class TTError(RuntimeError):
    def __init__(self, status: int, where: str):
        L = lib()
        self.status = status
        msg = L.tt_status_string(status).decode()
        detail = L.tt_last_error_detail().decode()
        super().__init__(f"{where}: {msg}" + (f" ({detail})" if detail else ""))


def _check(status: int, where: str):
    if status != TT_OK:
        raise TTError(status, where)


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, torch.Tensor):
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")
        return ctypes.c_void_p(t.data_ptr())
    return ctypes.c_void_p(int(t))


def _arg(t, name, numel, kind, device):
    """Check one tensor argument before its address reaches the library, whose kernels
    trust every size: ``kind`` "bf16" (any 2-byte type: bf16 values or their bit
    patterns), "f32", "i32", "w32" (any 4-byte integer), "u8" or "e4m3" (any 1-byte type); ``numel`` the element count the
    layout needs; ``device`` a CUDA ordinal, "host", or None (not checked).  None and raw integer addresses
    are passed through (the library rejects a null pointer it needs)."""
    if not isinstance(t, torch.Tensor):
        return
    ok = {"bf16": t.element_size() == 2 and not t.is_floating_point() or t.dtype == torch.bfloat16,
          "f32": t.dtype == torch.float32, "i32": t.dtype == torch.int32,
          "w32": t.element_size() == 4 and not t.is_floating_point(),
          "u8": t.element_size() == 1, "e4m3": t.element_size() == 1}[kind]
    if not ok:
        raise TypeError(f"{name}: dtype {t.dtype} where {kind} is expected")
    if t.numel() != numel:
        raise ValueError(f"{name}: {t.numel()} elements where the plan's shape needs {numel}")
    if device == "host":
        if t.is_cuda:
            raise ValueError(f"{name}: a host tensor is expected")
    elif device is not None and (not t.is_cuda or t.device.index != device):
        raise ValueError(f"{name}: expected on cuda:{device}, got {t.device}")


def _args(device, *items):
    """_arg over (tensor, name, numel, kind) items: every dtype and size first, then
    every device, so a wrong shape is reported before where a tensor lives."""
    for t, name, numel, kind in items:
        _arg(t, name, numel, kind, None)
    for t, name, numel, kind in items:
        _arg(t, name, numel, kind, device)


# The type each kind of argument usually has.
_USUAL = {"bf16": torch.bfloat16, "f32": torch.float32, "i32": torch.int32, "u8": torch.uint8,
          "e4m3": torch.float8_e4m3fn}


def _quick_py(device, tensors, want):
    """Addresses of tensors that are all of the usual type, the right size, contiguous and on the device
    (-1: the CPU): one look at each, since a small call's host time is what it waits for.  ``want``:
    (dtype, numel) of each.  None if one is not (or is no tensor): _addrs then says what is wrong, or
    takes it."""
    at = []
    try:
        for t, (dtype, numel) in zip(tensors, want):
            if t.dtype is not dtype or t.numel() != numel or t.get_device() != device or not t.is_contiguous():
                return None
            at.append(t.data_ptr())
    except AttributeError:
        return None
    return at


def _pick_quick(module):
    """The same in C++ (csrc/marshal.cpp), a tenth of the time, where it was built against this very torch: it
    reads torch's tensors by the layout that it found in the headers."""
    if getattr(module, "built_for", None) == torch.__version__:
        return module.addresses
    return _quick_py


try:   # built beside the library
    from . import _marshal
except ImportError:
    _marshal = None
_quick = _pick_quick(_marshal)


def _addrs(device, items):
    """Addresses of (tensor, name, numel, kind) items after the checks of _args."""
    _args(device, *items)
    return [_ptr(t) for t, _, _, _ in items]


def _stream(stream):
    """A torch stream, a raw handle, or a Plan: the current stream of its device."""
    if isinstance(stream, Plan):
        return torch._C._cuda_getCurrentRawStream(stream.device)
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


@dataclass
class Shape:
    batch: int
    q_heads: int
    kv_heads: int
    head_dim: int
    block: int
    ctx_capacity: int = 0
    seq_len: int = 0


class MxCache:
    """A context cache in microscaled e4m3 (the header's tt_mx_cache): values k, v in any 1-byte type
    and scale bytes k_scale, v_scale with the last dimension D / 32.  Slabs [B, Hkv, Lcap, D], or with
    `page_table` [B, pages_per_seq] pools [num_pages, Hkv, P, D].  Holds the tensors it describes, whose contents
    may change but not their memory."""

    def __init__(self, k, k_scale, v, v_scale, page_table=None):
        shape = k.shape
        if len(shape) != 4 or shape[3] % 32:
            raise ValueError(f"k: shape {tuple(shape)}, expected four dimensions, the last a multiple of 32")
        self._tensors = k, k_scale, v, v_scale, page_table
        self.shape = shape
        self._device = k.get_device() if k.is_cuda else -1
        n = k.numel()
        values, scales = (torch.float8_e4m3fn, n), (torch.uint8, n // 32)
        tensors, want = (k, v, k_scale, v_scale), (values, values, scales, scales)
        num_pages = page_size = pages_per_seq = table = 0
        if page_table is not None:
            if page_table.dim() != 2:
                raise ValueError(f"page_table: shape {tuple(page_table.shape)}, expected [B, pages_per_seq]")
            num_pages, page_size, pages_per_seq, table = shape[0], shape[2], page_table.shape[1], page_table.numel()
            tensors, want = tensors + (page_table,), want + ((torch.int32, table),)
        at = _quick(self._device, tensors, want)
        if at is None:
            # (a device cache's tensors are all on that device; a host one is refused by the calls)
            items = [(k, "k", n, "e4m3"), (v, "v", n, "e4m3"), (k_scale, "k_scale", n // 32, "u8"),
                     (v_scale, "v_scale", n // 32, "u8"), (page_table, "page_table", table, "i32")]
            at = _addrs(self._device if self._device >= 0 else None, items)
        # (a table without entries has no address, and none means slabs to the library: it gets one that nothing
        # reads, since no position lies below a capacity of 0)
        self._d = MxCacheDesc(at[0], at[1], at[2], at[3], None if page_table is None else at[4] if table else 16,
                              num_pages, page_size, pages_per_seq)
        self._ref = ctypes.byref(self._d)

    # (read-only: the library has the addresses of these tensors; write into them in place, or make another cache)
    k = property(lambda self: self._tensors[0])
    k_scale = property(lambda self: self._tensors[1])
    v = property(lambda self: self._tensors[2])
    v_scale = property(lambda self: self._tensors[3])
    page_table = property(lambda self: self._tensors[4])

    @classmethod
    def empty(cls, rows_of, kv_heads, positions, head_dim, device="cuda", page_table=None):
        """A new cache of zeros: `rows_of` sequences of `positions` rows, or (with a page table) that
        many pages of `positions` rows."""
        shape = (rows_of, kv_heads, positions, head_dim)
        new = [torch.zeros(shape[:3] + (head_dim // w,), dtype=t, device=device)
               for w, t in ((1, torch.float8_e4m3fn), (32, torch.uint8)) for _ in range(2)]
        return cls(new[0], new[2], new[1], new[3], page_table=page_table)

    def _fits(self, plan):
        """The cache's layout against a plan's shape and device."""
        s = plan.shape
        shape = self.shape
        if self._device != plan.device:
            raise ValueError(f"cache: expected on cuda:{plan.device}, got {self.k.device}")
        page_table = self._tensors[4]
        if page_table is None:
            want = (s.batch, s.kv_heads, s.ctx_capacity, s.head_dim)
            if shape != want:
                raise ValueError(f"cache: shape {tuple(shape)}, expected {want}")
        elif shape[1] != s.kv_heads or shape[3] != s.head_dim or page_table.shape[0] != s.batch:
            raise ValueError(f"cache: pages {tuple(shape)} with a table {tuple(page_table.shape)}, expected "
                             f"[num_pages, {s.kv_heads}, P, {s.head_dim}] and [{s.batch}, pages_per_seq]")
        return self._ref


class Plan:
    """Owns a tt_plan_t (device scratch, work split) for one shape on one device.  With ``window`` every
    attention call sees, of a block's context, the last ``window`` positions and the first ``sinks``."""

    out_dtype = torch.float32   # torch.bfloat16 for a plan made with out_bf16=True

    def __init__(self, batch, q_heads, kv_heads, head_dim, block, ctx_capacity=0, seq_len=0, scale=0.0,
                 kernel=KERNEL_AUTO, num_ctas=0, host_io=False, wait_timeout_us=0, device=None, out_bf16=False,
                 window=0, sinks=0):
        if device is None:
            device = torch.cuda.current_device()
        self.shape = Shape(batch, q_heads, kv_heads, head_dim, block, ctx_capacity, seq_len)
        self.device = int(device)
        self.out_dtype = torch.bfloat16 if out_bf16 else torch.float32
        d = Desc(batch, q_heads, kv_heads, head_dim, block, ctx_capacity, seq_len, float(scale), kernel,
                 num_ctas, (PLAN_HOST_IO if host_io else 0) | (PLAN_OUT_BF16 if out_bf16 else 0), wait_timeout_us)
        h = ctypes.c_void_p()
        _check(lib().tt_block_attn_plan_window(ctypes.byref(d), int(window), int(sinks), self.device,
                                               ctypes.byref(h)), "tt_block_attn_plan")
        self._h = h

    def close(self):
        if getattr(self, "_h", None):
            lib().tt_block_attn_plan_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def info(self) -> PlanInfo:
        inf = PlanInfo()
        _check(lib().tt_block_attn_plan_get_info(self._h, ctypes.byref(inf)), "tt_block_attn_plan_get_info")
        return inf

    # --- decode ------------------------------------------------------------
    # Each call hands the addresses of its tensors on: by _quick, or where that finds something to look
    # at, by the checks of _addrs in their order (every size and type first, then every device).
    def _outputs(self, q, out, lse, want_lse, tokens):
        """out and lse as given, or new ones ([B, tokens, Hq, D], and [B, Hq, tokens] where wanted)."""
        s = self.shape
        if out is None:
            shape = (s.batch, tokens, s.q_heads, s.head_dim)
            if q.dtype is self.out_dtype and q.shape == shape and q.is_contiguous():
                out = torch.empty_like(q)
            else:
                out = torch.empty(shape, dtype=self.out_dtype, device=q.device)
        if lse is None and want_lse:
            lse = torch.empty((s.batch, s.q_heads, tokens), dtype=torch.float32, device=q.device)
        return out, lse

    @functools.cached_property
    def _usual(self):
        """What _quick wants of a decode call's tensors: q, k_blk, v_blk, ctx_lens, out; k_ctx and v_ctx;
        parents; lse."""
        s = self.shape
        rows = s.batch * s.block
        nq, nb = rows * s.q_heads * s.head_dim, rows * s.kv_heads * s.head_dim
        nc = s.batch * s.kv_heads * s.ctx_capacity * s.head_dim
        b, i = torch.bfloat16, torch.int32
        return (((b, nq), (b, nb), (b, nb), (i, s.batch), (self.out_dtype, nq)), ((b, nc), (b, nc)), ((i, rows),),
                ((torch.float32, rows * s.q_heads),))

    def _decode_args(self, q, k_blk, v_blk, ctx_lens, out, lse, more, want, items):
        """Addresses of q, k_blk, v_blk, ctx_lens, out, lse and then of ``more`` (wanted as ``want``;
        ``items`` gives the same for _addrs)."""
        usual = self._usual
        first = (q, k_blk, v_blk, ctx_lens, out)
        if lse is None:
            at = _quick(self.device, first + more, usual[0] + want)
            if at is not None:
                at.insert(5, None)
        else:
            at = _quick(self.device, first + (lse,) + more, usual[0] + usual[3] + want)
        return at or _addrs(self.device, self._decode_items(q, k_blk, v_blk, ctx_lens, out, lse) + items())

    def _decode_items(self, q, k_blk, v_blk, ctx_lens, out, lse):
        s = self.shape
        rows = s.batch * s.block
        nq, nb = rows * s.q_heads * s.head_dim, rows * s.kv_heads * s.head_dim
        return ((q, "q", nq, "bf16"), (k_blk, "k_blk", nb, "bf16"), (v_blk, "v_blk", nb, "bf16"),
                (ctx_lens, "ctx_lens", s.batch, "i32"), (out, "out", nq, self._out_kind()),
                (lse, "lse", rows * s.q_heads, "f32"))

    def _slab_items(self, k_ctx, v_ctx):
        s = self.shape
        nc = s.batch * s.kv_heads * s.ctx_capacity * s.head_dim
        return (k_ctx, "k_ctx", nc, "bf16"), (v_ctx, "v_ctx", nc, "bf16")

    def _page_items(self, k_pages, v_pages, page_table):
        """(num_pages, page_size, pages_per_seq, items to check, what _quick wants) of a paged context."""
        s = self.shape
        if k_pages is None:
            num_pages, page_size = 0, 16      # no pool: valid only without context (the library checks)
        else:
            shape = k_pages.shape
            if len(shape) != 4 or shape[1] != s.kv_heads or shape[3] != s.head_dim:
                raise ValueError(f"k_pages: shape {tuple(k_pages.shape)}, expected [num_pages, {s.kv_heads}, P, "
                                 f"{s.head_dim}]")
            num_pages, page_size = shape[0], shape[2]
        pool_numel = k_pages.numel() if k_pages is not None else 0
        pages_per_seq = 0
        if page_table is not None:
            shape = page_table.shape
            if len(shape) != 2 or shape[0] != s.batch:
                raise ValueError(f"page_table: shape {tuple(shape)}, expected [{s.batch}, pages_per_seq]")
            pages_per_seq = shape[1]
        return num_pages, page_size, pages_per_seq, lambda: (
            (k_pages, "k_pages", pool_numel, "bf16"), (v_pages, "v_pages", pool_numel, "bf16"),
            (page_table, "page_table", s.batch * pages_per_seq, "i32")), (
            (torch.bfloat16, pool_numel), (torch.bfloat16, pool_numel), (torch.int32, s.batch * pages_per_seq))

    def _parents_item(self, parents):
        return (parents, "parents", self.shape.batch * self.shape.block, "i32")

    def _out_kind(self):
        return "bf16" if self.out_dtype == torch.bfloat16 else "f32"

    def _on(self, stream):
        return _stream(self if stream is None else stream)

    def block_attn(self, q, k_ctx, v_ctx, k_blk, v_blk, ctx_lens, out=None, lse=None, stream=None,
                   want_lse=False):
        out, lse = self._outputs(q, out, lse, want_lse, self.shape.block)
        q_, kb, vb, lens, o, l, kc, vc = self._decode_args(
            q, k_blk, v_blk, ctx_lens, out, lse, (k_ctx, v_ctx), self._usual[1],
            lambda: self._slab_items(k_ctx, v_ctx))
        _check(lib().tt_block_attn(self._h, q_, kc, vc, kb, vb, lens, o, l, self._on(stream)), "tt_block_attn")
        return (out, lse) if lse is not None else out

    def block_attn_paged(self, q, k_pages, v_pages, page_table, k_blk, v_blk, ctx_lens, out=None, lse=None,
                         stream=None, want_lse=False):
        """Decode over a paged context cache: k_pages / v_pages [num_pages, Hkv, P, D] bf16
        pools, page_table [B, pages_per_seq] int32 (device); P = k_pages.shape[2].  With no
        context at all, the pools and the table may be None."""
        out, lse = self._outputs(q, out, lse, want_lse, self.shape.block)
        num_pages, page_size, pages_per_seq, items, want = self._page_items(k_pages, v_pages, page_table)
        q_, kb, vb, lens, o, l, kp, vp, tab = self._decode_args(
            q, k_blk, v_blk, ctx_lens, out, lse, (k_pages, v_pages, page_table), want, items)
        _check(lib().tt_block_attn_paged(self._h, q_, kp, vp, tab, num_pages, page_size, pages_per_seq, kb, vb, lens,
                                         o, l, self._on(stream)), "tt_block_attn_paged")
        return (out, lse) if lse is not None else out

    def block_attn_tree(self, q, k_ctx, v_ctx, k_blk, v_blk, ctx_lens, parents, out=None, lse=None, stream=None,
                        want_lse=False):
        """Decode whose block is a tree of drafted tokens: parents [B, S] int32 (-1: hangs on the last
        committed token, -2: absent).  Otherwise as block_attn."""
        out, lse = self._outputs(q, out, lse, want_lse, self.shape.block)
        q_, kb, vb, lens, o, l, kc, vc, par = self._decode_args(
            q, k_blk, v_blk, ctx_lens, out, lse, (k_ctx, v_ctx, parents), self._usual[1] + self._usual[2],
            lambda: self._slab_items(k_ctx, v_ctx) + (self._parents_item(parents),))
        _check(lib().tt_block_attn_tree(self._h, q_, kc, vc, kb, vb, lens, par, o, l, self._on(stream)),
               "tt_block_attn_tree")
        return (out, lse) if lse is not None else out

    def block_attn_tree_paged(self, q, k_pages, v_pages, page_table, k_blk, v_blk, ctx_lens, parents, out=None,
                              lse=None, stream=None, want_lse=False):
        """block_attn_tree over a paged context cache (pages as block_attn_paged)."""
        out, lse = self._outputs(q, out, lse, want_lse, self.shape.block)
        num_pages, page_size, pages_per_seq, items, want = self._page_items(k_pages, v_pages, page_table)
        q_, kb, vb, lens, o, l, kp, vp, tab, par = self._decode_args(
            q, k_blk, v_blk, ctx_lens, out, lse, (k_pages, v_pages, page_table, parents), want + self._usual[2],
            lambda: items() + (self._parents_item(parents),))
        _check(lib().tt_block_attn_tree_paged(self._h, q_, kp, vp, tab, num_pages, page_size, pages_per_seq, kb, vb,
                                              lens, par, o, l, self._on(stream)), "tt_block_attn_tree_paged")
        return (out, lse) if lse is not None else out

    # --- quantised context cache ---------------------------------------------
    def block_attn_mx(self, q, cache, k_blk, v_blk, ctx_lens, parents=None, out=None, lse=None, stream=None,
                      want_lse=False):
        """Decode over a quantised context cache (MxCache); with ``parents`` the block is a drafted tree."""
        out, lse = self._outputs(q, out, lse, want_lse, self.shape.block)
        tree = parents is not None
        q_, kb, vb, lens, o, l, *par = self._decode_args(
            q, k_blk, v_blk, ctx_lens, out, lse, (parents,) if tree else (), self._usual[2] if tree else (),
            lambda: (self._parents_item(parents),) if tree else ())
        _check(lib().tt_block_attn_mx(self._h, q_, cache._fits(self), kb, vb, lens, par[0] if tree else None,
                                      o, l, self._on(stream)),
               "tt_block_attn_mx")
        return (out, lse) if lse is not None else out

    def _rows_args(self, k, v, n, ctx_lens, per_seq, names):
        """Addresses of the rows k and v of n elements each, ctx_lens, and one optional int32 per sequence."""
        B = self.shape.batch
        want = (torch.bfloat16, n), (torch.bfloat16, n), (torch.int32, B), (torch.int32, B)
        if per_seq is not None:
            at = _quick(self.device, (k, v, ctx_lens, per_seq), want)
        else:
            at = _quick(self.device, (k, v, ctx_lens), want[:3])
            if at is not None:
                at.append(None)
        return at or _addrs(self.device, ((k, names[0], n, "bf16"), (v, names[1], n, "bf16"),
                                          (ctx_lens, "ctx_lens", B, "i32"), (per_seq, names[2], B, "i32")))

    def kv_append_mx(self, k_new, v_new, cache, ctx_lens, counts=None, advance=True, stream=None):
        """Quantise k_new/v_new [B, rows, Hkv, D] into the cache at [L_n, L_n + counts[n]) (all rows
        without ``counts``) and advance ctx_lens (device int32) when ``advance``."""
        s = self.shape
        shape = k_new.shape
        if len(shape) != 4 or shape[0] != s.batch or shape[2] != s.kv_heads or shape[3] != s.head_dim:
            raise ValueError(f"k_new: shape {tuple(k_new.shape)}, expected [{s.batch}, rows, {s.kv_heads}, "
                             f"{s.head_dim}]")
        n = k_new.numel()
        kn, vn, lens, cnt = self._rows_args(k_new, v_new, n, ctx_lens, counts, ("k_new", "v_new", "counts"))
        _check(lib().tt_kv_append_mx(self._h, kn, vn, shape[1], cnt, cache._fits(self), lens,
                                     int(bool(advance)), self._on(stream)), "tt_kv_append_mx")

    def kv_read_mx(self, cache, ctx_lens, starts, k_out, v_out, stream=None):
        """Positions [starts[n], starts[n] + rows) below ctx_lens[n] back as bf16 into k_out/v_out
        [B, Hkv, rows, D] (``starts`` None: 0); other rows are left as they were."""
        s = self.shape
        shape = k_out.shape
        if len(shape) != 4 or shape[0] != s.batch or shape[1] != s.kv_heads or shape[3] != s.head_dim:
            raise ValueError(f"k_out: shape {tuple(k_out.shape)}, expected [{s.batch}, {s.kv_heads}, rows, "
                             f"{s.head_dim}]")
        n = k_out.numel()
        ko, vo, lens, st = self._rows_args(k_out, v_out, n, ctx_lens, starts, ("k_out", "v_out", "starts"))
        _check(lib().tt_kv_read_mx(self._h, cache._fits(self), lens, st, shape[2], ko, vo, self._on(stream)),
               "tt_kv_read_mx")
        return k_out, v_out

    def block_attn_host(self, q, k_ctx, v_ctx, k_blk, v_blk, ctx_lens, out, lse=None, stream=None):
        """Host (ideally pinned) CPU tensors in and out; copies happen inside the library."""
        _args("host", *self._decode_items(q, k_blk, v_blk, ctx_lens, out, lse), *self._slab_items(k_ctx, v_ctx))
        _check(lib().tt_block_attn_host(self._h, _ptr(q), _ptr(k_ctx), _ptr(v_ctx), _ptr(k_blk), _ptr(v_blk),
                                        _ptr(ctx_lens), _ptr(out), _ptr(lse), self._on(stream)),
               "tt_block_attn_host")
        return out

    # --- block-causal ------------------------------------------------------
    def block_attn_block_causal(self, q, k_ctx, v_ctx, k_blk, v_blk, out=None, lse=None, stream=None,
                                want_lse=False):
        out, lse = self._outputs(q, out, lse, want_lse, self.shape.seq_len)
        want = self._usual_causal
        x, w = (q, k_ctx, v_ctx, k_blk, v_blk, out), want[0] + ((self.out_dtype, want[0][0][1]),)
        if lse is None:
            at = _quick(self.device, x, w)
            if at is not None:
                at.append(None)
        else:
            at = _quick(self.device, x + (lse,), w + (want[1],))
        q_, kc, vc, kb, vb, o, l = at or _addrs(
            self.device, self._causal_items(q, k_ctx, v_ctx, k_blk, v_blk, out, lse, self._out_kind()))
        _check(lib().tt_block_attn_block_causal(self._h, q_, kc, vc, kb, vb, o, l, self._on(stream)),
               "tt_block_attn_block_causal")
        return (out, lse) if lse is not None else out

    @functools.cached_property
    def _usual_causal(self):
        """What _quick wants of q, k_ctx, v_ctx, k_blk and v_blk of a block-causal call, and of its lse."""
        s = self.shape
        n, b = s.batch * s.seq_len, torch.bfloat16
        k = (b, n * s.kv_heads * s.head_dim)
        return ((b, n * s.q_heads * s.head_dim), k, k, k, k), (torch.float32, n * s.q_heads)

    def _causal_items(self, q, k_ctx, v_ctx, k_blk, v_blk, out, lse, out_kind="f32"):
        s = self.shape
        nq = s.batch * s.seq_len * s.q_heads * s.head_dim
        nk = s.batch * s.seq_len * s.kv_heads * s.head_dim
        return ((q, "q", nq, "bf16"), (k_ctx, "k_ctx", nk, "bf16"), (v_ctx, "v_ctx", nk, "bf16"),
                (k_blk, "k_blk", nk, "bf16"), (v_blk, "v_blk", nk, "bf16"), (out, "out", nq, out_kind),
                (lse, "lse", s.batch * s.q_heads * s.seq_len, "f32"))

    def block_causal_backward(self, q, k_ctx, v_ctx, k_blk, v_blk, out, lse, dout, dq=None, dk_blk=None,
                              dv_blk=None, stream=None):
        """Gradients (dq, dk_blk, dv_blk) of sum(dout * out) for the block-causal attention;
        out and lse are the forward's outputs (fp32), dout is bf16."""
        s = self.shape
        if dq is None:
            dq = torch.empty((s.batch, s.seq_len, s.q_heads, s.head_dim), dtype=torch.float32, device=q.device)
        if dk_blk is None:
            dk_blk = torch.empty((s.batch, s.seq_len, s.kv_heads, s.head_dim), dtype=torch.float32,
                                 device=q.device)
        if dv_blk is None:
            dv_blk = torch.empty_like(dk_blk)
        nq = s.batch * s.seq_len * s.q_heads * s.head_dim
        nk = s.batch * s.seq_len * s.kv_heads * s.head_dim
        want, f = self._usual_causal, torch.float32
        at = _quick(self.device, (q, k_ctx, v_ctx, k_blk, v_blk, out, lse, dout, dq, dk_blk, dv_blk),
                    want[0] + ((f, nq), want[1], (torch.bfloat16, nq), (f, nq), (f, nk), (f, nk)))
        q_, kc, vc, kb, vb, o, l, do, dq_, dk, dv = at or _addrs(
            self.device, self._causal_items(q, k_ctx, v_ctx, k_blk, v_blk, out, lse)
            + ((dout, "dout", nq, "bf16"), (dq, "dq", nq, "f32"), (dk_blk, "dk_blk", nk, "f32"),
               (dv_blk, "dv_blk", nk, "f32")))
        _check(lib().tt_block_attn_block_causal_backward(self._h, q_, kc, vc, kb, vb, o, l, do, dq_, dk, dv,
                                                         self._on(stream)), "tt_block_attn_block_causal_backward")
        return dq, dk_blk, dv_blk

    # --- committed-block cache update ------------------------------------------
    def kv_append(self, k_new, v_new, k_ctx, v_ctx, ctx_lens, advance=True, stream=None):
        """Write k_new/v_new [B,S,Hkv,D] into k_ctx/v_ctx [B,Hkv,Lcap,D] at [L_n, L_n+S) in
        place; advance ctx_lens (device int32) by S when `advance`."""
        s = self.shape
        nb = s.batch * s.block * s.kv_heads * s.head_dim
        usual = self._usual
        at = _quick(self.device, (k_new, v_new, k_ctx, v_ctx, ctx_lens), usual[0][1:3] + usual[1] + usual[0][3:4])
        kn, vn, kc, vc, lens = at or _addrs(
            self.device, ((k_new, "k_new", nb, "bf16"), (v_new, "v_new", nb, "bf16"))
            + self._slab_items(k_ctx, v_ctx) + ((ctx_lens, "ctx_lens", s.batch, "i32"),))
        _check(lib().tt_kv_append(self._h, kn, vn, kc, vc, lens, int(bool(advance)), self._on(stream)),
               "tt_kv_append")

    # --- status / timing ---------------------------------------------------
    def check(self, stream=None):
        """Synchronise and read the device error word; raise TTError on a device-side error."""
        _check(lib().tt_block_attn_check(self._h, self._on(stream)), "tt_block_attn_check")

    def check_status(self, stream=None) -> int:
        return lib().tt_block_attn_check(self._h, self._on(stream))

    def profile(self, enable: bool):
        _check(lib().tt_block_attn_profile(self._h, int(enable)), "tt_block_attn_profile")

    def profile_read(self, kernel_id: int):
        n = ctypes.c_int()
        ms = ctypes.c_double()
        _check(lib().tt_block_attn_profile_read(self._h, kernel_id, ctypes.byref(n), ctypes.byref(ms)),
               "tt_block_attn_profile_read")
        return n.value, ms.value


def confidence_unmask(logits, tokens, masked, gamma=0.8, min_one=True, stream=None):
    """One unmasking step on CUDA tensors: logits [B,S,V] bf16, tokens [B,S] int32 and
    masked [B,S] uint8 (updated in place).  Returns (p_max [B,S] fp32, argmax [B,S] int32,
    n_committed [B] int32)."""
    B, S, V = logits.shape
    dev = logits.device.index if logits.device.index is not None else torch.cuda.current_device()
    _args(dev, (logits, "logits", B * S * V, "bf16"), (tokens, "tokens", B * S, "i32"),
          (masked, "masked", B * S, "u8"))
    p_max = torch.empty((B, S), dtype=torch.float32, device=logits.device)
    arg = torch.empty((B, S), dtype=torch.int32, device=logits.device)
    n_c = torch.empty((B,), dtype=torch.int32, device=logits.device)
    lib().tt_confidence_unmask.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_float,
                                           ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                           ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]
    _check(lib().tt_confidence_unmask(_ptr(logits), B, S, V, float(gamma), int(bool(min_one)), _ptr(tokens),
                                      _ptr(masked), _ptr(p_max), _ptr(arg), _ptr(n_c), _stream(stream)),
           "tt_confidence_unmask")
    return p_max, arg, n_c


_plans = {}


def _cached_plan(key, **kw):
    p = _plans.get(key)
    if p is None:
        p = Plan(**kw)
        _plans[key] = p
    return p


def block_attn(q, k_ctx, v_ctx, k_blk, v_blk, ctx_lens, scale=0.0, kernel=KERNEL_AUTO, want_lse=False):
    """Decode block attention on torch CUDA tensors (shapes as in the C header)."""
    B, S, Hq, D = q.shape
    Hkv, Lcap = k_ctx.shape[1], k_ctx.shape[2]
    dev = q.device.index if q.device.index is not None else torch.cuda.current_device()
    key = ("dec", B, S, Hq, Hkv, D, Lcap, float(scale), kernel, dev)
    plan = _cached_plan(key, batch=B, q_heads=Hq, kv_heads=Hkv, head_dim=D, block=S, ctx_capacity=Lcap,
                        scale=scale, kernel=kernel, device=dev)
    return plan.block_attn(q, k_ctx, v_ctx, k_blk, v_blk, ctx_lens, want_lse=want_lse)


def block_attn_block_causal(q, k_ctx, v_ctx, k_blk, v_blk, block_size, scale=0.0, kernel=KERNEL_AUTO,
                            want_lse=False):
    B, N, Hq, D = q.shape
    Hkv = k_ctx.shape[1]
    dev = q.device.index if q.device.index is not None else torch.cuda.current_device()
    key = ("bc", B, N, block_size, Hq, Hkv, D, float(scale), kernel, dev)
    plan = _cached_plan(key, batch=B, q_heads=Hq, kv_heads=Hkv, head_dim=D, block=block_size, seq_len=N,
                        scale=scale, kernel=kernel, device=dev)
    return plan.block_attn_block_causal(q, k_ctx, v_ctx, k_blk, v_blk, want_lse=want_lse)


def selftest_wait_timeout(device=0, timeout_us=20000, stream=None) -> int:
    return lib().tt_selftest_wait_timeout(int(device), int(timeout_us), _stream(stream))


def selftest_exp2(x, device=0):
    """The softmax's FMA-pipe exp2 evaluated on the device for float32 values x."""
    import numpy as np
    x = np.ascontiguousarray(x, dtype=np.float32)
    y = np.empty_like(x)
    _check(lib().tt_selftest_exp2(int(device), x.ctypes.data, y.ctypes.data, x.size), "tt_selftest_exp2")
    return y


def work_split(tiles_per_unit, num_ctas):
    """Host-only: the library's range split for the given per-unit tile counts."""
    n = len(tiles_per_unit)
    tiles = (ctypes.c_int * max(n, 1))(*tiles_per_unit)
    starts = (ctypes.c_longlong * (num_ctas + 1))()
    first = (ctypes.c_int * max(n, 1))()
    last = (ctypes.c_int * max(n, 1))()
    _check(lib().tt_debug_work_split(n, tiles, num_ctas, starts, first, last), "tt_debug_work_split")
    return list(starts), list(first)[:n], list(last)[:n]


def causal_split(batch, num_kv_heads, seq_len, block_size, key_tile, num_ctas, unit_cost=-1, window=0, sinks=0):
    """Host-only: the range boundaries of a block-causal call on the default tcgen05 kernel
    (unit_cost -1: the library's default fixed cost per unit; 0: the even split)."""
    starts = (ctypes.c_longlong * (num_ctas + 1))()
    _check(lib().tt_debug_causal_split_window(batch, num_kv_heads, seq_len, block_size, key_tile, num_ctas, unit_cost,
                                              window, sinks, starts), "tt_debug_causal_split")
    return list(starts)


def decode_split(seq_tiles, num_kv_heads, num_ctas, unit_cost=0, whole_tiles=0):
    """Host-only: the split of a decode call over sequences whose units have seq_tiles[n] tiles, as (range
    boundaries, cost taken, [(range, unit, first tile, end tile, slot or -1)], [(cut unit or -1, last range,
    first slot) of each range])."""
    n = len(seq_tiles)
    most = n * num_kv_heads + num_ctas
    starts, rec = (ctypes.c_longlong * (num_ctas + 1))(), (ctypes.c_int * (3 * num_ctas))()
    seg, cost, num = (ctypes.c_int * (5 * most))(), ctypes.c_int(), ctypes.c_int()
    _check(lib().tt_debug_decode_split(n, (ctypes.c_int * n)(*seq_tiles), num_kv_heads, num_ctas, unit_cost,
                                       whole_tiles, starts, rec, most, seg, ctypes.byref(cost), ctypes.byref(num)),
           "tt_debug_decode_split")
    return (list(starts), cost.value, [tuple(seg[5 * i:5 * i + 5]) for i in range(num.value)],
            [tuple(rec[3 * c:3 * c + 3]) for c in range(num_ctas)])


def mx_scale_words(head_dim, page_size, slice_rows, count):
    """Host-only: the copies of one tile's scale bytes of a quantised cache, as (byte of the buffer, byte
    offset in the scales, bytes), and the byte of the buffer where its first row's scales lie."""
    rows = (ctypes.c_int * len(slice_rows))(*slice_rows)
    at, num, first = (ctypes.c_longlong * 64)(), (ctypes.c_int * 64)(), ctypes.c_int()
    _check(lib().tt_debug_mx_scale_words(head_dim, page_size, rows, count, at, num, ctypes.byref(first)),
           "tt_debug_mx_scale_words")
    return [(4 * w, at[w], num[w]) for w in range(64) if num[w]], first.value


def block_attn_noalloc(q, k_ctx, v_ctx, k_blk, v_blk, ctx_lens, out, lse=None, status=None, scale=0.0,
                       kernel=KERNEL_AUTO, num_ctas=0, stream=None):
    """Decode through tt_block_attn_noalloc: no plan, no device allocation inside the
    library (its scratch is a fixed 40 MiB device array).  Outputs are caller-owned;
    `status` is an optional one-element uint32/int32 device tensor for the error bits."""
    B, S, Hq, D = q.shape
    Hkv, Lcap = k_ctx.shape[1], k_ctx.shape[2]
    dev = q.device.index if q.device.index is not None else torch.cuda.current_device()
    _args(dev, (q, "q", B * S * Hq * D, "bf16"), (k_ctx, "k_ctx", B * Hkv * Lcap * D, "bf16"),
          (v_ctx, "v_ctx", B * Hkv * Lcap * D, "bf16"), (k_blk, "k_blk", B * S * Hkv * D, "bf16"),
          (v_blk, "v_blk", B * S * Hkv * D, "bf16"), (ctx_lens, "ctx_lens", B, "i32"),
          (out, "out", B * S * Hq * D, "f32"), (lse, "lse", B * Hq * S, "f32"), (status, "status", 1, "w32"))
    d = Desc(B, Hq, Hkv, D, S, Lcap, 0, float(scale), kernel, num_ctas, 0, 0)
    return lib().tt_block_attn_noalloc(ctypes.byref(d), _ptr(q), _ptr(k_ctx), _ptr(v_ctx), _ptr(k_blk),
                                       _ptr(v_blk), _ptr(ctx_lens), _ptr(out), _ptr(lse), _ptr(status),
                                       _stream(stream))
