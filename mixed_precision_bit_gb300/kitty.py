"""ctypes binding of libkitty.so (C ABI in include/kitty.h).

Argument marshalling only: every step runs in the library's CUDA kernels.
Tensors are torch tensors on the GPU (their data pointers are passed through);
the stream defaults to torch's current stream.  There is no fallback: if the
library cannot be built or loaded, the calls raise.
"""

from __future__ import annotations

import ctypes
import dataclasses
import os

from . import build as _build

OK = 0
ERR = {-1: "KITTY_ERR_INVALID_ARG", -2: "KITTY_ERR_UNSUPPORTED", -3: "KITTY_ERR_CUDA",
       -4: "KITTY_ERR_WORKSPACE", -5: "KITTY_ERR_OOM"}
ST = dict(OK=0, EMPTY=1, RANGE=2, NONFINITE=3, BAD_PAGE=4, BAD_LEN=5, TAIL_FULL=6,
          BAD_FLUSH=7, TABLE_FULL=8, BAD_SEQ=9, TIMEOUT=10, NO_PAGES=11, BAD_TREE=12)
F16, BF16, F32 = 0, 1, 2
RANK_PAGE, RANK_RUNNING, RANK_SEQUENCE = 0, 1, 2
D = 128  # channels of a head
ROPE_HALF, ROPE_INTERLEAVED = 0, 1
MAX_NODES = 64  # drafted tokens of a tree
ROPE_PLAIN, ROPE_LINEAR, ROPE_NTK, ROPE_YARN, ROPE_BANDS = 0, 1, 2, 3, 4


class KittyError(RuntimeError):
    def __init__(self, fn, code):
        super().__init__("%s returned %s (%d)" % (fn, ERR.get(code, "?"), code))
        self.code = code


class _Cfg(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "head_dim", "num_kv_heads", "num_q_heads", "page_tokens", "n_hi", "hi_bit", "lo_bit",
        "v_group", "rank_mode", "in_dtype", "decode_pages_per_split", "decode_total_pages",
        "decode_max_pages", "decode_wait_polls", "v_bit")]


@dataclasses.dataclass
class Config:
    num_kv_heads: int
    num_q_heads: int
    n_hi: int = 32
    in_dtype: int = BF16
    rank_mode: int = RANK_PAGE
    decode_pages_per_split: int = 0
    decode_total_pages: int = 0     # planning hint: the batch's total page count (0: unknown)
    decode_max_pages: int = 0       # planning hint: the longest sequence's page count (0: unknown)
    decode_wait_polls: int = 0      # bound of the decode page waits in polls (0: the library's)
    head_dim: int = 128
    page_tokens: int = 32
    hi_bit: int = 4
    lo_bit: int = 2
    v_group: int = 32
    v_bit: int = 2                  # Value code width: 2, or 4 with lo_bit 4

    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        self.__dict__.pop("_ref", None)

    def __getstate__(self):
        return {k: v for k, v in self.__dict__.items() if k != "_ref"}

    def ref(self):
        """A reference to the C structure, kept until a field changes."""
        r = self.__dict__.get("_ref")
        if r is None:
            r = self.__dict__["_ref"] = ctypes.byref(self.c())
        return r

    def c(self):
        return _Cfg(self.head_dim, self.num_kv_heads, self.num_q_heads, self.page_tokens,
                    self.n_hi, self.hi_bit, self.lo_bit, self.v_group, self.rank_mode,
                    self.in_dtype, self.decode_pages_per_split, self.decode_total_pages,
                    self.decode_max_pages, self.decode_wait_polls, self.v_bit)


class _Rope(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("amplitude", ctypes.c_float), ("eps", ctypes.c_float), ("turns", ctypes.c_void_p),
                ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p)]


class _RopeScaling(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("trained", ctypes.c_int32), ("factor", ctypes.c_double),
                ("fast", ctypes.c_double), ("slow", ctypes.c_double)]


_lib = None
EXPORTS = ("kitty_abi_version", "kitty_page_bytes", "kitty_avg_bits", "kitty_alloc_create",
           "kitty_alloc_pages", "kitty_free_pages", "kitty_alloc_free_count",
           "kitty_alloc_destroy", "kitty_quantize_pages", "kitty_append_token",
           "kitty_decode_workspace_bytes", "kitty_decode_attention", "kitty_decode_plan",
           "kitty_decode_attention_noalloc", "kitty_append_decode", "kitty_f16kv_page_bytes",
           "kitty_f16kv_write_pages", "kitty_f16kv_append", "kitty_f16kv_workspace_bytes",
           "kitty_f16kv_decode", "kitty_rope_frequencies", "kitty_rope_turns", "kitty_norm_rope",
           "kitty_append_rope", "kitty_f16kv_append_rope", "kitty_shared_workspace_bytes",
           "kitty_decode_attention_shared", "kitty_f16kv_shared_workspace_bytes",
           "kitty_f16kv_decode_shared", "kitty_tree_plan", "kitty_page_tables",
           "kitty_tree_workspace_bytes", "kitty_tree_attention", "kitty_f16kv_tree_workspace_bytes",
           "kitty_f16kv_tree_attention", "kitty_tree_commit", "kitty_f16kv_tree_commit")
NOALLOC_SCRATCH_BYTES = 8 << 20


def lib_path() -> str:
    return _build.LIB


def load():
    """Load libkitty.so, building it first if it is missing or stale."""
    global _lib
    if _lib is None:
        path = _build.build()
        L = ctypes.CDLL(path)
        P, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        C = ctypes.POINTER(_Cfg)
        sig = {
            "kitty_abi_version": (ctypes.c_int, []),
            "kitty_page_bytes": (ctypes.c_int, [C, ctypes.POINTER(sz), ctypes.POINTER(sz)]),
            "kitty_avg_bits": (ctypes.c_float, [C]),
            "kitty_alloc_create": (ctypes.c_int, [i32, ctypes.POINTER(P)]),
            "kitty_alloc_pages": (ctypes.c_int, [P, i32, P]),
            "kitty_free_pages": (ctypes.c_int, [P, i32, P]),
            "kitty_alloc_free_count": (i32, [P]),
            "kitty_alloc_destroy": (None, [P]),
            "kitty_quantize_pages": (ctypes.c_int, [C, P, P, i32, P, P, i32, P, P, P, P, i32, P, P]),
            "kitty_append_token": (ctypes.c_int, [C, P, P, P, P, P, P, P, P, P, P, i32, P, P, i32,
                                                  i32, P, P]),
            "kitty_decode_workspace_bytes": (ctypes.c_int, [C, i32, i32, ctypes.POINTER(sz)]),
            "kitty_decode_attention": (ctypes.c_int, [C, P, P, i32, P, i32, P, P, P, P,
                                                      ctypes.c_float, P, i32, P, sz, i32, P, P]),
            "kitty_decode_attention_noalloc": (ctypes.c_int, [C, P, P, i32, P, i32, P, P, P, P,
                                                              ctypes.c_float, P, i32, i32, P, P]),
            "kitty_append_decode": (ctypes.c_int, [C, P, P, P, P, P, P, P, P, P, P, P, i32, P, P, i32,
                                                   ctypes.c_float, P, i32, P, sz, i32, P, P]),
            "kitty_decode_plan": (ctypes.c_int, [C, i32, i32, ctypes.POINTER(i32),
                                                 ctypes.POINTER(i32)]),
            "kitty_f16kv_page_bytes": (ctypes.c_int, [C, ctypes.POINTER(sz), ctypes.POINTER(sz)]),
            "kitty_f16kv_write_pages": (ctypes.c_int, [C, P, P, i32, P, P, i32, P, P]),
            "kitty_f16kv_append": (ctypes.c_int, [C, P, P, P, i32, P, i32, P, P, i32, P, P]),
            "kitty_f16kv_workspace_bytes": (ctypes.c_int, [C, i32, i32, ctypes.POINTER(sz)]),
            "kitty_rope_frequencies": (ctypes.c_int, [i32, ctypes.c_double, ctypes.POINTER(_RopeScaling),
                                                      P, ctypes.POINTER(ctypes.c_double)]),
            "kitty_rope_turns": (ctypes.c_int, [P, i32, P]),
            "kitty_norm_rope": (ctypes.c_int, [C, ctypes.POINTER(_Rope), P, i64, P, i64, P, i32, P,
                                               i64, P, i64, P]),
            "kitty_append_rope": (ctypes.c_int, [C, ctypes.POINTER(_Rope), P, i64, P, i64, P, i64, P,
                                                 i64, P, P, P, P, P, P, P, P, i32, P, P, i32, P, i32,
                                                 i32, P, P]),
            "kitty_f16kv_append_rope": (ctypes.c_int, [C, ctypes.POINTER(_Rope), P, i64, P, i64, P,
                                                       i64, i32, P, i64, P, i32, P, i32, P, P, P, P,
                                                       i32, i32, P, P]),
            "kitty_shared_workspace_bytes": (ctypes.c_int, [C, i32, i32, i32, ctypes.POINTER(sz)]),
            "kitty_decode_attention_shared": (ctypes.c_int, [C, P, P, i32, P, i32, P, P, i32, P, P, P,
                                                             P, ctypes.c_float, P, i32, P, sz, i32, P,
                                                             P]),
            "kitty_f16kv_shared_workspace_bytes": (ctypes.c_int, [C, i32, i32, i32,
                                                                  ctypes.POINTER(sz)]),
            "kitty_f16kv_decode_shared": (ctypes.c_int, [C, P, P, i32, P, i32, P, P, i32, P,
                                                         ctypes.c_float, P, i32, P, sz, i32, P, P]),
            "kitty_f16kv_decode": (ctypes.c_int, [C, P, P, i32, P, i32, P, ctypes.c_float, P, i32,
                                                  P, sz, i32, P, P]),
            "kitty_tree_plan": (ctypes.c_int, [P, P, i32, P, P, P, P, P, i32, P, P]),
            "kitty_page_tables": (ctypes.c_int, [P, P, P, i32, i32, i32, i32, P, P, i32, P, P, i32, P, P,
                                                 i32, P, P]),
            "kitty_tree_workspace_bytes": (ctypes.c_int, [C, i32, i32, i32, i32, i32, ctypes.POINTER(sz)]),
            "kitty_f16kv_tree_workspace_bytes": (ctypes.c_int, [C, i32, i32, i32, i32, i32,
                                                                ctypes.POINTER(sz)]),
            "kitty_tree_attention": (ctypes.c_int, [C, P, i64, P, i64, P, i64, i32, P, P, i32, P, i32, P,
                                                    i32, P, P, i32, P, P, P, P, ctypes.c_float, P, i32, P,
                                                    sz, i32, P, P]),
            "kitty_f16kv_tree_attention": (ctypes.c_int, [C, P, i64, P, i64, P, i64, i32, P, P, i32, P, i32,
                                                          P, i32, P, P, i32, P, ctypes.c_float, P, i32, P,
                                                          sz, i32, P, P]),
            "kitty_tree_commit": (ctypes.c_int, [C, P, i64, P, i64, i32, P, P, i32, P, P, P, P, P, P, P, P,
                                                 i32, P, P, i32, i32, i32, P, P]),
            "kitty_f16kv_tree_commit": (ctypes.c_int, [C, P, i64, P, i64, i32, P, P, i32, P, P, i32, P, i32,
                                                       P, i32, i32, P, P]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _chk(name, rc):
    if rc != OK:
        raise KittyError(name, rc)


def _ptr(t):
    """Device address of a tensor argument.  The library reads and writes plain
    dense arrays in device memory, so a view with gaps or a host tensor is
    refused here (it would be read wrongly, or fault)."""
    if t is None:
        return None
    if isinstance(t, int):
        return ctypes.c_void_p(t)
    if not t.is_cuda:
        raise ValueError("kitty: tensor arguments must be in device memory (got %s)" % t.device)
    if not t.is_contiguous():
        raise ValueError("kitty: tensor arguments must be contiguous (shape %s, strides %s)"
                         % (tuple(t.shape), t.stride()))
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        import torch
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def page_bytes(cfg: Config):
    b, p = ctypes.c_size_t(), ctypes.c_size_t()
    _chk("kitty_page_bytes", load().kitty_page_bytes(ctypes.byref(cfg.c()), ctypes.byref(b),
                                                     ctypes.byref(p)))
    return b.value, p.value


def avg_bits(cfg: Config) -> float:
    return float(load().kitty_avg_bits(ctypes.byref(cfg.c())))


class PageAllocator:
    """Host free list of physical page ids (kitty_alloc_*)."""

    def __init__(self, num_pages: int):
        h = ctypes.c_void_p()
        _chk("kitty_alloc_create", load().kitty_alloc_create(num_pages, ctypes.byref(h)))
        self._h = h

    def alloc(self, n: int):
        import numpy as np
        out = np.zeros(n, np.int32)
        _chk("kitty_alloc_pages", load().kitty_alloc_pages(self._h, n, out.ctypes.data))
        return out

    def free(self, ids):
        import numpy as np
        ids = np.ascontiguousarray(ids, np.int32)
        _chk("kitty_free_pages", load().kitty_free_pages(self._h, ids.size, ids.ctypes.data))

    @property
    def free_count(self) -> int:
        return int(load().kitty_alloc_free_count(self._h))

    def close(self):
        if self._h:
            load().kitty_alloc_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def quantize_pages(cfg: Config, k, v, page_ids, pool, pool_pages: int, seq_of_page=None,
                   n_seqs: int = 0, run_sum=None, run_sumsq=None, run_count=None, status=None,
                   stream=None):
    n_pages = page_ids.numel()
    _chk("kitty_quantize_pages", load().kitty_quantize_pages(
        ctypes.byref(cfg.c()), _ptr(k), _ptr(v), n_pages, _ptr(page_ids), _ptr(seq_of_page),
        n_seqs, _ptr(run_sum), _ptr(run_sumsq), _ptr(run_count), _ptr(pool), pool_pages,
        _ptr(status), _stream(stream)))


def append_token(cfg: Config, k_new, v_new, tail_k, tail_v, tail_len, run_sum, run_sumsq,
                 run_count, flush_page_ids, block_table, num_pages, pool, pool_pages: int,
                 status=None, stream=None):
    B = tail_len.numel()
    _chk("kitty_append_token", load().kitty_append_token(
        ctypes.byref(cfg.c()), _ptr(k_new), _ptr(v_new), _ptr(tail_k), _ptr(tail_v),
        _ptr(tail_len), _ptr(run_sum), _ptr(run_sumsq), _ptr(run_count), _ptr(flush_page_ids),
        _ptr(block_table), block_table.shape[1], _ptr(num_pages), _ptr(pool), pool_pages, B,
        _ptr(status), _stream(stream)))


def decode_workspace_bytes(cfg: Config, B: int, max_pages: int) -> int:
    n = ctypes.c_size_t()
    _chk("kitty_decode_workspace_bytes", load().kitty_decode_workspace_bytes(
        ctypes.byref(cfg.c()), B, max_pages, ctypes.byref(n)))
    return n.value


def decode_plan(cfg: Config, B: int, max_pages: int):
    s, c = ctypes.c_int32(), ctypes.c_int32()
    _chk("kitty_decode_plan", load().kitty_decode_plan(ctypes.byref(cfg.c()), B, max_pages,
                                                       ctypes.byref(s), ctypes.byref(c)))
    return s.value, c.value


def decode_attention(cfg: Config, q, pool, pool_pages: int, block_table, num_pages, tail_k,
                     tail_v, tail_len, sm_scale: float, out, workspace=None, status=None,
                     stream=None, out_dtype=None):
    import torch
    B = num_pages.numel()
    if out_dtype is None:
        out_dtype = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}[out.dtype]
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _chk("kitty_decode_attention", load().kitty_decode_attention(
        ctypes.byref(cfg.c()), _ptr(q), _ptr(pool), pool_pages, _ptr(block_table),
        block_table.shape[1], _ptr(num_pages), _ptr(tail_k), _ptr(tail_v), _ptr(tail_len),
        float(sm_scale), _ptr(out), out_dtype, _ptr(workspace), ws_bytes, B, _ptr(status),
        _stream(stream)))


def decode_attention_noalloc(cfg: Config, q, pool, pool_pages: int, block_table, num_pages,
                             tail_k, tail_v, tail_len, sm_scale: float, out, status=None,
                             stream=None, out_dtype=None):
    """kitty_decode_attention without a workspace: the library keeps the split-K
    partials in its own fixed device array (no allocation during the call)."""
    import torch
    B = num_pages.numel()
    if out_dtype is None:
        out_dtype = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}[out.dtype]
    _chk("kitty_decode_attention_noalloc", load().kitty_decode_attention_noalloc(
        ctypes.byref(cfg.c()), _ptr(q), _ptr(pool), pool_pages, _ptr(block_table),
        block_table.shape[1], _ptr(num_pages), _ptr(tail_k), _ptr(tail_v), _ptr(tail_len),
        float(sm_scale), _ptr(out), out_dtype, B, _ptr(status), _stream(stream)))


def append_decode(cfg: Config, k_new, v_new, q, tail_k, tail_v, tail_len, run_sum, run_sumsq,
                  run_count, flush_page_ids, block_table, num_pages, pool, pool_pages: int,
                  sm_scale: float, out, workspace=None, status=None, stream=None, out_dtype=None):
    """append_token followed by decode_attention, as one fused launch."""
    import torch
    B = tail_len.numel()
    if out_dtype is None:
        out_dtype = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}[out.dtype]
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _chk("kitty_append_decode", load().kitty_append_decode(
        ctypes.byref(cfg.c()), _ptr(k_new), _ptr(v_new), _ptr(q), _ptr(tail_k), _ptr(tail_v),
        _ptr(tail_len), _ptr(run_sum), _ptr(run_sumsq), _ptr(run_count), _ptr(flush_page_ids),
        _ptr(block_table), block_table.shape[1], _ptr(num_pages), _ptr(pool), pool_pages,
        float(sm_scale), _ptr(out), out_dtype, _ptr(workspace), ws_bytes, B, _ptr(status),
        _stream(stream)))


# ------------------------------------------------------------------ positions
def rope_frequencies(rot_dim: int, base: float = 10000.0, kind: int = ROPE_PLAIN,
                     factor: float = 1.0, trained: int = 0, fast: float = None, slow: float = 1.0):
    """(frequencies, amplitude): radians a position of each of the rot_dim / 2 pairs, in 64
    bits, and the factor on the rotated channels, stretched by `kind` (ROPE_*) to `factor`
    times the `trained` length (kitty_rope_frequencies)."""
    import numpy as np
    if fast is None:
        fast = 32.0 if kind == ROPE_YARN else 4.0
    f = np.zeros(max(rot_dim // 2, 1), np.float64)
    amp = ctypes.c_double()
    sc = _RopeScaling(kind, trained, factor, fast, slow)
    _chk("kitty_rope_frequencies", load().kitty_rope_frequencies(
        rot_dim, base, ctypes.byref(sc), f.ctypes.data, ctypes.byref(amp)))
    return f[:rot_dim // 2], amp.value


class Rope:
    """A position rotation with the norms before it (kitty_rope): the frequencies' table on
    the device, the pairs' layout, and the norms' weights (16-bit [128]; None: not normed).
    inv_freq: radians a position of each pair (rope_frequencies, or a model's own); empty
    for norms alone."""

    def __init__(self, inv_freq, layout: int = ROPE_HALF, amplitude: float = 1.0, q_weight=None,
                 k_weight=None, eps: float = 1e-6, device="cuda"):
        import numpy as np
        import torch
        f = np.ascontiguousarray(inv_freq, np.float64)
        turns = np.zeros(f.size, np.uint64)
        _chk("kitty_rope_turns", load().kitty_rope_turns(f.ctypes.data, f.size, turns.ctypes.data))
        self.rot_dim, self.layout, self.amplitude, self.eps = 2 * f.size, layout, amplitude, eps
        self.q_weight, self.k_weight = q_weight, k_weight
        self.turns = torch.from_numpy(turns.view(np.int64)).to(device)
        for w in (q_weight, k_weight):
            self._check_weight(w)

    @staticmethod
    def _check_weight(w, in_dtype=None):
        if w is not None and (w.numel() != D or w.element_size() != 2):
            raise ValueError("kitty: norm weights are 16-bit [%d]" % D)
        if w is not None:
            _same_type(w, in_dtype)
        _ptr(w)

    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        self.__dict__.pop("_ref", None)

    def __getstate__(self):
        return {k: v for k, v in self.__dict__.items() if k != "_ref"}

    def ref(self, dev: int, in_dtype: int = None):
        """A reference to the C structure of the fields as they are, kept until one changes, a
        tensor's memory moves, or the device or the rows' type does."""
        t, q, k = self.turns, self.q_weight, self.k_weight
        at = (dev, in_dtype, t.data_ptr(), q is not None and q.data_ptr(), k is not None and k.data_ptr())
        r = self.__dict__.get("_ref")
        if r is None or r[0] != at:
            for w in (q, k):
                self._check_weight(w, in_dtype)
            if t.element_size() != 8 or not 0 <= self.rot_dim <= 2 * t.numel():
                raise ValueError("kitty: turns are 64-bit, one of each pair (got %s, %s, rot_dim %d)"
                                 % (tuple(t.shape), t.dtype, self.rot_dim))
            c = _Rope(self.rot_dim, self.layout, self.amplitude, self.eps, _dense(t, dev),
                      _dense(q, dev), _dense(k, dev))
            r = self.__dict__["_ref"] = (at, ctypes.byref(c))
        return r[1]


def _device():
    """The current CUDA device, which the calls below launch on: every tensor must be there."""
    import torch
    return torch.cuda.current_device()


# Each check below is one expression over a tensor's attributes, and says what was wrong only
# when it fails: a call of a few microseconds on the device takes a dozen tensors.
def _here(t, dev: int):
    if t.get_device() != dev:  # -1: host memory
        if not t.is_cuda:
            raise ValueError("kitty: tensor arguments must be in device memory (got %s)" % t.device)
        raise ValueError("kitty: a tensor is on %s, the current device is cuda:%d" % (t.device, dev))


def _dense(t, dev: int):
    """Device address of a dense array on the current device (None: null)."""
    if t is None:
        return None
    if t.get_device() != dev or not t.is_contiguous():
        _here(t, dev)
        raise ValueError("kitty: tensor arguments must be contiguous (shape %s, strides %s)"
                         % (tuple(t.shape), t.stride()))
    return t.data_ptr()


class _RowTypes(dict):
    """Types that 16-bit values may have, by the configuration's input type: its own, or integers
    that hold its bits.  As the other 16-bit type they would be read as other numbers."""

    def __missing__(self, in_dtype):
        import torch
        mine = {F16: (torch.float16,), BF16: (torch.bfloat16,)}.get(in_dtype, (torch.float16, torch.bfloat16))
        self[in_dtype] = frozenset((*mine, torch.int16, torch.uint16))
        return self[in_dtype]


_row_types = _RowTypes()


def _same_type(t, in_dtype: int):
    if t.element_size() == 2 and t.dtype not in _row_types[in_dtype]:
        raise ValueError("kitty: %s values where the configuration has %s"
                         % (t.dtype, "bfloat16" if in_dtype == BF16 else "float16"))


def _rows(t, n: int, heads: int, dev: int, in_dtype: int = None):
    """(device address, elements from token to token) of rows [n, heads, 128]: 16-bit, each
    token's heads dense, any stride between tokens."""
    if t is None:
        return None, 0
    if t.shape != (n, heads, D) or t.dtype not in _row_types[in_dtype]:
        _same_type(t, in_dtype)
        raise ValueError("kitty: expected 16-bit rows [%d, %d, %d] (got %s, %s)"
                         % (n, heads, D, tuple(t.shape), t.dtype))
    s0, s1, s2 = t.stride()
    if s2 != 1 or (s1 != D and heads > 1) or t.get_device() != dev:
        _here(t, dev)
        raise ValueError("kitty: the heads of a token must be contiguous (strides %s)" % (t.stride(),))
    # the stride between tokens of one token says nothing
    return t.data_ptr(), s0 if n > 1 else heads * D


def _tail(t, cfg: Config, B: int, dev: int):
    """Address of tails [>= B, Hkv, 32, 128], 16-bit (None: null)."""
    if t is None:
        return None
    if t.numel() < B * cfg.num_kv_heads * 32 * D or t.dtype not in _row_types[cfg.in_dtype]:
        _same_type(t, cfg.in_dtype)
        raise ValueError("kitty: tails are 16-bit [%d, %d, 32, %d] (got %s, %s)"
                         % (B, cfg.num_kv_heads, D, tuple(t.shape), t.dtype))
    if t.get_device() != dev or not t.is_contiguous():
        _dense(t, dev)
    return t.data_ptr()


def _ints(name: str, t, n: int, dev: int):
    """Address of a dense int32 array of at least n entries (None: null)."""
    if t is None:
        return None
    if t.element_size() != 4 or t.is_floating_point() or t.numel() < n:
        raise ValueError("kitty: %s must be int32 with %d entries (got %s, %s)"
                         % (name, n, tuple(t.shape), t.dtype))
    if t.get_device() != dev or not t.is_contiguous():
        _dense(t, dev)
    return t.data_ptr()


def _table(t, B: int, dev: int):
    """(address, entries of a row) of a block table [>= B, max_pages]."""
    shape = t.shape
    if len(shape) != 2 or shape[0] < B:
        raise ValueError("kitty: the block table must be [%d, max_pages] (got %s)" % (B, tuple(shape)))
    return _ints("block_table", t, 0, dev), shape[1]


def _raw_stream(stream, dev: int):
    """As _stream, for the current device's current stream without making a stream object."""
    if stream is None:
        import torch
        return torch._C._cuda_getCurrentRawStream(dev)
    return stream if isinstance(stream, int) else stream.cuda_stream


def norm_rope(cfg: Config, rope: Rope, q, k, positions, q_out, k_out, stream=None):
    """Per-head norms and the position rotation of queries q [n, Hq, 128] and keys k
    [n, Hkv, 128] at positions [n] into q_out and k_out (which may be q and k); q or k may
    be None.  Rows may be slices of a joint projection (any token stride)."""
    dev, n, dt = _device(), positions.numel(), cfg.in_dtype
    if (q is None) != (q_out is None) or (k is None) != (k_out is None):
        raise ValueError("kitty: rows in need rows out")
    qp, qs = _rows(q, n, cfg.num_q_heads, dev, dt)
    kp, ks = _rows(k, n, cfg.num_kv_heads, dev, dt)
    qo, qos = _rows(q_out, n, cfg.num_q_heads, dev, dt)
    ko, kos = _rows(k_out, n, cfg.num_kv_heads, dev, dt)
    _chk("kitty_norm_rope", load().kitty_norm_rope(
        cfg.ref(), rope.ref(dev, dt), qp, qs, kp, ks, _ints("positions", positions, n, dev), n, qo, qos,
        ko, kos, _raw_stream(stream, dev)))


def append_rope(cfg: Config, rope: Rope, q, k_new, v_new, q_out, tail_k, tail_v, tail_len, run_sum,
                run_sumsq, run_count, flush_page_ids, block_table, num_pages, pool,
                pool_pages: int, pos_base=None, counted: bool = False, status=None, stream=None):
    """append_token with norm and rotation on the way (kitty_append_rope): the rotated query
    rows go to q_out (q and q_out may be None), the rotated key into the tail."""
    dev, B, dt = _device(), tail_len.numel(), cfg.in_dtype
    qp, qs = _rows(q, B, cfg.num_q_heads, dev, dt)
    qo, qos = _rows(q_out, B, cfg.num_q_heads, dev, dt)
    kp, ks = _rows(k_new, B, cfg.num_kv_heads, dev, dt)
    vp, vs = _rows(v_new, B, cfg.num_kv_heads, dev, dt)
    table, max_pages = _table(block_table, B, dev)
    _chk("kitty_append_rope", load().kitty_append_rope(
        cfg.ref(), rope.ref(dev, dt), qp, qs, kp, ks, vp, vs, qo, qos, _tail(tail_k, cfg, B, dev),
        _tail(tail_v, cfg, B, dev), _ints("tail_len", tail_len, B, dev), _dense(run_sum, dev),
        _dense(run_sumsq, dev), _dense(run_count, dev),
        _ints("flush_page_ids", flush_page_ids, B, dev), table, max_pages,
        _ints("num_pages", num_pages, B, dev), _dense(pool, dev), pool_pages,
        _ints("pos_base", pos_base, B, dev), int(counted), B, _dense(status, dev),
        _raw_stream(stream, dev)))


def f16kv_append_rope(cfg: Config, rope: Rope, q, k_new, v_new, q_out, pool, pool_pages: int,
                      block_table, ctx_len, new_page_ids, seq_start=None, pos_base=None,
                      counted: bool = False, status=None, stream=None):
    """Norm, rotation and append into the 16-bit paged cache (kitty_f16kv_append_rope): one
    token a sequence, or the runs that seq_start [B + 1] marks; rows behind the last run
    are left alone."""
    dev, B, n, dt = _device(), ctx_len.numel(), k_new.shape[0], cfg.in_dtype
    qp, qs = _rows(q, n, cfg.num_q_heads, dev, dt)
    qo, qos = _rows(q_out, n, cfg.num_q_heads, dev, dt)
    kp, ks = _rows(k_new, n, cfg.num_kv_heads, dev, dt)
    vp, vs = _rows(v_new, n, cfg.num_kv_heads, dev, dt)
    table, max_pages = _table(block_table, B, dev)
    _chk("kitty_f16kv_append_rope", load().kitty_f16kv_append_rope(
        cfg.ref(), rope.ref(dev, dt), qp, qs, kp, ks, vp, vs, n, qo, qos, _dense(pool, dev), pool_pages,
        table, max_pages, _ints("ctx_len", ctx_len, B, dev),
        _ints("new_page_ids", new_page_ids, n, dev), _ints("seq_start", seq_start, B + 1, dev),
        _ints("pos_base", pos_base, B, dev), int(counted), B, _dense(status, dev),
        _raw_stream(stream, dev)))


# ------------------------------------------------------------------ 16-bit paged baseline
def f16kv_page_bytes(cfg: Config):
    b, p = ctypes.c_size_t(), ctypes.c_size_t()
    _chk("kitty_f16kv_page_bytes", load().kitty_f16kv_page_bytes(
        ctypes.byref(cfg.c()), ctypes.byref(b), ctypes.byref(p)))
    return b.value, p.value


def f16kv_write_pages(cfg: Config, k, v, page_ids, pool, pool_pages: int, status=None,
                      stream=None):
    _chk("kitty_f16kv_write_pages", load().kitty_f16kv_write_pages(
        ctypes.byref(cfg.c()), _ptr(k), _ptr(v), page_ids.numel(), _ptr(page_ids), _ptr(pool),
        pool_pages, _ptr(status), _stream(stream)))


def f16kv_append(cfg: Config, k_new, v_new, pool, pool_pages: int, block_table, ctx_len,
                 new_page_ids, status=None, stream=None):
    _chk("kitty_f16kv_append", load().kitty_f16kv_append(
        ctypes.byref(cfg.c()), _ptr(k_new), _ptr(v_new), _ptr(pool), pool_pages,
        _ptr(block_table), block_table.shape[1], _ptr(ctx_len), _ptr(new_page_ids),
        ctx_len.numel(), _ptr(status), _stream(stream)))


def f16kv_workspace_bytes(cfg: Config, B: int, max_pages: int) -> int:
    n = ctypes.c_size_t()
    _chk("kitty_f16kv_workspace_bytes", load().kitty_f16kv_workspace_bytes(
        ctypes.byref(cfg.c()), B, max_pages, ctypes.byref(n)))
    return n.value


def f16kv_decode(cfg: Config, q, pool, pool_pages: int, block_table, ctx_len, sm_scale: float,
                 out, workspace=None, status=None, stream=None, out_dtype=None):
    import torch
    B = ctx_len.numel()
    if out_dtype is None:
        out_dtype = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}[out.dtype]
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _chk("kitty_f16kv_decode", load().kitty_f16kv_decode(
        ctypes.byref(cfg.c()), _ptr(q), _ptr(pool), pool_pages, _ptr(block_table),
        block_table.shape[1], _ptr(ctx_len), float(sm_scale), _ptr(out), out_dtype,
        _ptr(workspace), ws_bytes, B, _ptr(status), _stream(stream)))


# ------------------------------------------------------------------ shared prefix
def _out_dtype(out):
    import torch
    return {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}[out.dtype]


def _shared_bytes(name, cfg, B, n_prefix, max_pages):
    n = ctypes.c_size_t()
    _chk(name, getattr(load(), name)(ctypes.byref(cfg.c()), B, n_prefix, max_pages, ctypes.byref(n)))
    return n.value


def shared_workspace_bytes(cfg: Config, B: int, n_prefix: int, max_pages: int) -> int:
    return _shared_bytes("kitty_shared_workspace_bytes", cfg, B, n_prefix, max_pages)


def f16kv_shared_workspace_bytes(cfg: Config, B: int, n_prefix: int, max_pages: int) -> int:
    return _shared_bytes("kitty_f16kv_shared_workspace_bytes", cfg, B, n_prefix, max_pages)


def _attended(cfg, q, out, B, dev):
    """Addresses of q (16-bit) and out, both [B, Hq, 128]."""
    shape = (B, cfg.num_q_heads, D)
    if q.shape != shape or out.shape != shape or q.dtype not in _row_types[cfg.in_dtype]:
        _same_type(q, cfg.in_dtype)
        raise ValueError("kitty: q (16-bit) and out must be [%d, %d, %d] (got %s, %s)"
                         % (*shape, tuple(q.shape), tuple(out.shape)))
    return _dense(q, dev), _dense(out, dev)


def decode_attention_shared(cfg: Config, q, pool, pool_pages: int, prefix_table, prefix_pages,
                            block_table, num_pages, tail_k, tail_v, tail_len, sm_scale: float, out,
                            workspace=None, status=None, stream=None):
    """decode_attention of a batch that shares a prefix (kitty_decode_attention_shared):
    sequence b attends the first prefix_pages[b] pages of prefix_table (prefix_pages None: all
    of them), then its own pages and tail."""
    dev, B = _device(), num_pages.numel()
    qp, op = _attended(cfg, q, out, B, dev)
    table, max_pages = _table(block_table, B, dev)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _chk("kitty_decode_attention_shared", load().kitty_decode_attention_shared(
        cfg.ref(), qp, _dense(pool, dev), pool_pages, _ints("prefix_table", prefix_table, 0, dev),
        prefix_table.numel(), _ints("prefix_pages", prefix_pages, B, dev), table, max_pages,
        _ints("num_pages", num_pages, B, dev), _tail(tail_k, cfg, B, dev), _tail(tail_v, cfg, B, dev),
        _ints("tail_len", tail_len, B, dev), float(sm_scale), op, _out_dtype(out),
        _dense(workspace, dev), ws_bytes, B, _dense(status, dev), _raw_stream(stream, dev)))


def f16kv_decode_shared(cfg: Config, q, pool, pool_pages: int, prefix_table, prefix_pages,
                        block_table, ctx_len, sm_scale: float, out, workspace=None, status=None,
                        stream=None):
    """f16kv_decode of a batch that shares a prefix (kitty_f16kv_decode_shared); ctx_len counts
    a sequence's own tokens."""
    dev, B = _device(), ctx_len.numel()
    qp, op = _attended(cfg, q, out, B, dev)
    table, max_pages = _table(block_table, B, dev)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _chk("kitty_f16kv_decode_shared", load().kitty_f16kv_decode_shared(
        cfg.ref(), qp, _dense(pool, dev), pool_pages, _ints("prefix_table", prefix_table, 0, dev),
        prefix_table.numel(), _ints("prefix_pages", prefix_pages, B, dev), table, max_pages,
        _ints("ctx_len", ctx_len, B, dev), float(sm_scale), op, _out_dtype(out),
        _dense(workspace, dev), ws_bytes, B, _dense(status, dev), _raw_stream(stream, dev)))


# ------------------------------------------------------------------ drafted tokens
def _longs(name: str, t, n: int, dev: int):
    """Address of a dense 64-bit integer array of at least n entries (None: null)."""
    if t is None:
        return None
    if t.element_size() != 8 or t.is_floating_point() or t.is_complex() or t.numel() < n:
        raise ValueError("kitty: %s must be 64-bit integers, %d entries (got %s, %s)"
                         % (name, n, tuple(t.shape), t.dtype))
    if t.get_device() != dev or not t.is_contiguous():
        _dense(t, dev)
    return t.data_ptr()


def tree_plan(parents, seq_start, lens, visible, positions, num_pages=None, pos_base=None, status=None,
              stream=None):
    """Ancestor masks (visible, 64-bit [n]) and positions (int32 [n]) of the drafted trees whose
    parents [n] are given as places in the own tree, -1 for a node that follows the cached tokens
    (kitty_tree_plan); seq_start [B + 1] marks the sequences' rows.  visible or positions may be
    None."""
    dev, n, B = _device(), parents.numel(), lens.numel()
    _chk("kitty_tree_plan", load().kitty_tree_plan(
        _ints("parents", parents, n, dev), _ints("seq_start", seq_start, B + 1, dev), n,
        _ints("num_pages", num_pages, B, dev), _ints("lens", lens, B, dev),
        _ints("pos_base", pos_base, B, dev), _longs("visible", visible, n, dev),
        _ints("positions", positions, n, dev), B, _dense(status, dev), _raw_stream(stream, dev)))


def page_tables(lens, held, block_table, free_ids, free_count, num_pages=None, seq_start=None,
                extra: int = 0, partial: bool = True, shrink: bool = False, slots=None,
                new_page_ids=None, status=None, stream=None):
    """Pages for 32 * num_pages + lens tokens of each sequence, the new ones that seq_start [B + 1]
    marks and `extra` more (of these as many as the row has room for), from the stack
    free_ids[:free_count] on the device into the block table, whose rows hold `held` pages; shrink:
    those beyond go back (kitty_page_tables).  slots (64-bit) and new_page_ids (int32), one entry a
    new token, may be None."""
    dev, B = _device(), lens.numel()
    table, max_pages = _table(block_table, B, dev)
    # without a map no rows are written: any starts will do
    n = max((t.numel() for t in (slots, new_page_ids) if t is not None), default=0 if seq_start is None else 0x7FFFFFFF)
    _chk("kitty_page_tables", load().kitty_page_tables(
        _ints("num_pages", num_pages, B, dev), _ints("lens", lens, B, dev),
        _ints("seq_start", seq_start, B + 1, dev), n, extra, int(partial), int(shrink),
        _ints("held", held, B, dev), table, max_pages, _ints("free_ids", free_ids, 0, dev),
        _ints("free_count", free_count, 1, dev), free_ids.numel(), _longs("slots", slots, n, dev),
        _ints("new_page_ids", new_page_ids, n, dev), B, _dense(status, dev), _raw_stream(stream, dev)))


def _tree_bytes(name, cfg, B, n_tokens, max_nodes, n_prefix, max_pages):
    n = ctypes.c_size_t()
    _chk(name, getattr(load(), name)(cfg.ref(), B, n_tokens, max_nodes, n_prefix, max_pages, ctypes.byref(n)))
    return n.value


def tree_workspace_bytes(cfg: Config, B: int, n_tokens: int, max_nodes: int, max_pages: int,
                         n_prefix: int = 0) -> int:
    return _tree_bytes("kitty_tree_workspace_bytes", cfg, B, n_tokens, max_nodes, n_prefix, max_pages)


def f16kv_tree_workspace_bytes(cfg: Config, B: int, n_tokens: int, max_nodes: int, max_pages: int,
                               n_prefix: int = 0) -> int:
    return _tree_bytes("kitty_f16kv_tree_workspace_bytes", cfg, B, n_tokens, max_nodes, n_prefix, max_pages)


def _tree_rows(cfg, q, k, v, out, dev):
    """(rows, the addresses and strides of q, k, v, the address of out [n, Hq, 128])."""
    n = q.shape[0]
    if out.shape != (n, cfg.num_q_heads, D):
        raise ValueError("kitty: out must be [%d, %d, %d] (got %s)" % (n, cfg.num_q_heads, D, tuple(out.shape)))
    return n, (*_rows(q, n, cfg.num_q_heads, dev, cfg.in_dtype), *_rows(k, n, cfg.num_kv_heads, dev, cfg.in_dtype),
               *_rows(v, n, cfg.num_kv_heads, dev, cfg.in_dtype)), _dense(out, dev)


def tree_attention(cfg: Config, q, k, v, seq_start, visible, max_nodes: int, pool, pool_pages: int,
                   block_table, num_pages, tail_k, tail_v, tail_len, sm_scale: float, out,
                   prefix_table=None, prefix_pages=None, workspace=None, status=None, stream=None):
    """Attention of drafted tokens q [n, Hq, 128] to their sequences' cached tokens and to the
    drafted tokens k, v [n, Hkv, 128] of their masks (kitty_tree_attention); seq_start [B + 1]
    marks the sequences' rows, visible (64-bit [n]; None: chains) which nodes each sees."""
    dev, B = _device(), num_pages.numel()
    n, rows, op = _tree_rows(cfg, q, k, v, out, dev)
    table, max_pages = _table(block_table, B, dev)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _chk("kitty_tree_attention", load().kitty_tree_attention(
        cfg.ref(), *rows, n, _ints("seq_start", seq_start, B + 1, dev), _longs("visible", visible, n, dev),
        max_nodes, _dense(pool, dev), pool_pages, _ints("prefix_table", prefix_table, 0, dev),
        0 if prefix_table is None else prefix_table.numel(), _ints("prefix_pages", prefix_pages, B, dev),
        table, max_pages, _ints("num_pages", num_pages, B, dev), _tail(tail_k, cfg, B, dev),
        _tail(tail_v, cfg, B, dev), _ints("tail_len", tail_len, B, dev), float(sm_scale), op,
        _out_dtype(out), _dense(workspace, dev), ws_bytes, B, _dense(status, dev), _raw_stream(stream, dev)))


def f16kv_tree_attention(cfg: Config, q, k, v, seq_start, visible, max_nodes: int, pool, pool_pages: int,
                         block_table, ctx_len, sm_scale: float, out, prefix_table=None, prefix_pages=None,
                         workspace=None, status=None, stream=None):
    """tree_attention over 16-bit pages (kitty_f16kv_tree_attention)."""
    dev, B = _device(), ctx_len.numel()
    n, rows, op = _tree_rows(cfg, q, k, v, out, dev)
    table, max_pages = _table(block_table, B, dev)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _chk("kitty_f16kv_tree_attention", load().kitty_f16kv_tree_attention(
        cfg.ref(), *rows, n, _ints("seq_start", seq_start, B + 1, dev), _longs("visible", visible, n, dev),
        max_nodes, _dense(pool, dev), pool_pages, _ints("prefix_table", prefix_table, 0, dev),
        0 if prefix_table is None else prefix_table.numel(), _ints("prefix_pages", prefix_pages, B, dev),
        table, max_pages, _ints("ctx_len", ctx_len, B, dev), float(sm_scale), op, _out_dtype(out),
        _dense(workspace, dev), ws_bytes, B, _dense(status, dev), _raw_stream(stream, dev)))


def _path(path, path_len, B, dev):
    """(address, entries a row, address of the counts) of accepted paths [>= B, width]."""
    if path.dim() != 2 or path.shape[0] < B:
        raise ValueError("kitty: paths must be [%d, width] (got %s)" % (B, tuple(path.shape)))
    return _ints("path", path, 0, dev), path.shape[1], _ints("path_len", path_len, B, dev)


def tree_commit(cfg: Config, k, v, seq_start, path, path_len, tail_k, tail_v, tail_len, run_sum, run_sumsq,
                run_count, block_table, num_pages, pool, pool_pages: int, counted: bool = False,
                status=None, stream=None):
    """The accepted drafted tokens, rows path[b, :path_len[b]] of each sequence's in k, v
    [n, Hkv, 128], into the packed cache (kitty_tree_commit); full tails are quantized into the
    pages that the block table holds behind num_pages already (page_tables).  path_len of a sequence
    that is refused becomes 0.  counted: lengths shared by several layers, which the first layer's
    call has advanced: the later layers', with the path_len that it left."""
    dev, n, B, dt = _device(), k.shape[0], tail_len.numel(), cfg.in_dtype
    kp, ks = _rows(k, n, cfg.num_kv_heads, dev, dt)
    vp, vs = _rows(v, n, cfg.num_kv_heads, dev, dt)
    table, max_pages = _table(block_table, B, dev)
    _chk("kitty_tree_commit", load().kitty_tree_commit(
        cfg.ref(), kp, ks, vp, vs, n, _ints("seq_start", seq_start, B + 1, dev), *_path(path, path_len, B, dev),
        _tail(tail_k, cfg, B, dev), _tail(tail_v, cfg, B, dev), _ints("tail_len", tail_len, B, dev),
        _dense(run_sum, dev), _dense(run_sumsq, dev), _dense(run_count, dev), table, max_pages,
        _ints("num_pages", num_pages, B, dev), _dense(pool, dev), pool_pages, int(counted), B,
        _dense(status, dev), _raw_stream(stream, dev)))


def f16kv_tree_commit(cfg: Config, k, v, seq_start, path, path_len, pool, pool_pages: int, block_table, ctx_len,
                      counted: bool = False, status=None, stream=None):
    """The accepted drafted tokens into the 16-bit pages that the block table holds
    (kitty_f16kv_tree_commit)."""
    dev, n, B, dt = _device(), k.shape[0], ctx_len.numel(), cfg.in_dtype
    kp, ks = _rows(k, n, cfg.num_kv_heads, dev, dt)
    vp, vs = _rows(v, n, cfg.num_kv_heads, dev, dt)
    table, max_pages = _table(block_table, B, dev)
    _chk("kitty_f16kv_tree_commit", load().kitty_f16kv_tree_commit(
        cfg.ref(), kp, ks, vp, vs, n, _ints("seq_start", seq_start, B + 1, dev), *_path(path, path_len, B, dev),
        _dense(pool, dev), pool_pages, table, max_pages, _ints("ctx_len", ctx_len, B, dev), int(counted), B,
        _dense(status, dev), _raw_stream(stream, dev)))
