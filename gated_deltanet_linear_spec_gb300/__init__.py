"""GB300-native Gated DeltaNet speculative-decoding hot path: Python binding of ``libgdn.so``.

The functions here mirror the C entry points in ``include/gdn.h`` one for one
(``gdn_conv_update``, ``gdn_recurrent_step``, ``gdn_chunk_prefill``, ``gdn_mixed_batch``,
``gdn_workspace_bytes``, and the paged key-value cache's ``gdn_paged_attention``, ``gdn_kv_append``,
``gdn_kv_reserve``, ``gdn_kv_release``, ``gdn_kv_fork``, ``gdn_kv_copy_pages``, ``gdn_kv_compact``,
``gdn_copy_slots``, ``gdn_shared_attention``, ``gdn_kv_common_prefix``, and rotary positions' ``gdn_rope``,
``gdn_kv_append_rope``) and only marshal arguments: torch CUDA tensors become device
pointers, the current torch stream becomes the ``cudaStream_t``, and a negative return code
becomes a ``GdnError``.  Every step of the path runs in the library's CUDA kernels; there is
no fallback, and a missing library raises at the first call.
"""
from __future__ import annotations

import ctypes
import os
import threading
from dataclasses import dataclass
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgdn.so")

GDN_F32, GDN_BF16 = 0, 1
GDN_QKV_PACKED, GDN_QKV_PER_KHEAD = 0, 1
GDN_CONV_ROLLED, GDN_CONV_PER_SLOT = 0, 1
GDN_ROPE_HALF, GDN_ROPE_INTERLEAVED = 0, 1
GDN_ROPE_PLAIN, GDN_ROPE_LINEAR, GDN_ROPE_NTK, GDN_ROPE_BANDS, GDN_ROPE_RAMP = 0, 1, 2, 3, 4
STATUS_SLOT_RANGE, STATUS_NUM_ACCEPTED, STATUS_TOKEN_RANGE, STATUS_ROW_RANGE = 0x1, 0x2, 0x4, 0x8
STATUS_WAIT_TIMEOUT = 0x10
STATUS_PAGE_RANGE, STATUS_PAGE_SHARED, STATUS_NO_PAGES = 0x20, 0x40, 0x80
ERRORS = {-1: "NULL_ARG", -2: "SPEC_PAIR", -3: "SHAPE", -4: "CONSERVATION", -5: "WORKSPACE",
          -6: "DTYPE", -7: "CUDA", -8: "ALIGN"}


class GdnError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{ERRORS.get(code, code)}: {msg}")
        self.code = code
        self.name = ERRORS.get(code, str(code))


class _LayerDesc(ctypes.Structure):
    _fields_ = [("num_k_heads", ctypes.c_int32), ("num_v_heads", ctypes.c_int32),
                ("head_k_dim", ctypes.c_int32), ("head_v_dim", ctypes.c_int32),
                ("conv_width", ctypes.c_int32), ("conv_state_len", ctypes.c_int32),
                ("act_dtype", ctypes.c_int32), ("scale", ctypes.c_float),
                ("qkv_layout", ctypes.c_int32), ("conv_layout", ctypes.c_int32)]


class _LayerParams(ctypes.Structure):
    _fields_ = [("conv_weight", ctypes.c_void_p), ("conv_bias", ctypes.c_void_p),
                ("A_log", ctypes.c_void_p), ("dt_bias", ctypes.c_void_p)]


class _Pools(ctypes.Structure):
    _fields_ = [("conv_pool", ctypes.c_void_p), ("ssm_pool", ctypes.c_void_p), ("num_slots", ctypes.c_int64)]


class _Rows(ctypes.Structure):
    _fields_ = [("num_seqs", ctypes.c_int32), ("num_tokens", ctypes.c_int32),
                ("query_start_loc", ctypes.c_void_p), ("token_indx", ctypes.c_void_p),
                ("state_indices", ctypes.c_void_p), ("has_initial_state", ctypes.c_void_p),
                ("spec_state_indices", ctypes.c_void_p), ("num_accepted_tokens", ctypes.c_void_p),
                ("spec_cols", ctypes.c_int32)]


class _KvCache(ctypes.Structure):
    _fields_ = [("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p), ("page_stride", ctypes.c_int64),
                ("block_table", ctypes.c_void_p), ("refcount", ctypes.c_void_p), ("num_pages", ctypes.c_int32),
                ("num_table_rows", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class _KvRows(ctypes.Structure):
    _fields_ = [("num_seqs", ctypes.c_int32), ("num_tokens", ctypes.c_int32), ("query_start_loc", ctypes.c_void_p),
                ("token_indx", ctypes.c_void_p), ("table_rows", ctypes.c_void_p), ("kv_lens", ctypes.c_void_p),
                ("max_query_len", ctypes.c_int32)]


class _AttnDesc(ctypes.Structure):
    _fields_ = [("num_q_heads", ctypes.c_int32), ("scale", ctypes.c_float), ("window", ctypes.c_int32),
                ("num_sinks", ctypes.c_int32)]


class _KvGroups(ctypes.Structure):
    _fields_ = [("num_groups", ctypes.c_int32), ("group_start_loc", ctypes.c_void_p), ("prefix_lens", ctypes.c_void_p)]


class _RopeDesc(ctypes.Structure):
    _fields_ = [("turns", ctypes.c_void_p), ("rotary_dim", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("magnitude", ctypes.c_float)]


class _RopeFreq(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int32), ("scaling", ctypes.c_int32), ("base", ctypes.c_double),
                ("factor", ctypes.c_double), ("original_len", ctypes.c_double), ("low", ctypes.c_double),
                ("high", ctypes.c_double)]


EXPORTS = ("gdn_workspace_bytes", "gdn_prefill_workspace_bytes", "gdn_conv_update", "gdn_recurrent_step", "gdn_chunk_prefill",
           "gdn_mixed_batch", "gdn_mixed_batch_static_workspace", "gdn_status_string", "gdn_kv_append", "gdn_paged_attention",
           "gdn_attention_workspace_bytes", "gdn_kv_reserve", "gdn_kv_release", "gdn_kv_fork", "gdn_kv_copy_pages",
           "gdn_kv_compact", "gdn_kv_workspace_bytes", "gdn_copy_slots", "gdn_shared_attention",
           "gdn_shared_attention_workspace_bytes", "gdn_kv_common_prefix", "gdn_rope", "gdn_rope_turns", "gdn_rope_turns_of",
           "gdn_kv_append_rope")
# include/gdn_testing.h: hooks that let tests drive the kernels' failure paths
TESTING_EXPORTS = ("gdn_testing_set_prefill_faults", "gdn_testing_set_shared_faults")
STATIC_WORKSPACE_BYTES = 16 << 20

_lib = None
_lock = threading.Lock()


def library() -> ctypes.CDLL:
    """Loads ``libgdn.so`` (built by ``build.py``); raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing: run gated_deltanet_linear_spec_gb300.build first")
            lib = ctypes.CDLL(LIB_PATH)
            P, I32, VP = ctypes.POINTER, ctypes.c_int32, ctypes.c_void_p
            lib.gdn_status_string.restype = ctypes.c_char_p
            lib.gdn_status_string.argtypes = [ctypes.c_int]
            lib.gdn_workspace_bytes.restype = ctypes.c_size_t
            lib.gdn_workspace_bytes.argtypes = [P(_LayerDesc), P(_Rows), P(_Rows)]
            lib.gdn_prefill_workspace_bytes.restype = ctypes.c_size_t
            lib.gdn_prefill_workspace_bytes.argtypes = [P(_LayerDesc), P(_Rows), I32]
            lib.gdn_conv_update.restype = ctypes.c_int
            lib.gdn_conv_update.argtypes = [P(_LayerDesc), P(_LayerParams), P(_Pools), VP, I32, P(_Rows), VP,
                                            ctypes.c_int, VP, VP]
            lib.gdn_recurrent_step.restype = ctypes.c_int
            lib.gdn_recurrent_step.argtypes = [P(_LayerDesc), P(_LayerParams), P(_Pools), VP, ctypes.c_int, VP,
                                               VP, I32, P(_Rows), VP, VP, VP]
            lib.gdn_chunk_prefill.restype = ctypes.c_int
            lib.gdn_chunk_prefill.argtypes = [P(_LayerDesc), P(_LayerParams), P(_Pools), VP, ctypes.c_int, VP,
                                              VP, I32, P(_Rows), I32, VP, VP, ctypes.c_size_t, VP, VP]
            lib.gdn_mixed_batch.restype = ctypes.c_int
            lib.gdn_mixed_batch.argtypes = [P(_LayerDesc), P(_LayerParams), P(_Pools), VP, VP, VP, I32, P(_Rows),
                                            I32, I32, P(_Rows), VP, VP, ctypes.c_size_t, VP, VP]
            lib.gdn_mixed_batch_static_workspace.restype = ctypes.c_int
            lib.gdn_mixed_batch_static_workspace.argtypes = [P(_LayerDesc), P(_LayerParams), P(_Pools), VP, VP, VP,
                                                             I32, P(_Rows), I32, I32, P(_Rows), VP, VP, VP]
            I64, SZ = ctypes.c_int64, ctypes.c_size_t
            for name, res, args in (
                    ("gdn_kv_append", ctypes.c_int, [P(_KvCache), P(_KvRows), VP, I64, VP, I64, I32, VP, VP]),
                    ("gdn_paged_attention", ctypes.c_int, [P(_AttnDesc), P(_KvCache), P(_KvRows), VP, I64, I32, VP,
                                                           I64, VP, SZ, VP, VP]),
                    ("gdn_attention_workspace_bytes", SZ, [P(_AttnDesc), P(_KvCache), P(_KvRows)]),
                    ("gdn_kv_reserve", ctypes.c_int, [P(_KvCache), I32, VP, VP, VP, VP, SZ, VP, VP]),
                    ("gdn_kv_release", ctypes.c_int, [P(_KvCache), I32, VP, VP, VP, VP, VP]),
                    ("gdn_kv_fork", ctypes.c_int, [P(_KvCache), I32, VP, VP, VP, VP, SZ, VP, VP]),
                    ("gdn_kv_copy_pages", ctypes.c_int, [P(_KvCache), I32, VP, VP, VP, VP]),
                    ("gdn_kv_compact", ctypes.c_int, [P(_KvCache), VP, VP, SZ, VP, VP]),
                    ("gdn_kv_workspace_bytes", SZ, [P(_KvCache), I32]),
                    ("gdn_copy_slots", ctypes.c_int, [P(_LayerDesc), P(_Pools), I32, VP, VP, VP, VP]),
                    ("gdn_shared_attention", ctypes.c_int, [P(_AttnDesc), P(_KvCache), P(_KvRows), P(_KvGroups), VP, I64, I32,
                                                            VP, I64, VP, SZ, VP, VP]),
                    ("gdn_shared_attention_workspace_bytes", SZ, [P(_AttnDesc), P(_KvCache), P(_KvRows), P(_KvGroups)]),
                    ("gdn_kv_common_prefix", ctypes.c_int, [P(_KvCache), P(_KvRows), P(_KvGroups), VP, VP]),
                    ("gdn_rope", ctypes.c_int, [P(_RopeDesc), I32, I32, I32, VP, I32, VP, I64, VP, I64, VP]),
                    ("gdn_rope_turns", ctypes.c_int, [P(_RopeFreq), P(ctypes.c_uint64), P(ctypes.c_float)]),
                    ("gdn_rope_turns_of", ctypes.c_int, [P(ctypes.c_double), I32, P(ctypes.c_uint64)]),
                    ("gdn_kv_append_rope", ctypes.c_int, [P(_KvCache), P(_KvRows), P(_RopeDesc), VP, I64, VP, I64, I32, VP,
                                                          I64, VP, I64, I32, VP, VP])):
                fn = getattr(lib, name)
                fn.restype, fn.argtypes = res, args
            for hook in TESTING_EXPORTS:
                getattr(lib, hook).restype = ctypes.c_int
                getattr(lib, hook).argtypes = [ctypes.c_uint64, I32]
            _lib = lib
    return _lib


# ------------------------------------------------------------------------------------------
# Descriptors (Python views of the C structs)

def _dtype_code(dt: torch.dtype) -> int:
    if dt == torch.bfloat16:
        return GDN_BF16
    if dt == torch.float32:
        return GDN_F32
    raise TypeError(f"unsupported dtype {dt}")


def _ptr(t: Optional[torch.Tensor], dtype: Optional[torch.dtype] = None, name: str = "",
         device: Optional[int] = None) -> Optional[int]:
    if t is None:
        return None
    at = t.get_device()
    if at < 0:
        raise TypeError(f"{name}: expected a CUDA tensor")
    if device is not None and at != device:
        raise ValueError(f"{name} is on cuda:{at}, other tensors of the call on cuda:{device}")
    if not t.is_contiguous():
        raise TypeError(f"{name}: expected a contiguous tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    return t.data_ptr()


@dataclass
class Layer:
    num_k_heads: int
    num_v_heads: int
    head_k_dim: int
    head_v_dim: int
    conv_width: int
    conv_state_len: int
    act_dtype: torch.dtype = torch.bfloat16
    scale: float = 0.0  # <= 0: 1/sqrt(head_k_dim)
    qkv_layout: int = 0   # GDN_QKV_PACKED / GDN_QKV_PER_KHEAD (channel order of x)
    conv_layout: int = 0  # GDN_CONV_ROLLED / GDN_CONV_PER_SLOT (spec conv history)

    @property
    def channels(self) -> int:
        return 2 * self.num_k_heads * self.head_k_dim + self.num_v_heads * self.head_v_dim

    def c(self) -> _LayerDesc:
        return _LayerDesc(self.num_k_heads, self.num_v_heads, self.head_k_dim, self.head_v_dim, self.conv_width,
                          self.conv_state_len, _dtype_code(self.act_dtype), float(self.scale), int(self.qkv_layout),
                          int(self.conv_layout))


@dataclass
class Params:
    conv_weight: torch.Tensor
    A_log: torch.Tensor
    dt_bias: torch.Tensor
    conv_bias: Optional[torch.Tensor] = None

    def c(self, act: torch.dtype) -> _LayerParams:
        return _LayerParams(_ptr(self.conv_weight, act, "conv_weight"), _ptr(self.conv_bias, act, "conv_bias"),
                            _ptr(self.A_log, torch.float32, "A_log"), _ptr(self.dt_bias, torch.float32, "dt_bias"))


@dataclass
class Pools:
    conv_pool: Optional[torch.Tensor]
    ssm_pool: torch.Tensor

    def c(self, act: torch.dtype) -> _Pools:
        return _Pools(_ptr(self.conv_pool, act, "conv_pool"), _ptr(self.ssm_pool, torch.float32, "ssm_pool"),
                      int(self.ssm_pool.shape[0]))


@dataclass
class Rows:
    """One subset of rows (int32 CUDA tensors).  Speculative when spec_state_indices is set."""
    query_start_loc: torch.Tensor
    num_tokens: int
    token_indx: Optional[torch.Tensor] = None
    state_indices: Optional[torch.Tensor] = None
    has_initial_state: Optional[torch.Tensor] = None
    spec_state_indices: Optional[torch.Tensor] = None
    num_accepted_tokens: Optional[torch.Tensor] = None

    @property
    def num_seqs(self) -> int:
        return self.query_start_loc.numel() - 1

    def c(self) -> _Rows:
        i32 = torch.int32
        cols = 0 if self.spec_state_indices is None else int(self.spec_state_indices.shape[-1])
        return _Rows(self.num_seqs, int(self.num_tokens), _ptr(self.query_start_loc, i32, "query_start_loc"),
                     _ptr(self.token_indx, i32, "token_indx"), _ptr(self.state_indices, i32, "state_indices"),
                     _ptr(self.has_initial_state, i32, "has_initial_state"),
                     _ptr(self.spec_state_indices, i32, "spec_state_indices"),
                     _ptr(self.num_accepted_tokens, i32, "num_accepted_tokens"), cols)


def _int32(t: Optional[torch.Tensor], name: str, count: Optional[int] = None,
           device: Optional[int] = None) -> Optional[int]:
    if t is not None and count is not None and t.numel() != count:
        raise ValueError(f"{name}: expected {count} entries, got {t.numel()}")
    return _ptr(t, torch.int32, name, device)


def _fits32(value: int, name: str) -> int:
    """ctypes cuts what a 32-bit field does not hold."""
    if not -(1 << 31) <= int(value) < 1 << 31:
        raise ValueError(f"{name}: {value} does not fit 32 bits")
    return int(value)


def _token_rows(t: torch.Tensor, dtype: torch.dtype, heads: int, dim: int, name: str, device: int):
    """Pointer, token stride and tokens of a [tokens, heads, dim] tensor; the token dimension may be strided."""
    at = t.get_device()
    if at < 0:
        raise TypeError(f"{name}: expected a CUDA tensor")
    if at != device:
        raise ValueError(f"{name} is on cuda:{at}, other tensors of the call on cuda:{device}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    shape, st = t.shape, t.stride()
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim:
        raise ValueError(f"{name}: expected [tokens, {heads}, {dim}], got {tuple(shape)}")
    tokens = shape[0]
    if (dim > 1 and st[2] != 1) or (heads > 1 and st[1] != dim):
        raise TypeError(f"{name}: the heads of a token must be contiguous")
    if tokens <= 1:
        return t.data_ptr(), 0, tokens
    if tokens >= 1 << 31:
        raise ValueError(f"{name}: {tokens} tokens do not fit 32 bits")
    if st[0] < heads * dim:  # (0, an expanded tensor's stride, means dense in the C descriptors)
        raise TypeError(f"{name}: tokens share memory (an expanded tensor needs a copy)")
    return t.data_ptr(), st[0], tokens


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)  # 1 us less than the public call


def _on_current(device: int, rows: Optional["KvRows"] = None) -> int:
    """The library launches on the current device: every tensor of a call has to be there."""
    if _current_device() != device:
        raise ValueError(f"the call's tensors are on cuda:{device}, the current device is cuda:{_current_device()}")
    if rows is not None and rows._device != device:
        raise ValueError(f"the rows are on cuda:{rows._device}, other tensors of the call on cuda:{device}")
    return device


@dataclass(frozen=True)
class KvCache:
    """The paged key-value cache of an attention layer (``gdn_kv_cache``): pools
    [num_pages, num_kv_heads, page_size, head_dim], whose page dimension may be strided (K and V as
    halves of one allocation), the block table [table rows, max_pages] and the pages' holder
    counts, both int32.  The tensors stay the caller's; the descriptor is checked once, here."""
    k_pool: torch.Tensor
    v_pool: torch.Tensor
    block_table: torch.Tensor
    refcount: Optional[torch.Tensor] = None

    def __post_init__(self):
        k, v = self.k_pool, self.v_pool
        if not (k.is_cuda and v.is_cuda):
            raise TypeError("k_pool, v_pool: expected CUDA tensors")
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype:
            raise ValueError("k_pool and v_pool: one [num_pages, num_kv_heads, page_size, head_dim] shape and dtype")
        for t, name in ((k, "k_pool"), (v, "v_pool")):
            if not t[:1].is_contiguous():
                raise TypeError(f"{name}: a page must be contiguous")
            if t.shape[0] > 1 and t.stride(0) < t[0].numel():
                raise TypeError(f"{name}: pages share memory")
        if k.shape[0] > 1 and k.stride(0) != v.stride(0):
            raise ValueError("k_pool and v_pool: expected one page stride")
        if self.block_table.dim() != 2:
            raise ValueError("block_table: expected [table rows, max_pages]")
        pages, heads, size, dim = k.shape
        if max(pages, heads, size, dim, *self.block_table.shape) >= 1 << 31:
            raise ValueError("a dimension does not fit 32 bits")
        device = k.get_device()
        if v.get_device() != device:
            raise ValueError(f"v_pool is on cuda:{v.get_device()}, k_pool on cuda:{device}")
        desc = _KvCache(k.data_ptr(), v.data_ptr(), k.stride(0) if pages > 1 else 0,
                        _int32(self.block_table, "block_table", None, device),
                        _int32(self.refcount, "refcount", pages, device), pages,
                        self.block_table.shape[0], self.block_table.shape[1], size, heads, dim, _dtype_code(k.dtype))
        object.__setattr__(self, "_desc", desc)
        object.__setattr__(self, "_ref", ctypes.byref(desc))
        object.__setattr__(self, "_device", device)

    @property
    def dtype(self) -> torch.dtype:
        return self.k_pool.dtype


@dataclass(frozen=True)
class KvRows:
    """The rows of one subset as an attention layer sees them (``gdn_kv_rows``, int32 CUDA tensors):
    row n's new tokens are the last of its ``kv_lens[n]`` tokens, its pages those of table row
    ``table_rows[n]`` (None: n).  ``from_rows`` takes the GDN layers' rows over."""
    query_start_loc: torch.Tensor
    num_tokens: int
    kv_lens: torch.Tensor
    max_query_len: int
    table_rows: Optional[torch.Tensor] = None
    token_indx: Optional[torch.Tensor] = None

    def __post_init__(self):
        n = self.query_start_loc.numel() - 1
        device = self.query_start_loc.get_device()
        desc = _KvRows(n, _fits32(self.num_tokens, "num_tokens"), _int32(self.query_start_loc, "query_start_loc"),
                       _int32(self.token_indx, "token_indx", int(self.num_tokens), device),
                       _int32(self.table_rows, "table_rows", n, device), _int32(self.kv_lens, "kv_lens", n, device),
                       _fits32(self.max_query_len, "max_query_len"))
        object.__setattr__(self, "_device", device)
        object.__setattr__(self, "_desc", desc)
        object.__setattr__(self, "_ref", ctypes.byref(desc))

    @classmethod
    def from_rows(cls, rows: "Rows", kv_lens: torch.Tensor, max_query_len: int,
                  table_rows: Optional[torch.Tensor] = None) -> "KvRows":
        return cls(rows.query_start_loc, rows.num_tokens, kv_lens, max_query_len, table_rows, rows.token_indx)

    @property
    def num_seqs(self) -> int:
        return self.query_start_loc.numel() - 1


@dataclass(frozen=True)
class Attention:
    """``gdn_attn_desc``: scale <= 0 selects 1/sqrt(head_dim), window <= 0 none; with a window the
    first ``num_sinks`` positions stay visible."""
    num_q_heads: int
    scale: float = 0.0
    window: int = 0
    num_sinks: int = 0

    def __post_init__(self):
        desc = _AttnDesc(_fits32(self.num_q_heads, "num_q_heads"), float(self.scale), _fits32(self.window, "window"),
                         _fits32(self.num_sinks, "num_sinks"))
        object.__setattr__(self, "_desc", desc)
        object.__setattr__(self, "_ref", ctypes.byref(desc))


@dataclass(frozen=True)
class KvGroups:
    """Groups of rows that share the beginning of their caches (``gdn_kv_groups``, int32 CUDA tensors): group g is
    rows [group_start_loc[g], group_start_loc[g + 1]) of a call, which hold the same pages for their first prefix_lens[g]
    tokens."""
    group_start_loc: torch.Tensor
    prefix_lens: torch.Tensor

    def __post_init__(self):
        n = self.prefix_lens.numel()
        device = self.prefix_lens.get_device()
        desc = _KvGroups(n, _int32(self.group_start_loc, "group_start_loc", n + 1, device),
                         _int32(self.prefix_lens, "prefix_lens"))
        object.__setattr__(self, "_device", device)
        object.__setattr__(self, "_desc", desc)
        object.__setattr__(self, "_ref", ctypes.byref(desc))

    @property
    def num_groups(self) -> int:
        return self.prefix_lens.numel()


@dataclass(frozen=True)
class Rope:
    """Rotary positions (``gdn_rope_desc``): the first ``rotary_dim`` values of a head turn, pairs as ``layout`` says
    (GDN_ROPE_HALF or GDN_ROPE_INTERLEAVED).  The frequencies base^(-2i/rotary_dim) are scaled as ``scaling`` says
    (GDN_ROPE_PLAIN, _LINEAR, _NTK, _BANDS, _RAMP: include/gdn.h), or given in radians a position as ``frequencies``.
    ``magnitude`` 0 selects that of the scaling.  The table of frequencies is made once, here, on ``device`` (the current CUDA
    device)."""
    rotary_dim: int
    base: float = 10000.0
    layout: int = GDN_ROPE_HALF
    scaling: int = GDN_ROPE_PLAIN
    factor: float = 1.0
    original_len: float = 0.0
    low: float = 0.0
    high: float = 0.0
    magnitude: float = 0.0
    frequencies: Optional[tuple] = None
    device: Optional[torch.device] = None

    def __post_init__(self):
        r = _fits32(self.rotary_dim, "rotary_dim")
        if r < 2 or r > 256 or r % 2:
            raise ValueError(f"rotary_dim: {r} is not an even number of 2 to 256")
        turns, size = (ctypes.c_uint64 * (r // 2))(), ctypes.c_float(1.0)
        if self.frequencies is not None:
            f = torch.as_tensor(self.frequencies, dtype=torch.float64).flatten().tolist()
            if len(f) != r // 2:
                raise ValueError(f"frequencies: expected {r // 2}, got {len(f)}")
            _check(library().gdn_rope_turns_of((ctypes.c_double * len(f))(*f), len(f), turns))
        else:
            freq = _RopeFreq(r, _fits32(self.scaling, "scaling"), self.base, self.factor, self.original_len, self.low, self.high)
            _check(library().gdn_rope_turns(ctypes.byref(freq), turns, ctypes.byref(size)))
        table = torch.tensor([t - (1 << 64) if t >> 63 else t for t in turns], dtype=torch.int64)
        table = table.to("cuda" if self.device is None else self.device)
        desc = _RopeDesc(table.data_ptr(), r, _fits32(self.layout, "layout"), float(self.magnitude) or size.value)
        object.__setattr__(self, "turns", table)
        object.__setattr__(self, "_device", table.get_device())
        object.__setattr__(self, "_desc", desc)
        object.__setattr__(self, "_ref", ctypes.byref(desc))


def _rows_ref(r: Optional[Rows]):
    return None if r is None else ctypes.byref(r.c())


def _stream(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # 3 us less than a Stream object


def _stream_of(t: torch.Tensor, stream) -> Optional[int]:
    """``stream``, by default the current one of the tensor's device."""
    if stream is None and _raw_stream is not None:
        return _raw_stream(t.get_device())
    return _stream(stream)


def _scratch(nbytes: int, device, stream) -> torch.Tensor:
    """A workspace, allocated on the stream that works on it: a block of another stream's could still be in use by
    work queued there, and would be free for more of it as soon as the call returns."""
    if stream is None:
        return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        handle = _stream(stream)
        stream = torch.cuda.ExternalStream(handle, device=device) if handle else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)


def _check(rc: int) -> None:
    if rc != 0:
        raise GdnError(rc, library().gdn_status_string(rc).decode())


# ------------------------------------------------------------------------------------------
# The entry points

def gdn_workspace_bytes(layer: Layer, non_spec: Optional[Rows], spec: Optional[Rows]) -> int:
    return int(library().gdn_workspace_bytes(ctypes.byref(layer.c()), _rows_ref(non_spec), _rows_ref(spec)))


def gdn_prefill_workspace_bytes(layer: Layer, rows: Optional[Rows], num_prefills: int) -> int:
    return int(library().gdn_prefill_workspace_bytes(ctypes.byref(layer.c()), _rows_ref(rows), int(num_prefills)))


def mixed_batch_workspace_bytes(layer: Layer, non_spec: Optional[Rows], num_prefills: int,
                                spec: Optional[Rows]) -> int:
    """Total workspace gdn_mixed_batch needs for this batch."""
    return gdn_workspace_bytes(layer, non_spec, spec) + gdn_prefill_workspace_bytes(layer, non_spec, num_prefills)


def gdn_conv_update(layer: Layer, params: Params, pools: Pools, x: torch.Tensor, rows: Rows, y: torch.Tensor,
                    status: Optional[torch.Tensor] = None, stream=None) -> None:
    act = layer.act_dtype
    rc = library().gdn_conv_update(ctypes.byref(layer.c()), ctypes.byref(params.c(act)), ctypes.byref(pools.c(act)),
                                   _ptr(x, act, "x"), int(x.shape[0]), ctypes.byref(rows.c()), _ptr(y, None, "y"),
                                   _dtype_code(y.dtype), _ptr(status, torch.int32, "status"), _stream(stream))
    _check(rc)


def gdn_recurrent_step(layer: Layer, params: Params, pools: Pools, qkv: torch.Tensor, a: torch.Tensor,
                       b: torch.Tensor, rows: Rows, out: torch.Tensor, status: Optional[torch.Tensor] = None,
                       stream=None) -> None:
    act = layer.act_dtype
    rc = library().gdn_recurrent_step(ctypes.byref(layer.c()), ctypes.byref(params.c(act)),
                                      ctypes.byref(pools.c(act)), _ptr(qkv, None, "qkv"), _dtype_code(qkv.dtype), _ptr(a, act, "a"),
                                      _ptr(b, act, "b"), int(a.shape[0]), ctypes.byref(rows.c()),
                                      _ptr(out, act, "out"), _ptr(status, torch.int32, "status"), _stream(stream))
    _check(rc)


def gdn_chunk_prefill(layer: Layer, params: Params, pools: Pools, qkv: torch.Tensor, a: torch.Tensor,
                      b: torch.Tensor, rows: Rows, out: torch.Tensor, workspace: Optional[torch.Tensor] = None,
                      chunk_size: int = 64, status: Optional[torch.Tensor] = None, stream=None) -> None:
    act = layer.act_dtype
    need = gdn_prefill_workspace_bytes(layer, rows, rows.num_seqs)
    if workspace is None and need:
        workspace = _scratch(need, qkv.device, stream)
    ws_ptr = _ptr(workspace, torch.uint8, "workspace")
    ws_bytes = 0 if workspace is None else workspace.numel()
    rc = library().gdn_chunk_prefill(ctypes.byref(layer.c()), ctypes.byref(params.c(act)), ctypes.byref(pools.c(act)),
                                     _ptr(qkv, None, "qkv"), _dtype_code(qkv.dtype), _ptr(a, act, "a"),
                                     _ptr(b, act, "b"), int(a.shape[0]), ctypes.byref(rows.c()), int(chunk_size),
                                     _ptr(out, act, "out"), ws_ptr, ws_bytes, _ptr(status, torch.int32, "status"),
                                     _stream(stream))
    _check(rc)


def gdn_mixed_batch(layer: Layer, params: Params, pools: Pools, x: torch.Tensor, a: torch.Tensor,
                    b: torch.Tensor, non_spec: Optional[Rows], num_decodes: int, num_prefills: int,
                    spec: Optional[Rows], out: torch.Tensor, workspace: Optional[torch.Tensor] = None,
                    status: Optional[torch.Tensor] = None, stream=None,
                    num_actual_tokens: Optional[int] = None) -> None:
    """``num_actual_tokens`` (default x.shape[0]) may be smaller than the row count of x, a, b
    and out, e.g. for inputs padded to a CUDA-graph bucket; rows past it are never touched."""
    act = layer.act_dtype
    if num_actual_tokens is None:
        num_actual_tokens = int(x.shape[0])
    if workspace is None:
        need = mixed_batch_workspace_bytes(layer, non_spec, num_prefills, spec)
        workspace = _scratch(need, x.device, stream)
    rc = library().gdn_mixed_batch(ctypes.byref(layer.c()), ctypes.byref(params.c(act)), ctypes.byref(pools.c(act)),
                                   _ptr(x, act, "x"), _ptr(a, act, "a"), _ptr(b, act, "b"), int(num_actual_tokens),
                                   _rows_ref(non_spec), int(num_decodes), int(num_prefills), _rows_ref(spec),
                                   _ptr(out, act, "out"), _ptr(workspace, torch.uint8, "workspace"),
                                   workspace.numel(), _ptr(status, torch.int32, "status"), _stream(stream))
    _check(rc)


def gdn_mixed_batch_static_workspace(layer: Layer, params: Params, pools: Pools, x: torch.Tensor, a: torch.Tensor,
                                     b: torch.Tensor, non_spec: Optional[Rows], num_decodes: int, num_prefills: int,
                                     spec: Optional[Rows], out: torch.Tensor, status: Optional[torch.Tensor] = None,
                                     stream=None) -> None:
    """gdn_mixed_batch with the library's fixed device scratch, for callers that cannot
    allocate device memory (see include/gdn.h); allocates nothing itself."""
    act = layer.act_dtype
    rc = library().gdn_mixed_batch_static_workspace(
        ctypes.byref(layer.c()), ctypes.byref(params.c(act)), ctypes.byref(pools.c(act)), _ptr(x, act, "x"),
        _ptr(a, act, "a"), _ptr(b, act, "b"), int(x.shape[0]), _rows_ref(non_spec), int(num_decodes),
        int(num_prefills), _rows_ref(spec), _ptr(out, act, "out"), _ptr(status, torch.int32, "status"),
        _stream(stream))
    _check(rc)


# ------------------------------------------------------------------------------------------
# The paged key-value cache

def gdn_kv_append(cache: KvCache, rows: KvRows, k: torch.Tensor, v: torch.Tensor,
                  status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Writes the new tokens' k, v [num_global_tokens, num_kv_heads, head_dim] into the rows' pages."""
    _, heads, _, dim = cache.k_pool.shape
    kp, ks, tokens = _token_rows(k, cache.dtype, heads, dim, "k", cache._device)
    vp, vs, of_v = _token_rows(v, cache.dtype, heads, dim, "v", cache._device)
    if tokens != of_v:
        raise ValueError("k and v: expected one token count")
    device = _on_current(cache._device, rows)
    _check(library().gdn_kv_append(cache._ref, rows._ref, kp, ks, vp, vs, tokens,
                                   _ptr(status, torch.int32, "status", device), _stream_of(cache.k_pool, stream)))


def gdn_attention_workspace_bytes(attn: Attention, cache: KvCache, rows: KvRows) -> int:
    return int(library().gdn_attention_workspace_bytes(attn._ref, cache._ref, rows._ref))


def gdn_paged_attention(attn: Attention, cache: KvCache, rows: KvRows, q: torch.Tensor, out: torch.Tensor,
                        workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                        stream=None) -> None:
    """Causal attention of the rows' new tokens over their pages (which already hold them);
    q, out [num_global_tokens, num_q_heads, head_dim]."""
    dim = cache.k_pool.shape[3]
    qp, qs, tokens = _token_rows(q, cache.dtype, attn.num_q_heads, dim, "q", cache._device)
    op, os_, of_out = _token_rows(out, cache.dtype, attn.num_q_heads, dim, "out", cache._device)
    if tokens != of_out:
        raise ValueError("q and out: expected one token count")
    device = _on_current(cache._device, rows)
    if workspace is None:
        workspace = _scratch(gdn_attention_workspace_bytes(attn, cache, rows), q.device, stream)
    _check(library().gdn_paged_attention(attn._ref, cache._ref, rows._ref, qp, qs, tokens, op, os_,
                                         _ptr(workspace, torch.uint8, "workspace", device), workspace.numel(),
                                         _ptr(status, torch.int32, "status", device), _stream_of(cache.k_pool, stream)))


def gdn_shared_attention_workspace_bytes(attn: Attention, cache: KvCache, rows: KvRows, groups: KvGroups) -> int:
    return int(library().gdn_shared_attention_workspace_bytes(attn._ref, cache._ref, rows._ref, groups._ref))


def _of_device(part, device: int, name: str) -> None:
    if part._device != device:
        where = "the CPU" if part._device < 0 else f"cuda:{part._device}"
        raise ValueError(f"the {name} is on {where}, other tensors of the call on cuda:{device}")


def gdn_shared_attention(attn: Attention, cache: KvCache, rows: KvRows, groups: KvGroups, q: torch.Tensor,
                         out: torch.Tensor, workspace: Optional[torch.Tensor] = None,
                         status: Optional[torch.Tensor] = None, stream=None) -> None:
    """gdn_paged_attention with the pages that the rows of a group share read once for all of them."""
    dim = cache.k_pool.shape[3]
    qp, qs, tokens = _token_rows(q, cache.dtype, attn.num_q_heads, dim, "q", cache._device)
    op, os_, of_out = _token_rows(out, cache.dtype, attn.num_q_heads, dim, "out", cache._device)
    if tokens != of_out:
        raise ValueError("q and out: expected one token count")
    device = _on_current(cache._device, rows)
    _of_device(groups, device, "groups' table")
    if workspace is None:
        workspace = _scratch(gdn_shared_attention_workspace_bytes(attn, cache, rows, groups), q.device, stream)
    _check(library().gdn_shared_attention(attn._ref, cache._ref, rows._ref, groups._ref, qp, qs, tokens, op, os_,
                                          _ptr(workspace, torch.uint8, "workspace", device), workspace.numel(),
                                          _ptr(status, torch.int32, "status", device), _stream_of(cache.k_pool, stream)))


def gdn_kv_common_prefix(cache: KvCache, rows: KvRows, groups: KvGroups, status: Optional[torch.Tensor] = None,
                         stream=None) -> None:
    """Writes to groups.prefix_lens how many leading tokens the rows of each group hold in the same pages."""
    device = _on_current(cache._device, rows)
    _of_device(groups, device, "groups' table")
    _check(library().gdn_kv_common_prefix(cache._ref, rows._ref, groups._ref, _ptr(status, torch.int32, "status", device),
                                          _stream_of(cache.k_pool, stream)))


def gdn_rope(rope: Rope, positions: torch.Tensor, x: torch.Tensor, out: torch.Tensor, stream=None) -> None:
    """Turns the heads of x [tokens, heads, head_dim] by ``positions`` (int32, one per token, or of the first tokens) into
    ``out``, which may be x.  At negated positions it is the gradient with respect to x."""
    shape = x.shape
    if len(shape) != 3:
        raise ValueError(f"x: expected [tokens, heads, head_dim], got {tuple(shape)}")
    _, heads, dim = shape
    device, dtype = x.get_device(), x.dtype
    xp, xs, tokens = _token_rows(x, dtype, heads, dim, "x", device)
    op, os_, of_out = (xp, xs, tokens) if out is x else _token_rows(out, dtype, heads, dim, "out", device)
    n = positions.numel()
    if tokens != of_out or n > tokens:
        raise ValueError("positions, x and out: expected one token count, or fewer positions")
    if _current_device() != device:
        _on_current(device)
    if rope._device != device:
        _of_device(rope, device, "frequencies' table")
    _check(library().gdn_rope(rope._ref, heads, dim, _dtype_code(dtype), _int32(positions, "positions", None, device), n,
                              xp, xs, op, os_, _stream_of(x, stream)))


def gdn_kv_append_rope(cache: KvCache, rows: KvRows, rope: Rope, k: torch.Tensor, v: torch.Tensor,
                       q: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
                       status: Optional[torch.Tensor] = None, stream=None) -> None:
    """gdn_kv_append with the new tokens' keys turned by their positions on the way, and the queries q
    [num_global_tokens, num_q_heads, head_dim] of the same tokens turned into ``q_out`` (None: in place)."""
    _, heads, _, dim = cache.k_pool.shape
    dtype, device = cache.dtype, cache._device
    kp, ks, tokens = _token_rows(k, dtype, heads, dim, "k", device)
    vp, vs, of_v = _token_rows(v, dtype, heads, dim, "v", device)
    if tokens != of_v:
        raise ValueError("k and v: expected one token count")
    hq, qp, qs, op, os_ = 0, None, 0, None, 0
    if q is not None:
        if q.dim() != 3:
            raise ValueError(f"q: expected [tokens, heads, head_dim], got {tuple(q.shape)}")
        hq = q.shape[1]
        qp, qs, of_q = _token_rows(q, dtype, hq, dim, "q", device)
        op, os_, of_out = (qp, qs, of_q) if q_out is None else _token_rows(q_out, dtype, hq, dim, "q_out", device)
        if tokens != of_q or tokens != of_out:
            raise ValueError("k, v, q and q_out: expected one token count")
    elif q_out is not None:
        raise ValueError("q_out without q")
    _on_current(device, rows)
    if rope._device != device:
        _of_device(rope, device, "frequencies' table")
    _check(library().gdn_kv_append_rope(cache._ref, rows._ref, rope._ref, kp, ks, vp, vs, hq, qp, qs, op, os_, tokens,
                                        _ptr(status, torch.int32, "status", device), _stream_of(cache.k_pool, stream)))


def gdn_kv_workspace_bytes(cache: KvCache, count: int) -> int:
    """Workspace of gdn_kv_reserve and gdn_kv_fork over ``count`` rows, and of gdn_kv_compact."""
    return int(library().gdn_kv_workspace_bytes(cache._ref, int(count)))


def _kv_workspace(cache: KvCache, count: int, workspace: Optional[torch.Tensor], stream) -> torch.Tensor:
    return _scratch(gdn_kv_workspace_bytes(cache, count), cache.k_pool.device, stream) if workspace is None else workspace


def gdn_kv_reserve(cache: KvCache, table_rows: Optional[torch.Tensor], from_lens: torch.Tensor, to_lens: torch.Tensor,
                   workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                   stream=None) -> None:
    """Gives each listed table row free pages for its tokens [from_lens, to_lens)."""
    n = from_lens.numel()
    device = _on_current(cache._device)
    ws = _kv_workspace(cache, n, workspace, stream)
    _check(library().gdn_kv_reserve(cache._ref, n, _int32(table_rows, "table_rows", n, device),
                                    _int32(from_lens, "from_lens", None, device), _int32(to_lens, "to_lens", n, device),
                                    _ptr(ws, torch.uint8, "workspace", device), ws.numel(),
                                    _ptr(status, torch.int32, "status", device), _stream_of(cache.k_pool, stream)))


def gdn_kv_release(cache: KvCache, table_rows: torch.Tensor, first_page: Optional[torch.Tensor] = None,
                   last_page: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                   stream=None) -> None:
    """Gives back the pages of entries [first_page, last_page) of each listed table row."""
    n = table_rows.numel()
    device = _on_current(cache._device)
    _check(library().gdn_kv_release(cache._ref, n, _int32(table_rows, "table_rows", None, device),
                                    _int32(first_page, "first_page", n, device), _int32(last_page, "last_page", n, device),
                                    _ptr(status, torch.int32, "status", device), _stream_of(cache.k_pool, stream)))


def gdn_kv_fork(cache: KvCache, src_rows: torch.Tensor, dst_rows: torch.Tensor, lens: torch.Tensor,
                workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Table row dst_rows[i] becomes a holder of the first lens[i] tokens of src_rows[i]."""
    n = src_rows.numel()
    device = _on_current(cache._device)
    ws = _kv_workspace(cache, n, workspace, stream)
    _check(library().gdn_kv_fork(cache._ref, n, _int32(src_rows, "src_rows", None, device),
                                 _int32(dst_rows, "dst_rows", n, device), _int32(lens, "lens", n, device),
                                 _ptr(ws, torch.uint8, "workspace", device), ws.numel(),
                                 _ptr(status, torch.int32, "status", device), _stream_of(cache.k_pool, stream)))


def gdn_kv_copy_pages(cache: KvCache, src_pages: torch.Tensor, dst_pages: torch.Tensor,
                      status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Copies page src_pages[i] onto dst_pages[i] in both pools."""
    n = src_pages.numel()
    device = _on_current(cache._device)
    _check(library().gdn_kv_copy_pages(cache._ref, n, _int32(src_pages, "src_pages", None, device),
                                       _int32(dst_pages, "dst_pages", n, device),
                                       _ptr(status, torch.int32, "status", device), _stream_of(cache.k_pool, stream)))


def gdn_kv_compact(cache: KvCache, num_live: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                   status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Moves the live pages to ids 1..M; ``num_live`` (int32, one entry) receives M."""
    device = _on_current(cache._device)
    ws = _kv_workspace(cache, 0, workspace, stream)
    _check(library().gdn_kv_compact(cache._ref, _int32(num_live, "num_live", 1, device),
                                    _ptr(ws, torch.uint8, "workspace", device), ws.numel(),
                                    _ptr(status, torch.int32, "status", device), _stream_of(cache.k_pool, stream)))


def gdn_copy_slots(layer: Layer, pools: Pools, src_slots: torch.Tensor, dst_slots: torch.Tensor,
                   status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Copies GDN state: slot src_slots[i] of both pools onto dst_slots[i] (a NULL source reads as zeros)."""
    n = src_slots.numel()
    act = layer.act_dtype
    device = _on_current(pools.ssm_pool.get_device())
    _ptr(pools.conv_pool, act, "conv_pool", device)
    _check(library().gdn_copy_slots(ctypes.byref(layer.c()), ctypes.byref(pools.c(act)), n,
                                    _int32(src_slots, "src_slots", None, device), _int32(dst_slots, "dst_slots", n, device),
                                    _ptr(status, torch.int32, "status", device), _stream_of(pools.ssm_pool, stream)))


def gdn_testing_set_prefill_faults(wait_ns: int = 0, drop_copy_chunk: int = -1) -> None:
    """Test hook (include/gdn_testing.h): the wall-clock limit of the chunked prefill's bounded
    waits (0 = the default, one second) and a chunk whose record copy the scan leaves out on
    purpose (< 0 = none), for every later prefill launch in this process."""
    _check(library().gdn_testing_set_prefill_faults(int(wait_ns), int(drop_copy_chunk)))


def gdn_testing_set_shared_faults(wait_ns: int = 0, stop_tile: int = -1) -> None:
    """Test hook (include/gdn_testing.h): the limit of the waits in gdn_shared_attention's tensor-core pass (0 = the default) and
    the tile of a CTA's share at which its fetches end (< 0 = none), for every later call in this process."""
    _check(library().gdn_testing_set_shared_faults(int(wait_ns), int(stop_tile)))


__all__ = ["Layer", "Params", "Pools", "Rows", "GdnError", "library", "LIB_PATH", "EXPORTS",
           "gdn_workspace_bytes", "gdn_prefill_workspace_bytes", "mixed_batch_workspace_bytes", "STATUS_WAIT_TIMEOUT", "gdn_conv_update", "gdn_recurrent_step", "gdn_chunk_prefill",
           "gdn_mixed_batch", "gdn_mixed_batch_static_workspace", "STATIC_WORKSPACE_BYTES",
           "TESTING_EXPORTS", "gdn_testing_set_prefill_faults", "gdn_testing_set_shared_faults", "GDN_F32", "GDN_BF16", "STATUS_SLOT_RANGE", "STATUS_NUM_ACCEPTED",
           "STATUS_TOKEN_RANGE", "STATUS_ROW_RANGE", "KvCache", "KvRows", "Attention", "gdn_kv_append",
           "gdn_paged_attention", "gdn_attention_workspace_bytes", "gdn_kv_reserve", "gdn_kv_release", "gdn_kv_fork",
           "gdn_kv_copy_pages", "gdn_kv_compact", "gdn_kv_workspace_bytes", "gdn_copy_slots", "STATUS_PAGE_RANGE",
           "STATUS_PAGE_SHARED", "STATUS_NO_PAGES", "KvGroups", "gdn_shared_attention",
           "gdn_shared_attention_workspace_bytes", "gdn_kv_common_prefix", "Rope", "gdn_rope", "gdn_kv_append_rope",
           "GDN_ROPE_HALF", "GDN_ROPE_INTERLEAVED", "GDN_ROPE_PLAIN", "GDN_ROPE_LINEAR", "GDN_ROPE_NTK", "GDN_ROPE_BANDS",
           "GDN_ROPE_RAMP"]
