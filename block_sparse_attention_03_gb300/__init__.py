"""GB300-native MiniMax Sparse Attention (MSA) decode hot path.

Thin Python binding over the C ABI of ``libmsa.so`` (declared in
``include/msa.h``): every function here only marshals arguments (torch tensors
-> device pointers, the current CUDA stream) and raises on a non-OK status.
All computation runs in the library's CUDA kernels; there is no fallback.
"""

from __future__ import annotations

import ctypes
import dataclasses
import os
import struct as _struct
import threading
from typing import Optional

from . import roofline  # noqa: F401  (host-side byte model)

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmsa.so")

MSA_OK = 0
STATUS_NAMES = {0: "MSA_OK", 1: "MSA_ERR_INVALID_ARGUMENT", 2: "MSA_ERR_UNSUPPORTED",
                3: "MSA_ERR_WORKSPACE_TOO_SMALL", 4: "MSA_ERR_CUDA", 5: "MSA_ERR_DEVICE_FAULT",
                6: "MSA_ERR_TIMEOUT"}
DTYPES = {"bf16": 0, "fp8": 1, "nvfp4": 2}

# every symbol include/msa.h declares
EXPORTS = ("msa_workspace_size", "msa_workspace_init", "msa_indexer_score", "msa_topk_blocks",
           "msa_sparse_attend", "msa_decode", "msa_read_device_status", "msa_status_string",
           "msa_dequant_debug", "msa_decode_noalloc", "msa_cache_insert", "msa_dense_workspace_size",
           "msa_dense_attend", "msa_rope_init", "msa_rope_insert", "msa_build_tables")


class MsaError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}")
        self.status = status


class MsaCacheT(ctypes.Structure):
    _fields_ = [("kv_dtype", ctypes.c_int), ("index_dtype", ctypes.c_int),
                ("num_blocks", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("index_dim", ctypes.c_int32),
                ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_sf", ctypes.c_void_p), ("v_sf", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("idx", ctypes.c_void_p), ("idx_sf", ctypes.c_void_p), ("idx_scale", ctypes.c_void_p),
                ("k_global", ctypes.c_float), ("v_global", ctypes.c_float), ("idx_global", ctypes.c_float),
                ("nvfp4_mode", ctypes.c_int32)]


class MsaBatchT(ctypes.Structure):
    _fields_ = [("num_seqs", ctypes.c_int32), ("q_per_seq", ctypes.c_int32),
                ("max_blocks_per_seq", ctypes.c_int32),
                ("seq_lens", ctypes.c_void_p), ("block_table", ctypes.c_void_p)]


class MsaConfigT(ctypes.Structure):
    _fields_ = [("topk", ctypes.c_int32), ("init_blocks", ctypes.c_int32),
                ("local_blocks", ctypes.c_int32), ("index_scale", ctypes.c_float),
                ("sm_scale", ctypes.c_float), ("score_type", ctypes.c_int32), ("prefill_select", ctypes.c_int32)]


SCORE_TYPES = {"max": 0}  # msa_score_type_t: the block pooling of the index scores
# msa_nvfp4_mode_t: "exact" e2m1 x e4m3 products, or "e4m3": rounded to E4M3 first
NVFP4_MODES = {"exact": 0, "e4m3": 1}
# msa_prefill_select_t: a prefill chunk's selection by a top-k launch over the
# pooled scores, or in the tcgen05 indexer's epilogue (candidate lists)
PREFILL_SELECT = {"topk": 0, "indexer": 1}


class MsaQueryT(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int), ("scale", ctypes.c_float)]


ROPE_LAYOUTS = {"halves": 0, "adjacent": 1}  # msa_rope_layout_t


class MsaRopeT(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int32), ("axes", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("axis", ctypes.c_uint8 * 64), ("turns", ctypes.c_uint64 * 64)]


class MsaRowsT(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("stride", ctypes.c_int64)]


class MsaQkNormT(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("index_q", ctypes.c_void_p),
                ("index_k", ctypes.c_void_p), ("eps", ctypes.c_float), ("offset", ctypes.c_float)]


_lib_handle = None


def lib() -> ctypes.CDLL:
    """Load libmsa.so (built in-tree by __graft_entry__.build()); raises if absent."""
    global _lib_handle
    if _lib_handle is None:  # (every call after the first returns at once)
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built; run __graft_entry__.build() first "
                               "(there is no non-CUDA implementation)")
        h = ctypes.CDLL(LIB_PATH)
        P = ctypes.c_void_p
        h.msa_workspace_size.restype = ctypes.c_size_t
        h.msa_workspace_size.argtypes = [P, P, P, ctypes.c_int32]
        h.msa_workspace_init.argtypes = [P, ctypes.c_size_t, P]
        h.msa_indexer_score.argtypes = [P, P, P, P, P, P, ctypes.c_size_t, P]
        h.msa_topk_blocks.argtypes = [P, P, ctypes.c_int32, P, P, P, P, ctypes.c_size_t, P]
        h.msa_sparse_attend.argtypes = [P, P, P, P, ctypes.c_int32, P, P, P, P, ctypes.c_size_t, P]
        h.msa_decode.argtypes = [P, P, P, P, P, ctypes.c_int32, P, P, P, P, ctypes.c_size_t, P]
        h.msa_read_device_status.argtypes = [P, P, P]
        h.msa_status_string.restype = ctypes.c_char_p
        h.msa_status_string.argtypes = [ctypes.c_int]
        h.msa_dequant_debug.argtypes = [P, ctypes.c_int32, P, ctypes.c_int32, P, P]
        h.msa_decode_noalloc.argtypes = [P, P, P, P, P, ctypes.c_int32, P, P, P, P, P]
        h.msa_cache_insert.argtypes = [P, ctypes.c_int32, P, P, P, P, P, ctypes.c_size_t, P]
        I = ctypes.c_int32
        h.msa_dense_workspace_size.restype = ctypes.c_size_t
        h.msa_dense_workspace_size.argtypes = [P, P, I]
        h.msa_dense_attend.argtypes = [P, P, P, P, I, P, P, P, ctypes.c_size_t, P]
        h.msa_rope_init.argtypes = [P, I, ctypes.c_double, I, P, I]
        h.msa_rope_insert.argtypes = [P, P, I, P, P, I, P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
        h.msa_build_tables.argtypes = [I, I, P, P, I, P, I, P, P, P, P, P, I, P, P, P, ctypes.c_size_t, P]
        for name in EXPORTS:
            if name not in ("msa_workspace_size", "msa_status_string", "msa_dense_workspace_size"):
                getattr(h, name).restype = ctypes.c_int
        _lib_handle = h
    return _lib_handle


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


_raw_stream = None


def _stream(stream, device=None) -> Optional[int]:
    if stream is None:
        global _raw_stream
        if _raw_stream is None:
            import torch
            # the current stream's handle without a Stream object around it (a microsecond less)
            raw, current = getattr(torch._C, "_cuda_getCurrentRawStream", None), torch.cuda.current_device
            _raw_stream = (lambda d: raw(current() if d is None else d)) if raw else \
                (lambda d: torch.cuda.current_stream(d).cuda_stream)
        return _raw_stream(device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check(status: int, where: str) -> None:
    if status != MSA_OK:
        raise MsaError(status, where)


# ---------------------------------------------------------------- argument holders

@dataclasses.dataclass
class PagedCache:
    """Device tensors of one layer's paged K/V cache and index-key cache (layout in include/msa.h)."""
    kv_dtype: str
    index_dtype: str
    num_blocks: int
    num_kv_heads: int
    k: object
    v: object
    idx: object
    k_sf: object = None
    v_sf: object = None
    k_scale: object = None
    v_scale: object = None
    idx_sf: object = None
    idx_scale: object = None
    k_global: float = 0.0
    v_global: float = 0.0
    idx_global: float = 0.0
    head_dim: int = 128
    index_dim: int = 128
    nvfp4_mode: str = "exact"

    def __setattr__(self, name, value):
        # the serving calls look at the tensors once (_checked), and again when a field is set
        self.__dict__["_seen"] = ()
        self.__dict__[name] = value

    def struct(self) -> MsaCacheT:
        return MsaCacheT(DTYPES[self.kv_dtype], DTYPES[self.index_dtype], self.num_blocks, 128,
                         self.num_kv_heads, self.head_dim, self.index_dim,
                         _ptr(self.k), _ptr(self.v), _ptr(self.k_sf), _ptr(self.v_sf),
                         _ptr(self.k_scale), _ptr(self.v_scale), _ptr(self.idx), _ptr(self.idx_sf),
                         _ptr(self.idx_scale), self.k_global, self.v_global, self.idx_global,
                         NVFP4_MODES.get(self.nvfp4_mode, -1))


@dataclasses.dataclass
class Batch:
    seq_lens: object      # int32 [S] on the device
    block_table: object   # int32 [S][max_blocks] on the device
    q_per_seq: int = 1

    def struct(self) -> MsaBatchT:
        return MsaBatchT(self.seq_lens.shape[0], self.q_per_seq, self.block_table.shape[1],
                         _ptr(self.seq_lens), _ptr(self.block_table))


@dataclasses.dataclass
class Config:
    topk: int = 16
    init_blocks: int = 0
    local_blocks: int = 0
    index_scale: float = 128 ** -0.5
    sm_scale: float = 128 ** -0.5
    score_type: str = "max"
    prefill_select: str = "topk"

    def struct(self) -> MsaConfigT:
        # an unknown score type reaches the library as -1, which rejects it
        return MsaConfigT(self.topk, self.init_blocks, self.local_blocks, self.index_scale, self.sm_scale,
                          SCORE_TYPES.get(self.score_type, -1), PREFILL_SELECT.get(self.prefill_select, -1))


@dataclasses.dataclass
class Query:
    data: object          # bf16 tensor, or uint8 e4m3 codes
    dtype: str = "bf16"   # "bf16" | "fp8"
    scale: float = 1.0

    def struct(self) -> MsaQueryT:
        return MsaQueryT(_ptr(self.data), DTYPES[self.dtype], self.scale)


@dataclasses.dataclass
class QkNorm:
    """bf16 [128] weights of the per-head RMS norm before the rotation (None: that kind is not normed)."""
    q: object = None
    k: object = None
    index_q: object = None
    index_k: object = None
    eps: float = 1e-6
    offset: float = 0.0   # the norm multiplies by offset + weight

    def struct(self) -> MsaQkNormT:
        return MsaQkNormT(_ptr(self.q), _ptr(self.k), _ptr(self.index_q), _ptr(self.index_k), self.eps, self.offset)


def _ref(x):
    return ctypes.byref(x)


# The structs of the serving calls, packed side by side into a per-thread host
# buffer in one go (a ctypes object for each costs several microseconds a
# call, as long as the kernels of a decode step).  The library copies what it needs before it returns.
_tls = threading.local()
_CACHE, _BATCH, _CONFIG, _QUERY, _ROWS, _NORM = "7i9P3fi", "3i2P", "3i2f2i", "Pif", "Pq", "4P2f"


class _Layout:
    """Consecutive structs, each 8-byte aligned: the packer and each one's offset."""

    def __init__(self, *formats):
        self.offsets, fmt = [], "@"
        for f in formats:
            fmt += "0P"
            self.offsets.append(_struct.calcsize(fmt))
            fmt += f
        self.packer = _struct.Struct(fmt + "0P")

    def pack(self, *values):
        """Pack into this thread's buffer; returns the address of its start."""
        buf = getattr(_tls, "buf", None)
        if buf is None:
            _tls.buf = buf = ctypes.create_string_buffer(1024)
            _tls.addr = ctypes.addressof(buf)
        self.packer.pack_into(buf, 0, *values)
        return _tls.addr


def _p(t) -> int:
    return 0 if t is None else t.data_ptr()


def _checked(c: PagedCache, index: bool, dev: int, where: str) -> None:
    """The cache's tensors (the index keys' too, if the call writes them): dense, on the device, of
    their formats' types and at least num_blocks blocks long."""
    import torch
    codes = (torch.uint8, torch.int8, torch.float8_e4m3fn)
    wanted = [("k", c.kv_dtype, c.num_kv_heads), ("v", c.kv_dtype, c.num_kv_heads)] + [("idx", c.index_dtype, 1)] * index
    for name, kind, heads in wanted:
        rows = c.num_blocks * heads * 128
        parts = {"bf16": [(name, (torch.bfloat16,), 128)], "fp8": [(name, codes, 128), (name + "_scale", (torch.float32,), 1)],
                 "nvfp4": [(name, (torch.uint8, torch.int8), 64), (name + "_sf", codes, 8)]}.get(kind, [])
        for field, types, width in parts:
            t = getattr(c, field)
            if t is not None and (t.dtype not in types or t.numel() < rows * width or not t.is_contiguous() or t.get_device() != dev):
                raise MsaError(1, where)
    c.__dict__["_seen"] = (dev, index or (c._seen[:1] == (dev,) and c._seen[1]))


def _cache_values(c: PagedCache, index: bool, dev: int, where: str):
    seen = c._seen
    if not seen or seen[0] != dev or (index and not seen[1]):
        _checked(c, index, dev, where)
    return (DTYPES[c.kv_dtype], DTYPES[c.index_dtype], c.num_blocks, 128, c.num_kv_heads, c.head_dim, c.index_dim,
            c.k.data_ptr(), c.v.data_ptr(), _p(c.k_sf), _p(c.v_sf), _p(c.k_scale), _p(c.v_scale), _p(c.idx), _p(c.idx_sf),
            _p(c.idx_scale), c.k_global, c.v_global, c.idx_global, NVFP4_MODES.get(c.nvfp4_mode, -1))


_DENSE = _Layout(_CACHE, _BATCH, _CONFIG, _QUERY)
_ROPE = _Layout(_CACHE, _ROWS, _QUERY, _ROWS, _QUERY, _ROWS, _ROWS, _ROWS, _NORM)


_int32 = _bf16 = _f32 = _device = None
_query_types = {}  # the element types of a query of each kind


def _torch_names() -> None:
    global _int32, _bf16, _f32, _device
    import torch
    _int32, _bf16, _f32, _device = torch.int32, torch.bfloat16, torch.float32, torch.cuda.current_device
    _query_types.update(bf16=(torch.bfloat16,), fp8=(torch.uint8, torch.float8_e4m3fn, torch.int8))


# The serving calls refuse what the kernels would misread: other types, strides and
# sizes, and tensors that are not on the current device, where the kernels run.  The
# checks stand in one expression a call (a helper's call costs as much as a check).

def _rows(t, shape, where: str, dev: int):
    """(pointer, token stride) of a projection's bf16 rows of the given shape ([tokens][heads][128], or
    [tokens][128] for one head), the heads side by side."""
    strides = t.stride()
    if t.shape != shape or strides[-1] != 1 or (len(shape) == 3 and strides[1] != 128 and shape[1] != 1) or t.dtype is not _bf16 \
            or t.get_device() != dev:
        raise MsaError(1, where)
    return t.data_ptr(), strides[0]


def _nbytes(t) -> int:
    return t.numel() * t.element_size()


# ---------------------------------------------------------------- entry points (same names as the C ABI)

def msa_workspace_size(cache: PagedCache, batch: Batch, cfg: Config, num_q_heads: int) -> int:
    c, b, f = cache.struct(), batch.struct(), cfg.struct()
    n = lib().msa_workspace_size(_ref(c), _ref(b), _ref(f), num_q_heads)
    if n == 0:
        raise MsaError(1, "msa_workspace_size")
    return int(n)


def msa_workspace_init(workspace, stream=None) -> None:
    _check(lib().msa_workspace_init(_ptr(workspace), workspace.numel() * workspace.element_size(),
                                    _stream(stream)), "msa_workspace_init")


def msa_indexer_score(cache, batch, cfg, index_q: Query, pooled, workspace, stream=None) -> None:
    c, b, f, q = cache.struct(), batch.struct(), cfg.struct(), index_q.struct()
    _check(lib().msa_indexer_score(_ref(c), _ref(b), _ref(f), _ref(q), _ptr(pooled), _ptr(workspace),
                                   workspace.numel() * workspace.element_size(), _stream(stream)),
           "msa_indexer_score")


def msa_topk_blocks(batch, cfg, num_groups: int, pooled, topk_idx, topk_score, workspace, stream=None) -> None:
    b, f = batch.struct(), cfg.struct()
    _check(lib().msa_topk_blocks(_ref(b), _ref(f), num_groups, _ptr(pooled), _ptr(topk_idx), _ptr(topk_score),
                                 _ptr(workspace), workspace.numel() * workspace.element_size(),
                                 _stream(stream)), "msa_topk_blocks")


def msa_sparse_attend(cache, batch, cfg, q: Query, num_q_heads: int, topk_idx, out, lse, workspace,
                      stream=None) -> None:
    c, b, f, qq = cache.struct(), batch.struct(), cfg.struct(), q.struct()
    _check(lib().msa_sparse_attend(_ref(c), _ref(b), _ref(f), _ref(qq), num_q_heads, _ptr(topk_idx), _ptr(out),
                                   _ptr(lse), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                   _stream(stream)), "msa_sparse_attend")


def msa_decode(cache, batch, cfg, index_q: Query, q: Query, num_q_heads: int, topk_idx, out, lse, workspace,
               stream=None) -> None:
    c, b, f, iq, qq = cache.struct(), batch.struct(), cfg.struct(), index_q.struct(), q.struct()
    _check(lib().msa_decode(_ref(c), _ref(b), _ref(f), _ref(iq), _ref(qq), num_q_heads, _ptr(topk_idx),
                            _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel() * workspace.element_size(),
                            _stream(stream)), "msa_decode")


def msa_read_device_status(workspace, stream=None):
    """Synchronise, read and clear the device status word: (status code, raw flags)."""
    detail = ctypes.c_int32(0)
    st = lib().msa_read_device_status(_ptr(workspace), _stream(stream), ctypes.byref(detail))
    return int(st), int(detail.value)


def msa_status_string(status: int) -> str:
    return lib().msa_status_string(status).decode()


def msa_dequant_debug(cache, which: int, phys_blocks, out, stream=None) -> None:
    c = cache.struct()
    _check(lib().msa_dequant_debug(_ref(c), which, _ptr(phys_blocks), phys_blocks.numel(), _ptr(out),
                                   _stream(stream)), "msa_dequant_debug")


def msa_decode_noalloc(cache, batch, cfg, index_q: Query, q: Query, num_q_heads: int, topk_idx, out, lse,
                       status_out=None, stream=None) -> None:
    """msa_decode without a caller workspace, for callers that cannot allocate
    device memory (e.g. code living inside another framework's memory pool):
    the library's own fixed scratch array is used instead.  Problems whose
    workspace exceeds the scratch size are rejected; calls must not overlap on
    the GPU because they share that scratch.  status_out: optional device
    int32[2] that receives the call's device status flags."""
    c, b, f, iq, qq = cache.struct(), batch.struct(), cfg.struct(), index_q.struct(), q.struct()
    _check(lib().msa_decode_noalloc(_ref(c), _ref(b), _ref(f), _ref(iq), _ref(qq), num_q_heads, _ptr(topk_idx),
                                    _ptr(out), _ptr(lse), _ptr(status_out), _stream(stream)),
           "msa_decode_noalloc")


def msa_cache_insert(cache, slot_mapping, k, v, index_k, workspace, stream=None) -> None:
    """Quantize and write new tokens' K, V (bf16 [T][H][128]) and index keys (bf16
    [T][128], or None) into the paged caches at slot_mapping (int32 [T])."""
    c = cache.struct()
    _check(lib().msa_cache_insert(_ref(c), int(slot_mapping.numel()), _ptr(slot_mapping), _ptr(k), _ptr(v),
                                  _ptr(index_k), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                  _stream(stream)), "msa_cache_insert")


def msa_dense_workspace_size(cache: PagedCache, batch: Batch, num_q_heads: int) -> int:
    c, b = cache.struct(), batch.struct()
    n = lib().msa_dense_workspace_size(_ref(c), _ref(b), num_q_heads)
    if n == 0:
        raise MsaError(1, "msa_dense_workspace_size")
    return int(n)


def msa_dense_attend(cache, batch, cfg, q: Query, num_q_heads: int, out, lse, workspace, stream=None) -> None:
    """Attention of each new token (up to 8 a sequence) over its whole sequence in the paged cache.
    q.data, out: [S * q_per_seq][num_q_heads][128], lse: fp32 [S * q_per_seq][num_q_heads] or None, all dense."""
    if _int32 is None:
        _torch_names()
    lens, table, data = batch.seq_lens, batch.block_table, q.data
    shape, rows, dev = table.shape, lens.numel() * batch.q_per_seq * num_q_heads, cache.k.get_device()
    if (dev < 0 or dev != _device() or len(shape) != 2 or shape[0] != lens.numel()
            or lens.dtype is not _int32 or table.dtype is not _int32 or not lens.is_contiguous() or not table.is_contiguous()
            or data.numel() != rows * 128 or not data.is_contiguous() or data.dtype not in _query_types.get(q.dtype, ())
            or out.numel() != rows * 128 or not out.is_contiguous() or out.dtype is not _bf16
            or (lse is not None and (lse.numel() != rows or not lse.is_contiguous() or lse.dtype is not _f32
                                    or lse.get_device() != dev))
            or lens.get_device() != dev or table.get_device() != dev or data.get_device() != dev or out.get_device() != dev
            or workspace.get_device() != dev):
        raise MsaError(1, "msa_dense_attend")
    at = _DENSE.pack(*_cache_values(cache, False, dev, "msa_dense_attend"),
                     shape[0], batch.q_per_seq, shape[1], lens.data_ptr(), table.data_ptr(),
                     cfg.topk, cfg.init_blocks, cfg.local_blocks, cfg.index_scale, cfg.sm_scale,
                     SCORE_TYPES.get(cfg.score_type, -1), PREFILL_SELECT.get(cfg.prefill_select, -1),
                     data.data_ptr(), DTYPES[q.dtype], q.scale)
    o = _DENSE.offsets
    _check(lib().msa_dense_attend(at + o[0], at + o[1], at + o[2], at + o[3], num_q_heads, out.data_ptr(), _p(lse),
                                  workspace.data_ptr(), _nbytes(workspace), _stream(stream, dev)), "msa_dense_attend")


def msa_rope_init(rotary_dim: int, theta: float, sections=None, layout: str = "halves") -> MsaRopeT:
    """Rotary positions with one axis, or with len(sections) axes of sections[a] frequency pairs each."""
    sections = [rotary_dim // 2] if sections is None else list(sections)
    r = MsaRopeT()
    arr = (ctypes.c_int32 * max(1, len(sections)))(*sections)
    _check(lib().msa_rope_init(_ref(r), rotary_dim, theta, len(sections), arr, ROPE_LAYOUTS.get(layout, -1)),
           "msa_rope_init")
    return r


def msa_rope_insert(cache, rope: MsaRopeT, positions, slot_mapping, q, q_out: Query, index_q, index_q_out: Optional[Query],
                    k, v, index_k, norm: Optional[QkNorm], workspace, stream=None) -> None:
    """Norm and rotate q, index q, k and index k (bf16 [T][H][128], any token stride), write the
    queries to q_out / index_q_out (dense) and k, v, index k into the paged caches at slot_mapping (int32 [T]).
    positions: int32 [axes][T], or [T] for one axis."""
    if _int32 is None:
        _torch_names()
    where = "msa_rope_insert"
    T, H, dev, qd = slot_mapping.numel(), cache.num_kv_heads, cache.k.get_device(), q_out.data
    if (dev < 0 or dev != _device() or q.dim() != 3
            or positions.numel() != rope.axes * T or positions.dtype is not _int32 or not positions.is_contiguous()
            or slot_mapping.dtype is not _int32 or not slot_mapping.is_contiguous()
            or qd.numel() != q.numel() or not qd.is_contiguous() or qd.dtype not in _query_types.get(q_out.dtype, ())
            or positions.get_device() != dev or slot_mapping.get_device() != dev or q.get_device() != dev or qd.get_device() != dev
            or workspace.get_device() != dev):
        raise MsaError(1, where)
    hq = q.shape[1]
    none, kv = (0, 0), (T, H, 128)
    iqo, w = (0, 0, 0.0), (0, 0, 0, 0, 0.0, 0.0)
    if index_q_out is not None:
        x = index_q_out.data
        if x.numel() != T * H * 128 or not x.is_contiguous() or x.dtype not in _query_types.get(index_q_out.dtype, ()) \
                or x.get_device() != dev:
            raise MsaError(1, where)
        iqo = (x.data_ptr(), DTYPES[index_q_out.dtype], index_q_out.scale)
    if norm is not None:
        w = norm.q, norm.k, norm.index_q, norm.index_k
        for x in w:
            if x is not None and (x.numel() != 128 or x.dtype is not _bf16 or not x.is_contiguous() or x.get_device() != dev):
                raise MsaError(1, where)
        w = (_p(norm.q), _p(norm.k), _p(norm.index_q), _p(norm.index_k), norm.eps, norm.offset)
    at = _ROPE.pack(*_cache_values(cache, index_k is not None, dev, where),
                    *_rows(q, (T, hq, 128), where, dev), qd.data_ptr(), DTYPES[q_out.dtype], q_out.scale,
                    *(none if index_q is None else _rows(index_q, kv, where, dev)), *iqo, *_rows(k, kv, where, dev),
                    *_rows(v, kv, where, dev), *(none if index_k is None else
                                             _rows(index_k, (T, 128) if index_k.dim() == 2 else (T, 1, 128), where, dev)), *w)
    o = _ROPE.offsets
    _check(lib().msa_rope_insert(at, ctypes.byref(rope), T, positions.data_ptr(), slot_mapping.data_ptr(), hq, at + o[1], at + o[2],
                                 0 if index_q is None else at + o[3], 0 if index_q_out is None else at + o[4], at + o[5],
                                 at + o[6], 0 if index_k is None else at + o[7], 0 if norm is None else at + o[8],
                                 workspace.data_ptr(), _nbytes(workspace), _stream(stream, dev)), where)


def msa_build_tables(num_blocks: int, cached_lens, new_lens, block_table, free_blocks, free_count, seq_lens, token_offsets,
                     slot_mapping, positions, free_count_out, workspace, stream=None) -> None:
    """Block tables, lengths, slots and positions of a step from the requests' lengths (all int32 on the
    device): block_table [S][max_blocks] and the stack free_blocks are updated in place; seq_lens [S],
    token_offsets [S + 1], slot_mapping and positions [max_tokens] and free_count_out [1] are written."""
    if _int32 is None:
        _torch_names()
    where, dev = "msa_build_tables", block_table.get_device()
    S, shape, tokens = cached_lens.numel(), block_table.shape, slot_mapping.numel()
    if (dev < 0 or dev != _device() or new_lens.numel() != S or len(shape) != 2 or shape[0] != S
            or seq_lens.numel() != S or token_offsets.numel() != S + 1 or positions.numel() != tokens or workspace.get_device() != dev):
        raise MsaError(1, where)
    for t in (cached_lens, new_lens, block_table, free_blocks, free_count, seq_lens, token_offsets, slot_mapping, positions,
              free_count_out):
        if t.dtype is not _int32 or t.get_device() != dev or not t.is_contiguous():
            raise MsaError(1, where)
    _check(lib().msa_build_tables(S, num_blocks, cached_lens.data_ptr(), new_lens.data_ptr(), shape[1], block_table.data_ptr(),
                                  free_blocks.numel(), free_blocks.data_ptr(), free_count.data_ptr(), free_count_out.data_ptr(),
                                  seq_lens.data_ptr(), token_offsets.data_ptr(), tokens, slot_mapping.data_ptr(),
                                  positions.data_ptr(), workspace.data_ptr(), _nbytes(workspace), _stream(stream, dev)), where)


def default_config(topk: int = 16, head_dim: int = 128, index_dim: int = 128) -> Config:
    """The model's settings: index and softmax scales head_dim ** -0.5."""
    return Config(topk=topk, index_scale=index_dim ** -0.5, sm_scale=head_dim ** -0.5)


__all__ = ["PagedCache", "Batch", "Config", "Query", "QkNorm", "MsaError", "lib", "EXPORTS", "default_config",
           "msa_workspace_size", "msa_workspace_init", "msa_indexer_score", "msa_topk_blocks",
           "msa_sparse_attend", "msa_decode", "msa_read_device_status", "msa_status_string",
           "msa_dequant_debug", "msa_decode_noalloc", "msa_cache_insert", "msa_dense_workspace_size", "msa_dense_attend",
           "msa_rope_init", "msa_rope_insert", "msa_build_tables", "roofline"]
