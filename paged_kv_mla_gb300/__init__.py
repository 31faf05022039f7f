"""Python binding of the GB300 paged-KV MLA library (libpaged_kv_mla.so).

Argument marshalling only: torch tensors are turned into device pointers and the current
torch CUDA stream is passed as the cudaStream_t; every step of the computation runs in the
library's sm_103a kernels.  There is no CPU path: if the shared library is missing this
module refuses to import, and every call raises on a non-OK status.

Entry points (same names as the C ABI in include/paged_kv_mla.h):
  mla_decompress_k_paged              generic_flare_mla_decompress_k_cache_ragged_paged (bf16)
  mla_decompress_kv_paged             the same gather feeding the K and the V (w_uv) projections
  mla_decompress_k_paged_fp8          the K-decompress stage of mla_prefill_decode_graph_fp8
                                      (+ mla_decompress_k_paged_fp8_workspace_size)
  mla_decompress_kv_paged_fp8         its K and V form
  mla_decompress_k_paged_fp8_noalloc  the FP8 decompress with a fixed in-library workspace
  mla_decompress_k_paged_fp8_qcache   the FP8 decompress reading a quantised paged cache
  mla_cache_write_paged               RMSNorm + RoPE of new latent rows into the paged cache
  mla_cache_write_paged_qcache        the same into a quantised paged cache
  mla_cache_write_paged_at            both with rotary positions given apart from the slots
    (+ _qcache_at)
  mla_tree_attention_paged            attention of new tokens (one, a chain, a drafted tree)
    (+ _qcache, _workspace_size)      over the paged latent cache, in latent space
  mla_rope_heads                      rotation of the queries' rope columns at given positions
  mla_cache_compact_paged (+ _qcache) accepted drafts moved to the front of their region
  kv_matmul_paged                     kv_matmul_ragged_paged (bf16)
  kv_matmul_paged_fp8                 its FP8 block-scaled form (+ kv_matmul_paged_fp8_workspace_size)
  pkm_check_wait_timeout              the bounded-wait self-check
  pkm_validate_row_offsets            the opt-in check that an offset array is non-decreasing
  status_string, last_cuda_error      pkm_status_string, pkm_last_cuda_error
"""
from __future__ import annotations

import ctypes
import os
import threading
from dataclasses import dataclass
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpaged_kv_mla.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build the CUDA library first "
        "(python paged_kv_mla_gb300/build.py, or __graft_entry__.build()).")

_lib = ctypes.CDLL(LIB_PATH)

PKM_OK = 0
PKM_ERR_INVALID_ARG = 1
PKM_ERR_UNSUPPORTED = 2
PKM_ERR_CUDA = 3
PKM_ERR_OUT_OF_RANGE = 4
PKM_ERR_TIMEOUT = 5


class PkmError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        msg = f"{where}: {status_string(code)} ({code})"
        if code == PKM_ERR_CUDA:
            msg += f": {last_cuda_error()}"
        super().__init__(msg)


class _CCache(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("layer_stride", ctypes.c_int64),
                ("page_stride", ctypes.c_int64), ("slot_stride", ctypes.c_int64),
                ("kv_stride", ctypes.c_int64), ("num_layers", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("row_elems", ctypes.c_int32), ("page_table", ctypes.c_void_p),
                ("max_pages_per_seq", ctypes.c_int32), ("cache_lengths", ctypes.c_void_p)]


class _CQuantCache(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("layer_stride", ctypes.c_int64),
                ("page_stride", ctypes.c_int64), ("slot_stride", ctypes.c_int64),
                ("num_layers", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("kv_lora_rank", ctypes.c_int32),
                ("rope_dim", ctypes.c_int32), ("page_table", ctypes.c_void_p),
                ("max_pages_per_seq", ctypes.c_int32), ("cache_lengths", ctypes.c_void_p)]


_vp, _i32, _u32, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_uint32, ctypes.c_size_t
_lib.pkm_status_string.argtypes = [ctypes.c_int]
_lib.pkm_status_string.restype = ctypes.c_char_p
_lib.pkm_last_cuda_error.argtypes = []
_lib.pkm_last_cuda_error.restype = ctypes.c_char_p
_lib.mla_decompress_k_paged.argtypes = [ctypes.POINTER(_CCache), _u32, _vp, _vp, _i32, _i32, _i32,
                                        _i32, _vp, _i32, _vp, _vp, _vp, _vp]
_lib.mla_decompress_k_paged.restype = ctypes.c_int
_lib.mla_decompress_k_paged_fp8_workspace_size.argtypes = [_i32, _i32]
_lib.mla_decompress_k_paged_fp8_workspace_size.restype = _sz
_lib.mla_decompress_k_paged_fp8.argtypes = [ctypes.POINTER(_CCache), _u32, _vp, _vp, _i32, _i32,
                                            _i32, _i32, _vp, _vp, _i32, _vp, _vp, _vp, _sz, _vp,
                                            _vp]
_lib.mla_decompress_k_paged_fp8.restype = ctypes.c_int
_lib.mla_decompress_k_paged_fp8_qcache.argtypes = [ctypes.POINTER(_CQuantCache), _u32, _vp, _vp,
                                                   _i32, _i32, _vp, _vp, _i32, _vp, _vp, _vp,
                                                   _sz, _vp, _vp]
_lib.mla_decompress_k_paged_fp8_qcache.restype = ctypes.c_int
_lib.mla_cache_write_paged_qcache.argtypes = [_vp, _vp, _i32, _i32, _vp, ctypes.c_float, _vp,
                                              _i32, ctypes.POINTER(_CQuantCache), _u32, _vp, _vp]
_lib.mla_cache_write_paged_qcache.restype = ctypes.c_int
_f32, _i64 = ctypes.c_float, ctypes.c_int64
_lib.mla_cache_write_paged_at.argtypes = [_vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp, _f32, _vp,
                                          _i32, ctypes.POINTER(_CCache), _u32, _vp, _vp]
_lib.mla_cache_write_paged_at.restype = ctypes.c_int
_lib.mla_cache_write_paged_qcache_at.argtypes = [_vp, _vp, _vp, _i32, _i32, _vp, _f32, _vp, _i32,
                                                 ctypes.POINTER(_CQuantCache), _u32, _vp, _vp]
_lib.mla_cache_write_paged_qcache_at.restype = ctypes.c_int
_lib.mla_rope_heads.argtypes = [_vp, _i64, _i64, _vp, _i32, _i32, _i32, _vp, _i32, _i32, _vp, _i64,
                                _i64, _vp, _vp]
_lib.mla_rope_heads.restype = ctypes.c_int
_lib.mla_tree_attention_paged_workspace_size.argtypes = [_i32, _i32, _i32]
_lib.mla_tree_attention_paged_workspace_size.restype = _sz
_lib.mla_tree_attention_paged.argtypes = [_vp, _vp, _i32, _i32, _i32, _i32, _i32, _f32, _vp, _i32,
                                          ctypes.POINTER(_CCache), _u32, _vp, _vp, _vp, _sz, _vp,
                                          _vp]
_lib.mla_tree_attention_paged.restype = ctypes.c_int
_lib.mla_tree_attention_paged_qcache.argtypes = [_vp, _vp, _i32, _i32, _i32, _f32, _vp, _i32,
                                                 ctypes.POINTER(_CQuantCache), _u32, _vp, _vp,
                                                 _vp, _sz, _vp, _vp]
_lib.mla_tree_attention_paged_qcache.restype = ctypes.c_int
_lib.mla_cache_compact_paged.argtypes = [ctypes.POINTER(_CCache), _u32, _i32, _i32, _vp, _i32, _vp,
                                         _vp, _vp, _vp]
_lib.mla_cache_compact_paged.restype = ctypes.c_int
_lib.mla_cache_compact_paged_qcache.argtypes = [ctypes.POINTER(_CQuantCache), _u32, _i32, _i32,
                                                _vp, _i32, _vp, _vp, _vp, _vp]
_lib.mla_cache_compact_paged_qcache.restype = ctypes.c_int
_lib.mla_decompress_kv_paged.argtypes = [ctypes.POINTER(_CCache), _u32, _vp, _vp, _i32, _i32, _i32,
                                         _i32, _vp, _i32, _vp, _i32, _i32, _vp, _vp, _vp, _vp, _vp]
_lib.mla_decompress_kv_paged.restype = ctypes.c_int
_lib.mla_decompress_kv_paged_fp8.argtypes = [ctypes.POINTER(_CCache), _u32, _vp, _vp, _i32, _i32,
                                             _i32, _i32, _vp, _vp, _i32, _vp, _vp, _i32, _i32, _vp,
                                             _vp, _vp, _vp, _sz, _vp, _vp]
_lib.mla_decompress_kv_paged_fp8.restype = ctypes.c_int
_lib.mla_cache_write_paged.argtypes = [_vp, _vp, _i32, _i32, _i32, _i32, _vp, ctypes.c_float, _vp,
                                       _i32, ctypes.POINTER(_CCache), _u32, _vp, _vp]
_lib.mla_cache_write_paged.restype = ctypes.c_int
_lib.kv_matmul_paged_fp8_workspace_size.argtypes = [_i32, _i32]
_lib.kv_matmul_paged_fp8_workspace_size.restype = _sz
_lib.kv_matmul_paged_fp8.argtypes = [_vp, _vp, _i32, _i32, _i32, _vp, _vp, _i32,
                                     ctypes.POINTER(_CCache), _u32, _vp, _sz, _vp, _vp]
_lib.kv_matmul_paged_fp8.restype = ctypes.c_int
_lib.kv_matmul_paged.argtypes = [_vp, _vp, _i32, _i32, _i32, _vp, _i32, ctypes.POINTER(_CCache),
                                 _u32, _vp, _vp]
_lib.kv_matmul_paged.restype = ctypes.c_int
_lib.mla_decompress_k_paged_fp8_noalloc.argtypes = [ctypes.POINTER(_CCache), _u32, _vp, _vp, _i32,
                                                    _i32, _i32, _i32, _vp, _vp, _i32, _vp, _vp,
                                                    _vp, _vp]
_lib.mla_decompress_k_paged_fp8_noalloc.restype = ctypes.c_int
FP8_NOALLOC_SCRATCH_BYTES = 16 << 20
_lib.pkm_checks_only.argtypes = [_i32]
_lib.pkm_checks_only.restype = None
_lib.pkm_check_wait_timeout.argtypes = [_vp, _u32, _vp]
_lib.pkm_check_wait_timeout.restype = ctypes.c_int
_lib.pkm_validate_row_offsets.argtypes = [_vp, _i32, _vp, _vp]
_lib.pkm_validate_row_offsets.restype = ctypes.c_int


def status_string(code: int) -> str:
    return _lib.pkm_status_string(int(code)).decode()


def last_cuda_error() -> str:
    """What lies behind the last PKM_ERR_CUDA the library returned on this thread."""
    return _lib.pkm_last_cuda_error().decode()


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        return int(t)
    return t.data_ptr()


def _current_stream() -> int:
    """torch.cuda.current_stream().cuda_stream, without building the stream object: that takes
    a quarter of a small call's time on the host."""
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


if not (hasattr(torch._C, "_cuda_getCurrentRawStream") and hasattr(torch._C, "_cuda_getDevice")):
    def _current_stream() -> int:  # noqa: F811
        return torch.cuda.current_stream().cuda_stream


def _stream(stream) -> Optional[int]:
    if stream is None:
        return _current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


class _Descriptor:
    """Keeps the C struct of a cache descriptor from call to call, as long as no field is
    assigned; the tensors' addresses and the table's width are read anew for every call.

    Every assignment is followed by a new mark, and a struct is kept together with the mark that
    was there before its fields were read: one that was built beside an assignment in another
    thread is not used again.  Each thread keeps its own, so that no other one changes a struct
    while a call reads it."""

    def __setattr__(self, name, value):
        self.__dict__[name] = value
        self.__dict__["_mark"] = object()

    def __getstate__(self):  # copies and pickles make their own
        return {k: v for k, v in self.__dict__.items() if k not in ("_mark", "_kept")}

    def c_struct(self):
        d = self.__dict__
        kept = d.get("_kept")
        if kept is None:
            kept = d.setdefault("_kept", threading.local())
        mark = d.get("_mark")
        try:
            c, made = kept.struct
        except AttributeError:
            c = made = None
        if c is None or made is not mark:
            c = self._new_struct()
            kept.struct = c, mark
        else:
            table = self.page_table
            c.data = self.data.data_ptr()
            c.page_table = table.data_ptr()
            c.max_pages_per_seq = table.shape[-1]
            c.cache_lengths = _ptr(self.cache_lengths)
        return c


@dataclass
class PagedCache(_Descriptor):
    """A paged cache (all layers) described by element strides; see pkm_paged_cache.

    data: bf16 storage (any shape; only its base pointer is used).
    page_table: uint32/int32 [batch, max_pages_per_seq].
    cache_lengths: uint32/int32 [batch] (every call but the decompress ones).
    """
    data: torch.Tensor
    page_table: torch.Tensor
    layer_stride: int
    page_stride: int
    slot_stride: int
    num_layers: int
    num_pages: int
    page_size: int
    row_elems: int
    kv_stride: int = 0
    cache_lengths: Optional[torch.Tensor] = None

    def _new_struct(self) -> _CCache:
        table = self.page_table  # once: another thread may assign it
        return _CCache(self.data.data_ptr(), int(self.layer_stride), int(self.page_stride),
                       int(self.slot_stride), int(self.kv_stride), int(self.num_layers),
                       int(self.num_pages), int(self.page_size), int(self.row_elems),
                       table.data_ptr(), int(table.shape[-1]),
                       _ptr(self.cache_lengths))


@dataclass
class QuantCache(_Descriptor):
    """A quantised paged latent cache described by byte strides; see pkm_quant_cache.

    data: storage of the slots (any dtype and shape; only its base pointer is used).  A slot
    holds kv_lora_rank e4m3 codes, rope_dim bf16 values and kv_lora_rank/128 fp32 scales.
    """
    data: torch.Tensor
    page_table: torch.Tensor
    layer_stride: int
    page_stride: int
    slot_stride: int
    num_layers: int
    num_pages: int
    page_size: int
    kv_lora_rank: int
    rope_dim: int
    cache_lengths: Optional[torch.Tensor] = None

    def _new_struct(self) -> _CQuantCache:
        table = self.page_table  # once: another thread may assign it
        return _CQuantCache(self.data.data_ptr(), int(self.layer_stride), int(self.page_stride),
                            int(self.slot_stride), int(self.num_layers), int(self.num_pages),
                            int(self.page_size), int(self.kv_lora_rank), int(self.rope_dim),
                            table.data_ptr(), int(table.shape[-1]),
                            _ptr(self.cache_lengths))


def _check(code: int, where: str, check: bool) -> int:
    if check and code != PKM_OK:
        raise PkmError(code, where)
    return code


def mla_decompress_k_paged(cache: PagedCache, layer_idx: int, buffer_row_offsets: torch.Tensor,
                           cache_offsets: torch.Tensor, buffer_length: int, kv_lora_rank: int,
                           rope_dim: int, w_k: torch.Tensor, k_latent_buffer: torch.Tensor,
                           k_buffer: torch.Tensor, dev_status: Optional[torch.Tensor] = None,
                           stream=None, check: bool = True) -> int:
    c = cache.c_struct()
    batch = int(buffer_row_offsets.shape[0]) - 1
    code = _lib.mla_decompress_k_paged(ctypes.byref(c), int(layer_idx), _ptr(buffer_row_offsets),
                                       _ptr(cache_offsets), batch, int(buffer_length),
                                       int(kv_lora_rank), int(rope_dim), _ptr(w_k),
                                       int(w_k.shape[0]), _ptr(k_latent_buffer), _ptr(k_buffer),
                                       _ptr(dev_status), _stream(stream))
    return _check(code, "mla_decompress_k_paged", check)


def mla_decompress_kv_paged(cache: PagedCache, layer_idx: int, buffer_row_offsets: torch.Tensor,
                            cache_offsets: torch.Tensor, buffer_length: int, kv_lora_rank: int,
                            rope_dim: int, w_k: torch.Tensor, w_uv: torch.Tensor,
                            k_latent_buffer: torch.Tensor, k_buffer: torch.Tensor,
                            v_buffer: torch.Tensor, dev_status: Optional[torch.Tensor] = None,
                            stream=None, check: bool = True) -> int:
    """K and V from one gather; w_uv is [num_heads, v_head_dim, kv_lora_rank]."""
    c = cache.c_struct()
    batch = int(buffer_row_offsets.shape[0]) - 1
    code = _lib.mla_decompress_kv_paged(ctypes.byref(c), int(layer_idx), _ptr(buffer_row_offsets),
                                        _ptr(cache_offsets), batch, int(buffer_length),
                                        int(kv_lora_rank), int(rope_dim), _ptr(w_k),
                                        int(w_k.shape[0]), _ptr(w_uv), int(w_uv.shape[0]),
                                        int(w_uv.shape[1]), _ptr(k_latent_buffer), _ptr(k_buffer),
                                        _ptr(v_buffer), _ptr(dev_status), _stream(stream))
    return _check(code, "mla_decompress_kv_paged", check)


def mla_decompress_k_paged_fp8_workspace_size(buffer_length: int, kv_lora_rank: int) -> int:
    return int(_lib.mla_decompress_k_paged_fp8_workspace_size(int(buffer_length), int(kv_lora_rank)))


def fp8_workspace_views(workspace: torch.Tensor, buffer_length: int, kv_lora_rank: int):
    """(q_latent [L, R] uint8, q_scale [L, R/128] float32) views of an FP8 workspace."""
    L, R = int(buffer_length), int(kv_lora_rank)
    q = workspace[: L * R].view(L, R)
    off = (L * R + 255) // 256 * 256
    s = workspace[off: off + L * (R // 128) * 4].view(torch.float32).view(L, R // 128)
    return q, s


def mla_decompress_k_paged_fp8(cache: PagedCache, layer_idx: int,
                               buffer_row_offsets: torch.Tensor, cache_offsets: torch.Tensor,
                               buffer_length: int, kv_lora_rank: int, rope_dim: int,
                               w_k_e4m3: torch.Tensor, w_k_scale: torch.Tensor,
                               k_latent_buffer: torch.Tensor, k_buffer: torch.Tensor,
                               workspace: torch.Tensor, dev_status: Optional[torch.Tensor] = None,
                               stream=None, check: bool = True) -> int:
    c = cache.c_struct()
    batch = int(buffer_row_offsets.shape[0]) - 1
    code = _lib.mla_decompress_k_paged_fp8(
        ctypes.byref(c), int(layer_idx), _ptr(buffer_row_offsets), _ptr(cache_offsets), batch,
        int(buffer_length), int(kv_lora_rank), int(rope_dim), _ptr(w_k_e4m3), _ptr(w_k_scale),
        int(w_k_e4m3.shape[0]), _ptr(k_latent_buffer), _ptr(k_buffer), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(dev_status), _stream(stream))
    return _check(code, "mla_decompress_k_paged_fp8", check)


def mla_decompress_k_paged_fp8_qcache(cache: QuantCache, layer_idx: int,
                                      buffer_row_offsets: torch.Tensor, cache_offsets: torch.Tensor,
                                      buffer_length: int, w_k_e4m3: torch.Tensor,
                                      w_k_scale: torch.Tensor, k_latent_buffer: Optional[torch.Tensor],
                                      k_buffer: torch.Tensor, workspace: torch.Tensor,
                                      dev_status: Optional[torch.Tensor] = None, stream=None,
                                      check: bool = True) -> int:
    """FP8 decompress reading codes and scales straight from a quantised cache;
    k_latent_buffer (dequantised bf16 rows) may be None."""
    c = cache.c_struct()
    batch = int(buffer_row_offsets.shape[0]) - 1
    code = _lib.mla_decompress_k_paged_fp8_qcache(
        ctypes.byref(c), int(layer_idx), _ptr(buffer_row_offsets), _ptr(cache_offsets), batch,
        int(buffer_length), _ptr(w_k_e4m3), _ptr(w_k_scale), int(w_k_e4m3.shape[0]),
        _ptr(k_latent_buffer), _ptr(k_buffer), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(dev_status), _stream(stream))
    return _check(code, "mla_decompress_k_paged_fp8_qcache", check)


def mla_cache_write_paged_qcache(latent: torch.Tensor, input_row_offsets: torch.Tensor,
                                 kv_norm_gamma: torch.Tensor, epsilon: float,
                                 freqs_cis: torch.Tensor, cache: QuantCache, layer_idx: int,
                                 dev_status: Optional[torch.Tensor] = None, stream=None,
                                 check: bool = True) -> int:
    """RMSNorm + RoPE of new latent rows, quantised into a quantised cache's slots."""
    c = cache.c_struct()
    batch = int(input_row_offsets.shape[0]) - 1
    code = _lib.mla_cache_write_paged_qcache(_ptr(latent), _ptr(input_row_offsets), batch,
                                             int(latent.shape[0]), _ptr(kv_norm_gamma),
                                             float(epsilon), _ptr(freqs_cis),
                                             int(freqs_cis.shape[0]), ctypes.byref(c),
                                             int(layer_idx), _ptr(dev_status), _stream(stream))
    return _check(code, "mla_cache_write_paged_qcache", check)


def mla_decompress_kv_paged_fp8(cache: PagedCache, layer_idx: int,
                                buffer_row_offsets: torch.Tensor, cache_offsets: torch.Tensor,
                                buffer_length: int, kv_lora_rank: int, rope_dim: int,
                                w_k_e4m3: torch.Tensor, w_k_scale: torch.Tensor,
                                w_uv_e4m3: torch.Tensor, w_uv_scale: torch.Tensor,
                                k_latent_buffer: torch.Tensor, k_buffer: torch.Tensor,
                                v_buffer: torch.Tensor, workspace: torch.Tensor,
                                dev_status: Optional[torch.Tensor] = None, stream=None,
                                check: bool = True) -> int:
    """FP8 K and V from one gather and one activation quantisation."""
    c = cache.c_struct()
    batch = int(buffer_row_offsets.shape[0]) - 1
    code = _lib.mla_decompress_kv_paged_fp8(
        ctypes.byref(c), int(layer_idx), _ptr(buffer_row_offsets), _ptr(cache_offsets), batch,
        int(buffer_length), int(kv_lora_rank), int(rope_dim), _ptr(w_k_e4m3), _ptr(w_k_scale),
        int(w_k_e4m3.shape[0]), _ptr(w_uv_e4m3), _ptr(w_uv_scale), int(w_uv_e4m3.shape[0]),
        int(w_uv_e4m3.shape[1]), _ptr(k_latent_buffer), _ptr(k_buffer), _ptr(v_buffer),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(dev_status),
        _stream(stream))
    return _check(code, "mla_decompress_kv_paged_fp8", check)


def mla_cache_write_paged(latent: torch.Tensor, input_row_offsets: torch.Tensor,
                          kv_norm_gamma: torch.Tensor, epsilon: float, freqs_cis: torch.Tensor,
                          cache: PagedCache, layer_idx: int, kv_lora_rank: int, rope_dim: int,
                          dev_status: Optional[torch.Tensor] = None, stream=None,
                          check: bool = True) -> int:
    """RMSNorm + RoPE of new latent rows [total_rows, R + P] into the paged latent cache."""
    c = cache.c_struct()
    batch = int(input_row_offsets.shape[0]) - 1
    code = _lib.mla_cache_write_paged(_ptr(latent), _ptr(input_row_offsets), batch,
                                      int(latent.shape[0]), int(kv_lora_rank), int(rope_dim),
                                      _ptr(kv_norm_gamma), float(epsilon), _ptr(freqs_cis),
                                      int(freqs_cis.shape[0]), ctypes.byref(c), int(layer_idx),
                                      _ptr(dev_status), _stream(stream))
    return _check(code, "mla_cache_write_paged", check)


_initialized = torch.cuda.is_initialized


# Element types that the C calls read as what they are named for: bf16 values or their bits.
_BF16 = (torch.bfloat16, torch.int16, torch.uint16)
_WORD = (torch.int32, torch.uint32)
_FLOAT = (torch.float32,)


def _plain(types: tuple, *tensors) -> bool:
    """Whether the tensors have one of the types and no gaps (None and addresses pass)."""
    for t in tensors:
        if t is None or t.__class__ is int:
            continue
        if t.dtype not in types or not t.is_contiguous():
            return False
    return True


def _here(*tensors) -> bool:
    """Whether the tensors lie on the device that the call runs on (None and addresses pass).
    While CUDA is not initialised no tensor does."""
    device = torch._C._cuda_getDevice() if _initialized() else None
    for t in tensors:
        if t is not None and t.__class__ is not int and t.get_device() != device:
            return False
    return True


def _refuse(f, *args) -> int:
    """The status of a call whose tensors are not _here: what its own checks find, if anything.
    `args` end before the stream."""
    _lib.pkm_checks_only(1)
    try:
        code = f(*args, None)
    finally:
        _lib.pkm_checks_only(0)
    return PKM_ERR_INVALID_ARG if code == PKM_ERR_CUDA else code


def _has(n: int, t) -> bool:
    """At least n elements, as far as can be seen."""
    return t is None or t.__class__ is int or t.numel() >= n


def _cache_ok(cache, batch: int) -> bool:
    """A table row and a length for each request (and maybe for more)."""
    table, lengths = cache.page_table, cache.cache_lengths
    return (table.ndim == 2 and table.shape[0] >= batch and _has(batch, lengths) and
            _plain(_WORD, table, lengths))


def _rows_ok(latent, offsets, positions, gamma, freqs, cache, rank, rope) -> bool:
    """Rows of R + P columns with a position each, R factors of the norm, P of a position (or for a
    P of 0 any), and a descriptor for the requests that the offsets tell of."""
    return (latent.ndim == 2 and latent.shape[1] == rank + rope and
            _has(latent.shape[0], positions) and _has(rank, gamma) and
            (rope == 0 or (freqs.ndim == 2 and freqs.shape[1] == rope)) and
            _cache_ok(cache, offsets.shape[0] - 1) and _plain(_BF16, latent) and
            _plain(_WORD, offsets, positions) and _plain(_FLOAT, gamma, freqs))


def mla_cache_write_paged_at(latent: torch.Tensor, input_row_offsets: torch.Tensor,
                             positions: torch.Tensor, kv_norm_gamma: torch.Tensor,
                             epsilon: float, freqs_cis: torch.Tensor, cache: PagedCache,
                             layer_idx: int, kv_lora_rank: int, rope_dim: int,
                             dev_status: Optional[torch.Tensor] = None, stream=None,
                             check: bool = True) -> int:
    """mla_cache_write_paged with row r rotated by freqs_cis[positions[r]] (positions:
    uint32/int32 [total_rows]), wherever its slot is."""
    if not _rows_ok(latent, input_row_offsets, positions, kv_norm_gamma, freqs_cis, cache,
                    kv_lora_rank, rope_dim):
        return _check(PKM_ERR_INVALID_ARG, "mla_cache_write_paged_at", check)
    c = cache.c_struct()
    rows, batch = latent.shape[0], input_row_offsets.shape[0] - 1
    args = (_ptr(latent), _ptr(input_row_offsets), _ptr(positions), batch, rows,
            int(kv_lora_rank), int(rope_dim), _ptr(kv_norm_gamma), float(epsilon),
            _ptr(freqs_cis), freqs_cis.shape[0], ctypes.byref(c), int(layer_idx),
            _ptr(dev_status))
    f = _lib.mla_cache_write_paged_at
    here = _here(latent, input_row_offsets, positions, kv_norm_gamma, freqs_cis, cache.data,
                 cache.page_table, cache.cache_lengths)
    code = f(*args, _stream(stream)) if here else _refuse(f, *args)
    return _check(code, "mla_cache_write_paged_at", check)


def mla_cache_write_paged_qcache_at(latent: torch.Tensor, input_row_offsets: torch.Tensor,
                                    positions: torch.Tensor, kv_norm_gamma: torch.Tensor,
                                    epsilon: float, freqs_cis: torch.Tensor, cache: QuantCache,
                                    layer_idx: int, dev_status: Optional[torch.Tensor] = None,
                                    stream=None, check: bool = True) -> int:
    """mla_cache_write_paged_qcache with row r rotated by freqs_cis[positions[r]]."""
    if not _rows_ok(latent, input_row_offsets, positions, kv_norm_gamma, freqs_cis, cache,
                    cache.kv_lora_rank, cache.rope_dim):
        return _check(PKM_ERR_INVALID_ARG, "mla_cache_write_paged_qcache_at", check)
    c = cache.c_struct()
    rows, batch = latent.shape[0], input_row_offsets.shape[0] - 1
    args = (_ptr(latent), _ptr(input_row_offsets), _ptr(positions), batch, rows,
            _ptr(kv_norm_gamma), float(epsilon), _ptr(freqs_cis), int(freqs_cis.shape[0]),
            ctypes.byref(c), int(layer_idx), _ptr(dev_status))
    f = _lib.mla_cache_write_paged_qcache_at
    here = _here(latent, input_row_offsets, positions, kv_norm_gamma, freqs_cis, cache.data,
                 cache.page_table, cache.cache_lengths)
    code = f(*args, _stream(stream)) if here else _refuse(f, *args)
    return _check(code, "mla_cache_write_paged_qcache_at", check)


def mla_rope_heads(x: torch.Tensor, positions: torch.Tensor, freqs_cis: torch.Tensor,
                   y: torch.Tensor, half: bool = False,
                   dev_status: Optional[torch.Tensor] = None, stream=None,
                   check: bool = True) -> int:
    """Rotates x [rows, heads, P] into y [rows, heads, P] (bf16 views with contiguous last
    dimensions; y may be x) by the (cos, sin) pairs of freqs_cis[positions[row]]: pairs
    (2j, 2j + 1), or (j, j + P/2) with `half`."""
    shape, sx, sy = x.shape, x.stride(), y.stride()
    if y.shape != shape or len(shape) != 3 or sx[2] != 1 or sy[2] != 1 \
            or x.dtype not in _BF16 or y.dtype not in _BF16 or positions.numel() != shape[0] \
            or freqs_cis.shape[-1] != shape[2] or not _plain(_WORD, positions) \
            or not _plain(_FLOAT, freqs_cis):
        return _check(PKM_ERR_INVALID_ARG, "mla_rope_heads", check)
    args = (x.data_ptr(), sx[0], sx[1], _ptr(positions), shape[0], shape[1], shape[2],
            freqs_cis.data_ptr(), freqs_cis.shape[0], 1 if half else 0, y.data_ptr(), sy[0],
            sy[1], _ptr(dev_status))
    f = _lib.mla_rope_heads
    code = f(*args, _stream(stream)) if _here(x, positions, freqs_cis, y) else _refuse(f, *args)
    return _check(code, "mla_rope_heads", check)


def mla_tree_attention_paged_workspace_size(total_rows: int, num_heads: int,
                                            kv_lora_rank: int) -> int:
    return int(_lib.mla_tree_attention_paged_workspace_size(int(total_rows), int(num_heads),
                                                            int(kv_lora_rank)))


def _tree_shapes_ok(q, offsets, tree_mask, cache, out, lse, workspace, rank, rope) -> bool:
    """Shapes that the C call cannot see; an empty mask would pass for no mask there."""
    if q.ndim != 3:
        return False
    rows, heads, cols = q.shape
    return (cols == rank + rope and out.shape == (rows, heads, rank) and
            (lse is None or lse.shape == (rows, heads)) and
            (tree_mask is None or (tree_mask.ndim == 2 and tree_mask.shape[0] == rows and
                                   tree_mask.shape[1] > 0)) and
            _cache_ok(cache, offsets.shape[0] - 1) and
            _plain(_BF16, q, out) and _plain(_WORD, offsets, tree_mask) and
            _plain(_FLOAT, lse) and workspace.is_contiguous())


def mla_tree_attention_paged(q: torch.Tensor, input_row_offsets: torch.Tensor,
                             softmax_scale: float, cache: PagedCache, layer_idx: int,
                             kv_lora_rank: int, rope_dim: int, out: torch.Tensor,
                             workspace: torch.Tensor, tree_mask: Optional[torch.Tensor] = None,
                             lse: Optional[torch.Tensor] = None,
                             dev_status: Optional[torch.Tensor] = None, stream=None,
                             check: bool = True) -> int:
    """Attention of the new tokens' latent-space queries q [total_rows, heads, R + P] over the
    cache: each over its request's cached tokens and those new ones that its tree_mask row
    (uint32/int32 [total_rows, words], one bit a token; None: the tokens up to itself) names.
    out [total_rows, heads, R] bf16, lse [total_rows, heads] fp32 or None."""
    if not _tree_shapes_ok(q, input_row_offsets, tree_mask, cache, out, lse, workspace,
                           kv_lora_rank, rope_dim):
        return _check(PKM_ERR_INVALID_ARG, "mla_tree_attention_paged", check)
    c = cache.c_struct()
    rows, heads, _ = q.shape
    args = (q.data_ptr(), input_row_offsets.data_ptr(), input_row_offsets.shape[0] - 1, rows,
            heads, int(kv_lora_rank), int(rope_dim), float(softmax_scale), _ptr(tree_mask),
            0 if tree_mask is None else tree_mask.shape[1], ctypes.byref(c), int(layer_idx),
            out.data_ptr(), _ptr(lse), workspace.data_ptr(), workspace.nbytes, _ptr(dev_status))
    f = _lib.mla_tree_attention_paged
    here = _here(q, input_row_offsets, tree_mask, out, lse, workspace, cache.data,
                 cache.page_table, cache.cache_lengths)
    code = f(*args, _stream(stream)) if here else _refuse(f, *args)
    return _check(code, "mla_tree_attention_paged", check)


def mla_tree_attention_paged_qcache(q: torch.Tensor, input_row_offsets: torch.Tensor,
                                    softmax_scale: float, cache: QuantCache, layer_idx: int,
                                    out: torch.Tensor, workspace: torch.Tensor,
                                    tree_mask: Optional[torch.Tensor] = None,
                                    lse: Optional[torch.Tensor] = None,
                                    dev_status: Optional[torch.Tensor] = None, stream=None,
                                    check: bool = True) -> int:
    """mla_tree_attention_paged over a quantised cache."""
    if not _tree_shapes_ok(q, input_row_offsets, tree_mask, cache, out, lse, workspace,
                           cache.kv_lora_rank, cache.rope_dim):
        return _check(PKM_ERR_INVALID_ARG, "mla_tree_attention_paged_qcache", check)
    c = cache.c_struct()
    rows, heads, _ = q.shape
    args = (q.data_ptr(), input_row_offsets.data_ptr(), input_row_offsets.shape[0] - 1, rows,
            heads, float(softmax_scale), _ptr(tree_mask),
            0 if tree_mask is None else tree_mask.shape[1], ctypes.byref(c), int(layer_idx),
            out.data_ptr(), _ptr(lse), workspace.data_ptr(), workspace.nbytes, _ptr(dev_status))
    f = _lib.mla_tree_attention_paged_qcache
    here = _here(q, input_row_offsets, tree_mask, out, lse, workspace, cache.data,
                 cache.page_table, cache.cache_lengths)
    code = f(*args, _stream(stream)) if here else _refuse(f, *args)
    return _check(code, "mla_tree_attention_paged_qcache", check)


def _accepted_ok(shape, cache, accepted, counts, new_lengths) -> bool:
    """A table row, length, count and new length for each list of accepted drafts (and maybe for
    more)."""
    return (len(shape) == 2 and _cache_ok(cache, shape[0]) and
            _has(shape[0], counts) and _has(shape[0], new_lengths) and
            _plain(_WORD, accepted, counts, new_lengths))


def mla_cache_compact_paged(cache: PagedCache, layer_begin: int, layer_count: int,
                            accepted: torch.Tensor, accepted_counts: torch.Tensor,
                            new_lengths: Optional[torch.Tensor] = None,
                            dev_status: Optional[torch.Tensor] = None, stream=None,
                            check: bool = True) -> int:
    """Moves request b's accepted drafts accepted[b, :accepted_counts[b]] (strictly increasing
    indices behind cache_lengths[b]) to the front of its drafted region in every layer of the
    range, and writes the grown lengths to new_lengths (memory of its own, which none of the
    other arguments has)."""
    shape = accepted.shape
    if not _accepted_ok(shape, cache, accepted, accepted_counts, new_lengths):
        return _check(PKM_ERR_INVALID_ARG, "mla_cache_compact_paged", check)
    c = cache.c_struct()
    args = (ctypes.byref(c), layer_begin, layer_count, shape[0], accepted.data_ptr(), shape[1],
            _ptr(accepted_counts), _ptr(new_lengths), _ptr(dev_status))
    f = _lib.mla_cache_compact_paged
    here = _here(accepted, accepted_counts, new_lengths, cache.data, cache.page_table,
                 cache.cache_lengths)
    code = f(*args, _stream(stream)) if here else _refuse(f, *args)
    return _check(code, "mla_cache_compact_paged", check)


def mla_cache_compact_paged_qcache(cache: QuantCache, layer_begin: int, layer_count: int,
                                   accepted: torch.Tensor, accepted_counts: torch.Tensor,
                                   new_lengths: Optional[torch.Tensor] = None,
                                   dev_status: Optional[torch.Tensor] = None, stream=None,
                                   check: bool = True) -> int:
    """mla_cache_compact_paged for a quantised cache."""
    shape = accepted.shape
    if not _accepted_ok(shape, cache, accepted, accepted_counts, new_lengths):
        return _check(PKM_ERR_INVALID_ARG, "mla_cache_compact_paged_qcache", check)
    c = cache.c_struct()
    args = (ctypes.byref(c), layer_begin, layer_count, shape[0], accepted.data_ptr(), shape[1],
            _ptr(accepted_counts), _ptr(new_lengths), _ptr(dev_status))
    f = _lib.mla_cache_compact_paged_qcache
    here = _here(accepted, accepted_counts, new_lengths, cache.data, cache.page_table,
                 cache.cache_lengths)
    code = f(*args, _stream(stream)) if here else _refuse(f, *args)
    return _check(code, "mla_cache_compact_paged_qcache", check)


def kv_matmul_paged_fp8_workspace_size(total_rows: int, k_in: int) -> int:
    return int(_lib.kv_matmul_paged_fp8_workspace_size(int(total_rows), int(k_in)))


def kv_matmul_paged_fp8(hidden_state: torch.Tensor, input_row_offsets: torch.Tensor,
                        w_e4m3: torch.Tensor, w_scale: torch.Tensor, kv_cache: PagedCache,
                        layer_idx: int, workspace: torch.Tensor,
                        dev_status: Optional[torch.Tensor] = None, stream=None,
                        check: bool = True) -> int:
    """FP8 kv_matmul: hidden_state bf16 [M, k_in], w_e4m3 [n_out, k_in] with fp32 block scales
    [n_out/128, k_in/128]; the quantised rows land in `workspace`."""
    c = kv_cache.c_struct()
    batch = int(input_row_offsets.shape[0]) - 1
    code = _lib.kv_matmul_paged_fp8(_ptr(hidden_state), _ptr(input_row_offsets), batch,
                                    int(hidden_state.shape[0]), int(hidden_state.shape[1]),
                                    _ptr(w_e4m3), _ptr(w_scale), int(w_e4m3.shape[0]),
                                    ctypes.byref(c), int(layer_idx), _ptr(workspace),
                                    workspace.numel() * workspace.element_size(),
                                    _ptr(dev_status), _stream(stream))
    return _check(code, "kv_matmul_paged_fp8", check)


def mla_decompress_k_paged_fp8_noalloc(cache: PagedCache, layer_idx: int,
                                       buffer_row_offsets: torch.Tensor,
                                       cache_offsets: torch.Tensor, buffer_length: int,
                                       kv_lora_rank: int, rope_dim: int, w_k_e4m3: torch.Tensor,
                                       w_k_scale: torch.Tensor, k_latent_buffer: torch.Tensor,
                                       k_buffer: torch.Tensor,
                                       dev_status: Optional[torch.Tensor] = None, stream=None,
                                       check: bool = True) -> int:
    """The FP8 decompress without a caller workspace, for callers that cannot allocate
    device memory: the library's fixed 16 MiB device array holds the quantised latent."""
    c = cache.c_struct()
    batch = int(buffer_row_offsets.shape[0]) - 1
    code = _lib.mla_decompress_k_paged_fp8_noalloc(
        ctypes.byref(c), int(layer_idx), _ptr(buffer_row_offsets), _ptr(cache_offsets), batch,
        int(buffer_length), int(kv_lora_rank), int(rope_dim), _ptr(w_k_e4m3), _ptr(w_k_scale),
        int(w_k_e4m3.shape[0]), _ptr(k_latent_buffer), _ptr(k_buffer), _ptr(dev_status),
        _stream(stream))
    return _check(code, "mla_decompress_k_paged_fp8_noalloc", check)


def kv_matmul_paged(hidden_state: torch.Tensor, input_row_offsets: torch.Tensor,
                    weight: torch.Tensor, kv_cache: PagedCache, layer_idx: int,
                    dev_status: Optional[torch.Tensor] = None, stream=None,
                    check: bool = True) -> int:
    c = kv_cache.c_struct()
    batch = int(input_row_offsets.shape[0]) - 1
    code = _lib.kv_matmul_paged(_ptr(hidden_state), _ptr(input_row_offsets), batch,
                                int(hidden_state.shape[0]), int(hidden_state.shape[1]),
                                _ptr(weight), int(weight.shape[1]), ctypes.byref(c),
                                int(layer_idx), _ptr(dev_status), _stream(stream))
    return _check(code, "kv_matmul_paged", check)


def pkm_check_wait_timeout(dev_status: torch.Tensor, timeout_ms: int, stream=None,
                           check: bool = True) -> int:
    code = _lib.pkm_check_wait_timeout(_ptr(dev_status), int(timeout_ms), _stream(stream))
    return _check(code, "pkm_check_wait_timeout", check)


__all__ = ["pkm_check_wait_timeout", "mla_decompress_k_paged_fp8_noalloc",
           "FP8_NOALLOC_SCRATCH_BYTES", "PagedCache", "PkmError", "mla_decompress_k_paged", "mla_decompress_k_paged_fp8",
           "mla_decompress_k_paged_fp8_workspace_size", "fp8_workspace_views", "kv_matmul_paged",
           "mla_cache_write_paged_at", "mla_cache_write_paged_qcache_at", "mla_rope_heads",
           "mla_tree_attention_paged", "mla_tree_attention_paged_qcache",
           "mla_tree_attention_paged_workspace_size", "mla_cache_compact_paged",
           "mla_cache_compact_paged_qcache", "status_string", "LIB_PATH", "PKM_OK", "PKM_ERR_INVALID_ARG", "PKM_ERR_UNSUPPORTED",
           "PKM_ERR_CUDA", "PKM_ERR_OUT_OF_RANGE", "PKM_ERR_TIMEOUT"]


def pkm_validate_row_offsets(offsets: torch.Tensor, dev_status: torch.Tensor, stream=None,
                             check: bool = True) -> int:
    """Merges PKM_ERR_INVALID_ARG into dev_status when the offset array (batch + 1 entries)
    decreases somewhere; writes nothing else."""
    code = _lib.pkm_validate_row_offsets(_ptr(offsets), int(offsets.shape[0]) - 1,
                                         _ptr(dev_status), _stream(stream))
    return _check(code, "pkm_validate_row_offsets", check)
