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
    if t.__class__ is not torch.Tensor and not isinstance(t, torch.Tensor):
        return int(t)
    return t.data_ptr()


def _current_stream() -> int:
    """torch.cuda.current_stream().cuda_stream, without building the stream object: that takes
    a quarter of a small call's time on the host."""
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
if _raw_stream is None or not hasattr(torch._C, "_cuda_getDevice"):
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
        table, lengths = self.page_table, self.cache_lengths
        return self._struct_of((self.data.data_ptr(), table.data_ptr(), table.shape[-1],
                                _ptr(lengths)))

    def _struct_of(self, tensors: tuple):
        """The struct with what it says of the tensors: data, page_table, max_pages_per_seq and
        cache_lengths."""
        d = self.__dict__
        kept = d.get("_kept")
        if kept is None:
            kept = d.setdefault("_kept", threading.local())
        mark = d.get("_mark")
        try:
            c, made, said = kept.struct
        except AttributeError:
            c = made = said = None
        if c is None or made is not mark:
            c, said = self._new_struct(), None
        if tensors != said:  # assigning to the struct takes longer than comparing
            c.data, c.page_table, c.max_pages_per_seq, c.cache_lengths = tensors
            kept.struct = c, mark, tensors
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
        return _CCache(None, int(self.layer_stride), int(self.page_stride), int(self.slot_stride),
                       int(self.kv_stride), int(self.num_layers), int(self.num_pages),
                       int(self.page_size), int(self.row_elems))


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
        return _CQuantCache(None, int(self.layer_stride), int(self.page_stride),
                            int(self.slot_stride), int(self.num_layers), int(self.num_pages),
                            int(self.page_size), int(self.kv_lora_rank), int(self.rope_dim))


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


# Element types that the C calls read as what they are named for: bf16 values or their bits.
_BF16 = (torch.bfloat16, torch.int16, torch.uint16)
_WORD = (torch.int32, torch.uint32)
_FLOAT = (torch.float32,)
_Tensor = torch.Tensor


def _look(tensors: tuple) -> tuple:
    """The device of the tensors in (types, elements at least, tensor) and their addresses.  The
    device is -1 for host memory or several, -2 if there is none to be seen (None and addresses
    pass), and None if a tensor has fewer elements, another type or, unless its types are None,
    gaps.  One pass over all of them: it is much of a small call."""
    device, addresses = -2, []
    for types, n, t in tensors:
        if t.__class__ is not _Tensor and (t is None or t.__class__ is int):
            addresses.append(t)
            continue
        if types is not None and (t.dtype not in types or not t.is_contiguous()) \
                or n > 0 and t.numel() < n:
            return None, addresses
        at = t.get_device()
        if at != device:
            device = at if device == -2 else -1
        addresses.append(t.data_ptr())
    return device, addresses


def _here(device: int) -> bool:
    """Whether tensors of that device are where the call runs.  (A tensor on a GPU has initialised
    CUDA; before, there are only others.)"""
    return device == -2 or (device >= 0 and device == torch._C._cuda_getDevice())


def _run(f, where: str, args: tuple, device: int, stream, check: bool) -> int:
    """f(*args, stream) for tensors of the call's device.  For others the status of what the
    call's own checks find, if anything, and nothing is launched."""
    if _here(device):
        if stream is None and device >= 0 and _raw_stream is not None:
            code = f(*args, _raw_stream(device))
        else:
            code = f(*args, _stream(stream))
    else:
        _lib.pkm_checks_only(1)
        try:
            code = f(*args, None)
        finally:
            _lib.pkm_checks_only(0)
        if code == PKM_ERR_CUDA:
            code = PKM_ERR_INVALID_ARG
    return code if code == PKM_OK else _check(code, where, check)


def _write_at(f, where, latent, offsets, positions, gamma, epsilon, freqs, cache, layer_idx, rank,
              rope, widths, dev_status, stream, check) -> int:
    """Both cache writes at positions: rows of R + P columns with a position each, R factors of the
    norm, P of a position (any for a P of 0), and a table row and a length for each request."""
    table = cache.page_table
    shape, factors, pages, batch = latent.shape, freqs.shape, table.shape, offsets.shape[0] - 1
    device, at = _look(((_BF16, 0, latent), (_WORD, 0, offsets), (_WORD, shape[0] if shape else 0, positions),
                        (_FLOAT, rank, gamma), (_FLOAT, 0, freqs), (None, 0, cache.data),
                        (_WORD, 0, table), (_WORD, batch, cache.cache_lengths)))
    if device is None or len(shape) != 2 or shape[1] != rank + rope \
            or (rope != 0 and (len(factors) != 2 or factors[1] != rope)) \
            or len(pages) != 2 or pages[0] < batch:
        return _check(PKM_ERR_INVALID_ARG, where, check)
    c = cache._struct_of((at[5], at[6], pages[1], at[7]))
    args = (at[0], at[1], at[2], batch, shape[0], *widths, at[3], float(epsilon), at[4], factors[0],
            ctypes.byref(c), int(layer_idx), _ptr(dev_status))
    return _run(f, where, args, device, stream, check)


def mla_cache_write_paged_at(latent: torch.Tensor, input_row_offsets: torch.Tensor,
                             positions: torch.Tensor, kv_norm_gamma: torch.Tensor,
                             epsilon: float, freqs_cis: torch.Tensor, cache: PagedCache,
                             layer_idx: int, kv_lora_rank: int, rope_dim: int,
                             dev_status: Optional[torch.Tensor] = None, stream=None,
                             check: bool = True) -> int:
    """mla_cache_write_paged with row r rotated by freqs_cis[positions[r]] (positions:
    uint32/int32 [total_rows]), wherever its slot is."""
    return _write_at(_lib.mla_cache_write_paged_at, "mla_cache_write_paged_at", latent,
                     input_row_offsets, positions, kv_norm_gamma, epsilon, freqs_cis, cache,
                     layer_idx, kv_lora_rank, rope_dim, (int(kv_lora_rank), int(rope_dim)),
                     dev_status, stream, check)


def mla_cache_write_paged_qcache_at(latent: torch.Tensor, input_row_offsets: torch.Tensor,
                                    positions: torch.Tensor, kv_norm_gamma: torch.Tensor,
                                    epsilon: float, freqs_cis: torch.Tensor, cache: QuantCache,
                                    layer_idx: int, dev_status: Optional[torch.Tensor] = None,
                                    stream=None, check: bool = True) -> int:
    """mla_cache_write_paged_qcache with row r rotated by freqs_cis[positions[r]]."""
    return _write_at(_lib.mla_cache_write_paged_qcache_at, "mla_cache_write_paged_qcache_at", latent,
                     input_row_offsets, positions, kv_norm_gamma, epsilon, freqs_cis, cache,
                     layer_idx, cache.kv_lora_rank, cache.rope_dim, (), dev_status, stream, check)


def mla_rope_heads(x: torch.Tensor, positions: torch.Tensor, freqs_cis: torch.Tensor,
                   y: torch.Tensor, half: bool = False,
                   dev_status: Optional[torch.Tensor] = None, stream=None,
                   check: bool = True) -> int:
    """Rotates x [rows, heads, P] into y [rows, heads, P] (bf16 views with contiguous last
    dimensions; y may be x) by the (cos, sin) pairs of freqs_cis[positions[row]]: pairs
    (2j, 2j + 1), or (j, j + P/2) with `half`.  The cache writes turn keys in pairs (2j, 2j + 1);
    for queries in the half layout, turn the keys with this call too (x and y the rope columns of
    the latent rows, one head) and write them with factors (1, 0)."""
    shape, sx, sy, table = x.shape, x.stride(), y.stride(), freqs_cis.shape
    device, at = _look(((None, 0, x), (None, 0, y), (_WORD, 0, positions), (_FLOAT, 0, freqs_cis)))
    if device is None or y.shape != shape or len(shape) != 3 or sx[2] != 1 or sy[2] != 1 \
            or x.dtype not in _BF16 or y.dtype not in _BF16 or positions.numel() != shape[0] \
            or len(table) != 2 or table[1] != shape[2]:
        return _check(PKM_ERR_INVALID_ARG, "mla_rope_heads", check)
    args = (at[0], sx[0], sx[1], at[2], shape[0], shape[1], shape[2], at[3], table[0],
            1 if half else 0, at[1], sy[0], sy[1], _ptr(dev_status))
    return _run(_lib.mla_rope_heads, "mla_rope_heads", args, device, stream, check)


def mla_tree_attention_paged_workspace_size(total_rows: int, num_heads: int,
                                            kv_lora_rank: int) -> int:
    return int(_lib.mla_tree_attention_paged_workspace_size(int(total_rows), int(num_heads),
                                                            int(kv_lora_rank)))


def _attention(f, where, q, offsets, scale, cache, layer_idx, rank, rope, widths, out, workspace,
               mask, lse, dev_status, stream, check) -> int:
    """Both attentions, with the shapes that the C call cannot see (an empty mask would pass for no
    mask there), and a table row and a length for each request."""
    table = cache.page_table
    shape, pages, batch, words = q.shape, table.shape, offsets.shape[0] - 1, 0
    device, at = _look(((_BF16, 0, q), (_WORD, 0, offsets), (_BF16, 0, out), (None, 0, workspace),
                        (_WORD, 0, mask), (_FLOAT, 0, lse), (None, 0, cache.data), (_WORD, 0, table),
                        (_WORD, batch, cache.cache_lengths)))
    if mask is not None:
        m = mask.shape
        words = m[1] if len(m) == 2 and m[:1] == shape[:1] else 0
    if device is None or len(shape) != 3 or shape[2] != rank + rope \
            or out.shape != (shape[0], shape[1], rank) or not workspace.is_contiguous() \
            or (lse is not None and lse.shape != shape[:2]) or (mask is not None and words == 0) \
            or len(pages) != 2 or pages[0] < batch:
        return _check(PKM_ERR_INVALID_ARG, where, check)
    c = cache._struct_of((at[6], at[7], pages[1], at[8]))
    args = (at[0], at[1], batch, shape[0], shape[1], *widths, float(scale), at[4], words,
            ctypes.byref(c), int(layer_idx), at[2], at[5], at[3], workspace.nbytes, _ptr(dev_status))
    return _run(f, where, args, device, stream, check)


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
    return _attention(_lib.mla_tree_attention_paged, "mla_tree_attention_paged", q,
                      input_row_offsets, softmax_scale, cache, layer_idx, kv_lora_rank, rope_dim,
                      (int(kv_lora_rank), int(rope_dim)), out, workspace, tree_mask, lse,
                      dev_status, stream, check)


def mla_tree_attention_paged_qcache(q: torch.Tensor, input_row_offsets: torch.Tensor,
                                    softmax_scale: float, cache: QuantCache, layer_idx: int,
                                    out: torch.Tensor, workspace: torch.Tensor,
                                    tree_mask: Optional[torch.Tensor] = None,
                                    lse: Optional[torch.Tensor] = None,
                                    dev_status: Optional[torch.Tensor] = None, stream=None,
                                    check: bool = True) -> int:
    """mla_tree_attention_paged over a quantised cache."""
    return _attention(_lib.mla_tree_attention_paged_qcache, "mla_tree_attention_paged_qcache", q,
                      input_row_offsets, softmax_scale, cache, layer_idx, cache.kv_lora_rank,
                      cache.rope_dim, (), out, workspace, tree_mask, lse, dev_status, stream, check)


def _compact(f, where, cache, layer_begin, layer_count, accepted, counts, new_lengths, dev_status,
             stream, check) -> int:
    """Both compactions: a table row, length, count and new length for each list of accepted drafts
    (and maybe for more)."""
    table = cache.page_table
    shape, pages = accepted.shape, table.shape
    n = shape[0] if shape else 0
    device, at = _look(((_WORD, 0, accepted), (_WORD, n, counts), (_WORD, n, new_lengths),
                        (None, 0, cache.data), (_WORD, 0, table), (_WORD, n, cache.cache_lengths)))
    if device is None or len(shape) != 2 or len(pages) != 2 or pages[0] < n:
        return _check(PKM_ERR_INVALID_ARG, where, check)
    c = cache._struct_of((at[3], at[4], pages[1], at[5]))
    args = (ctypes.byref(c), layer_begin, layer_count, n, at[0], shape[1], at[1], at[2],
            _ptr(dev_status))
    return _run(f, where, args, device, stream, check)


def mla_cache_compact_paged(cache: PagedCache, layer_begin: int, layer_count: int,
                            accepted: torch.Tensor, accepted_counts: torch.Tensor,
                            new_lengths: Optional[torch.Tensor] = None,
                            dev_status: Optional[torch.Tensor] = None, stream=None,
                            check: bool = True) -> int:
    """Moves request b's accepted drafts accepted[b, :accepted_counts[b]] (strictly increasing
    indices behind cache_lengths[b]) to the front of its drafted region in every layer of the
    range, and writes the grown lengths to new_lengths (memory of its own, which none of the
    other arguments has)."""
    return _compact(_lib.mla_cache_compact_paged, "mla_cache_compact_paged", cache, layer_begin,
                    layer_count, accepted, accepted_counts, new_lengths, dev_status, stream, check)


def mla_cache_compact_paged_qcache(cache: QuantCache, layer_begin: int, layer_count: int,
                                   accepted: torch.Tensor, accepted_counts: torch.Tensor,
                                   new_lengths: Optional[torch.Tensor] = None,
                                   dev_status: Optional[torch.Tensor] = None, stream=None,
                                   check: bool = True) -> int:
    """mla_cache_compact_paged for a quantised cache."""
    return _compact(_lib.mla_cache_compact_paged_qcache, "mla_cache_compact_paged_qcache", cache,
                    layer_begin, layer_count, accepted, accepted_counts, new_lengths, dev_status,
                    stream, check)


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
