"""Thin binding of liboscar.so (include/oscar.h): ctypes, and for the calls
made once per layer and step around the cache (rotary, reading back, group
index and selection, decode over listed groups) the compiled _calls module
(csrc/binding.cpp), whose argument checks take a tenth of the time.

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  Device buffers are torch tensors (PyTorch supplies device memory
and streams); host integer arrays are Python sequences.  Every function
raises OscarError when the C call returns a non-zero status.  There is no
CPU fallback: importing this module fails loudly if the library is missing.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "liboscar.so")

OSCAR_OK = 0
OSCAR_ERR_INVALID_ARG = 1
OSCAR_ERR_CAPACITY = 2
OSCAR_ERR_CUDA = 3
OSCAR_ERR_UNSUPPORTED = 4
OSCAR_ERR_DEVICE_TIMEOUT = 5

OSCAR_BYTES_USED = 0
OSCAR_BYTES_BF16_EQUIVALENT = 1
OSCAR_BYTES_ARENA = 2

OSCAR_BF16 = 0
OSCAR_F32 = 1

ROTARY_SCALING = {"none": 0, "linear": 1, "banded": 2, "yarn": 3}

HEAD_DIM = 128
GROUP = 128
VALUE_GROUP = 32
BLOCK_BYTES = 13824
BLOCK_BYTES_META16 = 11008
WINDOW_BYTES = 65536


class OscarError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"oscar status {status}: {message}")
        self.status = status


class oscar_cache_config(ctypes.Structure):
    _fields_ = [("max_batch", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("max_seq_len", ctypes.c_int32),
                ("group_size", ctypes.c_int32), ("value_group", ctypes.c_int32),
                ("device", ctypes.c_int32), ("meta_bits", ctypes.c_int32)]


class oscar_rotary_config(ctypes.Structure):
    _fields_ = [("head_dim", ctypes.c_int32), ("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("scaling", ctypes.c_int32), ("base", ctypes.c_double), ("factor", ctypes.c_double),
                ("original_length", ctypes.c_double), ("low", ctypes.c_double), ("high", ctypes.c_double),
                ("attention_factor", ctypes.c_double)]


class oscar_rotary_table(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("factor", ctypes.c_float),
                ("reserved", ctypes.c_int32), ("phase", ctypes.c_uint64 * (128 // 2))]


class oscar_score_rule(ctypes.Structure):
    _fields_ = [("cap", ctypes.c_float), ("reserved", ctypes.c_int32), ("slopes", ctypes.c_void_p)]


class oscar_rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class oscar_rotary_rows(ctypes.Structure):
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p),
                ("src_token_stride", ctypes.c_int64), ("src_head_stride", ctypes.c_int64),
                ("dst_token_stride", ctypes.c_int64), ("dst_head_stride", ctypes.c_int64),
                ("heads", ctypes.c_int32)]


def _load() -> ctypes.CDLL:
    if not os.path.exists(_LIB_PATH):
        raise ImportError(f"{_LIB_PATH} is missing: build it with int2_kv_cache_oscar_gb300.build.build()")
    lib = ctypes.CDLL(_LIB_PATH)
    P = ctypes.c_void_p
    I32 = ctypes.c_int32
    SZ = ctypes.c_size_t
    I32P = ctypes.POINTER(ctypes.c_int32)
    sigs = {
        "oscar_cache_required_bytes": [ctypes.POINTER(oscar_cache_config), ctypes.POINTER(SZ)],
        "oscar_cache_create": [ctypes.POINTER(oscar_cache_config), P, SZ, ctypes.POINTER(P)],
        "oscar_cache_destroy": [P],
        "oscar_cache_reset": [P, I32, P],
        "oscar_cache_length": [P, I32, I32P],
        "oscar_quantize_append": [P, I32, I32P, I32P, P, P, P],
        "oscar_decode_workspace_bytes": [P, I32, I32, ctypes.POINTER(SZ)],
        "oscar_decode_attention": [P, I32, I32P, P, I32, ctypes.c_float, P, P, SZ, P],
        "oscar_decode_attention_f32": [P, I32, I32P, P, I32, ctypes.c_float, P, P, SZ, P],
        "oscar_cache_bytes": [P, I32, I32, ctypes.POINTER(SZ)],
        "oscar_cache_block_offset": [P, I32, I32, I32, ctypes.POINTER(SZ)],
        "oscar_cache_window_offset": [P, I32, I32, ctypes.POINTER(SZ)],
        "oscar_cache_check": [P, P],
        "oscar_bf16_decode_workspace_bytes": [I32, I32, I32, ctypes.POINTER(SZ)],
        "oscar_bf16_decode_attention": [I32, I32P, I32P, P, P, I32, I32, P, I32, ctypes.c_float, P, P,
                                        SZ, P],
        "oscar_set_timing_events": [P, P],
        "oscar_test_arm_wait_timeout": [],
        "oscar_test_settled_groups": [P, I32, I32P, P, I32P],
        "oscar_decode_attention_noalloc": [P, I32, I32P, P, I32, ctypes.c_float, P, P],
        "oscar_append_decode": [P, I32, I32P, P, P, P, I32, ctypes.c_float, P, P, SZ, P],
        "oscar_prefill_attention": [P, I32, I32, P, I32, ctypes.c_float, P, P, P, SZ, P],
        "oscar_prefill_workspace_bytes": [P, I32, I32, I32, ctypes.POINTER(SZ)],
        "oscar_rotary_frequencies": [ctypes.POINTER(oscar_rotary_config), ctypes.POINTER(ctypes.c_double),
                                     ctypes.POINTER(ctypes.c_double)],
        "oscar_rotary_prepare": [ctypes.POINTER(oscar_rotary_config), ctypes.POINTER(oscar_rotary_table)],
        "oscar_rotary": [P, ctypes.c_int64, P, I32, ctypes.POINTER(oscar_rotary_rows),
                         ctypes.POINTER(oscar_rotary_rows), I32, P],
        "oscar_cache_get_config": [P, ctypes.POINTER(oscar_cache_config)],
        "oscar_cache_read": [P, I32, I32P, I32P, I32P, I32, P, P, P],
        "oscar_cache_export": [P, I32, P, P, P, P],
        "oscar_cache_import": [P, I32, I32, P, P, P, P],
        "oscar_index_required_bytes": [P, ctypes.POINTER(SZ)],
        "oscar_index_attach": [P, P, SZ],
        "oscar_index_update": [P, I32, I32P, I32, P],
        "oscar_select_groups": [P, I32, I32P, P, I32, I32, I32, I32, P, P],
        "oscar_cache_fork": [P, I32, I32P, I32P, I32P, P],
        "oscar_cache_keep_groups": [P, I32, I32P, I32P, I32P, I32P, P],
        "oscar_scored_decode_attention": [P, I32, I32P, P, I32, ctypes.c_float, ctypes.POINTER(oscar_score_rule), I32,
                                          P, P, SZ, P],
        "oscar_scored_prefill_attention": [P, I32, I32, P, I32, ctypes.c_float, ctypes.POINTER(oscar_score_rule), P, P,
                                           P, SZ, P],
        "oscar_chunk_attention": [I32, I32P, I32P, ctypes.POINTER(oscar_rows), ctypes.POINTER(oscar_rows),
                                  ctypes.POINTER(oscar_rows), I32, I32, ctypes.c_float,
                                  ctypes.POINTER(oscar_score_rule), P, P, P, P, P],
        "oscar_sparse_decode_attention": [P, I32, I32P, P, I32, ctypes.c_float, P, I32, I32, P, P, P, SZ, P],
    }
    for name, args in sigs.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = ctypes.c_int
    lib.oscar_last_error.argtypes = []
    lib.oscar_last_error.restype = ctypes.c_char_p
    return lib


_lib = _load()

try:                      # linked against the library just loaded
    from int2_kv_cache_oscar_gb300 import _calls  # noqa: E402
except ImportError as e:
    raise ImportError(f"_calls.so cannot be loaded beside {_LIB_PATH} ({e}): "
                      "build it with int2_kv_cache_oscar_gb300.build.build()") from e

# The current stream's handle without building a Stream object (3 us a call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def library_path() -> str:
    return _LIB_PATH


def raw_library() -> ctypes.CDLL:
    return _lib


def oscar_last_error() -> str:
    return _lib.oscar_last_error().decode()


def _check(status: int):
    if status != OSCAR_OK:
        raise OscarError(status, oscar_last_error())


def _i32(seq: Sequence[int]):
    try:
        return (ctypes.c_int32 * len(seq))(*seq)
    except TypeError:      # entries that are not plain ints
        return (ctypes.c_int32 * len(seq))(*[int(x) for x in seq])


_cuda_ready = False


def _stream(stream) -> int:
    """Handle of a torch stream, a raw handle, or (None) the current stream of
    the current device."""
    global _cuda_ready
    if stream is None:
        if _raw_stream is not None and (_cuda_ready or torch.cuda.is_initialized()):
            _cuda_ready = True
            return _raw_stream(_raw_device())
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _torch_stream(stream, device) -> torch.cuda.Stream:
    """The torch stream of a call's stream argument (raw handles included)."""
    if stream is None:
        return torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return stream
    handle = int(stream)       # 0 and 1: the legacy default stream
    return torch.cuda.default_stream(device) if handle in (0, 1) else torch.cuda.ExternalStream(handle, device)


def _in_use(stream, device, *tensors) -> None:
    """Marks tensors as used by the copies just enqueued on `stream`: torch does
    not hand out their memory again before these have run, also when the caller
    drops them now.  (Not within a graph capture: the captured copies read or
    write these addresses at every replay, so the caller keeps the tensors.)"""
    s = _torch_stream(stream, device)
    with torch.cuda.stream(s):
        if torch.cuda.is_current_stream_capturing():
            return
    for t in tensors:
        if t is None or t.numel() == 0:
            continue
        if t.is_cuda:
            t.record_stream(s)
        else:
            _calls.host_in_use(t, s.stream_id, s.device_index, s.device_type)


def _ptr(t: Optional[torch.Tensor]) -> ctypes.c_void_p:
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _buf(t, dtype, shape, name: str, optional: bool = False) -> ctypes.c_void_p:
    """Pointer of a caller buffer after the checks the C ABI cannot make (it
    receives bare pointers): a torch tensor of `dtype`, dense row-major, whose
    leading dimension is at least shape[0] (the kernels use that many rows) and
    whose other dimensions equal the rest of `shape` (they set the strides);
    None entries are unchecked.  A smaller or differently strided buffer would
    otherwise let a kernel read or write past it."""
    if t is None and optional:
        return ctypes.c_void_p(0)
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None:
        ok = t.dim() == len(shape) and (shape[0] is None or t.shape[0] >= shape[0]) and \
            all(e is None or t.shape[i] == e for i, e in enumerate(shape) if i > 0)
        if not ok:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)} "
                             "(leading dimension at least, None: any)")
    return ctypes.c_void_p(t.data_ptr())


def make_config(max_batch: int, num_kv_heads: int, max_seq_len: int, device: int = 0,
                head_dim: int = HEAD_DIM, group_size: int = GROUP,
                value_group: int = VALUE_GROUP, meta_bits: int = 32) -> oscar_cache_config:
    return oscar_cache_config(max_batch, num_kv_heads, head_dim, max_seq_len, group_size,
                              value_group, device, meta_bits)


def oscar_cache_required_bytes(cfg: oscar_cache_config) -> int:
    out = ctypes.c_size_t(0)
    _check(_lib.oscar_cache_required_bytes(ctypes.byref(cfg), ctypes.byref(out)))
    return out.value


def oscar_cache_create(cfg: oscar_cache_config, arena: torch.Tensor) -> ctypes.c_void_p:
    h = ctypes.c_void_p(0)
    _check(_lib.oscar_cache_create(ctypes.byref(cfg), _buf(arena, torch.uint8, None, "arena"),
                                   arena.numel() * arena.element_size(), ctypes.byref(h)))
    h.num_kv_heads = cfg.num_kv_heads      # (per-call checks read it here, not through the library)
    return h


def _kv_heads(handle) -> Optional[int]:
    """KV heads of the cache, also of a bare handle (None for no handle, which
    the library refuses)."""
    n = getattr(handle, "num_kv_heads", None)
    return n if n is not None or handle is None else oscar_cache_get_config(handle).num_kv_heads


def oscar_cache_destroy(handle) -> None:
    _check(_lib.oscar_cache_destroy(handle))


def oscar_cache_reset(handle, seq: int = -1, stream=None) -> None:
    _check(_lib.oscar_cache_reset(handle, seq, _stream(stream)))


def oscar_cache_length(handle, seq: int) -> int:
    out = ctypes.c_int32(0)
    _check(_lib.oscar_cache_length(handle, seq, ctypes.byref(out)))
    return out.value


def oscar_cache_get_config(handle) -> oscar_cache_config:
    out = oscar_cache_config()
    _check(_lib.oscar_cache_get_config(handle, ctypes.byref(out)))
    return out


def oscar_quantize_append(handle, seq_ids: Sequence[int], cu_new: Sequence[int],
                          k: torch.Tensor, v: torch.Tensor, stream=None) -> None:
    rows = int(cu_new[-1]) if len(seq_ids) > 0 else 0
    if rows == 0:
        kp = vp = ctypes.c_void_p(0)
    else:
        kp = _buf(k, torch.bfloat16, (rows, _kv_heads(handle), HEAD_DIM), "k")
        vp = _buf(v, torch.bfloat16, (rows,) + tuple(k.shape[1:]), "v")
    _check(_lib.oscar_quantize_append(handle, len(seq_ids), _i32(seq_ids), _i32(cu_new), kp, vp,
                                      _stream(stream)))


def oscar_decode_workspace_bytes(handle, n_seqs: int, num_q_heads: int) -> int:
    out = ctypes.c_size_t(0)
    _check(_lib.oscar_decode_workspace_bytes(handle, n_seqs, num_q_heads, ctypes.byref(out)))
    return out.value


def oscar_decode_attention(handle, seq_ids: Sequence[int], q: torch.Tensor, num_q_heads: int,
                           softmax_scale: float, out: torch.Tensor, workspace: torch.Tensor,
                           stream=None) -> None:
    shape = (len(seq_ids), num_q_heads, HEAD_DIM)
    _check(_lib.oscar_decode_attention(handle, len(seq_ids), _i32(seq_ids), _buf(q, torch.bfloat16, shape, "q"),
                                       num_q_heads, ctypes.c_float(softmax_scale),
                                       _buf(out, torch.bfloat16, shape, "out"),
                                       _buf(workspace, torch.uint8, None, "workspace"),
                                       workspace.numel() * workspace.element_size(), _stream(stream)))


def oscar_decode_attention_f32(handle, seq_ids: Sequence[int], q: torch.Tensor, num_q_heads: int,
                               softmax_scale: float, out: torch.Tensor, workspace: torch.Tensor,
                               stream=None) -> None:
    """The same decode with float32 outputs (the merged result before any
    bf16 rounding)."""
    shape = (len(seq_ids), num_q_heads, HEAD_DIM)
    _check(_lib.oscar_decode_attention_f32(handle, len(seq_ids), _i32(seq_ids), _buf(q, torch.bfloat16, shape, "q"),
                                           num_q_heads, ctypes.c_float(softmax_scale),
                                           _buf(out, torch.float32, shape, "out"),
                                           _buf(workspace, torch.uint8, None, "workspace"),
                                           workspace.numel() * workspace.element_size(), _stream(stream)))


def oscar_decode_attention_noalloc(handle, seq_ids: Sequence[int], q: torch.Tensor, num_q_heads: int,
                                   softmax_scale: float, out: torch.Tensor, stream=None) -> None:
    """Decode without a workspace: the partials go to the library's built-in
    device scratch (for callers that cannot allocate device memory)."""
    shape = (len(seq_ids), num_q_heads, HEAD_DIM)
    _check(_lib.oscar_decode_attention_noalloc(handle, len(seq_ids), _i32(seq_ids),
                                               _buf(q, torch.bfloat16, shape, "q"), num_q_heads,
                                               ctypes.c_float(softmax_scale),
                                               _buf(out, torch.bfloat16, shape, "out"), _stream(stream)))


def oscar_append_decode(handle, seq_ids: Sequence[int], k_new: torch.Tensor, v_new: torch.Tensor,
                        q: torch.Tensor, num_q_heads: int, softmax_scale: float, out: torch.Tensor,
                        workspace: torch.Tensor, stream=None) -> None:
    """Append one token per sequence and decode, in one call (one launch when
    no group closes)."""
    shape = (len(seq_ids), num_q_heads, HEAD_DIM)
    kp = _buf(k_new, torch.bfloat16, (len(seq_ids), _kv_heads(handle), HEAD_DIM), "k_new")
    vp = _buf(v_new, torch.bfloat16, (len(seq_ids),) + tuple(k_new.shape[1:]), "v_new")
    _check(_lib.oscar_append_decode(handle, len(seq_ids), _i32(seq_ids), kp, vp,
                                    _buf(q, torch.bfloat16, shape, "q"), num_q_heads,
                                    ctypes.c_float(softmax_scale), _buf(out, torch.bfloat16, shape, "out"),
                                    _buf(workspace, torch.uint8, None, "workspace"),
                                    workspace.numel() * workspace.element_size(), _stream(stream)))


def oscar_prefill_workspace_bytes(handle, seq: int, n_q: int, num_q_heads: int) -> int:
    out = ctypes.c_size_t(0)
    _check(_lib.oscar_prefill_workspace_bytes(handle, seq, n_q, num_q_heads, ctypes.byref(out)))
    return out.value


def oscar_prefill_attention(handle, seq: int, q: torch.Tensor, num_q_heads: int, softmax_scale: float,
                            out: torch.Tensor, lse: Optional[torch.Tensor] = None,
                            workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Attention of a chunk's queries q [n_q, num_q_heads, 128] over the
    sequence's cached tokens; out gets the rows, lse (fp32 [n_q, heads]) their
    log-sum-exp.  With a workspace (uint8, see oscar_prefill_workspace_bytes)
    the history is split across more CTAs and merged."""
    qp = _buf(q, torch.bfloat16, (None, num_q_heads, HEAD_DIM), "q")
    n_q = q.shape[0]
    ws_bytes = 0 if workspace is None else workspace.numel()
    _check(_lib.oscar_prefill_attention(handle, seq, n_q, qp, num_q_heads, ctypes.c_float(softmax_scale),
                                        _buf(out, torch.bfloat16, (n_q, num_q_heads, HEAD_DIM), "out"),
                                        _buf(lse, torch.float32, (n_q, num_q_heads), "lse", optional=True),
                                        _buf(workspace, torch.uint8, (None,), "workspace", optional=True),
                                        ctypes.c_size_t(ws_bytes), _stream(stream)))


class RotaryConfig:
    """A rotary configuration and its prepared table (keep it beside the model)."""

    def __init__(self, cfg: oscar_rotary_config):
        self.cfg = cfg
        self.rotary_dim = cfg.rotary_dim
        self.interleaved = bool(cfg.interleaved)
        self._table = oscar_rotary_table()
        _check(_lib.oscar_rotary_prepare(ctypes.byref(cfg), ctypes.byref(self._table)))

    @property
    def address(self) -> int:      # of this object's own table: copies have theirs
        return ctypes.addressof(self._table)


def make_rotary_config(rotary_dim: int = HEAD_DIM, base: float = 10000.0, interleaved: bool = False,
                       scaling: str = "none", factor: float = 1.0, original_length: float = 0.0,
                       low: float = 0.0, high: float = 0.0, attention_factor: float = 0.0,
                       head_dim: int = HEAD_DIM) -> RotaryConfig:
    """Rotary positions of 128-channel heads: layout, rotated channels and the
    scaling for long contexts ("none", "linear", "banded", "yarn"; see
    include/oscar.h)."""
    if scaling not in ROTARY_SCALING:
        raise ValueError(f"scaling must be one of {sorted(ROTARY_SCALING)}, got {scaling!r}")
    return RotaryConfig(oscar_rotary_config(head_dim, rotary_dim, int(bool(interleaved)), ROTARY_SCALING[scaling], base,
                                            factor, original_length, low, high, attention_factor))


def oscar_rotary_frequencies(config: RotaryConfig):
    """(frequencies in radians per position, factor on the rotated channels)."""
    f = (ctypes.c_double * (HEAD_DIM // 2))()
    m = ctypes.c_double(0.0)
    _check(_lib.oscar_rotary_frequencies(ctypes.byref(config.cfg), f, ctypes.byref(m)))
    return [f[i] for i in range(config.rotary_dim // 2)], m.value


def oscar_rotary(config: RotaryConfig, positions: torch.Tensor, q: torch.Tensor,
                 k: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
                 k_out: Optional[torch.Tensor] = None, transpose: bool = False, stream=None) -> None:
    """Rotates q [n, heads, 128] and k [n, kv heads, 128] (bf16 or float32, any
    strides with contiguous channels) by their tokens' positions (int32 [n])
    into q_out and k_out, or in place without them.  transpose: the transposed
    rotation (the gradient)."""
    _check(_calls.rotary(config.address, positions, q, k, q_out, k_out, transpose, stream))


def oscar_cache_read(handle, seq_ids: Sequence[int], start: Sequence[int], end: Sequence[int],
                     k_out: Optional[torch.Tensor], v_out: Optional[torch.Tensor], stream=None, *,
                     num_kv_heads: int = -1) -> None:
    """Tokens start[i] .. end[i] - 1 of each slot seq_ids[i] as rows of k_out
    and v_out [rows, kv heads, 128] (bf16 or float32; either may be None).
    Here and below the KV heads must be the cache's; num_kv_heads (-1: not
    given) is checked beside them."""
    _check(_calls.read(handle, num_kv_heads, seq_ids, start, end, k_out, v_out, stream))


def _state_buffers(handle, length: int, blocks, window, maxima):
    """The cache's device and the pointers of a moved sequence's buffers, large enough for `length` tokens
    of the cache (the copies take sizes from the cache; a length that the
    library refuses anyway is left to it)."""
    cfg = oscar_cache_get_config(handle)
    if 0 <= length <= cfg.max_seq_len and isinstance(blocks, torch.Tensor):
        need = cfg.num_kv_heads * (length // GROUP) * (BLOCK_BYTES_META16 if cfg.meta_bits == 16 else BLOCK_BYTES)
        if blocks.numel() < need:
            raise ValueError(f"blocks has {blocks.numel()} bytes, {length} tokens of the cache need {need}")
    rows = cfg.num_kv_heads if length % GROUP else None
    return (cfg.device, _buf(blocks, torch.uint8, None, "blocks", optional=True),
            _buf(window, torch.bfloat16, (rows, 2, GROUP, HEAD_DIM), "window", optional=True),
            _buf(maxima, torch.float32, (2, cfg.num_kv_heads), "maxima"))


def oscar_cache_export(handle, seq: int, blocks: Optional[torch.Tensor], window: Optional[torch.Tensor],
                       maxima: torch.Tensor, stream=None) -> None:
    """The caller may drop the buffers at once: memory of torch's allocators is
    not reused before the copies have run (import too); other page-locked
    memory, and every buffer of a captured call, stays the caller's to keep."""
    device, *bufs = _state_buffers(handle, oscar_cache_length(handle, seq), blocks, window, maxima)
    _check(_lib.oscar_cache_export(handle, seq, *bufs, _stream(stream)))
    _in_use(stream, device, blocks, window, maxima)


def oscar_cache_import(handle, seq: int, length: int, blocks: Optional[torch.Tensor],
                       window: Optional[torch.Tensor], maxima: torch.Tensor, stream=None) -> None:
    device, *bufs = _state_buffers(handle, length, blocks, window, maxima)
    _check(_lib.oscar_cache_import(handle, seq, length, *bufs, _stream(stream)))
    _in_use(stream, device, blocks, window, maxima)


def oscar_cache_fork(handle, src: Sequence[int], dst: Sequence[int], length: Sequence[int], stream=None) -> None:
    """The first length[i] tokens of slot src[i] into slot dst[i]; with dst[i] =
    src[i] the slot is cut to them in place."""
    _check(_calls.fork(handle, src, dst, length, stream))


def oscar_cache_keep_groups(handle, src: Sequence[int], dst: Sequence[int], groups: Sequence[Sequence[int]],
                            stream=None) -> None:
    """Slot dst[i] := groups[i] (ascending) of slot src[i], and its window; with
    dst[i] = src[i] in place."""
    _check(_calls.keep_groups(handle, src, dst, groups, stream))


def oscar_index_required_bytes(handle) -> int:
    out = ctypes.c_size_t(0)
    _check(_lib.oscar_index_required_bytes(handle, ctypes.byref(out)))
    return out.value


def oscar_index_attach(handle, index: Optional[torch.Tensor]) -> None:
    _check(_lib.oscar_index_attach(handle, _buf(index, torch.uint8, (None,), "index", optional=True),
                                   0 if index is None else index.numel()))


def oscar_index_update(handle, seq_ids: Sequence[int], rebuild: bool = False, stream=None) -> None:
    _check(_calls.index_update(handle, seq_ids, rebuild, stream))


def oscar_select_groups(handle, seq_ids: Sequence[int], q: torch.Tensor, num_q_heads: int, groups: torch.Tensor,
                        keep_first: int = 0, keep_last: int = 0, stream=None, *, num_kv_heads: int = -1) -> None:
    """The groups with the largest scores of each (sequence, KV head), into
    groups int32 [n_seqs, kv heads, n_select]."""
    _check(_calls.select_groups(handle, num_kv_heads, seq_ids, q, num_q_heads, groups, keep_first, keep_last, stream))


def oscar_sparse_decode_attention(handle, seq_ids: Sequence[int], q: torch.Tensor, num_q_heads: int,
                                  softmax_scale: float, groups: torch.Tensor, out: torch.Tensor,
                                  workspace: torch.Tensor, lse: Optional[torch.Tensor] = None, stream=None, *,
                                  num_kv_heads: int = -1) -> None:
    """Decode attention over the listed groups (int32 [n_seqs, kv heads,
    n_select], entries outside a sequence's groups are empty) and the window;
    out bf16 or float32."""
    _check(_calls.sparse_decode(handle, num_kv_heads, seq_ids, q, num_q_heads, softmax_scale, groups, out, workspace,
                                lse, stream))


def oscar_scored_decode_attention(handle, seq_ids: Sequence[int], q: torch.Tensor, num_q_heads: int,
                                  softmax_scale: float, out: torch.Tensor, workspace: torch.Tensor, cap: float = 0.0,
                                  slopes: Optional[torch.Tensor] = None, stream=None) -> None:
    """Decode attention with scores capped to cap tanh(s / cap) and lowered by
    slopes[head] (float32 [num_q_heads]) per token between a cached token and the
    newest one; out bf16 or float32."""
    _check(_calls.scored_decode(handle, seq_ids, q, num_q_heads, softmax_scale, cap, slopes, out, workspace, stream))


def oscar_scored_prefill_attention(handle, seq: int, q: torch.Tensor, num_q_heads: int, softmax_scale: float,
                                   out: torch.Tensor, lse: Optional[torch.Tensor] = None,
                                   workspace: Optional[torch.Tensor] = None, cap: float = 0.0,
                                   slopes: Optional[torch.Tensor] = None, stream=None) -> None:
    """oscar_prefill_attention under the same rule; query i stands i tokens
    behind the cached ones."""
    _check(_calls.scored_prefill(handle, seq, q, num_q_heads, softmax_scale, cap, slopes, out, lse, workspace, stream))


def oscar_chunk_attention(cu_seqlens: Sequence[int], q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                          out: torch.Tensor, lse: Optional[torch.Tensor] = None,
                          prefix: Optional[Sequence[int]] = None, cap: float = 0.0,
                          slopes: Optional[torch.Tensor] = None, prior_out: Optional[torch.Tensor] = None,
                          prior_lse: Optional[torch.Tensor] = None, softmax_scale: float = 0.0,
                          stream=None) -> None:
    """Attention within a chunk of packed documents (rows cu_seqlens[d] ..
    cu_seqlens[d + 1] - 1 of q [n, heads, 128], k and v [n, kv heads, 128],
    bf16, any strides with contiguous channels): causal, the first prefix[d]
    tokens of a document seen by all of its tokens, scores capped to cap
    tanh(s / cap) and lowered by slopes[head] per token of distance, merged with
    prior_out and prior_lse (which may be out and lse themselves)."""
    _check(_calls.chunk(cu_seqlens, prefix, q, k, v, softmax_scale, cap, slopes, prior_out, prior_lse, out, lse, stream))


def oscar_cache_bytes(handle, seq: int, kind: int) -> int:
    out = ctypes.c_size_t(0)
    _check(_lib.oscar_cache_bytes(handle, seq, kind, ctypes.byref(out)))
    return out.value


def oscar_cache_block_offset(handle, seq: int, kv_head: int, group: int) -> int:
    out = ctypes.c_size_t(0)
    _check(_lib.oscar_cache_block_offset(handle, seq, kv_head, group, ctypes.byref(out)))
    return out.value


def oscar_cache_window_offset(handle, seq: int, kv_head: int) -> int:
    out = ctypes.c_size_t(0)
    _check(_lib.oscar_cache_window_offset(handle, seq, kv_head, ctypes.byref(out)))
    return out.value


def oscar_cache_check(handle, stream=None) -> None:
    _check(_lib.oscar_cache_check(handle, _stream(stream)))


def oscar_bf16_decode_workspace_bytes(n_seqs: int, num_kv_heads: int, num_q_heads: int) -> int:
    out = ctypes.c_size_t(0)
    _check(_lib.oscar_bf16_decode_workspace_bytes(n_seqs, num_kv_heads, num_q_heads,
                                                  ctypes.byref(out)))
    return out.value


def oscar_bf16_decode_attention(seq_ids: Sequence[int], seq_lens: Sequence[int],
                                k_cache: torch.Tensor, v_cache: torch.Tensor, num_kv_heads: int,
                                max_seq_len: int, q: torch.Tensor, num_q_heads: int,
                                softmax_scale: float, out: torch.Tensor, workspace: torch.Tensor,
                                stream=None) -> None:
    cshape = (None, num_kv_heads, max_seq_len, HEAD_DIM)
    if isinstance(k_cache, torch.Tensor) and len(seq_ids) > 0 and k_cache.dim() == 4 and \
            max(int(s) for s in seq_ids) >= k_cache.shape[0]:
        raise ValueError("seq_ids index past the caches' first dimension")
    shape = (len(seq_ids), num_q_heads, HEAD_DIM)
    _check(_lib.oscar_bf16_decode_attention(
        len(seq_ids), _i32(seq_ids), _i32(seq_lens), _buf(k_cache, torch.bfloat16, cshape, "k_cache"),
        _buf(v_cache, torch.bfloat16, cshape, "v_cache"), num_kv_heads, max_seq_len,
        _buf(q, torch.bfloat16, shape, "q"), num_q_heads, ctypes.c_float(softmax_scale),
        _buf(out, torch.bfloat16, shape, "out"), _buf(workspace, torch.uint8, None, "workspace"),
        workspace.numel() * workspace.element_size(), _stream(stream)))


def oscar_test_arm_wait_timeout() -> None:
    """Test hook: the next INT2 decode, read-back, cut inside a group, selection or tiled chunk
    attention on this thread leaves one copy unissued so that a bounded device wait runs out
    (see include/oscar.h)."""
    _check(_lib.oscar_test_arm_wait_timeout())


def oscar_test_settled_groups(cache, seq_ids: Sequence[int], stream=None) -> list:
    """Test hook: per slot, the leading groups the next decode on `stream`
    would copy before its grid dependency wait (see include/oscar.h)."""
    handle = cache.handle if isinstance(cache, OscarCache) else cache
    out = (ctypes.c_int32 * max(len(seq_ids), 1))()
    _check(_lib.oscar_test_settled_groups(handle, len(seq_ids), _i32(seq_ids), _stream(stream), out))
    return [int(out[i]) for i in range(len(seq_ids))]


def oscar_set_timing_events(start: Optional[torch.cuda.Event], stop: Optional[torch.cuda.Event]):
    s = ctypes.c_void_p(0 if start is None else start.cuda_event)
    e = ctypes.c_void_p(0 if stop is None else stop.cuda_event)
    _check(_lib.oscar_set_timing_events(s, e))


class OscarCache:
    """Owns a device arena (a torch uint8 tensor) and the library handle."""

    def __init__(self, max_batch: int, num_kv_heads: int, max_seq_len: int,
                 device: Optional[torch.device] = None, meta_bits: int = 32):
        device = torch.device("cuda", torch.cuda.current_device()) if device is None else device
        self.cfg = make_config(max_batch, num_kv_heads, max_seq_len, device.index or 0, meta_bits=meta_bits)
        self.meta_bits = meta_bits
        nbytes = oscar_cache_required_bytes(self.cfg)
        self.arena = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.handle = oscar_cache_create(self.cfg, self.arena)
        self.num_kv_heads = num_kv_heads
        self.index = None
        self.max_batch = max_batch
        self.max_seq_len = max_seq_len

    def close(self):
        if self.handle is not None and self.handle.value:
            oscar_cache_destroy(self.handle)
        self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def length(self, seq: int) -> int:
        return oscar_cache_length(self.handle, seq)

    def append(self, seq_ids, cu_new, k, v, stream=None):
        if isinstance(k, torch.Tensor) and k.dim() == 3 and k.shape[1] != self.num_kv_heads:
            raise ValueError(f"k has {k.shape[1]} KV heads, the cache {self.num_kv_heads}")
        oscar_quantize_append(self.handle, seq_ids, cu_new, k, v, stream)

    def workspace(self, n_seqs: int, num_q_heads: int) -> torch.Tensor:
        n = oscar_decode_workspace_bytes(self.handle, n_seqs, num_q_heads)
        return torch.empty(max(n, 16), dtype=torch.uint8, device=self.arena.device)

    def decode(self, seq_ids, q, num_q_heads, out, workspace, softmax_scale=0.0, stream=None):
        oscar_decode_attention(self.handle, seq_ids, q, num_q_heads, softmax_scale, out, workspace,
                               stream)

    def decode_f32(self, seq_ids, q, num_q_heads, out, workspace, softmax_scale=0.0, stream=None):
        oscar_decode_attention_f32(self.handle, seq_ids, q, num_q_heads, softmax_scale, out, workspace,
                                   stream)

    def append_decode(self, seq_ids, k_new, v_new, q, num_q_heads, out, workspace, softmax_scale=0.0,
                      stream=None):
        if isinstance(k_new, torch.Tensor) and k_new.dim() == 3 and k_new.shape[1] != self.num_kv_heads:
            raise ValueError(f"k_new has {k_new.shape[1]} KV heads, the cache {self.num_kv_heads}")
        oscar_append_decode(self.handle, seq_ids, k_new, v_new, q, num_q_heads, softmax_scale, out, workspace,
                            stream)

    def _heads(self, t, dim: int, name: str):
        """A buffer's KV-head dimension against the cache's (the C ABI cannot see it)."""
        if isinstance(t, torch.Tensor) and t.dim() > dim and t.shape[dim] != self.num_kv_heads:
            raise ValueError(f"{name} has {t.shape[dim]} KV heads, the cache {self.num_kv_heads}")

    def read(self, seq_ids, start, end, k_out=None, v_out=None, stream=None):
        oscar_cache_read(self.handle, seq_ids, start, end, k_out, v_out, stream)

    @property
    def block_bytes(self) -> int:
        return BLOCK_BYTES_META16 if self.meta_bits == 16 else BLOCK_BYTES

    def _slot_buffers(self, length: int, blocks, window, maxima):
        g = length // GROUP
        if isinstance(blocks, torch.Tensor) and tuple(blocks.shape) != (self.num_kv_heads, g, self.block_bytes):
            raise ValueError(f"blocks has shape {tuple(blocks.shape)}, expected "
                             f"{(self.num_kv_heads, g, self.block_bytes)}")
        self._heads(window, 0, "window")
        self._heads(maxima, 1, "maxima")

    def export_sequence(self, seq: int, pinned: bool = False, stream=None):
        """The packed state of a slot, (length, blocks, window, maxima), in new
        tensors on the cache's device or in page-locked host memory: complete
        once the stream has been waited for."""
        n = self.length(seq)
        where = dict(pin_memory=True) if pinned else dict(device=self.arena.device)
        # device tensors belong to the stream that fills them
        with torch.cuda.stream(_torch_stream(stream, self.arena.device)):
            blocks = torch.empty((self.num_kv_heads, n // GROUP, self.block_bytes), dtype=torch.uint8, **where)
            window = torch.empty((self.num_kv_heads, 2, GROUP, HEAD_DIM), dtype=torch.bfloat16, **where)
            maxima = torch.empty((2, self.num_kv_heads), dtype=torch.float32, **where)
        oscar_cache_export(self.handle, seq, blocks, window, maxima, stream)
        return n, blocks, window, maxima

    def import_sequence(self, seq: int, length: int, blocks, window, maxima, stream=None):
        self._slot_buffers(length, blocks, window, maxima)
        oscar_cache_import(self.handle, seq, length, blocks, window, maxima, stream)

    def enable_index(self):
        """Allocates and attaches the group index (kept with the cache; called
        again, it is emptied: queued calls may still use its memory)."""
        if self.index is None:
            n = oscar_index_required_bytes(self.handle)
            self.index = torch.empty(n, dtype=torch.uint8, device=self.arena.device)
        oscar_index_attach(self.handle, self.index)

    def update_index(self, seq_ids, rebuild: bool = False, stream=None):
        oscar_index_update(self.handle, seq_ids, rebuild, stream)

    def select_groups(self, seq_ids, q, num_q_heads, groups, keep_first=0, keep_last=0, stream=None):
        oscar_select_groups(self.handle, seq_ids, q, num_q_heads, groups, keep_first, keep_last, stream)

    def sparse_decode(self, seq_ids, q, num_q_heads, groups, out, workspace, lse=None, softmax_scale=0.0,
                      stream=None):
        oscar_sparse_decode_attention(self.handle, seq_ids, q, num_q_heads, softmax_scale, groups, out, workspace,
                                      lse, stream)

    def scored_decode(self, seq_ids, q, num_q_heads, out, workspace, cap=0.0, slopes=None, softmax_scale=0.0,
                      stream=None):
        oscar_scored_decode_attention(self.handle, seq_ids, q, num_q_heads, softmax_scale, out, workspace, cap, slopes,
                                      stream)

    def scored_prefill(self, seq, q, num_q_heads, out, lse=None, workspace=None, cap=0.0, slopes=None,
                       softmax_scale=0.0, stream=None):
        oscar_scored_prefill_attention(self.handle, seq, q, num_q_heads, softmax_scale, out, lse, workspace, cap, slopes,
                                       stream)

    def fork(self, src, dst, lengths=None, stream=None):
        """Copies the first lengths[i] tokens (None: all) of each slot src[i] to slot dst[i]."""
        if lengths is None:
            lengths = [self.length(s) for s in src]
        oscar_cache_fork(self.handle, src, dst, lengths, stream)

    def truncate(self, seq_ids, lengths, stream=None):
        """Cuts each slot to its first lengths[i] tokens."""
        oscar_cache_fork(self.handle, seq_ids, seq_ids, lengths, stream)

    def keep_groups(self, src, groups, dst=None, stream=None):
        """Leaves groups[i] of each slot src[i] and its window, in slot dst[i] or (None) in place."""
        oscar_cache_keep_groups(self.handle, src, src if dst is None else dst, groups, stream)
