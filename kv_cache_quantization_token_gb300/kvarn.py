"""Thin ctypes binding of libkvarn.so (include/kvarn.h).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels. PyTorch supplies device memory and the current stream. There is no
fallback: if the library has not been built, every call raises.
"""
from __future__ import annotations

import ctypes
import os
import re

import torch

from . import _build

TILE = 128
DEFAULT_ITERS = 4
LAUNCH_PDL = 1       # KVARN_LAUNCH_PDL
LAUNCH_PREFETCH = 2  # KVARN_LAUNCH_PREFETCH
DEVERR_WAIT = 1      # KVARN_DEVERR_WAIT
DEVERR_RECORD = 2    # KVARN_DEVERR_RECORD
DEVERR_WINDOW = 4    # KVARN_DEVERR_WINDOW
DEVERR_SELFTEST = 8  # KVARN_DEVERR_SELFTEST

CODE8 = {"i8": 0, "e4m3": 1}  # KVARN_CODE8_*
PAIRINGS = {"halves": 0, "adjacent": 1}  # KVARN_PAIRS_*
IO_TYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}  # KVARN_IO_*

_lib = None


class KvarnError(RuntimeError):
    def __init__(self, fn: str, status: int):
        msg = _L().kvarn_status_string(status).decode() if _lib is not None else str(status)
        super().__init__(f"{fn} failed: {msg} ({status})")
        self.status = status


class Layout(ctypes.Structure):
    """Mirror of kvarn_layout_t."""
    _fields_ = [("version", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("tile_tokens", ctypes.c_int32), ("sinkhorn_iters", ctypes.c_int32),
                ("k_bits", ctypes.c_int32), ("v_bits", ctypes.c_int32),
                ("v_group", ctypes.c_int32), ("v_groups", ctypes.c_int32),
                ("record_bytes", ctypes.c_int64),
                ("off_k_codes", ctypes.c_int64), ("off_v_codes", ctypes.c_int64),
                ("off_k_delta", ctypes.c_int64), ("off_k_lo", ctypes.c_int64),
                ("off_k_s", ctypes.c_int64), ("off_k_r", ctypes.c_int64),
                ("off_v_delta", ctypes.c_int64), ("off_v_lo", ctypes.c_int64),
                ("off_v_r", ctypes.c_int64), ("off_v_s", ctypes.c_int64)]


class Layout8(ctypes.Structure):
    """Mirror of kvarn_layout8_t."""
    _fields_ = [("version", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("tile_tokens", ctypes.c_int32), ("code_format", ctypes.c_int32),
                ("block_tokens", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("record_bytes", ctypes.c_int64),
                ("off_k_codes", ctypes.c_int64), ("off_v_codes", ctypes.c_int64),
                ("off_k_scale", ctypes.c_int64), ("off_v_scale", ctypes.c_int64)]


class Layout4(ctypes.Structure):
    """Mirror of kvarn_layout4_t."""
    _fields_ = [("version", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("tile_tokens", ctypes.c_int32), ("run_tokens", ctypes.c_int32),
                ("group_channels", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("record_bytes", ctypes.c_int64), ("run_bytes", ctypes.c_int64),
                ("off_k_codes", ctypes.c_int64), ("off_v_codes", ctypes.c_int64),
                ("off_k_scale", ctypes.c_int64), ("off_v_scale", ctypes.c_int64)]


class Rotary(ctypes.Structure):
    """Mirror of kvarn_rotary_t."""
    _fields_ = [("version", ctypes.c_int32), ("rotary_dim", ctypes.c_int32),
                ("pairing", ctypes.c_int32), ("n_axes", ctypes.c_int32),
                ("turn", ctypes.c_uint64 * 128), ("axis", ctypes.c_uint8 * 128)]


def library_path() -> str:
    return _build.LIB


def _L():
    global _lib
    if _lib is None:
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(f"libkvarn.so is not built ({path}); run __graft_entry__.build()")
        lib = ctypes.CDLL(path)
        vp, i64, c_int, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
        u32, f32, lay = ctypes.c_uint, ctypes.c_float, ctypes.POINTER(Layout)
        lib.kvarn_status_string.restype = ctypes.c_char_p
        lib.kvarn_status_string.argtypes = [c_int]
        lib.kvarn_layout.argtypes = [c_int, c_int, lay]
        lib.kvarn_layout_scales.argtypes = [c_int, c_int, c_int, lay]
        lib.kvarn_layout_ex.argtypes = [c_int, c_int, c_int, c_int, lay]
        lib.kvarn_get_device_error.argtypes = [ctypes.POINTER(u32), c_int]
        lib.kvarn_selftest_bounded_wait.argtypes = [u32, vp]
        lib.kvarn_rotate_query.argtypes = [vp, vp, i64, c_int, vp]
        lib.kvarn_compress_tile.argtypes = [vp, vp, i64, i64, vp, vp, i64, vp, i64, lay, vp]
        lib.kvarn_append_window.argtypes = [vp, vp, i64, vp, vp, c_int, vp, vp, c_int, c_int, c_int,
                                            u32, vp]
        lib.kvarn_decode_workspace_bytes.argtypes = [c_int, c_int, c_int, c_int, c_int, c_int,
                                                     ctypes.POINTER(sz)]
        lib.kvarn_decode_attention.argtypes = [vp, vp, i64, vp, vp, vp, vp, vp, vp, c_int, c_int,
                                               c_int, c_int, c_int, c_int, f32, lay, vp, sz, vp,
                                               u32, vp]
        lib.kvarn_decode_attention_noalloc.argtypes = [vp, vp, i64, vp, vp, vp, vp, vp, vp, c_int,
                                                       c_int, c_int, c_int, c_int, c_int, f32, lay,
                                                       vp, u32, vp]
        lib.kvarn_decode_split.argtypes = [vp, vp, i64, vp, vp, vp, vp, vp, vp, c_int, c_int, c_int,
                                           c_int, c_int, c_int, f32, lay, vp, sz, u32, vp]
        lib.kvarn_decode_combine.argtypes = [vp, sz, c_int, c_int, c_int, c_int, c_int, c_int, vp,
                                             u32, vp]
        lib.kvarn_window_advance.argtypes = [vp, vp, vp, c_int, c_int, c_int, c_int, u32, vp]
        lib.kvarn_prefill_attention.argtypes = [vp, c_int, i64, vp, i64, vp, c_int, c_int, vp, vp,
                                                c_int, c_int, c_int, c_int, c_int, c_int, f32, lay,
                                                vp, sz, vp, vp]
        lib.kvarn_prefill_attention_cached.argtypes = [vp, c_int, i64, vp, i64, vp, c_int, c_int,
                                                       vp, vp, c_int, c_int, c_int, c_int, c_int,
                                                       c_int, f32, lay, vp, sz, c_int, c_int, vp, vp]
        lib.kvarn_prefill_workspace_bytes.argtypes = [c_int, c_int, c_int, c_int, ctypes.POINTER(sz)]
        lay8 = ctypes.POINTER(Layout8)
        lib.kvarn_layout8.argtypes = [c_int, c_int, c_int, lay8]
        lib.kvarn_compress_tile8.argtypes = [vp, vp, i64, i64, vp, vp, i64, vp, i64, lay8, vp]
        lib.kvarn_expand_tile8.argtypes = [vp, i64, vp, vp, vp, i64, i64, vp, i64, lay8, vp]
        lib.kvarn_decode8_workspace_bytes.argtypes = [c_int, c_int, c_int, c_int, c_int, c_int,
                                                      ctypes.POINTER(sz)]
        lib.kvarn_decode_attention8.argtypes = [vp, c_int, vp, i64, vp, vp, vp, vp, vp, vp, c_int,
                                                c_int, c_int, c_int, c_int, c_int, f32, lay8, vp, vp,
                                                vp, sz, vp, u32, vp]
        lib.kvarn_prefill8_workspace_bytes.argtypes = [c_int, c_int, c_int, c_int, c_int, c_int,
                                                       ctypes.POINTER(sz)]
        lib.kvarn_prefill_attention8.argtypes = [vp, c_int, c_int, i64, vp, i64, vp, c_int, c_int, vp,
                                                 vp, c_int, c_int, c_int, c_int, c_int, c_int, f32,
                                                 lay8, vp, sz, vp, vp]
        lib.kvarn_evict_tiles.argtypes = [vp, vp, vp, vp, vp, vp, vp, c_int, c_int, c_int, c_int, c_int,
                                          c_int, u32, vp]
        lay4, rot = ctypes.POINTER(Layout4), ctypes.POINTER(Rotary)
        lib.kvarn_layout4.argtypes = [c_int, lay4]
        lib.kvarn_write_rows4.argtypes = [vp, i64, vp, i64, c_int, vp, i64, vp, vp, vp, c_int, c_int, c_int,
                                          c_int, c_int, lay4, u32, vp]
        lib.kvarn_read_rows4.argtypes = [vp, i64, vp, vp, vp, vp, i64, vp, i64, c_int, c_int, c_int, c_int,
                                         c_int, c_int, lay4, u32, vp]
        lib.kvarn_decode4_workspace_bytes.argtypes = [c_int, c_int, c_int, c_int, c_int, ctypes.POINTER(sz)]
        lib.kvarn_decode_attention4.argtypes = [vp, c_int, vp, i64, vp, vp, c_int, c_int, c_int, c_int, c_int,
                                                f32, lay4, vp, vp, vp, sz, vp, u32, vp]
        lib.kvarn_prefill4_workspace_bytes.argtypes = [c_int, c_int, c_int, c_int, c_int, ctypes.POINTER(sz)]
        lib.kvarn_prefill_attention4.argtypes = [vp, c_int, c_int, i64, vp, i64, vp, c_int, c_int, c_int, c_int,
                                                 f32, lay4, vp, sz, vp, vp]
        lib.kvarn_rotary.argtypes = [c_int, c_int, ctypes.POINTER(ctypes.c_double),
                                     ctypes.POINTER(ctypes.c_uint8), c_int, rot]
        lib.kvarn_norm_rotate.argtypes = [vp, i64, vp, i64, c_int, i64, c_int, c_int, c_int, vp, vp, f32, vp, rot,
                                          c_int, vp, i64, vp, i64, u32, vp]
        for name in ("kvarn_layout4", "kvarn_write_rows4", "kvarn_read_rows4",
                     "kvarn_decode4_workspace_bytes", "kvarn_decode_attention4",
                     "kvarn_prefill4_workspace_bytes", "kvarn_prefill_attention4", "kvarn_rotary",
                     "kvarn_norm_rotate"):
            getattr(lib, name).restype = c_int
        for name in ("kvarn_layout8", "kvarn_compress_tile8", "kvarn_expand_tile8",
                     "kvarn_decode8_workspace_bytes", "kvarn_decode_attention8",
                     "kvarn_prefill8_workspace_bytes", "kvarn_prefill_attention8",
                     "kvarn_evict_tiles"):
            getattr(lib, name).restype = c_int
        for name in ("kvarn_layout", "kvarn_layout_scales", "kvarn_layout_ex", "kvarn_rotate_query",
                     "kvarn_compress_tile", "kvarn_get_device_error", "kvarn_selftest_bounded_wait",
                     "kvarn_append_window", "kvarn_decode_workspace_bytes",
                     "kvarn_decode_attention", "kvarn_decode_attention_noalloc",
                     "kvarn_decode_split", "kvarn_decode_combine", "kvarn_window_advance",
                     "kvarn_prefill_attention", "kvarn_prefill_workspace_bytes",
                     "kvarn_prefill_attention_cached"):
            getattr(lib, name).restype = c_int
        _lib = lib
    return _lib


def declared_functions(header: str) -> list:
    """Names of the functions include/kvarn.h declares."""
    with open(header) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"^\s*(?:const\s+)?\w+\s*\**\s*(kvarn_\w+)\s*\(", text, flags=re.M)))


def _check(fn: str, rc: int):
    if rc != 0:
        raise KvarnError(fn, rc)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dev(t, name, dtype, device=None):
    """A contiguous CUDA tensor of `dtype` (on `device`, when given): anything
    else would reach the kernels as a pointer they cannot use."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda):
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    return t


def _all_dev(device, **tensors):
    """_dev for several (tensor, dtype) pairs that must share one device."""
    for name, (t, dtype) in tensors.items():
        _dev(t, name, dtype, device)


def device_error(clear: bool = True) -> int:
    """KVARN_DEVERR_* bits that kernels of this library set on the current
    device since the word was last cleared (kvarn_get_device_error; this
    synchronises the device)."""
    bits = ctypes.c_uint()
    _check("kvarn_get_device_error", _L().kvarn_get_device_error(ctypes.byref(bits), int(bool(clear))))
    return int(bits.value)


def selftest_bounded_wait(timeout_us: int, stream=None):
    """One kernel whose wait runs out after timeout_us and reports
    DEVERR_SELFTEST (kvarn_selftest_bounded_wait)."""
    _check("kvarn_selftest_bounded_wait",
           _L().kvarn_selftest_bounded_wait(int(timeout_us), _stream(stream)))


def layout(head_dim: int, iters: int = DEFAULT_ITERS, scale_bits: int = 32,
           v_bits: int = 2) -> Layout:
    """Record layout: fp32 scale fields (scale_bits 32, the default) or
    binary16 ones (16, the f16-scale layout; same codes), and 2-bit value
    codes (the k4v2 preset) or 4-bit ones (v_bits 4, the k4v4 variant)."""
    L = Layout()
    _check("kvarn_layout_ex",
           _L().kvarn_layout_ex(head_dim, iters, scale_bits, v_bits, ctypes.byref(L)))
    return L


def rotate_query(q: torch.Tensor, out: torch.Tensor = None, stream=None) -> torch.Tensor:
    """H q for every row (last axis = head_dim)."""
    _dev(q, "q", torch.float32)
    if out is None:
        out = torch.empty_like(q)
    _dev(out, "out", torch.float32)
    D = q.shape[-1]
    _check("kvarn_rotate_query",
           _L().kvarn_rotate_query(_ptr(q), _ptr(out), q.numel() // D, D, _stream(stream)))
    return out


def compress_tile(k_raw, v_raw, src_row0, tiles, dst_record, lay: Layout, stream=None):
    """k_raw, v_raw: fp32 [n_rows][row_stride] (2-D view of any row-major
    buffer); src_row0, dst_record: int64 [n_units] on the device."""
    _dev(k_raw, "k_raw", torch.float32)
    _all_dev(k_raw.device, v_raw=(v_raw, torch.float32), src_row0=(src_row0, torch.int64),
             dst_record=(dst_record, torch.int64), tiles=(tiles, torch.uint8))
    if k_raw.shape != v_raw.shape:
        raise ValueError("k_raw and v_raw must have the same shape")
    if src_row0.numel() != dst_record.numel():
        raise ValueError("src_row0 and dst_record must have one entry per unit")
    row_stride = k_raw.shape[-1]
    n_rows = k_raw.numel() // row_stride
    _check("kvarn_compress_tile",
           _L().kvarn_compress_tile(_ptr(k_raw), _ptr(v_raw), row_stride, n_rows, _ptr(src_row0),
                                    _ptr(tiles), tiles.numel(), _ptr(dst_record), src_row0.numel(),
                                    ctypes.byref(lay), _stream(stream)))


def append_window(k_new, v_new, win_k, win_v, win_start, win_len, stream=None, flags=0):
    """k_new, v_new: fp32 [n_seq][n_new][Hkv][D]; win_k, win_v: fp32
    [n_seq][Hkv][cap][D]; win_start, win_len: int32 [n_seq]."""
    _dev(k_new, "k_new", torch.float32)
    _all_dev(k_new.device, v_new=(v_new, torch.float32), win_k=(win_k, torch.float32),
             win_v=(win_v, torch.float32), win_start=(win_start, torch.int32),
             win_len=(win_len, torch.int32))
    n_seq, n_new, hkv, D = k_new.shape
    if v_new.shape != k_new.shape or win_k.shape != win_v.shape or win_k.shape[:2] != (n_seq, hkv) \
            or win_k.shape[3] != D or win_start.numel() != n_seq or win_len.numel() != n_seq:
        raise ValueError("append_window: inconsistent shapes")
    cap = win_k.shape[2]
    _check("kvarn_append_window",
           _L().kvarn_append_window(_ptr(k_new), _ptr(v_new), n_new, _ptr(win_k), _ptr(win_v), cap,
                                    _ptr(win_start), _ptr(win_len), n_seq, hkv, D, int(flags),
                                    _stream(stream)))


def decode_workspace_bytes(B, Hq, Hkv, head_dim, max_tiles, win_capacity) -> int:
    n = ctypes.c_size_t()
    _check("kvarn_decode_workspace_bytes",
           _L().kvarn_decode_workspace_bytes(B, Hq, Hkv, head_dim, max_tiles, win_capacity,
                                             ctypes.byref(n)))
    return n.value


def _decode_inputs(q, tiles, tile_table, n_tiles, win_k, win_v, win_start, win_len, what):
    """Checks the decode inputs (q fp32 [B][Hq][D]; tile_table int64
    [B][Hkv][max_tiles]; n_tiles int32 [B]; win_k/v fp32 [B][Hkv][cap][D];
    win_start/len int32 [B]) and returns (B, Hq, D, Hkv, max_tiles, cap)."""
    _dev(q, "q", torch.float32)
    _all_dev(q.device, tiles=(tiles, torch.uint8), tile_table=(tile_table, torch.int64),
             n_tiles=(n_tiles, torch.int32), win_k=(win_k, torch.float32),
             win_v=(win_v, torch.float32), win_start=(win_start, torch.int32),
             win_len=(win_len, torch.int32))
    B, Hq, D = q.shape
    Hkv, max_tiles = tile_table.shape[1], tile_table.shape[2]
    cap = win_k.shape[2]
    if (tile_table.shape[0] != B or n_tiles.numel() != B or win_start.numel() != B
            or win_len.numel() != B or win_k.shape != win_v.shape
            or tuple(win_k.shape[:2]) != (B, Hkv) or win_k.shape[3] != D):
        raise ValueError(f"{what}: inconsistent shapes")
    return B, Hq, D, Hkv, max_tiles, cap


def decode_attention(q, tiles, tile_table, n_tiles, win_k, win_v, win_start, win_len,
                     lay: Layout, softmax_scale=None, ws=None, out=None, stream=None, flags=0):
    """q fp32 [B][Hq][D]; tiles uint8 record pool; tile_table int64
    [B][Hkv][max_tiles]; n_tiles int32 [B]; win_k/v fp32 [B][Hkv][cap][D];
    win_start/len int32 [B]; flags: LAUNCH_* bits of this call."""
    B, Hq, D, Hkv, max_tiles, cap = _decode_inputs(q, tiles, tile_table, n_tiles, win_k, win_v,
                                                   win_start, win_len, "decode_attention")
    if softmax_scale is None:
        softmax_scale = D ** -0.5
    need = decode_workspace_bytes(B, Hq, Hkv, D, max_tiles, cap)
    if ws is None:
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    if out is None:
        out = torch.empty_like(q)
    _all_dev(q.device, ws=(ws, torch.uint8), out=(out, torch.float32))
    _check("kvarn_decode_attention",
           _L().kvarn_decode_attention(_ptr(q), _ptr(tiles), tiles.numel(), _ptr(tile_table),
                                       _ptr(n_tiles), _ptr(win_k), _ptr(win_v), _ptr(win_start),
                                       _ptr(win_len), cap, B, Hq, Hkv, D, max_tiles,
                                       float(softmax_scale), ctypes.byref(lay), _ptr(ws),
                                       ws.numel(), _ptr(out), int(flags), _stream(stream)))
    return out


def decode_split(q, tiles, tile_table, n_tiles, win_k, win_v, win_start, win_len, lay: Layout,
                 ws, softmax_scale=None, stream=None, flags=0):
    """First decode kernel: per-item partials into ws (see decode_attention)."""
    B, Hq, D, Hkv, max_tiles, cap = _decode_inputs(q, tiles, tile_table, n_tiles, win_k, win_v,
                                                   win_start, win_len, "decode_split")
    _dev(ws, "ws", torch.uint8, q.device)
    if softmax_scale is None:
        softmax_scale = D ** -0.5
    _check("kvarn_decode_split",
           _L().kvarn_decode_split(_ptr(q), _ptr(tiles), tiles.numel(), _ptr(tile_table),
                                   _ptr(n_tiles), _ptr(win_k), _ptr(win_v), _ptr(win_start),
                                   _ptr(win_len), cap, B, Hq, Hkv, D, max_tiles,
                                   float(softmax_scale), ctypes.byref(lay), _ptr(ws), ws.numel(),
                                   int(flags), _stream(stream)))


def decode_combine(ws, out, Hkv, max_tiles, win_capacity, stream=None, flags=0):
    """Second decode kernel: LSE combine of the partials in ws into out [B][Hq][D]."""
    _dev(out, "out", torch.float32)
    _dev(ws, "ws", torch.uint8, out.device)
    B, Hq, D = out.shape
    _check("kvarn_decode_combine",
           _L().kvarn_decode_combine(_ptr(ws), ws.numel(), B, Hq, Hkv, D, max_tiles, win_capacity,
                                     _ptr(out), int(flags), _stream(stream)))
    return out


def window_advance(win_start, win_len, n_tiles, d_len, promote, win_capacity, stream=None, flags=0):
    """Device-side window bookkeeping (length += d_len, then promote tiles)."""
    _dev(win_start, "win_start", torch.int32)
    _dev(win_len, "win_len", torch.int32, win_start.device)
    if n_tiles is not None:
        _dev(n_tiles, "n_tiles", torch.int32, win_start.device)
    _check("kvarn_window_advance",
           _L().kvarn_window_advance(_ptr(win_start), _ptr(win_len), _ptr(n_tiles),
                                     win_start.numel(), int(d_len), int(promote),
                                     int(win_capacity), int(flags), _stream(stream)))


def prefill_workspace_bytes(n_tiles, win_len, Hkv, head_dim) -> int:
    n = ctypes.c_size_t()
    _check("kvarn_prefill_workspace_bytes",
           _L().kvarn_prefill_workspace_bytes(int(n_tiles), int(win_len), Hkv, head_dim,
                                              ctypes.byref(n)))
    return n.value


def prefill_attention(q_chunk, pos0, tiles, tile_table, n_tiles, win_k, win_v, win_start,
                      win_len, lay: Layout, softmax_scale=None, ws=None, out=None, stream=None,
                      ws_blocks=None, cached_tiles=0):
    """Causal attention of a chunk of one sequence: q_chunk fp32 [C][Hq][D] at
    positions pos0 + i; tile_table int64 [Hkv][stride]; win_k/v fp32
    [Hkv][cap][D]; n_tiles, win_start, win_len host ints; ws a uint8 device
    workspace of prefill_workspace_bytes() (allocated here when None). With
    ws_blocks (images per KV head of a ws kept for the whole prompt), the call
    goes through kvarn_prefill_attention_cached and converts only the tiles
    from cached_tiles on."""
    _dev(q_chunk, "q_chunk", torch.float32)
    _all_dev(q_chunk.device, tiles=(tiles, torch.uint8), tile_table=(tile_table, torch.int64),
             win_k=(win_k, torch.float32), win_v=(win_v, torch.float32))
    C, Hq, D = q_chunk.shape
    Hkv, stride = tile_table.shape
    cap = win_k.shape[1]
    if win_k.shape != win_v.shape or win_k.shape[0] != Hkv or win_k.shape[2] != D:
        raise ValueError("prefill_attention: inconsistent shapes")
    if softmax_scale is None:
        softmax_scale = D ** -0.5
    if out is None:
        out = torch.empty_like(q_chunk)
    if ws is None:
        need = prefill_workspace_bytes(n_tiles, win_len, Hkv, D)
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device=q_chunk.device)
    _all_dev(q_chunk.device, ws=(ws, torch.uint8), out=(out, torch.float32))
    if ws_blocks is not None:
        _check("kvarn_prefill_attention_cached",
               _L().kvarn_prefill_attention_cached(
                   _ptr(q_chunk), C, int(pos0), _ptr(tiles), tiles.numel(), _ptr(tile_table),
                   stride, int(n_tiles), _ptr(win_k), _ptr(win_v), int(win_start), int(win_len),
                   cap, Hq, Hkv, D, float(softmax_scale), ctypes.byref(lay), _ptr(ws),
                   ws.numel(), int(ws_blocks), int(cached_tiles), _ptr(out), _stream(stream)))
        return out
    _check("kvarn_prefill_attention",
           _L().kvarn_prefill_attention(_ptr(q_chunk), C, int(pos0), _ptr(tiles), tiles.numel(),
                                        _ptr(tile_table), stride, int(n_tiles), _ptr(win_k),
                                        _ptr(win_v), int(win_start), int(win_len), cap, Hq, Hkv, D,
                                        float(softmax_scale), ctypes.byref(lay), _ptr(ws),
                                        ws.numel(), _ptr(out), _stream(stream)))
    return out


def decode_attention_noalloc(q, tiles, tile_table, n_tiles, win_k, win_v, win_start, win_len,
                             lay: Layout, softmax_scale=None, out=None, stream=None, flags=0):
    """decode_attention for callers that cannot allocate device memory: the
    partials go to the library's own fixed scratch array instead of a
    workspace (see kvarn_decode_attention_noalloc in include/kvarn.h).
    `out` must be passed by such callers; it is created here only as a
    convenience for everyone else."""
    B, Hq, D, Hkv, max_tiles, cap = _decode_inputs(q, tiles, tile_table, n_tiles, win_k, win_v,
                                                   win_start, win_len, "decode_attention_noalloc")
    if softmax_scale is None:
        softmax_scale = D ** -0.5
    if out is None:
        out = torch.empty_like(q)
    _dev(out, "out", torch.float32, q.device)
    _check("kvarn_decode_attention_noalloc",
           _L().kvarn_decode_attention_noalloc(
               _ptr(q), _ptr(tiles), tiles.numel(), _ptr(tile_table), _ptr(n_tiles), _ptr(win_k),
               _ptr(win_v), _ptr(win_start), _ptr(win_len), cap, B, Hq, Hkv, D, max_tiles,
               float(softmax_scale), ctypes.byref(lay), _ptr(out), int(flags), _stream(stream)))
    return out


# ---------------------------------------------------------------------------
# the 8-bit cache and eviction

def layout8(head_dim: int, code: str = "i8", block_tokens: int = 64) -> Layout8:
    """Layout of an 8-bit tile record: code "i8" (integers -127..127) or "e4m3"
    (8-bit floating point), one fp32 scale for each block of block_tokens (16,
    32, 64 or 128) tokens of a head's K and of its V."""
    if code not in CODE8:
        raise ValueError(f"code must be one of {sorted(CODE8)}, got {code!r}")
    L = Layout8()
    _check("kvarn_layout8", _L().kvarn_layout8(head_dim, CODE8[code], block_tokens, ctypes.byref(L)))
    return L


def _fit(device, *checks):
    """Each (name, tensor, dtype) is a contiguous tensor of dtype on the CUDA device of
    index `device`. One pass over what a decode step calls often; the tensor that does
    not fit is named by _dev."""
    for name, t, dtype in checks:
        if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == device
                and t.is_contiguous()):
            _dev(t, name, dtype, torch.device("cuda", max(device, 0)))


def _io(t, name):
    """A contiguous CUDA tensor of a query/output type: its KVARN_IO_* code and device index."""
    if isinstance(t, torch.Tensor) and t.is_cuda and t.is_contiguous():
        io = IO_TYPES.get(t.dtype)
        if io is not None:
            return io, t.get_device()
    if isinstance(t, torch.Tensor) and t.is_cuda and t.dtype not in IO_TYPES:
        raise TypeError(f"{name} must be float32, float16 or bfloat16, got {t.dtype}")
    _dev(t, name, getattr(t, "dtype", None))
    return IO_TYPES[t.dtype], t.get_device()


def _call(device, fn, stream, *args):
    """fn(*args, stream) with the tensors' device current: the kernels, the error word and
    the default stream are that device's."""
    if torch.cuda.current_device() != device:
        with torch.cuda.device(device):
            return _call(device, fn, stream, *args)
    if stream is None:  # (the handle itself: a Stream object takes a microsecond to make)
        handle = torch._C._cuda_getCurrentRawStream(device)
    elif stream.device.index != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{device}")
    else:
        handle = stream.cuda_stream
    rc = getattr(_lib or _L(), fn)(*args, handle)
    if rc != 0:
        raise KvarnError(fn, rc)


def _scratch(nbytes, device, stream):
    """A workspace in the memory of the stream that will use it: it is given back on
    return, and only later work of that stream may take it."""
    if stream is None:
        return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def _result(like, stream):
    if stream is None:
        return torch.empty_like(like)
    with torch.cuda.stream(stream):
        return torch.empty_like(like)


def _rows8(k, v, rows, tiles, records, names):
    _dev(k, names[0], torch.float32)
    device = k.get_device()
    _fit(device, (names[1], v, torch.float32), (names[2], rows, torch.int64),
         (names[3], records, torch.int64), ("tiles", tiles, torch.uint8))
    if k.shape != v.shape or k.dim() < 1:
        raise ValueError(f"{names[0]} and {names[1]} must have the same shape")
    if rows.numel() != records.numel():
        raise ValueError(f"{names[2]} and {names[3]} must have one entry per unit")
    stride = k.shape[-1]
    return device, stride, (k.numel() // stride if stride else 0)


def compress_tile8(k_raw, v_raw, src_row0, tiles, dst_record, lay: Layout8, stream=None):
    """128 raw rows per unit into 8-bit records: arguments as compress_tile's
    (k_raw, v_raw fp32 [n_rows][row_stride]; src_row0, dst_record int64 [n_units])."""
    device, stride, n_rows = _rows8(k_raw, v_raw, src_row0, tiles, dst_record,
                                    ("k_raw", "v_raw", "src_row0", "dst_record"))
    _call(device, "kvarn_compress_tile8", stream, k_raw.data_ptr(), v_raw.data_ptr(), stride, n_rows,
          src_row0.data_ptr(), tiles.data_ptr(), tiles.numel(), dst_record.data_ptr(),
          src_row0.numel(), ctypes.byref(lay))


def expand_tile8(tiles, src_record, k_out, v_out, dst_row0, lay: Layout8, stream=None):
    """The records at src_record (int64 [n_units]) as fp32 rows dst_row0[u] .. + 127
    of k_out and v_out, fp32 [n_rows][row_stride]; other rows stay as they are."""
    device, stride, n_rows = _rows8(k_out, v_out, dst_row0, tiles, src_record,
                                    ("k_out", "v_out", "dst_row0", "src_record"))
    _call(device, "kvarn_expand_tile8", stream, tiles.data_ptr(), tiles.numel(), src_record.data_ptr(),
          k_out.data_ptr(), v_out.data_ptr(), stride, n_rows, dst_row0.data_ptr(), dst_row0.numel(),
          ctypes.byref(lay))


def decode8_workspace_bytes(B, Hq, Hkv, head_dim, max_tiles, win_capacity) -> int:
    n = ctypes.c_size_t()
    _check("kvarn_decode8_workspace_bytes",
           _L().kvarn_decode8_workspace_bytes(B, Hq, Hkv, head_dim, max_tiles, win_capacity,
                                              ctypes.byref(n)))
    return n.value


def decode_attention8(q, tiles, tile_table, n_tiles, win_k, win_v, win_start, win_len,
                      lay: Layout8, softmax_scale=None, mass_in=None, mass_out=None, ws=None,
                      out=None, stream=None, flags=0):
    """decode_attention over 8-bit records: q and out fp32, fp16 or bf16 [B][Hq][D],
    the other arguments as decode_attention's. With mass_out (fp32, tile_table's
    shape) the softmax weight each tile received, summed over the query heads of
    its KV head, is added to mass_in (None: zeros; may be mass_out itself)."""
    io, device = _io(q, "q")
    _fit(device, ("tiles", tiles, torch.uint8), ("tile_table", tile_table, torch.int64),
         ("n_tiles", n_tiles, torch.int32), ("win_k", win_k, torch.float32),
         ("win_v", win_v, torch.float32), ("win_start", win_start, torch.int32),
         ("win_len", win_len, torch.int32))
    if q.dim() != 3 or tile_table.dim() != 3 or win_k.dim() != 4:
        raise ValueError("decode_attention8: q [B][Hq][D], tile_table [B][Hkv][max_tiles], "
                         "win_k [B][Hkv][cap][D] expected")
    B, Hq, D = q.shape
    Bt, Hkv, max_tiles = tile_table.shape
    Bw, Hw, cap, Dw = win_k.shape
    if (Bt != B or n_tiles.numel() != B or win_start.numel() != B or win_len.numel() != B
            or win_k.shape != win_v.shape or (Bw, Hw, Dw) != (B, Hkv, D)):
        raise ValueError("decode_attention8: inconsistent shapes")
    for name, m in (("mass_in", mass_in), ("mass_out", mass_out)):
        if m is not None:
            _fit(device, (name, m, torch.float32))
            if m.shape != tile_table.shape:
                raise ValueError(f"{name} must have tile_table's shape")
    if ws is None:
        with torch.cuda.device(device):  # the split of the work depends on the device
            need = decode8_workspace_bytes(B, Hq, Hkv, D, max_tiles, cap)
        ws = _scratch(need, q.device, stream)
    if out is None:
        out = _result(q, stream)
    _fit(device, ("ws", ws, torch.uint8), ("out", out, q.dtype))
    if out.shape != q.shape:
        raise ValueError("out must have q's shape")
    _call(device, "kvarn_decode_attention8", stream, q.data_ptr(), io, tiles.data_ptr(), tiles.numel(),
          tile_table.data_ptr(), n_tiles.data_ptr(), win_k.data_ptr(), win_v.data_ptr(),
          win_start.data_ptr(), win_len.data_ptr(), cap, B, Hq, Hkv, D, max_tiles,
          D ** -0.5 if softmax_scale is None else float(softmax_scale), ctypes.byref(lay),
          None if mass_in is None else mass_in.data_ptr(),
          None if mass_out is None else mass_out.data_ptr(), ws.data_ptr(), ws.numel(), out.data_ptr(),
          int(flags))
    return out


def prefill8_workspace_bytes(C, n_tiles, win_len, Hq, Hkv, head_dim) -> int:
    n = ctypes.c_size_t()
    _check("kvarn_prefill8_workspace_bytes",
           _L().kvarn_prefill8_workspace_bytes(int(C), int(n_tiles), int(win_len), Hq, Hkv, head_dim,
                                               ctypes.byref(n)))
    return n.value


def prefill_attention8(q_chunk, pos0, tiles, tile_table, n_tiles, win_k, win_v, win_start, win_len,
                       lay: Layout8, softmax_scale=None, ws=None, out=None, stream=None):
    """prefill_attention over 8-bit records: q_chunk and out fp32, fp16 or bf16
    [C][Hq][D], the other arguments as prefill_attention's; ws a uint8 device
    workspace of prefill8_workspace_bytes() for these sizes or larger ones
    (allocated here when None)."""
    io, device = _io(q_chunk, "q_chunk")
    _fit(device, ("tiles", tiles, torch.uint8), ("tile_table", tile_table, torch.int64),
         ("win_k", win_k, torch.float32), ("win_v", win_v, torch.float32))
    if q_chunk.dim() != 3 or tile_table.dim() != 2 or win_k.dim() != 3:
        raise ValueError("prefill_attention8: q_chunk [C][Hq][D], tile_table [Hkv][stride], "
                         "win_k [Hkv][cap][D] expected")
    C, Hq, D = q_chunk.shape
    Hkv, stride = tile_table.shape
    Hw, cap, Dw = win_k.shape
    if win_k.shape != win_v.shape or (Hw, Dw) != (Hkv, D):
        raise ValueError("prefill_attention8: inconsistent shapes")
    if out is None:
        out = _result(q_chunk, stream)
    if ws is None:
        with torch.cuda.device(device):
            need = prefill8_workspace_bytes(C, n_tiles, win_len, Hq, Hkv, D)
        ws = _scratch(need, q_chunk.device, stream)
    _fit(device, ("ws", ws, torch.uint8), ("out", out, q_chunk.dtype))
    if out.shape != q_chunk.shape:
        raise ValueError("out must have q_chunk's shape")
    _call(device, "kvarn_prefill_attention8", stream, q_chunk.data_ptr(), io, C, int(pos0),
          tiles.data_ptr(), tiles.numel(), tile_table.data_ptr(), stride, int(n_tiles),
          win_k.data_ptr(), win_v.data_ptr(), int(win_start), int(win_len), cap, Hq, Hkv, D,
          D ** -0.5 if softmax_scale is None else float(softmax_scale), ctypes.byref(lay),
          ws.data_ptr(), ws.numel(), out.data_ptr())
    return out


def evict_tiles(tile_table, tile_mass, n_tiles, keep, sinks=0, recent=0, table_out=None,
                mass_out=None, n_tiles_out=None, evicted=None, stream=None, flags=0):
    """Drops tiles by accumulated weight (kvarn_evict_tiles): per KV head, of more
    than `keep` tiles stay the first `sinks`, the last `recent` and the heaviest
    between (tile_mass: what decode_attention8 or decode_attention4 adds up, or the caller's own). tile_table int64 and tile_mass fp32 [B][Hkv][max_tiles], n_tiles int32
    [B]. Outputs default to the inputs (in place); evicted (int64, tile_table's
    shape) receives the offsets that left. Returns (table, mass, n_tiles, evicted)."""
    _dev(tile_table, "tile_table", torch.int64)
    device = tile_table.get_device()
    table_out = tile_table if table_out is None else table_out
    mass_out = tile_mass if mass_out is None else mass_out
    n_tiles_out = n_tiles if n_tiles_out is None else n_tiles_out
    _fit(device, ("tile_mass", tile_mass, torch.float32), ("n_tiles", n_tiles, torch.int32),
         ("table_out", table_out, torch.int64), ("mass_out", mass_out, torch.float32),
         ("n_tiles_out", n_tiles_out, torch.int32))
    if evicted is not None:
        _fit(device, ("evicted", evicted, torch.int64))
    if tile_table.dim() != 3:
        raise ValueError("tile_table must be [B][Hkv][max_tiles]")
    shape = tile_table.shape
    B, Hkv, max_tiles = shape
    if (tile_mass.shape != shape or table_out.shape != shape or mass_out.shape != shape
            or n_tiles.numel() != B or n_tiles_out.numel() != B
            or (evicted is not None and evicted.shape != shape)):
        raise ValueError("evict_tiles: inconsistent shapes")
    _call(device, "kvarn_evict_tiles", stream, tile_table.data_ptr(), tile_mass.data_ptr(),
          n_tiles.data_ptr(), table_out.data_ptr(), mass_out.data_ptr(), n_tiles_out.data_ptr(),
          None if evicted is None else evicted.data_ptr(), B, Hkv, max_tiles, int(keep), int(sinks),
          int(recent), int(flags))
    return table_out, mass_out, n_tiles_out, evicted


# ---------------------------------------------------------------------------
# the 4-bit cache, and queries and keys made ready for any cache

def layout4(head_dim: int) -> Layout4:
    """Layout of a 4-bit tile record: integers -7..7 with a scale for each 32
    channels of a token of a head (4.5 bits per value)."""
    L = Layout4()
    _check("kvarn_layout4", _L().kvarn_layout4(head_dim, ctypes.byref(L)))
    return L


def _rows_of(t, name, dims, dtype=None, device=None):
    """A CUDA tensor [..., heads, D] of `dims` (3 or 4) dimensions whose heads lie side by side and whose
    rows (all but the last two axes) are a constant stride apart, as a slice of a packed
    product's result: its stride in elements, and its shape."""
    if (isinstance(t, torch.Tensor) and t.is_cuda and (t.dtype in IO_TYPES if dtype is None else t.dtype is dtype)
            and (device is None or t.get_device() == device)):
        shape = t.shape  # (the usual strides, without more ado)
        if len(shape) == dims:
            if t.is_contiguous():
                return shape[-1] * shape[-2], shape
            if dims == 3:
                row, head, one = t.stride()
                if one == 1 and head == shape[2] and shape[0] > 1:
                    return row, shape
    return _rows_checked(t, name, dims, dtype, device), t.shape


def _rows_checked(t, name, dims, dtype, device):
    if not (isinstance(t, torch.Tensor) and t.is_cuda):
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype not in IO_TYPES:
        raise TypeError(f"{name} must be float32, float16 or bfloat16, got {t.dtype}")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if device is not None and t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{device}")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {t.dim()}")
    shape = t.shape
    width = shape[-2] * shape[-1]
    if t.is_contiguous() or t.numel() == 0:
        return width
    stride = t.stride()
    if (shape[-1] > 1 and stride[-1] != 1) or (shape[-2] > 1 and stride[-2] != shape[-1]):
        raise ValueError(f"the heads of a row of {name} must be contiguous")
    # (the stride of an axis of one element says nothing)
    row, span = None, 1
    for n, s in zip(shape[-3::-1], stride[-3::-1]):
        if n != 1:
            if row is None:
                row = s // span if s % span == 0 else -1
            if s != row * span:
                raise ValueError(f"the rows of {name} must be a constant stride apart")
        span *= n
    return width if row is None else row


def _layout4_for(lay, D, what):
    if lay.head_dim != D:
        raise ValueError(f"{what}: the layout is for head_dim {lay.head_dim}, the rows have {D}")
    return ctypes.byref(lay)


def _counts4(counts, B, device):
    if counts is None:
        return None
    _fit(device, ("counts", counts, torch.int32))
    if counts.numel() != B:
        raise ValueError("counts must have one entry per sequence")
    return counts.data_ptr()


def _rows4(k, v, tiles, tile_table, first, lay, counts, names, what):
    """What write_rows4 and read_rows4 check alike: the strides, sizes and pointers of a call."""
    k_stride, shape = _rows_of(k, names[0], 4)
    device, dtype = k.get_device(), k.dtype
    v_stride, v_shape = _rows_of(v, names[1], 4, dtype, device)
    _fit(device, ("tiles", tiles, torch.uint8), ("tile_table", tile_table, torch.int64), (names[2], first, torch.int32))
    table = tile_table.shape
    B, T, Hkv, D = shape
    if v_shape != shape or len(table) != 3 or table[0] != B or table[1] != Hkv or first.numel() != B:
        raise ValueError(f"{what}: inconsistent shapes")
    return device, k_stride, v_stride, _counts4(counts, B, device), (IO_TYPES[dtype], B, T, Hkv, D, table[2],
                                                                     _layout4_for(lay, D, what))


def write_rows4(k_new, v_new, tiles, tile_table, lens, lay: Layout4, counts=None, stream=None, flags=0):
    """Quantises rows into the 4-bit cache: k_new, v_new fp32, fp16 or bf16 [B][T][Hkv][D] (slices of
    a packed tensor will do: heads contiguous, rows a constant stride apart); row (b, t), t <
    counts[b] (int32 [B]; None: T), becomes token lens[b] + t (int32 [B], not changed) of sequence b.
    tiles uint8 record pool; tile_table int64 [B][Hkv][max_tiles]."""
    device, ks, vs, n, (io, *sizes) = _rows4(k_new, v_new, tiles, tile_table, lens, lay, counts,
                                             ("k_new", "v_new", "lens"), "write_rows4")
    _call(device, "kvarn_write_rows4", stream, k_new.data_ptr(), ks, v_new.data_ptr(), vs, io, tiles.data_ptr(),
          tiles.numel(), tile_table.data_ptr(), lens.data_ptr(), n, *sizes, int(flags))


def read_rows4(tiles, tile_table, first, k_out, v_out, lay: Layout4, counts=None, stream=None, flags=0):
    """Cached tokens first[b] + t (int32 [B]) of the 4-bit cache as rows (b, t), t < counts[b], of k_out
    and v_out (as k_new and v_new of write_rows4); other rows stay as they are."""
    device, ks, vs, n, sizes = _rows4(k_out, v_out, tiles, tile_table, first, lay, counts,
                                      ("k_out", "v_out", "first"), "read_rows4")
    _call(device, "kvarn_read_rows4", stream, tiles.data_ptr(), tiles.numel(), tile_table.data_ptr(), first.data_ptr(),
          n, k_out.data_ptr(), ks, v_out.data_ptr(), vs, *sizes, int(flags))


def decode4_workspace_bytes(B, Hq, Hkv, head_dim, max_tiles, weights=True) -> int:
    """Bytes that decode_attention4 needs, with mass_out or (weights False) without."""
    n = ctypes.c_size_t()
    _check("kvarn_decode4_workspace_bytes",
           _L().kvarn_decode4_workspace_bytes(B, Hq, Hkv, head_dim, max_tiles, ctypes.byref(n)))
    return n.value if weights else n.value - 256 * B * Hkv * max_tiles


def decode_attention4(q, tiles, tile_table, lens, lay: Layout4, softmax_scale=None, mass_in=None,
                      mass_out=None, ws=None, out=None, stream=None, flags=0):
    """Attention of one query token per sequence over the first lens[b] (int32 [B]) cached tokens: q
    and out fp32, fp16 or bf16 [B][Hq][D]; tile_table int64 [B][Hkv][max_tiles]. mass_in and mass_out
    as decode_attention8's."""
    io, device = _io(q, "q")
    _fit(device, ("tiles", tiles, torch.uint8), ("tile_table", tile_table, torch.int64), ("lens", lens, torch.int32))
    shape, table = q.shape, tile_table.shape
    if len(shape) != 3 or len(table) != 3:
        raise ValueError("decode_attention4: q [B][Hq][D], tile_table [B][Hkv][max_tiles] expected")
    B, Hq, D = shape
    Bt, Hkv, max_tiles = table
    if Bt != B or lens.numel() != B:
        raise ValueError("decode_attention4: inconsistent shapes")
    for name, m in (("mass_in", mass_in), ("mass_out", mass_out)):
        if m is not None:
            _fit(device, (name, m, torch.float32))
            if m.shape != table:
                raise ValueError(f"{name} must have tile_table's shape")
    if ws is None:
        with torch.cuda.device(device):  # the split of the work depends on the device
            need = decode4_workspace_bytes(B, Hq, Hkv, D, max_tiles, weights=mass_out is not None)
        ws = _scratch(need, q.device, stream)
    if out is None:
        out = _result(q, stream)
    _fit(device, ("ws", ws, torch.uint8), ("out", out, q.dtype))
    if out.shape != shape:
        raise ValueError("out must have q's shape")
    _call(device, "kvarn_decode_attention4", stream, q.data_ptr(), io, tiles.data_ptr(), tiles.numel(),
          tile_table.data_ptr(), lens.data_ptr(), B, Hq, Hkv, D, max_tiles,
          D ** -0.5 if softmax_scale is None else float(softmax_scale), _layout4_for(lay, D, "decode_attention4"),
          None if mass_in is None else mass_in.data_ptr(),
          None if mass_out is None else mass_out.data_ptr(), ws.data_ptr(), ws.numel(), out.data_ptr(),
          int(flags))
    return out


def prefill4_workspace_bytes(C, n_tiles, Hq, Hkv, head_dim) -> int:
    n = ctypes.c_size_t()
    _check("kvarn_prefill4_workspace_bytes",
           _L().kvarn_prefill4_workspace_bytes(int(C), int(n_tiles), Hq, Hkv, head_dim, ctypes.byref(n)))
    return n.value


def prefill_attention4(q_chunk, pos0, tiles, tile_table, lay: Layout4, softmax_scale=None, ws=None,
                       out=None, stream=None):
    """Causal attention of a chunk of one sequence whose rows are in the 4-bit cache: q_chunk and out fp32,
    fp16 or bf16 [C][Hq][D] at positions pos0 + i; tile_table int64 [Hkv][stride]; ws a uint8 device
    workspace of prefill4_workspace_bytes() for C positions and ceil((pos0 + C) / 128) tiles, or more of
    either (allocated here when None)."""
    io, device = _io(q_chunk, "q_chunk")
    _fit(device, ("tiles", tiles, torch.uint8), ("tile_table", tile_table, torch.int64))
    shape, table = q_chunk.shape, tile_table.shape
    if len(shape) != 3 or len(table) != 2:
        raise ValueError("prefill_attention4: q_chunk [C][Hq][D], tile_table [Hkv][stride] expected")
    C, Hq, D = shape
    Hkv, stride = table
    if out is None:
        out = _result(q_chunk, stream)
    if ws is None:
        n_tiles = max(0, min(stride, -(-(int(pos0) + C) // TILE)))
        with torch.cuda.device(device):
            need = prefill4_workspace_bytes(C, n_tiles, Hq, Hkv, D)
        ws = _scratch(need, q_chunk.device, stream)
    _fit(device, ("ws", ws, torch.uint8), ("out", out, q_chunk.dtype))
    if out.shape != shape:
        raise ValueError("out must have q_chunk's shape")
    _call(device, "kvarn_prefill_attention4", stream, q_chunk.data_ptr(), io, C, int(pos0), tiles.data_ptr(),
          tiles.numel(), tile_table.data_ptr(), stride, Hq, Hkv, D,
          D ** -0.5 if softmax_scale is None else float(softmax_scale),
          _layout4_for(lay, D, "prefill_attention4"), ws.data_ptr(), ws.numel(), out.data_ptr())
    return out


def rotary(rotary_dim: int, theta: float = 10000.0, inv_freq=None, sections=None, pair_axis=None,
           pairing: str = "halves") -> Rotary:
    """Rotation plan of norm_rotate (kvarn_rotary): pair i of a head turns by inv_freq[i] (rotary_dim / 2
    numbers; None: theta ** (-2 i / rotary_dim)) radians per position. Positions of several axes: sections,
    pairs of each axis in order (their sum is rotary_dim / 2), or pair_axis, the axis of each pair.
    pairing "halves": channels (i, i + rotary_dim / 2); "adjacent": (2 i, 2 i + 1)."""
    if pairing not in PAIRINGS:
        raise ValueError(f"pairing must be one of {sorted(PAIRINGS)}, got {pairing!r}")
    pairs = rotary_dim // 2
    if inv_freq is None:
        inv_freq = [float(theta) ** (-2.0 * i / rotary_dim) for i in range(pairs)]
    inv_freq = [float(f) for f in inv_freq]
    if sections is not None:
        if pair_axis is not None:
            raise ValueError("sections or pair_axis, not both")
        pair_axis = [a for a, n in enumerate(sections) for _ in range(n)]
    if len(inv_freq) != pairs or (pair_axis is not None and len(pair_axis) != pairs):
        raise ValueError("inv_freq, sections and pair_axis must cover rotary_dim / 2 pairs")
    axes, n_axes = None, 1
    if pair_axis is not None:
        if any(not 0 <= int(a) < 4 for a in pair_axis):
            raise ValueError("a position has 1 to 4 axes")
        n_axes = len(sections) if sections is not None else max(int(a) for a in pair_axis) + 1
        axes = (ctypes.c_uint8 * max(pairs, 1))(*[int(a) for a in pair_axis])
    R = Rotary()
    _check("kvarn_rotary", _L().kvarn_rotary(rotary_dim, PAIRINGS[pairing],
                                             (ctypes.c_double * max(pairs, 1))(*inv_freq), axes, n_axes,
                                             ctypes.byref(R)))
    return R


def norm_rotate(q, k, positions, rot, q_weight=None, k_weight=None, eps=None, hadamard=False, q_out=None,
                k_out=None, stream=None, flags=0):
    """Queries and keys of new tokens made ready for a cache, in one pass: per head RMS norm (eps; None: no
    norm) with weights [D], rotation by position (rot: rotary(...), or None), and on request an orthonormal
    Walsh-Hadamard transform. q [T][Hq][D] and k [T][Hkv][D] (or None) fp32, fp16 or bf16, heads contiguous and
    tokens a constant stride apart; positions int64 [T], or [axes][T]. Outputs are new tensors, or q_out and
    k_out (q and k themselves: in place). Returns (q_out, k_out)."""
    q_stride, shape = _rows_of(q, "q", 3)
    device, dtype = q.get_device(), q.dtype
    T, Hq, D = shape
    if q_out is None:
        q_out = _result_rows(q, stream)
    qo_stride, o_shape = _rows_of(q_out, "q_out", 3, dtype, device)
    good = o_shape == shape
    if k is not None:
        k_stride, shape = _rows_of(k, "k", 3, dtype, device)
        if k_out is None:
            k_out = _result_rows(k, stream)
        ko_stride, o_shape = _rows_of(k_out, "k_out", 3, dtype, device)
        Hkv, k_in, k_to = shape[1], k.data_ptr(), k_out.data_ptr()
        good = good and shape[0] == T and shape[2] == D and o_shape == shape
    else:
        if k_out is not None or k_weight is not None:
            raise ValueError("norm_rotate: k_out or k_weight without k")
        Hkv, k_stride, ko_stride, k_in, k_to = 0, 0, 0, None, None
    if not good:
        raise ValueError("norm_rotate: inconsistent shapes")
    at = plan = None
    if rot is not None:
        _fit(device, ("positions", positions, torch.int64))
        axes = positions.shape
        if not axes or axes[-1] != T or positions.numel() != rot.n_axes * T:
            raise ValueError("positions must be [T], or [axes][T] with the plan's axes")
        at, plan = positions.data_ptr(), ctypes.byref(rot)
    q_scale = k_scale = None
    if q_weight is not None:
        q_scale = _weight_ptr(q_weight, "q_weight", device, dtype, D, eps)
    if k_weight is not None:
        k_scale = _weight_ptr(k_weight, "k_weight", device, dtype, D, eps)
    if eps is not None and not eps >= 0:
        raise ValueError("eps must not be negative")
    _call(device, "kvarn_norm_rotate", stream, q.data_ptr(), q_stride, k_in, k_stride, IO_TYPES[dtype], T, Hq, Hkv, D,
          q_scale, k_scale, -1.0 if eps is None else float(eps), at, plan, int(bool(hadamard)), q_out.data_ptr(),
          qo_stride, k_to, ko_stride, int(flags))
    return q_out, k_out


def _weight_ptr(w, name, device, dtype, D, eps):
    _fit(device, (name, w, dtype))
    if w.numel() != D:
        raise ValueError(f"{name} must have head_dim elements")
    if eps is None:
        raise ValueError(f"{name} without a norm (eps)")
    return w.data_ptr()


def _result_rows(like, stream):
    """_result, contiguous whatever the strides of `like`."""
    if stream is None:
        return torch.empty(like.shape, dtype=like.dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(like.shape, dtype=like.dtype, device=like.device)
