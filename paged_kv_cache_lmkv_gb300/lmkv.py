"""Python binding of liblmkv.so (argument marshalling only).

Every function here maps one-to-one onto an ``extern "C"`` entry point of
``include/lmkv.h``; all data movement runs in the library's CUDA kernels.
PyTorch tensors are used only as carriers of device memory and streams.  If
the library has not been built, the first call raises: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading
from typing import Sequence

import numpy as np
import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "liblmkv.so")

OK = 0
ERR_INVALID_ARG = 1
ERR_MISALIGNED = 2
ERR_CUDA = 3
ERR_UNSUPPORTED = 4
ERR_BAD_BLOCK = 5
ERR_BAD_POINTER = 6
ERR_TIMEOUT = 7
ERR_SCRATCH_LIMIT = 8
ERR_BAD_DATA = 9
ERR_BAD_LENGTH = 10
ERR_NO_PAGES = 11
BF16, FP16, FP32 = 0, 1, 2                  # lmkv_dtype_t
ROTARY_MAX_PAIRS = 128
ROTARY_SCALINGS = {"plain": 0, "linear": 1, "base": 2, "bands": 3, "ramp": 4, "yarn": 5}
NOALLOC_STAGING_BYTES = 64 << 20
CACHEGEN_BATCH = 256
CACHEGEN_MAX_CHANNELS = 2048
CACHEGEN_MAX_TOKENS = 4096
CACHEGEN_MAX_LAYERS = 128

ENTRY_POINTS = (
    "lmkv_count_chunks", "lmkv_enumerate_chunks", "lmkv_gather_chunks", "lmkv_scatter_chunks",
    "lmkv_gather_layer", "lmkv_scatter_layer", "lmkv_gather_chunks_fp8e4m3",
    "lmkv_scatter_chunks_fp8e4m3", "lmkv_status_string", "lmkv_abi_version",
    "lmkv_launch_count", "lmkv_store_layers", "lmkv_retrieve_layers",
    "lmkv_store_layers_staged", "lmkv_retrieve_layers_staged",
    "lmkv_store_layers_staged_noalloc", "lmkv_decode_store_ranges",
    "lmkv_offload_init", "lmkv_offload_plan", "lmkv_offload_copied", "lmkv_offload_allocate",
    "lmkv_offload_add_free", "lmkv_cachegen_default_bins", "lmkv_cachegen_layout",
    "lmkv_cachegen_workspace_bytes", "lmkv_cachegen_encode", "lmkv_cachegen_decode",
    "lmkv_cachegen_store_chunks", "lmkv_cachegen_retrieve_chunks",
    "lmkv_last_cuda_error", "lmkv_cuda_error_name",
    "lmkv_store_layers_overlapped", "lmkv_retrieve_layers_overlapped",
    "lmkv_rotary_init", "lmkv_append_layer", "lmkv_scatter_chunks_shifted",
    "lmkv_scatter_layer_shifted", "lmkv_attend_workspace_bytes", "lmkv_attend_layer",
    "lmkv_weigh_layer", "lmkv_evict_layer",
    "lmkv_append_layer_normed", "lmkv_attend_window_workspace_bytes", "lmkv_attend_layer_window",
    "lmkv_pages_workspace_bytes", "lmkv_copy_pages", "lmkv_fork_pages", "lmkv_resize_pages",
    "lmkv_compact_pages",
)


class LmkvError(RuntimeError):
    def __init__(self, code: int, what: str = ""):
        self.code = code
        msg = f"{what}: lmkv status {code} ({status_string(code)})"
        if code == ERR_CUDA:
            err = last_cuda_error()
            msg += f"; last CUDA error {err} ({cuda_error_name(err)})"
        super().__init__(msg)


class OffloadState(ctypes.Structure):
    """lmkv_offload_t: positions in the free-page order, start <= current <= end."""
    _fields_ = [("start", ctypes.c_int64), ("current", ctypes.c_int64), ("end", ctypes.c_int64),
                ("limit", ctypes.c_int64), ("window", ctypes.c_int64)]

    def as_tuple(self):
        return (self.start, self.current, self.end, self.limit, self.window)


class CachegenLayout(ctypes.Structure):
    """lmkv_cachegen_layout_t: byte offsets of one chunk's encoded blob."""
    _fields_ = [("max1_offset", ctypes.c_uint64), ("cdf_offset", ctypes.c_uint64),
                ("lengths_offset", ctypes.c_uint64), ("bytes_offset", ctypes.c_uint64),
                ("max_bytes", ctypes.c_uint64)]


class _RowsT(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class _BatchT(ctypes.Structure):
    _fields_ = [("q_start", ctypes.c_void_p), ("kv_len", ctypes.c_void_p),
                ("block_table", ctypes.c_void_p), ("max_blocks", ctypes.c_int32),
                ("num_req", ctypes.c_int32), ("num_tokens", ctypes.c_int32),
                ("max_new", ctypes.c_int32), ("max_kv_len", ctypes.c_int32)]


class _RotaryT(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("magnitude", ctypes.c_double), ("inv_freq", ctypes.c_double * ROTARY_MAX_PAIRS)]


class _PoolT(ctypes.Structure):
    _fields_ = [
        ("layer_base", ctypes.c_void_p),
        ("num_blocks", ctypes.c_int64),
        ("num_layers", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("block_size", ctypes.c_int32),
        ("elem_bytes", ctypes.c_int32),
    ]


_lib = None
_lock = threading.Lock()


def load() -> ctypes.CDLL:
    """Load liblmkv.so (raises if it is missing: build it with build.build())."""
    global _lib
    lib = _lib
    if lib is not None:
        return lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: the CUDA library must be built "
                               "(paged_kv_cache_lmkv_gb300.build.build()); there is no fallback")
        lib = ctypes.CDLL(LIB_PATH)
        P, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        pool_p = ctypes.POINTER(_PoolT)
        lib.lmkv_count_chunks.argtypes = [P, P, i32, i32, i32, P]
        lib.lmkv_decode_store_ranges.argtypes = [P, P, i32, i32, P, P, P]
        off_p = ctypes.POINTER(OffloadState)
        lib.lmkv_offload_init.argtypes = [off_p, i64, i64]
        lib.lmkv_offload_plan.argtypes = [off_p, i64, P, P]
        lib.lmkv_offload_copied.argtypes = [off_p, i64]
        lib.lmkv_offload_allocate.argtypes = [off_p, i64, P, P]
        lib.lmkv_offload_add_free.argtypes = [off_p, i64]
        lib.lmkv_enumerate_chunks.argtypes = [P, P, i32, i32, i32, P, P, P, i32]
        move = [pool_p, P, i32, P, P, i32, i32, i32, P, P, P]
        lib.lmkv_gather_chunks.argtypes = move
        lib.lmkv_scatter_chunks.argtypes = move
        layer = [pool_p, P, i32, P, P, i32, i32, i32, P, i32, P, P]
        lib.lmkv_gather_layer.argtypes = layer
        lib.lmkv_scatter_layer.argtypes = layer
        layers = [pool_p, P, i32, P, P, i32, i32, i32, P, i32, i32, P, P, P, P]
        lib.lmkv_store_layers.argtypes = layers
        lib.lmkv_retrieve_layers.argtypes = layers
        staged = [pool_p, P, i32, P, P, i32, i32, i32, P, P, i64, i32, i32, P, P, P, P]
        lib.lmkv_store_layers_staged.argtypes = staged
        lib.lmkv_retrieve_layers_staged.argtypes = staged
        lib.lmkv_store_layers_staged_noalloc.argtypes = [pool_p, P, i32, P, P, i32, i32, i32, P,
                                                         i32, i32, P, P, P, P]
        overlapped = [pool_p, P, i32, P, P, i32, i32, i32, P, P, i64, i32, i32, P, P, P, P, P, P]
        lib.lmkv_store_layers_overlapped.argtypes = overlapped
        lib.lmkv_retrieve_layers_overlapped.argtypes = overlapped
        fp8 = [pool_p, P, i32, P, P, i32, i32, i32, P, P, P, P]
        lib.lmkv_gather_chunks_fp8e4m3.argtypes = fp8
        lib.lmkv_scatter_chunks_fp8e4m3.argtypes = fp8
        lib.lmkv_cachegen_default_bins.argtypes = [i32, P]
        lib.lmkv_cachegen_layout.argtypes = [i32, i32, i32, P, ctypes.POINTER(CachegenLayout)]
        lib.lmkv_cachegen_workspace_bytes.argtypes = [i32, i32, P, i32, P]
        lib.lmkv_cachegen_encode.argtypes = [P, P, i32, i32, i32, P, P, P, P, ctypes.c_uint64, P, P]
        lib.lmkv_cachegen_decode.argtypes = [P, P, P, i32, i32, i32, P, P, P, ctypes.c_uint64, P, P]
        cg_pool = [pool_p, P, i32, P, P, i32, i32, i32, P, P, P, P, ctypes.c_uint64, P, P]
        lib.lmkv_cachegen_store_chunks.argtypes = cg_pool
        lib.lmkv_cachegen_retrieve_chunks.argtypes = cg_pool
        f64, f32 = ctypes.c_double, ctypes.c_float
        rows_p = batch_p = P
        rot_p = ctypes.POINTER(_RotaryT)
        lib.lmkv_rotary_init.argtypes = [rot_p, i32, i32, f64, i32, f64, f64, f64, f64]
        lib.lmkv_append_layer.argtypes = [pool_p, i32, i32, batch_p, i32, rows_p, rows_p, rows_p, rows_p,
                                          P, rot_p, P, P]
        shifted = [pool_p, i32, P, i32, P, P, i32, i32, i32, P, P, rot_p]
        lib.lmkv_scatter_chunks_shifted.argtypes = shifted + [P, P]
        lib.lmkv_scatter_layer_shifted.argtypes = shifted + [i32, P, P]
        lib.lmkv_attend_workspace_bytes.argtypes = [pool_p, i32, i32, i32, i32, i64, i32, P]
        lib.lmkv_attend_layer.argtypes = [pool_p, i32, i32, batch_p, i32, rows_p, P, i64, f32, rows_p, P,
                                          P, ctypes.c_uint64, P, P]
        lib.lmkv_weigh_layer.argtypes = [pool_p, i32, i32, batch_p, i32, rows_p, P, f32, f32, P, P, i64, P, P]
        lib.lmkv_evict_layer.argtypes = [pool_p, i32, P, i32, P, i32, i32, P, i64, i32, i32, i32, P, P, P,
                                         i64, P, P]
        lib.lmkv_append_layer_normed.argtypes = [pool_p, P, i32, i32, batch_p, i32, rows_p, rows_p, rows_p, rows_p,
                                                 P, rot_p, P, P, f32, P, P]
        lib.lmkv_attend_window_workspace_bytes.argtypes = [pool_p, i32, i32, i32, i32, i32, P]
        lib.lmkv_attend_layer_window.argtypes = [pool_p, P, i32, i32, batch_p, i32, rows_p, f32, i32, i32, rows_p, P,
                                                 P, ctypes.c_uint64, P, P]
        lib.lmkv_pages_workspace_bytes.argtypes = [pool_p, i32, P]
        lib.lmkv_copy_pages.argtypes = [pool_p, P, P, P, i32, P, P]
        lib.lmkv_fork_pages.argtypes = [pool_p, P, P, i32, P, i32, P, i32, P, P, P, P, P, ctypes.c_uint64, P, P]
        lib.lmkv_resize_pages.argtypes = [pool_p, P, i32, P, P, i32, P, P, P, P, ctypes.c_uint64, P, P]
        lib.lmkv_compact_pages.argtypes = [pool_p, P, P, i32, P, i32, P, P, P, P, P, ctypes.c_uint64, P, P]
        for name in ("lmkv_append_layer_normed", "lmkv_attend_window_workspace_bytes", "lmkv_attend_layer_window",
                     "lmkv_pages_workspace_bytes", "lmkv_copy_pages", "lmkv_fork_pages", "lmkv_resize_pages",
                     "lmkv_compact_pages", "lmkv_rotary_init", "lmkv_append_layer", "lmkv_scatter_chunks_shifted",
                     "lmkv_scatter_layer_shifted", "lmkv_attend_workspace_bytes", "lmkv_attend_layer",
                     "lmkv_weigh_layer", "lmkv_evict_layer",
                     "lmkv_count_chunks", "lmkv_enumerate_chunks", "lmkv_gather_chunks",
                     "lmkv_cachegen_default_bins", "lmkv_cachegen_layout",
                     "lmkv_cachegen_workspace_bytes", "lmkv_cachegen_encode", "lmkv_cachegen_decode",
                     "lmkv_cachegen_store_chunks", "lmkv_cachegen_retrieve_chunks",
                     "lmkv_decode_store_ranges", "lmkv_offload_init", "lmkv_offload_plan",
                     "lmkv_offload_copied", "lmkv_offload_allocate", "lmkv_offload_add_free",
                     "lmkv_scatter_chunks", "lmkv_gather_layer", "lmkv_scatter_layer",
                     "lmkv_gather_chunks_fp8e4m3", "lmkv_scatter_chunks_fp8e4m3",
                     "lmkv_abi_version", "lmkv_store_layers", "lmkv_retrieve_layers",
                     "lmkv_store_layers_staged", "lmkv_retrieve_layers_staged",
                     "lmkv_store_layers_staged_noalloc", "lmkv_store_layers_overlapped",
                     "lmkv_retrieve_layers_overlapped"):
            getattr(lib, name).restype = ctypes.c_int
        lib.lmkv_status_string.argtypes = [ctypes.c_int]
        lib.lmkv_status_string.restype = ctypes.c_char_p
        lib.lmkv_launch_count.argtypes = []
        lib.lmkv_launch_count.restype = ctypes.c_int64
        lib.lmkv_last_cuda_error.argtypes = []
        lib.lmkv_last_cuda_error.restype = ctypes.c_int
        lib.lmkv_cuda_error_name.argtypes = [ctypes.c_int]
        lib.lmkv_cuda_error_name.restype = ctypes.c_char_p
        _lib = lib
        return lib


def status_string(code: int) -> str:
    return load().lmkv_status_string(int(code)).decode()


def launch_count() -> int:
    return int(load().lmkv_launch_count())


def last_cuda_error() -> int:
    return int(load().lmkv_last_cuda_error())


def cuda_error_name(err: int) -> str:
    return load().lmkv_cuda_error_name(int(err)).decode()


def _i64_array(values) -> np.ndarray:
    """Contiguous int64 host array (no copy when it already is one)."""
    if isinstance(values, np.ndarray) and values.dtype == np.int64 and values.flags.c_contiguous:
        return values
    return np.ascontiguousarray(values, dtype=np.int64)


def _stream_handle(stream) -> int | None:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


class Pool:
    """A paged KV pool: per-layer device tensors [2][num_blocks][block_size][heads*head_dim].

    Holds the DEVICE array of layer base pointers the ABI takes.  scales: the
    tensors of an 8-bit pool's powers of two, per layer [2][num_blocks][heads] in
    float8_e8m0fnu or uint8 (value = code * 2^(byte - 127)); the layers then hold
    e4m3 codes, as float8_e4m3fn or uint8.  A scale belongs to a whole page, so the
    calls that move rows (gather, scatter, store, retrieve, the codec, evict_layer)
    refuse such a pool: whole pages move by copy_pages, fork_pages and compact_pages.
    """

    scales = scale_ptrs = None

    def __init__(self, layers: Sequence[torch.Tensor], num_kv_heads: int, head_dim: int,
                 scales: Sequence[torch.Tensor] | None = None):
        t0 = layers[0]
        if t0.dim() != 4 or t0.shape[0] != 2 or t0.shape[3] != num_kv_heads * head_dim:
            raise ValueError("pool layers must be [2][num_blocks][block_size][heads*head_dim]")
        for t in layers:
            if t.shape != t0.shape or t.dtype != t0.dtype or not t.is_contiguous() or not t.is_cuda:
                raise ValueError("pool layers must be contiguous CUDA tensors of one shape/dtype")
        self.layers = list(layers)
        self.num_kv_heads = num_kv_heads
        self.head_dim = head_dim
        self.block_size = t0.shape[2]
        self.num_blocks = t0.shape[1]
        self.elem_bytes = t0.element_size()
        self.ptrs = torch.tensor([t.data_ptr() for t in layers], dtype=torch.int64,
                                 device=t0.device)
        self._struct = _PoolT(self.ptrs.data_ptr(), self.num_blocks, len(layers), num_kv_heads,
                              head_dim, self.block_size, self.elem_bytes)
        if scales is not None:
            if t0.dtype not in (torch.float8_e4m3fn, torch.uint8):
                raise ValueError(f"scales belong to layers of e4m3 codes, got {t0.dtype}")
            if len(scales) != len(layers):
                raise ValueError("one tensor of scales for each layer")
            for t in scales:
                if t.shape != (2, self.num_blocks, num_kv_heads) or not t.is_contiguous() or t.device != t0.device or \
                        t.dtype not in (torch.float8_e8m0fnu, torch.uint8):
                    raise ValueError("scales must be contiguous float8_e8m0fnu or uint8 [2][num_blocks][heads] on the "
                                     "layers' device")
            self.scales = list(scales)
            self.scale_ptrs = torch.tensor([t.data_ptr() for t in scales], dtype=torch.int64, device=t0.device)

    @property
    def num_layers(self) -> int:
        return len(self.layers)

    @property
    def struct(self):
        return ctypes.byref(self._struct)


def pointer_array(tensors: Sequence[torch.Tensor], device) -> torch.Tensor:
    """DEVICE int64 array of the tensors' data pointers (chunk_ptrs / code_ptrs).

    The copy is queued on the current stream from pinned host memory, so the
    host does not wait for the device (the caching host allocator keeps the
    pinned block until the copy has run)."""
    host = torch.tensor([t.data_ptr() for t in tensors], dtype=torch.int64)
    if torch.device(device).type != "cuda":
        return host.to(device)
    return host.pin_memory().to(device, non_blocking=True)


def count_chunks(start, end, chunk_size: int, save_unfull: bool) -> int:
    lib = load()
    s, e = _i64_array(start), _i64_array(end)
    out = ctypes.c_int32(0)
    rc = lib.lmkv_count_chunks(s.ctypes.data, e.ctypes.data, len(s), chunk_size, int(save_unfull),
                               ctypes.byref(out))
    if rc != OK:
        raise LmkvError(rc, "lmkv_count_chunks")
    return out.value


def decode_store_ranges(stored_end, cur_end, chunk_size: int):
    """lmkv_decode_store_ranges -> (start, end, number of completed chunks)."""
    lib = load()
    s, e = _i64_array(stored_end), _i64_array(cur_end)
    out_s = np.zeros(len(s), np.int64)
    out_e = np.zeros(len(s), np.int64)
    n = ctypes.c_int32(0)
    rc = lib.lmkv_decode_store_ranges(s.ctypes.data, e.ctypes.data, len(s), chunk_size,
                                      out_s.ctypes.data, out_e.ctypes.data, ctypes.byref(n))
    if rc != OK:
        raise LmkvError(rc, "lmkv_decode_store_ranges")
    return out_s, out_e, n.value


class Offload:
    """Thin wrapper of the lmkv_offload_* calls on one caller-owned state."""

    def __init__(self, num_free: int, window: int):
        self.state = OffloadState()
        self._call("lmkv_offload_init", ctypes.byref(self.state), int(num_free), int(window))

    def _call(self, name, *args):
        rc = getattr(load(), name)(*args)
        if rc != OK:
            raise LmkvError(rc, name)

    def plan(self, max_pages: int):
        first, count = ctypes.c_int64(0), ctypes.c_int64(0)
        self._call("lmkv_offload_plan", ctypes.byref(self.state), int(max_pages),
                   ctypes.byref(first), ctypes.byref(count))
        return first.value, count.value

    def copied(self, count: int):
        self._call("lmkv_offload_copied", ctypes.byref(self.state), int(count))

    def allocate(self, want: int):
        g, s = ctypes.c_int64(0), ctypes.c_int64(0)
        self._call("lmkv_offload_allocate", ctypes.byref(self.state), int(want), ctypes.byref(g),
                   ctypes.byref(s))
        return g.value, s.value

    def add_free(self, n: int):
        self._call("lmkv_offload_add_free", ctypes.byref(self.state), int(n))


def enumerate_chunks(start, end, chunk_size: int, save_unfull: bool):
    """[(request, first token, n tokens)] in chunk order."""
    lib = load()
    n = count_chunks(start, end, chunk_size, save_unfull)
    s, e = _i64_array(start), _i64_array(end)
    req = (ctypes.c_int32 * max(n, 1))()
    tok0 = (ctypes.c_int64 * max(n, 1))()
    ntok = (ctypes.c_int32 * max(n, 1))()
    rc = lib.lmkv_enumerate_chunks(s.ctypes.data, e.ctypes.data, len(s), chunk_size,
                                   int(save_unfull), req, tok0, ntok, n)
    if rc != OK:
        raise LmkvError(rc, "lmkv_enumerate_chunks")
    return [(req[i], tok0[i], ntok[i]) for i in range(n)]


def _ptr(t):
    return None if t is None else t.data_ptr()


def _common(pool: Pool, block_table: torch.Tensor, start, end):
    """(pool, table, max_blocks, start, end, num_req) plus the host arrays to keep alive."""
    if pool.scales is not None:
        raise ValueError("rows of an 8-bit pool do not move apart from their page's scale (a Pool of the layers without "
                         "scales moves the codes alone)")
    if block_table.dtype != torch.int32:
        raise ValueError("block_table must be int32")
    s, e = _i64_array(start), _i64_array(end)
    if s.shape != e.shape:
        raise ValueError("start and end must have one entry per request")
    return (pool.struct, block_table.data_ptr(), block_table.shape[-1], s.ctypes.data,
            e.ctypes.data, len(s)), (s, e)


def gather_chunks(pool, block_table, start, end, chunk_size, save_unfull, chunk_ptrs,
                  status=None, stream=None) -> int:
    """lmkv_gather_chunks; returns the status code (0 = launched)."""
    a, _keep = _common(pool, block_table, start, end)
    return load().lmkv_gather_chunks(*a, chunk_size, int(save_unfull), _ptr(chunk_ptrs),
                                     _ptr(status), _stream_handle(stream))


def scatter_chunks(pool, block_table, start, end, chunk_size, save_unfull, chunk_ptrs,
                   status=None, stream=None) -> int:
    a, _keep = _common(pool, block_table, start, end)
    return load().lmkv_scatter_chunks(*a, chunk_size, int(save_unfull), _ptr(chunk_ptrs),
                                      _ptr(status), _stream_handle(stream))


def gather_layer(pool, block_table, start, end, chunk_size, save_unfull, chunk_ptrs, layer,
                 status=None, stream=None) -> int:
    a, _keep = _common(pool, block_table, start, end)
    return load().lmkv_gather_layer(*a, chunk_size, int(save_unfull), _ptr(chunk_ptrs),
                                    int(layer), _ptr(status), _stream_handle(stream))


def scatter_layer(pool, block_table, start, end, chunk_size, save_unfull, chunk_ptrs, layer,
                  status=None, stream=None) -> int:
    a, _keep = _common(pool, block_table, start, end)
    return load().lmkv_scatter_layer(*a, chunk_size, int(save_unfull), _ptr(chunk_ptrs),
                                     int(layer), _ptr(status), _stream_handle(stream))


def gather_chunks_fp8e4m3(pool, block_table, start, end, chunk_size, save_unfull, code_ptrs,
                          scales, status=None, stream=None) -> int:
    a, _keep = _common(pool, block_table, start, end)
    return load().lmkv_gather_chunks_fp8e4m3(*a, chunk_size, int(save_unfull), _ptr(code_ptrs),
                                             _ptr(scales), _ptr(status), _stream_handle(stream))


def scatter_chunks_fp8e4m3(pool, block_table, start, end, chunk_size, save_unfull, code_ptrs,
                           scales, status=None, stream=None) -> int:
    a, _keep = _common(pool, block_table, start, end)
    return load().lmkv_scatter_chunks_fp8e4m3(*a, chunk_size, int(save_unfull), _ptr(code_ptrs),
                                              _ptr(scales), _ptr(status), _stream_handle(stream))


def _event_array(events, n):
    """HOST array of n cudaEvent_t handles (0 = none) from torch.cuda.Event objects."""
    if events is None:
        return None
    if len(events) != n:
        raise ValueError("one event (or None) per layer")
    arr = (ctypes.c_void_p * max(n, 1))()
    for i, e in enumerate(events):
        if e is None:
            continue
        handle = e.cuda_event if isinstance(e, torch.cuda.Event) else int(e)
        if not handle:
            raise ValueError("event has no CUDA event yet: record it once first")
        arr[i] = handle
    return arr


def store_layers(pool, block_table, start, end, chunk_size, save_unfull, chunk_ptrs, layer_lo,
                 layer_n, layer_ready=None, layer_done=None, status=None, stream=None) -> int:
    """lmkv_store_layers: per layer, wait on layer_ready[i], gather, record layer_done[i]."""
    a, _keep = _common(pool, block_table, start, end)
    r, d = _event_array(layer_ready, layer_n), _event_array(layer_done, layer_n)
    return load().lmkv_store_layers(*a, chunk_size, int(save_unfull), _ptr(chunk_ptrs), int(layer_lo),
                                    int(layer_n), r, d, _ptr(status), _stream_handle(stream))


def retrieve_layers(pool, block_table, start, end, chunk_size, save_unfull, chunk_ptrs, layer_lo,
                    layer_n, layer_ready=None, layer_done=None, status=None, stream=None) -> int:
    """lmkv_retrieve_layers: per layer, wait on layer_ready[i], scatter, record layer_done[i]."""
    a, _keep = _common(pool, block_table, start, end)
    r, d = _event_array(layer_ready, layer_n), _event_array(layer_done, layer_n)
    return load().lmkv_retrieve_layers(*a, chunk_size, int(save_unfull), _ptr(chunk_ptrs),
                                       int(layer_lo), int(layer_n), r, d, _ptr(status),
                                       _stream_handle(stream))


def _host_ptr_array(tensors):
    """HOST array of the (pinned host) tensors' data pointers."""
    arr = (ctypes.c_void_p * max(len(tensors), 1))()
    for i, t in enumerate(tensors):
        arr[i] = t.data_ptr()
    return arr


def staging_bytes(pool, start, end, chunk_size, save_unfull) -> int:
    """Bytes of the one-layer staging buffer the staged pipeline needs."""
    n = sum(ntok for _, _, ntok in enumerate_chunks(start, end, chunk_size, save_unfull))
    return 2 * pool.num_kv_heads * pool.head_dim * pool.elem_bytes * n


def store_layers_staged(pool, block_table, start, end, chunk_size, save_unfull, host_chunks,
                        staging, layer_lo, layer_n, layer_ready=None, layer_done=None,
                        status=None, stream=None) -> int:
    """lmkv_store_layers_staged; host_chunks: pinned host tensors, staging: device tensor."""
    a, _keep = _common(pool, block_table, start, end)
    h = _host_ptr_array(host_chunks)
    r, d = _event_array(layer_ready, layer_n), _event_array(layer_done, layer_n)
    return load().lmkv_store_layers_staged(*a, chunk_size, int(save_unfull), h, _ptr(staging),
                                           staging.numel() * staging.element_size(), int(layer_lo),
                                           int(layer_n), r, d, _ptr(status), _stream_handle(stream))


def retrieve_layers_staged(pool, block_table, start, end, chunk_size, save_unfull, host_chunks,
                           staging, layer_lo, layer_n, layer_ready=None, layer_done=None,
                           status=None, stream=None) -> int:
    """lmkv_retrieve_layers_staged (host -> staging by 2-D copies, then scatter)."""
    a, _keep = _common(pool, block_table, start, end)
    h = _host_ptr_array(host_chunks)
    r, d = _event_array(layer_ready, layer_n), _event_array(layer_done, layer_n)
    return load().lmkv_retrieve_layers_staged(*a, chunk_size, int(save_unfull), h, _ptr(staging),
                                              staging.numel() * staging.element_size(),
                                              int(layer_lo), int(layer_n), r, d, _ptr(status),
                                              _stream_handle(stream))


def overlap_events(stream=None):
    """Four events for the overlapped pipeline (recorded once on `stream`, so
    that their CUDA handles exist)."""
    evs = [torch.cuda.Event() for _ in range(4)]
    for e in evs:
        e.record(stream)
    return evs


def _overlapped(fn, pool, block_table, start, end, chunk_size, save_unfull, host_chunks, staging,
                layer_lo, layer_n, sync_events, layer_ready, layer_done, status, stream, copy_stream):
    a, _keep = _common(pool, block_table, start, end)
    h = _host_ptr_array(host_chunks)
    r, d = _event_array(layer_ready, layer_n), _event_array(layer_done, layer_n)
    e = _event_array(sync_events, 4)
    if copy_stream is None:
        raise ValueError("the overlapped pipeline needs a copy stream")
    return fn(*a, chunk_size, int(save_unfull), h, _ptr(staging), staging.numel() * staging.element_size(),
              int(layer_lo), int(layer_n), r, d, e, _ptr(status), _stream_handle(stream),
              _stream_handle(copy_stream))


def store_layers_overlapped(pool, block_table, start, end, chunk_size, save_unfull, host_chunks,
                            staging, layer_lo, layer_n, sync_events, layer_ready=None,
                            layer_done=None, status=None, stream=None, copy_stream=None) -> int:
    """lmkv_store_layers_overlapped: two staging halves (staging holds 2 layers),
    kernels on `stream`, copies on `copy_stream`, 4 sync events (overlap_events())."""
    return _overlapped(load().lmkv_store_layers_overlapped, pool, block_table, start, end, chunk_size,
                       save_unfull, host_chunks, staging, layer_lo, layer_n, sync_events, layer_ready,
                       layer_done, status, stream, copy_stream)


def retrieve_layers_overlapped(pool, block_table, start, end, chunk_size, save_unfull, host_chunks,
                               staging, layer_lo, layer_n, sync_events, layer_ready=None,
                               layer_done=None, status=None, stream=None, copy_stream=None) -> int:
    """lmkv_retrieve_layers_overlapped (the inverse of store_layers_overlapped)."""
    return _overlapped(load().lmkv_retrieve_layers_overlapped, pool, block_table, start, end, chunk_size,
                       save_unfull, host_chunks, staging, layer_lo, layer_n, sync_events, layer_ready,
                       layer_done, status, stream, copy_stream)


def store_layers_staged_noalloc(pool, block_table, start, end, chunk_size, save_unfull,
                                host_chunks, layer_lo, layer_n, layer_ready=None, layer_done=None,
                                status=None, stream=None) -> int:
    """lmkv_store_layers_staged_noalloc: the staged store using the library's
    built-in 64 MiB device staging area instead of a caller buffer, for callers
    that cannot allocate device memory.  Make the first call on a device before
    any stream capture; calls that overlap on the GPU share the staging area."""
    a, _keep = _common(pool, block_table, start, end)
    h = _host_ptr_array(host_chunks)
    r, d = _event_array(layer_ready, layer_n), _event_array(layer_done, layer_n)
    return load().lmkv_store_layers_staged_noalloc(*a, chunk_size, int(save_unfull), h,
                                                   int(layer_lo), int(layer_n), r, d,
                                                   _ptr(status), _stream_handle(stream))


# ---- CacheGen codec ----

def _i32_array(values) -> np.ndarray:
    return np.ascontiguousarray(np.asarray(values).reshape(-1), dtype=np.int32)


def cachegen_default_bins(num_layers: int) -> np.ndarray:
    """int32 [2][num_layers] bins (row 0 K, row 1 V)."""
    out = np.zeros(2 * num_layers, np.int32)
    check(load().lmkv_cachegen_default_bins(num_layers, out.ctypes.data), "lmkv_cachegen_default_bins")
    return out.reshape(2, num_layers)


def cachegen_layout(num_layers: int, num_tokens: int, channels: int, bins) -> CachegenLayout:
    b = _i32_array(bins)
    out = CachegenLayout()
    check(load().lmkv_cachegen_layout(num_layers, num_tokens, channels, b.ctypes.data,
                                      ctypes.byref(out)), "lmkv_cachegen_layout")
    return out


def cachegen_workspace_bytes(num_layers: int, channels: int, num_tokens) -> int:
    n = _i32_array(num_tokens)
    out = ctypes.c_uint64(0)
    check(load().lmkv_cachegen_workspace_bytes(num_layers, channels, n.ctypes.data, len(n),
                                               ctypes.byref(out)), "lmkv_cachegen_workspace_bytes")
    return out.value


def cachegen_encode(chunk_ptrs, num_tokens, num_layers, channels, bins, blob_ptrs, sizes,
                    workspace, status=None, stream=None) -> int:
    """chunk_ptrs / blob_ptrs: DEVICE int64 pointer arrays; sizes: DEVICE uint64
    (int64 tensor) [num_chunks]; workspace: a DEVICE uint8 tensor."""
    n, b = _i32_array(num_tokens), _i32_array(bins)
    return load().lmkv_cachegen_encode(_ptr(chunk_ptrs), n.ctypes.data, len(n), num_layers, channels,
                                       b.ctypes.data, _ptr(blob_ptrs), _ptr(sizes), _ptr(workspace),
                                       workspace.numel() * workspace.element_size(), _ptr(status),
                                       _stream_handle(stream))


def cachegen_decode(blob_ptrs, sizes, num_tokens, num_layers, channels, bins, chunk_ptrs,
                    workspace, status=None, stream=None) -> int:
    n, b = _i32_array(num_tokens), _i32_array(bins)
    return load().lmkv_cachegen_decode(_ptr(blob_ptrs), _ptr(sizes), n.ctypes.data, len(n), num_layers,
                                       channels, b.ctypes.data, _ptr(chunk_ptrs), _ptr(workspace),
                                       workspace.numel() * workspace.element_size(), _ptr(status),
                                       _stream_handle(stream))


def cachegen_store_chunks(pool, block_table, start, end, chunk_size, save_unfull, bins, blob_ptrs,
                          sizes, workspace, status=None, stream=None) -> int:
    """Encode a store call's chunks straight from the pool's pages."""
    a, _keep = _common(pool, block_table, start, end)
    b = _i32_array(bins)
    return load().lmkv_cachegen_store_chunks(*a, chunk_size, int(save_unfull), b.ctypes.data,
                                             _ptr(blob_ptrs), _ptr(sizes), _ptr(workspace),
                                             workspace.numel() * workspace.element_size(), _ptr(status),
                                             _stream_handle(stream))


def cachegen_retrieve_chunks(pool, block_table, start, end, chunk_size, save_unfull, bins, blob_ptrs,
                             sizes, workspace, status=None, stream=None) -> int:
    """Decode blobs straight into the pages of a retrieve call's chunks."""
    a, _keep = _common(pool, block_table, start, end)
    b = _i32_array(bins)
    return load().lmkv_cachegen_retrieve_chunks(*a, chunk_size, int(save_unfull), b.ctypes.data,
                                                _ptr(blob_ptrs), _ptr(sizes), _ptr(workspace),
                                                workspace.numel() * workspace.element_size(),
                                                _ptr(status), _stream_handle(stream))


class CachegenCodec:
    """Chunk buffers [2][L][n][H] bf16 <-> CacheGen blobs, through
    lmkv_cachegen_encode / lmkv_cachegen_decode, and pool pages <-> blobs
    through the fused store / retrieve.  Holds the bins and a device workspace
    that grows to the largest batch seen (PyTorch memory); calls that share
    one codec object must be ordered on one stream (they share the
    workspace)."""

    _POINTER_CACHE = 32      # pointer arrays kept for reuse

    def __init__(self, num_layers: int, channels: int, bins=None, device="cuda"):
        self.num_layers, self.channels = num_layers, channels
        self.bins = _i32_array(cachegen_default_bins(num_layers) if bins is None else bins)
        self.device = torch.device(device)
        self.workspace = torch.empty(0, dtype=torch.uint8, device=self.device)
        self._need = {}          # token counts -> workspace bytes
        self._ptrs = {}          # data pointers -> (device pointer array, event after its copy)

    def layout(self, num_tokens: int) -> CachegenLayout:
        return cachegen_layout(self.num_layers, num_tokens, self.channels, self.bins)

    def _workspace(self, ntok):
        key = tuple(ntok)
        need = self._need.get(key)
        if need is None:
            need = self._need[key] = cachegen_workspace_bytes(self.num_layers, self.channels, ntok)
        if self.workspace.numel() < need:
            self.workspace = torch.empty(need, dtype=torch.uint8, device=self.device)
        return self.workspace

    def _pointers(self, tensors):
        """The device pointer array of the tensors, reused while the same
        addresses come back (a serving loop with fixed buffers builds it once).
        The current stream waits for the copy that filled it (outside a
        stream capture; warm up before capturing)."""
        key = tuple(t.data_ptr() for t in tensors)
        hit = self._ptrs.pop(key, None)
        if hit is None:
            arr = pointer_array(tensors, self.device)
            ev = torch.cuda.Event()
            ev.record(torch.cuda.current_stream(self.device))
            hit = (arr, ev)
            if len(self._ptrs) >= self._POINTER_CACHE:
                self._ptrs.pop(next(iter(self._ptrs)))
        else:
            cur = torch.cuda.current_stream(self.device)
            if not torch.cuda.is_current_stream_capturing():
                cur.wait_event(hit[1])
            hit[0].record_stream(cur)    # evicted later: freed only after this stream's use
        self._ptrs[key] = hit            # most recently used last
        return hit[0]

    def encode(self, chunks, blobs=None, sizes=None, status=None, stream=None):
        """Encode the chunk tensors; returns (blobs, sizes): device uint8 tensors
        of each layout's max_bytes and a device int64 tensor of the sizes."""
        ntok = [int(c.shape[2]) for c in chunks]
        if blobs is None:
            blobs = [torch.empty(self.layout(n).max_bytes, dtype=torch.uint8, device=self.device)
                     for n in ntok]
        if sizes is None:
            sizes = torch.zeros(len(chunks), dtype=torch.int64, device=self.device)
        ws = self._workspace(ntok)
        cptr, bptr = self._pointers(chunks), self._pointers(blobs)
        self._order(stream, cptr, bptr)
        check(cachegen_encode(cptr, ntok, self.num_layers, self.channels, self.bins, bptr, sizes, ws,
                              status, stream), "lmkv_cachegen_encode")
        return blobs, sizes

    def _order(self, stream, *arrays):
        """The pointer arrays are written on the current stream: a different
        `stream` waits for them and keeps them alive until it has read them."""
        if stream is None:
            return
        cur = torch.cuda.current_stream(self.device)
        if isinstance(stream, torch.cuda.Stream) and stream != cur:
            stream.wait_stream(cur)
            for a in arrays:
                a.record_stream(stream)

    def store(self, pool, block_table, start, end, chunk_size, save_unfull, blobs=None, sizes=None,
              status=None, stream=None):
        """Encode a store call's chunks straight from the pool; returns (blobs, sizes)."""
        ntok = [n for _, _, n in enumerate_chunks(start, end, chunk_size, save_unfull)]
        if blobs is None:
            blobs = [torch.empty(self.layout(n).max_bytes, dtype=torch.uint8, device=self.device)
                     for n in ntok]
        if sizes is None:
            sizes = torch.zeros(len(ntok), dtype=torch.int64, device=self.device)
        ws = self._workspace(ntok)
        bptr = self._pointers(blobs)
        self._order(stream, bptr)
        check(cachegen_store_chunks(pool, block_table, start, end, chunk_size, save_unfull, self.bins,
                                    bptr, sizes, ws, status, stream), "lmkv_cachegen_store_chunks")
        return blobs, sizes

    def retrieve(self, pool, block_table, start, end, chunk_size, save_unfull, blobs, sizes,
                 status=None, stream=None):
        """Decode blobs straight into the pool's pages of a retrieve call's chunks."""
        ntok = [n for _, _, n in enumerate_chunks(start, end, chunk_size, save_unfull)]
        ws = self._workspace(ntok)
        bptr = self._pointers(blobs)
        self._order(stream, bptr)
        check(cachegen_retrieve_chunks(pool, block_table, start, end, chunk_size, save_unfull, self.bins,
                                       bptr, sizes, ws, status, stream), "lmkv_cachegen_retrieve_chunks")

    def decode(self, blobs, sizes, chunks, status=None, stream=None):
        """Decode into the chunk tensors (their token counts give n)."""
        ntok = [int(c.shape[2]) for c in chunks]
        ws = self._workspace(ntok)
        bptr, cptr = self._pointers(blobs), self._pointers(chunks)
        self._order(stream, bptr, cptr)
        check(cachegen_decode(bptr, sizes, ntok, self.num_layers, self.channels, self.bins, cptr, ws,
                              status, stream), "lmkv_cachegen_decode")
        return chunks


# ---- attention-side operators -------------------------------------------

_DTYPES = {torch.bfloat16: BF16, torch.float16: FP16, torch.float32: FP32}


class Rotary:
    """A rotary encoding (lmkv_rotary_t): inv_freq[i] = base^(-2i / rot_dim), scaled as
    lmkv_rotary_init describes, or the given inv_freq (radians per position).  scaling: "plain",
    "linear", "base", "bands", "yarn" (as checkpoints that name it are made) or "ramp" (between fractional
    pairs: no checkpoint's form)."""

    def __init__(self, rot_dim: int, base: float = 10000.0, interleaved: bool = False,
                 scaling: str = "plain", factor: float = 1.0, low: float = 1.0, high: float = 32.0,
                 original: float = 4096.0, inv_freq=None, magnitude: float | None = None):
        if scaling not in ROTARY_SCALINGS:
            raise ValueError(f"scaling must be one of {sorted(ROTARY_SCALINGS)}")
        self._struct = _RotaryT()
        rc = load().lmkv_rotary_init(ctypes.byref(self._struct), int(rot_dim), int(interleaved), float(base),
                                     ROTARY_SCALINGS[scaling], float(factor), float(low), float(high),
                                     float(original))
        if rc != OK:
            raise LmkvError(rc, "lmkv_rotary_init")
        if inv_freq is not None:
            f = np.ascontiguousarray(inv_freq, dtype=np.float64)
            if f.shape != (int(rot_dim) // 2,):
                raise ValueError("inv_freq must hold rot_dim / 2 frequencies")
            self._struct.inv_freq[:len(f)] = f.tolist()
        if magnitude is not None:
            self._struct.magnitude = float(magnitude)

    @property
    def rot_dim(self) -> int:
        return self._struct.rot_dim

    @property
    def magnitude(self) -> float:
        return self._struct.magnitude

    @property
    def inv_freq(self) -> np.ndarray:
        return np.array(self._struct.inv_freq[:self._struct.rot_dim // 2], np.float64)

    @property
    def struct(self):
        return ctypes.byref(self._struct)


# A decode step makes these calls once per layer with microseconds of GPU work
# in each, so the marshalling is written for few Python operations: structures
# are packed into bytes and the checks compare whole shapes.
_ROWS = struct.Struct("@Pqq")               # lmkv_rows_t
_BATCH = struct.Struct("@PPPiiiii")         # lmkv_batch_t
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_of(pool: Pool, dev: int, stream):
    """The stream handle of a call on the pool's device, which has to be the
    current one (the library launches there)."""
    if dev >= 0 and torch.cuda.current_device() != dev:
        raise ValueError(f"the pool's device cuda:{dev} is not the current one")
    if stream is None:
        return torch.cuda.current_stream(dev).cuda_stream if _raw_stream is None or dev < 0 else _raw_stream(dev)
    return _stream_handle(stream)


def _elsewhere(dev, names, tensors):
    """Raises for the first tensor that is not on the pool's device."""
    for name, t in zip(names, tensors):
        if t is not None and t.get_device() != dev:
            raise ValueError(f"{name} is on {t.device}, the pool on {'cuda:%d' % dev if dev >= 0 else 'the CPU'}")


def _dtype_of(t0: torch.Tensor) -> int:
    dtype = _DTYPES.get(t0.dtype)
    if dtype is None:
        raise ValueError(f"no operators for a pool of {t0.dtype}")
    return dtype


def _rows(name: str, t: torch.Tensor, dtype, dev: int, shape) -> bytes:
    """lmkv_rows_t of a [tokens][heads][head_dim] tensor of the pool's type, any
    strides over tokens and heads."""
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)} ([tokens][heads][head_dim]), got {list(t.shape)}")
    if t.dtype != dtype or t.get_device() != dev:
        raise ValueError(f"{name} must be {dtype} on the pool's device, got {t.dtype} on {t.device}")
    ts, hs, es = t.stride()
    if es != 1:
        raise ValueError(f"{name}: a head's elements must be contiguous")
    return _ROWS.pack(t.data_ptr(), ts, hs)


def _whole(name: str, t: torch.Tensor, dtype, dev: int, shape) -> int:
    """Pointer of a contiguous tensor of this type and shape on the pool's device."""
    if t.shape != shape or t.dtype != dtype or not t.is_contiguous() or t.get_device() != dev:
        raise ValueError(f"{name} must be contiguous {dtype} {list(shape)} on the pool's device, got {t.dtype} "
                         f"{list(t.shape)} on {t.device}")
    return t.data_ptr()


def _status(status, dev: int):
    if status is None:
        return None
    if status.dtype != torch.int32 or status.get_device() != dev:
        raise ValueError("status must be int32 on the pool's device")
    return status.data_ptr()


def _heads_of(name: str, t: torch.Tensor):
    """(tokens, heads) of a [tokens][heads][head_dim] tensor."""
    shape = t.shape
    if len(shape) != 3:
        raise ValueError(f"{name} must be [tokens][heads][head_dim], got {list(shape)}")
    return shape[0], shape[1]


def _batch(pool: Pool, dev: int, block_table, q_start, kv_len, num_tokens, max_new, max_kv_len):
    """(lmkv_batch_t, number of requests)."""
    n, cols = kv_len.shape[0], block_table.shape[-1]
    i32 = torch.int32
    return _BATCH.pack(_whole("q_start", q_start, i32, dev, (n + 1,)), _whole("kv_len", kv_len, i32, dev, (n,)),
                       _whole("block_table", block_table, i32, dev, (n, cols)), cols, n, num_tokens,
                       num_tokens if max_new is None else max_new,
                       cols * pool.block_size if max_kv_len is None else max_kv_len), n


def append_layer(pool, layer, block_table, q, k, v, q_out, q_start, kv_len, rotary, positions=None,
                 status=None, stream=None) -> int:
    """lmkv_append_layer: rotate q into q_out (may be q), rotate k and copy v into
    the pages of the last q_start[r+1] - q_start[r] cached tokens of each
    request.  q, k, v: [tokens][heads][head_dim]; returns the status code."""
    t0 = pool.layers[0]
    dt, dev = t0.dtype, t0.get_device()
    tokens, heads = _heads_of("q", q)
    qs, ks = (tokens, heads, pool.head_dim), (tokens, pool.num_kv_heads, pool.head_dim)
    b, _ = _batch(pool, dev, block_table, q_start, kv_len, tokens, None, None)
    return load().lmkv_append_layer(
        pool.struct, _dtype_of(t0), int(layer), b, heads, _rows("q", q, dt, dev, qs), _rows("k", k, dt, dev, ks),
        _rows("v", v, dt, dev, ks), _rows("q_out", q_out, dt, dev, qs),
        None if positions is None else _whole("positions", positions, torch.int64, dev, (tokens,)),
        rotary.struct, _status(status, dev), _stream_of(pool, dev, stream))


def _shifted_args(pool, block_table, start, end, chunk_size, save_unfull, chunk_ptrs, shift, rotary, status):
    t0 = pool.layers[0]
    dev = t0.get_device()
    _elsewhere(dev, ("block_table", "chunk_ptrs", "status"), (block_table, chunk_ptrs, status))
    s, e, sh = _i64_array(start), _i64_array(end), _i64_array(shift)
    if s.shape != e.shape or s.shape != sh.shape:
        raise ValueError("start, end and shift must have one entry per request")
    if block_table.dtype != torch.int32 or not block_table.is_contiguous() or block_table.dim() != 2 or \
            block_table.shape[0] < len(s):
        raise ValueError("block_table must be contiguous int32 [requests][blocks]")
    # the host arrays go as bytes: they are read during the call
    return (pool.struct, _dtype_of(t0), block_table.data_ptr(), block_table.shape[-1], s.tobytes(), e.tobytes(),
            len(s), chunk_size, int(save_unfull), _ptr(chunk_ptrs), sh.tobytes(), rotary.struct), dev


def scatter_chunks_shifted(pool, block_table, start, end, chunk_size, save_unfull, chunk_ptrs, shift, rotary,
                           status=None, stream=None) -> int:
    """lmkv_scatter_chunks_shifted: scatter_chunks with request r's keys turned by
    shift[r] positions."""
    a, dev = _shifted_args(pool, block_table, start, end, chunk_size, save_unfull, chunk_ptrs, shift, rotary, status)
    return load().lmkv_scatter_chunks_shifted(*a, _ptr(status), _stream_of(pool, dev, stream))


def scatter_layer_shifted(pool, block_table, start, end, chunk_size, save_unfull, chunk_ptrs, shift, rotary,
                          layer, status=None, stream=None) -> int:
    """lmkv_scatter_layer_shifted: scatter_layer with request r's keys turned by
    shift[r] positions."""
    a, dev = _shifted_args(pool, block_table, start, end, chunk_size, save_unfull, chunk_ptrs, shift, rotary, status)
    return load().lmkv_scatter_layer_shifted(*a, int(layer), _ptr(status), _stream_of(pool, dev, stream))


def attend_workspace_bytes(pool, num_q_heads: int, num_tokens: int, num_req: int, max_new: int,
                           prefix_len: int = 0, max_kv_len: int = 0) -> int:
    """Bytes of workspace for attend_layer calls within these bounds (smaller ones too)."""
    out = ctypes.c_uint64(0)
    check(load().lmkv_attend_workspace_bytes(pool.struct, int(num_q_heads), int(num_tokens), int(num_req),
                                             int(max_new), int(prefix_len), int(max_kv_len),
                                             ctypes.byref(out)), "lmkv_attend_workspace_bytes")
    return out.value


def attend_layer(pool, layer, q, out, q_start, kv_len, block_table, scale, workspace, prefix_table=None,
                 prefix_len=0, lse=None, max_new=None, max_kv_len=None, status=None, stream=None) -> int:
    """lmkv_attend_layer: attention of q [tokens][heads][head_dim] to the shared
    prefix and the requests' own cached tokens, into out (and lse, float32
    [tokens][heads]).  max_new and max_kv_len bound the lengths on the device
    (default: the rows of q, the table's width); tight ones cost less.
    workspace: uint8 of attend_workspace_bytes for the same bounds or larger ones."""
    t0 = pool.layers[0]
    dt, dev = t0.dtype, t0.get_device()
    tokens, heads = _heads_of("q", q)
    qs = (tokens, heads, pool.head_dim)
    b, _ = _batch(pool, dev, block_table, q_start, kv_len, tokens, max_new, max_kv_len)
    table = None
    if prefix_len > 0:
        if prefix_table is None or prefix_table.numel() * pool.block_size < prefix_len:
            raise ValueError("prefix_table does not cover prefix_len")
        table = _whole("prefix_table", prefix_table, torch.int32, dev, (prefix_table.numel(),))
    wp, size = None, 0
    if workspace is not None:
        wp = _whole("workspace", workspace, torch.uint8, dev, (workspace.numel(),))
        size = workspace.numel()
    return load().lmkv_attend_layer(
        pool.struct, _dtype_of(t0), int(layer), b, heads, _rows("q", q, dt, dev, qs), table, int(prefix_len),
        float(scale), _rows("out", out, dt, dev, qs),
        None if lse is None else _whole("lse", lse, torch.float32, dev, (tokens, heads)), wp, size,
        _status(status, dev), _stream_of(pool, dev, stream))


def weigh_layer(pool, layer, q, lse, q_start, kv_len, block_table, scale, scores, scores_out, decay=1.0,
                max_new=None, max_kv_len=None, status=None, stream=None) -> int:
    """lmkv_weigh_layer: scores_out = decay * scores + the attention weight every
    own cached token receives from q, per KV head.  scores, scores_out:
    float32 [requests][kv heads][stride]; scores_out may be scores, and scores
    None when decay is 0.  max_kv_len defaults to what the table and the
    scores have room for."""
    t0 = pool.layers[0]
    dt, dev = t0.dtype, t0.get_device()
    tokens, heads = _heads_of("q", q)
    stride = scores_out.shape[-1]
    if max_kv_len is None:
        max_kv_len = min(block_table.shape[-1] * pool.block_size, stride)
    b, n = _batch(pool, dev, block_table, q_start, kv_len, tokens, max_new, max_kv_len)
    shape = (n, pool.num_kv_heads, stride)
    return load().lmkv_weigh_layer(
        pool.struct, _dtype_of(t0), int(layer), b, heads, _rows("q", q, dt, dev, (tokens, heads, pool.head_dim)),
        _whole("lse", lse, torch.float32, dev, (tokens, heads)), float(scale), float(decay),
        None if scores is None else _whole("scores", scores, torch.float32, dev, shape),
        _whole("scores_out", scores_out, torch.float32, dev, shape), stride, _status(status, dev),
        _stream_of(pool, dev, stream))


def evict_layer(pool, layer, block_table, kv_len, scores, sinks, recent, keep, new_len, kept_scores=None,
                max_kv_len=None, status=None, stream=None) -> int:
    """lmkv_evict_layer: keep the first `sinks`, the last `recent` and the highest
    scores of each request's cached tokens, keep.shape[-1] in all, per KV head,
    and move their rows to the front of the request's pages.  Writes keep
    (int32 [requests][kv heads][budget]), new_len and kept_scores; the caller
    then takes new_len as kv_len and frees the pages behind it.  max_kv_len
    defaults to what the table and the scores have room for.  Not for an 8-bit
    pool with scales, which belong to whole pages."""
    dev = pool.layers[0].get_device()
    if pool.scales is not None:
        raise ValueError("rows of an 8-bit pool do not move apart from their page's scale")
    n, cols, kh = kv_len.shape[0], block_table.shape[-1], pool.num_kv_heads
    stride, budget = scores.shape[-1], keep.shape[-1]
    i32, f32 = torch.int32, torch.float32
    kp, kept_stride = None, 0
    if kept_scores is not None:
        kept_stride = kept_scores.shape[-1]
        kp = _whole("kept_scores", kept_scores, f32, dev, (n, kh, kept_stride))
    if max_kv_len is None:
        max_kv_len = min(cols * pool.block_size, stride)
    return load().lmkv_evict_layer(
        pool.struct, int(layer), _whole("block_table", block_table, i32, dev, (n, cols)), cols,
        _whole("kv_len", kv_len, i32, dev, (n,)), n, int(max_kv_len),
        _whole("scores", scores, f32, dev, (n, kh, stride)), stride, budget, int(sinks), int(recent), _whole("keep", keep, i32, dev, (n, kh, budget)),
        _whole("new_len", new_len, i32, dev, (n,)), kp, kept_stride, _status(status, dev),
        _stream_of(pool, dev, stream))


# ---- the 8-bit cache ------------------------------------------------------

def _cache_dtype(pool, name: str, t: torch.Tensor):
    """(element type of the rows, lmkv_dtype_t, DEVICE array of scales or None) of a call on a
    16-bit pool, whose type the rows have, or an 8-bit one."""
    dt, scales = t.dtype, pool.scale_ptrs
    code = _DTYPES.get(dt)
    if code is None or code == FP32:
        raise ValueError(f"{name} must be bfloat16 or float16, got {dt}")
    if scales is not None:
        return dt, code, scales.data_ptr()
    t0 = pool.layers[0]
    if t0.element_size() == 1:
        raise ValueError("an 8-bit pool needs its scales (Pool(..., scales=))")
    return t0.dtype, _dtype_of(t0), None


def append_layer_normed(pool, layer, block_table, q, k, v, q_out, q_start, kv_len, rotary=None, q_norm=None,
                        k_norm=None, eps=1e-6, positions=None, status=None, stream=None) -> int:
    """lmkv_append_layer_normed: append_layer for models that norm each head of q and k
    (q_norm, k_norm: float32 [head_dim], or None) before the rotation (rotary, or None),
    into 16-bit pages or, with the pool's scales, pages of e4m3 codes."""
    dev = pool.layers[0].get_device()
    tokens, heads = _heads_of("q", q)
    dt, code, scales = _cache_dtype(pool, "q", q)
    d = pool.head_dim
    qs, ks = (tokens, heads, d), (tokens, pool.num_kv_heads, d)
    b, _ = _batch(pool, dev, block_table, q_start, kv_len, tokens, None, None)
    f32 = torch.float32
    return load().lmkv_append_layer_normed(
        pool.struct, scales, code, int(layer), b, heads, _rows("q", q, dt, dev, qs), _rows("k", k, dt, dev, ks),
        _rows("v", v, dt, dev, ks), _rows("q_out", q_out, dt, dev, qs),
        None if positions is None else _whole("positions", positions, torch.int64, dev, (tokens,)),
        None if rotary is None else rotary.struct,
        None if q_norm is None else _whole("q_norm", q_norm, f32, dev, (d,)),
        None if k_norm is None else _whole("k_norm", k_norm, f32, dev, (d,)), float(eps), _status(status, dev),
        _stream_of(pool, dev, stream))


def _count(n) -> int:
    """A number of tokens for the library's 32 bits: as good as all of them where it is larger, refused below 0."""
    return max(-1, min(int(n), 2 ** 31 - 1))


def attend_window_workspace_bytes(pool, num_q_heads: int, num_tokens: int, num_req: int, max_new: int,
                                  max_kv_len: int = 0) -> int:
    """Bytes of workspace for attend_layer_window calls within these bounds (smaller ones too)."""
    out = ctypes.c_uint64(0)
    check(load().lmkv_attend_window_workspace_bytes(pool.struct, int(num_q_heads), int(num_tokens), int(num_req),
                                                    int(max_new), int(max_kv_len), ctypes.byref(out)),
          "lmkv_attend_window_workspace_bytes")
    return out.value


def attend_layer_window(pool, layer, q, out, q_start, kv_len, block_table, scale, workspace, window=0, sinks=0,
                        lse=None, max_new=None, max_kv_len=None, status=None, stream=None) -> int:
    """lmkv_attend_layer_window: attention of q [tokens][heads][head_dim] to the requests'
    own cached tokens, 16-bit or 8-bit, into out (and lse, float32 [tokens][heads]).  With a
    window (0: none) token t sees the last `window` tokens up to itself, and the first
    `sinks`.  max_new and max_kv_len bound the lengths on the device, as in attend_layer."""
    dev = pool.layers[0].get_device()
    tokens, heads = _heads_of("q", q)
    dt, code, scales = _cache_dtype(pool, "q", q)
    qs = (tokens, heads, pool.head_dim)
    b, _ = _batch(pool, dev, block_table, q_start, kv_len, tokens, max_new, max_kv_len)
    return load().lmkv_attend_layer_window(
        pool.struct, scales, code, int(layer), b, heads, _rows("q", q, dt, dev, qs), float(scale), _count(window),
        _count(sinks), _rows("out", out, dt, dev, qs),
        None if lse is None else _whole("lse", lse, torch.float32, dev, (tokens, heads)),
        _whole("workspace", workspace, torch.uint8, dev, (workspace.numel(),)), workspace.numel(),
        _status(status, dev), _stream_of(pool, dev, stream))


# ---- pages ----------------------------------------------------------------

def pages_workspace_bytes(pool, rows: int) -> int:
    """Bytes of workspace for fork_pages, resize_pages and compact_pages on tables of up to this many rows."""
    out = ctypes.c_uint64(0)
    check(load().lmkv_pages_workspace_bytes(pool.struct, int(rows), ctypes.byref(out)), "lmkv_pages_workspace_bytes")
    return out.value


def _scales(pool):
    return None if pool.scale_ptrs is None else pool.scale_ptrs.data_ptr()


def copy_pages(pool, src, dst, status=None, stream=None) -> int:
    """lmkv_copy_pages: page src[i] to page dst[i] (int32), all layers, K and V, and their scales."""
    dev = pool.layers[0].get_device()
    n = src.shape[0]
    return load().lmkv_copy_pages(pool.struct, _scales(pool), _whole("src", src, torch.int32, dev, (n,)),
                                  _whole("dst", dst, torch.int32, dev, (n,)), n, _status(status, dev),
                                  _stream_of(pool, dev, stream))


def fork_pages(pool, block_table, kv_len, parents, refs, table_out, len_out, refs_out, workspace, status=None,
               stream=None) -> int:
    """lmkv_fork_pages: row i of table_out (and len_out) continues row parents[i] of block_table,
    whose rows give their pages back; full pages are shared, a last one that is not full
    is copied for all rows but the first.  refs, refs_out: int32 [num_blocks], how many rows
    hold each page."""
    dev, i32 = pool.layers[0].get_device(), torch.int32
    rows, cols, rows_out = kv_len.shape[0], block_table.shape[-1], parents.shape[0]
    held = (pool.num_blocks,)
    return load().lmkv_fork_pages(
        pool.struct, _scales(pool), _whole("block_table", block_table, i32, dev, (rows, cols)), cols,
        _whole("kv_len", kv_len, i32, dev, (rows,)), rows, _whole("parents", parents, i32, dev, (rows_out,)), rows_out,
        _whole("refs", refs, i32, dev, held), _whole("table_out", table_out, i32, dev, (rows_out, cols)),
        _whole("len_out", len_out, i32, dev, (rows_out,)), _whole("refs_out", refs_out, i32, dev, held),
        _whole("workspace", workspace, torch.uint8, dev, (workspace.numel(),)), workspace.numel(), _status(status, dev),
        _stream_of(pool, dev, stream))


def resize_pages(pool, block_table, kv_len, new_len, refs, table_out, refs_out, workspace, status=None,
                 stream=None) -> int:
    """lmkv_resize_pages: rows of kv_len tokens become rows of new_len: pages behind give up a
    reference, missing ones are given.  table_out may be block_table, refs_out refs.
    A row cut back to inside a page that other rows hold keeps that page: fork_pages with
    parents 0, 1, 2, .. gives it a copy of its own, which an append to it needs."""
    dev, i32 = pool.layers[0].get_device(), torch.int32
    rows, cols = kv_len.shape[0], block_table.shape[-1]
    held = (pool.num_blocks,)
    return load().lmkv_resize_pages(
        pool.struct, _whole("block_table", block_table, i32, dev, (rows, cols)), cols,
        _whole("kv_len", kv_len, i32, dev, (rows,)), _whole("new_len", new_len, i32, dev, (rows,)), rows,
        _whole("refs", refs, i32, dev, held), _whole("table_out", table_out, i32, dev, (rows, cols)),
        _whole("refs_out", refs_out, i32, dev, held),
        _whole("workspace", workspace, torch.uint8, dev, (workspace.numel(),)), workspace.numel(), _status(status, dev),
        _stream_of(pool, dev, stream))


def compact_pages(pool, block_table, kv_len, refs, table_out, refs_out, page_map, workspace, status=None,
                  stream=None) -> int:
    """lmkv_compact_pages: the highest held pages move into the lowest free ones; page_map
    (int32 [num_blocks]) says where each page is now, and table_out, which may be
    block_table, follows it."""
    dev, i32 = pool.layers[0].get_device(), torch.int32
    rows, cols = kv_len.shape[0], block_table.shape[-1]
    held = (pool.num_blocks,)
    return load().lmkv_compact_pages(
        pool.struct, _scales(pool), _whole("block_table", block_table, i32, dev, (rows, cols)), cols,
        _whole("kv_len", kv_len, i32, dev, (rows,)), rows, _whole("refs", refs, i32, dev, held),
        _whole("table_out", table_out, i32, dev, (rows, cols)), _whole("refs_out", refs_out, i32, dev, held),
        _whole("page_map", page_map, i32, dev, held),
        _whole("workspace", workspace, torch.uint8, dev, (workspace.numel(),)), workspace.numel(), _status(status, dev),
        _stream_of(pool, dev, stream))


def check(rc: int, what: str = "lmkv") -> None:
    if rc != OK:
        raise LmkvError(rc, what)
