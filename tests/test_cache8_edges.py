"""The 8-bit cache's operators and pages at the ends of their ranges: what is found on the host,
before any CUDA call (CPU only)."""
import ctypes

import numpy as np
import pytest
import torch

from paged_kv_cache_lmkv_gb300 import build, lmkv

PTR = 0x10000
INV, UNS = lmkv.ERR_INVALID_ARG, lmkv.ERR_UNSUPPORTED
STEP = 8 * 1024                      # threads that go through the pages together, each by this many at a time
MOST = 2 ** 31 - 1 - STEP


@pytest.fixture(scope="module")
def lib():
    build.build()
    return lmkv.load()


def pages(lib, which, num_blocks=64, rows=1, cols=4, ws_bytes=64):
    """One of the calls, with too little workspace to go on."""
    p = ctypes.byref(lmkv._PoolT(0x20000, num_blocks, 2, 2, 64, 16, 1))
    if which == "fork":
        return lib.lmkv_fork_pages(p, PTR, PTR, cols, PTR, rows, PTR, rows, PTR, PTR * 3, PTR * 4, PTR, PTR, ws_bytes, None, None)
    if which == "resize":
        return lib.lmkv_resize_pages(p, PTR, cols, PTR, PTR, rows, PTR, PTR * 3, PTR, PTR, ws_bytes, None, None)
    return lib.lmkv_compact_pages(p, PTR, PTR, cols, PTR, rows, PTR, PTR * 3, PTR, PTR, PTR, ws_bytes, None, None)


@pytest.mark.parametrize("which", ["fork", "resize", "compact"])
def test_pages_that_a_counter_of_32_bits_would_step_past(lib, which):
    """A thread's counter of pages passes the last one by less than STEP, and has to hold that."""
    before = lmkv.launch_count()
    out = ctypes.c_uint64(0)
    size = lambda n: lib.lmkv_pages_workspace_bytes(ctypes.byref(lmkv._PoolT(0x20000, n, 2, 2, 64, 16, 1)), 5, ctypes.byref(out))
    for n in (MOST + 1, 2 ** 31 - 1 - 4096, 2 ** 31 - 1):
        assert pages(lib, which, num_blocks=n) == UNS and size(n) == UNS
    assert size(MOST) == lmkv.OK and out.value > 24 * MOST
    assert pages(lib, which, num_blocks=MOST) == INV                 # (the workspace)
    assert lmkv.launch_count() == before


@pytest.mark.parametrize("which", ["fork", "resize", "compact"])
def test_tables_whose_columns_a_counter_of_32_bits_would_step_past(lib, which):
    """A lane's counter of columns passes the last one by up to 31 (128 where four steps are taken at once)."""
    before = lmkv.launch_count()
    for rows, cols in ((1, 2 ** 31 - 1), (1, 2 ** 31 - 128), (1, MOST + 1), (2, MOST // 2 + 1)):
        assert pages(lib, which, rows=rows, cols=cols, ws_bytes=1 << 30) == INV, (rows, cols)
    assert lmkv.launch_count() == before


def movement_calls():
    """The calls that take rows out of pages or into them, on requests of no tokens."""
    table = torch.zeros((1, 4), dtype=torch.int32)
    a = (table, np.array([0]), np.array([16]), 16, True)
    chunks, staging = torch.zeros(1, dtype=torch.int64), torch.zeros(64, dtype=torch.uint8)
    host, bins, sizes = [staging], np.full((2, 2), 16, np.int32), torch.zeros(1, dtype=torch.int64)
    some = dict(stream=0)
    two = dict(stream=0, copy_stream=0)
    return {
        "gather_chunks": lambda p: lmkv.gather_chunks(p, *a, chunks, **some),
        "scatter_chunks": lambda p: lmkv.scatter_chunks(p, *a, chunks, **some),
        "gather_layer": lambda p: lmkv.gather_layer(p, *a, chunks, 0, **some),
        "scatter_layer": lambda p: lmkv.scatter_layer(p, *a, chunks, 0, **some),
        "gather_chunks_fp8e4m3": lambda p: lmkv.gather_chunks_fp8e4m3(p, *a, chunks, chunks, **some),
        "scatter_chunks_fp8e4m3": lambda p: lmkv.scatter_chunks_fp8e4m3(p, *a, chunks, chunks, **some),
        "store_layers": lambda p: lmkv.store_layers(p, *a, chunks, 0, 2, **some),
        "retrieve_layers": lambda p: lmkv.retrieve_layers(p, *a, chunks, 0, 2, **some),
        "store_layers_staged": lambda p: lmkv.store_layers_staged(p, *a, host, staging, 0, 2, **some),
        "retrieve_layers_staged": lambda p: lmkv.retrieve_layers_staged(p, *a, host, staging, 0, 2, **some),
        "store_layers_staged_noalloc": lambda p: lmkv.store_layers_staged_noalloc(p, *a, host, 0, 2, **some),
        "store_layers_overlapped": lambda p: lmkv.store_layers_overlapped(p, *a, host, staging, 0, 2, None, **two),
        "retrieve_layers_overlapped": lambda p: lmkv.retrieve_layers_overlapped(p, *a, host, staging, 0, 2, None, **two),
        "cachegen_store_chunks": lambda p: lmkv.cachegen_store_chunks(p, *a, bins, chunks, sizes, staging, **some),
        "cachegen_retrieve_chunks": lambda p: lmkv.cachegen_retrieve_chunks(p, *a, bins, chunks, sizes, staging, **some),
    }


@pytest.mark.parametrize("name", list(movement_calls()))
@pytest.mark.parametrize("scales", [False, True])
def test_rows_of_a_pool_with_scales_do_not_move_without_them(lib, name, scales):
    """The calls that move chunks know of no scales: codes in another page's scale are other values.  A Pool of the same
    layers without scales is taken as bytes, as before (here its layers are null, which the library says)."""
    pool = lmkv.Pool.__new__(lmkv.Pool)
    pool.num_kv_heads, pool.head_dim, pool.elem_bytes, pool.block_size, pool.num_blocks = 2, 64, 1, 16, 4
    pool._struct = lmkv._PoolT(None, 4, 2, 2, 64, 16, 1)
    call = movement_calls()[name]
    if not scales:
        assert call(pool) == INV
        return
    pool.scales = [None, None]
    with pytest.raises(ValueError, match="scale"):
        call(pool)


@pytest.mark.parametrize("name,value", [("window", 2 ** 32 + 5), ("sinks", 2 ** 32 + 1), ("window", 2 ** 31), ("sinks", 2 ** 40)])
def test_windows_and_sinks_beyond_32_bits_are_all_keys(monkeypatch, name, value):
    """Not what is left of them in 32 bits, which would be another window; below zero they are refused all the same."""
    seen = {}

    class Library:
        def lmkv_attend_layer_window(self, pool, scales, code, layer, batch, heads, q, scale, window, sinks, *rest):
            seen.update(window=window, sinks=sinks)
            return lmkv.OK
    monkeypatch.setattr(lmkv, "load", lambda: Library())
    monkeypatch.setattr(lmkv, "_stream_of", lambda *a: 0)
    pool = lmkv.Pool.__new__(lmkv.Pool)
    pool.layers, pool.num_kv_heads, pool.head_dim, pool.block_size = [torch.zeros((2, 4, 16, 128), dtype=torch.float16)], 2, 64, 16
    pool._struct = lmkv._PoolT(None, 4, 1, 2, 64, 16, 2)
    q, i32 = torch.zeros((1, 2, 64), dtype=torch.float16), torch.int32
    call = lambda **kw: lmkv.attend_layer_window(
        pool, 0, q, torch.zeros_like(q), torch.tensor([0, 1], dtype=i32), torch.tensor([3], dtype=i32),
        torch.zeros((1, 4), dtype=i32), 0.125, torch.zeros(64, dtype=torch.uint8), **kw)
    assert call(**{name: value}) == lmkv.OK and seen[name] == 2 ** 31 - 1
    assert call(**{name: 7}) == lmkv.OK and seen[name] == 7
    call(**{name: -2 ** 40})
    assert -2 ** 31 <= seen[name] < 0
