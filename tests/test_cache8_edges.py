"""The 8-bit cache's operators and pages at the ends of their ranges: what is found on the host,
before any CUDA call (CPU only)."""
import ctypes

import pytest

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
