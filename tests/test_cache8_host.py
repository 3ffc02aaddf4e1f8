"""Refusals of the 8-bit cache's operators: argument errors are found on the host, before any
CUDA call (CPU only)."""
import ctypes
import math

import pytest

from paged_kv_cache_lmkv_gb300 import build, lmkv

PTR = 0x10000
ROWS = dict(data=PTR, token_stride=256, head_stride=64)
INV, MIS, UNS = lmkv.ERR_INVALID_ARG, lmkv.ERR_MISALIGNED, lmkv.ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build.build()
    return lmkv.load()


def pool(**kw):
    a = dict(num_blocks=64, num_layers=2, num_kv_heads=2, head_dim=64, block_size=16, elem_bytes=1) | kw
    return lmkv._PoolT(0x20000, a["num_blocks"], a["num_layers"], a["num_kv_heads"], a["head_dim"], a["block_size"],
                       a["elem_bytes"])


def batch(**kw):
    a = dict(q_start=PTR, kv_len=PTR, block_table=PTR, max_blocks=8, num_req=2, num_tokens=2, max_new=1,
             max_kv_len=128) | kw
    return lmkv._BatchT(**a)


def ref(x):
    return None if x is None else ctypes.byref(x)


def append(lib, p=None, b=None, scales=PTR, dtype=lmkv.BF16, layer=0, heads=4, missing=None, data=PTR, rot=None,
           qn=None, kn=None, eps=1e-6):
    rows = [ref(None if n == missing else lmkv._RowsT(**(ROWS | dict(data=data)))) for n in "qkvo"]
    return lib.lmkv_append_layer_normed(ref(p or pool()), scales, dtype, layer, ref(b or batch()), heads, *rows, None,
                                        None if rot is None else rot.struct, qn, kn, eps, None, None)


def attend(lib, p=None, b=None, scales=PTR, dtype=lmkv.BF16, layer=0, heads=4, q=ROWS, out=ROWS | dict(data=PTR * 2),
           scale=0.125, window=0, sinks=0, ws=PTR, ws_bytes=1 << 40):
    r = lambda x: None if x is None else ctypes.byref(lmkv._RowsT(**x))
    return lib.lmkv_attend_layer_window(ref(p or pool()), scales, dtype, layer, ref(b or batch()), heads, r(q), scale,
                                        window, sinks, r(out), None, ws, ws_bytes, None, None)


@pytest.mark.parametrize("call", [append, attend])
def test_batch_refusals(lib, call):
    before = lmkv.launch_count()
    for bad in (dict(num_req=-1), dict(num_tokens=-1), dict(max_new=-1), dict(max_kv_len=-1), dict(max_kv_len=129),
                dict(max_blocks=-1), dict(q_start=None), dict(kv_len=None), dict(block_table=None),
                dict(num_tokens=1 << 30, max_new=1)):
        assert call(lib, b=batch(**bad)) == INV, bad
    for bad in (dict(heads=0), dict(heads=3), dict(heads=-2), dict(layer=2), dict(layer=-1)):
        assert call(lib, **bad) == INV, bad
    assert call(lib, p=pool(num_layers=0)) == INV
    for dtype in (lmkv.FP32, 3, -1):
        assert call(lib, dtype=dtype) == UNS
    assert call(lib, p=pool(elem_bytes=4)) == UNS
    assert call(lib, p=pool(head_dim=96)) == UNS
    assert call(lib, scales=None) == INV                               # an 8-bit pool without scales
    assert call(lib, p=pool(elem_bytes=2)) == INV                      # a 16-bit pool with scales
    assert call(lib, b=batch(num_req=0)) == lmkv.OK                    # nothing to do
    assert call(lib, b=batch(num_tokens=0)) == lmkv.OK
    assert call(lib, p=pool(elem_bytes=2), scales=None, b=batch(num_tokens=0)) == lmkv.OK
    assert lmkv.launch_count() == before


def test_append_refusals(lib):
    for missing in "qkvo":
        assert append(lib, missing=missing) == INV
    assert append(lib, data=PTR + 1) == INV
    assert append(lib, data=None) == INV
    for eps in (-1e-6, math.nan, math.inf):
        assert append(lib, eps=eps) == INV
    assert append(lib, qn=PTR + 4) == MIS and append(lib, kn=PTR + 8) == MIS
    assert append(lib, rot=lmkv.Rotary(66)) == INV
    assert append(lib, rot=lmkv.Rotary(64, inv_freq=[math.nan] * 32)) == INV


def test_attend_refusals(lib):
    for bad in (dict(scale=math.nan), dict(scale=math.inf), dict(ws=None), dict(ws_bytes=16), dict(q=None),
                dict(out=None), dict(q=ROWS | dict(data=PTR + 1)), dict(window=-1), dict(sinks=-1), dict(out=ROWS)):
        assert attend(lib, **bad) == INV, bad
    assert attend(lib, ws=PTR + 8) == MIS


def test_attend_workspace(lib):
    out = ctypes.c_uint64(0)
    size = lambda *a, p=None: lib.lmkv_attend_window_workspace_bytes(ref(p or pool()), *a, ctypes.byref(out))
    assert size(4, 2, 2, 1, 128) == lmkv.OK and out.value > 0
    assert size(4, 0, 2, 1, 128) == lmkv.OK and out.value == 0
    for bad in ((0, 2, 2, 1, 128), (3, 2, 2, 1, 128), (4, -1, 2, 1, 128), (4, 2, -1, 1, 128), (4, 2, 2, -1, 128),
                (4, 2, 2, 1, -1), (4, 1 << 29, 2, 1, 128)):
        assert size(*bad) == INV, bad
    assert size(4, 2, 2, 1, 128, p=pool(elem_bytes=4)) == UNS
    assert lib.lmkv_attend_window_workspace_bytes(ref(pool()), 4, 2, 2, 1, 128, None) == INV


@pytest.mark.parametrize("elem", [1, 2])
@pytest.mark.parametrize("kv_heads,dim,page", [(1, 64, 16), (2, 128, 16), (8, 128, 64), (3, 64, 8)])
def test_attend_workspace_covers_smaller_calls(lib, elem, kv_heads, dim, page):
    """What a call of its own bounds needs is at most what larger bounds say: calls with that much are not refused for
    it (they are refused for their out, which is q, behind the check of the workspace)."""
    p = pool(elem_bytes=elem, num_kv_heads=kv_heads, head_dim=dim, block_size=page)
    out = ctypes.c_uint64(0)
    size = lambda *a: (lib.lmkv_attend_window_workspace_bytes(ref(p), *a, ctypes.byref(out)), out.value)[1]

    def need(heads, tokens, req, new, length):
        lo, hi = 0, 1 << 40
        b = batch(num_tokens=tokens, num_req=req, max_new=new, max_kv_len=length, max_blocks=-(-length // page))
        # out is misaligned by design of the probe: rows pass, the workspace is looked at before its alignment
        bad = lambda n: attend(lib, p=p, b=b, scales=PTR if elem == 1 else None, heads=heads, ws=PTR + 8, ws_bytes=n) == INV
        while lo < hi:
            mid = (lo + hi) // 2
            lo, hi = (mid + 1, hi) if bad(mid) else (lo, mid)
        return lo
    for group in (1, 5, 8):
        heads = kv_heads * group
        for big in ((700, 9, 300, 5000), (64, 64, 1, 9000), (40, 3, 40, 70), (8, 8, 1, 10)):
            most = size(heads, *big)
            for cut in ((1, 1, 1, 1), big, (big[0] // 2, 1, big[2], big[3]), (big[0], big[1], 1, big[3]),
                        (min(big[0], 16), 2, min(big[2], 8), big[3] // 3), (big[0], 1, big[2], big[3])):
                cut = tuple(max(1, c) for c in cut)
                assert need(heads, *cut) <= most, (group, big, cut)


def pages(lib, which, p=None, scales=PTR, table=PTR, cols=4, kv_len=PTR, rows=3, extra=PTR, refs=PTR, table_out=PTR * 3,
          refs_out=PTR, ws=PTR, ws_bytes=1 << 30, rows_out=3, len_out=PTR * 4):
    a = (ref(p or pool()),)
    if which == "fork":
        return lib.lmkv_fork_pages(*a, scales, table, cols, kv_len, rows, extra, rows_out, refs, table_out, len_out, refs_out,
                                   ws, ws_bytes, None, None)
    if which == "resize":
        return lib.lmkv_resize_pages(*a, table, cols, kv_len, extra, rows, refs, table_out, refs_out, ws, ws_bytes, None, None)
    return lib.lmkv_compact_pages(*a, scales, table, cols, kv_len, rows, refs, table_out, refs_out, extra, ws, ws_bytes, None, None)


@pytest.mark.parametrize("which", ["fork", "resize", "compact"])
def test_pages_refusals(lib, which):
    before = lmkv.launch_count()
    for bad in (dict(rows=-1), dict(cols=-1), dict(rows=1 << 25), dict(table=None), dict(kv_len=None), dict(extra=None),
                dict(refs=None), dict(refs_out=None), dict(table_out=None), dict(ws=None), dict(ws_bytes=64),
                dict(cols=1 << 30), dict(p=pool(num_layers=0))):
        assert pages(lib, which, **bad) == INV, bad
    for bad in (dict(refs=PTR + 4), dict(refs_out=PTR + 8), dict(ws=PTR + 8)):
        assert pages(lib, which, **bad) == MIS, bad
    assert pages(lib, which, p=pool(num_blocks=2 ** 31 - 1)) == UNS
    if which != "resize":
        assert pages(lib, which, p=pool(elem_bytes=2)) == INV            # scales of a 16-bit pool
    if which == "fork":
        assert pages(lib, which, table_out=PTR) == INV                   # rows of it may still be read
        assert pages(lib, which, len_out=PTR) == INV and pages(lib, which, len_out=None) == INV
        assert pages(lib, which, rows_out=-1) == INV
    assert lmkv.launch_count() == before


def test_pages_workspace_and_copy_refusals(lib):
    out = ctypes.c_uint64(0)
    assert lib.lmkv_pages_workspace_bytes(ref(pool()), 5, ctypes.byref(out)) == lmkv.OK and out.value > 0
    small = out.value
    assert lib.lmkv_pages_workspace_bytes(ref(pool()), 5000, ctypes.byref(out)) == lmkv.OK and out.value > small
    for rows in (-1, (1 << 24) + 1):
        assert lib.lmkv_pages_workspace_bytes(ref(pool()), rows, ctypes.byref(out)) == INV
    assert lib.lmkv_pages_workspace_bytes(ref(pool()), 5, None) == INV
    copy = lambda p=None, scales=PTR, src=PTR, dst=PTR, n=3: lib.lmkv_copy_pages(ref(p or pool()), scales, src, dst, n, None, None)
    assert copy(n=-1) == INV and copy(src=None) == INV and copy(dst=None) == INV
    assert copy(p=pool(elem_bytes=2)) == INV and copy(p=pool(num_layers=0)) == INV
    assert copy(n=0, src=None, dst=None) == lmkv.OK
    assert lmkv.status_string(lmkv.ERR_NO_PAGES) != "unknown status"
