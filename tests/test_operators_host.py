"""Rotary set-up against its formulas, and the refusals of the attention-side
operators: argument errors are found on the host, before any CUDA call (CPU only)."""
import ctypes
import math

import numpy as np
import pytest

from paged_kv_cache_lmkv_gb300 import build, lmkv

PTR = 0x10000
ROWS = dict(data=PTR, token_stride=256, head_stride=64)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return lmkv.load()


def pool(**kw):
    a = dict(num_blocks=64, num_layers=2, num_kv_heads=2, head_dim=64, block_size=16, elem_bytes=2) | kw
    return lmkv._PoolT(0x20000, a["num_blocks"], a["num_layers"], a["num_kv_heads"], a["head_dim"],
                       a["block_size"], a["elem_bytes"])


def batch(**kw):
    a = dict(q_start=PTR, kv_len=PTR, block_table=PTR, max_blocks=8, num_req=2, num_tokens=2, max_new=1,
             max_kv_len=128) | kw
    return lmkv._BatchT(**a)


def ref(x):
    return None if x is None else ctypes.byref(x)


@pytest.mark.parametrize("kind,kw", [
    ("plain", {}), ("linear", dict(factor=4.0)), ("base", dict(factor=8.0)),
    ("bands", dict(factor=8.0, low=1.0, high=4.0, original=8192.0)),
    ("ramp", dict(factor=16.0, low=1.0, high=32.0, original=4096.0))])
@pytest.mark.parametrize("rot", [2, 64, 128, 256])
def test_rotary_frequencies(lib, kind, kw, rot):
    if kind == "base" and rot == 2:
        with pytest.raises(lmkv.LmkvError):
            lmkv.Rotary(rot, base=10000.0, scaling=kind, **kw)
        return
    got = lmkv.Rotary(rot, base=10000.0, scaling=kind, **kw)
    i = np.arange(rot // 2)
    base, fac = 10000.0, kw.get("factor", 1.0)
    if kind == "base":
        base = base * fac ** (rot / (rot - 2))
    f = base ** (-2.0 * i / rot)
    if kind == "linear":
        f = f / fac
    elif kind == "bands":
        wave = 2 * math.pi / f
        smooth = (kw["original"] / wave - kw["low"]) / (kw["high"] - kw["low"])
        f = np.where(wave < kw["original"] / kw["high"], f,
                     np.where(wave > kw["original"] / kw["low"], f / fac, (1 - smooth) * f / fac + smooth * f))
    elif kind == "ramp":
        pair = lambda turns: rot * math.log(kw["original"] / (turns * 2 * math.pi)) / (2 * math.log(base))
        mix = np.clip((i - pair(kw["high"])) / (pair(kw["low"]) - pair(kw["high"])), 0, 1)
        f = f * (1 - mix) + f / fac * mix
    np.testing.assert_allclose(got.inv_freq, f, rtol=1e-13)
    assert got.magnitude == pytest.approx(0.1 * math.log(fac) + 1 if kind == "ramp" else 1.0, rel=1e-15)
    assert got.rot_dim == rot


def test_rotary_refusals(lib):
    for bad in (dict(rot_dim=3), dict(rot_dim=0), dict(rot_dim=258), dict(base=1.0), dict(base=math.nan),
                dict(scaling="linear", factor=0.5), dict(scaling="bands", factor=2, low=4, high=4),
                dict(scaling="ramp", factor=2, low=0.0), dict(scaling="bands", original=0.0),
                dict(factor=math.inf)):
        with pytest.raises(lmkv.LmkvError) as e:
            lmkv.Rotary(**(dict(rot_dim=64) | bad))
        assert e.value.code == lmkv.ERR_INVALID_ARG
    with pytest.raises(ValueError):
        lmkv.Rotary(64, scaling="other")
    with pytest.raises(ValueError):
        lmkv.Rotary(64, inv_freq=[1.0] * 31)
    out = lmkv._RotaryT()
    assert lib.lmkv_rotary_init(ctypes.byref(out), 64, 0, 1e4, 9, 1.0, 1.0, 2.0, 1.0) == lmkv.ERR_INVALID_ARG
    assert lib.lmkv_rotary_init(None, 64, 0, 1e4, 0, 1.0, 1.0, 2.0, 1.0) == lmkv.ERR_INVALID_ARG


def append(lib, p=None, b=None, dtype=lmkv.BF16, layer=0, heads=4, rot=None, rows=("q", "k", "v", "o"), **rk):
    r = {n: lmkv._RowsT(**(ROWS | rk)) if n in rows else None for n in ("q", "k", "v", "o")}
    rot = lmkv.Rotary(64) if rot is None else rot
    return lib.lmkv_append_layer(ref(pool() if p is None else p), dtype, layer, ref(batch() if b is None else b),
                                 heads, *(ref(r[n]) for n in ("q", "k", "v", "o")), None, rot.struct, None, None)


def attend(lib, p=None, b=None, dtype=lmkv.BF16, layer=0, heads=4, prefix=PTR, prefix_len=40, scale=0.125,
           ws=PTR, ws_bytes=1 << 30, q=ROWS, out=ROWS):
    q, out = (None if x is None else lmkv._RowsT(**x) for x in (q, out))
    return lib.lmkv_attend_layer(ref(pool() if p is None else p), dtype, layer, ref(batch() if b is None else b),
                                 heads, ref(q), prefix, prefix_len, scale, ref(out), None, ws, ws_bytes, None, None)


def weigh(lib, p=None, b=None, dtype=lmkv.BF16, layer=0, heads=4, q=ROWS, lse=PTR, scale=0.125, decay=1.0,
          scores=PTR, out=PTR, stride=128):
    q = None if q is None else lmkv._RowsT(**q)
    return lib.lmkv_weigh_layer(ref(pool() if p is None else p), dtype, layer, ref(batch() if b is None else b),
                                heads, ref(q), lse, scale, decay, scores, out, stride, None, None)


def evict(lib, p=None, layer=0, table=PTR, max_blocks=8, kv_len=PTR, num_req=2, max_kv_len=128, scores=PTR + 64,
          stride=128, budget=32, sinks=4, recent=8, keep=PTR, new_len=PTR + 32, kept=None, kept_stride=0):
    return lib.lmkv_evict_layer(ref(pool() if p is None else p), layer, table, max_blocks, kv_len, num_req,
                                max_kv_len, scores, stride, budget, sinks, recent, keep, new_len, kept,
                                kept_stride, None, None)


BATCHED = [append, attend, weigh]


@pytest.mark.parametrize("call", BATCHED)
def test_batch_refusals(lib, call):
    inv = lmkv.ERR_INVALID_ARG
    before = lmkv.launch_count()
    for bad in (dict(num_req=-1), dict(num_tokens=-1), dict(max_new=-1), dict(max_kv_len=-1), dict(max_kv_len=129),
                dict(max_blocks=-1), dict(q_start=None), dict(kv_len=None), dict(block_table=None),
                dict(num_tokens=1 << 30, max_new=1)):
        assert call(lib, b=batch(**bad)) == inv, bad
    for bad in (dict(heads=0), dict(heads=3), dict(heads=-2), dict(layer=2), dict(layer=-1)):
        assert call(lib, **bad) == inv, bad
    assert call(lib, p=pool(num_layers=0)) == inv
    assert call(lib, p=pool(num_kv_heads=1, head_dim=3)) == lmkv.ERR_MISALIGNED
    for dtype in (lmkv.FP32, 3, -1):
        assert call(lib, dtype=dtype) == lmkv.ERR_UNSUPPORTED
    assert call(lib, p=pool(elem_bytes=1), dtype=lmkv.BF16) == lmkv.ERR_UNSUPPORTED
    assert call(lib, b=batch(num_req=0)) == lmkv.OK                # nothing to do
    if call is not weigh:                                          # weights still decay without new tokens
        assert call(lib, b=batch(num_tokens=0)) == lmkv.OK
    assert lmkv.launch_count() == before


def test_append_refusals(lib):
    for missing in ("q", "k", "v", "o"):
        assert append(lib, rows=[n for n in ("q", "k", "v", "o") if n != missing]) == lmkv.ERR_INVALID_ARG
    assert append(lib, data=PTR + 1) == lmkv.ERR_INVALID_ARG
    assert append(lib, data=None) == lmkv.ERR_INVALID_ARG
    assert append(lib, rot=lmkv.Rotary(66)) == lmkv.ERR_INVALID_ARG     # more than head_dim
    assert append(lib, rot=lmkv.Rotary(64, inv_freq=[math.nan] * 32)) == lmkv.ERR_INVALID_ARG
    assert append(lib, rot=lmkv.Rotary(64, magnitude=math.inf)) == lmkv.ERR_INVALID_ARG


def test_attend_refusals(lib):
    inv = lmkv.ERR_INVALID_ARG
    assert attend(lib, p=pool(head_dim=96)) == lmkv.ERR_UNSUPPORTED
    assert attend(lib, p=pool(elem_bytes=4), dtype=lmkv.FP32) == lmkv.ERR_UNSUPPORTED
    for bad in (dict(prefix_len=-1), dict(prefix=None), dict(scale=math.nan), dict(scale=math.inf), dict(ws=None),
                dict(ws_bytes=16), dict(q=None), dict(out=None), dict(q=ROWS | dict(data=PTR + 1)),
                dict(prefix_len=2 ** 31)):
        assert attend(lib, **bad) == inv, bad
    assert attend(lib, ws=PTR + 8) == lmkv.ERR_MISALIGNED
    out = ctypes.c_uint64(0)
    size = lambda *a: lib.lmkv_attend_workspace_bytes(ctypes.byref(pool()), *a, ctypes.byref(out))
    assert size(4, 2, 2, 1, 40, 128) == lmkv.OK and out.value > 0
    assert size(4, 0, 2, 1, 40, 128) == lmkv.OK and out.value == 0
    for bad in ((3, 2, 2, 1, 40, 128), (4, -1, 2, 1, 40, 128), (4, 2, -2, 1, 40, 128), (4, 2, 2, -1, 40, 128),
                (4, 2, 2, 1, -40, 128), (4, 2, 2, 1, 40, -1)):
        assert size(*bad) == inv, bad


def test_weigh_refusals(lib):
    inv = lmkv.ERR_INVALID_ARG
    for bad in (dict(q=None), dict(lse=None), dict(scores=None), dict(out=None), dict(stride=127),
                dict(scale=math.nan), dict(decay=math.nan), dict(decay=math.inf)):
        assert weigh(lib, **bad) == inv, bad
    assert weigh(lib, p=pool(head_dim=96)) == lmkv.ERR_UNSUPPORTED


def test_evict_refusals(lib):
    inv = lmkv.ERR_INVALID_ARG
    before = lmkv.launch_count()
    for bad in (dict(layer=2), dict(layer=-1), dict(num_req=-1), dict(max_kv_len=-1), dict(max_kv_len=129),
                dict(stride=127), dict(budget=0), dict(sinks=-1), dict(recent=-1), dict(sinks=20, recent=13),
                dict(kv_len=None), dict(keep=None), dict(new_len=None), dict(new_len=PTR), dict(scores=None),
                dict(table=None), dict(kept=PTR, kept_stride=31), dict(kept=PTR + 64, kept_stride=32)):
        assert evict(lib, **bad) == inv, bad
    assert evict(lib, p=pool(num_kv_heads=1, head_dim=3)) == lmkv.ERR_MISALIGNED
    assert evict(lib, p=pool(num_blocks=2 ** 28)) == inv         # token slots are numbered with 32 bits
    assert evict(lib, num_req=0) == lmkv.OK
    assert lmkv.launch_count() == before


def test_refusals_of_scales_and_shared_rows(lib):
    before = lmkv.launch_count()
    for scale in (3e38, -3e38):                     # not finite once log2(e) is folded in
        assert attend(lib, scale=scale, out=ROWS | dict(data=PTR + 4096)) == lmkv.ERR_INVALID_ARG
        assert weigh(lib, scale=scale) == lmkv.ERR_INVALID_ARG
    assert attend(lib) == lmkv.ERR_INVALID_ARG      # out is q
    assert lmkv.launch_count() == before


def shifted(lib, p=None, dtype=lmkv.BF16, shift=(5,), rot=None, layer=None, start=(0,), end=(300,), chunk=256):
    s, e = np.array(start, np.int64), np.array(end, np.int64)
    sh = None if shift is None else np.array(shift, np.int64)
    rot = lmkv.Rotary(64) if rot is None else rot
    a = [ref(pool() if p is None else p), dtype, PTR, 64, s.ctypes.data, e.ctypes.data, len(s), chunk, 1, 0x30000,
         None if sh is None else sh.ctypes.data, rot.struct]
    if layer is None:
        return lib.lmkv_scatter_chunks_shifted(*a, None, None)
    return lib.lmkv_scatter_layer_shifted(*a, layer, None, None)


def test_shifted_refusals(lib):
    before = lmkv.launch_count()
    for kw in ({}, dict(layer=0)):
        assert shifted(lib, shift=None, **kw) == lmkv.ERR_INVALID_ARG
        assert shifted(lib, rot=lmkv.Rotary(66), **kw) == lmkv.ERR_INVALID_ARG
        assert shifted(lib, start=(17,), **kw) == lmkv.ERR_INVALID_ARG
        assert shifted(lib, chunk=24, **kw) == lmkv.ERR_INVALID_ARG
        assert shifted(lib, end=(4096,), **kw) == lmkv.ERR_INVALID_ARG
        assert shifted(lib, p=pool(elem_bytes=1), **kw) == lmkv.ERR_UNSUPPORTED
        assert shifted(lib, dtype=lmkv.FP32, **kw) == lmkv.ERR_UNSUPPORTED
        assert shifted(lib, start=(0,), end=(0,), **kw) == lmkv.OK
    assert shifted(lib, layer=2) == lmkv.ERR_INVALID_ARG
    assert shifted(lib, layer=-1) == lmkv.ERR_INVALID_ARG
    assert lmkv.launch_count() == before


def test_binding_refusals(lib):
    """The Python calls check shapes, types, devices and strides before the library is called."""
    import torch
    layers = [torch.zeros((2, 8, 16, 128), dtype=torch.bfloat16) for _ in range(2)]
    p = lmkv.Pool.__new__(lmkv.Pool)
    p.layers, p.num_kv_heads, p.head_dim, p.block_size, p.num_blocks, p.elem_bytes = layers, 2, 64, 16, 8, 2
    p._struct = pool(num_blocks=8)
    table = torch.zeros((2, 4), dtype=torch.int32)
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    kv = torch.zeros((2, 2, 64), dtype=torch.bfloat16)
    qs, ln = torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    ws, lse = torch.zeros(1 << 20, dtype=torch.uint8), torch.zeros((2, 4))
    sc = torch.zeros((2, 2, 64))
    rot = lmkv.Rotary(64)

    def bad(fn, *a, **k):
        with pytest.raises(ValueError):
            fn(*a, **k)

    def app(table=table, q=q, k=kv, v=kv, o=q, qs=qs, ln=ln, **kw):
        return lmkv.append_layer(p, 0, table, q, k, v, o, qs, ln, rot, **kw)
    for kw in (dict(q=q.float()), dict(k=q), dict(v=kv[:1]), dict(o=q[:, :, ::2]), dict(qs=qs.long()), dict(qs=qs[:2]),
               dict(table=table.long()), dict(table=table[:1]), dict(positions=torch.zeros(2, dtype=torch.int32)),
               dict(positions=torch.zeros(3, dtype=torch.int64)), dict(q=torch.zeros((2, 4, 128))[:, :, ::2])):
        bad(app, **kw)

    def att(q=q, o=q, lse=lse, prefix=table[0], n=40, table=table):
        return lmkv.attend_layer(p, 0, q, o, qs, ln, table, 0.1, ws, prefix_table=prefix, prefix_len=n, lse=lse)
    for kw in (dict(n=65), dict(prefix=None), dict(prefix=table[0].long()), dict(lse=lse.double()),
               dict(lse=lse[:, :3]), dict(o=q[:1]), dict(q=q[0])):
        bad(att, **kw)

    def wei(q=q, lse=lse, a=sc, b=sc):
        return lmkv.weigh_layer(p, 0, q, lse, qs, ln, table, 0.1, a, b)
    for kw in (dict(lse=lse[:1]), dict(a=sc[:, :, :32]), dict(b=sc.double()), dict(b=sc[:1]), dict(a=sc[:, :1])):
        bad(wei, **kw)

    def evi(s=sc, keep=torch.zeros((2, 2, 8), dtype=torch.int32), nl=ln.clone(), kept=None, table=table):
        return lmkv.evict_layer(p, 0, table, ln, s, 1, 1, keep, nl, kept_scores=kept)
    for kw in (dict(s=sc.double()), dict(s=sc[:1]), dict(keep=torch.zeros((2, 2, 8))), dict(nl=ln.long()),
               dict(kept=sc[:, :, :4]), dict(table=table[:1])):
        bad(evi, **kw)
    bad(lmkv.scatter_chunks_shifted, p, table, [0, 0], [64, 64], 64, True, ws, [1], rot)
    p.layers = [x.to(torch.uint8) for x in layers]
    bad(app)


def test_binding_refuses_shifted_tables(lib):
    import torch
    p = lmkv.Pool.__new__(lmkv.Pool)
    p.layers = [torch.zeros((2, 8, 16, 128), dtype=torch.bfloat16)]
    p.num_kv_heads, p.head_dim, p.block_size, p.num_blocks, p.elem_bytes = 2, 64, 16, 8, 2
    p._struct = pool(num_blocks=8, num_layers=1)
    table, ptrs = torch.zeros((2, 8), dtype=torch.int32), torch.zeros(2, dtype=torch.int64)
    for t in (table[:1], table[:, ::2], table[0], table.long()):
        for fn, more in ((lmkv.scatter_chunks_shifted, ()), (lmkv.scatter_layer_shifted, (0,))):
            with pytest.raises(ValueError):
                fn(p, t, [0, 0], [64, 64], 64, True, ptrs, [1, 1], lmkv.Rotary(64), *more)
