"""The attention-side operators against 64-bit formulas: rotary append, shifted
retrieve, shared-prefix attention, attention weights, eviction, and a decode
step of them together (eager, captured and replayed)."""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import paged_kv_cache_lmkv_gb300 as pkg
from paged_kv_cache_lmkv_gb300 import lmkv
from gpu_util import require_gpu
from operator_util import DEV, HALF_STEP, TINY, Batch, rotate64, within

pytestmark = pytest.mark.gpu
BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(autouse=True)
def gpu():
    require_gpu()


# ---- rotary append ------------------------------------------------------

def append_case(new, kv, heads, kv_heads, dim, dtype, rot, interleaved=False, page=16, positions=None, offset=0,
                in_place=False, magnitude=1.0, extra=0, seed=0):
    b = Batch(new, kv, heads, kv_heads, dim, dtype, page=page, seed=seed, extra_rows=extra)
    g = torch.Generator().manual_seed(seed + 1)
    t, width = b.tokens, heads + 2 * kv_heads
    # q, k and v of one projection, `offset` elements into their storage
    store = torch.randn(t * width * dim + offset, generator=g).to(dtype)
    qkv_cpu = store[offset:].view(t, width, dim)
    store_d = store.to(DEV)
    qkv = store_d[offset:].view(t, width, dim)
    q, k, v = qkv[:, :heads], qkv[:, heads:heads + kv_heads], qkv[:, heads + kv_heads:]
    q_out = q if in_place else torch.full((t, heads, dim), 7.0, dtype=dtype, device=DEV)
    before = q_out.clone().cpu()
    index = torch.cat([torch.arange(m - n, m) for n, m in zip(new, kv)] + [torch.zeros(extra, dtype=torch.long)])
    pos = index if positions is None else torch.tensor(positions, dtype=torch.int64)
    rotary = pkg.Rotary(rot, base=10000.0, interleaved=interleaved, magnitude=magnitude)
    pkg.check(pkg.append_layer(b.pool, b.layer, b.table_d, q, k, v, q_out, b.q_start_d, b.kv_len_d, rotary,
                               positions=None if positions is None else pos.to(DEV), status=b.status))
    torch.cuda.synchronize()
    assert b.status.item() == 0
    live = int(b.q_start[-1])
    step, tiny = HALF_STEP[dtype], TINY[dtype]

    def near(got, x, what):
        want, mag = rotate64(x.double(), pos[:live], rotary.inv_freq, interleaved, magnitude)
        # fp32: cos and sin within 2^-22 (their rounding and that of the fraction of a turn), two products and a
        # sum; the frequency's own rounding is 2^-53 of its angle
        angle = pos[:live].abs().max().item() * 2.0 ** -51 if live else 0.0
        tol = step * 1.001 * want.abs() + (2.0 ** -21 + angle) * mag + tiny
        rest = slice(rot, None)
        tol[..., rest] = 0
        within(got, want, tol, what)

    near(q_out[:live], qkv_cpu[:live, :heads], "q")
    assert torch.equal(q_out[live:].cpu(), before[live:])
    want_pool = b.pool_cpu.clone()
    flat = b.pool.layers[b.layer].cpu().view(2, -1, kv_heads, dim)
    where = torch.cat([b.slots(r)[m - n:] for r, (n, m) in enumerate(zip(new, kv))])
    near(flat[0][where], qkv_cpu[:live, heads:heads + kv_heads], "k")
    want = want_pool[b.layer].view(2, -1, kv_heads, dim)
    want[1, where] = qkv_cpu[:live, heads + kv_heads:]
    want[0, where] = flat[0][where]
    for i, l in enumerate(b.pool.layers):       # every other slot, layer and row as it was
        assert torch.equal(l.cpu().view(torch.uint8), want_pool[i].view(torch.uint8))


@pytest.mark.parametrize("dtype", [BF, FP, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [64, 32, 2, 34])
def test_append_types_and_layouts(dtype, interleaved, rot):
    append_case([1, 3, 0, 17], [5, 3, 9, 50], 6, 2, 64, dtype, rot, interleaved, extra=3)


@pytest.mark.parametrize("page", [1, 5, 16, 24, 64])
def test_append_pages_and_long(page):
    append_case([400, 1, 33], [431, 70, 33], 8, 8, 128, BF, 128, page=page, magnitude=1.25)


@pytest.mark.parametrize("offset", [0, 1, 4])
@pytest.mark.parametrize("in_place", [False, True])
def test_append_alignment_and_in_place(offset, in_place):
    append_case([2, 5], [8, 5], 4, 2, 64, BF, 64, offset=offset, in_place=in_place)


def test_append_odd_head_dims():
    append_case([2, 5], [8, 5], 4, 4, 20, BF, 10)
    append_case([2, 5], [8, 5], 4, 4, 20, FP, 20, interleaved=True)
    append_case([1, 2], [1, 2], 3, 1, 256, F32, 256)


@pytest.mark.parametrize("dtype,rot,interleaved", [(BF, 64, True), (F32, 2, True), (FP, 64, False)])
def test_append_head_dim_of_no_multiple_of_two(dtype, rot, interleaved):
    append_case([2, 5], [8, 5], 16, 16, 65, dtype, rot, interleaved)


def test_append_far_positions():
    p = [0, 1, -1, 131071, 2 ** 20 + 1, -(2 ** 24) - 3, 2 ** 31 + 5, 123456789]
    append_case([8], [8], 4, 2, 64, F32, 64, positions=p)
    append_case([8], [8], 4, 2, 64, BF, 64, positions=p, interleaved=True)


def test_append_many_requests():
    new = [(i * 7) % 3 for i in range(1100)]
    append_case(new, [n + (i % 5) for i, n in enumerate(new)], 2, 1, 64, BF, 64)


def test_append_bad_blocks_and_lengths():
    b = Batch([2, 2], [20, 6], 4, 2, 64, BF)
    g = torch.Generator().manual_seed(1)
    qkv = torch.randn((4, 8, 64), generator=g).to(BF).to(DEV)
    q, k, v = qkv[:, :4], qkv[:, 4:6], qkv[:, 6:]
    rot = pkg.Rotary(64)

    def go(table, kv_len):
        out = torch.full_like(q, 7.0)
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        pkg.check(pkg.append_layer(b.pool, 1, table, q, k, v, out, b.q_start_d, kv_len, rot, status=st))
        torch.cuda.synchronize()
        assert not bool((out == 7.0).all(-1).any())
        return st.item()
    before = b.pool.layers[1][:, b.table[0, 1].item()].clone()
    for bad in (-1, b.num_blocks, 2 ** 31 - 1, -2 ** 31):
        t = b.table_d.clone()
        t[0, 1] = bad
        assert go(t, b.kv_len_d) == lmkv.ERR_BAD_BLOCK
        now = b.pool.layers[1][:, b.table[0, 1].item()]
        assert torch.equal(now.view(torch.int16), before.view(torch.int16))
    for bad in ([1, 6], [20, 10 ** 6], [20, -5]):
        assert go(b.table_d, torch.tensor(bad, dtype=torch.int32, device=DEV)) == lmkv.ERR_BAD_LENGTH


# ---- shifted retrieve ---------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, FP, F32])
@pytest.mark.parametrize("interleaved,rot,heads,dim,page", [
    (False, 64, 2, 64, 16), (True, 64, 2, 64, 16), (False, 32, 2, 64, 16), (False, 128, 8, 128, 16),
    (False, 6, 4, 20, 16), (True, 10, 4, 20, 8), (False, 128, 8, 128, 64), (False, 64, 1, 64, 1)])
def test_shifted_scatter(dtype, interleaved, rot, heads, dim, page):
    ends, shifts = [300, 0, 37, 256], [1000, 5, -131072, 0]
    layers = 3
    b = Batch([0] * 4, ends, heads, heads, dim, dtype, page=page, layers=layers)
    chunk = 128
    chunks = pkg.enumerate_chunks([0] * 4, ends, chunk, True)
    g = torch.Generator().manual_seed(5)
    bufs = [torch.randn((2, layers, n, heads * dim), generator=g).to(dtype) for _, _, n in chunks]
    bufs_d = [x.to(DEV) for x in bufs]
    ptrs = pkg.pointer_array(bufs_d, DEV)
    rotary = pkg.Rotary(rot, interleaved=interleaved, magnitude=1.5)       # the magnitude is not applied again
    step, tiny = HALF_STEP[dtype], TINY[dtype]
    a = (b.pool, b.table_d, [0] * 4, ends, chunk, True, ptrs, shifts, rotary)
    start = [l.clone() for l in b.pool.layers]

    def look(done):
        torch.cuda.synchronize()
        assert b.status.item() == 0
        for l in range(layers):
            if l not in done:
                assert torch.equal(b.pool.layers[l].view(torch.uint8), start[l].view(torch.uint8))
                continue
            flat = b.pool.layers[l].cpu().view(2, -1, heads, dim)
            rest = start[l].cpu().view(2, -1, heads, dim).clone()
            for (r, t0, n), x in zip(chunks, bufs):
                at = b.slots(r)[t0:t0 + n]
                want, mag = rotate64(x[0, l].view(n, heads, dim).double(), torch.full((n,), shifts[r]),
                                     rotary.inv_freq, interleaved)
                tol = step * 1.001 * want.abs() + 2.0 ** -21 * mag + tiny
                tol[..., rot:] = 0
                if shifts[r] == 0:
                    tol[:] = 0
                within(flat[0][at], want, tol, f"layer {l} chunk of {r}")
                assert torch.equal(flat[1][at].flatten(1), x[1, l])
                rest[:, at] = flat[:, at]
            assert torch.equal(flat.view(torch.uint8), rest.view(torch.uint8))

    pkg.check(pkg.scatter_layer_shifted(*a, 1, status=b.status))
    look({1})
    pkg.check(pkg.scatter_chunks_shifted(*a, status=b.status))
    look({0, 1, 2})


@pytest.mark.parametrize("dtype,rot,interleaved", [(BF, 64, True), (F32, 2, True), (FP, 64, False)])
def test_shifted_scatter_head_dim_of_no_multiple_of_two(dtype, rot, interleaved):
    test_shifted_scatter(dtype, interleaved, rot, 16, 65, 16)


def test_shifted_scatter_many_requests_and_bad_block():
    n = 300                                     # two launches
    ends = [1 + i % 40 for i in range(n)]
    shifts = [i - 150 for i in range(n)]
    b = Batch([0] * n, ends, 2, 2, 64, BF, layers=1, layer=0)
    chunks = pkg.enumerate_chunks([0] * n, ends, 64, True)
    g = torch.Generator().manual_seed(5)
    bufs = [torch.randn((2, 1, m, 128), generator=g).to(BF) for _, _, m in chunks]
    bufs_d = [x.to(DEV) for x in bufs]
    ptrs = pkg.pointer_array(bufs_d, DEV)
    rotary = pkg.Rotary(64)
    table = b.table_d.clone()
    table[7, 0] = -1
    pkg.check(pkg.scatter_chunks_shifted(b.pool, table, [0] * n, ends, 64, True, ptrs, shifts, rotary, b.status))
    torch.cuda.synchronize()
    assert b.status.item() == lmkv.ERR_BAD_BLOCK
    flat = b.pool.layers[0].cpu().view(2, -1, 2, 64)
    for (r, t0, m), x in zip(chunks, bufs):
        if r == 7:
            continue
        at = b.slots(r)[t0:t0 + m]
        want, mag = rotate64(x[0, 0].view(m, 2, 64).double(), torch.full((m,), shifts[r]), rotary.inv_freq, False)
        within(flat[0][at], want, 2.0 ** -8 * 1.001 * want.abs() + 2.0 ** -21 * mag, f"request {r}")


# ---- attention ----------------------------------------------------------

def attend(b, q=None, out=None, lse=True, table=None, prefix_table=None, max_new=None, max_kv=None, status=None,
           stream=None, q_start=None, kv_len=None):
    q = b.q if q is None else q
    out = torch.full(b.q.shape, 7.0, dtype=b.dtype, device=DEV) if out is None else out
    max_new = max(b.new + [0]) if max_new is None else max_new
    max_kv = max(b.kv + [0]) if max_kv is None else max_kv
    n = pkg.attend_workspace_bytes(b.pool, b.heads, b.tokens, len(b.new), max_new, b.prefix, max_kv)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)             # NaN wherever it is read unwritten
    lse = torch.full((b.tokens, b.heads), 7.0, device=DEV) if lse else None
    pkg.check(pkg.attend_layer(b.pool, b.layer, q, out, b.q_start_d if q_start is None else q_start,
                               b.kv_len_d if kv_len is None else kv_len, b.table_d if table is None else table,
                               b.scale, ws, prefix_table=b.prefix_table_d if prefix_table is None else prefix_table,
                               prefix_len=b.prefix, lse=lse, max_new=max_new, max_kv_len=max_kv,
                               status=b.status if status is None else status, stream=stream))
    return out, lse


def attend_case(*a, hide=None, **kw):
    b = Batch(*a, **kw)
    out, lse = attend(b)
    torch.cuda.synchronize()
    assert b.status.item() == 0
    want, want_l, tol, tol_l = b.attend()
    live = int(b.q_start[-1])
    within(out[:live], want[:live], tol[:live], "out")
    within(lse[:live], want_l[:live], tol_l[:live], "lse")
    assert bool((out[live:] == 7.0).all()) and bool((lse[live:] == 7.0).all())
    return b


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("prefix", [0, 1, 16, 129, 700])
def test_attend_decode(dtype, dim, prefix):
    attend_case([1, 1, 1, 1, 1], [1, 16, 17, 300, 40], 8, 2, dim, dtype, prefix=prefix, extra_rows=2)


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (2, 2), (3, 1), (12, 2), (40, 8), (64, 1)])
def test_attend_head_groups(heads, kv_heads):
    attend_case([1, 2, 5], [70, 2, 33], heads, kv_heads, 128, BF, prefix=77)


@pytest.mark.parametrize("page", [1, 5, 8, 24, 64])
def test_attend_pages(page):
    attend_case([3, 1], [101, 64], 4, 2, 64, BF, prefix=203, page=page)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("new,kv,prefix", [
    ([40, 1, 130], [40, 200, 131], 0), ([40, 1, 130], [40, 200, 131], 300), ([257], [257], 0), ([64, 65], [500, 65], 1),
    ([5, 0, 3], [5, 0, 9], 0), ([128] * 3, [128, 129, 400], 128)])
def test_attend_extend(dtype, new, kv, prefix):
    attend_case(new, kv, 8, 2, 128, dtype, prefix=prefix, extra_rows=1)


def test_attend_extend_small_heads():
    attend_case([200, 31], [333, 31], 4, 4, 64, BF, prefix=190)
    attend_case([150, 150], [150, 170], 10, 2, 64, FP, prefix=515)


def test_attend_long():
    attend_case([1, 1], [5000, 3], 4, 1, 128, BF, prefix=4100)
    attend_case([300], [2500], 2, 1, 64, BF, prefix=2049)


@pytest.mark.parametrize("dtype,dim", [(BF, 128), (FP, 64)])
@pytest.mark.parametrize("prefix", [0, 200])
def test_attend_longer_own_contexts(dtype, dim, prefix):
    """Contexts that several warps share, short and empty ones and several row tiles among them."""
    attend_case([1, 1, 1, 1, 0, 1], [600, 3, 0, 1100, 700, 16], 8, 2, dim, dtype, prefix=prefix, extra_rows=1)
    attend_case([3, 15, 1, 7], [700, 900, 0, 20], 8, 2, dim, dtype, prefix=prefix, page=24)
    attend_case([2, 30, 5], [1, 650, 513], 8, 2, dim, dtype, prefix=prefix)     # unseen keys, a big request
    attend_case([1, 15], [3000, 2], 16, 4, dim, dtype, prefix=prefix)


@pytest.mark.parametrize("dtype,dim", [(BF, 128), (FP, 64)])
def test_attend_longer_own_contexts_unseen_keys(dtype, dim):
    attend_case([2, 30, 5], [1, 1100, 1030], 8, 2, dim, dtype)
    attend_case([15, 3], [1500, 9], 8, 2, dim, dtype, prefix=30, page=24)


@pytest.mark.parametrize("dtype,dim", [(BF, 128), (FP, 64)])
@pytest.mark.parametrize("longest", [60, 900])
def test_attend_long_prefix_of_many_rows(dtype, dim, longest):
    """Rows and keys enough for tiles of the prefix, with short own contexts and with
    longer ones (beside the tiles)."""
    new = [1] * 78 + [0, 3]
    attend_case(new, [1 + (i * 17) % 60 for i in range(78)] + [longest, longest - 7], 8, 2, dim, dtype, prefix=20011,
                extra_rows=2)


def test_attend_many_requests():
    n = 200
    attend_case([1] * n, [1 + (i * 13) % 60 for i in range(n)], 4, 1, 64, BF, prefix=333)
    attend_case([i % 3 for i in range(n)], [i % 3 + (i * 7) % 20 for i in range(n)], 2, 2, 64, BF, prefix=0)


def test_attend_rows_that_see_nothing():
    """No prefix: requests without tokens, and new tokens before the first cached one (kv_len < new)."""
    b = attend_case([2, 4, 1], [0, 2, 3], 4, 2, 64, BF)
    out, lse = attend(b)
    torch.cuda.synchronize()
    empty = [0, 1, 2, 3]                          # both rows of request 0, two of request 1
    assert bool((out[empty] == 0).all()) and bool((lse[empty] == -math.inf).all())
    attend_case([2, 130], [0, 100], 4, 2, 64, BF)
    attend_case([2, 3], [0, 1], 4, 2, 64, BF, prefix=5)
    attend_case([1, 1], [0, 0], 4, 2, 64, BF, prefix=0)
    attend_case([1, 1], [0, 0], 4, 2, 64, BF, prefix=33)


def test_attend_strides_and_alignment():
    b = Batch([1, 20], [30, 41], 8, 2, 64, BF, prefix=50)
    want, want_l, tol, tol_l = b.attend()
    t = b.tokens
    for off in (0, 1, 2):                         # q inside a wider projection, odd starts
        store = torch.full((t * 14 * 64 + off,), 9.0, dtype=BF, device=DEV)
        wide = store[off:].view(t, 14, 64)
        wide[:, 2:10] = b.q
        heads_first = torch.full((8 * t * 65 + off,), 7.0, dtype=BF, device=DEV)[off:].view(8, t, 65)
        out = heads_first.transpose(0, 1)[..., :64]
        o, lse = attend(b, q=wide[:, 2:10], out=out)
        torch.cuda.synchronize()
        within(o, want, tol, "out")
        within(lse, want_l, tol_l, "lse")
        assert bool((heads_first[..., 64] == 7.0).all())
    rev = b.q.flip(1)                             # a head stride below zero cannot be made in torch: check equality by data
    o2, _ = attend(b, q=rev.flip(1), lse=False)
    torch.cuda.synchronize()
    within(o2, want, tol, "out")


def test_attend_loose_bounds():
    """Bounds far above the lengths change nothing but the split."""
    b = Batch([1, 1, 6], [30, 41, 9], 8, 2, 64, BF, prefix=50)
    wide = torch.full((3, 400), -1, dtype=torch.int32, device=DEV)
    wide[:, :b.table.shape[1]] = b.table_d
    out, lse = attend(b, table=wide, max_kv=400 * 16, max_new=b.tokens)
    torch.cuda.synchronize()
    assert b.status.item() == 0
    want, want_l, tol, tol_l = b.attend()
    within(out, want, tol, "out")
    within(lse, want_l, tol_l, "lse")


@pytest.mark.parametrize("new,kv", [([1, 1], [70, 100]), ([40, 90], [70, 100])])
def test_attend_bad_blocks(new, kv):
    b = Batch(new, kv, 8, 2, 64, BF, prefix=100)
    table, prefix = b.table_d.clone(), b.prefix_table_d.clone()
    table[1, 2] = -1
    prefix[3] = b.num_blocks

    def hide(r, n):
        j = torch.arange(n) // 16
        return (j == 3) if r is None else (j == 2) if r == 1 else torch.zeros(n, dtype=torch.bool)
    out, lse = attend(b, table=table, prefix_table=prefix)
    torch.cuda.synchronize()
    assert b.status.item() == lmkv.ERR_BAD_BLOCK
    want, want_l, tol, tol_l = b.attend(hide)
    within(out, want, tol, "out")
    within(lse, want_l, tol_l, "lse")


def test_attend_large_values():
    """Scores far from zero, masked places at the type's lowest value, equal scores."""
    b = Batch([1, 40], [60, 90], 4, 2, 64, BF, prefix=30, spread=60.0)
    out, lse = attend(b)
    torch.cuda.synchronize()
    want, want_l, tol, tol_l = b.attend()
    within(out, want, tol, "out")
    within(lse, want_l, tol_l, "lse")


@pytest.mark.parametrize("scale", [0.0, -0.11, 1.0, -1e-6])
def test_attend_scales(scale):
    b = Batch([1, 40, 2], [60, 90, 17], 4, 2, 64, BF, prefix=130)
    b.scale = scale
    out, lse = attend(b)
    torch.cuda.synchronize()
    want, want_l, tol, tol_l = b.attend()
    within(out, want, tol, "out")
    within(lse, want_l, tol_l, "lse")


def test_attend_not_finite():
    """A NaN key reaches exactly the rows that see it; an infinite score makes a row NaN."""
    b = Batch([1, 1], [40, 40], 2, 1, 64, BF, prefix=20)
    b.pool.layers[1].view(2, -1, 64)[0, b.slots(0)[5]] = math.nan
    out, lse = attend(b)
    torch.cuda.synchronize()
    assert bool(out[0].isnan().all()) and bool(lse[0].isnan().all())
    want, want_l, tol, tol_l = b.attend()
    within(out[1], want[1], tol[1], "the other request")
    assert bool(lse[1].isfinite().all())


@pytest.mark.parametrize("scale", [None, -0.25, 0.0])
@pytest.mark.parametrize("dtype,dim,prefix,heads", [(BF, 128, 20, 8), (FP, 64, 0, 8), (BF, 64, 2000, 4), (FP, 128, 300, 6)])
def test_attend_values_of_other_requests_not_finite(dtype, dim, prefix, heads, scale):
    """Requests whose rows share a tile: one's infinite and NaN values stay its own."""
    b = Batch([34, 33, 3, 40], [60, 200, 50, 40], heads, 2, dim, dtype, prefix=prefix, page=24)
    b.scale = b.scale if scale is None else scale
    flat = b.pool.layers[1].view(2, -1, 2 * dim)
    flat[1, b.slots(1)[3]] = math.inf
    flat[1, b.slots(1)[150]] = math.nan
    flat[1, b.slots(3)[0]] = -math.inf
    out, lse = attend(b)
    torch.cuda.synchronize()
    assert b.status.item() == 0
    want, want_l, tol, tol_l = b.attend()
    within(lse, want_l, tol_l, "lse")
    for r in (0, 2):
        at = slice(int(b.q_start[r]), int(b.q_start[r + 1]))
        within(out[at], want[at], tol[at], f"request {r}")
    at = slice(int(b.q_start[1]), int(b.q_start[2]))
    assert not bool(out[at].isfinite().any())
    at = slice(int(b.q_start[3]), int(b.q_start[4]))
    assert not bool(out[at].isfinite().any())


def test_attend_bad_lengths():
    b = Batch([1, 3], [40, 50], 4, 2, 64, BF, prefix=20)
    for qs, kv in (([0, 1, 9], [40, 50]), ([0, 1, 4], [40, 10 ** 6]), ([0, 1, 4], [-3, 50]), ([-2, 1, 4], [40, 50]),
                   ([3, 1, 4], [40, 50])):
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        attend(b, q_start=torch.tensor(qs, dtype=torch.int32, device=DEV),
               kv_len=torch.tensor(kv, dtype=torch.int32, device=DEV), status=st)
        torch.cuda.synchronize()
        assert st.item() == lmkv.ERR_BAD_LENGTH, (qs, kv)


@pytest.mark.parametrize("prefix,kv", [(0, 50), (20, 50), (20, 900)])
def test_attend_bound_of_no_new_tokens(prefix, kv):
    """Tokens beyond a bound of 0 are reported and their rows left."""
    b = Batch([1, 2], [40, kv], 4, 2, 64, BF, prefix=prefix)
    out, lse = attend(b, max_new=0)
    torch.cuda.synchronize()
    assert b.status.item() == lmkv.ERR_BAD_LENGTH
    assert bool((out == 7.0).all()) and bool((lse == 7.0).all())


# ---- attention weights --------------------------------------------------

def weigh_case(*a, decay=1.0, fresh=False, in_place=False, **kw):
    b = Batch(*a, **kw)
    _, lse, _, _ = b.attend()
    lse = lse.float()
    g = torch.Generator().manual_seed(9)
    stride = max(b.kv) + 5
    scores = torch.rand((len(b.new), b.kv_heads, stride), generator=g)
    old = scores.to(DEV)
    out = old if in_place else torch.full_like(old, 7.0)
    pkg.check(pkg.weigh_layer(b.pool, b.layer, b.q, lse.to(DEV), b.q_start_d, b.kv_len_d, b.table_d, b.scale,
                              None if fresh else old, out, decay=decay, max_new=max(b.new), max_kv_len=max(b.kv),
                              status=b.status))
    torch.cuda.synchronize()
    assert b.status.item() == 0
    want, tol = b.weigh(lse, scores, decay)
    for r, n in enumerate(b.kv):
        within(out[r, :, :n], want[r, :, :n], tol[r, :, :n], f"request {r}")
        rest = out[r, :, n:].cpu()
        assert torch.equal(rest, scores[r, :, n:]) if in_place else bool((rest == 7.0).all())


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,kv_heads", [(8, 2), (3, 3), (5, 1)])
def test_weigh_decode(dtype, dim, heads, kv_heads):
    weigh_case([1, 1, 1, 0], [1, 300, 47, 20], heads, kv_heads, dim, dtype, prefix=21, decay=0.75)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("page", [1, 16, 24])
def test_weigh_window(dtype, page):
    weigh_case([64, 7, 33], [700, 7, 290], 8, 2, 64, dtype, page=page)
    weigh_case([64, 1], [64, 900], 16, 2, 128, dtype, page=page, prefix=40, in_place=True)


def test_weigh_options():
    weigh_case([2, 3], [40, 0], 4, 2, 64, BF, decay=0.0, fresh=True)
    weigh_case([2, 3], [40, 9], 4, 2, 64, BF, decay=0.0)
    weigh_case([2, 4], [40, 2], 4, 2, 64, BF, in_place=True)           # tokens that see nothing
    weigh_case([0, 0], [40, 9], 4, 2, 64, BF, decay=0.5)


@pytest.mark.parametrize("scale", [2.0 ** -14, -2.0 ** -14, 0.0])
@pytest.mark.parametrize("dtype,dim", [(BF, 64), (FP, 128)])
def test_weigh_scales_near_zero(dtype, dim, scale):
    b = Batch([70, 3, 1], [200, 90, 33], 8, 2, dim, dtype)
    b.scale = scale
    lse = b.attend()[1].float()
    scores = torch.rand((3, 2, 200), generator=torch.Generator().manual_seed(4))
    out = scores.to(DEV)
    pkg.check(pkg.weigh_layer(b.pool, 1, b.q, lse.to(DEV), b.q_start_d, b.kv_len_d, b.table_d, scale, out, out, decay=0.5,
                              status=b.status))
    torch.cuda.synchronize()
    assert b.status.item() == 0
    want, tol = b.weigh(lse, scores, 0.5)
    for r, n in enumerate(b.kv):
        within(out[r, :, :n], want[r, :, :n], tol[r, :, :n], f"request {r}")


@pytest.mark.parametrize("dtype", [BF, FP])
def test_weigh_window_of_large_products(dtype):
    """Products of 2^28, whose weight against an lse of their size is exactly 1: powers of
    two all along, which the product of a tile and -lse / scale leave as they are."""
    b = Batch([70], [200], 2, 2, 64, dtype)
    b.q.zero_()
    b.q[:, :, 0] = 2.0 ** 14
    flat = b.pool.layers[1].view(2, -1, 2, 64)
    flat[0, b.slots(0)] = 0.0
    flat[0, b.slots(0)[9], :, 0] = 2.0 ** 14
    lse = torch.full((70, 2), 2.0 ** 24, device=DEV)
    out = torch.full((1, 2, 200), 7.0, device=DEV)
    pkg.check(pkg.weigh_layer(b.pool, 1, b.q, lse, b.q_start_d, b.kv_len_d, b.table_d, 2.0 ** -4, None, out, decay=0.0,
                              status=b.status))
    torch.cuda.synchronize()
    want = torch.zeros(200)
    want[9] = 70.0
    assert torch.equal(out[0].cpu(), want.repeat(2, 1))


def test_weigh_repeats_bits_and_bad_block():
    b = Batch([20, 1], [300, 77], 8, 2, 128, BF)
    _, lse, _, _ = b.attend()
    table = b.table_d.clone()
    table[0, 3] = -7
    outs = []
    for _ in range(3):
        out = torch.zeros((2, 2, 300), device=DEV)
        pkg.check(pkg.weigh_layer(b.pool, 1, b.q, lse.float().to(DEV), b.q_start_d, b.kv_len_d, table, b.scale, None,
                                  out, decay=0.0, status=b.status))
        outs.append(out)
    torch.cuda.synchronize()
    assert b.status.item() == lmkv.ERR_BAD_BLOCK
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    assert bool((outs[0][0, :, 48:64] == 0).all()) and bool((outs[0][0, :, :48] > 0).all())


# ---- eviction -----------------------------------------------------------

def choose(scores, n, budget, sinks, recent):
    """Kept token numbers of one head, by sorting."""
    if n <= budget:
        return list(range(n))
    s = scores[:n].tolist()
    rank = sorted(range(sinks, n - recent), key=lambda j: (math.inf if math.isnan(s[j]) else 0, -s[j] if
                                                           not math.isnan(s[j]) else 0, j))
    return sorted(list(range(sinks)) + rank[:budget - sinks - recent] + list(range(n - recent, n)))


def evict_case(kv, budget, sinks, recent, kv_heads=2, dim=64, dtype=BF, page=16, scores=None, kept=True, seed=0,
               max_kv=None):
    b = Batch([0] * len(kv), kv, kv_heads, kv_heads, dim, dtype, page=page, seed=seed)
    m = max(kv + [1]) if max_kv is None else max_kv
    g = torch.Generator().manual_seed(seed + 3)
    if scores is None:
        scores = torch.exp(3 * torch.randn((len(kv), kv_heads, m), generator=g))
        scores[torch.rand(scores.shape, generator=g) < 0.3] = 0.0
    keep = torch.full((len(kv), kv_heads, budget), 99, dtype=torch.int32, device=DEV)
    new_len = torch.full((len(kv),), 99, dtype=torch.int32, device=DEV)
    ks = torch.full((len(kv), kv_heads, budget + 3), 99.0, device=DEV) if kept else None
    pkg.check(pkg.evict_layer(b.pool, b.layer, b.table_d, b.kv_len_d, scores.to(DEV), sinks, recent, keep, new_len,
                              kept_scores=ks, max_kv_len=m, status=b.status))
    torch.cuda.synchronize()
    assert b.status.item() == 0
    want = b.pool_cpu.clone()
    flat, old = want[b.layer].view(2, -1, kv_heads, dim), b.pool_cpu[b.layer].view(2, -1, kv_heads, dim)
    assert new_len.tolist() == [min(n, budget) for n in kv]
    for r, n in enumerate(kv):
        at = b.slots(r)
        for h in range(kv_heads):
            idx = choose(scores[r, h], n, budget, sinks, recent)
            assert keep[r, h].tolist() == idx + [-1] * (budget - len(idx)), (r, h)
            flat[:, at[:len(idx)], h] = old[:, at[idx], h]
            if kept:
                assert torch.equal(ks[r, h, :len(idx)].cpu().nan_to_num(5.5), scores[r, h, idx].nan_to_num(5.5))
                assert bool((ks[r, h, len(idx):budget] == 0).all()) and bool((ks[r, h, budget:] == 99.0).all())
    for i, l in enumerate(b.pool.layers):
        assert torch.equal(l.cpu().view(torch.uint8), want[i].view(torch.uint8))


@pytest.mark.parametrize("dtype", [BF, FP, F32])
@pytest.mark.parametrize("page", [1, 16, 24])
def test_evict(dtype, page):
    evict_case([500, 31, 32, 33, 0, 1, 100], 32, 4, 8, dtype=dtype, page=page)


@pytest.mark.parametrize("budget,sinks,recent", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (32, 32, 0), (32, 0, 32), (32, 16, 16),
                                                 (33, 0, 0), (600, 4, 4), (299, 0, 1)])
def test_evict_budgets(budget, sinks, recent):
    evict_case([300, 40, 200], budget, sinks, recent, kv_heads=3, dim=128)


def test_evict_long():
    evict_case([9000, 4097, 2500], 2048, 4, 100, kv_heads=1, dim=64)
    evict_case([40000], 100, 4, 10, kv_heads=2, dim=64)
    evict_case([20011], 15000, 0, 0, kv_heads=1, dim=128)
    evict_case([60001, 300, 51201], 5000, 4, 10, kv_heads=1, dim=64)      # more keys than shared memory holds


def test_evict_odd_rows():
    evict_case([100, 60], 20, 2, 3, kv_heads=4, dim=20, dtype=BF)       # 40-byte heads
    evict_case([100, 60], 20, 2, 3, kv_heads=8, dim=3, dtype=BF)        # 6-byte heads
    evict_case([100, 60], 20, 2, 3, kv_heads=1, dim=256, dtype=BF)


def test_evict_ties_and_special_scores():
    s = torch.zeros((2, 2, 100))
    s[0, 0] = -0.0
    s[0, 0, ::3] = 0.0
    s[0, 1] = torch.arange(100).float() % 4
    s[1, 0] = math.nan
    s[1, 0, 40:60] = -math.inf
    s[1, 0, 50] = math.inf
    s[1, 1] = -torch.arange(100).float()
    s[1, 1, 7] = math.nan
    for budget, sinks, recent in ((30, 0, 0), (30, 4, 5), (70, 0, 1)):
        evict_case([100, 90], budget, sinks, recent, scores=s)
    evict_case([100, 90], 30, 4, 5, scores=s, kept=False)


def test_evict_repeated_call_is_the_same_move():
    evict_case([64] * 40, 48, 0, 0, kv_heads=1, dim=64, max_kv=64)
    evict_case([17] * 300, 16, 0, 0, kv_heads=1, dim=64)


def test_evict_nothing_cached():
    """A batch with no room for cached tokens: no scores, no table."""
    b = Batch([0, 0], [0, 0], 2, 2, 64, BF)
    keep = torch.full((2, 2, 3), 7, dtype=torch.int32, device=DEV)
    new_len = torch.full((2,), 7, dtype=torch.int32, device=DEV)
    pkg.check(pkg.evict_layer(b.pool, 1, b.table_d, b.kv_len_d, torch.empty((2, 2, 0), device=DEV), 1, 1, keep, new_len,
                              status=b.status))
    torch.cuda.synchronize()
    assert b.status.item() == 0
    assert bool((keep == -1).all()) and bool((new_len == 0).all())


def test_evict_bad_block_and_length():
    b = Batch([0], [100], 2, 2, 64, BF)
    table = b.table_d.clone()
    table[0, 5] = b.num_blocks
    scores = torch.arange(100, 0, -1).float().repeat(1, 2, 1).to(DEV)
    scores[0, :, 81] = 1000.0                 # in the bad page
    scores[0, :, 97] = 1000.0
    keep = torch.empty((1, 2, 20), dtype=torch.int32, device=DEV)
    new_len = torch.empty(1, dtype=torch.int32, device=DEV)
    pkg.check(pkg.evict_layer(b.pool, 1, table, b.kv_len_d, scores, 0, 0, keep, new_len, status=b.status))
    torch.cuda.synchronize()
    assert b.status.item() == lmkv.ERR_BAD_BLOCK
    assert keep[0, 0].tolist() == list(range(18)) + [81, 97]
    flat, old = b.pool.layers[1].cpu().view(2, -1, 128), b.pool_cpu[1].view(2, -1, 128)
    at = b.slots(0)
    assert torch.equal(flat[:, at[18]], old[:, at[18]]) and torch.equal(flat[:, at[19]], old[:, at[97]])
    b.status.zero_()
    ln = torch.tensor([5000], dtype=torch.int32, device=DEV)
    pkg.check(pkg.evict_layer(b.pool, 1, b.table_d, ln, scores, 0, 0, keep, new_len, max_kv_len=100, status=b.status))
    torch.cuda.synchronize()
    assert b.status.item() == lmkv.ERR_BAD_LENGTH and new_len.item() == 20


# ---- together -----------------------------------------------------------

def step_buffers(b, budget):
    n, m = len(b.new), max(b.kv)
    ws = pkg.attend_workspace_bytes(b.pool, b.heads, b.tokens, n, max(b.new), b.prefix, m)
    return dict(ws=torch.empty(ws, dtype=torch.uint8, device=DEV), q=torch.empty_like(b.q), out=torch.empty_like(b.q),
                lse=torch.empty((b.tokens, b.heads), device=DEV), scores=torch.zeros((n, b.kv_heads, m), device=DEV),
                keep=torch.empty((n, b.kv_heads, budget), dtype=torch.int32, device=DEV),
                new_len=torch.empty(n, dtype=torch.int32, device=DEV),
                kept=torch.empty((n, b.kv_heads, budget), device=DEV))


def decode_step(b, s, k, v, rotary, stream=None):
    a = dict(max_new=max(b.new), max_kv_len=max(b.kv), status=b.status, stream=stream)
    pkg.check(pkg.append_layer(b.pool, 1, b.table_d, b.q, k, v, s["q"], b.q_start_d, b.kv_len_d, rotary,
                               status=b.status, stream=stream))
    pkg.check(pkg.attend_layer(b.pool, 1, s["q"], s["out"], b.q_start_d, b.kv_len_d, b.table_d, b.scale, s["ws"],
                               prefix_table=b.prefix_table_d, prefix_len=b.prefix, lse=s["lse"], **a))
    pkg.check(pkg.weigh_layer(b.pool, 1, s["q"], s["lse"], b.q_start_d, b.kv_len_d, b.table_d, b.scale, s["scores"],
                              s["scores"], **a))
    pkg.check(pkg.evict_layer(b.pool, 1, b.table_d, b.kv_len_d, s["scores"], 2, 6, s["keep"], s["new_len"],
                              kept_scores=s["kept"], max_kv_len=max(b.kv), status=b.status, stream=stream))


@pytest.mark.parametrize("new,kv,heads,kv_heads,dim", [
    ([1, 1, 1], [200, 31, 90], 8, 2, 64), ([60, 1, 33], [200, 31, 90], 16, 2, 128)])
def test_decode_step_eager_and_captured(new, kv, heads, kv_heads, dim):
    """Append, attend, weigh and evict in a row on one stream, eager, then captured
    on another stream and replayed from the same start: the same bits.  The
    eager step is checked against the formulas on what it wrote."""
    b = Batch(new, kv, heads, kv_heads, dim, BF, prefix=150)
    g = torch.Generator().manual_seed(4)
    k, v = (torch.randn((b.tokens, kv_heads, dim), generator=g).to(BF).to(DEV) for _ in range(2))
    rotary = pkg.Rotary(dim)
    start = b.pool.layers[1].clone()
    eager, graphed = step_buffers(b, 48), step_buffers(b, 48)
    decode_step(b, eager, k, v, rotary)
    torch.cuda.synchronize()
    assert b.status.item() == 0
    after = b.pool.layers[1].clone()
    # the formulas, on the rotated rows that the append wrote
    b.pool.layers[1].copy_(start)
    pkg.check(pkg.append_layer(b.pool, 1, b.table_d, b.q, k, v, graphed["q"], b.q_start_d, b.kv_len_d, rotary))
    torch.cuda.synchronize()
    b.pool_cpu[1] = b.pool.layers[1].cpu()
    b.q_cpu = eager["q"].cpu()
    want, want_l, tol, tol_l = b.attend()
    within(eager["out"], want, tol, "out")
    within(eager["lse"], want_l, tol_l, "lse")
    ws, ts = b.weigh(eager["lse"].cpu(), torch.zeros_like(eager["scores"]).cpu(), 1.0)
    within(eager["scores"], ws, ts, "scores")
    for r, n in enumerate(kv):
        for h in range(kv_heads):
            idx = choose(eager["scores"][r, h].cpu(), n, 48, 2, 6)
            assert eager["keep"][r, h].tolist() == idx + [-1] * (48 - len(idx))
            at = b.slots(r)
            x = after.cpu().view(2, -1, kv_heads, dim)[:, at[:len(idx)], h]
            assert torch.equal(x, b.pool_cpu[1].view(2, -1, kv_heads, dim)[:, at[idx], h])
    # captured
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        decode_step(b, graphed, k, v, rotary)
    for _ in range(2):
        b.pool.layers[1].copy_(start)
        graphed["scores"].zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert b.status.item() == 0
        for n in ("q", "out", "lse", "scores", "keep", "new_len", "kept"):
            assert torch.equal(eager[n], graphed[n]), n
        assert torch.equal(after.view(torch.int16), b.pool.layers[1].view(torch.int16))


def test_captured_step_follows_the_lengths():
    """A captured call reads the lengths on the device: replays with other lengths equal eager calls."""
    b = Batch([1, 1, 1], [200, 31, 90], 8, 2, 64, BF, prefix=100)
    out, lse = torch.zeros_like(b.q), torch.zeros((3, 8), device=DEV)
    n = pkg.attend_workspace_bytes(b.pool, 8, 3, 3, 1, 100, 200)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)

    def go(o, l, w):
        pkg.check(pkg.attend_layer(b.pool, 1, b.q, o, b.q_start_d, b.kv_len_d, b.table_d, b.scale, w,
                                   prefix_table=b.prefix_table_d, prefix_len=100, lse=l, max_new=1, max_kv_len=200,
                                   status=b.status))
    go(out, lse, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(out, lse, ws)
    for lens in ([200, 31, 90], [1, 30, 17], [0, 31, 64]):
        b.kv_len_d.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        o2, l2 = torch.zeros_like(out), torch.zeros_like(lse)
        go(o2, l2, torch.empty_like(ws))
        torch.cuda.synchronize()
        assert torch.equal(out, o2) and torch.equal(lse, l2)
        assert b.status.item() == 0


def test_two_streams_at_once():
    """Two calls in flight on two streams, a workspace each."""
    b = Batch([1] * 20, [100 + 13 * i for i in range(20)], 8, 2, 128, BF, prefix=1500)
    ref, _ = attend(b)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    n = pkg.attend_workspace_bytes(b.pool, 8, 20, 20, 1, 1500, max(b.kv))
    bufs = [(torch.empty(n, dtype=torch.uint8, device=DEV), torch.zeros_like(b.q)) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, (w, o) in zip((s1, s2), bufs):
            pkg.check(pkg.attend_layer(b.pool, 1, b.q, o, b.q_start_d, b.kv_len_d, b.table_d, b.scale, w,
                                       prefix_table=b.prefix_table_d, prefix_len=1500, max_new=1,
                                       max_kv_len=max(b.kv), stream=s))
    torch.cuda.synchronize()
    assert torch.equal(bufs[0][1], ref) and torch.equal(bufs[1][1], ref)


def test_first_calls_are_captured():
    """A process whose first calls of the operators are made under capture."""
    code = """
import torch
import paged_kv_cache_lmkv_gb300 as pkg
from operator_util import Batch, DEV
b = Batch([70, 1], [200, 90], 8, 2, 64, torch.bfloat16, prefix=150)
c = Batch([1, 1], [1000, 90], 8, 2, 64, torch.bfloat16)
k = torch.randn((71, 2, 64), device=DEV).bfloat16()
rot = pkg.Rotary(64)
s = torch.cuda.Stream()

def run(b):
    n, m, w = len(b.new), max(b.kv), max(b.new)
    ws = torch.empty(pkg.attend_workspace_bytes(b.pool, b.heads, b.tokens, n, w, b.prefix, m), dtype=torch.uint8,
                     device=DEV)
    out, q = torch.zeros_like(b.q), torch.zeros_like(b.q)
    lse = torch.zeros((b.tokens, b.heads), device=DEV)
    scores = torch.zeros((n, b.kv_heads, m), device=DEV)
    keep = torch.zeros((n, b.kv_heads, 32), dtype=torch.int32, device=DEV)
    new_len = torch.zeros(n, dtype=torch.int32, device=DEV)
    kk = k[:b.tokens]

    def go():
        pkg.check(pkg.append_layer(b.pool, 1, b.table_d, b.q, kk, kk, q, b.q_start_d, b.kv_len_d, rot, status=b.status))
        pkg.check(pkg.attend_layer(b.pool, 1, q, out, b.q_start_d, b.kv_len_d, b.table_d, b.scale, ws,
                                   prefix_table=b.prefix_table_d, prefix_len=b.prefix, lse=lse, max_new=w,
                                   max_kv_len=m, status=b.status))
        pkg.check(pkg.weigh_layer(b.pool, 1, q, lse, b.q_start_d, b.kv_len_d, b.table_d, b.scale, scores, scores,
                                  max_new=w, status=b.status))
        pkg.check(pkg.evict_layer(b.pool, 1, b.table_d, b.kv_len_d, scores, 2, 6, keep, new_len, status=b.status))
    start = [x.clone() for x in b.pool.layers]
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        go()
    g.replay()
    torch.cuda.synchronize()
    first = [x.clone() for x in (q, out, lse, scores, keep, new_len, *b.pool.layers)]
    for x, y in zip(b.pool.layers, start):
        x.copy_(y)
    scores.zero_()
    go()
    torch.cuda.synchronize()
    assert b.status.item() == 0
    for x, y in zip(first, (q, out, lse, scores, keep, new_len, *b.pool.layers)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))

run(b)
run(c)
print("same")
"""
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([os.path.dirname(here), here, os.environ.get("PYTHONPATH", "")]))
    r = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]
