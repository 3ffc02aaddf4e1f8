"""The 8-bit cache's operators against 64-bit formulas: append with norms of q and k, attention
with a window and sinks over 16-bit and 8-bit pages, and both beside forked, resized and
compacted pages, eager, captured and replayed."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_lmkv_gb300 as pkg
from paged_kv_cache_lmkv_gb300 import lmkv
from cache8_util import E4M3, E8M0, LOWEST, Cache, codes_of, exponent, normed64, turned64
from gpu_util import require_gpu
from operator_util import DEV, HALF_STEP, TINY, within

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16
BITS = {BF: torch.int16, FP: torch.int16, E4M3: torch.uint8}


@pytest.fixture(autouse=True)
def gpu():
    require_gpu()


def make_rotary(rot, interleaved=False, magnitude=1.0):
    r = pkg.Rotary(rot, base=10000.0, interleaved=interleaved, magnitude=magnitude)
    r.interleaved = interleaved
    return r


# ---- append with norms ----------------------------------------------------

def append_case(new, kv, heads, kv_heads, dim, dtype, wide, rot=0, interleaved=False, norms=True, page=16, offset=0,
                in_place=False, positions=None, extra=0, seed=0, spread=1.0, exps=(-9, -3), eps=1e-6, split=True):
    b = Cache(new, kv, heads, kv_heads, dim, dtype, wide, page, seed, extra, exps=exps)
    g = torch.Generator().manual_seed(seed + 1)
    t, width = b.tokens, heads + 2 * kv_heads
    store = (torch.randn(t * width * dim + offset, generator=g) * spread).to(dtype)
    store_d = store.to(DEV)
    cut = (lambda s: [s[offset:].view(t, width, dim)[:, a:z] for a, z in
                      ((0, heads), (heads, heads + kv_heads), (heads + kv_heads, width))])
    q, k, v = cut(store_d)
    qc, kc, vc = cut(store)
    q_out = q if in_place else torch.full((t, heads, dim), 7.0, dtype=dtype, device=DEV)
    before = q_out.clone().cpu()
    live = int(b.q_start[-1])
    index = torch.cat([torch.arange(m - n, m) for n, m in zip(new, kv)]) if new else torch.zeros(0)
    pos = index if positions is None else torch.tensor(positions, dtype=torch.int64)
    rotary = make_rotary(rot, interleaved, 1.25) if rot else None
    qn, kn = ((torch.randn(dim, generator=g) * 0.3 + 1.0) for _ in range(2)) if norms else (None, None)
    put = lambda x: None if x is None else x.to(DEV)
    call = lambda: pkg.check(pkg.append_layer_normed(
        b.pool, b.layer, b.table_d, q, k, v, q_out, b.q_start_d, b.kv_len_d, rotary, put(qn), put(kn), eps,
        positions=None if positions is None else torch.cat((pos, torch.zeros(extra, dtype=torch.int64))).to(DEV),
        status=b.status))
    call()
    torch.cuda.synchronize()
    assert b.status.item() == 0
    step, tiny = HALF_STEP[dtype], TINY[dtype]
    # In fp32: a norm's mean of dim squares is off by (dim + 2) 2^-24, its root by half of that and 2^-22; three more
    # products; cosine, sine within 2^-21.1, two products and a sum; the frequency's rounding is 2^-53 of its angle.
    angle = pos[:live].abs().max().item() * 2.0 ** -51 if live else 0.0
    rel = (dim + 2) * 2.0 ** -25 + 8 * 2.0 ** -24 + 2.0 ** -21 + 2.0 ** -20 + angle

    want, mag = turned64(normed64(qc[:live], qn, eps), pos[:live], rotary)
    within(q_out[:live], want, step * 1.001 * want.abs() + rel * mag + tiny, "q")
    assert torch.equal(q_out[live:].cpu(), before[live:])

    k64, k_mag = turned64(normed64(kc[:live], kn, eps), pos[:live], rotary)
    v64 = vc[:live].double()
    where = torch.cat([b.slots(r)[m - n:] for r, (n, m) in enumerate(zip(new, kv))])
    got = b.pool.layers[b.layer].cpu()
    got = got if wide else got.view(torch.uint8)
    flat = got.view(2, -1, kv_heads, dim)
    expect = b.pool_cpu[b.layer].clone().view(2, -1, kv_heads, dim)
    if wide:
        within(flat[0, where], k64, step * 1.001 * k64.abs() + rel * k_mag + tiny, "k")
        assert torch.equal(flat[1, where].view(torch.int16), vc[:live].contiguous().view(torch.int16))
        expect[:, where] = flat[:, where]
    else:
        blk = where // page
        sc = b.scales_cpu[b.layer].long() - 127                           # [2, pages, heads]
        now = b.scales_d[b.layer].cpu().long() - 127
        x64, x_mag = torch.stack((k64, v64)), torch.stack((rel * k_mag, torch.zeros_like(v64)))
        assert x64.isfinite().all()
        amax = torch.zeros(2, b.num_blocks, kv_heads, dtype=torch.float64).index_reduce_(1, blk, x64.abs().amax(-1), "amax")
        err = torch.zeros_like(amax).index_reduce_(1, blk, x_mag.amax(-1), "amax")
        held = torch.zeros(b.num_blocks, dtype=torch.bool)
        touched = torch.zeros(b.num_blocks, dtype=torch.bool)
        touched[blk] = True
        for r, (n, m) in enumerate(zip(new, kv)):
            if n and (m - n) % page:
                held[int(b.table[r, (m - n) // page])] = True
        before_e = torch.where(held[None, :, None], sc, LOWEST)
        lo, hi = torch.maximum(exponent((amax - err).clamp(min=0)), before_e), torch.maximum(exponent(amax + err), before_e)
        at = touched[None, :, None]
        assert bool(torch.where(at, (now >= lo) & (now <= hi), now == sc).all())
        # the new tokens' codes
        power = torch.exp2(now.double())[:, blk][..., None]
        unit = x64 / power
        half = torch.maximum(unit.abs() * 2.0 ** -4, torch.full((), 2.0 ** -10, dtype=torch.float64))
        within(flat[:, where].contiguous().view(E4M3).double(), unit, half * 1.001 + 1.1 * x_mag / power, "codes")
        expect[:, where] = flat[:, where]
        # earlier tokens of the same pages, rounded again where the scale has grown
        for r, (n, m) in enumerate(zip(new, kv)):
            a = (m - n) % page
            if n and a:
                p = int(b.table[r, (m - n) // page])
                old = b.pool_cpu[b.layer][:, p, :a].contiguous().view(2, a, kv_heads, dim).view(E4M3).double()
                by = torch.exp2((sc - now)[:, p].double())[:, None, :, None]
                expect.view(2, b.num_blocks, page, kv_heads, dim)[:, p, :a] = codes_of(old * by)
    for i, l in enumerate(b.pool.layers):           # every other slot, layer and row as it was
        want_l = expect.view(got.shape) if i == b.layer else b.pool_cpu[i]
        assert torch.equal(l.cpu().view(torch.uint8), want_l.contiguous().view(torch.uint8)), i
    if not wide and not in_place:
        call()
        torch.cuda.synchronize()
        assert torch.equal(b.pool.layers[b.layer].cpu().view(torch.uint8), got.view(torch.uint8))     # the same codes again


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("dim,rot", [(64, 64), (64, 0), (64, 34), (64, 2), (128, 128), (128, 64), (128, 20), (128, 16)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_layouts(wide, dtype, dim, rot, interleaved):
    append_case([1, 3, 0, 17, 33], [5, 3, 9, 50, 40], 6, 2, dim, dtype, wide, rot, interleaved, extra=3)


@pytest.mark.parametrize("page", [1, 5, 8, 16, 24, 64])
@pytest.mark.parametrize("wide", [False, True])
def test_append_pages_and_long(page, wide):
    append_case([400, 1, 33, 2], [431, 70, 33, 18], 8, 8, 128, BF, wide, 128, page=page)


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (5, 5), (40, 8), (6, 3), (70, 7)])
def test_append_head_counts(heads, kv_heads):
    append_case([1, 20], [4, 37], heads, kv_heads, 64, BF, False, 64)


@pytest.mark.parametrize("offset", [0, 1, 4])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("wide", [False, True])
def test_append_alignment_and_in_place(offset, in_place, wide):
    append_case([2, 5, 40], [8, 5, 41], 4, 2, 64, BF, wide, 64, offset=offset, in_place=in_place)
    append_case([2, 5, 40], [8, 5, 41], 4, 2, 64, BF, wide, 34, offset=offset, in_place=in_place)


def test_append_without_norms_or_with_large_eps():
    append_case([3, 20], [7, 25], 4, 2, 128, FP, False, 128, norms=False)
    append_case([3, 20], [7, 25], 4, 2, 128, FP, False, 128, eps=10.0)


def test_append_far_positions():
    append_case([8], [8], 4, 2, 64, BF, False, 64, positions=[0, 1, -1, 131071, 2 ** 20 + 1, -(2 ** 24) - 3, 2 ** 31 + 5, 123456789])


def test_append_many_requests():
    new = [(i * 7) % 3 for i in range(1100)]
    append_case(new, [n + (i % 37) for i, n in enumerate(new)], 2, 1, 64, BF, False, 64)


@pytest.mark.parametrize("exps", [(-20, -15), (2, 30), (40, 60)])
def test_append_scales_far_from_the_values(exps):
    """Values much larger and much smaller than the page's earlier scale."""
    append_case([1, 3, 17], [9, 30, 40], 4, 2, 64, BF, False, 64, exps=exps)


def one_page(values, before=0, byte=127, dtype=BF):
    """Appends rows of one head of 64 to a page behind `before` tokens; (codes, scale byte, old codes)."""
    n = values.shape[0]
    b = Cache([n], [before + n], 1, 1, 64, dtype, seed=3)
    b.scales_d.fill_(byte)
    old = b.pool.layers[1].view(torch.uint8).clone()
    z = torch.zeros((n, 1, 64), dtype=dtype, device=DEV)
    v = values.to(dtype).to(DEV)[:, None]
    pkg.check(pkg.append_layer_normed(b.pool, 1, b.table_d, z, z, v, z, b.q_start_d, b.kv_len_d, status=b.status))
    torch.cuda.synchronize()
    assert b.status.item() == 0
    p = int(b.table[0, 0])
    return b.pool.layers[1].view(torch.uint8)[1, p].cpu(), int(b.scales_d[1, 1, p, 0]), old[1, p].cpu(), int(b.scales_d[1, 0, p, 0])


def test_append_borders_of_the_scale():
    """448 * 2^e is the last value of exponent e; K of zeros has the lowest."""
    for top, e in ((448.0, 0), (450.0, 1), (447.0, 0), (7.0, -6), (7.03125, -5), (2.0 ** -40, -48), (1e30, 60), (2.0 ** -100, -60)):
        x = torch.zeros(2, 64)
        x[1, 5] = -top
        codes, byte, _, k_byte = one_page(x)
        assert byte == e + 127 and k_byte == -60 + 127, top
        want = codes_of(torch.tensor(float(torch.tensor(-top).to(BF))).double() * 2.0 ** -e)
        assert int(codes[1, 5]) == int(want)
        assert int(codes.view(E4M3).float()[:2].abs().sum() - codes.view(E4M3).float()[1, 5].abs()) == 0


def test_append_values_that_are_not_finite():
    x = torch.ones(3, 64)
    x[0, 0], x[1, 1], x[2, 2], x[2, 3] = math.nan, math.inf, -math.inf, 3.0
    codes, byte, _, _ = one_page(x)
    assert byte == 127 - 7                      # of 3.0
    got = codes.view(E4M3).float()[:3]
    bad = torch.zeros(3, 64, dtype=torch.bool)
    bad[0, 0] = bad[1, 1] = bad[2, 2] = True
    assert bool((got.isnan() == bad).all())
    assert bool((got[~bad] * 2.0 ** -7 == x[~bad]).all())


def test_append_keeps_a_larger_scale_and_a_nan_scale():
    x = torch.ones(1, 64)
    codes, byte, old, _ = one_page(x, before=4, byte=130)
    assert byte == 130 and torch.equal(codes[:4], old[:4]) and bool((codes[4].view(E4M3).float() == 0.125).all())
    _, byte, _, _ = one_page(x, before=4, byte=255)
    assert byte == 255
    _, byte, _, _ = one_page(x, before=0, byte=255)           # no earlier tokens: the page begins anew
    assert byte == 127 - 8


def test_append_bad_blocks_and_lengths():
    b = Cache([2, 2], [20, 6], 4, 2, 64, BF)
    g = torch.Generator().manual_seed(1)
    qkv = torch.randn((4, 8, 64), generator=g).to(BF).to(DEV)
    q, k, v = qkv[:, :4], qkv[:, 4:6], qkv[:, 6:]
    before = b.pool.layers[1].view(torch.uint8).clone(), b.scales_d.clone()

    def go(table, kv_len, q_start=None):
        out = torch.full_like(q, 7.0)
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        pkg.check(pkg.append_layer_normed(b.pool, 1, table, q, k, v, out, b.q_start_d if q_start is None else q_start,
                                          kv_len, make_rotary(64), status=st))
        torch.cuda.synchronize()
        return st.item(), out
    p0 = int(b.table[0, 1])
    for bad in (-1, b.num_blocks, 2 ** 31 - 1, -2 ** 31):
        t = b.table_d.clone()
        t[0, 1] = bad
        code, out = go(t, b.kv_len_d)
        assert code == lmkv.ERR_BAD_BLOCK and not bool((out == 7.0).all(-1).any())
        assert torch.equal(b.pool.layers[1].view(torch.uint8)[:, p0], before[0][:, p0])
        assert torch.equal(b.scales_d[:, :, p0], before[1][:, :, p0])
    for bad in ([1, 6], [20, 10 ** 6], [20, -5]):
        assert go(b.table_d, torch.tensor(bad, dtype=torch.int32, device=DEV))[0] == lmkv.ERR_BAD_LENGTH
    assert go(b.table_d, b.kv_len_d, torch.tensor([0, 9, 4], dtype=torch.int32, device=DEV))[0] == lmkv.ERR_BAD_LENGTH
    # a null entry among the scales
    b.pool.scale_ptrs[1] = 0
    assert go(b.table_d, b.kv_len_d)[0] == lmkv.ERR_BAD_POINTER


# ---- attention with a window and sinks ------------------------------------

def run_attend(b, window=0, sinks=0, q=None, out=None, lse=True, ws=None, scale=None, **kw):
    q = b.q if q is None else q
    out = torch.full((b.tokens, b.heads, b.dim), 7.0, dtype=b.dtype, device=DEV) if out is None else out
    l = torch.full((b.tokens, b.heads), 7.0, device=DEV) if lse else None
    max_new, max_len = max(b.new, default=0), max(b.kv, default=0)
    if ws is None:
        n = pkg.attend_window_workspace_bytes(b.pool, b.heads, b.tokens, len(b.new), max_new, max(max_len, 0))
        ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV)
    kw = dict(max_new=max_new, max_kv_len=max(max_len, 0), status=b.status) | kw
    pkg.check(pkg.attend_layer_window(b.pool, b.layer, q, out, b.q_start_d, b.kv_len_d, b.table_d,
                                      b.scale if scale is None else scale, ws, window, sinks, l, **kw))
    torch.cuda.synchronize()
    return out, l


def attend_case(b, window=0, sinks=0, status=0, hide=None, **kw):
    out, l = run_attend(b, window, sinks, **kw)
    assert b.status.item() == status
    want, want_l, tol, tol_l = b.attend(window, sinks, hide, kw.get("scale"))
    live = int(b.q_start[-1])
    within(out[:live], want[:live], tol[:live], "out")
    within(l[:live], want_l[:live], tol_l[:live], "lse")
    assert bool((out[live:] == 7.0).all()) and bool((l[live:] == 7.0).all())
    return out, l


WINDOWS = [(0, 0), (1, 0), (7, 3), (40, 4), (40, 37), (1000, 2)]


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_attend_decode(wide, dtype, dim, window, sinks):
    b = Cache([1, 1, 1, 0, 1, 1], [1, 200, 17, 9, 16, 533], 8, 2, dim, dtype, wide, extra_rows=2)
    attend_case(b, window, sinks)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_attend_few_new_tokens(wide, dtype, window, sinks):
    b = Cache([5, 2, 0, 3, 1], [205, 2, 40, 47, 90], 16, 2, 128, dtype, wide, extra_rows=1, seed=1)
    attend_case(b, window, sinks)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 1), (50, 5), (130, 200)])
def test_attend_tiles(wide, dtype, dim, window, sinks):
    """Requests of 64 rows and more beside small ones; 256 rows and more; a tile of few rows."""
    b = Cache([70, 3, 16, 33, 1], [300, 50, 16, 161, 400], 8, 2, dim, dtype, wide, extra_rows=2, seed=2)
    attend_case(b, window, sinks)


@pytest.mark.parametrize("page", [1, 5, 8, 16, 24, 48, 64])
@pytest.mark.parametrize("wide", [False, True])
def test_attend_pages(page, wide):
    b = Cache([1, 4, 40], [333, 70, 141], 8, 2, 64, BF, wide, page)
    attend_case(b)
    attend_case(b, 33, 3)


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (5, 1), (9, 3), (16, 1), (24, 8), (80, 1)])
@pytest.mark.parametrize("new", [1, 4, 21])
def test_attend_head_counts(heads, kv_heads, new):
    b = Cache([new, 1], [100, 35], heads, kv_heads, 64, BF)
    attend_case(b, 60, 2)


@pytest.mark.parametrize("wide", [False, True])
def test_attend_long_contexts_in_parts(wide):
    """Few rows against many keys: streams and parts of tiles that are joined."""
    attend_case(Cache([1, 1], [9000, 3000], 4, 1, 128, BF, wide))
    attend_case(Cache([40], [5000], 4, 2, 128, BF, wide))
    attend_case(Cache([40], [5000], 4, 2, 64, FP, wide), 3000, 4)


def test_attend_one_long_context_among_many():
    """Rows of many parts beside many rows of one."""
    attend_case(Cache([1] * 200, [9000] + [5 + i % 20 for i in range(199)], 4, 1, 64, BF))


def test_attend_more_items_than_sms():
    b = Cache([130, 90, 75], [131, 300, 75], 64, 16, 64, BF, False)
    attend_case(b)
    b = Cache([20] * 60, [20 + i for i in range(60)], 16, 4, 64, BF, True)
    attend_case(b, 9, 1)


def test_attend_many_requests():
    new = [1 + (i % 3 == 0) for i in range(1100)]
    attend_case(Cache(new, [n + (i * 5) % 41 for i, n in enumerate(new)], 2, 1, 64, BF, False), 20, 2)


@pytest.mark.parametrize("new", [2, 40])
def test_attend_rows_that_see_nothing(new):
    """More new tokens than cached ones, no cached ones, none new."""
    b = Cache([new, new, 0], [new - 1, 0, 5], 8, 2, 64, BF)
    for window, sinks in ((0, 0), (3, 1)):
        out, l = attend_case(b, window, sinks, status=0)
        assert bool((out[0] == 0).all()) and bool((l[0] == -math.inf).all())
        assert bool((out[new:2 * new] == 0).all()) and bool((l[new:2 * new] == -math.inf).all())


@pytest.mark.parametrize("new", [1, 3, 40])
@pytest.mark.parametrize("wide", [False, True])
def test_attend_pages_outside_the_window_are_not_there(new, wide):
    """Entries of pages that no row sees any of may be anything, and what lies in seen pages but is not seen by
    any row does not reach a row, whatever it is."""
    n, window, sinks, page = 900, 70, 5, 16
    b = Cache([new], [n], 8, 2, 64, BF, wide)
    want = run_attend(b, window, sinks)[0].clone()
    attend_case(b, window, sinks)
    first = n - new + 1 - window                   # first key that the first row sees behind the sinks
    b.table_d[0, 1:first // page] = torch.tensor([-1, 10 ** 9, -7] * 100, dtype=torch.int32)[:first // page - 1].to(DEV)
    flat = b.pool.layers[1].view(2, -1, 2 * 64)
    hidden = torch.cat((b.slots(0)[sinks:page], b.slots(0)[first // page * page:first])).to(DEV)
    assert len(hidden) > 0
    flat.view(torch.uint8 if not wide else torch.int16)[:, hidden] = 0x7F if not wide else 0x7FC0     # NaN
    got = run_attend(b, window, sinks)[0]
    assert b.status.item() == 0
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("new", [1, 40])
def test_attend_bad_blocks(new):
    b = Cache([new, 1], [300, 40], 8, 2, 64, BF)
    for bad in (-1, b.num_blocks, -2 ** 31):
        b.status.zero_()
        b.table_d[0, 3] = bad
        attend_case(b, status=lmkv.ERR_BAD_BLOCK, hide=lambda r, n: (torch.arange(n) // 16 == 3) & (r == 0))


@pytest.mark.parametrize("new", [1, 40])
def test_attend_lengths_beyond_their_bounds(new):
    b = Cache([new, 1], [300, 40], 8, 2, 64, BF)
    for field, bad in (("kv_len_d", [10 ** 6, 40]), ("kv_len_d", [-4, 40]), ("q_start_d", [0, 10 ** 6, new + 1])):
        b.status.zero_()
        keep = getattr(b, field)
        setattr(b, field, torch.tensor(bad, dtype=torch.int32, device=DEV))
        run_attend(b)
        assert b.status.item() == lmkv.ERR_BAD_LENGTH
        setattr(b, field, keep)


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("scale", [-0.2, 0.0, 1e-6, 3.0])
def test_attend_scales_of_scores(new, wide, scale):
    attend_case(Cache([new, 2], [200, 30], 8, 2, 64, BF, wide), 100, 2, scale=scale)


@pytest.mark.parametrize("new", [1, 5, 40])
@pytest.mark.parametrize("exps", [(-60, -55), (50, 60), (-30, 10), (-89, -80), (90, 105)])
def test_attend_page_scales(new, exps):
    """Scales far from 1 and far from one another; q is made to fit K's."""
    b = Cache([new], [300], 8, 2, 128, BF, exps=exps, seed=5)
    b.scales_cpu[:, 0] = 127 - 6 + (b.scales_cpu[:, 0] % 3)
    b.to(DEV)
    attend_case(b)
    attend_case(b, 64, 17)


def test_attend_all_scale_bytes_of_k():
    """Scores of scales down to 2^-127 vanish, and those of large ones decide."""
    b = Cache([1, 40], [256, 300], 4, 1, 64, BF)
    b.scales_cpu[1, 0] = torch.arange(b.num_blocks, dtype=torch.uint8)[:, None] % 122
    b.to(DEV)
    attend_case(b)


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("kv", [0, 1])
def test_attend_scale_of_nan(new, kv):
    """A NaN scale makes every row that sees its page NaN, in that KV head alone."""
    b = Cache([new, 1], [300, 40], 8, 2, 64, BF)
    want = run_attend(b, 20, 0)[0]
    b.scales_d[1, kv, int(b.table[0, 290 // 16]), 1] = 255
    got, l = run_attend(b, 20, 0)
    assert bool(got[:new, 4:].isnan().all(-1)[-1].all()) and bool(got[new - 1, 4:].isnan().all())
    same = torch.ones(b.tokens, 8, dtype=torch.bool)
    same[:new, 4:] = False
    assert torch.equal(got[same].view(torch.int16), want[same].view(torch.int16))


@pytest.mark.parametrize("new", [1, 5, 40])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_attend_far_scores(new, dtype):
    """One key far above all others, first or last, and rows of very large and very small q."""
    for at in (0, 150, 255):
        b = Cache([new], [256 + new - 1], 8, 2, 64, dtype, wide=True, seed=7)
        flat = b.pool_cpu[1].view(2, -1, 2, 64)
        flat[0, b.slots(0)[at]] *= 30
        b.q_cpu[:, 1] *= 40
        b.q_cpu[:, 2] *= 2.0 ** -10
        b.to(DEV)
        attend_case(b)
    b = Cache([new], [256], 8, 2, 64, dtype, seed=7)
    b.q_cpu[:, 1] *= 2.0 ** -10
    b.q_cpu[:, 2] = 0
    b.q_cpu[:, 3, 1:] *= 2.0 ** -9
    if dtype == BF:
        b.q_cpu[:, 4] *= 2.0 ** -50
    b.to(DEV)
    attend_case(b)


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("wide", [False, True])
def test_attend_strides_and_alignment(new, wide):
    """Rows of q and out at odd addresses, heads before tokens, strides below zero; the same bits."""
    b = Cache([new, 2], [90, 33], 6, 2, 64, BF, wide)
    want, want_l = run_attend(b, 30, 2)
    t, h, d = b.tokens, b.heads, b.dim
    for offset in (1, 2, 8):
        q = torch.empty(t * h * d + offset, dtype=BF, device=DEV)[offset:].view(h, t, d).transpose(0, 1)
        o = torch.empty(t * (h * d + 5) + offset, dtype=BF, device=DEV)[offset:].view(t, h * d + 5)[:, :h * d].view(t, h, d)
        q.copy_(b.q)
        out, l = run_attend(b, 30, 2, q=q, out=o)
        assert torch.equal(out, want) and torch.equal(l, want_l)
    assert torch.equal(run_attend(b, 30, 2, lse=False)[0], want)


@pytest.mark.parametrize("new", [1, 40])
def test_attend_values_that_are_not_finite(new):
    """They stay with the rows that see them (one new token a request), or with their request."""
    b = Cache([new, new], [300, 300], 8, 2, 64, BF, wide=True)
    want = run_attend(b, 50, 2)[0]
    flat = b.pool.layers[1].view(2, -1, 2, 64)
    flat[1, b.slots(0)[299], 1, 3] = math.inf
    flat[0, b.slots(0)[298], 0, 3] = math.nan
    got = run_attend(b, 50, 2)[0]
    assert torch.equal(got[new:].view(torch.int16), want[new:].view(torch.int16))
    assert bool((got[new - 1, 4:, 3] == math.inf).all()) and bool(got[new - 1, :4].isnan().all())


def test_attend_repeated_and_two_streams():
    """The same bits again, and from two calls side by side with workspaces of their own."""
    bs = [Cache([60, 1, 3], [700, 3000, 90], 8, 2, 128, BF, seed=s) for s in (1, 2)]
    want = [run_attend(b, 500, 4) for b in bs]
    streams = [torch.cuda.Stream() for _ in bs]
    wss = [torch.empty(pkg.attend_window_workspace_bytes(b.pool, 8, b.tokens, 3, 60, 3000), dtype=torch.uint8, device=DEV) for b in bs]
    for _ in range(3):
        outs = []
        torch.cuda.synchronize()
        for b, s, ws in zip(bs, streams, wss):
            out, l = torch.empty_like(b.q), torch.empty((b.tokens, 8), device=DEV)
            s.wait_stream(torch.cuda.current_stream())
            pkg.check(pkg.attend_layer_window(b.pool, 1, b.q, out, b.q_start_d, b.kv_len_d, b.table_d, b.scale, ws, 500, 4, l,
                                              max_new=60, max_kv_len=3000, stream=s))
            outs.append((out, l))
        torch.cuda.synchronize()
        for (o, l), (wo, wl) in zip(outs, want):
            assert torch.equal(o, wo) and torch.equal(l, wl)


def test_attend_one_workspace_serves_smaller_batches():
    big = Cache([130, 30, 1], [900, 40, 9], 8, 2, 64, BF)
    n = pkg.attend_window_workspace_bytes(big.pool, 8, 161, 3, 130, 900)
    ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV)
    for new, kv in (([130, 30, 1], [900, 40, 9]), ([1, 1, 1], [900, 800, 7]), ([16, 2], [50, 900]), ([1], [1])):
        attend_case(Cache(new, kv, 8, 2, 64, BF), ws=ws)


def test_attend_captured_follows_the_lengths():
    b = Cache([1, 1, 40], [200, 31, 90], 8, 2, 64, BF)
    n = pkg.attend_window_workspace_bytes(b.pool, 8, 42, 3, 40, 208)
    ws = [torch.empty(n, dtype=torch.uint8, device=DEV) for _ in range(2)]
    out, l = torch.empty_like(b.q), torch.empty((42, 8), device=DEV)
    go = lambda o, ll, w: pkg.check(pkg.attend_layer_window(
        b.pool, 1, b.q, o, b.q_start_d, b.kv_len_d, b.table_d, b.scale, w, 64, 4, ll, max_new=40, max_kv_len=208, status=b.status))
    go(out, l, ws[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(out, l, ws[0])
    for kv in ([200, 31, 90], [3, 30, 40], [150, 1, 77]):
        b.kv_len_d.copy_(torch.tensor(kv, dtype=torch.int32))
        graph.replay()
        o, ll = torch.empty_like(out), torch.empty_like(l)
        go(o, ll, ws[1])
        torch.cuda.synchronize()
        assert torch.equal(out, o) and torch.equal(l, ll) and b.status.item() == 0


# ---- a step of them together ----------------------------------------------

def test_a_step_of_beams_eager_and_captured():
    """Two requests of three beams: fork by parents, grow, append, attend, then free and compact, and attend again: the
    compacted cache gives the same bits; captured and replayed, the same state."""
    page, heads, kv_heads, dim, layers = 16, 8, 2, 64, 2
    new, kv = [1] * 6, [40, 40, 40, 33, 33, 33]
    b = Cache(new, kv, heads, kv_heads, dim, BF, layers=layers, spare=20, seed=9)
    i32 = dict(dtype=torch.int32, device=DEV)
    refs0 = torch.zeros(b.num_blocks, dtype=torch.int32)
    for r in range(6):
        refs0[b.table[r, :-(-kv[r] // page)].long()] += 1
    refs0, start_pool, start_scales = refs0.to(DEV), [l.clone() for l in b.pool.layers], b.scales_d.clone()
    parents = torch.tensor([1, 1, 0, 3, 4, 3], **i32)
    g = torch.Generator().manual_seed(11)
    k, v = (torch.randn((6, kv_heads, dim), generator=g).to(BF).to(DEV) for _ in range(2))
    w = (torch.rand(dim, generator=g) + 0.5).to(DEV)
    rotary = make_rotary(dim)
    cols = b.table.shape[1]
    ws = torch.empty(pkg.pages_workspace_bytes(b.pool, 6), dtype=torch.uint8, device=DEV)
    aws = torch.empty(pkg.attend_window_workspace_bytes(b.pool, heads, 6, 6, 1, cols * page), dtype=torch.uint8, device=DEV)
    s = dict(table=torch.empty((6, cols), **i32), refs=torch.empty(b.num_blocks, **i32), lens=torch.empty(6, **i32),
             map=torch.empty(b.num_blocks, **i32), q=torch.empty_like(b.q), out=torch.empty_like(b.q), again=torch.empty_like(b.q),
             q_start=torch.arange(7, **i32))

    def step():
        pkg.check(pkg.fork_pages(b.pool, b.table_d, b.kv_len_d, parents, refs0, s["table"], s["lens"], s["refs"], ws, b.status))
        grown = s["lens"] + 1
        pkg.check(pkg.resize_pages(b.pool, s["table"], s["lens"], grown, s["refs"], s["table"], s["refs"], ws, b.status))
        pkg.check(pkg.append_layer_normed(b.pool, 1, s["table"], b.q, k, v, s["q"], s["q_start"], grown, rotary, w, w,
                                          status=b.status))
        a = dict(window=32, sinks=2, max_new=1, max_kv_len=cols * page, status=b.status)
        pkg.check(pkg.attend_layer_window(b.pool, 1, s["q"], s["out"], s["q_start"], grown, s["table"], b.scale, aws, **a))
        pkg.check(pkg.compact_pages(b.pool, s["table"], grown, s["refs"], s["table"], s["refs"], s["map"], ws, b.status))
        pkg.check(pkg.attend_layer_window(b.pool, 1, s["q"], s["again"], s["q_start"], grown, s["table"], b.scale, aws, **a))

    def restart():
        for l, l0 in zip(b.pool.layers, start_pool):
            l.copy_(l0)
        b.scales_d.copy_(start_scales)
        torch.cuda.synchronize()
    step()
    torch.cuda.synchronize()
    assert b.status.item() == 0
    assert torch.equal(s["out"], s["again"])
    held = torch.unique(s["table"][s["table"] >= 0])
    assert held.tolist() == list(range(len(held)))                   # no gaps
    assert s["refs"].sum().item() == int((s["table"] >= 0).sum())
    # against the formula: each beam's cache is its parent's and the new token
    want = Cache([1] * 6, [kv[p] + 1 for p in parents.tolist()], heads, kv_heads, dim, BF, layers=layers, seed=9)
    want.num_blocks, want.table = b.num_blocks, s["table"].cpu()
    want.pool_cpu = torch.stack([l.view(torch.uint8).cpu() for l in b.pool.layers])
    want.scales_cpu, want.q_cpu = b.scales_d.cpu(), s["q"].cpu()
    o, _, tol, _ = want.attend(32, 2)
    within(s["out"], o, tol, "out")
    parent_rows = torch.cat([b.rows64(b.slots(p), 0, 0) for p in parents.tolist()])
    child_rows = torch.cat([want.rows64(want.slots(r)[:-1], 0, 0) for r in range(6)])
    scale = torch.cat([want.sizes(want.slots(r)[:-1], 0, 0) for r in range(6)])[:, None]
    assert bool(((parent_rows - child_rows).abs() <= torch.maximum(parent_rows.abs() * 2.0 ** -4, scale * 2.0 ** -18)).all())
    eager = {n: t.clone() for n, t in s.items()}
    pool, scales = [l.clone() for l in b.pool.layers], b.scales_d.clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for _ in range(2):
        restart()
        graph.replay()
        torch.cuda.synchronize()
        assert b.status.item() == 0
        for n in eager:
            assert torch.equal(eager[n].view(torch.int16) if eager[n].dtype == BF else eager[n],
                               s[n].view(torch.int16) if s[n].dtype == BF else s[n]), n
        for l, l1 in zip(b.pool.layers, pool):
            assert torch.equal(l.view(torch.uint8), l1.view(torch.uint8))
        assert torch.equal(b.scales_d, scales)


def test_python_refusals():
    b = Cache([1], [20], 4, 2, 64, BF)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    out, f32 = torch.empty_like(b.q), torch.zeros((1, 4, 64), device=DEV)
    bare = pkg.Pool(b.pool.layers, 2, 64)
    a = (b.q_start_d, b.kv_len_d, b.table_d, b.scale, ws)
    with pytest.raises(ValueError, match="scales"):
        pkg.attend_layer_window(bare, 1, b.q, out, *a)
    with pytest.raises(ValueError, match="bfloat16 or float16"):
        pkg.attend_layer_window(b.pool, 1, f32, out, *a)
    with pytest.raises(ValueError, match="out must"):
        pkg.attend_layer_window(b.pool, 1, b.q, f32, *a)
    with pytest.raises(ValueError, match="scale"):
        scores = torch.zeros((1, 2, 32), device=DEV)
        keep = torch.zeros((1, 2, 4), dtype=torch.int32, device=DEV)
        pkg.evict_layer(b.pool, 1, b.table_d, b.kv_len_d, scores, 1, 1, keep, b.kv_len_d.clone())
    with pytest.raises(ValueError, match="one tensor of scales"):
        pkg.Pool(b.pool.layers, 2, 64, scales=list(b.scales_d)[:1])
    with pytest.raises(ValueError, match="float8_e8m0fnu"):
        pkg.Pool(b.pool.layers, 2, 64, scales=[t.float() for t in b.scales_d])
    with pytest.raises(ValueError, match="e4m3"):
        pkg.Pool([l.view(torch.int8) for l in b.pool.layers], 2, 64, scales=list(b.scales_d))
    assert pkg.Pool(b.pool.layers, 2, 64, scales=[t.view(E8M0) for t in b.scales_d]).scales is not None
