"""The attention-side operators where bounds, roundings and values are at their edges."""
import math

import pytest
import torch

import paged_kv_cache_lmkv_gb300 as pkg
from paged_kv_cache_lmkv_gb300 import lmkv
from gpu_util import require_gpu
from operator_util import DEV, HALF_STEP, TINY, Batch, within

pytestmark = pytest.mark.gpu
BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(autouse=True)
def gpu():
    require_gpu()


def attend(b, max_new=None, max_kv=None, ws=None):
    """One call with every row of out and lse at 7 before it: (out, lse)."""
    max_new = max(b.new + [0]) if max_new is None else max_new
    max_kv = max(b.kv + [0]) if max_kv is None else max_kv
    if ws is None:
        n = pkg.attend_workspace_bytes(b.pool, b.heads, b.tokens, len(b.new), max_new, b.prefix, max_kv)
        ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)
    out = torch.full(b.q.shape, 7.0, dtype=b.dtype, device=DEV)
    lse = torch.full((b.tokens, b.heads), 7.0, device=DEV)
    pkg.check(pkg.attend_layer(b.pool, b.layer, b.q, out, b.q_start_d, b.kv_len_d, b.table_d, b.scale, ws,
                               prefix_table=b.prefix_table_d, prefix_len=b.prefix, lse=lse, max_new=max_new,
                               max_kv_len=max_kv, status=b.status))
    return out, lse


# ---- scores far from zero -------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("new,kv,prefix", [([1, 2], [60, 900], 30), ([1, 70], [60, 90], 300)])
def test_attend_keys_near_the_lowest_value(dtype, new, kv, prefix):
    """Keys whose products are as low as fp32 has room for weigh nothing beside others; a row that sees only
    such keys, all alike, takes the mean of their values."""
    b = Batch(new, kv, 4, 2, 64, dtype, prefix=prefix)
    b.q_cpu.copy_(b.q_cpu.abs() + 1)
    b.q.copy_(b.q_cpu)
    assert float(b.q_cpu.max()) < 16
    # 64 products with |q| < 16 stay below the largest fp32 number
    low = torch.tensor(torch.finfo(dtype).min / (4096 if dtype == BF else 1)).to(dtype)
    for x in (b.pool_cpu[1], b.pool.layers[1]):
        k = x.view(2, -1, 128)[0]
        k[b.prefix_slots()] = low.to(x.device)      # the prefix, every other key of the first request,
        k[b.slots(0)[::2]] = low.to(x.device)
        k[b.slots(1)] = low.to(x.device)            # and all keys of the second
    out, lse = attend(b)
    torch.cuda.synchronize()
    assert b.status.item() == 0
    step, lo = HALF_STEP[dtype], int(b.q_start[1])
    # the other requests' rows see equal scores, which make every weight exactly 1
    vis = torch.cat((torch.ones((new[1], prefix), dtype=torch.bool), b.visible(1)), 1).double()
    for h in range(2):
        k, v = b.rows64(b.slots(0)[1::2], h, 0), b.rows64(b.slots(0)[1::2], h, 1)
        v1 = torch.cat((b.rows64(b.prefix_slots(), h, 1), b.rows64(b.slots(1), h, 1)))
        count = vis.sum(1, keepdim=True)
        mean, size = vis @ v1 / count, vis @ v1.abs() / count
        for a in (2 * h, 2 * h + 1):
            q = b.q_cpu[0, a].double()
            x = k @ q * b.scale
            p = torch.softmax(x, 0)
            # as Batch.attend counts: 64 products a score, the sum of 30 weights, each weight's half step
            dx = 72 * 2.0 ** -23 * float((k.abs() @ q.abs()).max()) * b.scale
            tol = (1.01 * step + 2 * dx + 46 * 2.0 ** -23 + 2.0 ** -21) * (p @ v.abs()) + 1.01 * step * (p @ v).abs() + \
                (30 * 2.0 ** -25 * float(v.abs().max()) if dtype == FP else 0.0)
            within(out[0, a], p @ v, tol, "others beside them")
            want = torch.logsumexp(x, 0)
            within(lse[0, a], want, dx + 46 * 2.0 ** -23 + 2.0 ** -21 * (1 + want.abs()), "their lse")
            within(out[lo:, a], mean, 1.01 * step * mean.abs() + (count + 16) * 2.0 ** -23 * size + TINY[dtype], "mean")


# ---- values that are not finite -----------------------------------------

def call_time(b):
    """Shortest time of five calls, ms."""
    n = pkg.attend_workspace_bytes(b.pool, b.heads, b.tokens, len(b.new), max(b.new), b.prefix, max(b.kv))
    ws, out, times = torch.empty(n, dtype=torch.uint8, device=DEV), torch.empty_like(b.q), []
    for _ in range(6):
        first, last = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        first.record()
        pkg.check(pkg.attend_layer(b.pool, 1, b.q, out, b.q_start_d, b.kv_len_d, b.table_d, b.scale, ws,
                                   prefix_table=b.prefix_table_d, prefix_len=b.prefix, max_new=max(b.new),
                                   max_kv_len=max(b.kv)))
        last.record()
        torch.cuda.synchronize()
        times.append(first.elapsed_time(last))
    return min(times[1:])


def test_attend_one_bad_value_does_not_stall_the_batch():
    """Rows that share a tile with a request whose values are not finite are taken again sixteen at a time, at
    six times the clean call's cost here (a row a warp: 144 times)."""
    b = Batch([70, 70, 70, 30], [200, 300, 70, 90], 16, 2, 128, BF, prefix=12000)
    clean = call_time(b)
    b.pool.layers[1].view(2, -1, 256)[1, b.slots(1)[0]] = math.nan
    bad = call_time(b)
    assert bad < 20 * clean, (clean, bad)


@pytest.mark.parametrize("scale", [None, -0.25, 0.0])
@pytest.mark.parametrize("dtype,dim,prefix,new,kv", [
    (BF, 128, 3000, [34, 3, 0, 40, 90], [60, 50, 9, 400, 90]),          # parts of the prefix, small requests between
    (FP, 64, 0, [70, 66, 1, 100], [70, 300, 5, 1200]), (BF, 64, 40, [64, 3, 65], [64, 900, 2000])])
def test_attend_bad_values_in_parts(dtype, dim, prefix, new, kv, scale):
    """Infinite and NaN values of one request, in its first and its last page, and a block that is not there."""
    b = Batch(new, kv, 8, 2, dim, dtype, prefix=prefix, page=16)
    b.scale = b.scale if scale is None else scale
    r = len(new) - 1
    flat = b.pool.layers[1].view(2, -1, 2 * dim)
    flat[1, b.slots(r)[0]] = math.inf
    flat[1, b.slots(r)[kv[r] - new[r]], dim + 3] = math.nan
    table = b.table_d.clone()
    table[0, 1] = -1
    b.table_d = table
    out, lse = attend(b)
    torch.cuda.synchronize()
    assert b.status.item() == lmkv.ERR_BAD_BLOCK

    def hide(i, n):
        return torch.arange(n) // 16 == 1 if i == 0 else torch.zeros(n, dtype=torch.bool)
    want, want_l, tol, tol_l = b.attend(hide)
    within(lse, want_l, tol_l, "lse")
    at = int(b.q_start[r])
    within(out[:at], want[:at], tol[:at], "the others")
    assert not bool(out[at:, 4:].isfinite().all(-1).any()) and not bool(out[at:, :4].isfinite().any())


# ---- bounds of no cached tokens -----------------------------------------

@pytest.mark.parametrize("new,kv,prefix", [
    ([1, 2], [40, 50], 0), ([1, 2], [40, 50], 20), ([0, 1], [40, 0], 20), ([70, 0], [0, 40], 0),
    ([70, 0], [0, 40], 300), ([70, 0], [0, 40], 3000), ([1] * 80, [0] * 79 + [3], 20011), ([1, 1], [0, -4], 20)])
def test_attend_bound_of_no_cached_tokens(new, kv, prefix):
    """Cached tokens beyond a bound of 0 are reported, of requests without new tokens too, and not attended to."""
    b = Batch(new, [max(n, 0) for n in kv], 8, 2, 64, BF, prefix=prefix)
    b.kv_len_d = torch.tensor(kv, dtype=torch.int32, device=DEV)
    out, lse = attend(b, max_kv=0)
    torch.cuda.synchronize()
    assert b.status.item() == lmkv.ERR_BAD_LENGTH
    want, want_l, tol, tol_l = b.attend(lambda r, n: torch.full((n,), r is not None))
    within(out, want, tol, "out")
    within(lse, want_l, tol_l, "lse")


def test_attend_bound_of_no_cached_tokens_kept():
    b = Batch([1, 70, 0], [0, 0, 0], 8, 2, 64, BF, prefix=90)
    out, lse = attend(b, max_kv=0)
    torch.cuda.synchronize()
    assert b.status.item() == 0
    want, want_l, tol, tol_l = b.attend()
    within(out, want, tol, "out")
    within(lse, want_l, tol_l, "lse")


def weigh(b, lse, scores, out, decay=1.0, max_new=None, max_kv=None):
    pkg.check(pkg.weigh_layer(b.pool, b.layer, b.q, lse, b.q_start_d, b.kv_len_d, b.table_d, b.scale, scores, out,
                              decay=decay, max_new=max(b.new) if max_new is None else max_new,
                              max_kv_len=max(b.kv) if max_kv is None else max_kv, status=b.status))


@pytest.mark.parametrize("new", [[1, 1], [30, 1], [0, 0]])
def test_weigh_bound_of_no_cached_tokens(new):
    """Cached tokens beyond a bound of 0 are reported, and no score is touched."""
    b = Batch(new, [40, 50], 8, 2, 64, BF, extra_rows=1)
    lse, out = torch.zeros((b.tokens, 8), device=DEV), torch.full((2, 2, 50), 7.0, device=DEV)
    weigh(b, lse, out, out, max_kv=0)
    torch.cuda.synchronize()
    assert b.status.item() == lmkv.ERR_BAD_LENGTH
    assert bool((out == 7.0).all())
    b.status.zero_()
    b.kv_len_d.zero_()
    weigh(b, lse, out, out, max_kv=0)
    torch.cuda.synchronize()
    assert b.status.item() == 0


@pytest.mark.parametrize("max_new", [1, 20])
def test_weigh_lengths_of_requests_without_cached_tokens(max_new):
    """New tokens beyond their bound are reported of a request that has no cached ones too."""
    b = Batch([1, max_new + 1], [40, 0], 8, 2, 64, BF)
    lse, out = torch.zeros((b.tokens, 8), device=DEV), torch.full((2, 2, 40), 7.0, device=DEV)
    weigh(b, lse, None, out, decay=0.0, max_new=max_new)
    torch.cuda.synchronize()
    assert b.status.item() == lmkv.ERR_BAD_LENGTH
    assert bool((out[1] == 7.0).all())


@pytest.mark.parametrize("new", [1, 3])
def test_weigh_many_requests(new):
    n = 150
    b = Batch([new] * n, [(i * 13) % 70 for i in range(n)], 8, 2, 64, BF)
    _, lse, _, _ = b.attend()
    scores = torch.rand((n, 2, 75), generator=torch.Generator().manual_seed(2))
    out = scores.to(DEV)
    weigh(b, lse.float().to(DEV), out, out, decay=0.5)
    torch.cuda.synchronize()
    assert b.status.item() == 0
    want, tol = b.weigh(lse.float(), scores, 0.5)
    for r, m in enumerate(b.kv):
        within(out[r, :, :m], want[r, :, :m], tol[r, :, :m], f"request {r}")
        assert torch.equal(out[r, :, m:].cpu(), scores[r, :, m:])


# ---- rotary -------------------------------------------------------------

@pytest.mark.parametrize("share", [0.25, 0.75])
def test_append_slow_frequencies_at_far_positions(share):
    """A frequency of (1000 + share) 2^-64 turns a position is taken to the nearest 2^-64 of a
    turn, so at position 2^60 its angle is a whole number of sixteenths of a turn."""
    k = 1000 + round(share)
    f = 2 * math.pi * (1000 + share) * 2.0 ** -64
    rotary = pkg.Rotary(64, inv_freq=[f] * 32)
    b = Batch([1], [1], 2, 2, 64, F32)
    x = torch.randn((1, 2, 64), generator=torch.Generator().manual_seed(3))
    q, out = x.to(DEV), torch.empty((1, 2, 64), device=DEV)
    pos = torch.tensor([2 ** 60], dtype=torch.int64, device=DEV)
    pkg.check(pkg.append_layer(b.pool, 1, b.table_d, q, q, q, out, b.q_start_d, b.kv_len_d, rotary, positions=pos,
                               status=b.status))
    torch.cuda.synchronize()
    assert b.status.item() == 0
    t = 2 * math.pi * (k % 16) / 16
    a, c = x.double()[..., :32], x.double()[..., 32:]
    want = torch.cat((a * math.cos(t) - c * math.sin(t), a * math.sin(t) + c * math.cos(t)), -1)
    mag = (a.abs() + c.abs()).repeat(1, 1, 2)
    within(out, want, 2.0 ** -24 * 1.001 * want.abs() + 2.0 ** -21 * mag, "q")


# ---- workspace ----------------------------------------------------------

@pytest.mark.parametrize("prefix,max_kv,calls", [
    (0, 1024, [([200, 250], [300, 1024]), ([64], [700]), ([1, 1, 30], [1000, 5, 30]), ([1], [1])]),
    (0, 3000, [([1, 1, 1], [2900, 5, 30]), ([1, 80], [900, 2000]), ([1], [3000])]),
    (700, 600, [([1] * 6, [40, 3, 600, 1, 1, 90]), ([90, 1], [90, 600]), ([2, 2], [9, 2])])])
def test_attend_workspace_of_the_largest_batch_serves_smaller_ones(prefix, max_kv, calls):
    """One workspace, sized for bounds that no call exceeds."""
    b = Batch([1], [1], 8, 2, 64, BF, prefix=prefix)
    n = pkg.attend_workspace_bytes(b.pool, 8, 8192, 8, 2048, prefix, max_kv)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)
    for new, kv in calls:
        for p in sorted({prefix, prefix // 3}):
            b = Batch(new, kv, 8, 2, 64, BF, prefix=p)
            out, lse = attend(b, ws=ws)
            torch.cuda.synchronize()
            assert b.status.item() == 0
            want, want_l, tol, tol_l = b.attend()
            within(out, want, tol, "out")
            within(lse, want_l, tol_l, "lse")


# ---- strides, ties, repeated calls ----------------------------------------

def test_attend_strides_below_zero():
    """Rows whose tokens and heads lie in falling order, as the C structure can say."""
    b = Batch([1, 40, 2], [30, 41, 900], 8, 2, 64, BF, prefix=50)
    t, d = b.tokens, 64
    q = b.q.flip((0, 1)).contiguous()
    out = torch.full_like(q, 7.0)
    lse = torch.full((t, 8), 7.0, device=DEV)
    n = pkg.attend_workspace_bytes(b.pool, 8, t, 3, 40, 50, 900)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)
    last = 2 * d * (t * 8 - 1)                    # bytes to the last row, which is token 0's head 0
    batch = lmkv._BatchT(b.q_start_d.data_ptr(), b.kv_len_d.data_ptr(), b.table_d.data_ptr(), b.table_d.shape[1], 3, t, 40, 900)
    rows = [bytes(lmkv._RowsT(x.data_ptr() + last, -8 * d, -d)) for x in (q, out)]
    pkg.check(lmkv.load().lmkv_attend_layer(
        b.pool.struct, lmkv.BF16, 1, bytes(batch), 8, rows[0], b.prefix_table_d.data_ptr(), 50, b.scale, rows[1],
        lse.data_ptr(), ws.data_ptr(), n, b.status.data_ptr(), torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    assert b.status.item() == 0
    want, want_l, tol, tol_l = b.attend()
    within(out.flip((0, 1)), want, tol, "out")
    within(lse, want_l, tol_l, "lse")


@pytest.mark.parametrize("new,kv,prefix", [([1, 2], [60, 900], 30), ([1, 70], [60, 90], 300)])
def test_attend_equal_scores(new, kv, prefix):
    """All keys alike: every weight is 1, lse is the score and the logarithm of the count."""
    b = Batch(new, kv, 4, 2, 64, BF, prefix=prefix)
    for x in (b.pool_cpu[1], b.pool.layers[1]):
        k = x.view(2, -1, 128)[0]
        for at in [b.slots(0), b.slots(1), b.prefix_slots()]:
            k[at] = 0.5
    out, lse = attend(b)
    torch.cuda.synchronize()
    want, want_l, tol, tol_l = b.attend()
    within(out, want, tol, "out")
    within(lse, want_l, tol_l, "lse")


@pytest.mark.parametrize("kv,budget,kv_heads", [([64] * 40, 48, 1), ([17] * 300, 16, 1), ([9000, 300, 60000], 2000, 2)])
def test_evict_same_start_same_bits(kv, budget, kv_heads):
    """Calls from one start, again and again: pool, keep, new_len and kept scores have the same bits."""
    b = Batch([0] * len(kv), kv, kv_heads, kv_heads, 64, BF)
    g = torch.Generator().manual_seed(6)
    scores = torch.randint(0, 9, (len(kv), kv_heads, max(kv)), generator=g).float().to(DEV)     # ties all over
    start, first = b.pool.layers[1].clone(), None
    for _ in range(4):
        b.pool.layers[1].copy_(start)
        keep = torch.full((len(kv), kv_heads, budget), 99, dtype=torch.int32, device=DEV)
        new_len = torch.full((len(kv),), 99, dtype=torch.int32, device=DEV)
        kept = torch.full((len(kv), kv_heads, budget), 99.0, device=DEV)
        pkg.check(pkg.evict_layer(b.pool, 1, b.table_d, b.kv_len_d, scores, 2, 3, keep, new_len, kept_scores=kept,
                                  status=b.status))
        torch.cuda.synchronize()
        assert b.status.item() == 0
        now = [keep, new_len, kept, b.pool.layers[1].view(torch.int16).clone()]
        first = now if first is None else first
        for x, y in zip(first, now):
            assert torch.equal(x, y)
    before = start.view(2, -1, kv_heads, 64)
    after = b.pool.layers[1].view(2, -1, kv_heads, 64)
    for r in range(len(kv)):
        at = b.slots(r).to(DEV)
        n = min(kv[r], budget)
        for h in range(kv_heads):
            idx = keep[r, h, :n].long()
            assert torch.equal(after[:, at[:n], h], before[:, at[idx], h])


@pytest.mark.parametrize("scale", [0.125, -0.125])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("new,kv,prefix", [
    ([1, 2], [60, 90], 30), ([1, 70], [60, 90], 300), ([70, 3], [90, 40], 0), ([1, 1], [1500, 40], 50),
    ([1] * 78 + [0, 3], [1 + (i * 17) % 60 for i in range(78)] + [0, 9], 20011)])
def test_attend_one_key_far_above(dtype, new, kv, prefix, scale):
    """A key whose score is near the largest that fp32 has room for is all that its rows see: its value is
    the result, its score lse, whichever kernel comes upon it; other requests' rows are as without it."""
    b = Batch(new, kv, 8, 2, 64, dtype, prefix=prefix)
    b.scale = scale
    b.q_cpu.copy_(b.q_cpu.abs() + 1)
    b.q.copy_(b.q_cpu)
    top = torch.tensor(torch.finfo(dtype).max / (4096 if dtype == BF else 1)).to(dtype)
    top = top if scale > 0 else -top
    in_prefix = prefix > 0
    at = int(b.prefix_slots()[prefix // 2]) if in_prefix else int(b.slots(0)[5])
    for x in (b.pool_cpu[1], b.pool.layers[1]):
        x.view(2, -1, 128)[0, at] = top.to(x.device)
    out, lse = attend(b)
    torch.cuda.synchronize()
    assert b.status.item() == 0
    for r, n in enumerate(new):
        if not in_prefix and r > 0:
            continue
        for i in range(int(b.q_start[r]), int(b.q_start[r + 1])):
            for h in range(2):
                v = b.pool_cpu[1, 1].view(-1, 128)[at, h * 64:(h + 1) * 64]
                for a in range(4 * h, 4 * h + 4):
                    assert torch.equal(out[i, a].cpu(), v), (r, i, a)
            score = b.q_cpu[i].double().sum(-1) * float(top) * scale
            within(lse[i], score, 2.0 ** -18 * score.abs(), "lse")
    if not in_prefix:
        ref = Batch(new, kv, 8, 2, 64, dtype, prefix=prefix)
        ref.scale = scale
        ref.q_cpu.copy_(b.q_cpu)
        want, want_l, tol, tol_l = ref.attend()
        lo = int(b.q_start[1])
        within(out[lo:], want[lo:], tol[lo:], "the others")
        within(lse[lo:], want_l[lo:], tol_l[lo:], "lse of the others")
