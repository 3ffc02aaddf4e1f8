"""The 8-bit cache's operators and pages at the ends of their ranges, against 64-bit formulas."""
import pytest
import torch

import paged_kv_cache_lmkv_gb300 as pkg
from cache8_util import Cache
from gpu_util import require_gpu
from paged_kv_cache_lmkv_gb300 import lmkv
from test_gpu_cache8 import attend_case, run_attend

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(autouse=True)
def gpu():
    require_gpu()


@pytest.mark.parametrize("new,heads", [(8, 2), (8, 8), (70, 8)])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("window", [2 ** 30, 2 ** 31 - 12, 2 ** 31 - 3, 2 ** 31 - 2, 2 ** 31 - 1])
def test_attend_windows_that_end_near_32_bits(new, heads, wide, window):
    """They take in every key, of requests with fewer cached tokens than new ones too, whose first rows have
    tokens before the cache's first."""
    b = Cache([new, 2], [new - 5, 40], heads, 2, 64, BF, wide)
    out, lse = attend_case(b, window, 0)
    want, want_l = attend_case(b)
    assert torch.equal(out, want) and torch.equal(lse, want_l)
    attend_case(b, window, 3)


@pytest.mark.parametrize("wide", [False, True])
def test_a_beam_goes_back_into_a_page_that_it_shares(wide):
    """Two beams of 40 tokens share two full pages; the second goes back to 20.  Its last page is then the first's full one,
    until a fork of all rows by their own numbers gives it one of its own, which it may append to."""
    page, dim, heads = 16, 64, 2
    b = Cache([1], [40], heads, heads, dim, BF, wide, page, spare=8, layers=1, layer=0, seed=4)
    i32 = dict(dtype=torch.int32, device=b.device)
    refs = torch.zeros(b.num_blocks, **i32)
    refs[b.table_d[0, :3].long()] = 1
    cols = b.table.shape[1]
    ws = torch.empty(pkg.pages_workspace_bytes(b.pool, 2), dtype=torch.uint8, device=b.device)
    bits = torch.int16 if wide else torch.uint8

    def fork(table, lens, parents):
        out, n = torch.empty((2, cols), **i32), torch.empty(2, **i32)
        pkg.check(pkg.fork_pages(b.pool, table, lens, torch.tensor(parents, **i32), refs, out, n, refs, ws, b.status))
        return out, n

    def resize(table, lens, to):
        to = torch.tensor(to, **i32)
        pkg.check(pkg.resize_pages(b.pool, table, lens, to, refs, table, refs, ws, b.status))
        return to

    def of_row(row, n):
        """Bits of a row's tokens, and its pages' scales."""
        j = torch.arange(n, device=b.device)
        slots = table[row].long()[j // page] * page + j % page
        rows = b.pool.layers[0].view(bits).view(2, -1, heads * dim)[:, slots].clone()
        return rows, None if wide else b.scales_d[0][:, table[row, :-(-n // page)].long()].clone()

    table, lens = fork(b.table_d, b.kv_len_d, [0, 0])
    assert table[0, :2].tolist() == table[1, :2].tolist() and refs[table[0, 1]] == 2
    lens = resize(table, lens, [40, 20])
    assert refs[table[1, 1]] == 2                   # a last page, not full, that another row holds too
    first, second = of_row(0, 40), of_row(1, 20)
    table, lens = fork(table, lens, [0, 1])
    for r, n in enumerate((40, 20)):
        assert refs[table[r, (n - 1) // page]] == 1
    grown = resize(table, lens, [41, 21])
    g = torch.Generator().manual_seed(5)
    q, k, v = ((torch.randn((2, heads, dim), generator=g) * 1000).to(BF).to(b.device) for _ in range(3))
    pkg.check(pkg.append_layer_normed(b.pool, 0, table, q, k, v, q, torch.arange(3, **i32), grown, status=b.status))
    torch.cuda.synchronize()
    assert b.status.item() == 0
    got = of_row(0, 32)                             # the pages that the append does not write to
    assert torch.equal(got[0], first[0][:, :32]) and (wide or torch.equal(got[1], first[1][:, :2]))
    got = of_row(1, 16)
    assert torch.equal(got[0], second[0][:, :16]) and (wide or torch.equal(got[1], second[1][:, :1]))
    if wide:
        assert torch.equal(of_row(0, 40)[0], first[0]) and torch.equal(of_row(1, 20)[0], second[0])
        assert torch.equal(of_row(1, 21)[0][1, 20], v[1].view(torch.int16).flatten())
    else:                                           # the last pages' earlier codes, to the new token's scale
        now, then = of_row(1, 20), second
        assert bool((now[1][:, 1] > then[1][:, 1]).all())
        code = lambda x: x.view(torch.float8_e4m3fn).double().view(2, -1, heads, dim)
        value = lambda x, s: code(x[:, 16:20]) * torch.exp2(s[:, 1].double() - 127)[:, None, :, None]
        step = torch.exp2(now[1][:, 1].double() - 127 - 10)[:, None, :, None]
        a, z = value(*then), value(*now)
        assert bool(((a - z).abs() <= torch.maximum(a.abs() * 2.0 ** -4, step)).all())


@pytest.mark.parametrize("new", [1, 5, 40])
@pytest.mark.parametrize("large", [0, 1, 2])
def test_attend_scales_of_v_that_differ_by_2_to_the_64(new, large):
    """Pages of 2^-24 beside pages of 2^40, every second page or one of them; scores alike, and far in favour of a page of
    small values."""
    b = Cache([new], [300], 8, 2, 128, BF, seed=5)
    pages = b.table[0, :19].long()
    b.scales_cpu[:, 0] = 127 - 7                    # (of K)
    b.scales_cpu[:, 1] = 127 - 24
    b.scales_cpu[:, 1, pages[::2] if large == 0 else pages[3 * large]] = 127 + 40
    b.to(b.device)
    attend_case(b)
    attend_case(b, 64, 17)
    if large:
        flat = b.pool_cpu[1, 0].view(-1, 2, 128)
        flat[b.slots(0)[[5, 290]]] = (b.q_cpu[:, ::4].float().mean(0) * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        b.to(b.device)
        attend_case(b)


def back_to_front(x):
    """Rows of a copy of x [tokens][heads][dim] laid out last token and last head first, and that copy."""
    store = x.flip(0, 1).contiguous()
    t, h, d = x.shape
    return lmkv._RowsT(store.data_ptr() + (t * h - 1) * d * x.element_size(), -h * d, -d), store


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("wide", [False, True])
def test_attend_strides_below_zero(new, wide):
    b = Cache([new, 2], [90, 33], 6, 2, 64, BF, wide)
    want, want_l = run_attend(b, 30, 2)
    q, q_store = back_to_front(b.q)
    out, out_store = back_to_front(torch.zeros_like(b.q))
    lse = torch.zeros_like(want_l)
    n = pkg.attend_window_workspace_bytes(b.pool, 6, b.tokens, 2, new if new > 2 else 2, 90)
    ws = torch.empty(n, dtype=torch.uint8, device=b.device)
    batch, _ = lmkv._batch(b.pool, ws.get_device(), b.table_d, b.q_start_d, b.kv_len_d, b.tokens, max(new, 2), 90)
    pkg.check(lmkv.load().lmkv_attend_layer_window(
        b.pool.struct, None if wide else b.pool.scale_ptrs.data_ptr(), lmkv.BF16, 1, batch, 6, bytes(q), b.scale, 30, 2,
        bytes(out), lse.data_ptr(), ws.data_ptr(), n, b.status.data_ptr(), torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    assert b.status.item() == 0
    assert torch.equal(out_store.flip(0, 1), want) and torch.equal(lse, want_l)


@pytest.mark.parametrize("rot", [0, 34, 64])
@pytest.mark.parametrize("wide", [False, True])
def test_append_strides_below_zero(rot, wide):
    """The same bits in the pages and in q_out."""
    bs = [Cache([3, 20], [9, 41], 4, 2, 64, BF, wide, seed=8) for _ in range(2)]
    g = torch.Generator().manual_seed(9)
    q, k, v = (torch.randn((23, h, 64), generator=g).to(BF).to(bs[0].device) for h in (4, 2, 2))
    norm = (torch.rand(64, generator=g) + 0.5).to(q.device)
    rotary = pkg.Rotary(rot) if rot else None
    want = torch.zeros_like(q)
    b = bs[0]
    pkg.check(pkg.append_layer_normed(b.pool, 1, b.table_d, q, k, v, want, b.q_start_d, b.kv_len_d, rotary, norm, norm,
                                      status=b.status))
    b = bs[1]
    rows = [back_to_front(x) for x in (q, k, v, torch.zeros_like(q))]
    batch, _ = lmkv._batch(b.pool, q.get_device(), b.table_d, b.q_start_d, b.kv_len_d, 23, None, None)
    pkg.check(lmkv.load().lmkv_append_layer_normed(
        b.pool.struct, None if wide else b.pool.scale_ptrs.data_ptr(), lmkv.BF16, 1, batch, 4, *(bytes(r) for r, _ in rows), None,
        None if rotary is None else rotary.struct, norm.data_ptr(), norm.data_ptr(), 1e-6, b.status.data_ptr(),
        torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    assert bs[0].status.item() == 0 and b.status.item() == 0
    assert torch.equal(rows[3][1].flip(0, 1), want)
    for x, y in zip(bs[0].pool.layers, b.pool.layers):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert wide or torch.equal(bs[0].scales_d, b.scales_d)


@pytest.mark.parametrize("wide", [False, True])
def test_pages_beyond_32_bits_of_bytes(wide):
    """A layer whose halves have more than 2^32 bytes each, with pages at their ends: append, attention (few rows and
    tiles), copies and forks give the bits that they give in a small pool."""
    page, heads, kv_heads, dim = 16, 16, 8, 128
    small = Cache([1, 40, 3], [300, 200, 35], heads, kv_heads, dim, BF, wide, page, layers=1, layer=0, spare=6, seed=6)
    size = 2 if wide else 1
    blocks = 2 ** 32 // (page * kv_heads * dim * size) + 5000
    dev = small.device
    where = blocks - 1 - 7 * torch.arange(small.num_blocks, device=dev)        # of the small pool's pages
    layer = torch.empty((2, blocks, page, kv_heads * dim), dtype=BF if wide else torch.uint8, device=dev)
    bits = torch.int16 if wide else torch.uint8
    layer[:, where] = small.pool.layers[0].view(layer.dtype)
    scales = None
    if not wide:
        scales = torch.full((2, blocks, kv_heads), 255, dtype=torch.uint8, device=dev)
        scales[:, where] = small.scales_d[0]
    big = pkg.Pool([layer], kv_heads, dim, scales=None if wide else [scales])
    far = torch.where(small.table_d >= 0, where[small.table_d.long().clamp(min=0)], -1).to(torch.int32)

    def same():
        torch.cuda.synchronize()
        assert small.status.item() == 0
        assert torch.equal(layer[:, where].view(bits), small.pool.layers[0].view(bits))
        assert wide or torch.equal(scales[:, where], small.scales_d[0])

    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn((44, kv_heads, dim), generator=g).to(BF).to(dev) for _ in range(2))
    rotary = pkg.Rotary(dim)
    got = []
    for pool, table in ((small.pool, small.table_d), (big, far)):
        q = torch.empty_like(small.q)
        pkg.check(pkg.append_layer_normed(pool, 0, table, small.q, k, v, q, small.q_start_d, small.kv_len_d, rotary,
                                          status=small.status))
        n = pkg.attend_window_workspace_bytes(pool, heads, 44, 3, 40, 300)
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
        for window in (0, 33):
            out, lse = torch.empty_like(q), torch.empty((44, heads), device=dev)
            pkg.check(pkg.attend_layer_window(pool, 0, q, out, small.q_start_d, small.kv_len_d, table, small.scale, ws, window,
                                              2, lse, max_new=40, max_kv_len=300, status=small.status))
            got.append((q, out, lse))
    same()
    for a, b in zip(got[:2], got[2:]):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    # forks copy the last pages: from and to the far end
    parents = torch.tensor([0, 0, 1, 2, 2], dtype=torch.int32, device=dev)
    lens = torch.empty(5, dtype=torch.int32, device=dev)
    rows = []
    for pool, table, held in ((small.pool, small.table_d, torch.zeros(small.num_blocks, dtype=torch.int32, device=dev)),
                              (big, far, torch.full((blocks,), -1, dtype=torch.int32, device=dev))):
        if pool is big:
            held[where] = 0
        held[table[table >= 0].long()] = 1
        out = torch.empty((5, table.shape[1]), dtype=torch.int32, device=dev)
        ws = torch.empty(pkg.pages_workspace_bytes(pool, 5), dtype=torch.uint8, device=dev)
        pkg.check(pkg.fork_pages(pool, table, small.kv_len_d, parents, held, out, lens, held, ws, small.status))
        torch.cuda.synchronize()
        rows.append([pool.layers[0].view(bits).view(2, -1, kv_heads * dim)[:, s] for s in (
            (t.long()[j // page] * page + j % page) for t, j in zip(out, (torch.arange(int(n), device=dev) for n in lens)))])
    assert small.status.item() == 0
    assert all(torch.equal(a, b) for a, b in zip(*rows))
    free = (held == 0).nonzero()[:2, 0].to(torch.int32)
    src = far[0, :2].contiguous()
    pkg.check(pkg.copy_pages(big, src, free, small.status))
    torch.cuda.synchronize()
    assert torch.equal(layer[:, free.long()].view(bits), layer[:, src.long()].view(bits)) and small.status.item() == 0
