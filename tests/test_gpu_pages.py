"""Pages copied, forked, resized and compacted on the device against a model of them in Python."""
import numpy as np
import pytest
import torch

import paged_kv_cache_lmkv_gb300 as pkg
from paged_kv_cache_lmkv_gb300 import lmkv
from gpu_util import require_gpu
from operator_util import DEV

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


@pytest.fixture(autouse=True)
def gpu():
    require_gpu()


class Model:
    """Tables, references and the pages' bytes as numpy arrays; what the calls say, step by step."""

    def __init__(self, table, lens, refs, pool, scales, page):
        self.table, self.lens, self.refs = table.copy(), lens.copy(), refs.copy()
        self.pool, self.scales, self.page, self.status = pool.copy(), None if scales is None else scales.copy(), page, 0

    def ok(self, i):
        if 0 <= i < len(self.refs):
            return True
        self.status = self.status or lmkv.ERR_BAD_BLOCK
        return False

    def clamp(self, lens):
        most = self.table.shape[1] * self.page
        out = np.clip(lens, 0, most)
        if (out != lens).any():
            self.status = self.status or lmkv.ERR_BAD_LENGTH
        return out

    def pages(self, n):
        return -(-int(n) // self.page)

    def add(self, i, by):
        if self.ok(i) and self.refs[i] >= 0:
            self.refs[i] += by

    def take(self):
        free = np.nonzero(self.refs == 0)[0]
        if len(free) == 0:
            self.status = self.status or lmkv.ERR_NO_PAGES
            return -1
        self.refs[free[0]] = 1
        return int(free[0])

    def copy(self, src, dst, tokens):
        self.pool[:, :, dst, :tokens] = self.pool[:, :, src, :tokens]
        if self.scales is not None:
            self.scales[:, :, dst] = self.scales[:, :, src]

    def fork(self, parents):
        lens = self.clamp(self.lens)
        for row, n in zip(self.table, lens):
            for c in range(self.pages(n)):
                self.add(row[c], -1)
        out, new_lens, part = [], [], {}
        for i, p in enumerate(parents):
            row, n = np.full(self.table.shape[1], -1, np.int32), 0
            if 0 <= p < len(lens):
                n = int(lens[p])
                row[:self.pages(n)] = self.table[p][:self.pages(n)]
            for c in range(n // self.page):
                self.add(row[c], 1)
            out.append(row)
            new_lens.append(n)
        want = []
        for i, (row, n) in enumerate(zip(out, new_lens)):
            if n % self.page == 0 or not self.ok(row[n // self.page]):
                continue
            src = int(row[n // self.page])
            if part.setdefault(src, i) == i and self.refs[src] == 0:
                self.refs[src] = 1
            else:
                want.append((i, src, n))
        for i, src, n in want:
            dst = self.take()
            out[i][n // self.page] = dst
            if dst >= 0:
                self.copy(src, dst, n % self.page)
        self.table = np.stack(out) if out else np.zeros((0, self.table.shape[1]), np.int32)
        self.lens = np.array(new_lens, np.int32)

    def resize(self, new_lens):
        lens, new = self.clamp(self.lens), self.clamp(new_lens)
        for row, a, z in zip(self.table, lens, new):
            for c in range(self.pages(z), self.pages(a)):
                self.add(row[c], -1)
            row[min(self.pages(a), self.pages(z)):] = -1
        for row, a, z in zip(self.table, lens, new):
            for c in range(self.pages(a), self.pages(z)):
                row[c] = self.take()
        self.lens = new

    def compact(self):
        where = np.arange(len(self.refs), dtype=np.int32)
        gaps, held = np.nonzero(self.refs == 0)[0], np.nonzero(self.refs > 0)[0][::-1]
        for to, src in zip(gaps, held):
            if to >= src:
                break
            self.copy(src, to, self.page)
            self.refs[to], self.refs[src] = self.refs[src], 0
            where[src] = to
        for row, n in zip(self.table, self.clamp(self.lens)):
            for c in range(self.pages(n)):
                if self.ok(row[c]):
                    row[c] = where[row[c]]
            row[self.pages(n):] = -1
        return where


class State:
    """The same on the device."""

    def __init__(self, lens, shared=0, page=16, layers=3, kv_heads=2, dim=64, spare=10, bits=8, cols=None, seed=0, groups=1):
        rng = np.random.default_rng(seed)
        lens = np.asarray(lens, np.int32)
        need = [-(-int(n) // page) for n in lens]
        cols = max(need + [1]) + 2 if cols is None else cols
        self.num_blocks = sum(need) + spare
        ids = rng.permutation(self.num_blocks)
        table, at = np.full((len(lens), cols), -1, np.int32), 0
        for r, n in enumerate(need):
            table[r, :n] = ids[at:at + n]
            at += n
            k = min(shared, n, need[r - r % groups])
            if r % groups:
                table[r, :k] = table[r - r % groups, :k]
        refs = np.bincount(np.concatenate([t[:n] for t, n in zip(table, need)] + [np.zeros(0, np.int64)]).astype(np.int64),
                           minlength=self.num_blocks).astype(np.int32)
        row = kv_heads * dim * (bits // 8)
        pool = rng.integers(0, 256, (layers, 2, self.num_blocks, page, row), dtype=np.uint8)
        scales = rng.integers(0, 256, (layers, 2, self.num_blocks, kv_heads), dtype=np.uint8) if bits == 8 else None
        self.m = Model(table, lens, refs, pool, scales, page)
        d = torch.from_numpy(pool).to(DEV)
        self.layers = list(d.view(E4M3 if bits == 8 else torch.bfloat16 if bits == 16 else torch.float32))
        self.scales = None if scales is None else torch.from_numpy(scales).to(DEV)
        self.pool = pkg.Pool(self.layers, kv_heads, dim, scales=None if scales is None else list(self.scales))
        self.table, self.lens = torch.from_numpy(table).to(DEV), torch.from_numpy(lens).to(DEV)
        self.refs = torch.from_numpy(refs).to(DEV)
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.cols = cols

    def ws(self, rows):
        return torch.full((pkg.pages_workspace_bytes(self.pool, rows),), 255, dtype=torch.uint8, device=DEV)

    def fork(self, parents, in_place=True):
        n = len(parents)
        table = torch.full((n, self.cols), 77, dtype=torch.int32, device=DEV)
        lens = torch.full((n,), 77, dtype=torch.int32, device=DEV)
        refs = self.refs if in_place else torch.empty_like(self.refs)
        p = torch.tensor(parents, dtype=torch.int32, device=DEV)
        pkg.check(pkg.fork_pages(self.pool, self.table, self.lens, p, self.refs, table, lens, refs, self.ws(n), self.status))
        self.table, self.lens, self.refs = table, lens, refs
        self.m.fork(parents)
        self.check()

    def resize(self, lens, in_place=True):
        new = torch.tensor(lens, dtype=torch.int32, device=DEV)
        table = self.table if in_place else torch.full_like(self.table, 77)
        refs = self.refs if in_place else torch.empty_like(self.refs)
        pkg.check(pkg.resize_pages(self.pool, self.table, self.lens, new, self.refs, table, refs, self.ws(len(lens)), self.status))
        self.table, self.refs = table, refs
        self.m.resize(np.asarray(lens, np.int32))
        self.lens = torch.from_numpy(self.m.lens).to(DEV)
        self.check()

    def compact(self, in_place=True):
        table = self.table if in_place else torch.full_like(self.table, 77)
        refs = self.refs if in_place else torch.empty_like(self.refs)
        where = torch.full_like(self.refs, 77)
        pkg.check(pkg.compact_pages(self.pool, self.table, self.lens, self.refs, table, refs, where, self.ws(len(self.lens)),
                                    self.status))
        self.table, self.refs = table, refs
        want = self.m.compact()
        self.check()
        assert where.cpu().numpy().tolist() == want.tolist()

    def check(self):
        torch.cuda.synchronize()
        assert self.status.item() == self.m.status
        assert self.refs.cpu().numpy().tolist() == self.m.refs.tolist()
        assert self.table.cpu().numpy().tolist() == self.m.table.tolist()
        assert self.lens.cpu().numpy().tolist() == self.m.lens.tolist()
        for l, x in zip(self.layers, self.m.pool):
            assert np.array_equal(l.view(torch.uint8).cpu().numpy().reshape(x.shape), x)
        if self.scales is not None:
            assert np.array_equal(self.scales.cpu().numpy(), self.m.scales)


@pytest.mark.parametrize("bits", [8, 16, 32])
@pytest.mark.parametrize("page", [1, 5, 16, 64])
@pytest.mark.parametrize("in_place", [False, True])
def test_fork(bits, page, in_place):
    s = State([40, 40, 40, 33, 33, 33, 0, 16], shared=2, groups=3, page=page, bits=bits)
    s.fork([1, 1, 1, 4, 3, 3, 6, 7], in_place)
    s.fork([0, 2, 1, 5, 5, 5, 7, 7], in_place)


def test_fork_to_more_and_fewer_rows():
    s = State([30, 20], spare=60)
    s.fork([0, 0, 0, 0, 1, 1, 1])
    s.fork([6, 2, 2])
    s.fork([-1, 5, 1])               # no such parents: empty rows
    s.fork([])
    assert int(s.refs.sum()) == 0


def test_fork_of_rows_that_share_their_last_page():
    s = State([20, 20, 20])
    s.m.table[1] = s.m.table[0]
    s.m.refs[:] = np.bincount(s.m.table[s.m.table >= 0], minlength=s.num_blocks)
    s.table, s.refs = torch.from_numpy(s.m.table).to(DEV), torch.from_numpy(s.m.refs).to(DEV)
    s.fork([1, 0, 2])                # one of the first two goes on with the page
    assert int(s.refs.max()) == 2    # only the full page is shared
    s.m.refs[s.m.table[2, 1]] += 1   # held by somebody else: not written to
    s.refs[int(s.m.table[2, 1])] += 1
    s.fork([2, 2, 0])


def test_fork_uses_pages_that_it_frees_and_says_when_there_are_none():
    s = State([20, 20, 20], spare=0)
    s.fork([0, 0, 0])                # two are freed, two are given
    assert s.status.item() == 0
    s.fork([0, 1, 2, 0, 0, 0, 0, 0])
    assert s.status.item() == lmkv.ERR_NO_PAGES


def test_resize_gives_and_frees():
    s = State([40, 0, 17, 16, 64], spare=12)
    s.resize([0, 50, 18, 15, 65])
    s.resize([33, 50, 0, 200 // 3, 1], in_place=False)
    s.resize([0] * 5)
    assert int(s.refs.abs().sum()) == 0
    s.resize([16 * s.cols, 0, 0, 0, 0])


def test_resize_without_enough_pages():
    s = State([16, 16], spare=2, cols=8)
    s.resize([70, 70])
    assert s.status.item() == lmkv.ERR_NO_PAGES


def test_resize_many_rows_and_pages():
    rng = np.random.default_rng(1)
    s = State(rng.integers(0, 60, 2500), page=4, layers=1, spare=30000, kv_heads=1)
    s.resize(rng.integers(0, 60, 2500).tolist())
    s.resize(rng.integers(0, 60, 2500).tolist())
    s.compact()


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("page", [1, 16, 24])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(bits, page, in_place):
    s = State([40, 100, 17, 3, 64, 0], shared=2, groups=2, page=page, bits=bits, spare=25)
    s.resize([0, 70, 17, 0, 20, 0], in_place)
    s.compact(in_place)
    s.compact(in_place)              # nothing is left to do
    s.resize([1] * 6, in_place)


def test_compact_when_nothing_or_everything_is_held():
    s = State([32, 32], spare=0)
    s.compact()
    s.resize([0, 0])
    s.compact()


def test_pages_out_of_reach_stay():
    s = State([40, 50, 20], spare=10)
    free = np.nonzero(s.m.refs == 0)[0][:4]
    s.m.refs[free] = -3
    own = int(s.m.table[1, 0])
    s.m.refs[own] = -1
    s.refs = torch.from_numpy(s.m.refs).to(DEV)
    s.resize([0, 50, 60])
    s.fork([1, 1, 2])
    s.compact()
    assert s.refs[free].cpu().tolist() == [-3] * 4 and int(s.refs[own]) == -1


def test_entries_and_lengths_out_of_range():
    for bad in (-1, -2 ** 31, 10 ** 9):
        s = State([40, 50, 20])
        s.table[0, 1] = bad
        s.m.table[0, 1] = bad
        s.resize([40, 20, 20])
        assert s.status.item() == 0
        s.compact()
        assert s.status.item() == lmkv.ERR_BAD_BLOCK
        s.fork([0, 0, 1])
        s.table[2, 1] = bad          # a page that is not full
        s.m.table[2, 1] = bad
        s.fork([2, 2])
    for bad in (-5, 10 ** 6):
        s = State([40, 50, 20], cols=4)
        s.lens[2] = bad
        s.m.lens[2] = bad
        s.resize([40, 20, 20])
        assert s.status.item() == lmkv.ERR_BAD_LENGTH


def test_random_walk():
    rng = np.random.default_rng(3)
    s = State(rng.integers(0, 90, 12), page=8, spare=300, layers=2, kv_heads=1, cols=14)
    for _ in range(25):
        what = rng.integers(0, 4)
        n = len(s.m.lens)
        if what == 0:
            s.fork(rng.integers(-1, n, rng.integers(4, 14)).tolist(), bool(rng.integers(2)))
        elif what == 3:
            s.compact(bool(rng.integers(2)))
        else:
            s.resize(np.clip(s.m.lens + rng.integers(-30, 30, n), 0, 112).tolist(), bool(rng.integers(2)))
    assert s.status.item() == 0


@pytest.mark.parametrize("bits", [8, 16, 32])
def test_copy_pages(bits):
    s = State([200, 30], spare=30, bits=bits)
    free = np.nonzero(s.m.refs == 0)[0]
    src = np.array([s.m.table[0, 0], s.m.table[0, 3], s.m.table[1, 1], 5, -1, s.num_blocks], np.int32)
    dst = np.array([free[0], free[1], free[2], 5, free[3], free[4]], np.int32)
    put = lambda x: torch.from_numpy(x).to(DEV)
    pkg.check(pkg.copy_pages(s.pool, put(src), put(dst), s.status))
    for a, z in list(zip(src, dst))[:3]:
        s.m.copy(a, z, s.m.page)
    s.m.status = lmkv.ERR_BAD_BLOCK
    s.check()
    s.status.zero_()
    s.m.status = 0
    pkg.check(pkg.copy_pages(s.pool, put(src[:0]), put(dst[:0]), s.status))
    s.check()


def test_copies_of_many_layers_and_pages():
    s = State([16 * 300], spare=300, layers=40, kv_heads=1)
    src = torch.from_numpy(s.m.table[0, :300].copy()).to(DEV)
    free = np.nonzero(s.m.refs == 0)[0][:300].astype(np.int32)
    pkg.check(pkg.copy_pages(s.pool, src, torch.from_numpy(free).to(DEV), s.status))
    for a, z in zip(s.m.table[0, :300], free):
        s.m.copy(a, z, 16)
    s.check()


def test_null_layers_are_reported():
    s = State([40, 40])
    s.pool.ptrs[1] = 0
    free = torch.from_numpy(np.nonzero(s.m.refs == 0)[0][:2].astype(np.int32)).to(DEV)
    pkg.check(pkg.copy_pages(s.pool, s.table[0, :2].contiguous(), free, s.status))
    torch.cuda.synchronize()
    assert s.status.item() == lmkv.ERR_BAD_POINTER


def test_captured_walk_on_another_stream():
    """fork, resize and compact captured on a side stream; replayed from the same start, the same state."""
    s = State([40, 40, 33, 7], spare=30)
    parents = torch.tensor([1, 1, 0, 3], dtype=torch.int32, device=DEV)
    new = torch.tensor([20, 70, 0, 9], dtype=torch.int32, device=DEV)
    table, lens = torch.empty_like(s.table), torch.empty_like(s.lens)
    refs, where, ws = torch.empty_like(s.refs), torch.empty_like(s.refs), s.ws(4)

    def go():
        pkg.check(pkg.fork_pages(s.pool, s.table, s.lens, parents, s.refs, table, lens, refs, ws, s.status))
        pkg.check(pkg.resize_pages(s.pool, table, lens, new, refs, table, refs, ws, s.status))
        pkg.check(pkg.compact_pages(s.pool, table, new, refs, table, refs, where, ws, s.status))
    start = [l.clone() for l in s.layers], s.scales.clone()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        go()
    s.m.fork([1, 1, 0, 3])
    s.m.resize(np.array([20, 70, 0, 9], np.int32))
    want = s.m.compact()
    for _ in range(2):
        for l, l0 in zip(s.layers, start[0]):
            l.copy_(l0)
        s.scales.copy_(start[1])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert s.status.item() == 0
        assert table.cpu().numpy().tolist() == s.m.table.tolist() and refs.cpu().numpy().tolist() == s.m.refs.tolist()
        assert where.cpu().numpy().tolist() == want.tolist()
        held = s.m.refs > 0
        for l, x in zip(s.layers, s.m.pool):
            assert np.array_equal(l.view(torch.uint8).cpu().numpy()[:, held], x[:, held])
        assert np.array_equal(s.scales.cpu().numpy()[:, :, held], s.m.scales[:, :, held])
