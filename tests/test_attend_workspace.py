"""The attention workspace's size grows with every bound, so that the largest batch's serves all (CPU only)."""
import ctypes
import random

import pytest

from paged_kv_cache_lmkv_gb300 import build, lmkv


@pytest.fixture(scope="module")
def size():
    build.build()
    lib = lmkv.load()

    def call(kv_heads, dim, *bounds):
        pool = lmkv._PoolT(0x20000, 64, 2, kv_heads, dim, 16, 2)
        out = ctypes.c_uint64(0)
        assert lib.lmkv_attend_workspace_bytes(ctypes.byref(pool), *bounds, ctypes.byref(out)) == lmkv.OK
        return out.value
    return call


def test_fewer_tokens_need_no_more(size):
    """32 heads on 8 of 128, no prefix, contexts up to 1024: batches of 1 to 8192 tokens."""
    by_tokens = [size(8, 128, 32, t, 8, 2048, 0, 1024) for t in (1, 8, 64, 512, 1024, 2048, 8192)]
    assert by_tokens == sorted(by_tokens) and by_tokens[3] > 0


def test_grows_with_every_bound(size):
    rng = random.Random(5)
    up = lambda top: int(top ** rng.random())
    for _ in range(3000):
        kv_heads, group, dim = rng.choice((1, 2, 3, 8, 16, 160)), rng.choice((1, 4, 8, 3, 64)), rng.choice((64, 128))
        most = [up(20000), up(600), up(4000), rng.choice((0, up(300000))), rng.choice((0, up(200000)))]
        less = [rng.choice((x, rng.randint(min(x, 1), x), rng.randint(0, x))) for x in most]
        assert size(kv_heads, dim, kv_heads * group, *less) <= size(kv_heads, dim, kv_heads * group, *most), (less, most)


def test_stays_small(size):
    """Less than a GB for batches of 16384 rows a head, whatever the prefix; none where nothing is joined."""
    assert size(8, 128, 64, 16384, 256, 16384, 1 << 20, 1 << 17) < 1 << 30
    assert size(8, 128, 64, 64, 64, 1, 16384, 600) < 64 << 20
    assert size(8, 128, 64, 64, 64, 1, 0, 1024) == 0
