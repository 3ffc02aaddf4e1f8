"""The 8-bit cache's operators and pages at the ends of their ranges, against 64-bit formulas."""
import pytest
import torch

import paged_kv_cache_lmkv_gb300 as pkg
from cache8_util import Cache
from gpu_util import require_gpu
from test_gpu_cache8 import attend_case

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
