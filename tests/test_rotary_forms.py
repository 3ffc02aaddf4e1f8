"""The rotary scaling of released long-context checkpoints: a ramp between whole pairs (CPU only)."""
import math

import numpy as np
import pytest

from paged_kv_cache_lmkv_gb300 import build, lmkv


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return lmkv.load()


# The ends by hand from d ln(L / (2 pi n)) / (2 ln b), n turns over L positions:
#   d 128, b 1e4, L 4096:   n 32 -> 20.94, n 1 -> 45.03;    d 128, b 1e6, L 32768: 23.60, 39.65
#   d 64,  b 1e4, L 256:    0.84, 12.88;                    d 64,  b 1e4, L 128:  -1.57, 10.47
#   d 8,   b 10,  L 1000:   2.79, 8.81 (the last is above d - 1);  d 64, b 1e4, L 5: -12.8, -0.79
@pytest.mark.parametrize("dim,base,original,factor,first,last", [
    (128, 1e4, 4096, 16.0, 20, 46), (128, 1e6, 32768, 4.0, 23, 40), (64, 1e4, 256, 8.0, 0, 13),
    (64, 1e4, 128, 8.0, 0, 11), (8, 10.0, 1000, 2.0, 2, 7), (64, 1e4, 5, 2.0, 0, 0)])
def test_ramp_between_whole_pairs(dim, base, original, factor, first, last):
    got = lmkv.Rotary(dim, base=base, scaling="yarn", factor=factor, low=1.0, high=32.0, original=original)
    want = []
    for i in range(dim // 2):
        f = base ** (-2.0 * i / dim)
        slow = 0.0 if i <= first else 1.0 if i >= last else (i - first) / (last - first)
        want.append(f / factor * slow + f * (1.0 - slow))
    np.testing.assert_allclose(got.inv_freq, want, rtol=1e-13)
    assert got.magnitude == pytest.approx(0.1 * math.log(factor) + 1.0, rel=1e-15)


def test_ramp_between_whole_pairs_at_known_pairs():
    """Single values: pair 33 of 128 elements lies half way from 20 to 46."""
    got = lmkv.Rotary(128, base=1e4, scaling="yarn", factor=16.0, low=1.0, high=32.0, original=4096).inv_freq
    f = lambda i: 10.0 ** (-4.0 * i / 64)
    for i, share in ((0, 1.0), (20, 1.0), (33, (1 + 1 / 16) / 2), (46, 1 / 16), (63, 1 / 16)):
        assert got[i] == pytest.approx(f(i) * share, rel=1e-12)
    whole = lmkv.Rotary(128, base=1e4, scaling="ramp", factor=16.0, low=1.0, high=32.0, original=4096).inv_freq
    assert abs(whole[33] / got[33] - 1) > 1e-4                  # the form with fractional ends is another one


def test_ramp_between_whole_pairs_refusals():
    """Both ends before the first pair (original 1) or behind the last (base 10) among them."""
    for bad in (dict(original=1.0), dict(low=0.0), dict(low=32.0), dict(original=0.0), dict(factor=0.5),
                dict(original=1e6, base=10.0)):
        with pytest.raises(lmkv.LmkvError) as e:
            lmkv.Rotary(**(dict(rot_dim=64, base=1e4, scaling="yarn", factor=2.0, low=1.0, high=32.0, original=4096.0) | bad))
        assert e.value.code == lmkv.ERR_INVALID_ARG
