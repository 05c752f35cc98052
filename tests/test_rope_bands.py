"""The angles between YaRN's two borders, and what a table of one's own is for."""
import math

import numpy as np
import pytest

import sparse_moe_ffn_coli_amd as pkg


@pytest.mark.parametrize("rot,base,factor,length", [(64, 10000.0, 8.0, 4096), (128, 500000.0, 4.0, 8192), (40, 10000.0, 32.5, 2048), (576, 1e6, 1.5, 32768)])
def test_share_rises_with_the_turns(rot, base, factor, length):
    """Pair by pair: of the angle f a share of (turns - 1) / 31 is kept, the rest is divided by the factor (each of the five
    operations and the power off by a few half-steps of fp64)."""
    f, amp = pkg.coli_rope_freqs(rot, base, "yarn", factor, length)
    middle = 0
    for i in range(rot // 2):
        plain = math.exp(-2 * i / rot * math.log(base))
        turns = length * plain / (2 * math.pi)
        share = min(max((turns - 1) / 31, 0), 1)
        assert math.isclose(f[i], plain * (share + (1 - share) / factor), rel_tol=1e-13), i
        middle += 0 < share < 1
    assert middle >= 3 and math.isclose(amp, 0.1 * math.log(factor) + 1, rel_tol=2.0 ** -24)


def test_a_share_by_index_is_another_table():
    """What the documentation says of models that blend by the pair's index: other angles between the borders, up to 2.3 times
    these, the same outside of them."""
    rot, base, factor, length = 64, 10000.0, 8.0, 4096
    f = pkg.coli_rope_freqs(rot, base, "yarn", factor, length)[0].numpy()
    i = np.arange(rot // 2)
    plain = base ** (-2 * i / rot)
    border = lambda turns: rot / 2 * math.log(length / (turns * 2 * math.pi)) / math.log(base)
    lo, hi = math.floor(border(32)), math.ceil(border(1))
    share = np.clip((hi - i) / (hi - lo), 0, 1)
    other = plain * (share + (1 - share) / factor)
    ratio = other / f
    assert 2.2 < ratio.max() < 2.35 and (ratio[lo + 1:hi] > 1.05).all()
    assert np.allclose(ratio[:lo + 1], 1, rtol=1e-13) and np.allclose(ratio[hi:], 1, rtol=1e-13)
