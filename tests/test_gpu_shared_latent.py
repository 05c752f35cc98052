"""Latent rows behind shared pages: every split of the waves over a sequence's and a group's query heads, at rows as wide as the
kernel, narrower ones and ones narrower than its values' columns; and rows that are run again because large values met large
weights."""
import numpy as np
import pytest

from serve_reference import make_shared
from test_gpu_shared import queries, run

pytestmark = pytest.mark.gpu

# Heads, sequences of the groups: one, two or four query tiles for a sequence and for a group (by the mean).
SPLITS = {"1-1": (8, [4, 1, 4]), "1-2": (16, [6, 1, 5]), "1-4": (8, [20, 3, 13]), "2-2": (40, [1, 1, 1, 1]), "2-4": (64, [3, 1, 6]),
          "4-4": (100, [2, 1, 1])}
WIDTHS = [(320, 256), (288, 256), (256, 256), (264, 200), (192, 128), (136, 64), (576, 512), (520, 512), (512, 512), (328, 264), (400, 256)]


def groups_of(sizes, pages, rng):
    """Groups behind so many pages and one page more each; every fifth sequence ends inside them, one slot is empty."""
    out, at = [], 0
    for g, n in enumerate(sizes):
        tails = []
        for _ in range(n):
            t = int(rng.integers(0, 90))
            tails.append((int(rng.integers(1, pages * 16)),) if at % 5 == 3 else (0,) if at == 7 else t)
            at += 1
        out.append((pages + g, tails))
    return out


@pytest.mark.parametrize("split", SPLITS)
@pytest.mark.parametrize("Dk,Dv", WIDTHS)
def test_splits_and_widths(split, Dk, Dv):
    Hq, sizes = SPLITS[split]
    rng = np.random.default_rng(Dk + Hq)
    for pages in (3, 45):                  # rows that are not cut, and rows that are
        run(make_shared(groups_of(sizes, pages, rng), 1, Dk, Dv, 16, "bf16", True, seed=Dk + pages), Hq, 2.0 / np.sqrt(Dk))


@pytest.mark.parametrize("split", SPLITS)
@pytest.mark.parametrize("Dk,Dv", [(320, 256), (264, 256), (576, 512), (520, 512), (400, 256)])
@pytest.mark.parametrize("where", ["pages", "own"])
@pytest.mark.parametrize("growth", [50.0, 90.0])
def test_large_values(split, Dk, Dv, where, growth):
    """Values near 1e30 beside scores that grow by 2^50 or 2^90 over each 256 positions (the shortest part a row is cut into) of
    the pages, or behind them: sums under the first stage's reference pass fp32's end, the results are far inside it."""
    Hq, sizes = SPLITS[split]
    sizes = sizes[:2]
    for n in (240, 1100):                  # a whole row, one that is cut
        pages = -(-n // 16) if where == "pages" else 2
        c = make_shared([(pages, [n - 3 * i if where == "own" and i < 2 else 40 for i in range(s)]) for s in sizes], 1, Dk, Dv, 16,
                        "bf16", True, seed=n)
        q = queries(c, sum(sizes), Hq)
        q[..., :Dv] = 0                    # scores come from the columns that are no values
        q[..., Dv] = 1.0
        k = c["k"]
        k[..., :Dv] *= 1e30
        k[..., Dv:] *= 0.125
        k[..., Dv] = 0.25
        b0 = 0
        for s in sizes:
            for b in range(b0, b0 + s):
                first, end = (0, pages * 16) if where == "pages" else (pages * 16, int(c["lens"][b]))
                if where == "own" and end - first < 100:
                    continue
                p = np.arange(first, end)
                k[c["table"][b, p // 16].long(), 0, p % 16, Dv] = k.new_tensor((p - first) % 256 / 256)
            b0 += s
        run(c, Hq, growth * np.log(2.0), q=q)
