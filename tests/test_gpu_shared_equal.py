"""Equal scores weigh the same wherever their positions lie: in the pages that a group shares or behind them, read by 16-head
tiles or through LDS, however large the scores are."""
import numpy as np
import pytest

from serve_reference import U16, U32, make_shared
from test_gpu_shared import queries, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Dk,Dv", [(64, 64), (128, 128), (192, 128), (256, 256)])
@pytest.mark.parametrize("room", [0, 200000])
@pytest.mark.parametrize("scale,size,key", [(0.1, 65536.0, 129.0), (0.1, 1.5, 7.0), (-0.2, 65536.0, -253.0), (0.3, 4096.0, 129.0), (0.088388, 65536.0, 3.0),
                                            (0.125, 65536.0, 129.0), (3.0, 2.0 ** 20, 253.0)])
def test_equal_scores(Dk, Dv, room, scale, size, key):
    """One product a score, exact in fp32: scores up to 2^30 are the same number in both parts.  Values are 1 in the pages and
    -1 behind them, so the output is a quotient of whole numbers: off by half a step of it, and by the quotient's own
    three roundings."""
    tails = [3, 100, 0, 64, 1, 37, 250, 12, 5, 2]
    c = make_shared([(6, tails)], 1, Dk, Dv, 16, "bf16", seed=1, room=room)
    c["k"][:] = 0
    c["k"][..., 5] = key
    c["v"][:] = -1
    c["v"][c["table"][0, :6].long()] = 1
    q = queries(c, len(tails), 4) * 0
    q[..., 5] = size
    out, lse = run(c, 4, scale, q=q, want=False)
    n = 96 + np.array(tails)
    want = ((96 - np.array(tails)) / n)[:, None, None]
    got = out.double().numpy()
    assert np.all(np.abs(got - want) <= np.abs(want) * (U16 + 4 * U32))
    s = float(np.float32(scale)) * size * key
    assert np.all(np.abs(lse.double().numpy() - (s + np.log(n))[:, None]) <= 4 * U32 * np.abs(s + np.log(n))[:, None] + 8 * U32)


@pytest.mark.parametrize("Dk,Dv", [(64, 64), (128, 128), (256, 256)])
def test_infinite_keys_of_either_sign(Dk, Dv):
    # a score of minus infinity has no weight, through LDS too, whatever the sign of the scale
    import torch
    for scale in (0.1, -0.2, 0.125, 1.0):
        c = make_shared([(6, [3, 100, 0, 64, 1, 37, 250, 12, 5, 2])], 1, Dk, Dv, 16, "bf16", seed=2, room=200000)
        c["k"][:] = 0
        c["k"][..., 5] = float("-inf") if scale > 0 else float("inf")
        q = queries(c, 10, 4) * 0
        q[..., 5] = 1
        out, lse = run(c, 4, scale, q=q, want=False)
        assert bool((out == 0).all()) and bool((lse == float("-inf")).all())
        c["k"][c["table"][0, 2].long(), 0, 7, 5] = 2.0 if scale > 0 else -2.0
        v = c["v"][c["table"][0, 2].long(), 0, 7]
        out, lse = run(c, 4, scale, q=q, want=False)
        assert torch.equal(out, v.expand_as(out)) and torch.allclose(lse, torch.full_like(lse, 2 * abs(scale)))
