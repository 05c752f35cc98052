"""Cosines and sines of the rotation, seen through pairs (1, 0): relatively as near to those of the 64-bit angle as fp32 allows,
also next to their zeros and at far positions."""
import numpy as np
import pytest
import torch

from serve_reference import U32, pairs
from sparse_moe_ffn_coli_amd import COLI_F32, KvShape, Rope, coli_kv_rope, coli_rope_freqs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot,rot_at", [(64, 64, 0), (128, 128, 0), (256, 256, 0), (72, 40, 8), (80, 32, 0)])
@pytest.mark.parametrize("far", [300, 1 << 17, (1 << 31) - 1])
def test_relative_error(D, rot, rot_at, interleaved, far):
    """sincospif is off by at most two units in the last place (4 half-steps), the turn by the rest's angle rounds once, and
    the 64-bit angle's two products and fraction are off by 4 half-steps of it."""
    rng = np.random.default_rng(D + far)
    rows = 2000
    pos = rng.integers(0, far, size=rows).astype(np.int32)
    freq = coli_rope_freqs(rot)[0].numpy().copy()
    freq[1] = np.pi * (1 + 2.0 ** -26)                       # half turns, and a little
    freq[2] = np.pi / 2 * (1 - 2.0 ** -25)
    freq[3] = 2 * np.pi * (1 + 2.0 ** -27)
    a, b = pairs(rot, rot_at, interleaved)
    q = torch.zeros((rows, 1, D))
    q[:, 0, torch.from_numpy(a)] = 1
    shape = KvShape(B=0, Hq=1, Hkv=1, Dk=D, Dv=D, page=16, n_pages=1, max_pages=1, dtype=COLI_F32)
    out = torch.empty((rows, 1, D), device="cuda")
    coli_kv_rope(shape, q.cuda(), None, None, out, pos=torch.from_numpy(pos).cuda(), rope=Rope(torch.from_numpy(freq).cuda(), rot_at, interleaved))
    got = out[:, 0].double().cpu().numpy()
    angle = np.longdouble(pos)[:, None] * np.longdouble(freq)
    slack = (4 * 2.0 ** -53 * np.abs(angle)).astype(np.float64)
    for x, want in ((got[:, a], np.cos(angle)), (got[:, b], np.sin(angle))):
        want = want.astype(np.float64)
        over = np.abs(x - want) - 5 * U32 * np.abs(want) - slack - 1e-37
        i = np.unravel_index(over.argmax(), over.shape)
        assert over.max() <= 0, f"position {pos[i[0]]}, pair {i[1]}: {x[i]!r} for {want[i]!r}"
