"""Requests whose sums of tokens and of pages pass 32 bits: first come, first served all the same."""
import numpy as np
import pytest
import torch

from sparse_moe_ffn_coli_amd import KvShape, coli_kv_plan
from test_gpu_plan import dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [3000, 6000])              # in one launch, and in two
def test_sums_past_32_bits(rows):
    """256 sequences of 300 want 2^24 tokens in pages of one: 2^32 of both.  Kept in 32 bits, the sums would begin anew behind
    them, and the small requests there would be served before the large ones that came first."""
    B, mp, n_pages, head, count = 300, 1 << 24, 1000, 990, 700
    want = np.full(B, 2)
    want[3:259] = mp
    assert int(want[3:259].sum()) == 1 << 32
    table = torch.full((B, mp), -7, dtype=torch.int32, device="cuda")
    ring = np.random.default_rng(1).permutation(n_pages)
    d = dict(lens=dev(np.zeros(B)), ring=dev(ring), state=dev([head, count, 0, 0]), start=dev(np.full(B + 1, 5)), slot=dev(np.zeros(rows)),
             pos=dev(np.zeros(rows)))
    shape = KvShape(B=B, Hq=1, Hkv=1, Dk=8, Dv=8, page=1, n_pages=n_pages, max_pages=mp)
    coli_kv_plan(shape, table, d["lens"], dev(want), d["ring"], d["state"], d["start"], d["slot"], d["pos"])
    torch.cuda.synchronize()
    got = {k: v.cpu().numpy() for k, v in d.items()}
    pages = ring[(head + np.arange(6)) % n_pages]
    assert got["state"].tolist() == [(head + 6) % n_pages, count - 6, 6, 297] and np.array_equal(got["ring"], ring)
    assert got["lens"].tolist() == [2] * 3 + [0] * 297 and got["start"].tolist() == [0, 2, 4] + [6] * 298
    assert got["slot"][:6].tolist() == pages.tolist() and got["pos"][:6].tolist() == [0, 1] * 3
    assert (got["slot"][6:] == -1).all() and (got["pos"][6:] == -1).all()
    assert table[:3, :2].tolist() == pages.reshape(3, 2).tolist()
    table[:3, :2] = -7
    assert bool((table == -7).all())
