"""A prompt's life under a batch: brought by one sequence, read by others, the first of them ended while the others go on, its
place taken by another sequence, and the pages given back by the last; attention against the 64-bit form at every step."""
import numpy as np
import pytest
import torch

import kv_reference as kv
from serve_reference import to_np
from sparse_moe_ffn_coli_amd import COLI_BF16, COLI_F32, KvCache, KvShape, coli_kv_attn_shared, coli_kv_attn_shared_workspace_bytes, coli_kv_plan, coli_kv_rope
from test_gpu_kv import within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,latent,Hq,Hkv,Dk,Dv,room", [("f32", False, 4, 2, 64, 64, 0), ("bf16", False, 24, 2, 128, 128, 90000),
                                                            ("bf16", True, 40, 1, 320, 256, 0)])
def test_a_prompt_outlives_the_sequence_that_brought_it(dtype, latent, Hq, Hkv, Dk, Dv, room):
    rng = np.random.default_rng(3)
    B, page, n_pages, P, rows = 6, 8, 120, 9, 160
    mp = max(40, room // page)
    s = KvShape(B=B, Hq=Hq, Hkv=Hkv, Dk=Dk, Dv=Dv, page=page, n_pages=n_pages, max_pages=mp, dtype=COLI_F32 if dtype == "f32" else COLI_BF16)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")
    new = lambda *n: torch.from_numpy(rng.standard_normal(n).astype(np.float32)).cuda().to(dt)
    kpool = torch.full((n_pages, Hkv, page, Dk), float("nan"), dtype=dt, device="cuda")
    vpool = None if latent else torch.full((n_pages, Hkv, page, Dv), float("nan"), dtype=dt, device="cuda")
    table, lens, shared = i32(np.full((B, mp), -1)), i32([0] * B), i32([0] * B)
    ring, state = i32(rng.permutation(n_pages)), i32([0, n_pages, 0, 0])
    start, slot, pos = i32([0] * (B + 1)), i32([0] * rows), i32([0] * rows)
    cache = KvCache(kpool, vpool, table, lens)
    hist = [[] for _ in range(B)]

    def step(want, groups, refused=0):
        coli_kv_plan(s, table, lens, i32(want), ring, state, start, slot, pos, shared=shared)
        k, v = new(rows, Hkv, Dk), None if latent else new(rows, Hkv, Dv)
        coli_kv_rope(s, None, k, v, None, pos=pos, pool_k=kpool, pool_v=vpool, slot=slot)
        assert state.tolist()[3] == refused
        st, n = start.tolist(), lens.tolist()
        kn, vn = to_np(k), to_np(k)[..., :Dv] if latent else to_np(v)
        for b in range(B):
            hist[b] = hist[b][:n[b]] + [(kn[r], vn[r]) for r in range(st[b], st[b + 1])]
            assert len(hist[b]) == n[b]
        q = new(B, Hq, Dk)
        out = torch.empty((B, Hq, Dv), dtype=dt, device="cuda")
        ws = torch.empty(coli_kv_attn_shared_workspace_bytes(s, len(groups) - 1), dtype=torch.uint8, device="cuda")
        coli_kv_attn_shared(s, q, cache, out, 0.1, shared, i32(groups), ws=ws)
        # the history as a cache of its own, a page a sequence
        most = max(max(n), 1)
        at = 1 << (most - 1).bit_length()
        hk, hv = np.zeros((B, Hkv, at, Dk)), np.zeros((B, Hkv, at, Dv))
        for b in range(B):
            for p, (x, y) in enumerate(hist[b]):
                hk[b, :, p], hv[b, :, p] = x, y
        c = dict(k=torch.from_numpy(hk), v=torch.from_numpy(hv), table=torch.arange(B)[:, None], lens=lens.cpu(), page=at, n_pages=B, max_pages=1,
                 Hkv=Hkv, Dk=Dk, Dv=Dv, dtype=dtype)
        r = kv.attn(c, q.cpu(), 0.1)
        within(out.double().cpu().numpy(), r["out"], r["tol_out"], f"lengths {n}")
        return n

    def free():
        h = state.tolist()
        return set(ring.cpu().numpy()[(h[0] + np.arange(h[1])) % n_pages].tolist())

    step([P * page + 3, 0, 0, 0, 0, 0], [0, 1, 6])
    prompt = table[0, :P].tolist()
    for b in (1, 2, 3):
        table[b, :P] = table[0, :P]
        lens[b] = P * page
        hist[b] = hist[0][:P * page]
    shared[:4] = P
    step([P * page + 4, P * page + 1, P * page + 20, P * page + 1, 30, 0], [0, 4, 6])
    n = step([0, P * page + 2, P * page + 21, P * page + 2, 31, 1], [0, 4, 6])       # the first one has ended: read through its row
    assert not free() & set(prompt)
    n = step([50, n[1] + 1, n[2] + 1, n[3] + 1, n[4] + 1, n[5] + 1], [0, 4, 6], refused=1)   # no place for another one yet
    assert n[0] == 0 and table[0, :P].tolist() == prompt
    shared[0] = 0                                                                   # a group of three, and its place is free
    n = step([50, n[1] + 1, n[2] + 1, n[3] + 1, n[4] + 1, n[5] + 1], [0, 1, 4, 6])
    assert n[0] == 50 and not set(table[0, :7].tolist()) & set(prompt)
    n = step([51, P * page - 5, n[2] + 1, n[3] + 1, 0, n[5] + 1], [0, 1, 4, 6])      # one is cut into the prompt
    n = step([52, n[1], 0, n[3] + 1, 0, n[5] + 1], [0, 1, 4, 6])
    n = step([53, 0, 0, n[3] + 1, 0, n[5] + 1], [0, 1, 4, 6])
    assert not free() & set(prompt)
    shared[:] = 0                                                                   # the last one gives them back
    step([54, 0, 0, 0, 0, n[5] + 1], [0, 1, 4, 6])
    assert set(prompt) <= free()
    step([0] * B, [0, B])
    assert free() == set(range(n_pages))
