"""Attention of one new token per sequence where groups of sequences share their first pages, through the C ABI, against
the plain 64-bit form of the attention over each sequence's own row of the table (tests/kv_reference.py, with its bounds).
Rows of the pools that no position owns hold NaN and infinities throughout."""
import numpy as np
import pytest

import kv_reference as ref
from serve_reference import make_shared
from sparse_moe_ffn_coli_amd import (COLI_BF16, COLI_F32, KvCache, KvShape, coli_kv_append, coli_kv_attn, coli_kv_attn_shared,
                                     coli_kv_attn_shared_workspace_bytes, coli_kv_attn_workspace_bytes)
from test_gpu_kv import bits, guarded, queries, within

pytestmark = pytest.mark.gpu


def handles(c, Hq):
    B = len(c["lens"])
    s = KvShape(B=B, Hq=Hq, Hkv=c["Hkv"], Dk=c["Dk"], Dv=c["Dv"], page=c["page"], n_pages=c["n_pages"], max_pages=c["max_pages"],
                dtype=COLI_F32 if c["dtype"] == "f32" else COLI_BF16)
    cache = KvCache(c["k"].cuda(), None if c["v"] is None else c["v"].cuda(), c["table"].cuda(), c["lens"].cuda())
    return s, cache, c["shared"].cuda(), c["group_start"].cuda()


def run(c, Hq, scale, q=None, want=True, stream=None):
    import torch
    B = len(c["lens"])
    q = queries(c, B, Hq) if q is None else q
    s, cache, shared, start = handles(c, Hq)
    out, out_ok = guarded((B, Hq, c["Dv"]), q.dtype, 7.0)
    lse, lse_ok = guarded((B, Hq), torch.float32, 7.0)
    ws, ws_ok = guarded((coli_kv_attn_shared_workspace_bytes(s, len(start) - 1),), torch.uint8, 0xA5)
    qd = q.cuda()
    torch.cuda.synchronize()
    for _ in range(2):                     # a second pass on what the first left in the workspace
        coli_kv_attn_shared(s, qd, cache, out, scale, shared, start, lse=lse, ws=ws, stream=stream)
    torch.cuda.synchronize()
    for ok in (out_ok, lse_ok, ws_ok):
        ok()
    if want:
        r = ref.attn(c, q, scale)
        label = f"{c['dtype']} B={B} Hq={Hq} Hkv={c['Hkv']} D={c['Dk']}/{c['Dv']} page={c['page']}"
        within(out.double().cpu().numpy(), r["out"], r["tol_out"], label + " out")
        within(lse.cpu().numpy(), r["lse"], r["tol_lse"], label + " lse")
        print(label, "ok", flush=True)
    return out.cpu(), lse.cpu()


# Groups whose pages end inside tiles, one that shares nothing, one of one sequence, sequences that end before
# their group's pages or with them, empty slots (the first of a group among them).
def mixed(page):
    n = -(-150 // page)
    return [(n, [0, 1, 33, (n * page - 1,), (1,), 70]), (0, [5, 0, 64]), (-(-257 // page), [129]),
            (-(-40 // page), [(0,), 31, 32, (0,), 2])]


LAYOUTS = [(8, 2, 64, 64, 16, False), (3, 3, 8, 8, 1, False), (12, 12, 80, 80, 2, False), (14, 2, 128, 128, 64, False),
           (5, 1, 96, 40, 4, False), (4, 2, 72, 136, 8, False), (34, 2, 192, 128, 32, False), (16, 1, 256, 256, 128, False),
           (6, 2, 256, 200, 512, False), (32, 8, 128, 128, 16, False), (40, 1, 128, 128, 16, False), (32, 1, 128, 64, 16, True),
           (16, 1, 576, 512, 64, True), (20, 1, 576, 512, 16, True), (33, 1, 512, 512, 16, True), (100, 1, 320, 256, 32, True),
           (8, 4, 296, 264, 8, True), (64, 1, 576, 512, 64, True), (128, 1, 576, 512, 64, True), (2, 1, 256, 256, 16, True)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv,Dk,Dv,page,latent", LAYOUTS)
def test_layouts(dtype, Hq, Hkv, Dk, Dv, page, latent):
    run(make_shared(mixed(page), Hkv, Dk, Dv, page, dtype, latent, seed=Hq * 1000 + Dk), Hq, 2.0 / np.sqrt(Dk))


@pytest.mark.parametrize("dtype,Hq,Hkv,Dk,Dv,latent", [("bf16", 8, 2, 128, 128, False), ("bf16", 4, 2, 64, 64, False),
                                                       ("bf16", 2, 1, 256, 256, False), ("bf16", 2, 1, 192, 128, False),
                                                       ("f32", 2, 1, 64, 64, False), ("bf16", 16, 1, 576, 512, True)])
@pytest.mark.parametrize("n", [1, 2, 4, 5, 8, 16, 17, 32, 33, 70])
def test_group_sizes(dtype, Hq, Hkv, Dk, Dv, latent, n):
    # from one query tile that is not full to several, beside groups of other sizes
    rng = np.random.default_rng(n)
    for room in (0, 100000):
        c = make_shared([(20, list(rng.integers(0, 60, size=n))), (3, [9]), (11, list(rng.integers(0, 9, size=3)))], Hkv, Dk, Dv, 16,
                        dtype, latent, seed=n, room=room)
        run(c, Hq, 2.0 / np.sqrt(Dk))


@pytest.mark.parametrize("Hq,Hkv,Dk,Dv", [(8, 2, 128, 128), (4, 1, 64, 64), (8, 2, 256, 256), (4, 1, 192, 128), (4, 1, 80, 104),
                                          (4, 1, 40, 24), (4, 2, 128, 200), (32, 1, 96, 96)])
@pytest.mark.parametrize("n,pages", [(9, 40), (17, 3), (24, 70), (33, 21), (65, 129), (80, 2)])
def test_one_large_group(Hq, Hkv, Dk, Dv, n, pages):
    # every number of query tiles a workgroup has, and of waves that split the positions
    rng = np.random.default_rng(n + Dk)
    # (as wide a table as a long prefix has, and one that ends behind the sequences)
    for room in (200000, 0):
        run(make_shared([(pages, list(rng.integers(0, 50, size=n)))], Hkv, Dk, Dv, 16, "bf16", seed=n, room=room), Hq, 2.0 / np.sqrt(Dk))


def test_one_large_group_of_small_pages():
    # the shared pages end inside a stage; pages that do not exist
    rng = np.random.default_rng(3)
    for page, pages in ((1, 77), (2, 1030), (8, 5)):
        c = make_shared([(pages, list(rng.integers(0, 9, size=40)))], 1, 128, 128, page, "bf16", seed=page, room=60000)
        run(c, 4, 0.2)
        c["table"][:, [0, 3, pages - 1]] = -1
        run(c, 4, 0.2)


@pytest.mark.parametrize("dtype,latent,Hq,Hkv,Dk,Dv", [("bf16", False, 8, 2, 128, 128), ("f32", False, 2, 2, 64, 64),
                                                       ("bf16", True, 64, 1, 576, 512), ("bf16", False, 2, 1, 256, 256),
                                                       ("bf16", False, 48, 1, 128, 128), ("bf16", False, 64, 1, 64, 64)])
def test_long_prefix(dtype, latent, Hq, Hkv, Dk, Dv):
    # cut over every range
    run(make_shared([(1251, [1, 700, 40, 3])], Hkv, Dk, Dv, 16, dtype, latent, seed=5), Hq, 2.0 / np.sqrt(Dk))


@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scales(scale, dtype):
    run(make_shared([(30, [9, 100, 0]), (2, [1, 1])], 2, 128, 128, 16, dtype, seed=4), 8, scale)
    run(make_shared([(30, [9, 100, 0] * 5), (2, [1, 1])], 2, 128, 128, 16, dtype, seed=4, room=100000), 16, scale)
    run(make_shared([(30, [9, 100, 0]), (2, [1, 1])], 1, 576, 512, 16, dtype, True, seed=4), 16, scale / 3)


@pytest.mark.parametrize("dtype,Hq,Hkv,D", [("bf16", 8, 2, 128), ("f32", 8, 2, 64), ("bf16", 4, 2, 256)])
def test_many_sequences_and_groups(dtype, Hq, Hkv, D):
    rng = np.random.default_rng(6)
    groups = [(int(rng.integers(0, 12)), [int(x) if x < 40 else (0,) for x in rng.integers(0, 50, size=rng.integers(1, 9))]) for _ in range(130)]
    run(make_shared(groups, Hkv, D, D, 8, dtype, seed=6), Hq, 0.2)
    if D == 128:
        run(make_shared(groups[:70], Hkv, D, D, 8, dtype, seed=6, room=3000), 20, 0.2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("latent,Hq,Dk,Dv", [(False, 8, 128, 128), (True, 40, 576, 512)])
def test_hidden_pages(dtype, latent, Hq, Dk, Dv):
    c = make_shared([(20, [30, 50, 0, 7, 8, 9, 10]), (9, [90, 3])], 1 if latent else 2, Dk, Dv, 8, dtype, latent, seed=10)
    c["table"][:7, 3] = -1                 # in the shared pages of a group, for all of it
    c["table"][:7, 17:19] = c["n_pages"]
    c["table"][1, 22] = -7                 # in a sequence's own
    c["table"][7:, :9] = 1 << 30           # a group without any
    run(c, Hq, 0.1)
    c["table"][:] = -1                     # nothing anywhere
    out, lse = run(c, Hq, 0.1)
    assert bool((out == 0).all()) and bool((lse == -np.inf).all())


def test_values_outside_a_query_do_not_reach_it():
    """NaN and infinities in shared rows behind a short sequence's end, in other sequences' rows, behind the lengths."""
    import torch
    for latent, Hq, Dk, Dv, room in ((False, 8, 128, 128, 0), (False, 40, 128, 128, 200000), (True, 32, 576, 512, 0)):
        c = make_shared([(8, [5, (70,), (0,), 0]), (2, [9])], 1 if latent else 2, Dk, Dv, 16, "bf16", latent, seed=11, room=room)
        a = run(c, Hq, 0.1)
        for pool in (c["k"], c["v"]):
            if pool is not None:
                pool[c["table"][0, 4], :, 6:] = float("nan")           # position 70 on of the shared pages
                pool[c["table"][0, 5:8].long()] = float("inf")
        b = run(c, Hq, 0.1, want=False)
        keep = [1, 2, 4]
        assert torch.equal(a[0][keep], b[0][keep]) and torch.equal(a[1][keep], b[1][keep])
        assert bool(b[1][[0, 3]].isnan().all())


def test_infinite_and_missing_scores():
    import torch
    for dtype in ("bf16", "f32"):
        for Hq, room in ((2, 0), (40, 300000)):
            c = make_shared([(4, [20, 33, 0]), (4, [3])], 1, 64, 64, 16, dtype, seed=12, room=room)
            q = queries(c, 4, Hq)
            q[:, :, 1:] = 0
            q[:, :, 0] = 1
            c["k"][:, :, :, 0] = float("-inf")
            out, lse = run(c, Hq, 0.5, q=q, want=False)                     # no weight anywhere
            assert bool((out == 0).all()) and bool((lse == float("-inf")).all())
            c["k"][c["table"][0, 2].long(), :, 7, 0] = 3.0                 # one score in the first group's pages
            out, lse = run(c, Hq, 0.5, q=q, want=False)
            v = c["v"][c["table"][0, 2].long(), 0, 7]
            assert bool((out[:3] == v).all()) and torch.allclose(lse[:3], torch.full_like(lse[:3], 1.5)) and bool((out[3] == 0).all())
            c["k"][c["table"][0, 2].long(), :, 9, 0] = float("inf")
            out, lse = run(c, Hq, 0.5, q=q, want=False)
            assert bool(lse[:3].isnan().all()) and bool(out[:3].isnan().all()) and bool((lse[3] == float("-inf")).all())


def test_the_largest_score_anywhere():
    """A score far above the rest, in the pages or behind them, early or late."""
    for latent, Hq, Dk, Dv, room in ((False, 16, 128, 128, 0), (False, 16, 128, 128, 200000), (False, 16, 256, 256, 200000), (True, 16, 576, 512, 0)):
        for pos in (0, 40, 511, 512, 520):
            c = make_shared([(32, [30, 31, 45, 9, 10, 11])], 1, Dk, Dv, 16, "bf16", latent, seed=pos, room=room)
            for b in range(6):
                c["k"][c["table"][b, pos // 16].long(), :, pos % 16] *= 30
            run(c, Hq, 1.0)


def test_like_the_attention_over_each_row():
    """Beside coli_kv_attn on the same cache: both within the bound of the same value."""
    import torch
    c = make_shared([(40, [100, 7, 0, 31]), (0, [300, 20])], 2, 128, 128, 16, "bf16", seed=13)
    q = queries(c, 6, 8)
    out, lse = run(c, 8, 0.15, q=q)
    s, cache, shared, start = handles(c, 8)
    out2, lse2 = torch.empty_like(out, device="cuda"), torch.empty_like(lse, device="cuda")
    ws = torch.empty(coli_kv_attn_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    coli_kv_attn(s, q.cuda(), cache, out2, 0.15, lse=lse2, ws=ws)
    r = ref.attn(c, q, 0.15)
    within(out2.double().cpu().numpy(), r["out"], r["tol_out"], "out")
    assert np.abs((lse - lse2.cpu()).numpy()).max() <= 2 * r["tol_lse"].max()


def test_groups_that_are_no_partition_stay_inside():
    """Descending borders, borders outside the batch, counts outside the table: no fault, nothing outside the outputs."""
    import torch
    for Hq, room in ((4, 0), (80, 200000)):
        c = make_shared([(8, [5, 9]), (2, [9, 1, 4])], 2, 64, 64, 16, "bf16", seed=14, room=room)
        for start in ([0, -5, 99], [3, 1, 0], [5, 5, 5], [0, 5, 0], [2, 4, 4]):
            for shared in ([8, 8, 2, 2, 2], [-1, 100, 0, 1 << 30, -(1 << 31)]):
                c["group_start"], c["shared"] = torch.tensor(start, dtype=torch.int32), torch.tensor(shared, dtype=torch.int32)
                c["table"] = c["table"].clamp(min=0)
                run(c, Hq, 0.1, want=False)


@pytest.mark.parametrize("dtype,latent,n_groups", [("bf16", False, 64), ("bf16", False, 400), ("f32", False, 300), ("bf16", True, 64)])
def test_falling_borders_of_more_units_than_a_number_holds(dtype, latent, n_groups):
    """Borders 0, B, 0, B, .. of 4096 sequences count the batch n_groups / 2 times: some 2^33 units."""
    import torch
    B, Hq, page, mp, Dk, Dv = 4096, 8, 4096, 63, 264 if latent else 8, 8
    Hkv = 1 if latent else 8
    s = KvShape(B, Hq, Hkv, Dk, Dv, page, 2, mp, COLI_F32 if dtype == "f32" else COLI_BF16)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    zeros = lambda *n, dt=torch.int32: torch.zeros(n, dtype=dt, device="cuda")
    cache = KvCache(zeros(2, Hkv, page, Dk, dt=dt), None if latent else zeros(2, Hkv, page, Dv, dt=dt), zeros(B, mp), zeros(B))
    start = zeros(n_groups + 1)
    start[1::2] = B
    q, out, lse = zeros(B, Hq, Dk, dt=dt), zeros(B, Hq, Dv, dt=dt), zeros(B, Hq, dt=torch.float32)
    ws = zeros(coli_kv_attn_shared_workspace_bytes(s, n_groups), dt=torch.uint8)
    coli_kv_attn_shared(s, q, cache, out, 0.1, zeros(B) + mp, start, lse=lse, ws=ws)
    torch.cuda.synchronize()
    assert bool((out == 0).all()) and bool((lse == -np.inf).all())       # (no sequence has a position)


@pytest.mark.parametrize("Dk,Dv", [(64, 64), (64, 40), (128, 128), (128, 64), (96, 72)])
@pytest.mark.parametrize("n", [11, 30, 70])
def test_narrow_latent_groups_of_many_heads(Dk, Dv, n):
    rng = np.random.default_rng(n)
    c = make_shared([(70, list(rng.integers(0, 50, size=n))), (2, [5])], 1, Dk, Dv, 16, "bf16", True, seed=n, room=200000)
    run(c, 8, 2.0 / np.sqrt(Dk))


def test_no_sequences():
    import torch
    s = KvShape(0, 4, 2, 64, 64, 16, 4, 2, COLI_F32)
    z = lambda *n, dt=torch.float32: torch.zeros(n, dtype=dt, device="cuda")
    i = lambda *n: z(*n, dt=torch.int32)
    cache = KvCache(z(4, 2, 16, 64), z(4, 2, 16, 64), i(0, 2), i(0))
    coli_kv_attn_shared(s, z(0, 4, 64), cache, z(0, 4, 64), 0.1, i(0), i(1), ws=z(coli_kv_attn_shared_workspace_bytes(s, 0), dt=torch.uint8))
    torch.cuda.synchronize()


def test_repeats_streams_and_graphs():
    import torch
    c = make_shared([(100, [300, 17, 9, 1]), (7, [4])], 2, 128, 128, 16, "bf16", seed=16)
    a = run(c, 8, 0.2, want=False)
    side = torch.cuda.Stream()
    wide = make_shared([(100, [300, 17, 9, 1] * 8), (7, [4])], 2, 128, 128, 16, "bf16", seed=16, room=200000)
    for _ in range(3):
        x, y = run(wide, 8, 0.2, want=False), run(wide, 8, 0.2, want=False, stream=side)
        assert torch.equal(bits(x[0]), bits(y[0])) and torch.equal(bits(x[1]), bits(y[1]))
    for st in (None, side, None):
        b = run(c, 8, 0.2, want=False, stream=st)
        assert torch.equal(bits(a[0]), bits(b[0])) and torch.equal(bits(a[1]), bits(b[1]))
    for latent, Hq, Hkv, Dk, Dv, room in ((False, 8, 2, 128, 128, 0), (False, 64, 2, 128, 128, 200000), (True, 64, 1, 576, 512, 0)):
        c = make_shared([(30, [40, 17, 9, 1]), (7, [4])], Hkv, Dk, Dv, 16, "bf16", latent, seed=17, room=room)
        s, cache, shared, start = handles(c, Hq)
        q = queries(c, 5, Hq).cuda()
        # two captured calls, each with a workspace, replayed at once
        calls = []
        for i in range(2):
            out = torch.empty((5, Hq, Dv), dtype=torch.bfloat16, device="cuda")
            ws = torch.empty(coli_kv_attn_shared_workspace_bytes(s, 2), dtype=torch.uint8, device="cuda")
            st = torch.cuda.Stream()
            qi = q * (i + 1)
            coli_kv_attn_shared(s, qi, cache, out, 0.1, shared, start, ws=ws)
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=st):
                coli_kv_attn_shared(s, qi, cache, out, 0.1, shared, start, ws=ws)
            calls.append((g, st, out, qi, ws))         # (a captured call's workspace lives as long as the graph)
        for step in range(4):
            cache.lens[:4] += 0 if step == 0 else 1
            cache.lens.clamp_(max=int(c["max_pages"]) * 16 - 16)
            torch.cuda.synchronize()
            for g, st, out, _, _ in calls:
                with torch.cuda.stream(st):
                    out.zero_()
                    g.replay()
            torch.cuda.synchronize()
            for _, _, out, qi, _ in calls:
                want = torch.empty_like(out)
                own = torch.empty(coli_kv_attn_shared_workspace_bytes(s, 2), dtype=torch.uint8, device="cuda")
                coli_kv_attn_shared(s, qi, cache, want, 0.1, shared, start, ws=own)
                assert torch.equal(bits(out), bits(want)), f"replay {step}"


def test_offsets_past_32_bits():
    """A pool of more than 2^32 elements; shared and own pages lie at its end and its start."""
    import torch
    page, D, Hkv = 4096, 256, 4
    n_pages = 1100
    g = torch.Generator(device="cuda").manual_seed(1)
    k = torch.zeros((n_pages, Hkv, page, D), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    ids = [n_pages - 1, 0, n_pages - 2]
    for pg in ids:
        k[pg] = torch.randn(k[pg].shape, generator=g, device="cuda").bfloat16()
        v[pg] = torch.randn(k[pg].shape, generator=g, device="cuda").bfloat16()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    table, lens = i32([[n_pages - 1, 0], [n_pages - 1, n_pages - 2]]), i32([page + 100, page + 1])
    s = KvShape(2, 4, Hkv, D, D, page, n_pages, 2, COLI_BF16)
    q = torch.randn((2, 4, D), generator=g, device="cuda").bfloat16()
    out = torch.empty_like(q)
    ws = torch.empty(coli_kv_attn_shared_workspace_bytes(s, 1), dtype=torch.uint8, device="cuda")
    coli_kv_attn_shared(s, q, KvCache(k, v, table, lens), out, 0.1, i32([1, 1]), i32([0, 2]), ws=ws)
    c = dict(k=k[ids].cpu(), v=v[ids].cpu(), table=torch.tensor([[0, 1], [0, 2]]), lens=lens.cpu(), page=page, n_pages=3, max_pages=2,
             Hkv=Hkv, Dk=D, Dv=D, dtype="bf16")
    r = ref.attn(c, q.cpu(), 0.1)
    within(out.double().cpu().numpy(), r["out"], r["tol_out"], "out")


def test_refusals_of_the_binding():
    import torch
    c = make_shared([(2, [5, 9])], 2, 64, 64, 16, "bf16", seed=18)
    s, cache, shared, start = handles(c, 4)
    q = queries(c, 2, 4).cuda()
    out = torch.empty_like(q)
    ws = torch.empty(coli_kv_attn_shared_workspace_bytes(s, 1), dtype=torch.uint8, device="cuda")
    for kw in (dict(shared=shared.long()), dict(shared=shared[:1]), dict(shared=shared.cpu()), dict(group_start=start.view(1, 2)),
               dict(group_start=start[:0]), dict(group_start=start.float())):
        with pytest.raises(ValueError):
            coli_kv_attn_shared(s, q, cache, out, 0.1, **(dict(shared=shared, group_start=start, ws=ws) | kw))
    with pytest.raises(ValueError):
        coli_kv_attn_shared(s, q.float(), cache, out, 0.1, shared, start, ws=ws)
    with pytest.raises(ValueError):
        coli_kv_attn_shared(s, q, cache, out, 0.1, shared, start, ws=ws.cpu())


def test_a_serving_step():
    """The plan, the rotated keys' way into the pages and the attention behind a shared prompt, step after step: prompts
    that are appended, tokens that are decoded, a sequence that ends and one that begins, against 64-bit forms over the
    whole history."""
    import torch
    import serve_reference as sr
    from sparse_moe_ffn_coli_amd import QkNorm, Rope, coli_kv_plan, coli_kv_rope, coli_rope_freqs
    rng = np.random.default_rng(19)
    B, Hq, Hkv, D, page, n_pages, mp, P = 6, 8, 2, 64, 8, 200, 24, 5
    s = KvShape(B=B, Hq=Hq, Hkv=Hkv, Dk=D, Dv=D, page=page, n_pages=n_pages, max_pages=mp, dtype=COLI_F32)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    f32 = lambda *n: torch.from_numpy(rng.standard_normal(n).astype(np.float32)).cuda()
    kpool, vpool = torch.full((n_pages, Hkv, page, D), float("nan"), device="cuda"), torch.full((n_pages, Hkv, page, D), float("nan"), device="cuda")
    table, lens, shared = i32(np.full((B, mp), -1)), i32([0] * B), i32([0] * B)
    ring, state = i32(rng.permutation(n_pages)), i32([0, n_pages, 0, 0])
    rows = 80
    start, slot, pos = i32([0] * (B + 1)), i32([0] * rows), i32([0] * rows)
    freq, amp = coli_rope_freqs(32)
    norm = QkNorm(1 + 0.1 * f32(D), 1 + 0.1 * f32(D))
    rope = Rope(freq.cuda(), 8, True, amp)
    cache = KvCache(kpool, vpool, table, lens)
    hist = [[] for _ in range(B)]          # (key, value) of every position, in 64 bits

    def step(want):
        """New tokens of random content up to the wanted lengths; the queries of the last ones."""
        coli_kv_plan(s, table, lens, i32(want), ring, state, start, slot, pos, shared=shared)
        x = f32(rows, (Hq + 2 * Hkv) * D)
        q, k = x[:, :Hq * D].unflatten(1, (Hq, D)), x[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
        v = x[:, (Hq + Hkv) * D:].unflatten(1, (Hkv, D))
        q_out = torch.zeros((rows, Hq, D), device="cuda")
        coli_kv_rope(s, q, k, v, q_out, pos=pos, rope=rope, norm=norm, pool_k=kpool, pool_v=vpool, slot=slot)
        st, ps = start.tolist(), pos.cpu().numpy()
        assert state.tolist()[3] == 0 and lens.tolist() == list(want)
        kk, _ = sr.norm_rope(sr.to_np(k), sr.to_np(norm.k_w), 1e-6, ps, freq.numpy(), 8, True, amp, False)
        for b in range(B):
            hist[b] = hist[b][:want[b]]
            hist[b] += [(kk[r], sr.to_np(v[r])) for r in range(st[b], st[b + 1])]
            assert len(hist[b]) == want[b]
        return q_out, st

    step([P * page + 3, 0, 0, 0, 0, 0])    # the prompt, with three tokens of the first sequence's own
    for b in (1, 2, 3):                    # its full pages are lent to three others
        table[b, :P] = table[0, :P]
        lens[b] = P * page
        hist[b] = hist[0][:P * page]
    shared[:4] = P
    group_start = i32([0, 4, 6])
    ws = torch.empty(coli_kv_attn_shared_workspace_bytes(s, 2), dtype=torch.uint8, device="cuda")
    free = []
    for t in range(12):
        n = lens.tolist()
        want = [x + 1 if x or b < 4 else 0 for b, x in enumerate(n)]
        if t == 2:
            want[4] = 21                   # a prompt of its own
        if t == 5:
            want[2] += 17                  # drafted tokens ...
        if t == 6:
            want[2] -= 9                   # ... of which some are taken back
        if t == 8:
            want[4], want[5] = 0, 30       # one ends, another begins
        q_out, st = step(want)
        last = [max(e - 1, 0) for e in st[1:]]
        q = q_out[last].contiguous()
        out = torch.empty((B, Hq, D), device="cuda")
        lse = torch.empty((B, Hq), device="cuda")
        coli_kv_attn_shared(s, q, cache, out, 0.2, shared, group_start, lse=lse, ws=ws)
        qn = sr.to_np(q)
        for b in range(B):
            if not hist[b]:
                assert bool((out[b] == 0).all())
                continue
            K, V = np.stack([h[0] for h in hist[b]], 1), np.stack([h[1] for h in hist[b]], 1)      # [Hkv, n, D]
            for i in range(Hq):
                h, m = i // (Hq // Hkv), len(hist[b])
                tt = 0.2 * K[h] @ qn[b, i]
                w = np.exp(tt - tt.max())
                w /= w.sum()
                # a key is off by its own bound (75 half-steps of each element: norm 38, angle 34, rounding), then as the attention
                delta = (75 + D + 8) * 2.0 ** -24 * 0.2 * 2 * (np.abs(K[h]) @ np.abs(qn[b, i])).max()
                tol = (2 * delta + (m + 40) * 2.0 ** -24) * (w @ np.abs(V[h])) + 2.0 ** -23 * np.abs(w @ V[h])
                assert np.all(np.abs(out[b, i].double().cpu().numpy() - w @ V[h]) <= tol), f"step {t}, sequence {b}, head {i}"
        free.append(state.tolist()[1])
    held = sum(-(-x // page) for x in lens.tolist()) - 3 * P
    assert free[-1] == n_pages - held
