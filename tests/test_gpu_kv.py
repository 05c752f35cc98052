"""Paged key-value cache (append, attention of one new token, eviction by
running weight) through the C ABI against plain 64-bit forms
(tests/kv_reference.py, which also derives the bounds).  Rows of the pools
that no position owns hold NaN and infinities throughout."""
import numpy as np
import pytest

import kv_reference as ref
from sparse_moe_ffn_coli_amd import (COLI_BF16, COLI_F32, KvCache, KvShape, coli_index_topk, coli_kv_append,
                                     coli_kv_attn, coli_kv_attn_workspace_bytes, coli_kv_evict)

pytestmark = pytest.mark.gpu


def shape_of(c, B, Hq):
    return KvShape(B=B, Hq=Hq, Hkv=c["Hkv"], Dk=c["Dk"], Dv=c["Dv"], page=c["page"], n_pages=c["n_pages"],
                   max_pages=c["max_pages"], dtype=COLI_F32 if c["dtype"] == "f32" else COLI_BF16)


def cache_of(c):
    return KvCache(c["k"].cuda(), None if c["v"] is None else c["v"].cuda(), c["table"].cuda(), c["lens"].cuda())


def bits(t):
    import torch
    return t.view(torch.int32 if t.dtype == torch.float32 else torch.int16)


def guarded(shape, dtype, fill):
    """A tensor inside a larger buffer of `fill`; the second value checks that the buffer's rest is untouched."""
    import torch
    n = int(np.prod(shape))
    buf = torch.full((n + 512,), fill, dtype=dtype, device="cuda")
    view = buf[256:256 + n].view(shape)

    def check():
        rest = torch.cat([buf[:256], buf[256 + n:]])
        assert bool((rest == fill).all()), "written outside an output"
    return view, check


def queries(c, B, Hq, seed=1):
    import torch
    q = np.random.default_rng(seed).standard_normal((B, Hq, c["Dk"])).astype(np.float32)
    return torch.from_numpy(q).to(torch.float32 if c["dtype"] == "f32" else torch.bfloat16)


def within(got, want, tol, label):
    got = np.asarray(got, np.float64)
    empty = np.isneginf(want)
    assert np.array_equal(np.isneginf(got), empty), f"{label}: other rows are empty"
    got, want, tol = got[~empty], want[~empty], tol[~empty]
    assert np.all(np.isfinite(got)), f"{label}: not finite"
    over = np.abs(got - want) - tol
    assert over.size == 0 or over.max() <= 0, f"{label}: {over.max():.3e} over the bound, worst error {np.abs(got - want).max():.3e}"


def run_attn(c, Hq, scale, idx=None, acc_in=None, in_place=False, q=None, want=True):
    import torch
    B = len(c["lens"])
    q = queries(c, B, Hq) if q is None else q
    s, cache = shape_of(c, B, Hq), cache_of(c)
    dt = q.dtype
    out, out_ok = guarded((B, Hq, c["Dv"]), dt, 7.0)
    lse, lse_ok = guarded((B, Hq), torch.float32, 7.0)
    kw, checks = {}, [out_ok, lse_ok]
    if idx is not None:
        kw["idx"] = torch.from_numpy(idx).cuda()
    acc_out = None
    if acc_in is not None:
        acc_out, ok = guarded(acc_in.shape, torch.float32, 7.0)
        checks.append(ok)
        kw["acc_out"] = acc_out
        if in_place:
            acc_out.copy_(torch.from_numpy(acc_in))
            kw["acc_in"] = acc_out
        else:
            kw["acc_in"] = torch.from_numpy(acc_in).cuda()
    nb = coli_kv_attn_workspace_bytes(s, idx_k=0 if idx is None else idx.shape[1], acc=acc_in is not None)
    ws, ws_ok = guarded((nb,), torch.uint8, 0xA5)
    # a second pass on the same workspace: nothing may depend on what the first left there
    coli_kv_attn(s, q.cuda(), cache, out, scale, lse=lse, ws=ws, **kw)
    if not in_place:
        coli_kv_attn(s, q.cuda(), cache, out, scale, lse=lse, ws=ws, **kw)
    torch.cuda.synchronize()
    for ok in checks + [ws_ok]:
        ok()
    if not want:
        return out.cpu(), lse.cpu(), None if acc_out is None else acc_out.cpu()
    r = ref.attn(c, q, scale, idx, acc_in)
    label = f"{c['dtype']} B={B} Hq={Hq} Hkv={c['Hkv']} D={c['Dk']}/{c['Dv']} page={c['page']}"
    within(out.double().cpu().numpy(), r["out"], r["tol_out"], label + " out")
    within(lse.cpu().numpy(), r["lse"], r["tol_lse"], label + " lse")
    if acc_in is not None:
        got = acc_out.cpu().numpy()
        for b, n in enumerate(c["lens"].tolist()):
            within(got[b, :, :n], r["acc"][b, :, :n], r["tol_acc"][b, :, :n], label + " acc")
            rest = got[b, :, n:]
            assert np.array_equal(rest, acc_in[b, :, n:] if in_place else np.full_like(rest, 7.0)), "acc behind a length"
    print(label, "ok", flush=True)
    return out.cpu(), lse.cpu(), None if acc_out is None else acc_out.cpu()


BORDERS = [0, 1, 2, 31, 32, 33, 63, 65, 127, 128, 129, 257, 500]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv,Dk,Dv,page,latent", [
    (8, 2, 64, 64, 16, False),
    (3, 3, 8, 8, 1, False),               # the smallest heads, one position a page
    (12, 12, 80, 80, 2, False),           # widths that fill no tile
    (14, 2, 128, 128, 64, False),
    (5, 1, 96, 40, 4, False),             # values narrower than keys
    (4, 2, 72, 136, 8, False),            # and wider
    (34, 2, 192, 128, 32, False),         # 17 query heads: a second tile of one
    (16, 1, 256, 256, 128, False),
    (6, 2, 256, 200, 512, False),         # pages longer than every sequence
    (32, 1, 128, 64, 16, True),           # a latent cache of a small width
    (16, 1, 576, 512, 64, True),
    (20, 1, 576, 512, 16, True),
    (33, 1, 512, 512, 16, True),
    (100, 1, 320, 256, 32, True),
    (8, 4, 296, 264, 8, True),            # several latent heads, widths just past a tile
    (64, 1, 576, 512, 64, True),
    (128, 1, 576, 512, 64, True),
])
def test_attn_layouts(dtype, Hq, Hkv, Dk, Dv, page, latent):
    c = ref.make_cache(BORDERS, Hkv, Dk, Dv, page, dtype, latent, seed=Hq * 1000 + Dk)
    run_attn(c, Hq, 2.0 / np.sqrt(Dk))


@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0])
def test_attn_scales(scale):
    # 3.0: scores of several hundred, weights that underflow, references that move far
    c = ref.make_cache([700, 1, 45], 2, 128, 128, 16, "f32", seed=4)
    run_attn(c, 8, scale)


@pytest.mark.parametrize("dtype,latent,Hq,Dk,Dv", [("bf16", False, 8, 128, 128), ("f32", False, 2, 64, 64),
                                                   ("bf16", True, 64, 576, 512)])
def test_attn_one_long_sequence(dtype, latent, Hq, Dk, Dv):
    # cut over every range; the parts are joined
    c = ref.make_cache([20011], 1 if latent else 2, Dk, Dv, 16, dtype, latent, seed=5)
    run_attn(c, Hq, 2.0 / np.sqrt(Dk))


def test_attn_one_position():
    c = ref.make_cache([1], 2, 64, 64, 16, "bf16", seed=6)
    out, lse, _ = run_attn(c, 4, 0.125)


def test_attn_more_sequences_than_threads():
    rng = np.random.default_rng(7)
    lens = rng.integers(0, 150, size=700)
    lens[:300] = 0                        # a run of empty ones longer than a scan's width
    c = ref.make_cache(lens, 1, 64, 64, 16, "bf16", seed=7)
    run_attn(c, 3, 0.25)


def test_attn_nothing_anywhere():
    c = ref.make_cache([0, 0, 0], 2, 64, 64, 16, "bf16", seed=8)
    out, lse, _ = run_attn(c, 4, 0.125)
    assert bool((out == 0).all())


def test_attn_lengths_outside_the_table():
    import torch
    c = ref.make_cache([40, 64], 1, 64, 64, 16, "f32", seed=9, extra_cols=0)
    want = run_attn(c, 2, 0.2)
    c["lens"] = torch.tensor([40, 1 << 30], dtype=torch.int32)        # clamped to max_pages * page = 64
    got = run_attn(c, 2, 0.2, want=False)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    c["lens"] = torch.tensor([-5, 64], dtype=torch.int32)
    got = run_attn(c, 2, 0.2, want=False)
    assert bool((got[0][0] == 0).all()) and torch.equal(got[0][1], want[0][1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("latent,Hq,Dk,Dv", [(False, 6, 128, 128), (True, 40, 576, 512)])
def test_attn_hidden_pages(dtype, latent, Hq, Dk, Dv):
    # pages that do not exist inside a sequence; the second has none at all
    c = ref.make_cache([200, 90, 33], 1 if latent else 2, Dk, Dv, 8, dtype, latent, seed=10)
    c["table"][0, 3] = -1
    c["table"][0, 7:9] = c["n_pages"]
    c["table"][1, :] = -7
    c["table"][2, 0] = 1 << 30
    acc = np.random.default_rng(1).random((3, c["Hkv"], c["max_pages"] * 8)).astype(np.float32)
    run_attn(c, Hq, 0.1, acc_in=acc)


@pytest.mark.parametrize("dtype,Hq,Hkv,Dk,Dv,page,latent", [
    ("bf16", 8, 2, 128, 128, 16, False), ("f32", 4, 4, 80, 80, 32, False), ("bf16", 34, 2, 64, 64, 4, False),
    ("bf16", 64, 1, 576, 512, 64, True), ("f32", 18, 1, 576, 512, 64, True), ("bf16", 7, 1, 256, 256, 16, False)])
@pytest.mark.parametrize("in_place", [False, True])
def test_attn_running_weights(dtype, Hq, Hkv, Dk, Dv, page, latent, in_place):
    c = ref.make_cache([0, 1, 33, 1030, 515, 2048], Hkv, Dk, Dv, page, dtype, latent, seed=11)
    ld = -(-c["max_pages"] * page // 4) * 4 + 8
    acc = np.random.default_rng(2).random((6, Hkv, ld)).astype(np.float32)
    run_attn(c, Hq, 2.0 / np.sqrt(Dk), acc_in=acc, in_place=in_place)


def test_attn_running_weights_from_zero():
    import torch
    c = ref.make_cache([100, 64], 2, 64, 64, 16, "f32", seed=12)
    s, cache, q = shape_of(c, 2, 4), cache_of(c), queries(c, 2, 4)
    acc = torch.full((2, 2, c["max_pages"] * 16), 5.0, device="cuda")
    out = torch.empty((2, 4, 64), device="cuda")
    ws = torch.empty(coli_kv_attn_workspace_bytes(s, acc=True), dtype=torch.uint8, device="cuda")
    coli_kv_attn(s, q.cuda(), cache, out, 0.25, acc_out=acc, ws=ws)
    r = ref.attn(c, q, 0.25, acc_in=np.zeros(acc.shape, np.float32))
    for b, n in enumerate([100, 64]):
        within(acc[b, :, :n].cpu().numpy(), r["acc"][b, :, :n], r["tol_acc"][b, :, :n], "acc")
        # the weights of a cache head's query heads sum to their number
        assert np.abs(acc[b, :, :n].double().sum(-1).cpu().numpy() - 2.0).max() < 1e-4


@pytest.mark.parametrize("dtype,Hq,Hkv,Dk,Dv,page,latent,k", [
    ("bf16", 8, 2, 128, 128, 16, False, 77), ("f32", 3, 3, 64, 64, 1, False, 32), ("bf16", 64, 1, 576, 512, 64, True, 300),
    ("f32", 20, 1, 576, 512, 8, True, 65), ("bf16", 16, 1, 576, 512, 64, True, 1)])
def test_attn_listed_positions(dtype, Hq, Hkv, Dk, Dv, page, latent, k):
    lens = [0, 1, 40, 1000, 512, 77]
    c = ref.make_cache(lens, Hkv, Dk, Dv, page, dtype, latent, seed=13)
    rng = np.random.default_rng(3)
    idx = rng.integers(-3, 1200, size=(6, k)).astype(np.int32)       # -1s in between, positions past the end, doubles
    idx[4] = -1                                                      # nothing listed
    idx[5, :] = 5                                                    # one position, k times
    run_attn(c, Hq, 2.0 / np.sqrt(Dk), idx=idx)


def test_attn_listed_extreme_positions():
    c = ref.make_cache([100], 1, 64, 64, 16, "bf16", seed=14)
    idx = np.array([[-2 ** 31, 2 ** 31 - 1, 99, 100, 0, -1]], np.int32)
    run_attn(c, 4, 0.2, idx=idx)


def test_attn_over_an_index_selection():
    """The two together: positions selected by index scores, then attention over them."""
    import torch
    rng = np.random.default_rng(15)
    lens, k, tail = [900, 100, 2500, 0], 256, 4
    c = ref.make_cache(lens, 1, 576, 512, 64, "bf16", True, seed=15)
    L = c["max_pages"] * 64
    scores = torch.from_numpy(rng.standard_normal((4, L)).astype(np.float32)).cuda()
    idx = torch.empty((4, k), dtype=torch.int32, device="cuda")
    s, cache, q = shape_of(c, 4, 64), cache_of(c), queries(c, 4, 64)
    coli_index_topk(scores, k, idx, tail=tail, lens=cache.lens)
    out = torch.empty((4, 64, 512), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(coli_kv_attn_workspace_bytes(s, idx_k=k), dtype=torch.uint8, device="cuda")
    coli_kv_attn(s, q.cuda(), cache, out, 0.08, idx=idx, ws=ws)
    r = ref.attn(c, q, 0.08, idx=idx.cpu().numpy())
    within(out.double().cpu().numpy(), r["out"], r["tol_out"], "out")


def test_attn_repeats_bitwise():
    import torch
    c = ref.make_cache([3000, 17, 900], 2, 128, 128, 16, "bf16", seed=16)
    a = run_attn(c, 8, 0.2, want=False)
    for _ in range(3):
        b = run_attn(c, 8, 0.2, want=False)
        assert torch.equal(bits(a[0]), bits(b[0])) and torch.equal(bits(a[1]), bits(b[1]))


def test_attn_offsets_past_32_bits():
    """A pool of more than 2^32 elements; the sequence's pages lie at its end and its start."""
    import torch
    page, D, Hkv = 4096, 256, 4
    n_pages = 1100                        # 1100 * 4 * 4096 * 256 = 4.6e9 elements, 9.2 GB a pool
    g = torch.Generator(device="cuda").manual_seed(1)
    k = torch.zeros((n_pages, Hkv, page, D), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    for pg in (0, n_pages - 1):
        k[pg] = torch.randn(k[pg].shape, generator=g, device="cuda").bfloat16()
        v[pg] = torch.randn(k[pg].shape, generator=g, device="cuda").bfloat16()
    table = torch.tensor([[n_pages - 1, 0]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([page + 100], dtype=torch.int32, device="cuda")
    s = KvShape(1, 4, Hkv, D, D, page, n_pages, 2, COLI_BF16)
    q = torch.randn((1, 4, D), generator=g, device="cuda").bfloat16()
    out = torch.empty((1, 4, D), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(coli_kv_attn_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    coli_kv_attn(s, q, KvCache(k, v, table, lens), out, 0.1, ws=ws)
    c = dict(k=torch.cat([k[-1:], k[:1]]).cpu(), v=torch.cat([v[-1:], v[:1]]).cpu(), table=torch.tensor([[0, 1]]),
             lens=lens.cpu(), page=page, n_pages=2, max_pages=2, Hkv=Hkv, Dk=D, Dv=D, dtype="bf16")
    r = ref.attn(c, q.cpu(), 0.1)
    within(out.double().cpu().numpy(), r["out"], r["tol_out"], "out")


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------

def same_pool(got, want, label):
    import torch
    assert torch.equal(bits(got.cpu()), bits(want)), f"{label}: the pool differs"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("latent,Hkv,Dk,Dv,page", [(False, 2, 64, 64, 16), (False, 5, 80, 40, 1), (True, 1, 576, 512, 64),
                                                   (False, 12, 128, 128, 8), (False, 1, 8, 8, 2)])
def test_append_ragged(dtype, latent, Hkv, Dk, Dv, page):
    import torch
    lens, news = [50, 0, 7, 130, 1, 64], [50, 0, 3, 30, 1, 0]
    c = ref.make_cache(lens, Hkv, Dk, Dv, page, dtype, latent, seed=21)
    start = np.concatenate([[2], 2 + np.cumsum(news)]).astype(np.int32)      # two rows before the first sequence
    rows = int(start[-1]) + 3                                               # three behind the last
    rng = np.random.default_rng(1)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    k_new = torch.from_numpy(rng.standard_normal((rows, Hkv, Dk)).astype(np.float32)).to(dt)
    v_new = None if latent else torch.from_numpy(rng.standard_normal((rows, Hkv, Dv)).astype(np.float32)).to(dt)
    s, cache = shape_of(c, 6, Hkv), cache_of(c)
    coli_kv_append(s, k_new.cuda(), None if latent else v_new.cuda(), cache, start=torch.from_numpy(start).cuda())
    k2, v2 = ref.append(c, k_new, v_new, start)
    same_pool(cache.k, k2, "k")
    if not latent:
        same_pool(cache.v, v2, "v")


def test_append_one_each_and_more_rows_than_positions():
    import torch
    c = ref.make_cache([5, 0, 1, 33], 2, 64, 64, 16, "bf16", seed=22)
    s, cache = shape_of(c, 4, 2), cache_of(c)
    new = torch.randn(4, 2, 64).bfloat16()
    coli_kv_append(s, new.cuda(), new.cuda(), cache)
    k2, v2 = ref.append(c, new, new)
    same_pool(cache.k, k2, "k")
    same_pool(cache.v, v2, "v")
    # 9 rows for a sequence of 5 positions: the first 4 have no place; a page that does not exist takes nothing
    c["table"][3, 2] = -1
    start = torch.tensor([0, 9, 9, 10, 20], dtype=torch.int32)
    new = torch.randn(20, 2, 64).bfloat16()
    cache = cache_of(c)
    coli_kv_append(s, new.cuda(), new.cuda(), cache, start=start.cuda())
    k2, v2 = ref.append(c, new, new, start.numpy())
    same_pool(cache.k, k2, "k")
    same_pool(cache.v, v2, "v")


# ---------------------------------------------------------------------------
# evict
# ---------------------------------------------------------------------------

def run_evict(lens, Hkv, Dk, Dv, page, k, tail, dtype="bf16", latent=False, ties=False, new_extra=5, with_acc=True, seed=31,
              edit=None):
    import torch
    B = len(lens)
    cols = -(-k // page)
    c = ref.make_cache(lens, Hkv, Dk, Dv, page, dtype, latent, seed=seed, spare_pages=B * cols)
    ld = -(-c["max_pages"] * page // 4) * 4
    rng = np.random.default_rng(seed)
    acc = (rng.integers(0, 5, size=(B, Hkv, ld)) if ties else rng.random((B, Hkv, ld)) ** 4).astype(np.float32)
    for b, n in enumerate(lens):
        acc[b, :, n:] = np.nan            # behind a length: never looked at
    new_table = c["free"][:B * cols].reshape(B, cols).copy()
    if edit:
        edit(c, acc, new_table)
    s, cache = shape_of(c, B, Hkv), cache_of(c)
    new_lens, l_ok = guarded((B,), torch.int32, -9)
    kept, k_ok = guarded((B, Hkv, k), torch.int32, -9)
    new_acc, a_ok = guarded((B, Hkv, k + new_extra), torch.float32, -9.0)
    coli_kv_evict(s, cache, torch.from_numpy(acc).cuda(), k, torch.from_numpy(new_table).cuda(), new_lens, kept, tail=tail,
                  new_acc=new_acc if with_acc else None)
    torch.cuda.synchronize()
    for ok in (l_ok, k_ok, a_ok):
        ok()
    r = ref.evict(c, acc, k, tail, new_table, new_acc.cpu().numpy() if with_acc else None)
    assert np.array_equal(new_lens.cpu().numpy(), r["new_lens"])
    assert np.array_equal(kept.cpu().numpy(), r["kept"])
    if with_acc:
        assert np.array_equal(new_acc.cpu().numpy(), r["new_acc"])
    same_pool(cache.k, r["k"], "k")
    if not latent:
        same_pool(cache.v, r["v"], "v")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hkv,Dk,Dv,page,latent,k,tail", [
    (2, 64, 64, 16, False, 40, 4), (3, 80, 40, 1, False, 33, 0), (1, 576, 512, 64, True, 100, 7),
    (2, 8, 8, 2, False, 1, 0), (2, 128, 128, 8, False, 64, 1000), (1, 64, 64, 4, False, 1, 3),
])
def test_evict(dtype, Hkv, Dk, Dv, page, latent, k, tail):
    run_evict([0, 1, 39, 40, 41, 300], Hkv, Dk, Dv, page, k, tail, dtype, latent)


def test_evict_ties_and_no_weights_out():
    run_evict([500, 501], 2, 64, 64, 16, 128, 4, ties=True)
    run_evict([500, 20], 2, 64, 64, 16, 128, 4, with_acc=False)


def test_evict_budget_past_the_index_selections():
    run_evict([9000, 100, 4097], 1, 8, 8, 64, 4097, 16, ties=True)


def test_evict_budget_longer_than_the_table():
    run_evict([30, 17], 2, 64, 64, 16, 100, 4)


def test_evict_many_rows():
    run_evict(list(np.random.default_rng(3).integers(0, 90, size=70)), 4, 8, 8, 16, 24, 2, ties=True)


def test_evict_pages_that_do_not_exist():
    def edit(c, acc, new_table):
        c["table"][1, 1] = -1
        new_table[0, 1] = c["n_pages"]
    run_evict([100, 90], 2, 64, 64, 16, 40, 4, edit=edit)


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,latent,Hq,Hkv,Dk,Dv", [("bf16", False, 8, 2, 64, 64), ("f32", True, 6, 1, 320, 256)])
def test_serving_run(dtype, latent, Hq, Hkv, Dk, Dv):
    """Prompts go in, tokens are decoded with running weights kept, the cache is cut to a budget, decoding goes on in
    the new pages: every step against the plain forms."""
    import torch
    page, k, tail, steps = 8, 48, 4, 5
    prompts = [60, 3, 100]
    B = 3
    rng = np.random.default_rng(41)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    cols = -(-(max(prompts) + steps + 1) // page)
    n_pages = B * cols * 2
    ids = rng.permutation(n_pages).astype(np.int32)
    table, new_table = ids[:B * cols].reshape(B, cols), ids[B * cols:].reshape(B, cols)
    c = dict(k=torch.full((n_pages, Hkv, page, Dk), float("nan"), dtype=dt),
             v=None if latent else torch.full((n_pages, Hkv, page, Dv), float("nan"), dtype=dt),
             table=torch.from_numpy(table), lens=torch.tensor(prompts, dtype=torch.int32), page=page, n_pages=n_pages,
             max_pages=cols, Hkv=Hkv, Dk=Dk, Dv=Dv, dtype=dtype)
    s, dev = shape_of(c, B, Hq), cache_of(c)
    scale = 1.5 / np.sqrt(Dk)
    ws = torch.empty(coli_kv_attn_workspace_bytes(s, acc=True), dtype=torch.uint8, device="cuda")
    acc = torch.zeros((B, Hkv, cols * page), device="cuda")
    acc_ref, acc_tol = np.zeros(acc.shape), np.zeros(acc.shape)

    def fresh(*size):
        return torch.from_numpy(rng.standard_normal(size).astype(np.float32)).to(dt)

    def put(rows, start):
        kn, vn = fresh(rows, Hkv, Dk), None if latent else fresh(rows, Hkv, Dv)
        coli_kv_append(s, kn.cuda(), None if latent else vn.cuda(), dev, start=None if start is None else torch.from_numpy(start).cuda())
        c["k"], c["v"] = ref.append(c, kn, vn, start)

    def decode():
        nonlocal acc_ref, acc_tol
        q = fresh(B, Hq, Dk)
        out = torch.empty((B, Hq, Dv), dtype=dt, device="cuda")
        coli_kv_attn(s, q.cuda(), dev, out, scale, acc_in=acc, acc_out=acc, ws=ws)
        r = ref.attn(c, q, scale, acc_in=acc_ref)
        within(out.double().cpu().numpy(), r["out"], r["tol_out"], "out")
        acc_ref, acc_tol = r["acc"], acc_tol + r["tol_acc"]
        within(acc.cpu().numpy(), acc_ref, acc_tol, "acc")

    start = np.concatenate([[0], np.cumsum(prompts)]).astype(np.int32)
    put(int(start[-1]), start)
    decode()
    for _ in range(steps):
        c["lens"] += 1
        dev.lens.add_(1)
        put(B, None)
        decode()
    # the kept positions go by the weights that the device holds (ties and rounding are its own)
    host_acc = acc.cpu().numpy()
    new_lens = torch.empty(B, dtype=torch.int32, device="cuda")
    kept = torch.empty((B, Hkv, k), dtype=torch.int32, device="cuda")
    new_acc = torch.empty((B, Hkv, cols * page), device="cuda")
    nt = torch.from_numpy(new_table).cuda()
    coli_kv_evict(s, dev, acc, k, nt, new_lens, kept, tail=tail, new_acc=new_acc)
    r = ref.evict(c, host_acc, k, tail, new_table, new_acc.cpu().numpy())
    assert np.array_equal(kept.cpu().numpy(), r["kept"]) and np.array_equal(new_acc.cpu().numpy(), r["new_acc"])
    c.update(k=r["k"], v=r["v"], table=torch.from_numpy(new_table), lens=torch.from_numpy(r["new_lens"]))
    same_pool(dev.k, c["k"], "k after the eviction")
    dev = KvCache(dev.k, dev.v, nt, new_lens)
    acc, acc_ref, acc_tol = new_acc, new_acc.cpu().numpy().astype(np.float64), np.zeros(acc.shape)
    for _ in range(steps):
        c["lens"] += 1
        dev.lens.add_(1)
        put(B, None)
        decode()


def test_graph_replays():
    """A captured decode step (append, attention with running weights) replayed with eager work in between."""
    import torch
    c = ref.make_cache([300, 40, 0, 77], 2, 128, 128, 16, "bf16", seed=51)
    s, dev = shape_of(c, 4, 8), cache_of(c)
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randn((4, 8, 128), generator=g, device="cuda").bfloat16()
    new = torch.randn((4, 2, 128), generator=g, device="cuda").bfloat16()
    ld = c["max_pages"] * 16
    acc_in = torch.rand((4, 2, ld), generator=g, device="cuda")
    acc_out = torch.zeros((4, 2, ld), device="cuda")
    out, lse = torch.empty((4, 8, 128), dtype=torch.bfloat16, device="cuda"), torch.empty((4, 8), device="cuda")
    ws = torch.empty(coli_kv_attn_workspace_bytes(s, acc=True), dtype=torch.uint8, device="cuda")

    def step(stream=None):
        coli_kv_append(s, new, new, dev, stream=stream)
        coli_kv_attn(s, q, dev, out, 0.2, acc_in=acc_in, acc_out=acc_out, lse=lse, ws=ws, stream=stream)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        q.copy_(torch.randn((4, 8, 128), generator=g, device="cuda").bfloat16())
        new.copy_(torch.randn((4, 2, 128), generator=g, device="cuda").bfloat16())
        dev.lens.copy_(torch.tensor([300 - i, 40 + i, i, 77], dtype=torch.int32))
        step()
        want = [t.clone() for t in (out, lse, acc_out)]
        for t in (out, lse):
            t.fill_(3.0)
        ws.fill_(0x5A)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(bits(out), bits(want[0])) and torch.equal(lse, want[1]) and torch.equal(acc_out, want[2])


def test_two_streams_at_once():
    """Two calls in flight, a workspace each, on streams of their own."""
    import torch
    c = ref.make_cache([4000, 100], 2, 128, 128, 16, "bf16", seed=52)
    s, dev = shape_of(c, 2, 8), cache_of(c)
    qs = [queries(c, 2, 8, seed=i).cuda() for i in range(2)]
    outs = [torch.empty((2, 8, 128), dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    wss = [torch.empty(coli_kv_attn_workspace_bytes(s), dtype=torch.uint8, device="cuda") for _ in range(2)]
    for i in range(2):
        coli_kv_attn(s, qs[i], dev, outs[2 + i], 0.2, ws=wss[0])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for i in range(2):
            coli_kv_attn(s, qs[i], dev, outs[i], 0.2, ws=wss[i], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(bits(outs[i]), bits(outs[2 + i]))


def test_refusals_of_the_binding():
    import torch
    c = ref.make_cache([40], 2, 64, 64, 16, "bf16", seed=53)
    s, dev = shape_of(c, 1, 4), cache_of(c)
    q, out = queries(c, 1, 4).cuda(), torch.empty((1, 4, 64), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(coli_kv_attn_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    for bad in (dict(q=q.float()), dict(q=q[:, :2]), dict(q=q.cpu()), dict(out=out.float()),
                dict(q=q.transpose(0, 1).contiguous().transpose(0, 1).expand(1, 4, 64)[..., ::1].permute(0, 2, 1)),
                dict(lse=torch.empty(4, device="cuda")), dict(idx=torch.zeros((1, 3), dtype=torch.int64, device="cuda"))):
        kw = dict(q=q, out=out) | bad
        with pytest.raises(ValueError):
            coli_kv_attn(s, kw.pop("q"), dev, kw.pop("out"), 0.1, ws=ws, **kw)


@pytest.mark.parametrize("Hq,Dk,Dv", [(20, 576, 512), (64, 576, 512), (100, 576, 512), (40, 320, 256)])
@pytest.mark.parametrize("scale", [-0.2, 3.0])
def test_attn_latent_scores_far_apart(Hq, Dk, Dv, scale):
    # scores of several hundred, growing along the sequence: later ones pass the first stage's by far more than 2^60
    c = ref.make_cache([1500, 1, 70, 0], 1, Dk, Dv, 16, "bf16", True, seed=61)
    for b, n in enumerate(c["lens"].tolist()):
        for p in range(n):
            c["k"][c["table"][b, p // 16], :, p % 16] *= 0.05 + 1.5 * p / 1500
    run_attn(c, Hq, scale)


def test_attn_latent_growing_scores_of_one_head():
    # one query head of 64 meets ever larger scores, the others stay near zero
    import torch
    c = ref.make_cache([900], 1, 576, 512, 64, "bf16", True, seed=62)
    q = queries(c, 1, 64) * 0.01
    q[0, 37] = 0
    q[0, 37, 5] = 4.0
    for p in range(900):
        c["k"][c["table"][0, p // 64], :, p % 64, 5] = 0.25 * (p // 2)
    run_attn(c, 64, 1.0, q=q)


@pytest.mark.parametrize("Hq", [20, 64, 100])
def test_attn_latent_long_ranges(Hq):
    """Sequences that share their pages (a common prompt), so many positions that a workgroup's range is longer than
    the block of positions it looks up at a time, and spans several sequences."""
    import torch
    B, n, page = 70, 16000, 64
    c = ref.make_cache([n], 1, 320, 256, page, "bf16", True, seed=63)
    lens = np.full(B, n)
    lens[1::3] = np.random.default_rng(1).integers(0, n, size=len(lens[1::3]))
    c["table"] = c["table"].expand(B, -1).contiguous()
    c["lens"] = torch.from_numpy(lens.astype(np.int32))
    s, dev, q = shape_of(c, B, Hq), cache_of(c), queries(c, B, Hq)
    out = torch.empty((B, Hq, 256), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(coli_kv_attn_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    coli_kv_attn(s, q.cuda(), dev, out, 0.1, ws=ws)
    pick = [0, 1, 4, 35, 69]
    few = dict(c, table=c["table"][pick], lens=c["lens"][pick])
    r = ref.attn(few, q[pick], 0.1)
    within(out[pick].double().cpu().numpy(), r["out"], r["tol_out"], "out")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv,Dk,Dv,page,latent", [
    (8, 2, 64, 64, 16, False), (3, 3, 8, 8, 1, False), (12, 12, 80, 80, 2, False), (14, 2, 128, 128, 64, False),
    (5, 1, 96, 40, 4, False), (34, 2, 192, 128, 32, False), (16, 1, 256, 256, 128, False), (32, 1, 128, 64, 16, True),
    (16, 1, 576, 512, 64, True), (100, 1, 320, 256, 32, True), (8, 4, 296, 264, 8, True), (3, 1, 264, 8, 16, True),
    (64, 1, 512, 512, 64, True), (40, 1, 400, 384, 16, True)])
def test_attn_rows_cut_into_ranges(dtype, Hq, Hkv, Dk, Dv, page, latent):
    # a table long enough that rows are not taken whole: ranges begin and end inside them
    c = ref.make_cache(BORDERS + [1100, 0, 4000], Hkv, Dk, Dv, page, dtype, latent, seed=Hq * 1000 + Dk + 1)
    run_attn(c, Hq, 2.0 / np.sqrt(Dk))
    acc = np.random.default_rng(2).random((16, Hkv, c["max_pages"] * page // 4 * 4 + 4)).astype(np.float32)
    run_attn(c, Hq, 2.0 / np.sqrt(Dk), acc_in=acc)


@pytest.mark.parametrize("dtype,Hq,Dk,Dv,latent", [("bf16", 4, 128, 128, False), ("f32", 2, 576, 512, True)])
def test_attn_more_heads_than_a_workgroups_threads(dtype, Hq, Dk, Dv, latent):
    c = ref.make_cache([40, 3], 1, Dk, Dv, 16, dtype, latent, seed=71)
    acc = np.random.default_rng(2).random((2, 1, c["max_pages"] * 16)).astype(np.float32)
    run_attn(c, 260 * Hq // 2, 0.1, acc_in=acc)


@pytest.mark.parametrize("k,ties", [(300, False), (5000, True), (40000, False)])
def test_evict_rows_past_the_key_cache(k, ties):
    # rows of more than 32768 positions beside shorter ones, budgets that are staged and ones that are not
    run_evict([70001, 32769, 32768, 4096, 12], 1, 8, 8, 64, k, 5, ties=ties, dtype="f32")


def test_evict_weights_of_every_kind():
    # infinities, zeros of both signs, subnormals, one value everywhere: the last positions and the lowest stay
    def edit(c, acc, new_table):
        acc[0, 0, :400] = 0.0
        acc[0, 0, 1:400:2] = -0.0
        acc[0, 1, :400] = np.inf
        acc[1, 0, :300] = 1e-45
        acc[1, 0, 7] = -1e-45
        acc[1, 1, :300] = -np.inf
        acc[1, 1, 250:260] = 3.0
    run_evict([400, 300], 2, 8, 8, 16, 100, 4, edit=edit, dtype="f32")


def test_empty_arguments_do_not_count_as_absent():
    import torch
    c = ref.make_cache([40], 2, 64, 64, 16, "bf16", seed=61)
    s, dev = shape_of(c, 1, 4), cache_of(c)
    q, out = queries(c, 1, 4).cuda(), torch.empty((1, 4, 64), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(coli_kv_attn_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    for bad in (dict(idx=torch.empty((1, 0), dtype=torch.int32, device="cuda")), dict(acc_out=torch.empty((1, 2, 0), device="cuda"))):
        with pytest.raises(ValueError):
            coli_kv_attn(s, q, dev, out, 0.1, ws=ws, **bad)
    i32 = dict(dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        coli_kv_evict(s, dev, torch.zeros((1, 2, 48), device="cuda"), 8, torch.zeros((1, 1), **i32), torch.zeros(1, **i32),
                      torch.zeros((1, 2, 8), **i32), new_acc=torch.empty((1, 2, 0), device="cuda"))


@pytest.mark.parametrize("Hq,Dk,Dv,page", [(100, 576, 512, 64), (128, 320, 256, 32), (70, 264, 8, 64), (40, 256, 256, 64),
                                           (64, 136, 72, 32), (34, 200, 128, 16), (20, 192, 192, 1)])
def test_attn_latent_long_tables(Hq, Dk, Dv, page):
    # room for many more positions than there are: calls are laid out by the room
    c = ref.make_cache(BORDERS + [1100, 0, 2500], 1, Dk, Dv, page, "bf16", True, seed=Hq + Dk, extra_cols=(1 << 15) // page)
    run_attn(c, Hq, 2.0 / np.sqrt(Dk))
    acc = np.random.default_rng(2).random((16, 1, c["max_pages"] * page // 4 * 4 + 4)).astype(np.float32)
    run_attn(c, Hq, 2.0 / np.sqrt(Dk), acc_in=acc)
    idx = np.random.default_rng(3).integers(-1, 1200, size=(16, 2100)).astype(np.int32)
    run_attn(c, Hq, 2.0 / np.sqrt(Dk), idx=idx)


@pytest.mark.parametrize("Hq,Dk,Dv", [(100, 576, 512), (128, 320, 256), (33, 256, 256)])
def test_attn_latent_scores_far_apart_in_long_tables(Hq, Dk, Dv):
    c = ref.make_cache([1500, 1, 70, 0], 1, Dk, Dv, 16, "bf16", True, seed=64, extra_cols=1 << 13)
    for b, n in enumerate(c["lens"].tolist()):
        for p in range(n):
            c["k"][c["table"][b, p // 16], :, p % 16] *= 0.05 + 1.5 * p / 1500
    run_attn(c, Hq, 3.0)


@pytest.mark.parametrize("Hq", [16, 100])
def test_attn_latent_one_row_in_many_parts(Hq):
    # a row that every workgroup has a part of, alone and beside an empty one
    for lens in ([70000], [0, 66000, 3]):
        run_attn(ref.make_cache(lens, 1, 320, 256, 64, "bf16", True, seed=65), Hq, 0.1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hkv,D", [(8, 64), (5, 128), (3, 256)])
@pytest.mark.parametrize("B,longest", [(3, 40), (40, 60), (130, 130), (260, 30), (400, 250)])
def test_attn_short_rows_of_any_number(dtype, Hkv, D, B, longest):
    # rows that a workgroup takes whole, with one wave or several
    lens = np.random.default_rng(B).integers(0, longest + 1, size=B)
    lens[0], lens[-1] = longest, 0
    c = ref.make_cache(lens, Hkv, D, D, 16, dtype, seed=B + D, extra_cols=0)
    run_attn(c, 2 * Hkv, 1.0 / np.sqrt(D))
    if B == 40:
        acc = np.random.default_rng(2).random((B, Hkv, c["max_pages"] * 16)).astype(np.float32)
        run_attn(c, 2 * Hkv, 1.0 / np.sqrt(D), acc_in=acc)


def test_a_handle_whose_tensors_moved():
    import torch
    c = ref.make_cache([100, 37], 2, 64, 64, 16, "bf16", seed=66)
    s, dev, q = shape_of(c, 2, 4), cache_of(c), queries(c, 2, 4)
    ws = torch.empty(coli_kv_attn_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    outs = [torch.empty((2, 4, 64), dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    coli_kv_attn(s, q.cuda(), dev, outs[0], 0.1, ws=ws)
    half = torch.tensor([50, 37], dtype=torch.int32, device="cuda")
    dev.lens.set_(half)                          # the handle's tensor now has other memory
    coli_kv_attn(s, q.cuda(), dev, outs[1], 0.1, ws=ws)
    few = dict(c, lens=half.cpu())
    coli_kv_attn(s, q.cuda(), cache_of(few), outs[2], 0.1, ws=ws)
    assert torch.equal(bits(outs[1]), bits(outs[2])) and not torch.equal(bits(outs[0]), bits(outs[1]))


@pytest.mark.parametrize("Hq,Hkv,Dk,Dv", [(6, 2, 192, 192), (5, 5, 136, 192), (20, 1, 144, 136), (4, 2, 200, 248), (9, 3, 256, 72),
                                          (4, 4, 192, 256), (2, 2, 8, 184)])
def test_attn_f32_widths(Hq, Hkv, Dk, Dv):
    # every way a wide fp32 row is taken, whole and cut
    c = ref.make_cache(BORDERS + [700], Hkv, Dk, Dv, 16, "f32", seed=Dk + Dv)
    run_attn(c, Hq, 2.0 / np.sqrt(Dk))
    c = ref.make_cache([1, 1300, 0, 257], Hkv, Dk, Dv, 64, "f32", seed=Dk + Dv, extra_cols=40)
    acc = np.random.default_rng(2).random((4, Hkv, c["max_pages"] * 64)).astype(np.float32)
    run_attn(c, Hq, 2.0 / np.sqrt(Dk), acc_in=acc)


@pytest.mark.parametrize("Dk,tokens", [(520, 1), (344, 2)])
def test_append_of_more_rows_than_a_launch_holds(Dk, tokens):
    """New tokens on both sides of a launch's last workgroup (2^22 of them, of one or two tokens each).  Sequences of
    a few positions: the rows before their last ones have no place, and are not looked at."""
    import torch
    border, lens, page = tokens << 22, [8, 6], 4
    c = ref.make_cache(lens, 1, Dk, 64, page, "f32", True, seed=81)
    s, cache = shape_of(c, 2, 1), cache_of(c)
    start = torch.tensor([0, border + 4, border + 13], dtype=torch.int32)
    rows = border + 15
    new = torch.empty((rows, 1, Dk), device="cuda")
    new[border - 64:] = torch.randn((rows - border + 64, 1, Dk), generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    coli_kv_append(s, new, None, cache, start=start.cuda())
    k2, _ = ref.append(c, new[border - 64:].cpu(), None, start.numpy() - (border - 64) * (start.numpy() > 0))
    same_pool(cache.k, k2, "k")


def test_evict_keeps_the_newest_beside_nans():
    # running weights of a row that met a NaN: the newest positions stay all the same
    import torch
    c = ref.make_cache([300], 1, 8, 8, 16, "f32", seed=82, spare_pages=4)
    s, cache, k, tail = shape_of(c, 1, 1), cache_of(c), 64, 4
    acc = torch.full((1, 1, c["max_pages"] * 16), 0x7fffffff, dtype=torch.int32, device="cuda").view(torch.float32)
    new_lens, kept = torch.empty(1, dtype=torch.int32, device="cuda"), torch.empty((1, 1, k), dtype=torch.int32, device="cuda")
    coli_kv_evict(s, cache, acc, k, torch.from_numpy(c["free"][:4][None]).cuda(), new_lens, kept, tail=tail)
    assert kept[0, 0].tolist() == list(range(k - tail)) + list(range(300 - tail, 300))


INFINITE = [("bf16", 8, 2, 128, 128, False), ("bf16", 6, 3, 80, 80, False), ("bf16", 5, 1, 96, 40, False),
            ("bf16", 4, 2, 72, 136, False), ("bf16", 17, 1, 64, 64, False), ("bf16", 4, 2, 200, 248, False),
            ("f32", 4, 2, 128, 128, False), ("f32", 3, 3, 8, 8, False), ("f32", 4, 4, 192, 128, False),
            ("f32", 4, 2, 200, 256, False), ("f32", 18, 1, 576, 512, True), ("f32", 20, 1, 304, 256, True),
            ("bf16", 20, 1, 576, 512, True), ("bf16", 64, 1, 576, 512, True), ("bf16", 100, 1, 520, 512, True),
            ("bf16", 33, 1, 400, 384, True), ("bf16", 40, 1, 320, 256, True), ("bf16", 100, 1, 264, 8, True), ("bf16", 40, 1, 200, 128, True)]


def hidden_by_scores(c, q, column, bad, every=5):
    """Keys of every fifth position (pages of one; of a sequence of three all, if `bad` is infinite) get `bad` in a
    column where every query is positive, so that their scores are -inf or far below all others: the same cache with
    those pages hidden is what the plain form reads."""
    import torch
    q[..., column] = q[..., column].abs() + 0.5
    same = dict(c, table=c["table"].clone())
    for b, n in enumerate(c["lens"].tolist()):
        for p in range(n):
            if p % every == 1 or (n == 3 and np.isinf(bad)):
                c["k"][c["table"][b, p], :, 0, column] = bad
                same["table"][b, p] = -1
    return same


@pytest.mark.parametrize("dtype,Hq,Hkv,Dk,Dv,latent", INFINITE)
@pytest.mark.parametrize("bad", [-np.inf, "lowest"])
@pytest.mark.parametrize("room", [0, 1 << 13])
def test_attn_scores_of_minus_infinity(dtype, Hq, Hkv, Dk, Dv, latent, bad, room):
    """Live keys with an infinity or the type's lowest value: their positions have no weight, whatever the sign of the
    scale's rounding error, and a sequence of nothing but infinities is an empty row."""
    import torch
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    for scale in (2.0, 2.0 / np.sqrt(Dk), 2.0 / np.sqrt(96)):
        c = ref.make_cache([40, 3, 0, 300], Hkv, Dk, Dv, 1, dtype, latent, seed=91, extra_cols=room + 1)
        q = queries(c, 4, Hq)
        same = hidden_by_scores(c, q, Dk - 1, torch.finfo(dt).min if bad == "lowest" else bad)
        acc = np.random.default_rng(2).random((4, Hkv, c["max_pages"] // 4 * 4 + 4)).astype(np.float32)
        for acc_in in (None, acc):
            got = run_attn(c, Hq, scale, acc_in=acc_in, q=q, want=False)
            r = ref.attn(same, q, scale, acc_in=acc_in)
            within(got[0].double().numpy(), r["out"], r["tol_out"], "out")
            within(got[1].numpy(), r["lse"], r["tol_lse"], "lse")
            for b, n in enumerate(c["lens"].tolist()):
                if acc_in is not None:
                    within(got[2][b, :, :n].numpy(), r["acc"][b, :, :n], r["tol_acc"][b, :, :n], "acc")


@pytest.mark.parametrize("dtype,Hq,Hkv,Dk,Dv,latent", [
    ("bf16", 8, 2, 128, 128, False), ("f32", 6, 2, 80, 80, False), ("f32", 4, 2, 256, 256, False), ("f32", 20, 1, 576, 512, True),
    ("bf16", 20, 1, 576, 512, True), ("bf16", 100, 1, 576, 512, True), ("bf16", 40, 1, 320, 256, True)])
@pytest.mark.parametrize("room", [0, 1 << 13])
@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_attn_nan_and_infinite_queries(dtype, Hq, Hkv, Dk, Dv, latent, room, bad):
    """One query head of each sequence has a NaN (or an infinity, so that its scores are +inf, -inf and no number): its
    out, lse and its cache head's running weights are NaN, in rows taken whole and cut, and nothing else is."""
    import torch
    lens = [700, 1, 0, 300]
    c = ref.make_cache(lens, Hkv, Dk, Dv, 16, dtype, latent, seed=92, extra_cols=room // 16 + 1)
    q, G = queries(c, 4, Hq), Hq // Hkv
    heads = [Hq - 1, 0, 1, Hq // 2]
    clean = q.clone()
    for b, i in enumerate(heads):
        q[b, i, 3] = bad
    acc = np.random.default_rng(2).random((4, Hkv, c["max_pages"] * 16)).astype(np.float32)
    if np.isinf(bad):                        # a sequence of one position: its one score is +inf
        c["k"][c["table"][1, 0], :, 0, 3] = 1.0
    for acc_in in (None, acc):
        out, lse, got_acc = run_attn(c, Hq, 0.2, acc_in=acc_in, q=q, want=False)
        r = ref.attn(c, clean, 0.2, acc_in=acc_in)
        for b, n in enumerate(lens):
            hit = np.zeros(Hq, bool)
            hit[heads[b]] = n > 0
            assert bool(torch.isnan(out[b, hit]).all()) and bool(torch.isnan(lse[b, hit]).all()), f"sequence {b}"
            within(out[b, ~hit].double().numpy(), r["out"][b, ~hit], r["tol_out"][b, ~hit], "out")
            within(lse[b, ~hit].numpy(), r["lse"][b, ~hit], r["tol_lse"][b, ~hit], "lse")
            if acc_in is not None:
                h = hit.reshape(Hkv, G).any(1)
                assert bool(torch.isnan(got_acc[b, h, :n]).all()), f"running weights of sequence {b}"
                within(got_acc[b, ~h, :n].numpy(), r["acc"][b, ~h, :n], r["tol_acc"][b, ~h, :n], "acc")


def test_attn_nan_in_one_part_of_a_cut_row():
    # a live key that is all NaN: whatever part of the row it lies in, all heads that read it are NaN
    import torch
    for dtype, latent, Hq, D in (("bf16", False, 4, 128), ("bf16", True, 64, 576), ("f32", False, 3, 64)):
        for at in (0, 9000, 20010):
            c = ref.make_cache([20011, 50], 1, D, D if not latent else 512, 16, dtype, latent, seed=93)
            c["k"][c["table"][0, at // 16], :, at % 16] = float("nan")
            acc = np.zeros((2, 1, c["max_pages"] * 16), np.float32)
            out, lse, got = run_attn(c, Hq, 0.1, acc_in=acc, want=False)
            assert bool(torch.isnan(out[0]).all()) and bool(torch.isnan(lse[0]).all()) and bool(torch.isnan(got[0, 0, :20011]).all())
            assert not bool(torch.isnan(out[1]).any()) and not bool(torch.isnan(lse[1]).any()) and not bool(torch.isnan(got[1, 0, :50]).any())


@pytest.mark.parametrize("Hq,Dk,Dv", [(20, 576, 512), (64, 576, 512), (100, 576, 512), (100, 520, 512), (40, 320, 256), (100, 264, 256)])
@pytest.mark.parametrize("room", [0, 1 << 14])
@pytest.mark.parametrize("growth", [15.0, 50.0, 90.0])
def test_attn_latent_large_values(Hq, Dk, Dv, room, growth):
    """Values near 1e25 beside scores that grow by 2^15 to 2^90 along a sequence: sums under the first stage's reference
    pass fp32's end, the results are far inside it."""
    c = ref.make_cache([900, 0, 70, 1], 1, Dk, Dv, 16, "bf16", True, seed=94, extra_cols=room // 16 + 1)
    q = queries(c, 4, Hq)
    q[..., :Dv] = 0                          # scores come from the columns that are no values
    q[..., Dv] = 1.0
    for b, n in enumerate(c["lens"].tolist()):
        for p in range(n):
            row = c["k"][c["table"][b, p // 16], :, p % 16]
            row[..., :Dv] *= 1e25
            row[..., Dv:] *= 0.125
            row[..., Dv] = p / n
    run_attn(c, Hq, growth * np.log(2.0), q=q)
    acc = np.random.default_rng(2).random((4, 1, c["max_pages"] * 16)).astype(np.float32)
    run_attn(c, Hq, growth * np.log(2.0), q=q, acc_in=acc)


def test_a_handle_whose_tensors_change_in_place():
    # the memory stays, the sizes, the order or the type do not: refused, and taken again once they are as before
    import torch
    c = ref.make_cache([100, 37], 2, 64, 64, 16, "bf16", seed=67)
    s, q = shape_of(c, 2, 4), queries(c, 2, 4).cuda()
    ws = torch.empty(coli_kv_attn_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    outs = [torch.empty((2, 4, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    changes = [("lens", lambda t: t.set_(t[:1])), ("lens", lambda t: t.resize_(1)), ("table", lambda t: t.transpose_(0, 1)),
               ("table", lambda t: t.resize_(2, 3)), ("k", lambda t: t.transpose_(1, 2)), ("v", lambda t: t.transpose_(0, 3)),
               ("k", lambda t: setattr(t, "data", t.data.view(torch.float16))), ("lens", lambda t: setattr(t, "data", t.data.view(torch.float32)))]
    for name, change in changes:
        dev = cache_of(c)
        coli_kv_attn(s, q, dev, outs[0], 0.1, ws=ws)
        t = getattr(dev, name)
        before, at = t.detach(), t.data_ptr()
        change(t)
        assert t.data_ptr() == at
        new = torch.zeros((2, 2, 64), dtype=torch.bfloat16, device="cuda")
        with pytest.raises(ValueError):
            coli_kv_attn(s, q, dev, outs[1], 0.1, ws=ws)
        with pytest.raises(ValueError):
            coli_kv_append(s, new, new, dev)
        t.data = before
        coli_kv_attn(s, q, dev, outs[1], 0.1, ws=ws)
        assert torch.equal(bits(outs[0]), bits(outs[1]))


def big_pool(pages=1100):
    """Pools of more than 2^32 elements (9 GB each), zero but for the first and the last page."""
    import torch
    page, D, Hkv = 4096, 256, 4
    g = torch.Generator(device="cuda").manual_seed(1)
    k = torch.zeros((pages, Hkv, page, D), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    for pool in (k, v):
        for pg in (0, pages - 1):
            pool[pg] = torch.randn(pool[pg].shape, generator=g, device="cuda").bfloat16()
    return k, v, page, D, Hkv, g


def test_append_offsets_past_32_bits():
    import torch
    k, v, page, D, Hkv, g = big_pool()
    n = k.shape[0]
    table = torch.tensor([[n - 1, n - 2]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([page + 3], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    new = torch.randn((8, Hkv, D), generator=g, device="cuda").bfloat16()
    want = [torch.cat([p[n - 2:], p[:1]]) for p in (k, v)]
    for x in range(8):
        p = page + 3 - 8 + x
        for w, rows in zip(want, (new, -new)):
            w[1 if p < page else 0, :, p % page] = rows[x]
    coli_kv_append(KvShape(1, 4, Hkv, D, D, page, n, 2, COLI_BF16), new, -new, KvCache(k, v, table, lens), start=start)
    for pool, w in zip((k, v), want):
        assert torch.equal(bits(torch.cat([pool[n - 2:], pool[:1]])), bits(w))
        assert not bool(pool[1:n - 2].any()), "written elsewhere"


def test_evict_offsets_past_32_bits():
    import torch
    k, v, page, D, Hkv, g = big_pool()
    n, keep = k.shape[0], 700
    table = torch.tensor([[n - 1]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([page], dtype=torch.int32, device="cuda")
    acc = torch.stack([torch.randperm(page, generator=g, device="cuda") for _ in range(Hkv)])[None].float()
    new_lens, kept = torch.empty(1, dtype=torch.int32, device="cuda"), torch.empty((1, Hkv, keep), dtype=torch.int32, device="cuda")
    last = [p[n - 1:].clone() for p in (k, v)]
    coli_kv_evict(KvShape(1, 4, Hkv, D, D, page, n, 1, COLI_BF16), KvCache(k, v, table, lens), acc, keep,
                  torch.tensor([[n - 2]], dtype=torch.int32, device="cuda"), new_lens, kept)
    want = torch.topk(acc[0], keep, dim=-1).indices.sort(-1).values
    assert torch.equal(kept[0].long(), want)
    for pool, old in zip((k, v), last):
        assert torch.equal(bits(pool[n - 1:]), bits(old)) and not bool(pool[1:n - 2].any()) and not bool(pool[n - 2, :, keep:].any())
        for h in range(Hkv):
            assert torch.equal(bits(pool[n - 2, h, :keep]), bits(old[0, h, want[h]]))


@pytest.mark.parametrize("dtype,Hq,Hkv,D", [("bf16", 8, 2, 128), ("bf16", 4, 4, 64), ("f32", 4, 2, 128), ("f32", 2, 1, 256)])
def test_attn_large_values(dtype, Hq, Hkv, D):
    # the largest values the documentation allows for 900 positions, scores far apart
    c = ref.make_cache([900, 3, 0, 130], Hkv, D, D, 16, dtype, seed=95)
    c["v"] *= 2.0 ** 86
    run_attn(c, Hq, 1.0)


@pytest.mark.parametrize("Hq,Dk,Dv", [(20, 576, 512), (64, 576, 512), (128, 576, 512), (100, 512, 512), (100, 320, 256)])
@pytest.mark.parametrize("growth", [0.0, 90.0])
def test_attn_latent_replays_bitwise(Hq, Dk, Dv, growth):
    """Eager calls and replays of a captured one, with other calls on the workspace in between: the same bits, also in
    rows that are run again."""
    import torch
    c = ref.make_cache([3000, 0, 17, 900, 2100], 1, Dk, Dv, 16, "bf16", True, seed=96, extra_cols=1 << 10)
    if growth:
        for b, n in enumerate(c["lens"].tolist()):
            for p in range(0, n, 3):
                c["k"][c["table"][b, p // 16], :, p % 16] *= 1.0 + 2.0 * p / 3000
    s, dev, scale = shape_of(c, 5, Hq), cache_of(c), 0.1 if not growth else 3.0
    q, other = queries(c, 5, Hq).cuda(), queries(c, 5, Hq, seed=2).cuda()
    out, lse = torch.empty((5, Hq, Dv), dtype=torch.bfloat16, device="cuda"), torch.empty((5, Hq), device="cuda")
    acc = torch.zeros((5, 1, c["max_pages"] * 16), device="cuda")
    ws = torch.empty(coli_kv_attn_workspace_bytes(s, acc=True), dtype=torch.uint8, device="cuda")

    def step(q=q):
        coli_kv_attn(s, q, dev, out, scale, acc_out=acc, lse=lse, ws=ws)

    step()
    want = [t.clone() for t in (out, lse, acc)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(6):
        step(other)
        out.fill_(3.0)
        if i % 2:
            torch.cuda.synchronize()
            graph.replay()
        else:
            step()
        torch.cuda.synchronize()
        assert torch.equal(bits(out), bits(want[0])) and torch.equal(bits(lse), bits(want[1])) and torch.equal(bits(acc), bits(want[2]))


def test_evict_replays():
    # a captured eviction with work of the program's own between its replays
    import torch
    c = ref.make_cache([500, 40, 0, 300], 2, 64, 64, 16, "bf16", seed=97, spare_pages=32)
    s, dev, k = shape_of(c, 4, 2), cache_of(c), 100
    table = torch.from_numpy(c["free"][:28].reshape(4, 7)).cuda()
    acc = torch.zeros((4, 2, c["max_pages"] * 16), device="cuda")
    new_lens, kept = torch.empty(4, dtype=torch.int32, device="cuda"), torch.empty((4, 2, k), dtype=torch.int32, device="cuda")
    new_acc = torch.empty((4, 2, 112), device="cuda")

    def step():
        coli_kv_evict(s, dev, acc, k, table, new_lens, kept, tail=4, new_acc=new_acc)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    before = dev.k.clone(), dev.v.clone()
    for i in range(4):
        host = np.random.default_rng(i).random(tuple(acc.shape)).astype(np.float32)
        acc.copy_(torch.from_numpy(host))
        dev.lens.copy_(torch.tensor([500 - i, 40 + i, i, 300], dtype=torch.int32))
        dev.k.copy_(before[0])
        dev.v.copy_(before[1])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        now = dict(c, lens=dev.lens.cpu(), k=before[0].cpu(), v=before[1].cpu())
        r = ref.evict(now, host, k, 4, table.cpu().numpy(), new_acc.cpu().numpy())
        assert np.array_equal(kept.cpu().numpy(), r["kept"]) and np.array_equal(new_acc.cpu().numpy(), r["new_acc"])
        assert np.array_equal(new_lens.cpu().numpy(), r["new_lens"])
        same_pool(dev.k, r["k"], "k")
        same_pool(dev.v, r["v"], "v")
