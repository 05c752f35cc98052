"""Refusals of the serving step's entry points on the host, with device addresses that are never dereferenced: every call
fails a check before the library reaches the device (and those tests run only where there is none).  Then the angles of
the rotation, and the plain forms by hand."""
import ctypes as C
import dataclasses
import math

import numpy as np
import pytest
import torch

import serve_reference as ref
import sparse_moe_ffn_coli_amd as pkg
from sparse_moe_ffn_coli_amd import COLI_BF16, COLI_F32, CQkNorm, CRope, KvShape

OK, E_NULL, E_SHAPE, E_DTYPE, E_ALIGN, E_WS, E_DEVICE, E_LAUNCH, E_ALIAS = range(9)
no_gpu = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="fake device addresses must not reach a GPU")


def fake(i, off=0):
    return 0x7F0000000000 + i * (1 << 36) + off


def shape(**kw):
    return KvShape(**(dict(B=4, Hq=32, Hkv=8, Dk=128, Dv=128, page=16, n_pages=1000, max_pages=64, dtype=COLI_BF16) | kw))


def plan(s=None, table=fake(1), lens=fake(2), want=fake(3), shared=fake(4), ring=fake(5), state=fake(6), new_lens=fake(7),
         new_state=fake(8), start=fake(9), rows=100, slot=fake(10), pos=fake(11)):
    cs = (s or shape()).c()
    return pkg.lib().coli_kv_plan(C.byref(cs), table, lens, want, shared, ring, state, new_lens, new_state, start, rows, slot, pos, None)


def rope(s=None, rows=100, q=fake(1), q_ld=4096, k=fake(2), k_ld=1024, v=fake(3), v_ld=1024, norm=(fake(4), fake(5), 128, 1e-6),
         rot=(fake(6), 128, 0, 0, 1.0), pos=fake(7), slot=fake(8), q_out=fake(9), k_out=None, pool_k=fake(11), pool_v=fake(12)):
    cs = (s or shape()).c()
    cn = None if norm is None else C.byref(CQkNorm(*norm))
    cr = None if rot is None else C.byref(CRope(*rot))
    return pkg.lib().coli_kv_rope(C.byref(cs), rows, q, q_ld, k, k_ld, v, v_ld, cn, cr, pos, slot, q_out, k_out, pool_k, pool_v, None)


@no_gpu
def test_plan_refusals():
    assert plan() == E_DEVICE                                           # valid: reaches the device query
    assert plan(shared=None) == E_DEVICE
    assert plan(new_lens=fake(2), new_state=fake(6)) == E_DEVICE        # in place
    for k in ("table", "lens", "want", "ring", "state", "new_lens", "new_state", "start", "slot", "pos"):
        assert plan(**{k: None}) == E_NULL, k
        assert plan(**{k: fake(30, 4)}) == E_ALIGN, k
    assert plan(shared=fake(4, 8)) == E_ALIGN
    assert plan(rows=0, slot=None, pos=None) == E_DEVICE
    assert plan(shape(B=0), table=None, lens=None, want=None, shared=None, new_lens=None) == E_DEVICE
    assert plan(rows=-1) == E_SHAPE and plan(rows=(1 << 25) + 1) == E_SHAPE and plan(rows=1 << 25) == E_DEVICE
    for kw in (dict(B=-1), dict(page=24), dict(page=0), dict(n_pages=0), dict(max_pages=0), dict(max_pages=(1 << 20) + 1)):
        assert plan(shape(**kw)) == E_SHAPE, kw
    assert plan(shape(Hkv=1, Hq=1, page=1, n_pages=(1 << 30) + 1)) == E_SHAPE
    assert plan(shape(dtype=7)) == E_DTYPE
    assert plan(shape(Hkv=1, Dk=576, Dv=512)) == E_DEVICE               # a latent cache's shape
    # outputs over inputs and over each other
    for k in ("want", "shared"):
        for o in ("table", "ring", "new_lens", "new_state", "start", "slot", "pos"):
            assert plan(**{k: fake(20), o: fake(20)}) == E_ALIAS, (k, o)
    assert plan(new_lens=fake(2, 16)) == E_DEVICE                       # (four lengths: the next bytes)
    assert plan(shape(B=5), new_lens=fake(2, 16)) == E_ALIAS
    assert plan(slot=fake(10), pos=fake(10, 384)) == E_ALIAS and plan(slot=fake(10), pos=fake(10, 400)) == E_DEVICE
    assert pkg.lib().coli_kv_plan(None, *[fake(1)] * 9, 0, None, None, None) == E_NULL


@no_gpu
def test_rope_refusals():
    assert rope() == E_DEVICE
    assert rope(norm=None) == E_DEVICE and rope(rot=None) == E_DEVICE and rope(rot=None, pos=None) == E_DEVICE
    assert rope(pos=None) == E_NULL
    assert rope(q=None, q_out=None) == E_DEVICE and rope(q=None) == E_NULL and rope(q_out=None) == E_NULL
    keys = dict(k=None, v=None, slot=None, pool_k=None, pool_v=None)
    assert rope(**keys) == E_DEVICE and rope(**keys, k_out=fake(10)) == E_NULL and rope(**keys, q=None, q_out=None) == E_NULL
    assert rope(k_out=fake(10)) == E_DEVICE
    assert rope(slot=None) == E_NULL and rope(pool_k=None) == E_NULL and rope(pool_v=None) == E_NULL and rope(k=None) == E_NULL
    assert rope(slot=None, v=None, pool_k=None, pool_v=None) == E_NULL              # keys with nowhere to go
    assert rope(slot=None, v=None, pool_k=None, pool_v=None, k_out=fake(10)) == E_DEVICE
    for k in ("q", "k", "v", "pos", "slot", "q_out", "pool_k", "pool_v"):
        assert rope(**{k: fake(30, 8)}) == E_ALIGN, k
    assert rope(norm=(fake(4, 8), None, 128, 1e-6)) == E_ALIGN and rope(rot=(fake(6, 8), 128, 0, 0, 1.0)) == E_ALIGN
    assert rope(rot=(None, 128, 0, 0, 1.0)) == E_NULL
    assert rope(rows=0) == E_DEVICE and rope(rows=-1) == E_SHAPE and rope(rows=(1 << 25) + 1) == E_SHAPE
    for kw in (dict(q_ld=4088), dict(q_ld=4100), dict(k_ld=1016), dict(v_ld=1022), dict(q_ld=1 << 40)):
        assert rope(**kw) == E_SHAPE, kw
    for n in ((fake(4), None, 0, 0.0), (fake(4), None, 136, 0.0), (fake(4), None, 12, 0.0), (fake(4), None, 8, -1.0),
              (fake(4), None, 8, math.nan), (fake(4), None, 8, math.inf)):
        assert rope(norm=n) == E_SHAPE, n
    for r in ((fake(6), 0, 0, 0, 1.0), (fake(6), 136, 0, 0, 1.0), (fake(6), 12, 0, 0, 1.0), (fake(6), 64, 72, 0, 1.0),
              (fake(6), 64, 4, 0, 1.0), (fake(6), 64, -8, 0, 1.0), (fake(6), 64, 2 ** 31 - 8, 0, 1.0), (fake(6), 8, 0, 0, math.nan),
              (fake(6), 8, 0, 0, math.inf)):
        assert rope(rot=r) == E_SHAPE, r
    assert rope(shape(dtype=9)) == E_DTYPE and rope(shape(Dk=100)) == E_SHAPE
    lat = shape(Hkv=1, Dk=576, Dv=512)
    wide = dict(q_ld=32 * 576, k_ld=576)
    assert rope(lat, v=None, pool_v=None, **wide) == E_DEVICE and rope(lat, **wide) == E_SHAPE
    # in place: rows side by side only
    assert rope(q_out=fake(1)) == E_DEVICE and rope(q_out=fake(1), q_ld=4104) == E_ALIAS
    assert rope(k_out=fake(2)) == E_DEVICE and rope(k_out=fake(2), k_ld=1032) == E_ALIAS
    assert rope(q_out=fake(1, 16)) == E_ALIAS and rope(k_out=fake(1)) == E_ALIAS and rope(pool_k=fake(3)) == E_ALIAS
    assert rope(q_out=fake(11)) == E_ALIAS and rope(pool_v=fake(8)) == E_ALIAS and rope(q_out=fake(7)) == E_ALIAS


def attend(s=None, c=None, q=fake(5), scale=0.1, shared=fake(20), start=fake(21), groups=2, out=fake(6), lse=None, ws=fake(7), ws_bytes=1 << 40):
    cs = (s or shape()).c()
    cc = c or pkg.CKvCache(k=fake(1), v=fake(2), table=fake(3), lens=fake(4))
    return pkg.lib().coli_kv_attn_shared(C.byref(cs), q, C.byref(cc), scale, shared, start, groups, out, lse, ws, ws_bytes, None)


@no_gpu
def test_shared_attention_refusals():
    assert attend() == E_DEVICE and attend(lse=fake(22)) == E_DEVICE
    for k in ("q", "shared", "start", "out", "ws"):
        assert attend(**{k: None}) == E_NULL, k
        assert attend(**{k: fake(30, 4)}) == E_ALIGN, k
    assert attend(lse=fake(30, 4)) == E_ALIGN
    assert attend(groups=0) == E_SHAPE and attend(groups=5) == E_SHAPE and attend(groups=-1) == E_SHAPE and attend(groups=4) == E_DEVICE
    assert attend(shape(B=0), groups=0, q=None) == E_DEVICE
    for bad in (math.nan, math.inf, 3.4e38):
        assert attend(scale=bad) == E_SHAPE
    for kw in (dict(Hq=33), dict(Dk=600), dict(page=24), dict(B=1 << 20, max_pages=1 << 12)):
        assert attend(shape(**kw)) == E_SHAPE and pkg.coli_kv_attn_shared_workspace_bytes(shape(**kw), 1) == 0, kw
    assert attend(shape(dtype=5)) == E_DTYPE
    lat = pkg.CKvCache(k=fake(1), v=None, table=fake(3), lens=fake(4))
    assert attend(shape(Hkv=1, Dk=576, Dv=512), lat) == E_DEVICE and attend(shape(Hkv=1, Dk=576, Dv=512)) == E_SHAPE
    need = pkg.coli_kv_attn_shared_workspace_bytes(shape(), 2)
    assert need > 0 and attend(ws_bytes=need - 1) == E_WS and attend(ws_bytes=need) == E_DEVICE
    assert pkg.coli_kv_attn_shared_workspace_bytes(shape(), 0) == 0 == pkg.coli_kv_attn_shared_workspace_bytes(shape(), 5)
    assert pkg.coli_kv_attn_shared_workspace_bytes(shape(B=0), 0) > 0
    for other in (dict(q=fake(6)), dict(shared=fake(6)), dict(start=fake(7)), dict(lse=fake(6)), dict(out=fake(1)), dict(ws=fake(3)), dict(lse=fake(4))):
        assert attend(**other) == E_ALIAS, other


@no_gpu
def test_keys_that_go_to_no_cache():
    # normed and rotated keys of a cache of pairs whose values are the wider ones, which no latent cache has
    pair = dict(s=shape(Dk=64, Dv=128), q_ld=32 * 64, k_ld=8 * 64, rot=(fake(6), 64, 0, 0, 1.0), norm=None)
    out = dict(v=None, slot=None, pool_k=None, pool_v=None, k_out=fake(10))
    assert rope(**pair) == E_DEVICE and rope(**pair, **out) == E_DEVICE and rope(**pair, **(out | dict(q=None, q_out=None))) == E_DEVICE
    assert rope(**pair, v=None, pool_v=None) == E_SHAPE                              # with places: latent rows only


def test_a_shapes_copies_form_their_own_c_form():
    import copy
    import pickle
    s = shape()
    ref = pkg._shape_ref(s)
    assert pkg._shape_ref(s) is ref
    for t in (copy.copy(s), copy.deepcopy(s), pickle.loads(pickle.dumps(s)), dataclasses.replace(s, B=9)):
        assert "_ref" not in t.__dict__ and hash(t) is not None and (t == s or t.B == 9)
        assert pkg._shape_ref(t) is not ref and pkg._shape_ref(t)._obj.B == t.B


def test_the_binding_names_what_is_missing():
    i = torch.zeros(64, dtype=torch.int32)
    for ring, slot in ((None, i), (i, None)):
        with pytest.raises(ValueError, match="ring and slot"):
            pkg.coli_kv_plan(shape(), i.view(1, 64), i, i, ring, i, i, slot, i)


@no_gpu
def test_the_binding_takes_gpu_tensors_only():
    i = torch.zeros(64, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        pkg.coli_kv_plan(shape(), i.view(1, 64), i, i, i, i, i, i, i)
    with pytest.raises(ValueError, match="GPU"):
        pkg.coli_kv_rope(shape(), torch.zeros(1, 32, 128), None, None, None)


def test_freqs():
    f, amp = pkg.coli_rope_freqs(128)
    i = np.arange(64)
    assert amp == 1 and np.allclose(f.numpy(), 10000.0 ** (-2 * i / 128), rtol=1e-14, atol=0)
    g, amp = pkg.coli_rope_freqs(128, scaling="linear", factor=4)
    assert amp == 1 and np.allclose(g.numpy() * 4, f.numpy(), rtol=1e-14, atol=0)
    g, amp = pkg.coli_rope_freqs(128, scaling="ntk", factor=4)
    assert amp == 1 and g[0] == 1 and np.isclose(g[-1], f[-1] / 4, rtol=1e-13)       # the slowest pair is interpolated
    g, amp = pkg.coli_rope_freqs(128, scaling="yarn", factor=16, length=4096)
    turns = 4096 * f.numpy() / (2 * math.pi)
    fast, slow = turns >= 32, turns <= 1
    assert fast.any() and slow.any() and math.isclose(amp, 0.1 * math.log(16) + 1, rel_tol=1e-7)
    assert np.array_equal(g.numpy()[fast], f.numpy()[fast]) and np.allclose(g.numpy()[slow] * 16, f.numpy()[slow], rtol=1e-14)
    mid = ~fast & ~slow
    assert (g.numpy()[mid] < f.numpy()[mid]).all() and (g.numpy()[mid] * 16 > f.numpy()[mid]).all()
    for scaling in pkg.ROPE_SCALINGS:                                                # a factor of one changes nothing
        g, amp = pkg.coli_rope_freqs(40, 500000.0, scaling, 1.0, 8192)
        assert amp == 1 and np.allclose(g.numpy(), 500000.0 ** (-2 * np.arange(20) / 40), rtol=1e-14, atol=0)


def test_freqs_whose_base_passes_the_end():
    # base * factor^(rot / (rot - 2)) past the largest number would leave every angle but the first at 0
    with pytest.raises(pkg.ColiError):
        pkg.coli_rope_freqs(8, 1e300, "ntk", 1e7)
    f, _ = pkg.coli_rope_freqs(8, 1e300, "yarn", 1e7)
    assert f[0] == 1 and np.allclose(f[1:].numpy() * 1e7, 1e300 ** (-np.arange(1, 4) / 4), rtol=1e-13, atol=0)


def test_freqs_refusals():
    for bad in (dict(rot=0), dict(rot=12), dict(rot=584), dict(rot=64, base=1.0), dict(rot=64, base=math.nan), dict(rot=64, base=math.inf),
                dict(rot=64, factor=0.5), dict(rot=64, factor=math.inf), dict(rot=64, length=0), dict(rot=64, length=math.nan)):
        with pytest.raises(pkg.ColiError):
            pkg.coli_rope_freqs(**bad)
    with pytest.raises(ValueError):
        pkg.coli_rope_freqs(64, scaling="cubic")
    d, a = C.c_double(), C.c_float()
    assert pkg.lib().coli_rope_freqs(64, 1e4, 4, 1.0, 1.0, C.byref(d), C.byref(a)) == E_SHAPE
    assert pkg.lib().coli_rope_freqs(64, 1e4, 0, 1.0, 1.0, None, C.byref(a)) == E_NULL


def test_plain_plan_by_hand():
    # pages of 4; sequence 0 goes on into a new page, 1 ends, 2 is new and takes the page that 1 gives back
    table = np.array([[5, -1, -1], [2, 7, -1], [-1, -1, -1]], np.int32)
    r = ref.plan(4, table, np.array([4, 6, 0]), np.array([5, 0, 6]), None, np.array([9, 9, 9, 9, 9, 9, 1, 3], np.int32), 6, 2, 8)
    assert r["ring"].tolist() == [2, 7, 9, 9, 9, 9, 1, 3] and r["lens"].tolist() == [5, 0, 6] and r["start"].tolist() == [0, 1, 1, 7]
    assert r["table"].tolist() == [[5, 1, -1], [2, 7, -1], [3, 2, -1]]
    assert r["slot"].tolist() == [4, 12, 13, 14, 15, 8, 9, -1] and r["pos"].tolist() == [4, 0, 1, 2, 3, 4, 5, -1]
    assert r["state"].tolist() == [1, 1, 7, 0]
    # one page of its own left where the first is another's; the ring serves the first of two
    r = ref.plan(4, np.array([[5, 6], [1, -1], [2, -1]], np.int32), np.array([8, 4, 4]), np.array([0, 5, 5]), np.array([1, 0, 0]),
                 np.zeros(7, np.int32), 0, 0, 9)
    assert r["ring"].tolist() == [6, 0, 0, 0, 0, 0, 0] and r["lens"].tolist() == [0, 5, 4] and r["state"].tolist() == [1, 0, 1, 1]


def test_plain_rope_by_hand():
    x = np.array([[[3.0, 4.0, 1.0, 2.0]]])
    y, tol = ref.norm_rope(x, None, 0, np.array([1]), np.array([math.pi / 2]), 0, False, 1.0, False)
    assert np.allclose(y, [[[-4, 3, 1, 2]]]) and (tol < 1e-5).all()
    y, _ = ref.norm_rope(x, None, 0, np.array([2]), np.array([math.pi / 2, math.pi / 4]), 0, False, 2.0, False)
    assert np.allclose(y, [[[-6, -4, -2, 8]]])
    y, _ = ref.norm_rope(x, None, 0, np.array([2]), np.array([math.pi / 2, math.pi / 4]), 0, True, 1.0, False)
    assert np.allclose(y, [[[-3, -4, -2, 1]]])
    y, _ = ref.norm_rope(x, np.array([1.0, 2.0]), 0, np.array([0]), np.array([1.0]), 2, True, 1.0, False)
    assert np.allclose(y, [[[3 / math.sqrt(12.5), 8 / math.sqrt(12.5), 1, 2]]])
