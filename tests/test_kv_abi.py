"""Refusals of the paged cache's entry points on the host, with device
addresses that are never dereferenced: every call fails a check before the
library reaches the device (and the tests run only where there is none).
Then the plain forms themselves, by hand."""
import copy
import ctypes as C

import numpy as np
import pytest
import torch

import kv_reference as ref
import sparse_moe_ffn_coli_amd as pkg
from sparse_moe_ffn_coli_amd import COLI_BF16, COLI_F32, CKvCache, KvCache, KvShape

OK, E_NULL, E_SHAPE, E_DTYPE, E_ALIGN, E_WS, E_DEVICE, E_LAUNCH, E_ALIAS = range(9)
no_gpu = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="fake device addresses must not reach a GPU")


def fake(i, off=0):
    return 0x7F0000000000 + i * (1 << 36) + off


def shape(**kw):
    return KvShape(**(dict(B=4, Hq=32, Hkv=8, Dk=128, Dv=128, page=16, n_pages=1000, max_pages=64, dtype=COLI_BF16) | kw))


def cache(**kw):
    return CKvCache(**(dict(k=fake(1), v=fake(2), table=fake(3), lens=fake(4)) | kw))


def attn(s=None, c=None, q=fake(5), scale=0.1, idx=None, idx_k=0, acc_in=None, acc_out=None, ld=0, out=fake(6), lse=None,
         ws=fake(7), ws_bytes=1 << 40):
    cs, cc = (s or shape()).c(), c or cache()
    return pkg.lib().coli_kv_attn(C.byref(cs), q, C.byref(cc), scale, idx, idx_k, acc_in, acc_out, ld, out, lse, ws, ws_bytes, None)


def append(s=None, c=None, k_new=fake(8), v_new=fake(9), rows=4, start=None):
    cs, cc = (s or shape()).c(), c or cache()
    return pkg.lib().coli_kv_append(C.byref(cs), k_new, v_new, rows, start, C.byref(cc), None)


def evict(s=None, c=None, acc=fake(10), ld=1024, k=100, tail=4, new_table=fake(11), cols=64, new_lens=fake(12),
          kept=fake(13), new_acc=None, new_ld=0):
    cs, cc = (s or shape()).c(), c or cache()
    return pkg.lib().coli_kv_evict(C.byref(cs), C.byref(cc), acc, ld, k, tail, new_table, cols, new_lens, kept, new_acc, new_ld, None)


BAD_SHAPES = [dict(B=-1), dict(Hkv=0), dict(Hq=0), dict(Hq=33), dict(Hq=4), dict(Hq=2048), dict(Dk=0), dict(Dk=100), dict(Dv=12),
              dict(Dk=264), dict(Dv=512), dict(page=0), dict(page=24), dict(page=8192), dict(n_pages=0), dict(max_pages=0),
              dict(n_pages=1 << 25), dict(max_pages=(1 << 20) + 1), dict(B=1 << 20, max_pages=1 << 12)]


@no_gpu
@pytest.mark.parametrize("kw", BAD_SHAPES)
def test_shapes_are_refused_everywhere(kw):
    s = shape(**kw)
    rows = max(s.B, 0)
    assert attn(s) == E_SHAPE and append(s, rows=rows) == E_SHAPE and evict(s) == E_SHAPE


@no_gpu
def test_calls_past_the_launches_are_refused():
    # a launch holds fewer than 2^32 threads
    for kw in (dict(B=1 << 15, Hq=64), dict(B=1 << 20, Hq=8, max_pages=1), dict(B=1 << 12, max_pages=1 << 13)):
        s = shape(**kw)
        assert attn(s) == E_SHAPE and append(s, rows=s.B) == E_SHAPE and evict(s, ld=1 << 17) == E_SHAPE
        assert pkg.coli_kv_attn_workspace_bytes(s) == 0
    assert attn(shape(B=1 << 15, max_pages=1)) == E_DEVICE
    many = shape(B=1 << 15, max_pages=1)
    assert attn(many, idx=fake(20), idx_k=7904) == E_DEVICE and attn(many, idx=fake(20), idx_k=7936 + 32) == E_SHAPE
    assert pkg.coli_kv_attn_workspace_bytes(many, idx_k=7936 + 32) == 0
    assert append(rows=1 << 25, start=fake(20), c=cache()) == E_DEVICE
    assert append(rows=(1 << 25) + 1, start=fake(20)) == E_SHAPE
    assert evict(many, ld=16, k=1984 - 64, cols=128) == E_DEVICE and evict(many, ld=16, k=2048, cols=128) == E_SHAPE
    assert evict(many, ld=16, new_acc=fake(14), new_ld=2048) == E_SHAPE


@no_gpu
def test_other_types_are_refused():
    s = shape(dtype=2)
    assert attn(s) == E_DTYPE and append(s) == E_DTYPE and evict(s) == E_DTYPE
    assert pkg.coli_kv_attn_workspace_bytes(s) == 0


@no_gpu
def test_latent_limits():
    lat = cache(v=None)
    assert attn(shape(Hkv=1, Dk=576, Dv=512), lat) == E_DEVICE
    assert attn(shape(Hkv=1, Dk=576, Dv=512)) == E_SHAPE               # separate values: up to 256
    assert attn(shape(Dk=64, Dv=128), lat) == E_SHAPE                  # values wider than the key they lie in
    assert attn(shape(Dk=584, Dv=512), lat) == E_SHAPE
    assert append(shape(Hkv=1, Dk=576, Dv=512), lat) == E_NULL         # v_new for a cache without v
    assert append(shape(Hkv=1, Dk=576, Dv=512), lat, v_new=None) == E_DEVICE
    assert append(v_new=None) == E_NULL


@no_gpu
def test_attn_refusals():
    assert attn() == E_DEVICE                                          # valid: reaches the device query
    assert attn(q=None) == E_NULL and attn(out=None) == E_NULL and attn(ws=None) == E_NULL
    assert attn(c=cache(k=None)) == E_NULL and attn(c=cache(table=None)) == E_NULL and attn(c=cache(lens=None)) == E_NULL
    assert pkg.lib().coli_kv_attn(None, 1, None, 0.1, None, 0, None, None, 0, None, None, None, 0, None) == E_NULL
    cs = shape().c()
    assert pkg.lib().coli_kv_attn(C.byref(cs), 16, None, 0.1, None, 0, None, None, 0, 16, None, 16, 0, None) == E_NULL
    assert attn(q=fake(5, 8)) == E_ALIGN and attn(c=cache(k=fake(1, 4))) == E_ALIGN and attn(lse=fake(20, 4)) == E_ALIGN
    assert attn(ws_bytes=pkg.coli_kv_attn_workspace_bytes(shape()) - 1) == E_WS
    assert attn(ws_bytes=pkg.coli_kv_attn_workspace_bytes(shape())) == E_DEVICE
    for bad in (float("nan"), float("inf"), 3.4e38):
        assert attn(scale=bad) == E_SHAPE
    # listed positions
    assert attn(idx=fake(20), idx_k=0) == E_SHAPE and attn(idx_k=5) == E_SHAPE and attn(idx=fake(20), idx_k=2048) == E_DEVICE
    # running weights
    w = dict(acc_out=fake(21), ld=1024)
    assert attn(**w) == E_DEVICE and attn(**w, acc_in=fake(21)) == E_DEVICE and attn(**w, acc_in=fake(22)) == E_DEVICE
    assert attn(acc_out=fake(21), ld=1020) == E_SHAPE and attn(acc_out=fake(21), ld=1026) == E_SHAPE
    assert attn(acc_in=fake(21)) == E_NULL
    assert attn(**w, idx=fake(20), idx_k=8) == E_SHAPE
    need = pkg.coli_kv_attn_workspace_bytes(shape(), acc=True)
    assert need > pkg.coli_kv_attn_workspace_bytes(shape()) and attn(**w, ws_bytes=need - 1) == E_WS
    assert pkg.coli_kv_attn_workspace_bytes(shape(), idx_k=8, acc=True) == 0


@no_gpu
def test_attn_aliases():
    assert attn(out=fake(5, 1024)) == E_ALIAS                          # out inside q
    assert attn(out=fake(1, 4096)) == E_ALIAS                          # out inside the keys
    assert attn(lse=fake(6, 256)) == E_ALIAS                           # lse inside out
    assert attn(ws=fake(2, 65536)) == E_ALIAS                          # the workspace over the values
    assert attn(acc_out=fake(21), acc_in=fake(21, 64), ld=1024) == E_ALIAS
    assert attn(acc_out=fake(3), ld=1024) == E_ALIAS                   # over the page table


@no_gpu
def test_append_refusals():
    assert append() == E_DEVICE and append(rows=9, start=fake(20)) == E_DEVICE
    assert append(rows=5) == E_SHAPE and append(rows=-1, start=fake(20)) == E_SHAPE
    assert append(k_new=None) == E_NULL and append(k_new=fake(8, 8)) == E_ALIGN and append(start=fake(20, 4)) == E_ALIGN
    assert append(k_new=fake(1, 256)) == E_ALIAS and append(c=cache(v=fake(1, 4096))) == E_ALIAS


@no_gpu
def test_evict_refusals():
    assert evict() == E_DEVICE and evict(new_acc=fake(14), new_ld=100) == E_DEVICE
    assert evict(k=0) == E_SHAPE and evict(tail=-1) == E_SHAPE and evict(ld=1020) == E_SHAPE and evict(ld=1025) == E_SHAPE
    assert evict(cols=6) == E_SHAPE and evict(cols=7) == E_DEVICE and evict(cols=0) == E_SHAPE
    assert evict(new_acc=fake(14), new_ld=99) == E_SHAPE and evict(k=(1 << 24) + 1, cols=1 << 21) == E_SHAPE
    assert evict(acc=None) == E_NULL and evict(kept=None) == E_NULL and evict(new_lens=None) == E_NULL
    assert evict(new_table=None) == E_NULL and evict(kept=fake(13, 8)) == E_ALIGN
    assert evict(kept=fake(10, 256)) == E_ALIAS and evict(new_acc=fake(10), new_ld=100) == E_ALIAS
    assert evict(new_lens=fake(4)) == E_ALIAS and evict(new_table=fake(1, 64)) == E_ALIAS


@no_gpu
def test_no_sequences():
    s, c = shape(B=0), CKvCache()
    assert attn(s, cache(), q=None, out=None, ws=None, ws_bytes=0) == E_DEVICE
    assert append(s, cache(), k_new=None, v_new=None, rows=0) == E_DEVICE
    assert evict(s, cache(), acc=None, new_table=None, new_lens=None, kept=None) == E_DEVICE


def test_binding_checks_types_sizes_and_devices():
    s = shape(B=2, Hq=4, Hkv=2, Dk=64, Dv=64, n_pages=8, max_pages=3)
    k = torch.zeros((8, 2, 16, 64), dtype=torch.bfloat16)
    good = KvCache(k, k.clone(), torch.zeros((2, 3), dtype=torch.int32), torch.zeros(2, dtype=torch.int32))
    q, out = torch.zeros((2, 4, 64), dtype=torch.bfloat16), torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    bad_caches = [KvCache(k.float(), good.v, good.table, good.lens), KvCache(k[:7], good.v, good.table, good.lens),
                  KvCache(k, good.v, good.table.long(), good.lens), KvCache(k, good.v, good.table[:, :2], good.lens),
                  KvCache(k, good.v, good.table, good.lens[:1]), good]       # the last: on the CPU
    for c in bad_caches:
        with pytest.raises(ValueError):
            pkg.coli_kv_attn(s, q, c, out, 0.1)
        with pytest.raises(ValueError):
            pkg.coli_kv_append(s, torch.zeros((2, 2, 64), dtype=torch.bfloat16), torch.zeros((2, 2, 64), dtype=torch.bfloat16), c)
        with pytest.raises(ValueError):
            pkg.coli_kv_evict(s, c, torch.zeros((2, 2, 48)), 4, torch.zeros((2, 1), dtype=torch.int32),
                              torch.zeros(2, dtype=torch.int32), torch.zeros((2, 2, 4), dtype=torch.int32))


def test_plain_attention_by_hand():
    # two positions, one head: scores ln 1 and ln 3 give weights 1/4 and 3/4
    c = ref.make_cache([2], 1, 8, 8, 2, "f32", seed=1)
    pg = int(c["table"][0, 0])
    c["k"][pg, 0] = 0.0
    c["k"][pg, 0, 1, 0] = float(np.log(3.0))
    c["v"][pg, 0, 0], c["v"][pg, 0, 1] = 4.0, 8.0
    q = torch.zeros((1, 2, 8))
    q[0, 0, 0] = 1.0                                                   # head 1 asks for nothing: equal weights
    r = ref.attn(c, q, 1.0, acc_in=np.zeros((1, 1, 4), np.float32))
    assert np.allclose(r["out"][0, 0], 7.0, atol=1e-6) and np.allclose(r["out"][0, 1], 6.0)
    assert np.allclose(r["lse"][0], [np.log(4.0), np.log(2.0)], atol=1e-6)
    assert np.allclose(r["acc"][0, 0, :2], [0.75, 1.25], atol=1e-6) and np.all(r["acc"][0, 0, 2:] == 0)


def test_plain_eviction_by_hand():
    c = ref.make_cache([6], 1, 8, 8, 2, "f32", seed=2, spare_pages=2)
    acc = np.array([[[5, 1, 5, 5, 0, 2, 9, 9]]], np.float32)
    new_table = c["free"][:2][None]
    r = ref.evict(c, acc, 4, 1, new_table, np.zeros((1, 1, 6), np.float32))
    assert r["kept"].tolist() == [[[0, 2, 3, 5]]] and r["new_lens"].tolist() == [4]      # the newest, then 5 5 5
    assert r["new_acc"].tolist() == [[[5, 5, 5, 2, 0, 0]]]
    assert torch.equal(r["k"][int(new_table[0, 1]), 0, 1], c["k"][int(c["table"][0, 2]), 0, 1])


def test_a_copied_cache_forms_its_own_handles():
    t = torch.zeros(4)
    c = KvCache(t, None, t.clone(), t.clone())
    object.__setattr__(c, "_handles", (None, C.byref(C.c_int()), None))     # as after a call
    for d in (copy.copy(c), copy.deepcopy(c)):
        assert "_handles" not in d.__dict__ and torch.equal(d.k, c.k) and d.v is None
    assert copy.deepcopy(c).k.data_ptr() != c.k.data_ptr() and "_handles" in c.__dict__
