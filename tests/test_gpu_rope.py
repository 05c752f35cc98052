"""Norm and rotation of queries and keys on their way to the attention, through the C ABI, against plain forms in 64 bits
(tests/serve_reference.py, which derives the bounds)."""
import numpy as np
import pytest

import serve_reference as ref
from sparse_moe_ffn_coli_amd import COLI_BF16, COLI_F32, ColiError, KvShape, QkNorm, Rope, coli_kv_rope, coli_rope_freqs

pytestmark = pytest.mark.gpu


def dev(x, dt=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dt is None else t.to(dt)


def run(rows, Hq, Hkv, Dk, Dv, dtype="bf16", latent=False, rot=0, rot_at=0, interleaved=False, width=0, norms="qk", page=16,
        far=5000, scaling="plain", fused=True, in_place=False, to=("pool",), holes=True, seed=0, scale=1.0, stream=None, pos=None):
    import torch
    rng = np.random.default_rng(seed)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *s: (torch.randn(s, generator=g, device="cuda") * scale).to(dt)
    n_pages = -(-rows // page) + 2
    shape = KvShape(B=0, Hq=Hq, Hkv=Hkv, Dk=Dk, Dv=Dv, page=page, n_pages=n_pages, max_pages=1,
                    dtype=COLI_F32 if dtype == "f32" else COLI_BF16)
    if fused:
        pad = 8 * int(rng.integers(0, 3))                      # rows wider than what is used of them
        w = (Hq + Hkv) * Dk + (0 if latent else Hkv * Dv) + pad
        x = randn(rows, w)
        q, k = x[:, :Hq * Dk].unflatten(1, (Hq, Dk)), x[:, Hq * Dk:(Hq + Hkv) * Dk].unflatten(1, (Hkv, Dk))
        v = None if latent else x[:, (Hq + Hkv) * Dk:(Hq + Hkv) * Dk + Hkv * Dv].unflatten(1, (Hkv, Dv))
    else:
        q, k, v = randn(rows, Hq, Dk), randn(rows, Hkv, Dk), None if latent else randn(rows, Hkv, Dv)
    if pos is None:
        pos = rng.integers(0, far, size=rows)
        pos[0] = far - 1
    slot = rng.permutation(n_pages * page)[:rows]
    if holes and rows > 5:
        pos[2], slot[3], slot[4] = -1, -1, n_pages * page
        pos[rows - 1], slot[rows - 1] = -5, -1
    freq, amp = coli_rope_freqs(rot, scaling=scaling, factor=8.0, length=4096) if rot else (None, 1.0)
    wq = (1 + 0.2 * randn(width).float() / scale).to(dt) if width and "q" in norms else None
    wk = (1 + 0.2 * randn(width).float() / scale).to(dt) if width and "k" in norms else None
    qn, kn, vn = ref.to_np(q), ref.to_np(k), None if v is None else ref.to_np(v)
    k_out = None
    if in_place:
        q_out = q
        k_out = k if "out" in to else None
    else:
        q_out = torch.full((rows, Hq, Dk), 7.0, dtype=dt, device="cuda")
        k_out = torch.full((rows, Hkv, Dk), 7.0, dtype=dt, device="cuda") if "out" in to else None
    kw = {}
    if "pool" in to:
        kw = dict(pool_k=torch.full((n_pages, Hkv, page, Dk), 7.0, dtype=dt, device="cuda"), slot=dev(slot.astype(np.int32)),
                  pool_v=None if latent else torch.full((n_pages, Hkv, page, Dv), 7.0, dtype=dt, device="cuda"))
    coli_kv_rope(shape, q, k, v if "pool" in to else None, q_out, pos=dev(pos.astype(np.int32)), stream=stream,
                 rope=Rope(freq.cuda(), rot_at, interleaved, amp) if rot else None,
                 norm=QkNorm(wq, wk, 1e-6) if width else None, k_out=k_out, **kw)
    torch.cuda.synchronize()
    f = freq.numpy() if rot else None
    bf = dtype == "bf16"
    live = pos >= 0
    rq, tq = ref.norm_rope(qn, None if wq is None else ref.to_np(wq), 1e-6, pos, f, rot_at, interleaved, amp, bf)
    rk, tk = ref.norm_rope(kn, None if wk is None else ref.to_np(wk), 1e-6, pos, f, rot_at, interleaved, amp, bf)

    def close(got, want, tol, label):
        got = ref.to_np(got)
        assert np.all(np.isfinite(got)), label
        over = np.abs(got - want) - tol
        assert over.max() <= 0, f"{label}: {over.max():.3e} over the bound, worst error {np.abs(got - want).max():.3e}"

    close(q_out[dev(live)], rq[live], tq[live], "q")
    if not in_place:
        assert bool((q_out[dev(~live)] == 7).all()), "a row without a position was written"
        if k_out is not None:
            assert bool((k_out[dev(~live)] == 7).all())
    if k_out is not None:
        close(k_out[dev(live)], rk[live], tk[live], "k_out")
    if "pool" in to:
        ok = live & (slot >= 0) & (slot < n_pages * page)
        at = dev(slot[ok])
        pk = kw["pool_k"]
        close(pk[at // page, :, at % page], rk[ok], tk[ok], "pool_k")
        rest = torch.ones((n_pages, page), dtype=torch.bool, device="cuda")
        rest[at // page, at % page] = False
        assert bool((pk.transpose(1, 2)[rest] == 7).all()), "another place of the pool was written"
        if v is not None:
            assert np.array_equal(ref.to_np(kw["pool_v"][at // page, :, at % page]), vn[ok]), "values differ"
            assert bool((kw["pool_v"].transpose(1, 2)[rest] == 7).all())
    return q_out


LAYOUTS = [
    # Hq, Hkv, Dk, Dv, latent, rot, rot_at, width
    (32, 8, 128, 128, False, 128, 0, 128),
    (4, 2, 64, 64, False, 64, 0, 64),
    (3, 3, 8, 8, False, 8, 0, 8),
    (2, 1, 16, 40, False, 8, 8, 16),
    (12, 12, 80, 80, False, 32, 0, 80),
    (5, 1, 96, 40, False, 24, 40, 96),        # half of 24 is an odd number of fours
    (4, 2, 72, 136, False, 72, 0, 72),        # values wider than keys
    (7, 1, 192, 128, False, 64, 128, 192),
    (6, 2, 256, 200, False, 40, 8, 104),      # a norm of a part
    (16, 4, 256, 256, False, 256, 0, 0),
    (9, 3, 88, 24, False, 0, 0, 88),          # norm alone
    (64, 1, 576, 512, True, 64, 512, 512),
    (3, 1, 576, 512, True, 576, 0, 576),
    (2, 1, 520, 512, True, 520, 0, 512),      # lanes that hold a half of theirs
    (2, 1, 552, 512, True, 536, 8, 536),
    (2, 1, 568, 512, True, 40, 528, 8),
    (100, 1, 320, 256, True, 64, 256, 256),
]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv,Dk,Dv,latent,rot,rot_at,width", LAYOUTS)
def test_layouts(Hq, Hkv, Dk, Dv, latent, rot, rot_at, width, dtype, interleaved):
    run(37, Hq, Hkv, Dk, Dv, dtype, latent, rot, rot_at, interleaved, width, seed=Dk + Hq)


@pytest.mark.parametrize("rows", [1, 2, 5, 64, 511, 1025, 4100])
@pytest.mark.parametrize("Hq,Hkv,Dk,rot,width", [(1, 1, 64, 64, 64), (32, 8, 128, 128, 128), (2, 1, 32, 16, 0)])
def test_rows(rows, Hq, Hkv, Dk, rot, width):
    # narrow tokens share a workgroup, few wide ones are spread
    run(rows, Hq, Hkv, Dk, Dk, "bf16", rot=rot, width=width, seed=rows)
    run(rows, Hq, Hkv, Dk, Dk, "f32", rot=rot, width=width, interleaved=True, seed=rows)


@pytest.mark.parametrize("scaling", ["plain", "linear", "ntk", "yarn"])
@pytest.mark.parametrize("far", [1, 4096, 1 << 20, 1 << 24, (1 << 31) - 1])
def test_far_positions(scaling, far):
    run(60, 2, 1, 128, 128, "f32", rot=128, far=far, scaling=scaling, seed=3)
    run(60, 2, 1, 128, 128, "f32", rot=128, far=far, scaling=scaling, interleaved=True, seed=4)


@pytest.mark.parametrize("norms", ["q", "k", "qk"])
@pytest.mark.parametrize("to", [("pool",), ("out",), ("pool", "out")])
def test_targets_and_norms(norms, to):
    run(70, 8, 2, 128, 128, rot=64, width=128, norms=norms, to=to, seed=5)
    run(70, 8, 2, 128, 128, rot=64, width=128, norms=norms, to=to, fused=False, seed=6)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("Dk,latent", [(128, False), (72, False), (576, True), (552, True)])
def test_in_place(dtype, interleaved, Dk, latent):
    run(90, 6, 1 if latent else 2, Dk, 512 if latent else Dk, dtype, latent, rot=Dk // 16 * 16 if Dk != 552 else 536,
        interleaved=interleaved, width=Dk // 8 * 8, to=("pool", "out"), in_place=True, fused=False, seed=7)


def test_large_and_small_values():
    run(40, 4, 2, 128, 128, "f32", rot=128, width=128, scale=1e15, seed=8)
    run(40, 4, 2, 128, 128, "bf16", rot=128, width=128, scale=1e15, seed=8)
    run(40, 4, 2, 64, 64, "f32", rot=64, width=64, scale=1e-5, seed=9)


def test_zero_rows_of_a_norm():
    """A head of zeros stays zeros: eps keeps the root from zero."""
    import torch
    shape = KvShape(B=0, Hq=2, Hkv=1, Dk=64, Dv=64, page=16, n_pages=1, max_pages=1)
    q = torch.zeros((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    out = torch.ones_like(q)
    coli_kv_rope(shape, q, None, None, out, norm=QkNorm(q_w=torch.ones(64, dtype=torch.bfloat16, device="cuda")))
    assert bool((out == 0).all())


def test_other_heads_do_not_leak():
    """NaN and infinities in one token's head, in rows left out and in the gap behind the heads stay where they are."""
    import torch
    shape = KvShape(B=0, Hq=4, Hkv=2, Dk=40, Dv=40, page=16, n_pages=1, max_pages=1, dtype=COLI_F32)
    x = torch.randn(6, 8 * 40 + 8, device="cuda")
    q, k, v = x[:, :160].unflatten(1, (4, 40)), x[:, 160:240].unflatten(1, (2, 40)), x[:, 240:320].unflatten(1, (2, 40))
    freq, _ = coli_rope_freqs(40)
    call = lambda out, pk, pv: coli_kv_rope(shape, q, k, v, out, pos=dev(np.array([0, 5, -1, 9, 10, 11], np.int32)),
                                            rope=Rope(freq.cuda()), norm=QkNorm(torch.ones(40, device="cuda"), torch.ones(40, device="cuda")),
                                            pool_k=pk, pool_v=pv, slot=dev(np.arange(6, dtype=np.int32)))
    new = lambda: (torch.zeros(6, 4, 40, device="cuda"), torch.zeros(1, 2, 16, 40, device="cuda"), torch.zeros(1, 2, 16, 40, device="cuda"))
    a, b = new(), new()
    call(*a)
    x[1, 40:80] = float("nan")
    x[2] = float("inf")
    x[:, 320:] = float("nan")
    call(*b)
    assert bool(b[0][1, 1].isnan().all())
    b[0][1, 1] = a[0][1, 1]
    assert all(torch.equal(s, t) for s, t in zip(a, b))


def test_one_row_of_any_stride():
    # a single row says nothing about where the next one would be
    import torch
    shape = KvShape(B=0, Hq=2, Hkv=2, Dk=64, Dv=64, page=16, n_pages=1, max_pages=1, dtype=COLI_F32)
    x = torch.randn(2 * 64 + 4, device="cuda").as_strided((1, 2, 64), (132, 64, 1))
    out, want = torch.empty(1, 2, 64, device="cuda"), torch.empty(1, 2, 64, device="cuda")
    freq, pos = coli_rope_freqs(64)[0].cuda(), dev(np.array([77], np.int32))
    assert x.stride(0) % 8 == 4
    coli_kv_rope(shape, x, None, None, out, pos=pos, rope=Rope(freq))
    coli_kv_rope(shape, x.contiguous().view(1, 2, 64), None, None, want, pos=pos, rope=Rope(freq))
    assert torch.equal(out, want)
    two = torch.randn(2, 2 * 64 + 4, device="cuda")[:, :128].unflatten(1, (2, 64))
    with pytest.raises(ColiError):
        coli_kv_rope(shape, two, None, None, torch.empty(2, 2, 64, device="cuda"), pos=pos.repeat(2), rope=Rope(freq))


def test_queries_alone_and_keys_alone():
    import torch
    shape = KvShape(B=0, Hq=4, Hkv=2, Dk=64, Dv=64, page=16, n_pages=1, max_pages=1, dtype=COLI_F32)
    freq, _ = coli_rope_freqs(64)
    q, k = torch.randn(5, 4, 64, device="cuda"), torch.randn(5, 2, 64, device="cuda")
    pos = dev(np.arange(5, dtype=np.int32))
    both, ko = torch.empty_like(q), torch.empty_like(k)
    coli_kv_rope(shape, q, k, None, both, pos=pos, rope=Rope(freq.cuda()), k_out=ko)
    q1, k1 = torch.empty_like(q), torch.empty_like(k)
    coli_kv_rope(shape, q, None, None, q1, pos=pos, rope=Rope(freq.cuda()))
    coli_kv_rope(shape, None, k, None, None, pos=pos, rope=Rope(freq.cuda()), k_out=k1)
    assert torch.equal(both, q1) and torch.equal(ko, k1)
    # position 0 turns nothing, and a turn back by the negative angle gives the value again
    assert torch.equal(both[0], q[0])
    back = torch.empty_like(q)
    coli_kv_rope(shape, both, None, None, back, pos=pos, rope=Rope(-freq.cuda()))
    assert (back - q).abs().max() <= 40 * 2.0 ** -24 * 2 * q.abs().max()


def test_copies_are_exact_without_norm_and_rotation():
    import torch
    run(33, 4, 2, 64, 64, "bf16", seed=11)
    shape = KvShape(B=0, Hq=2, Hkv=1, Dk=64, Dv=64, page=16, n_pages=1, max_pages=1)
    q = torch.randint(-32768, 32767, (4, 2, 64), dtype=torch.int16, device="cuda").view(torch.bfloat16)
    out = torch.zeros_like(q)
    coli_kv_rope(shape, q, None, None, out)
    assert torch.equal(out.view(torch.int16), q.view(torch.int16))


def test_pools_past_32_bits():
    import torch
    page, D, Hkv, n_pages = 4096, 256, 4, 1100                  # 4.6e9 elements a pool
    shape = KvShape(B=0, Hq=4, Hkv=Hkv, Dk=D, Dv=D, page=page, n_pages=n_pages, max_pages=1)
    pk = torch.zeros((n_pages, Hkv, page, D), dtype=torch.bfloat16, device="cuda")
    pv = torch.zeros_like(pk)
    k, v = torch.randn(2, Hkv, D, device="cuda").bfloat16(), torch.randn(2, Hkv, D, device="cuda").bfloat16()
    slot = dev(np.array([n_pages * page - 1, 5], np.int32))
    coli_kv_rope(shape, None, k, v, None, pool_k=pk, pool_v=pv, slot=slot)
    assert torch.equal(pk[-1, :, -1], k[0]) and torch.equal(pk[0, :, 5], k[1])
    assert torch.equal(pv[-1, :, -1], v[0]) and torch.equal(pv[0, :, 5], v[1])
    assert int((pk[-1].abs().sum(-1) != 0).sum()) == Hkv


def test_streams_graphs_and_repeats():
    import torch
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = run(50, 8, 2, 128, 128, rot=128, width=128, seed=12)
    b = run(50, 8, 2, 128, 128, rot=128, width=128, seed=12, stream=side)
    assert torch.equal(a[:-1][dev(np.arange(49) != 2)], b[:-1][dev(np.arange(49) != 2)])
    shape = KvShape(B=0, Hq=4, Hkv=2, Dk=64, Dv=64, page=16, n_pages=1, max_pages=1)
    freq, _ = coli_rope_freqs(64)
    rope = Rope(freq.cuda())
    q, pos = torch.randn(7, 4, 64, device="cuda").bfloat16(), dev(np.arange(7, dtype=np.int32))
    out = torch.empty_like(q)
    coli_kv_rope(shape, q, None, None, out, pos=pos, rope=rope)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        coli_kv_rope(shape, q, None, None, out, pos=pos, rope=rope)
    for i in range(4):
        pos += 1000 * i
        q.copy_(torch.randn(7, 4, 64, device="cuda"))
        out.zero_()
        g.replay()
        want = torch.empty_like(q)
        coli_kv_rope(shape, q, None, None, want, pos=pos, rope=rope)
        assert torch.equal(out, want), f"replay {i}"


def test_refusals_of_the_binding():
    import torch
    shape = KvShape(B=0, Hq=4, Hkv=2, Dk=64, Dv=64, page=16, n_pages=1, max_pages=1)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16, device="cuda")
    out, pos = torch.zeros_like(q), dev(np.arange(3, dtype=np.int32))
    freq = coli_rope_freqs(64)[0].cuda()
    for bad in (q.float(), q[:, :3], q.transpose(0, 1), q[..., :32], q.cpu()):
        with pytest.raises(ValueError):
            coli_kv_rope(shape, bad, None, None, out)
    wide = torch.zeros(3, 4, 128, dtype=torch.bfloat16, device="cuda")[..., :64]        # heads apart
    with pytest.raises(ValueError):
        coli_kv_rope(shape, wide, None, None, out)
    with pytest.raises(ValueError):
        coli_kv_rope(shape, None, None, None, None)
    with pytest.raises(ValueError):
        coli_kv_rope(shape, q, None, None, out, pos=pos.long(), rope=Rope(freq))
    with pytest.raises(ValueError):
        coli_kv_rope(shape, q, None, None, out, pos=pos, rope=Rope(freq.float()))
    with pytest.raises(ColiError):
        coli_kv_rope(shape, q, None, None, out, rope=Rope(freq))                        # no positions
    with pytest.raises(ColiError):
        coli_kv_rope(shape, q, None, None, out, pos=pos, rope=Rope(freq, rot_at=8))     # past the head
    with pytest.raises(ColiError):
        coli_kv_rope(shape, q, None, None, out, pos=pos, rope=Rope(torch.empty(0, dtype=torch.float64, device="cuda")))
    with pytest.raises(ColiError):
        coli_kv_rope(shape, q, None, None, out, k_out=out[:, :2].contiguous())          # an output without keys
