"""A step's plan (pages from and to the ring, tables, places and positions) through the C ABI against a plain form in
whole numbers: everything has to be equal, also what is not to be written."""
import numpy as np
import pytest

import serve_reference as ref
from sparse_moe_ffn_coli_amd import KvShape, coli_kv_plan

pytestmark = pytest.mark.gpu


def make(rng, lens, page, free, spare=0, max_extra=3, most=None):
    """Sequences with pages in random order and a ring of `free` pages that begins anywhere."""
    lens = np.asarray(lens, np.int64)
    held = -(-lens // page)
    mp = int(max(held.max() if len(lens) else 0, -(-(most or 0) // page), 1)) + max_extra
    n_pages = max(int(held.sum()) + free + spare, 1)
    ids = rng.permutation(n_pages)
    table, at = np.full((len(lens), mp), -7, np.int32), 0
    for b, h in enumerate(held):
        table[b, :h] = ids[at:at + h]
        at += h
    ring, head = np.full(n_pages, -9, np.int32), int(rng.integers(n_pages))
    ring[(head + np.arange(free)) % n_pages] = ids[at:at + free]
    return dict(page=page, table=table, lens=lens.astype(np.int32), ring=ring, head=head, count=free)


def dev(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


def run(c, want, rows, shared=None, in_place=False, stream=None, label=""):
    import torch
    B, mp = c["table"].shape
    shape = KvShape(B=B, Hq=4, Hkv=2, Dk=64, Dv=64, page=c["page"], n_pages=len(c["ring"]), max_pages=mp)
    table, lens, ring = dev(c["table"]), dev(c["lens"]), dev(c["ring"])
    state = dev([c["head"], c["count"], 77, 77])
    guard = torch.full((3 * (B + rows) + 64,), 1234567, dtype=torch.int32, device="cuda")
    cut = lambda at, n: guard[at:at + n]
    up4 = lambda n: (n + 7) // 4 * 4
    start, slot = cut(0, B + 1), cut(up4(B + 1), rows)
    pos = cut(up4(B + 1) + up4(rows), rows)
    new_lens, new_state = (None, None) if in_place else (torch.full((B,), 55, dtype=torch.int32, device="cuda"), dev([5] * 4))
    kw = dict(shared=None if shared is None else dev(shared), new_lens=new_lens, new_state=new_state)
    coli_kv_plan(shape, table, lens, dev(want), ring, state, start, slot, pos, stream=stream, **kw)
    torch.cuda.synchronize()
    r = ref.plan(c["page"], c["table"], c["lens"], np.asarray(want), shared, c["ring"], c["head"], c["count"], rows)
    got = dict(table=table, ring=ring, lens=lens if in_place else new_lens, state=state if in_place else new_state, start=start,
               slot=slot, pos=pos)
    for k, v in got.items():
        assert np.array_equal(v.cpu().numpy(), r[k]), f"{label} {k} differs"
    if not in_place:
        assert np.array_equal(lens.cpu().numpy(), c["lens"]) and state.tolist() == [c["head"], c["count"], 77, 77]
    used = torch.zeros_like(guard, dtype=torch.bool)
    for at, n in ((0, B + 1), (up4(B + 1), rows), (up4(B + 1) + up4(rows), rows)):
        used[at:at + n] = True
    assert bool((guard[~used] == 1234567).all()), f"{label}: written outside the outputs"
    return r


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("page", [1, 2, 16, 4096])
@pytest.mark.parametrize("B", [1, 2, 63, 64, 65, 1000, 1024, 1025, 2500])
def test_steps_of_all_kinds(B, page, in_place):
    rng = np.random.default_rng(B * 7 + page)
    lens = rng.integers(0, 3 * page + 20, size=B)
    lens[rng.random(B) < 0.2] = 0
    want = np.where(rng.random(B) < 0.6, lens + 1, rng.integers(0, 3 * page + 20, size=B))
    want[rng.random(B) < 0.2] = 0
    shared = np.minimum(rng.integers(0, 3, size=B), np.minimum(-(-lens // page), -(-want // page)))
    need = int(np.maximum(-(-want // page) - -(-lens // page), 0).sum())
    rows = int(np.maximum(want - lens, 0).sum()) + int(rng.integers(0, 9))
    c = make(rng, lens, page, need, most=3 * page + 20)
    r = run(c, want, rows, shared if B % 2 else None, in_place)
    assert r["state"][3] == 0


@pytest.mark.parametrize("B,seed", [(1, 0), (40, 1), (40, 2), (1500, 3), (1500, 4), (3000, 5)])
@pytest.mark.parametrize("by", ["pages", "rows", "both"])
def test_first_come_first_served(B, seed, by):
    """The ring, or the step, serves only some; pages that come back in the same call are taken too."""
    rng = np.random.default_rng(seed)
    page = 8
    lens = rng.integers(0, 60, size=B)
    want = np.where(rng.random(B) < 0.3, 0, lens + rng.integers(0, 40, size=B))
    need = int(np.maximum(-(-want // page) - -(-lens // page), 0).sum())
    gone = int((-(-lens // page))[want == 0].sum())
    new = int(np.maximum(want - lens, 0).sum())
    free = max(need // 2 - gone, 0) if by != "rows" else need
    rows = new // 2 if by != "pages" else new + 3
    r = run(make(rng, lens, page, free, most=100), want, rows)
    if B > 1:
        assert r["state"][3] > 0


def test_large_steps():
    """Rows by the second launch: prompts of many sequences, one of very many pages."""
    rng = np.random.default_rng(9)
    for lens, want, page in (([0] * 300, rng.integers(0, 700, size=300), 16), ([5, 0, 70], [5, 40001, 71], 1),
                             (rng.integers(0, 50, size=5000), rng.integers(0, 50, size=5000), 4)):
        lens, want = np.asarray(lens), np.asarray(want)
        need = int(np.maximum(-(-want // page) - -(-lens // page), 0).sum())
        new = int(np.maximum(want - lens, 0).sum())
        for rows in (new, new + 5, max(4097, new // 2)):
            run(make(rng, lens, page, need, most=int(want.max())), want, rows, label=f"{len(lens)} sequences, {rows} rows")


def test_nothing_to_do_and_no_rows():
    rng = np.random.default_rng(10)
    run(make(rng, [5, 0, 16], 16, 0), [5, 0, 16], 0)
    run(make(rng, [5, 0, 16], 16, 3), [6, 1, 17], 0)        # no row: all refused
    run(make(rng, [16, 32], 16, 0), [0, 0], 4)              # everything comes back
    run(make(rng, [0, 0], 16, 0, spare=4), [1, 1], 4)       # an empty ring


def test_no_sequences():
    import torch
    shape = KvShape(B=0, Hq=4, Hkv=2, Dk=64, Dv=64, page=16, n_pages=8, max_pages=4)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    state, start = dev([3, 2, 9, 9]), dev([5])
    slot, pos = dev([7] * 5), dev([7] * 5)
    coli_kv_plan(shape, none.view(0, 4), none, none, dev([0] * 8), state, start, slot, pos)
    assert state.tolist() == [3, 2, 0, 0] and start.tolist() == [0] and slot.tolist() == [-1] * 5 == pos.tolist()


def test_lengths_outside_the_table_are_clamped():
    rng = np.random.default_rng(11)
    c = make(rng, [32, 10], 8, 8, max_extra=0)
    c["lens"] = np.array([1 << 30, 10], np.int32)           # four pages: 32
    run(c, [-5, 1 << 30], 40)


def test_page_ids_outside_the_pool():
    rng = np.random.default_rng(12)
    c = make(rng, [20, 3], 8, 4)
    c["table"][0, 2] = len(c["ring"])                       # the page that the next token falls into
    c["ring"][(c["head"] + 1) % len(c["ring"])] = -3
    r = run(c, [26, 20], 40)
    assert (r["slot"][:4] == -1).all() and (r["pos"][:4] == np.arange(20, 24)).all()


def test_a_state_that_is_none_stays_inside():
    """Heads and counts outside the ring, more pages coming back than it holds: nothing outside is touched."""
    import torch
    for head, count in ((-5, 3), (1 << 30, 3), (2, -4), (2, 1 << 30), (2, 6)):
        buf = torch.full((24,), 99, dtype=torch.int32, device="cuda")
        ring = buf[8:14]
        shape = KvShape(B=2, Hq=4, Hkv=2, Dk=64, Dv=64, page=4, n_pages=6, max_pages=5)
        table = dev(np.arange(10).reshape(2, 5) % 6)
        start, slot, pos = dev([0] * 3), dev([0] * 8), dev([0] * 8)
        coli_kv_plan(shape, table, dev([20, 3]), dev([0, 9]), ring, dev([head, count, 0, 0]), start, slot, pos,
                     new_lens=dev([0, 0]), new_state=dev([0] * 4))
        torch.cuda.synchronize()
        assert bool((buf[:8] == 99).all()) and bool((buf[14:] == 99).all())


def test_many_steps_keep_every_page():
    """A batch over 60 steps in place: tables and ring hold every page once, and lengths follow the wishes."""
    import torch
    rng = np.random.default_rng(13)
    B, page, mp, n_pages = 70, 4, 32, 900
    shape = KvShape(B=B, Hq=4, Hkv=2, Dk=64, Dv=64, page=page, n_pages=n_pages, max_pages=mp)
    table, lens = dev(np.full((B, mp), -1)), dev(np.zeros(B))
    ring, state = dev(rng.permutation(n_pages)), dev([0, n_pages, 0, 0])
    rows = 300
    start, slot, pos = dev(np.zeros(B + 1)), dev(np.zeros(rows)), dev(np.zeros(rows))
    host = dict(table=table.cpu().numpy(), lens=lens.cpu().numpy(), ring=ring.cpu().numpy(), head=0, count=n_pages)
    side = torch.cuda.Stream()
    for step in range(60):
        n = host["lens"].astype(np.int64)
        kind = rng.random(B)
        want = np.where(kind < 0.7, n + 1, np.where(kind < 0.8, 0, np.where(kind < 0.9, np.maximum(n - 3, 0), n + rng.integers(0, 30))))
        want = np.minimum(want, mp * page)
        r = ref.plan(page, host["table"], host["lens"], want, None, host["ring"], host["head"], host["count"], rows)
        w = dev(want)
        torch.cuda.synchronize()
        coli_kv_plan(shape, table, lens, w, ring, state, start, slot, pos, stream=side if step % 2 else None)
        torch.cuda.synchronize()
        for k, v in dict(table=table, lens=lens, ring=ring, state=state, start=start, slot=slot, pos=pos).items():
            assert np.array_equal(v.cpu().numpy(), r[k]), f"step {step}: {k}"
        host = dict(table=r["table"].astype(np.int32), lens=r["lens"].astype(np.int32), ring=r["ring"].astype(np.int32),
                    head=int(r["state"][0]), count=int(r["state"][1]))
        own = [p for b in range(B) for p in host["table"][b, :-(-host["lens"][b] // page)]]
        left = list(host["ring"][(host["head"] + np.arange(host["count"])) % n_pages])
        assert sorted(own + left) == list(range(n_pages))


def test_replayed_from_a_graph():
    import torch
    rng = np.random.default_rng(14)
    for B, rows in ((50, 200), (50, 9000)):
        lens = rng.integers(0, 50, size=B)
        c = make(rng, lens, 4, 500, most=300)
        table, mp = dev(c["table"]), c["table"].shape[1]
        shape = KvShape(B=B, Hq=4, Hkv=2, Dk=64, Dv=64, page=4, n_pages=len(c["ring"]), max_pages=mp)
        d = {k: dev(c[k]) for k in ("lens", "ring")}
        state, want = dev([c["head"], c["count"], 0, 0]), dev(lens)
        start, slot, pos = dev(np.zeros(B + 1)), dev(np.zeros(rows)), dev(np.zeros(rows))
        call = lambda: coli_kv_plan(shape, table, d["lens"], want, d["ring"], state, start, slot, pos)
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        host = dict(table=c["table"], lens=c["lens"], ring=c["ring"], head=c["head"], count=c["count"])
        for step in range(4):
            w = np.minimum(host["lens"] + rng.integers(0, 5, size=B), mp * 4)
            want.copy_(dev(w))
            r = ref.plan(4, host["table"], host["lens"], w, None, host["ring"], host["head"], host["count"], rows)
            g.replay()
            torch.cuda.synchronize()
            for k, v in dict(table=table, lens=d["lens"], ring=d["ring"], state=state, start=start, slot=slot, pos=pos).items():
                assert np.array_equal(v.cpu().numpy(), r[k]), f"replay {step}: {k}"
            host = dict(table=r["table"].astype(np.int32), lens=r["lens"].astype(np.int32), ring=r["ring"].astype(np.int32),
                        head=int(r["state"][0]), count=int(r["state"][1]))
