"""Pages that sequences borrow, over a step's plan: they stay out of the ring until the last one that reads them gives them
back, and a sequence that was cut below them, or has ended, gets no place inside them."""
import numpy as np
import pytest

import serve_reference as ref
from sparse_moe_ffn_coli_amd import KvShape, coli_kv_plan
from test_gpu_plan import dev, make

pytestmark = pytest.mark.gpu


def plain(page, table, lens, want, shared, ring, head, count, rows):
    """ref.plan, where a sequence that holds fewer pages than it shares does not grow and keeps nobody waiting."""
    lens, want = np.asarray(lens), np.asarray(want)
    below = (want > lens) & (-(-lens // page) < shared)
    r = ref.plan(page, table, lens, np.where(below, lens, want), shared, ring, head, count, rows)
    r["state"][3] += below.sum()
    return r


class Batch:
    """A batch in place, on the GPU and in whole numbers."""

    def __init__(self, B, page, mp, n_pages, rows, seed):
        rng = np.random.default_rng(seed)
        self.page, self.rows, self.n_pages = page, rows, n_pages
        self.shape = KvShape(B=B, Hq=4, Hkv=2, Dk=64, Dv=64, page=page, n_pages=n_pages, max_pages=mp)
        self.host = dict(table=np.full((B, mp), -1, np.int32), lens=np.zeros(B, np.int32), ring=rng.permutation(n_pages).astype(np.int32))
        self.head, self.count = 0, n_pages
        self.shared = np.zeros(B, np.int32)
        self.d = {k: dev(v) for k, v in self.host.items()}
        self.state = dev([0, n_pages, 0, 0])
        self.start, self.slot, self.pos = dev(np.zeros(B + 1)), dev(np.zeros(rows)), dev(np.zeros(rows))

    def step(self, want):
        import torch
        h = self.host
        r = plain(self.page, h["table"], h["lens"], want, self.shared, h["ring"], self.head, self.count, self.rows)
        coli_kv_plan(self.shape, self.d["table"], self.d["lens"], dev(want), self.d["ring"], self.state, self.start, self.slot, self.pos,
                     shared=dev(self.shared))
        torch.cuda.synchronize()
        got = dict(self.d, state=self.state, start=self.start, slot=self.slot, pos=self.pos)
        for k, v in got.items():
            assert np.array_equal(v.cpu().numpy(), r[k]), f"{k} differs"
        self.host = {k: r[k].astype(np.int32) for k in ("table", "lens", "ring")}
        self.head, self.count = int(r["state"][0]), int(r["state"][1])
        return r

    def lend(self, to, of, pages):
        """The first pages of sequence `of`, full ones, begin sequences `to` as well."""
        for b in to:
            self.host["table"][b, :pages] = self.host["table"][of, :pages]
            self.host["lens"][b] = pages * self.page
        self.shared[[of, *to]] = pages
        for k in ("table", "lens"):
            self.d[k].copy_(dev(self.host[k]))

    def free(self):
        return self.host["ring"][(self.head + np.arange(self.count)) % self.n_pages].tolist()


@pytest.mark.parametrize("rows", [200, 6000])              # in one launch, and in two
def test_a_prompt_is_given_back_by_the_last_that_reads_it(rows):
    t = Batch(B=5, page=8, mp=40, n_pages=90, rows=rows, seed=1)
    t.step([5 * 8 + 3, 0, 0, 0, 20])
    t.lend((1, 2), 0, 5)
    t.step([60, 41, 55, 0, 21])
    prompt = t.host["table"][0, :5].tolist()
    t.step([0, 42, 56, 0, 22])                             # the one that brought it ends: only its own pages go back
    assert not set(prompt) & set(t.free())
    r = t.step([0, 43, 0, 0, 23])                          # the next one
    assert r["state"][3] == 0 and not set(prompt) & set(t.free())
    assert t.host["table"][1, :5].tolist() == prompt
    t.shared[:] = 0                                        # the last one: they are its own now
    t.step([0, 0, 0, 0, 24])
    assert set(prompt) <= set(t.free())
    t.step([0, 0, 0, 0, 0])
    assert sorted(t.free()) == list(range(90))


@pytest.mark.parametrize("rows", [200, 6000])
def test_no_growth_below_the_shared_pages(rows):
    t = Batch(B=6, page=4, mp=40, n_pages=120, rows=rows, seed=2)
    t.step([4 * 4, 0, 0, 7, 0, 0])
    t.lend((1, 2, 4), 0, 4)
    t.step([17, 20, 18, 8, 30, 0])
    prompt = t.host["table"][0, :4].tolist()
    t.step([0, 9, 12, 9, 13, 0])                           # one ends, three are cut below the pages (one inside the last)
    assert not set(prompt) & set(t.free())
    free = t.free()
    r = t.step([30, 11, 13, 10, 13, 50])                   # no place for the first three, and the others are served
    assert r["state"].tolist()[2:] == [51, 3] and r["lens"].tolist() == [0, 9, 12, 10, 13, 50] and r["start"].tolist() == [0, 0, 0, 0, 1, 1, 51]
    assert t.host["table"][:3, :4].tolist() == [prompt] * 3
    assert not set(r["slot"][r["slot"] >= 0] // 4) & set(prompt) and len(free) == len(t.free()) + 13
    t.shared[0] = 0                                        # the ended one's place is another's: pages from the ring
    r = t.step([30, 9, 12, 10, 13, 50])
    assert not set(t.host["table"][0, :8]) & set(prompt)
    assert r["state"][3] == 0 and r["lens"][0] == 30


def test_refused_between_others():
    """Many sequences, some cut below what they share; the ring or the step's rows serve all, or only the first."""
    rng = np.random.default_rng(3)
    for B, page, tight in ((40, 8, False), (40, 8, True), (1500, 4, False), (1500, 4, True), (3000, 16, True)):
        lens = rng.integers(0, 60, size=B)
        held = -(-lens // page)
        want = np.where(rng.random(B) < 0.3, rng.integers(0, 60, size=B), lens + rng.integers(0, 30, size=B))
        shared = np.where(rng.random(B) < 0.3, held + rng.integers(1, 3, size=B), np.minimum(rng.integers(0, 3, size=B), held)).astype(np.int32)
        grows = (want > lens) & (held >= shared)
        need = int((-(-want // page) - held)[grows].sum())
        c = make(rng, lens, page, need // (2 if tight else 1), most=100)
        rows = int((want - lens)[grows].sum()) // (2 if tight else 1) + 2
        import torch
        table, dl, ring, state = dev(c["table"]), dev(lens), dev(c["ring"]), dev([c["head"], c["count"], 0, 0])
        shape = KvShape(B=B, Hq=4, Hkv=2, Dk=64, Dv=64, page=page, n_pages=len(c["ring"]), max_pages=c["table"].shape[1])
        start, slot, pos, nl, ns = dev(np.zeros(B + 1)), dev(np.zeros(rows)), dev(np.zeros(rows)), dev(np.zeros(B)), dev([0] * 4)
        coli_kv_plan(shape, table, dl, dev(want), ring, state, start, slot, pos, shared=dev(shared), new_lens=nl, new_state=ns)
        torch.cuda.synchronize()
        r = plain(page, c["table"], lens, want, shared, c["ring"], c["head"], c["count"], rows)
        for k, v in dict(table=table, lens=nl, ring=ring, state=ns, start=start, slot=slot, pos=pos).items():
            assert np.array_equal(v.cpu().numpy(), r[k]), f"{B} sequences: {k} differs"
        assert r["state"][3] >= ((want > lens) & ~grows).sum() > 0
