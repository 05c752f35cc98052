"""Cases of a serving step over the paged key-value cache and how one pass of each operator is run.

  plan    from the lengths that a batch's sequences have and want: pages taken from and given back to a ring of free
          pages, the page tables, and the place and position of every new token
  rope    queries and keys of new tokens: each head's norm and the rotation by its position in one pass; the queries
          come out, the keys and values go to their places in the pages
  shared  attention of one new token per sequence where groups of sequences begin with the same pages

``own`` false: elementary torch operations in 32 bits (angles in 64), rounded once at the end.  ``own`` true: the
library's entry points.  A case's lengths are fixed, the seed gives their order, the pages' places and all values.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _plan(name, B, page, lo, hi, new_lo, new_hi, mix=False, tight=False):
    """Lengths lo..hi, new tokens new_lo..new_hi of each; mix: some sequences end, lose tokens, rest or are new;
    tight: the ring holds too few pages for all."""
    return dict(name=name, op="plan", B=B, page=page, lo=lo, hi=hi, new_lo=new_lo, new_hi=new_hi, mix=mix, tight=tight)


def _rope(name, rows, Hq, Hkv, Dk, Dv, page, rot, rot_at, interleaved, norm, scaling, far, dtype="bf16", latent=False):
    """norm: elements of a head that are normed, from its first on (0: none); far: the largest position."""
    return dict(name=name, op="rope", rows=rows, Hq=Hq, Hkv=Hkv, Dk=Dk, Dv=Dv, page=page, rot=rot, rot_at=rot_at,
                interleaved=interleaved, norm=norm, scaling=scaling, far=far, dtype=dtype, latent=latent)


def _shared(name, B, groups, Hq, Hkv, Dk, Dv, page, pre_lo, pre_hi, lo, hi, idle=0, dtype="bf16", latent=False):
    """groups: runs of sequences with a prefix each, of pre_lo..pre_hi positions (whole pages); lo..hi: positions of a
    sequence's own behind it; idle: slots of length 0."""
    return dict(name=name, op="shared", B=B, groups=groups, Hq=Hq, Hkv=Hkv, Dk=Dk, Dv=Dv, page=page, pre_lo=pre_lo,
                pre_hi=pre_hi, lo=lo, hi=hi, idle=idle, dtype=dtype, latent=latent)


def listed():
    return [
        # decode: one token for each of 64 sequences; few of them need a page
        _plan("plan_decode", 64, 16, 1, 8192, 1, 1),
        # a step of a busy server: most sequences decode, some have ended, lost rejected tokens or bring a prompt
        _plan("plan_mixed", 500, 16, 1, 8192, 1, 2000, mix=True),
        # a long queue of prompts, more than the pool holds
        _plan("plan_prompts", 1024, 64, 0, 0, 1, 8192, tight=True),
        # one user's next token: latency is all that counts
        _rope("rope_one", 1, 32, 8, 128, 128, 16, 128, 0, False, 128, "none", 777),
        # a serving batch's decode step over latent rows: the latent part is normed, the 64 last elements rotated
        _rope("rope_latent_decode", 64, 64, 1, 576, 512, 64, 64, 512, True, 512, "yarn", 131071, latent=True),
        # prompts of a batch, heads normed and rotated whole
        _rope("rope_prompts", 16384, 32, 8, 128, 128, 16, 128, 0, False, 128, "ntk", 32768),
        # small fp32 model, a part of an odd head, positions of a million
        _rope("rope_f32_part", 4001, 12, 12, 80, 80, 32, 32, 0, True, 0, "linear", 1 << 20, dtype="f32"),
        # four samples of one prompt
        _shared("shared_samples", 4, 1, 32, 8, 128, 128, 16, 2000, 2000, 1, 300),
        # a serving batch behind one long system prompt
        _shared("shared_batch", 64, 1, 32, 8, 128, 128, 64, 32768, 32768, 0, 2048, idle=2),
        # several prompts, each with its users
        _shared("shared_groups", 95, 5, 32, 8, 128, 128, 16, 500, 16000, 1, 1000, idle=1),
        # latent rows, all heads on one cache head
        _shared("shared_latent", 32, 1, 64, 1, 576, 512, 64, 32768, 32768, 1, 1024, latent=True),
        # small fp32 model, a head for each query head
        _shared("shared_f32_odd", 13, 2, 12, 12, 80, 80, 32, 300, 1999, 1, 257, dtype="f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "rope", "rope", "shared", "shared", "shared"])
    latent = rng.random() < 0.3
    dtype = "f32" if rng.random() < 0.25 else "bf16"
    page = rng.choice([1, 8, 16, 32, 64, 128])
    if latent:
        Hkv, Dk, Dv = 1, *rng.choice([(576, 512), (512, 512), (320, 256), (288, 256)])
        G = rng.choice([8, 12, 16, 32, 64, 100, 128])
    else:
        Dk = Dv = rng.choice([64, 80, 96, 128, 128, 192, 256])
        if rng.random() < 0.2:
            Dk, Dv = 192, 128
        Hkv = rng.choice([1, 2, 4, 5, 8, 12])
        G = rng.choice([1, 1, 2, 3, 4, 7, 8, 16])
    elt = 4 if dtype == "f32" else 2
    if op == "plan":
        B = _log_int(rng, 1, 1024)
        hi = _log_int(rng, 1, 8192)
        new_hi = _log_int(rng, 1, 8192)
        c = _plan("", B, page, rng.choice([0, 1, hi]), hi, rng.choice([1, new_hi]) if B * new_hi < 1 << 20 else 1, new_hi,
                  rng.random() < 0.5, rng.random() < 0.3)
    elif op == "rope":
        row = (Hkv * (G * Dk + Dk + (0 if latent else Dv))) * elt
        rows = _log_int(rng, 1, max(2, min(65536, int(190e6 / row))))
        rot = min(Dk, 8 * rng.choice([1, 3, 4, 8, 8, 10, 16, 32]))
        rot_at = Dk - rot if latent or rng.random() < 0.3 else 0
        norm = rng.choice([0, Dk, Dk, Dv]) if not latent else Dv
        c = _rope("", rows, Hkv * G, Hkv, Dk, Dv, page, rot, rot_at, rng.random() < 0.5, norm,
                  rng.choice(["none", "linear", "ntk", "yarn"]), _log_int(rng, 2, 1 << 20), dtype, latent)
    else:
        B = _log_int(rng, 1, 96)
        groups = min(B, rng.choice([1, 1, 2, 3, 7]))
        pos = Hkv * (Dk + (0 if latent else Dv)) * elt         # bytes of one position
        # a prefix of up to 65536 positions, products of at most 140 GFLOP, and what the plain form keeps of them
        most = min(65536, int(140e9 / (2 * Hkv * G * (Dk + Dv) * B)), int(1e9 / (4 * Hkv * G * B)), int(0.5e9 / pos))
        if dtype == "f32":
            most = min(most, int(20e9 / (2 * Hkv * G * (Dk + Dv) * B)))
        pre_hi = _log_int(rng, 1, max(2, most))
        pre_lo = rng.choice([1, pre_hi])
        hi = _log_int(rng, 1, max(2, min(2048, pre_hi, int(0.3e9 / (pos * B)))))
        c = _shared("", B, groups, Hkv * G, Hkv, Dk, Dv, page, pre_lo, pre_hi, rng.choice([0, 1, hi]), hi,
                    rng.choice([0, 0, 1, 2]) if B > 2 else 0, dtype, latent)
    del c["name"]
    return c


def _spread(n, lo, hi):
    """n lengths from lo to hi, even over their logarithm; lo and hi are among them."""
    if n == 1:
        return [hi]
    base = max(lo, 1)
    mid = [int(round(base * (max(hi, 1) / base) ** (i / (n - 1)))) for i in range(n)]
    return [lo] + mid[1:-1] + [hi]


def _plan_lens(c):
    """(length, wanted length) of every sequence, in the cases' own order."""
    have, news = _spread(c["B"], c["lo"], c["hi"]), _spread(c["B"], c["new_lo"], c["new_hi"])
    if not c["mix"]:
        return [(n, n + a) for n, a in zip(have, news)]
    kinds = [lambda n, a: (n, n + 1)] * 9 + [lambda n, a: (n, 0), lambda n, a: (n, max(n - 3, 0)),
                                             lambda n, a: (n, n), lambda n, a: (0, a)]
    # (7 i: each kind meets short and long sequences)
    return [kinds[7 * i % len(kinds)](n, a) for i, (n, a) in enumerate(zip(have, news))]


def _pages(n, page):
    return -(-n // page)


def _group_sizes(c):
    """Sequences of each group: as even as an odd share lets them be, none empty."""
    left, sizes = c["B"], []
    for g in range(c["groups"], 0, -1):
        n = max(1, min(left - (g - 1), left // g + (g % 2) * (left // (3 * g))))
        sizes.append(n if g > 1 else left)
        left -= sizes[-1]
    return sizes


def _prefixes(c):
    """Pages of each group's prefix."""
    return [max(1, n // c["page"]) for n in _spread(c["groups"], c["pre_lo"], c["pre_hi"])]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


def _prepare_plan(c, host):
    B, page = c["B"], c["page"]
    order = host.permutation(B)
    lens, want = np.array(_plan_lens(c), np.int64)[order].T
    # every fourth long sequence begins with two pages that are not its own
    shared = np.where((np.arange(B) % 4 == 1) & (np.minimum(lens, want) > 2 * page), 2, 0)
    held, need = _pages(lens, page), _pages(want, page)
    take = int(np.maximum(need - held, 0).sum())
    free = take // 2 + 1 if c["tight"] else take + 5
    n_pages = int(held.sum()) + free + 2
    ids = host.permutation(n_pages)
    mp = int(max(need.max(), held.max(), 1)) + 1
    table = np.full((B, mp), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    ring, head = np.full(n_pages, -1, np.int32), int(host.integers(n_pages))
    ring[(head + np.arange(free)) % n_pages] = ids[at:at + free]
    rows = int(np.maximum(want - lens, 0).sum()) + 3           # a padded step
    new = dict(dtype=torch.int32, device="cuda")
    return dict(table=_i32(table), lens=_i32(lens), want=_i32(want), shared=_i32(shared), ring=_i32(ring),
                state=_i32([head, free, 0, 0]), new_lens=torch.empty(B, **new), new_state=torch.empty(4, **new),
                start=torch.empty(B + 1, **new), slot=torch.empty(rows, **new), pos=torch.empty(rows, **new))


def _freqs(c):
    """Angle per position of each pair, in 64 bits, and the factor on cosines and sines."""
    R = c["rot"]
    i, s, base = np.arange(R // 2, dtype=np.float64), 8.0, 10000.0
    f = base ** (-2 * i / R)
    if c["scaling"] == "linear":
        return f / s, 1.0
    if c["scaling"] == "ntk":
        return (base * s ** (R / (R - 2))) ** (-2 * i / R), 1.0
    if c["scaling"] == "yarn":
        turns = 4096 * f / (2 * math.pi)
        keep = np.clip((turns - 1) / 31, 0, 1)
        return f * keep + f / s * (1 - keep), 0.1 * math.log(s) + 1
    return f, 1.0


def _prepare_rope(c, host, g):
    dt, rows, page = DTYPES[c["dtype"]], c["rows"], c["page"]
    Hq, Hkv, Dk, Dv = c["Hq"], c["Hkv"], c["Dk"], c["Dv"]

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=dt)

    if c["latent"]:
        q, k, v = randn(rows, Hq, Dk), randn(rows, Hkv, Dk), None
    else:                                                      # one projection's output
        x = randn(rows, (Hq + Hkv) * Dk + Hkv * Dv)
        q = x[:, :Hq * Dk].unflatten(1, (Hq, Dk))
        k = x[:, Hq * Dk:(Hq + Hkv) * Dk].unflatten(1, (Hkv, Dk))
        v = x[:, (Hq + Hkv) * Dk:].unflatten(1, (Hkv, Dv))
    n_pages = _pages(rows, page) + 3
    # runs of up to 1000 tokens of one sequence, from any position on; some rows have no place, the last is none
    pos, at = np.empty(rows, np.int64), 0
    while at < rows:
        n = min(rows - at, int(host.integers(1, 1000)))
        pos[at:at + n] = host.integers(0, max(c["far"] - n, 1)) + np.arange(n)
        at += n
    slot = host.permutation(n_pages)[np.arange(rows) // page] * page + np.arange(rows) % page
    if rows > 8:
        slot[3], slot[-1], pos[-1] = -1, -1, -1
    f, amp = _freqs(c)
    nw = c["norm"]
    st = dict(q=q, k=k, v=v, pos=_i32(pos), slot=_i32(slot), freq=torch.from_numpy(f).cuda(), amp=amp,
              # (a row without a position stays as it is)
              q_out=torch.zeros((rows, Hq, Dk), dtype=dt, device="cuda"),
              pool_k=randn(n_pages, Hkv, page, Dk), pool_v=None if v is None else randn(n_pages, Hkv, page, Dv))
    # an absorbed query is not normed: its norm came before the absorption
    st["q_w"] = None if c["latent"] or not nw else (1 + 0.1 * randn(nw).float()).to(dt)
    st["k_w"] = (1 + 0.1 * randn(nw).float()).to(dt) if nw else None
    return st


def _prepare_shared(c, host, g):
    dt, B, page = DTYPES[c["dtype"]], c["B"], c["page"]
    Hq, Hkv, Dk, Dv = c["Hq"], c["Hkv"], c["Dk"], c["Dv"]
    sizes, pre = _group_sizes(c), _prefixes(c)
    start = np.concatenate([[0], np.cumsum(sizes)])
    shared = np.repeat(pre, sizes)
    tail = np.array(_spread(B, c["lo"], c["hi"]), np.int64)[host.permutation(B)]
    need = shared + _pages(tail, page)
    lens = shared * page + tail
    if c["idle"]:
        lens[host.choice(B, c["idle"], replace=False)] = 0
    mp = int(need.max()) + 1
    n_pages = sum(pre) + int(_pages(tail, page).sum()) + 2
    ids = host.permutation(n_pages)
    table = np.full((B, mp), -1, np.int32)
    at = 0
    for i in range(c["groups"]):
        table[start[i]:start[i + 1], :pre[i]] = ids[at:at + pre[i]]
        at += pre[i]
    for b in range(B):
        n = need[b] - shared[b]
        table[b, shared[b]:need[b]] = ids[at:at + n]
        at += n

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=dt)

    return dict(k=randn(n_pages, Hkv, page, Dk), v=None if c["latent"] else randn(n_pages, Hkv, page, Dv), table=_i32(table),
                lens=_i32(lens), shared=_i32(shared), group_start=_i32(start), q=randn(B, Hq, Dk),
                # trained heads look at few positions: scores spread by about 2
                scale=2.0 / math.sqrt(Dk), out=torch.empty((B, Hq, Dv), dtype=dt, device="cuda"),
                lse=torch.empty((B, Hq), dtype=torch.float32, device="cuda"))


def prepare(case, seed):
    host = np.random.default_rng(seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if case["op"] == "plan":
        st = _prepare_plan(case, host)
    else:
        st = (_prepare_rope if case["op"] == "rope" else _prepare_shared)(case, host, g)
    st["case"] = case
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _plain_plan(st):
    page, (B, mp) = st["case"]["page"], st["table"].shape
    n_pages, rows = st["ring"].shape[0], st["slot"].shape[0]
    table, ring = st["table"], st["ring"]
    cap = mp * page
    n, t = st["lens"].long().clamp(0, cap), st["want"].long().clamp(0, cap)
    held, need = (n + page - 1) // page, (t + page - 1) // page
    head, count = st["state"][0].long(), st["state"][1].long()
    col = torch.arange(mp, device=n.device)
    # pages that go back, in order of sequences and columns, to the ring's tail
    back = (col >= torch.maximum(need, st["shared"].long())[:, None]) & (col < held[:, None])
    at = torch.cumsum(back.view(-1), 0)
    n_back = at[-1]
    # (pages that stay write entry n_pages of a longer ring)
    longer = torch.cat([ring, ring.new_zeros(1)])
    longer[torch.where(back.view(-1), (head + count + at - 1) % n_pages, n_pages)] = table.view(-1)
    ring.copy_(longer[:-1])
    # who grows, first come first served
    more, tokens = (need - held).clamp(min=0), (t - n).clamp(min=0)
    upto = torch.cumsum(more, 0)
    fits = (tokens == 0) | ((upto <= count + n_back) & (torch.cumsum(tokens, 0) <= rows))
    t = torch.where(fits, t, n)
    need = torch.where(fits, need, held)
    new = (col >= held[:, None]) & (col < need[:, None])
    source = (head + torch.cumsum(new.view(-1), 0) - 1) % n_pages
    table.copy_(torch.where(new, ring[source].view(B, mp), table))
    taken = new.sum()
    tokens = (t - n).clamp(min=0)
    start = torch.cat([tokens.new_zeros(1), torch.cumsum(tokens, 0)])
    r = torch.arange(rows, device=n.device)
    b = (torch.searchsorted(start, r, right=True) - 1).clamp(max=B - 1)
    live = r < start[-1]
    pos = torch.where(live, t[b] - start[b + 1] + r, 0)
    slot = table[b, pos // page] * page + pos % page
    state = torch.stack([(head + taken) % n_pages, count + n_back - taken, start[-1], (~fits).sum()])
    i32 = torch.int32
    return dict(table=table, ring=ring, lens=t.to(i32), state=state.to(i32), start=start.to(i32),
                slot=torch.where(live, slot, -1).to(i32), pos=torch.where(live, pos, -1).to(i32))


def _plain_rope(st):
    c = st["case"]
    dt, page = st["q"].dtype, c["page"]
    pos, slot = st["pos"].long(), st["slot"].long()
    angle = pos.double()[:, None] * st["freq"]
    cos, sin = (angle.cos() * st["amp"]).float()[:, None], (angle.sin() * st["amp"]).float()[:, None]
    lo, hi = c["rot_at"], c["rot_at"] + c["rot"]

    def one(x, w):
        x = x.float()
        if w is not None:
            part = x[..., :c["norm"]]
            part = part * torch.rsqrt((part * part).mean(-1, keepdim=True) + 1e-6) * w.float()
            x = torch.cat([part, x[..., c["norm"]:]], -1)
        r = x[..., lo:hi]
        if c["interleaved"]:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = r[..., :c["rot"] // 2], r[..., c["rot"] // 2:]
            r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([x[..., :lo], r, x[..., hi:]], -1).to(dt)

    live = pos >= 0
    q_out = torch.where(live[:, None, None], one(st["q"], st["q_w"]), st["q_out"])
    ok = live & (slot >= 0)
    # (rows without a place write a page behind the pool)
    to = torch.where(ok, slot // page, st["pool_k"].shape[0])
    for pool, new in ((st["pool_k"], one(st["k"], st["k_w"])), (st["pool_v"], st["v"])):
        if pool is not None:
            longer = torch.cat([pool, pool[:1]])
            longer[to, :, slot % page] = new
            pool.copy_(longer[:-1])
    return dict(q=q_out, k=st["pool_k"], v=st["pool_v"])


def _plain_shared(st):
    c = st["case"]
    B, Hq, Hkv, Dk, Dv, page = c["B"], c["Hq"], c["Hkv"], c["Dk"], c["Dv"], c["page"]
    G, table, lens = Hq // Hkv, st["table"].long(), st["lens"].long()
    first = st["shared"].long() * page
    q = st["q"].float().view(B, Hkv, G, Dk) * st["scale"]
    vpool = st["k"] if st["v"] is None else st["v"]
    # the sequences' own positions
    n = max(c["hi"], 1)
    pos = first[:, None] + torch.arange(n, device=lens.device)
    own_ok = pos < lens[:, None]
    at = torch.where(own_ok, pos, 0)
    pages = torch.gather(table, 1, at // page).clamp(min=0)
    K = st["k"][pages, :, at % page].float().transpose(1, 2)                      # [B, Hkv, n, Dk]
    V = vpool[pages, :, at % page][..., :Dv].float().transpose(1, 2)
    s = torch.matmul(q, K.transpose(2, 3)).masked_fill(~own_ok[:, None, None], -math.inf)
    out = torch.empty((B, Hkv, G, Dv), device=q.device)
    lse = torch.empty((B, Hkv, G), device=q.device)
    b0 = 0
    for size, pre in zip(_group_sizes(c), _prefixes(c)):
        g = slice(b0, b0 + size)
        row = table[b0, :pre]
        pk = st["k"][row].float().transpose(0, 1).reshape(Hkv, pre * page, Dk)
        pv = vpool[row][..., :Dv].float().transpose(0, 1).reshape(Hkv, pre * page, Dv)
        ps = torch.matmul(q[g].transpose(0, 1).reshape(Hkv, size * G, Dk), pk.transpose(1, 2))
        ok = (torch.arange(pre * page, device=lens.device) < lens[g, None]).repeat_interleave(G, 0)
        ps = ps.masked_fill(~ok, -math.inf)
        so = s[g].transpose(0, 1).reshape(Hkv, size * G, n)
        m = torch.maximum(ps.amax(-1, keepdim=True), so.amax(-1, keepdim=True))
        m0 = torch.where(torch.isinf(m), 0.0, m)
        pe, oe = torch.exp(ps - m0), torch.exp(so - m0)
        total = pe.sum(-1, keepdim=True) + oe.sum(-1, keepdim=True)
        o = torch.matmul(pe, pv)
        oe = oe.view(Hkv, size, G, n).transpose(0, 1)
        o = o.view(Hkv, size, G, Dv).transpose(0, 1) + torch.matmul(oe, V[g])
        total = total.view(Hkv, size, G, 1).transpose(0, 1)
        out[g] = o / torch.where(total > 0, total, 1.0)
        lse[g] = (torch.log(total) + m0.view(Hkv, size, G, 1).transpose(0, 1))[..., 0]
        b0 += size
    return dict(out=out.view(B, Hq, Dv).to(st["q"].dtype), lse=lse.view(B, Hq))


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _handles(st):
    """What a serving program keeps beside its cache: the shape, the cache's handle, the rotation and the workspace."""
    import sparse_moe_ffn_coli_amd as coli
    c = st["case"]
    op = c["op"]
    if op == "plan":
        B, mp = st["table"].shape
        return coli, coli.KvShape(B=B, Hq=8, Hkv=8, Dk=128, Dv=128, page=c["page"], n_pages=st["ring"].shape[0], max_pages=mp)
    k, v = (st["pool_k"], st["pool_v"]) if op == "rope" else (st["k"], st["v"])
    mp = 1 if op == "rope" else st["table"].shape[1]
    shape = coli.KvShape(B=c.get("B", 0), Hq=c["Hq"], Hkv=c["Hkv"], Dk=c["Dk"], Dv=c["Dv"], page=c["page"], n_pages=k.shape[0],
                         max_pages=mp, dtype=coli.COLI_F32 if c["dtype"] == "f32" else coli.COLI_BF16)
    if op == "rope":
        rope = coli.Rope(freq=st["freq"], rot_at=c["rot_at"], interleaved=c["interleaved"], amp=st["amp"])
        norm = coli.QkNorm(q_w=st["q_w"], k_w=st["k_w"], eps=1e-6) if c["norm"] else None
        return coli, shape, rope, norm
    ws = torch.empty(coli.coli_kv_attn_shared_workspace_bytes(shape, c["groups"]), dtype=torch.uint8, device="cuda")
    return coli, shape, coli.KvCache(k, v, st["table"], st["lens"]), ws


def run(state):
    st = state
    op = st["case"]["op"]
    if not own:
        return {"plan": _plain_plan, "rope": _plain_rope, "shared": _plain_shared}[op](st)
    if "handles" not in st:
        st["handles"] = _handles(st)
    if op == "plan":
        coli, shape = st["handles"]
        coli.coli_kv_plan(shape, st["table"], st["lens"], st["want"], st["ring"], st["state"], st["start"], st["slot"], st["pos"],
                          shared=st["shared"], new_lens=st["new_lens"], new_state=st["new_state"])
        return dict(table=st["table"], ring=st["ring"], lens=st["new_lens"], state=st["new_state"], start=st["start"],
                    slot=st["slot"], pos=st["pos"])
    if op == "rope":
        coli, shape, rope, norm = st["handles"]
        coli.coli_kv_rope(shape, st["q"], st["k"], st["v"], st["q_out"], pos=st["pos"], rope=rope, norm=norm,
                          pool_k=st["pool_k"], pool_v=st["pool_v"], slot=st["slot"])
        return dict(q=st["q_out"], k=st["pool_k"], v=st["pool_v"])
    coli, shape, cache, ws = st["handles"]
    coli.coli_kv_attn_shared(shape, st["q"], cache, st["out"], st["scale"], st["shared"], st["group_start"], lse=st["lse"], ws=ws)
    return dict(out=st["out"], lse=st["lse"])


def work(case):
    c = case
    if c["op"] == "plan":
        pairs = _plan_lens(c)
        moved = sum(abs(_pages(t, c["page"]) - _pages(n, c["page"])) for n, t in pairs)
        tokens = sum(max(t - n, 0) for n, t in pairs)
        if c["tight"]:                                         # about half of them find a place
            moved, tokens = moved // 2, tokens // 2
        return {"bytes": 5 * 4 * c["B"] + 8 * moved + 8 * tokens, "flops": 0}
    elt = 4 if c["dtype"] == "f32" else 2
    row = c["Hkv"] * (c["Dk"] + (0 if c["latent"] else c["Dv"])) * elt
    if c["op"] == "rope":
        q = c["Hq"] * c["Dk"] * elt
        elements = c["rows"] * (c["Hq"] + c["Hkv"])
        return {"bytes": c["rows"] * (2 * (q + row) + 8), "flops": elements * (4 * c["norm"] + 3 * c["rot"])}
    sizes, pre = _group_sizes(c), _prefixes(c)
    tail = sum(_spread(c["B"], c["lo"], c["hi"]))
    positions = sum(pre) * c["page"] + tail
    nbytes = positions * row + c["B"] * c["Hq"] * ((c["Dk"] + c["Dv"]) * elt + 4) + _pages(positions, c["page"]) * 4
    seen = sum(n * p for n, p in zip(sizes, pre)) * c["page"] + tail
    return {"bytes": nbytes, "flops": 2 * c["Hq"] * (c["Dk"] + c["Dv"]) * seen}


# ---------------------------------------------------------------------------
# the definition in 64 bits, one sequence (or token) and head at a time
# ---------------------------------------------------------------------------

def _exact_rope(c, st):
    page, R, lo = c["page"], c["rot"], c["rot_at"]
    f, amp = _freqs(c)
    pos, slot = st["pos"].cpu().numpy(), st["slot"].cpu().numpy()
    # each pair's place in the head
    first = lo + (2 * np.arange(R // 2) if c["interleaved"] else np.arange(R // 2))
    second = first + (1 if c["interleaved"] else R // 2)
    angle = torch.from_numpy(np.where(pos < 0, 0, pos)[:, None] * f).cuda()
    z = torch.polar(torch.full_like(angle, amp), angle)
    first, second = torch.from_numpy(first).cuda(), torch.from_numpy(second).cuda()

    def head(x, w):
        x = x.double()                                         # [rows, D]
        if w is not None:
            m = c["norm"]
            x[:, :m] = x[:, :m] / torch.sqrt(x[:, :m].square().sum(-1, keepdim=True) / m + 1e-6) * w.double()
        y = torch.complex(x[:, first], x[:, second]) * z
        x[:, first], x[:, second] = y.real, y.imag
        return x

    rows = np.nonzero(pos >= 0)[0]
    put = rows[slot[rows] >= 0]
    rows = torch.from_numpy(rows).cuda()
    q = st["q_out"].double()
    for h in range(c["Hq"]):
        q[rows, h] = head(st["q"][:, h], st["q_w"])[rows]
    pg, off = torch.from_numpy(slot[put] // page).cuda(), torch.from_numpy(slot[put] % page).cuda()
    put = torch.from_numpy(put).cuda()
    k, v = st["pool_k"].double(), None if st["pool_v"] is None else st["pool_v"].double()
    for h in range(c["Hkv"]):
        k[pg, h, off] = head(st["k"][:, h], st["k_w"])[put]
        if v is not None:
            v[pg, h, off] = st["v"][put, h].double()
    return dict(q=q, k=k, v=v)


def _exact_shared(c, st):
    B, Hq, Hkv, Dv, page = c["B"], c["Hq"], c["Hkv"], c["Dv"], c["page"]
    G = Hq // Hkv
    table, lens = st["table"].cpu().numpy().astype(np.int64), st["lens"].cpu().numpy()
    out = torch.zeros((B, Hq, Dv), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(B):
        p = np.arange(lens[b])
        if not len(p):
            continue
        pg, off = torch.from_numpy(table[b, p // page]).cuda(), torch.from_numpy(p % page).cuda()
        for h in range(Hkv):
            K = st["k"][pg, h, off].double()
            V = K[:, :Dv] if st["v"] is None else st["v"][pg, h, off].double()
            s = (K @ st["q"][b, h * G:(h + 1) * G].double().T).T * st["scale"]
            lse[b, h * G:(h + 1) * G] = torch.logsumexp(s, -1)
            out[b, h * G:(h + 1) * G] = torch.softmax(s, -1) @ V
    return dict(out=out, lse=lse)


def exact(case, seed):
    if case["op"] == "plan":
        return None                                            # whole numbers: the plain form's are the definition's
    st = prepare(case, seed)
    return (_exact_rope if case["op"] == "rope" else _exact_shared)(case, st)
