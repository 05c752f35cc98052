"""Plain forms of a serving step's operators (the plan in whole numbers, one sequence at a time; norm and rotation in 64
bits, one head at a time) and error bounds that follow from the arithmetic the library documents."""
import numpy as np
import torch

U32 = 2.0 ** -24                         # half a step of fp32
U16 = 2.0 ** -8                          # half a step of bf16


def plan(page, table, lens, want, shared, ring, head, count, rows):
    """Everything after the call, and the row each token went to."""
    table, ring = table.copy(), ring.copy()
    B, mp = table.shape
    n_pages, cap = len(ring), mp * page
    n, t = np.clip(lens.astype(np.int64), 0, cap), np.clip(want.astype(np.int64), 0, cap)
    pages = lambda x: -(-int(x) // page)
    free = count
    for b in range(B):
        for col in range(max(pages(t[b]), 0 if shared is None else int(shared[b])), pages(n[b])):
            ring[(head + free) % n_pages] = table[b, col]
            free += 1
    new_lens, start, slot, pos = n.copy(), np.zeros(B + 1, np.int64), np.full(rows, -1, np.int64), np.full(rows, -1, np.int64)
    taken = at = refused = asked_pages = asked_rows = 0
    for b in range(B):
        start[b] = at
        if t[b] <= n[b]:
            new_lens[b] = t[b]
            continue
        asked_pages += pages(t[b]) - pages(n[b])
        asked_rows += int(t[b] - n[b])
        if asked_pages > free or asked_rows > rows:
            refused += 1
            continue
        new_lens[b] = t[b]
        for col in range(pages(n[b]), pages(t[b])):
            table[b, col] = ring[(head + taken) % n_pages]
            taken += 1
        for p in range(int(n[b]), int(t[b])):
            pg = int(table[b, p // page])
            slot[at], pos[at] = (pg * page + p % page if 0 <= pg < n_pages else -1), p
            at += 1
    start[B] = at
    state = np.array([(head + taken) % n_pages, free - taken, at, refused])
    return dict(table=table, ring=ring, lens=new_lens, start=start, slot=slot, pos=pos, state=state)


def pairs(rot, rot_at, interleaved):
    i = np.arange(rot // 2)
    return (rot_at + 2 * i, rot_at + 2 * i + 1) if interleaved else (rot_at + i, rot_at + i + rot // 2)


def norm_rope(x, w, eps, pos, freq, rot_at, interleaved, amp, bf16):
    """x [rows][heads][D] of which w normed, rotated by pos * freq: the values and their bounds (float64).

    The norm's sum of n squares, its mean, root and division and the two products are off by at most n / 2 + 6
    half-steps, relatively; the angle's product by 4 half-steps of fp64 and its fraction by 2 of fp32, cosine and
    sine by 4 and their factor by 1; the rotation's products and sum by 2; the result is rounded once."""
    x = np.asarray(x, np.float64).copy()
    rel = 0.0
    if w is not None:
        n = len(w)
        f = 1 / np.sqrt((x[..., :n] ** 2).mean(-1, keepdims=True) + eps)
        x[..., :n] *= f * np.asarray(w, np.float64)
        rel = (n / 2 + 6) * U32
    tol = np.abs(x) * rel
    if freq is not None:
        a, b = pairs(2 * len(freq), rot_at, interleaved)
        angle = pos[:, None].astype(np.float64) * freq
        c, s = amp * np.cos(angle)[:, None], amp * np.sin(angle)[:, None]
        off = (4 * 2.0 ** -53 * np.abs(angle) + 9 * U32)[:, None] * abs(amp)
        u, v = x[..., a], x[..., b]
        size = np.abs(u) + np.abs(v)
        x[..., a], x[..., b] = u * c - v * s, v * c + u * s
        tol[..., a] = tol[..., b] = size * (rel * abs(amp) + off)
    return x, tol * (1 + U16) + np.abs(x) * (U16 if bf16 else U32) + 1e-37


def to_np(t):
    return t.detach().cpu().to(torch.float64).numpy()


def make_shared(groups, Hkv, Dk, Dv, page, dtype="bf16", latent=False, seed=0, room=0):
    """A cache for kv_reference.attn whose sequences share pages: groups [(pages, [positions behind them])].  A value of
    (n,) in place of a number: a sequence of n positions all in all, within its group's pages.  room: positions that the
    table has columns for at least (how a call is cut goes by them)."""
    import kv_reference as kv
    tails = [t for _, ts in groups for t in ts]
    own = [0 if isinstance(t, tuple) else t for t in tails]
    c = kv.make_cache([p * page for p, _ in groups] + own, Hkv, Dk, Dv, page, dtype, latent, seed=seed)
    G, table = len(groups), c["table"].numpy()
    shared = np.repeat([p for p, _ in groups], [len(ts) for _, ts in groups]).astype(np.int32)
    group = np.repeat(np.arange(G), [len(ts) for _, ts in groups])
    mp = max(int(s) + -(-t // page) for s, t in zip(shared, own)) + 1
    mp = max(mp, 1, -(-room // page))
    new = np.full((len(tails), mp), -1, np.int32)
    lens = np.zeros(len(tails), np.int32)
    for b, t in enumerate(tails):
        new[b, :shared[b]] = table[group[b], :shared[b]]
        n = -(-own[b] // page)
        new[b, shared[b]:shared[b] + n] = table[G + b, :n]
        lens[b] = t[0] if isinstance(t, tuple) else shared[b] * page + t
    c.update(table=torch.from_numpy(new), lens=torch.from_numpy(lens), max_pages=mp, shared=torch.from_numpy(shared),
             group_start=torch.from_numpy(np.concatenate([[0], np.cumsum([len(ts) for _, ts in groups])]).astype(np.int32)))
    return c
