"""Plain 64-bit forms of the paged key-value cache's operators (numpy, one
sequence and head at a time), seeded caches, and error bounds that follow from
the arithmetic the library documents."""
import numpy as np
import torch

U32 = 2.0 ** -24                         # half a step of fp32
U16 = 2.0 ** -8                          # half a step of bf16


def make_cache(lens, Hkv, Dk, Dv, page, dtype="bf16", latent=False, seed=0, spare_pages=0, poison=True, extra_cols=1):
    """A cache with pages in random order.  Rows that no position owns hold NaN and infinities (poison)."""
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens, np.int64)
    B = len(lens)
    need = -(-lens // page)
    mp = int(max(need.max() if B else 0, 1)) + extra_cols
    n_pages = int(need.sum()) + spare_pages + 2
    ids = rng.permutation(n_pages)
    # behind a sequence's pages: ids that do not exist, and ids of others' pages
    table = rng.choice(np.array([-1, n_pages, 1 << 30, 0], np.int64), size=(B, mp)).astype(np.int32)
    at = 0
    live = np.zeros((n_pages, page), bool)
    for b in range(B):
        own = ids[at:at + need[b]]
        table[b, :need[b]] = own
        for i, pg in enumerate(own):
            live[pg, :min(page, lens[b] - i * page)] = True
        at += need[b]

    def pool(d):
        x = torch.from_numpy(rng.standard_normal((n_pages, Hkv, page, d)).astype(np.float32))
        if poison:
            dead = torch.from_numpy(~live)[:, None, :, None].expand(-1, Hkv, -1, d)
            bad = torch.from_numpy(rng.choice(np.array([np.nan, np.inf, -np.inf], np.float32), size=x.shape))
            x = torch.where(dead, bad, x)
        return x.to(torch.float32 if dtype == "f32" else torch.bfloat16)

    return dict(k=pool(Dk), v=None if latent else pool(Dv), table=torch.from_numpy(table),
                lens=torch.from_numpy(lens.astype(np.int32)), page=page, n_pages=n_pages, max_pages=mp,
                Hkv=Hkv, Dk=Dk, Dv=Dv, free=ids[at:].astype(np.int32), dtype=dtype)


def rows_at(c, b, h, pos, which):
    """Keys or values of head h at positions pos of sequence b (float64), and which pages exist."""
    pos = np.asarray(pos, np.int64)
    pg = c["table"].numpy()[b, pos // c["page"]].astype(np.int64)
    ok = (pg >= 0) & (pg < c["n_pages"])
    pool = c["k"] if which == "k" or c["v"] is None else c["v"]
    x = pool[torch.from_numpy(np.where(ok, pg, 0)), h, torch.from_numpy(pos % c["page"])].double().numpy()
    return (x if which == "k" else x[:, :c["Dv"]]), ok


def attn(c, q, scale, idx=None, acc_in=None):
    """out, lse, acc and their bounds (arrays).  The bounds: a score is a sum of Dk products rounded in fp32,
    off by at most (Dk + 8) half-steps of its products' magnitudes; a weight and the sum that divides it are
    each off by that much, relatively; sums over n positions add at most n half-steps, the base-2 exponential
    and the divisions a few; in bf16 a weight enters the products as two bf16 parts, off by 2^-16, and the
    output is rounded once."""
    B, Hq = q.shape[0], q.shape[1]
    Hkv, Dv = c["Hkv"], c["Dv"]
    G = Hq // Hkv
    lens = c["lens"].numpy()
    bf = c["dtype"] == "bf16"
    out, lse = np.zeros((B, Hq, Dv)), np.full((B, Hq), -np.inf)
    tol_out, tol_lse = np.zeros((B, Hq, Dv)), np.zeros((B, Hq))
    ld = 0 if acc_in is None else acc_in.shape[2]
    acc = None if acc_in is None else acc_in.astype(np.float64)
    tol_acc = None if acc_in is None else np.zeros(acc_in.shape)
    for b in range(B):
        pos = np.arange(lens[b])
        if idx is not None:
            pos = idx[b][(idx[b] >= 0) & (idx[b] < lens[b])]
        for h in range(Hkv):
            K, ok = rows_at(c, b, h, pos, "k")
            V, _ = rows_at(c, b, h, pos, "v")
            K, V, p = K[ok], V[ok], pos[ok]
            n = len(p)
            if n == 0:
                continue
            for i in range(h * G, (h + 1) * G):
                qi = q[b, i].double().numpy()
                t = scale * (K @ qi)
                m = t.max()
                e = np.exp(t - m)
                w = e / e.sum()
                out[b, i] = w @ V
                lse[b, i] = m + np.log(e.sum())
                delta = (c["Dk"] + 8) * U32 * abs(scale) * (np.abs(K) @ np.abs(qi)).max()
                rel = 2 * delta + (n + 32) * U32
                tol_out[b, i] = ((rel + (2.0 ** -16 if bf else 0)) * (w @ np.abs(V))
                                 + (U16 if bf else U32) * np.abs(out[b, i]) * (1 + rel) + 1e-30)
                tol_lse[b, i] = delta + (n + 32) * U32 + 4 * U32 * abs(lse[b, i])
                if acc is not None:
                    acc[b, h, p] += w
                    tol_acc[b, h, p] += w * rel
    if acc is not None:
        tol_acc += (G + 2) * U32 * np.abs(acc)
    return dict(out=out, lse=lse, acc=acc, tol_out=tol_out, tol_lse=tol_lse, tol_acc=tol_acc)


def evict(c, acc, k, tail, new_table, new_acc=None):
    """Moves the kept rows inside c's pools (copies are returned) and gives lens, kept and acc after it."""
    B, Hkv = len(c["lens"]), c["Hkv"]
    lens = c["lens"].numpy()
    k2, v2 = c["k"].clone(), None if c["v"] is None else c["v"].clone()
    kept = np.full((B, Hkv, k), -1, np.int32)
    new_lens = np.minimum(lens, k).astype(np.int32)
    if new_acc is not None:
        new_acc = np.zeros_like(new_acc)
    for b in range(B):
        n, m = int(lens[b]), int(new_lens[b])
        t = min(tail, m)
        for h in range(Hkv):
            best = np.lexsort((np.arange(n - t), -acc[b, h, :n - t].astype(np.float64)))[:m - t]
            keep = np.sort(np.concatenate([best, np.arange(n - t, n)])).astype(np.int64)
            kept[b, h, :m] = keep
            if new_acc is not None:
                new_acc[b, h, :m] = acc[b, h, keep]
            for j, p in enumerate(keep):
                src, dst = int(c["table"][b, p // c["page"]]), int(new_table[b, j // c["page"]])
                if 0 <= src < c["n_pages"] and 0 <= dst < c["n_pages"]:
                    k2[dst, h, j % c["page"]] = c["k"][src, h, p % c["page"]]
                    if v2 is not None:
                        v2[dst, h, j % c["page"]] = c["v"][src, h, p % c["page"]]
    return dict(k=k2, v=v2, kept=kept, new_lens=new_lens, new_acc=new_acc)


def append(c, k_new, v_new, start=None):
    B = len(c["lens"])
    lens = c["lens"].numpy()
    cap = c["max_pages"] * c["page"]
    k2, v2 = c["k"].clone(), None if c["v"] is None else c["v"].clone()
    for b in range(B):
        r = range(start[b], start[b + 1]) if start is not None else range(b, b + 1)
        for x in r:
            p = min(max(int(lens[b]), 0), cap) - (r.stop - x)
            if p < 0:
                continue
            pg = int(c["table"][b, p // c["page"]])
            if 0 <= pg < c["n_pages"]:
                k2[pg, :, p % c["page"]] = k_new[x]
                if v2 is not None:
                    v2[pg, :, p % c["page"]] = v_new[x]
    return k2, v2
