"""Cases of the paged key-value cache's operators and how one pass of each is run.

  append   the keys and values of new tokens go into the pages of their sequences
  attn     attention of one new token per sequence over its cached positions: all of them, or the ones an
           index selection lists; it can add each position's attention weight to a running sum
  evict    per sequence and cache head, the positions of largest running weight (the newest always) are
           copied into new pages

``own`` false: elementary torch operations in 32 bits, rounded once at the end.  ``own`` true: the library's entry
points.  Sequences of a batch differ in length; a case's lengths are fixed, the seed gives their order, the pages'
places and all values.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _attn(name, B, Hq, Hkv, Dk, Dv, page, lo, hi, dtype="bf16", latent=False, idx_k=0, acc=False):
    return dict(name=name, op="attn", B=B, Hq=Hq, Hkv=Hkv, Dk=Dk, Dv=Dv, page=page, lo=lo, hi=hi,
                dtype=dtype, latent=latent, idx_k=idx_k, acc=acc)


def _evict(name, B, Hkv, Dk, Dv, page, lo, hi, k, tail, dtype="bf16", latent=False):
    return dict(name=name, op="evict", B=B, Hq=Hkv, Hkv=Hkv, Dk=Dk, Dv=Dv, page=page, lo=lo, hi=hi,
                dtype=dtype, latent=latent, k=k, tail=tail)


def _append(name, B, Hkv, Dk, Dv, page, lo, hi, new_lo, new_hi, dtype="bf16", latent=False):
    return dict(name=name, op="append", B=B, Hq=Hkv, Hkv=Hkv, Dk=Dk, Dv=Dv, page=page, lo=lo, hi=hi,
                dtype=dtype, latent=latent, new_lo=new_lo, new_hi=new_hi)


def listed():
    return [
        # one user's chat, a few hundred tokens in: latency is all that counts
        _attn("attn_one_short", 1, 32, 8, 128, 128, 16, 777, 777),
        # one user with a long document: the work has to be split over the cache's length
        _attn("attn_one_long", 1, 32, 8, 128, 128, 16, 131071, 131071),
        # a serving batch with shared heads, from an empty slot to a full 32768-entry cache
        _attn("attn_batch", 64, 32, 8, 128, 128, 64, 0, 32768),
        # the sparse attention's decode step: 64 rows, 2048 positions each that the index selection took from a
        # 32768-entry latent cache
        _attn("attn_latent_selected", 64, 64, 1, 576, 512, 64, 32768, 32768, latent=True, idx_k=2048),
        # a latent cache of many heads read whole, ragged lengths: as much product as reading
        _attn("attn_latent_batch", 32, 128, 1, 576, 512, 32, 8000, 32768, latent=True),
        # small fp32 model, a head for each query head, a head width that fills no tile
        _attn("attn_f32_odd", 7, 12, 12, 80, 80, 32, 1, 1999, dtype="f32"),
        # a batch whose cache is to be evicted later: the running weights are kept up
        _attn("attn_weights", 16, 32, 8, 128, 128, 16, 1000, 8192, acc=True),
        # a batch over its budget: a quarter of a cache of shared heads stays
        _evict("evict_batch", 16, 8, 128, 128, 16, 4001, 8192, 2048, 4),
        # longer caches with a larger budget than the index selection's 4096
        _evict("evict_large_budget", 8, 8, 128, 128, 64, 32768, 32768, 8192, 64),
        # one long latent cache, an odd budget
        _evict("evict_latent_one", 1, 1, 576, 512, 64, 32768, 32768, 4001, 128, latent=True),
        # decode: one token for each of 64 sequences
        _append("append_decode", 64, 8, 128, 128, 16, 1, 8192, 1, 1),
        # prompts of a batch, ragged
        _append("append_prompts", 24, 8, 128, 128, 16, 40, 2000, 40, 2000),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "evict", "append"])
    latent = rng.random() < 0.35
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
        G = rng.choice([1, 1, 2, 3, 4, 7, 8, 16, 24])
    elt = 4 if dtype == "f32" else 2
    row = Hkv * (Dk + (0 if latent else Dv)) * elt       # bytes of one position
    B = _log_int(rng, 1, 96)
    # the longest length: up to 131072, a batch's cache at most 0.6 GB and its products at most 150 GFLOP
    hi = _log_int(rng, 1, max(2, min(131072, int(0.6e9 / (row * B)), int(150e9 / (2 * Hkv * G * (Dk + Dv) * B)))))
    lo = rng.choice([0, 1, hi, max(1, hi // 9)])
    lo = min(lo, hi)
    if op == "attn":
        idx_k = _log_int(rng, 1, 2048) if rng.random() < 0.3 else 0
        acc = idx_k == 0 and rng.random() < 0.4
        c = _attn("", B, Hkv * G, Hkv, Dk, Dv, page, lo, hi, dtype, latent, idx_k, acc)
    elif op == "evict":
        hi = min(hi, 65536)
        lo = min(lo, hi)
        k = min(_log_int(rng, 1, 8192), max(1, hi))
        c = _evict("", B, Hkv, Dk, Dv, page, lo, hi, k, rng.choice([0, 1, 4, 64, 5000]), dtype, latent)
    else:
        hi = min(hi, 8192)
        new_hi = _log_int(rng, 1, hi)
        c = _append("", B, Hkv, Dk, Dv, page, min(new_hi, hi), hi, rng.choice([1, new_hi]), new_hi, dtype, latent)
    del c["name"]
    return c


def _spread(n, lo, hi):
    """n lengths from lo to hi, even over their logarithm; lo and hi are among them."""
    if n == 1:
        return [hi]
    base = max(lo, 1)
    mid = [int(round(base * (hi / base) ** (i / (n - 1)))) for i in range(n)]
    return [lo] + mid[1:-1] + [hi]


def _lengths(c):
    return _spread(c["B"], c["lo"], c["hi"])


def _news(c):
    """New tokens of each sequence, none with more than its length after them."""
    return [min(a, b) for a, b in zip(_spread(c["B"], c["new_lo"], c["new_hi"]), _lengths(c))]


def _max_pages(c):
    return -(-c["hi"] // c["page"]) + 1                  # one column that no length reaches


def _ld(c):
    return -(-_max_pages(c) * c["page"] // 4) * 4


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    c = case
    dev, dt = "cuda", DTYPES[c["dtype"]]
    host = np.random.default_rng(seed)
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    B, Hq, Hkv, Dk, Dv, page = c["B"], c["Hq"], c["Hkv"], c["Dk"], c["Dv"], c["page"]
    order = host.permutation(B)
    lens = np.array(_lengths(c), np.int64)[order]
    mp = _max_pages(c)
    need = -(-lens // page)
    n_new = -(-c.get("k", 0) // page)
    n_pages = 1 + int(need.sum()) + B * n_new + 3        # page 0 stays free, and three more
    ids = 1 + host.permutation(n_pages - 1)
    table = np.full((B, mp), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :need[b]] = ids[at:at + need[b]]
        at += need[b]

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=dt)

    st = dict(case=c, k=randn(n_pages, Hkv, page, Dk), v=None if c["latent"] else randn(n_pages, Hkv, page, Dv),
              table=torch.from_numpy(table).to(dev), lens=torch.from_numpy(lens.astype(np.int32)).to(dev))
    if c["op"] == "attn":
        st["q"] = randn(B, Hq, Dk)
        # trained heads look at few positions: scores spread by about 2
        st["scale"] = 2.0 / math.sqrt(Dk)
        st["out"] = torch.empty((B, Hq, Dv), dtype=dt, device=dev)
        st["lse"] = torch.empty((B, Hq), dtype=torch.float32, device=dev)
        if c["idx_k"]:
            # the index selection's form: ascending positions of the row, -1 behind them
            kk = c["idx_k"]
            idx = np.full((B, kk), -1, np.int32)
            for b in range(B):
                n = min(kk, int(lens[b]))
                idx[b, :n] = np.sort(host.choice(int(lens[b]), n, replace=False)) if n else []
            st["idx"] = torch.from_numpy(idx).to(dev)
        if c["acc"]:
            live = torch.arange(_ld(c), device=dev) < st["lens"].long()[:, None, None]
            st["acc_in"] = torch.rand((B, Hkv, _ld(c)), generator=g, device=dev) * live
            st["acc_out"] = torch.zeros((B, Hkv, _ld(c)), device=dev)
    elif c["op"] == "evict":
        # running weights: few large ones, many near zero, some exactly equal
        live = torch.arange(_ld(c), device=dev) < st["lens"].long()[:, None, None]
        w = torch.rand((B, Hkv, _ld(c)), generator=g, device=dev)
        st["acc"] = torch.where(w < 0.3, torch.floor(w * 64) / 64, w ** 4) * live
        st["new_table"] = torch.from_numpy(ids[at:at + B * n_new].reshape(B, n_new).astype(np.int32)).to(dev)
        st["new_lens"] = torch.empty(B, dtype=torch.int32, device=dev)
        st["new_acc"] = torch.empty((B, Hkv, -(-c["k"] // 4) * 4 + 64), device=dev)
        st["kept"] = torch.empty((B, Hkv, c["k"]), dtype=torch.int32, device=dev)
    else:
        start = np.concatenate([[0], np.cumsum(np.array(_news(c), np.int64)[order])])
        rows = int(start[-1]) + 5                        # a padded batch: five rows behind the last sequence
        st["start"] = torch.from_numpy(start.astype(np.int32)).to(dev)
        st["k_new"] = randn(rows, Hkv, Dk)
        st["v_new"] = None if c["latent"] else randn(rows, Hkv, Dv)
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _gather(pool, table, pos, valid):
    """Rows of the listed positions: [B, n, Hkv, D] in 32 bits, zero where not valid."""
    page = pool.shape[2]
    p = pos.clamp(min=0)
    pages = torch.gather(table.long(), 1, (p // page).clamp(max=table.shape[1] - 1)).clamp(min=0)
    return torch.where(valid[:, :, None, None], pool[pages, :, p % page].float(), 0.0)


def _plain_attn(st):
    c = st["case"]
    B, Hq, Hkv, Dk, Dv = c["B"], c["Hq"], c["Hkv"], c["Dk"], c["Dv"]
    lens = st["lens"].long()
    if c["idx_k"]:
        pos = st["idx"].long()
    else:
        pos = torch.arange(c["hi"], device=lens.device).expand(B, -1)
    valid = (pos >= 0) & (pos < lens[:, None])
    K = _gather(st["k"], st["table"], pos, valid).transpose(1, 2)                # [B, Hkv, n, Dk]
    V = K[..., :Dv] if st["v"] is None else _gather(st["v"], st["table"], pos, valid).transpose(1, 2)
    q = st["q"].float().view(B, Hkv, Hq // Hkv, Dk)
    s = torch.matmul(q, K.transpose(2, 3)) * st["scale"]                         # [B, Hkv, G, n]
    s = s.masked_fill(~valid[:, None, None, :], -math.inf)
    m = s.amax(-1, keepdim=True)
    m0 = torch.where(torch.isinf(m), 0.0, m)
    e = torch.exp(s - m0)
    l = e.sum(-1, keepdim=True)
    w = e / torch.where(l > 0, l, 1.0)
    out = torch.matmul(w, V).reshape(B, Hq, Dv).to(st["q"].dtype)
    r = dict(out=out, lse=(torch.log(l) + m0).reshape(B, Hq))
    if c["acc"]:
        a = st["acc_in"].clone()
        a[:, :, :c["hi"]] += w.sum(2)
        r["acc"] = a
    return r


def _plain_evict(st):
    c = st["case"]
    k, page = c["k"], c["page"]
    lens = st["lens"].long()
    B, Hkv, ld = st["acc"].shape
    pos = torch.arange(ld, device=lens.device)
    n = lens[:, None, None]
    rank = torch.where(pos < n, st["acc"], -math.inf)
    rank = torch.where((pos >= n - min(c["tail"], k)) & (pos < n), math.inf, rank)
    first = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :k]
    if first.shape[-1] < k:
        first = torch.nn.functional.pad(first, (0, k - first.shape[-1]), value=ld)
    there = torch.arange(k, device=lens.device) < n                              # [B, 1, k]
    kept = torch.where(there, first, ld).sort(-1).values
    new_lens = lens.clamp(max=k)
    src = torch.where(there, kept, 0)                                            # [B, Hkv, k]
    new_acc = torch.zeros_like(st["new_acc"])
    new_acc[..., :k] = torch.where(there, st["acc"].gather(2, src), 0.0)
    h = torch.arange(Hkv, device=lens.device)[:, None]
    # what is not there reads and writes page 0, which no sequence holds: it stays as it is
    sp = torch.where(there, torch.gather(st["table"].long(), 1, (src // page).view(B, -1)).view(B, Hkv, k), 0)
    so = torch.where(there, src % page, 0)
    j = torch.arange(k, device=lens.device)
    dp = torch.where(there, st["new_table"].long()[:, j // page][:, None], 0).expand(B, Hkv, k)
    do = torch.where(there, j % page, 0).expand(B, Hkv, k)
    for pool in (st["k"], st["v"]):
        if pool is not None:
            pool[dp, h, do] = pool[sp, h, so]
    kept = torch.where(there, kept, -1).to(torch.int32)
    return dict(k=st["k"], v=st["v"], new_lens=new_lens.to(torch.int32), new_acc=new_acc, kept=kept)


def _plain_append(st):
    page = st["k"].shape[2]
    rows = torch.arange(st["k_new"].shape[0], device=st["k"].device)
    start, lens = st["start"].long(), st["lens"].long()
    b = (torch.searchsorted(start, rows, right=True) - 1).clamp(max=lens.shape[0] - 1)
    pos = lens[b] - start[b + 1] + rows
    ok = (rows < start[-1]) & (pos >= 0)
    p = pos.clamp(min=0)
    dp = torch.where(ok, st["table"].long()[b, (p // page).clamp(max=st["table"].shape[1] - 1)], 0)
    do = torch.where(ok, p % page, 0)
    for pool, new in ((st["k"], st["k_new"]), (st["v"], st["v_new"])):
        if pool is not None:
            # rows behind the last sequence write page 0's own values there
            pool[dp, :, do] = torch.where(ok[:, None, None], new, pool[0, :, 0])
    return dict(k=st["k"], v=st["v"])


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _handles(st):
    """What a serving program keeps beside its cache: the shape, the cache's handle and the workspace."""
    import sparse_moe_ffn_coli_amd as coli
    c = st["case"]
    shape = coli.KvShape(B=c["B"], Hq=c["Hq"], Hkv=c["Hkv"], Dk=c["Dk"], Dv=c["Dv"], page=c["page"],
                         n_pages=st["k"].shape[0], max_pages=st["table"].shape[1],
                         dtype=coli.COLI_F32 if c["dtype"] == "f32" else coli.COLI_BF16)
    cache = coli.KvCache(st["k"], st["v"], st["table"], st["lens"])
    ws = None
    if c["op"] == "attn":
        n = coli.coli_kv_attn_workspace_bytes(shape, idx_k=c["idx_k"], acc=c["acc"])
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    return coli, shape, cache, ws


def run(state):
    st = state
    op = st["case"]["op"]
    if not own:
        return {"attn": _plain_attn, "evict": _plain_evict, "append": _plain_append}[op](st)
    if "handles" not in st:
        st["handles"] = _handles(st)
    coli, shape, cache, ws = st["handles"]
    if op == "attn":
        coli.coli_kv_attn(shape, st["q"], cache, st["out"], st["scale"], idx=st.get("idx"),
                          acc_in=st.get("acc_in"), acc_out=st.get("acc_out"), lse=st["lse"], ws=ws)
        r = dict(out=st["out"], lse=st["lse"])
        if "acc_out" in st:
            r["acc"] = st["acc_out"]
        return r
    if op == "evict":
        coli.coli_kv_evict(shape, cache, st["acc"], st["case"]["k"], st["new_table"], st["new_lens"], st["kept"],
                           tail=st["case"]["tail"], new_acc=st["new_acc"])
        return dict(k=st["k"], v=st["v"], new_lens=st["new_lens"], new_acc=st["new_acc"], kept=st["kept"])
    coli.coli_kv_append(shape, st["k_new"], st["v_new"], cache, start=st["start"])
    return dict(k=st["k"], v=st["v"])


def work(case):
    c = case
    elt = 4 if c["dtype"] == "f32" else 2
    lens = _lengths(c)
    row = (c["Dk"] + (0 if c["latent"] else c["Dv"])) * elt
    if c["op"] == "attn":
        seen = sum(min(n, c["idx_k"]) for n in lens) if c["idx_k"] else sum(lens)
        nbytes = seen * c["Hkv"] * row + c["B"] * c["Hq"] * ((c["Dk"] + c["Dv"]) * elt + 4)
        nbytes += seen * 4 if c["idx_k"] else sum(-(-n // c["page"]) for n in lens) * 4
        nbytes += seen * c["Hkv"] * 8 if c["acc"] else 0
        return {"bytes": nbytes, "flops": 2 * c["Hq"] * (c["Dk"] + c["Dv"]) * seen}
    if c["op"] == "evict":
        kept = sum(min(n, c["k"]) for n in lens) * c["Hkv"]
        new_ld = -(-c["k"] // 4) * 4 + 64
        return {"bytes": sum(lens) * c["Hkv"] * 4 + 2 * kept * row + c["B"] * c["Hkv"] * (c["k"] + new_ld) * 4,
                "flops": 0}
    return {"bytes": 2 * sum(_news(c)) * c["Hkv"] * row, "flops": 0}


# ---------------------------------------------------------------------------
# the definition in 64 bits, one sequence and cache head at a time
# ---------------------------------------------------------------------------

def _positions(pool, table_row, h, pos):
    """Rows of head h at host positions `pos` of one sequence, in 64 bits."""
    page = pool.shape[2]
    at = torch.from_numpy(table_row[pos // page].astype(np.int64)).to(pool.device)
    return pool[at, h, torch.from_numpy(pos % page).to(pool.device)].double()


def exact(case, seed):
    c = case
    st = prepare(c, seed)
    table, lens = st["table"].cpu().numpy(), st["lens"].cpu().numpy().astype(np.int64)
    B, Hq, Hkv, Dv, page = c["B"], c["Hq"], c["Hkv"], c["Dv"], c["page"]
    G = Hq // Hkv
    if c["op"] == "attn":
        out = torch.zeros((B, Hq, Dv), dtype=torch.float64, device="cuda")
        lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")
        acc = st["acc_in"].double() if c["acc"] else None
        for b in range(B):
            pos = np.arange(lens[b])
            if c["idx_k"]:
                listed_here = st["idx"][b].cpu().numpy().astype(np.int64)
                pos = listed_here[(listed_here >= 0) & (listed_here < lens[b])]
            if not len(pos):
                continue
            for h in range(Hkv):
                K = _positions(st["k"], table[b], h, pos)
                V = K[:, :Dv] if st["v"] is None else _positions(st["v"], table[b], h, pos)
                s = (K @ st["q"][b, h * G:(h + 1) * G].double().T).T * st["scale"]
                lse[b, h * G:(h + 1) * G] = torch.logsumexp(s, -1)
                w = torch.softmax(s, -1)
                out[b, h * G:(h + 1) * G] = w @ V
                if acc is not None:
                    acc[b, h, :lens[b]] += w.sum(0)
        r = dict(out=out, lse=lse)
        if acc is not None:
            r["acc"] = acc
        return r
    if c["op"] == "evict":
        acc = st["acc"].cpu().numpy()
        new_table = st["new_table"].cpu().numpy()
        new_acc = torch.zeros_like(st["new_acc"])
        for b in range(B):
            n = int(lens[b])
            m = min(n, c["k"])
            t = min(c["tail"], m)
            for h in range(Hkv):
                head = acc[b, h, :n - t]
                best = np.lexsort((np.arange(n - t), -head))[:m - t]
                keep = np.sort(np.concatenate([best, np.arange(n - t, n)]))
                new_acc[b, h, :m] = torch.from_numpy(acc[b, h, keep]).to("cuda")
                to = torch.from_numpy(new_table[b, np.arange(m) // page].astype(np.int64)).to("cuda")
                for pool in (st["k"], st["v"]):
                    if pool is not None and m:
                        rows = _positions(pool, table[b], h, keep)
                        pool[to, h, torch.arange(m, device="cuda") % page] = rows.to(pool.dtype)
        return dict(k=st["k"], v=st["v"], new_lens=None, new_acc=new_acc, kept=None)
    start = st["start"].cpu().numpy()
    for b in range(B):
        r = np.arange(start[b], start[b + 1])
        pos = lens[b] - len(r) + np.arange(len(r))
        at = torch.from_numpy(table[b, pos // page].astype(np.int64)).to("cuda")
        off = torch.from_numpy(pos % page).to("cuda")
        for pool, new in ((st["k"], st["k_new"]), (st["v"], st["v_new"])):
            if pool is not None:
                pool[at, :, off] = new[torch.from_numpy(r).to("cuda")]
    return dict(k=st["k"], v=st["v"])
