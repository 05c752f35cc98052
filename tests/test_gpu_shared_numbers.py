"""Shared pages and what is no number: keys of minus infinity or the type's lowest value, queries and keys with NaN or
infinities, the largest values, by every kernel that a part may take."""
import numpy as np
import pytest
import torch

import kv_reference as ref
from serve_reference import make_shared
from test_gpu_kv import within
from test_gpu_shared import queries, run

pytestmark = pytest.mark.gpu

# dtype, Hq, Hkv, Dk, Dv, latent, room of the table (200000: bf16 pages through LDS)
KERNELS = [("bf16", 40, 1, 128, 128, False, 200000), ("bf16", 8, 2, 128, 128, False, 0), ("bf16", 40, 1, 64, 64, False, 200000),
           ("bf16", 40, 1, 192, 128, False, 200000), ("bf16", 40, 1, 256, 256, False, 200000), ("bf16", 40, 1, 120, 80, True, 200000),
           ("f32", 6, 2, 80, 80, False, 0), ("f32", 20, 1, 576, 512, True, 0), ("bf16", 20, 1, 576, 512, True, 0),
           ("bf16", 100, 1, 576, 512, True, 0), ("bf16", 40, 1, 320, 256, True, 0), ("bf16", 20, 1, 200, 128, True, 0)]


def close(out, lse, r, at=...):
    within(out[at].double().numpy(), r["out"][at], r["tol_out"][at], "out")
    within(lse[at].numpy(), r["lse"][at], r["tol_lse"][at], "lse")


@pytest.mark.parametrize("dtype,Hq,Hkv,Dk,Dv,latent,room", KERNELS)
@pytest.mark.parametrize("bad", [-np.inf, "lowest"])
def test_scores_of_minus_infinity(dtype, Hq, Hkv, Dk, Dv, latent, room, bad):
    """Every fifth position, in the pages and behind them, has no weight: the plain form reads the same cache with those
    pages (of one position) hidden.  The scale's second part has either sign."""
    for scale in (2.0, 2.0 / np.sqrt(Dk), 0.125, 2.0 / np.sqrt(96)):
        c = make_shared([(300, [40, 3, 0, (7,), (200,)]), (0, [9]), (33, [1, 500])], Hkv, Dk, Dv, 1, dtype, latent, seed=91, room=room)
        q = queries(c, len(c["lens"]), Hq)
        q[..., Dk - 1] = q[..., Dk - 1].abs() + 0.5
        same = dict(c, table=c["table"].clone())
        for b, n in enumerate(c["lens"].tolist()):
            at = np.arange(1, n, 5)
            c["k"][c["table"][b, at].long(), :, 0, Dk - 1] = torch.finfo(c["k"].dtype).min if bad == "lowest" else bad
            same["table"][b, at] = -1
        close(*run(c, Hq, scale, q=q, want=False), ref.attn(same, q, scale))


@pytest.mark.parametrize("dtype,Hq,Hkv,Dk,Dv,latent,room", KERNELS)
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_queries_that_are_no_numbers(dtype, Hq, Hkv, Dk, Dv, latent, room, bad):
    """One query head of each sequence: its own outputs are NaN (of one position the score may be minus infinity alone), and
    nothing else is."""
    for scale in (0.2, -0.2):
        c = make_shared([(30, [40, 3, 0, (70,), (1,)]), (0, [9]), (3, [1, 500])], Hkv, Dk, Dv, 16, dtype, latent, seed=92, room=room)
        q = queries(c, len(c["lens"]), Hq)
        r = ref.attn(c, q, scale)
        heads = np.arange(len(q)) * 7 % Hq
        q[np.arange(len(q)), heads, 3] = bad
        out, lse = run(c, Hq, scale, q=q, want=False)
        for b, n in enumerate(c["lens"].tolist()):
            rest = np.arange(Hq) != heads[b]
            close(out, lse, r, (b, rest))
            if n > 1:
                assert bool(out[b, heads[b]].isnan().all()) and bool(lse[b, heads[b]].isnan())


@pytest.mark.parametrize("dtype,Hq,Hkv,Dk,Dv,latent,room", KERNELS)
def test_a_key_that_is_no_number(dtype, Hq, Hkv, Dk, Dv, latent, room):
    # in the pages all that read them are NaN, behind them its own sequence
    for at in (0, 500, 959, 960, 1500):
        c = make_shared([(60, [40, 3, 900]), (3, [5])], Hkv, Dk, Dv, 16, dtype, latent, seed=93, room=room)
        who = [b for b in range(3) if at < int(c["lens"][b])]
        for b in who:
            c["k"][c["table"][b, at // 16], :, at % 16] = float("nan")
        out, lse = run(c, Hq, 0.1, want=False)
        for b in range(4):
            for x in (out[b], lse[b]):
                assert bool(x.isnan().all() if b in who else x.isfinite().all()), (at, b)


@pytest.mark.parametrize("dtype,Hq,Hkv,Dk,Dv,latent,room", [k for k in KERNELS if not k[5]])
def test_large_values(dtype, Hq, Hkv, Dk, Dv, latent, room):
    # scores far apart
    c = make_shared([(60, [40, 3, 0, (70,), 900]), (0, [9]), (3, [1, 500])], Hkv, Dk, Dv, 16, dtype, seed=95, room=room)
    c["v"] *= 2.0 ** 86
    run(c, Hq, 1.0)
