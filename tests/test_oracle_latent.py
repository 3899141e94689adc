"""Pins the fp64 reference of the latent operators: both forms of latent
attention agree with attention over explicitly expanded keys and values, and the
step tables with the host's own bookkeeping."""
import numpy as np

import paged_kv_cache_263_gb300 as pkv
from oracle import latent as ol
from paged_kv_cache_263_gb300 import build as pkv_build
from paged_kv_cache_263_gb300.workload import DeviceWorkload


def test_absorbed_and_expanded_forms_agree():
    rng = np.random.default_rng(1)
    H, T, n, scale = 3, 37, 5, 192 ** -0.5
    wk, wv = rng.normal(size=(H, 128, 512)) / 22, rng.normal(size=(H, 128, 512)) / 22
    cache = rng.normal(size=(4, 16, 576))
    table = np.array([[2, 0, 3]])
    q = rng.normal(size=(n, H, 192))
    x = ol.gather(cache, table[0], T)
    # expanded: keys and values per head from the latents
    kv = np.concatenate([np.einsum("hdl,tl->thd", wk, x[:, :512]), np.einsum("hdl,tl->thd", wv, x[:, :512])], axis=-1)
    exp, _ = ol.expanded(q, kv, x[:, 512:], [0, n], [0, T], scale)
    # absorbed: the key expansion goes into the query, the value expansion onto the output
    qa = np.concatenate([np.einsum("rhd,hdl->rhl", q[..., :128], wk), q[..., 128:]], axis=-1)
    lat, _ = ol.absorbed(qa, cache, table, [T], [0, n], scale)
    assert np.abs(np.einsum("rhl,hdl->rhd", lat, wv) - exp).max() < 1e-12
    # and a direct softmax, row by row
    for i in range(n):
        seen = T - n + 1 + i
        for h in range(H):
            s = scale * (kv[:seen, h, :128] @ q[i, h, :128] + x[:seen, 512:] @ q[i, h, 128:])
            p = np.exp(s) / np.exp(s).sum()
            assert np.abs(p @ kv[:seen, h, 128:] - exp[i, h]).max() < 1e-12


def test_rows_that_see_nothing_are_zero():
    rng = np.random.default_rng(2)
    out, tol = ol.expanded(rng.normal(size=(4, 2, 192)), rng.normal(size=(2, 2, 256)), rng.normal(size=(2, 64)),
                           [0, 4], [0, 2], 0.1)
    assert (out[:2] == 0).all() and (tol[:2] == 0).all() and (out[2:] != 0).any()


def test_step_tables_match_the_host_pool():
    """The same lengths put through the block manager by hand give the same tables and slots."""
    pkv_build.build()
    rng = np.random.default_rng(3)
    nb, B, mb = 400, 23, 12
    pool = pkv.KVPool(nb, rng.permutation(nb))
    ctx = rng.integers(0, 90, B)
    new = rng.integers(0, 90, B)
    tables = np.full((B, mb), -1)
    for s in range(B):
        have = -(-int(ctx[s]) // 16)
        tables[s, :have] = pool.alloc(have)
    need = [-(-int(c + n) // 16) - -(-int(c) // 16) for c, n in zip(ctx, new)]
    free = pool.alloc(sum(need) + 3)      # reserved beforehand, a few too many
    got, cu, lens, slots, pos, totals, flags = ol.step_tables(tables, ctx, new, free, nb, int(new.sum()))
    assert flags == 0 and totals == (new.sum(), sum(need))
    at = 0
    for s in range(B):
        have = -(-int(ctx[s]) // 16)
        row = tables[s].copy()
        row[have:have + need[s]] = free[at:at + need[s]]
        at += need[s]
        assert (row == got[s]).all()
        assert (slots[cu[s]:cu[s + 1]] == DeviceWorkload._slots(row, int(ctx[s]), int(ctx[s] + new[s]))).all()
        assert (pos[cu[s]:cu[s + 1]] == np.arange(ctx[s], ctx[s] + new[s])).all()
    assert (lens == ctx + new).all()


def test_step_tables_refusals():
    t = np.full((5, 2), 7)
    free = [10, 11, 12]
    # too long for the table, negative, blocks short, then one that needs none, then rows short
    _, cu, lens, slots, _, totals, flags = ol.step_tables(t, [20, 3, 0, 5, 16], [13, -1, 64 - 32, 2, 16], free[:1], 20,
                                                          40)
    assert cu.tolist() == [0, 0, 0, 0, 2, 2] and lens.tolist() == [20, 3, 0, 7, 16]
    assert totals == (2, 0) and flags == 4 | 16 and (slots[2:] == -1).all()
