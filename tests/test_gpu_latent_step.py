"""A decode step with a latent cache as one captured graph: tables, cache write and
attention one after the other, replayed with new lengths, tokens and free blocks."""
import numpy as np
import pytest
import torch

import paged_kv_cache_263_gb300 as pkv
from oracle import latent as ol
from tests.gpu_util import require_gpu
from tests.test_gpu_latent import SCALE, bf, check, cu_of, f64, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    require_gpu()


@pytest.mark.parametrize("heads", [8, 128])
def test_a_captured_step_replayed(heads):
    rng = np.random.default_rng(heads)
    B, width, nb, cap, reserve = 6, 14, 90, 30, 12
    order = rng.permutation(nb)
    empty = dict(dtype=torch.int32, device="cuda")
    cache = torch.full((nb, 16, 576), float("nan"), dtype=torch.bfloat16, device="cuda")
    tables, lens, new = torch.full((B, width), -1, **empty), torch.zeros(B, **empty), torch.zeros(B, **empty)
    free, cu, total = torch.zeros(reserve, **empty), torch.empty(B + 1, **empty), torch.empty(B, **empty)
    slots, pos = torch.empty(cap, dtype=torch.int64, device="cuda"), torch.empty(cap, **empty)
    totals, down = torch.empty(2, **empty), torch.zeros(cap, 576, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(cap, heads, 576, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(cap, heads, 512, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(pkv.paged_latent_attention_workspace_size(B, cap, heads, width), dtype=torch.uint8, device="cuda")

    def step():
        pkv.kv_build_step_tables(tables, lens, new, free, nb, cu, total, slots, pos, totals)
        pkv.reshape_and_cache_latent(down[:, :512], down[:, 512:], cache, slots)
        pkv.paged_latent_attention(out, q, cache, tables, total, cu_q_lens=cu, scale=SCALE, workspace=ws)
        lens.copy_(total)

    step()                                   # nothing to add yet: every buffer is set up
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    history, at = [np.zeros((0, 576))] * B, 0
    for n in ([9, 1, 0, 16, 3, 1], [1] * 6, [1, 1, 20, 1, 1, 0], [1] * 6, [4] * 6, [0, 1, 0, 1, 0, 1], [5] * 6, [1] * 6):
        rows, c = sum(n), cu_of(n)
        new.copy_(i32(n))
        free.copy_(i32(order[(at + np.arange(reserve)) % nb]))
        down.copy_(bf(rng.normal(size=(cap, 576))))
        q.copy_(bf(rng.normal(size=(cap, heads, 576))))
        out.fill_(float("nan"))
        graph.replay()
        assert pkv.kv_last_device_status() == 0
        at += int(totals[1])
        x, qs, got = f64(down), f64(q), f64(out)
        history = [np.concatenate([history[s], x[c[s]:c[s + 1]]]) for s in range(B)]
        assert lens.tolist() == [len(h) for h in history] and totals.tolist()[0] == rows
        for s in range(B):
            if n[s]:
                h = history[s]
                ref, tol = ol.attend(qs[c[s]:c[s + 1]], h, h[:, :512], SCALE, np.arange(len(h) - n[s] + 1, len(h) + 1))
                check(got[c[s]:c[s + 1]], ref, tol)
        assert np.isnan(got[rows:]).all()
    assert at <= nb
