"""Parity of the latent-attention operators and the step tables with their fp64
reference.  The attention tolerances are the reference's own bounds, per output
element, from the roundings that the kernels make (see oracle/latent.py)."""
import numpy as np
import pytest
import torch

import paged_kv_cache_263_gb300 as pkv
from oracle import latent as ol
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu
SCALE = 192 ** -0.5


@pytest.fixture(scope="module", autouse=True)
def gpu():
    require_gpu()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def bf(x):
    return torch.tensor(np.asarray(x, dtype=np.float32), device="cuda").to(torch.bfloat16)


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def cu_of(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int64)


def check(got, ref, tol, rows=None):
    rows = ~np.isnan(ref) if rows is None else rows
    off = np.abs(got - ref)[rows] - tol[rows]
    assert np.isfinite(got[rows]).all()
    assert off.size == 0 or off.max() <= 0, (off.max(), np.abs(got - ref)[rows].max())


# ----------------------------------------------------------------- step tables
def run_tables(ctx, new, free, nb, width, cap, tables=None, seed=0):
    B = len(ctx)
    rng = np.random.default_rng(seed)
    if tables is None:
        tables = rng.integers(0, nb, (B, width))
    t = i32(tables).reshape(B, width)
    out = [torch.full((B + 1,), -9, dtype=torch.int32, device="cuda"), torch.full((B,), -9, dtype=torch.int32, device="cuda"),
           torch.full((cap,), -9, dtype=torch.int64, device="cuda"), torch.full((cap,), -9, dtype=torch.int32, device="cuda"),
           torch.full((2,), -9, dtype=torch.int32, device="cuda")]
    pkv.kv_build_step_tables(t, i32(ctx), i32(new), i32(free), nb, *out)
    status = pkv.kv_last_device_status()
    flags = pkv.kv_last_device_status_flags()
    exp = ol.step_tables(tables, ctx, new, free, nb, cap)
    assert flags == exp[6] and status == (5 if exp[6] else 0)
    assert np.array_equal(t.cpu().numpy(), exp[0])
    for got, e in zip(out, exp[1:6]):
        assert np.array_equal(got.cpu().numpy(), np.asarray(e))
    return t, out


@pytest.mark.parametrize("B,ctx_hi,new_hi", [(1, 40, 1), (1, 0, 0), (5, 33, 50), (64, 4096, 1), (1023, 100, 3),
                                             (2048, 60, 20), (2049, 60, 20), (5000, 300, 17)])
def test_step_tables(B, ctx_hi, new_hi):
    rng = np.random.default_rng(B)
    ctx, new = rng.integers(0, ctx_hi + 1, B), rng.integers(0, new_hi + 1, B)
    need = int(sum(-(-int(c + n) // 16) - -(-int(c) // 16) for c, n in zip(ctx, new)))
    nb = 6000
    run_tables(ctx, new, rng.integers(0, nb, need + B % 3), nb, -(-(ctx_hi + new_hi) // 16) or 1, int(new.sum()) + B % 4)


@pytest.mark.parametrize("B", [6, 4100])
@pytest.mark.parametrize("what", ["blocks", "rows", "lengths", "ids", "all"])
def test_step_tables_refusals(B, what):
    rng = np.random.default_rng(7)
    ctx, new = rng.integers(0, 60, B), rng.integers(0, 40, B)
    need = int(sum(-(-int(c + n) // 16) - -(-int(c) // 16) for c, n in zip(ctx, new)))
    nb, width, cap = 500, 8, int(new.sum()) + 5
    free = rng.integers(0, nb, need)
    if what in ("blocks", "all"):
        free = free[:need // 2]
    if what in ("rows", "all"):
        cap = int(new.sum() * 0.7)
    if what in ("lengths", "all"):
        ctx[1], new[2], ctx[B - 1], new[3], ctx[3] = -5, -1, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1
        cap = min(cap, 300000)
    if what in ("ids", "all"):
        free = free.copy()
        free[::3] = nb + 7
        free[1::5] = -2
    run_tables(ctx, new, free, nb, width, cap)


def test_step_tables_without_rows_or_sequences():
    run_tables([3, 16], [0, 0], [4], 9, 2, 0)
    run_tables([3, 16], [0, 0], [], 9, 2, 5)
    z = torch.zeros
    cu, totals = torch.full((1,), 5, dtype=torch.int32, device="cuda"), torch.full((2,), 5, dtype=torch.int32, device="cuda")
    slots = z(3, dtype=torch.int64, device="cuda")
    empty = z(0, dtype=torch.int32, device="cuda")
    pkv.kv_build_step_tables(z((0, 4), dtype=torch.int32, device="cuda"), empty, empty, empty, 8, cu, empty.clone(),
                             slots, i32([7, 7, 7]), totals)
    assert pkv.kv_last_device_status() == 0
    assert cu.tolist() == [0] and totals.tolist() == [0, 0] and slots.tolist() == [-1] * 3


# ----------------------------------------------------------------- cache write
@pytest.mark.parametrize("T,pad", [(1, 0), (3, 2), (64, 0), (333, 7), (5000, 40)])
def test_latent_write(T, pad):
    g = torch.Generator(device="cuda").manual_seed(T)
    nb = -(-T // 16) + 2
    wide = torch.randn(T + pad, 704, generator=g, device="cuda").to(torch.bfloat16)
    lat, rope = wide[:, 8:520], wide[:, 600:664]
    cache = torch.full((nb, 16, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    slots = torch.full((T + pad,), -1, dtype=torch.int64, device="cuda")
    slots[:T] = torch.randperm(nb * 16, generator=g, device="cuda")[:T]
    if pad:
        slots = torch.cat([slots[T:], slots[:T]])      # the padding first
    exp = cache.clone().view(-1, 576)
    real = slots >= 0
    exp[slots[real]] = torch.cat([lat, rope], dim=1)[real]
    with pytest.raises(ValueError):
        pkv.reshape_and_cache_latent(lat.t(), rope, cache, slots)
    pkv.reshape_and_cache_latent(lat, rope, cache, slots)
    assert pkv.kv_last_device_status() == 0
    assert torch.equal(cache.view(-1, 576).view(torch.int16), exp.view(torch.int16))
    # one row to every slot, and a slot outside the pool
    slots[0] = nb * 16
    pkv.reshape_and_cache_latent(lat[:1].expand(T + pad, -1), rope, cache, slots)
    assert pkv.kv_last_device_status() == 5 and pkv.kv_last_device_status_flags() == 2
    exp[slots[1:][slots[1:] >= 0], :512] = lat[0]
    if pad or T == 1:
        assert torch.equal(cache.view(-1, 576)[:, :512], exp[:, :512])


# ----------------------------------------------------------------- absorbed form
class Paged:
    """Ragged sequences in a poisoned cache: every slot that no key fills is NaN,
    and every table entry that no key needs is out of range."""

    def __init__(self, heads, lens, rows, seed=0, extra_rows=0, k_std=1.0, v_mean=0.0, first_block=0, spare=3):
        rng = np.random.default_rng(seed)
        self.lens, self.rows, self.heads = list(lens), list(rows), heads
        blocks = [-(-x // 16) for x in lens]
        self.width = max(1, max(blocks)) + 1
        nb = first_block + sum(blocks) + spare
        order = first_block + rng.permutation(sum(blocks) + spare)
        self.tables = rng.choice([-1, nb, 2 ** 31 - 1], (len(lens), self.width))
        self.cache = torch.full((nb, 16, 576), float("nan"), dtype=torch.bfloat16, device="cuda")
        at = 0
        self.small = np.full((sum(blocks) + spare, 16, 576), np.nan)   # the blocks from first_block on
        for s, n in enumerate(lens):
            self.tables[s, :blocks[s]] = order[at:at + blocks[s]]
            at += blocks[s]
            x = rng.normal(size=(n, 576)) * k_std
            x[:, :512] += v_mean
            t = np.arange(n)
            self.small[self.tables[s, t // 16] - first_block, t % 16] = x
        self.cache[first_block:] = bf(self.small)
        self.small = f64(self.cache[first_block:])
        self.first_block = first_block
        self.cu = cu_of(rows)
        self.q = bf(rng.normal(size=(int(self.cu[-1]) + extra_rows, heads, 576)))
        self.out = torch.full((self.q.shape[0], heads, 512), float("nan"), dtype=torch.bfloat16, device="cuda")

    def args(self, decode=False):
        return dict(out=self.out, q=self.q, cache=self.cache, block_tables=i32(self.tables),
                    context_lens=i32(self.lens), cu_q_lens=None if decode else i32(self.cu), scale=SCALE)

    def run(self, decode=False, **kw):
        self.out.fill_(float("nan"))
        pkv.paged_latent_attention(**{**self.args(decode), **kw})
        return f64(self.out)

    def expected(self, scale=SCALE):
        return ol.absorbed(f64(self.q), self.small, self.tables - self.first_block, self.lens, self.cu, scale)


LENGTHS = [1, 2, 15, 16, 17, 63, 64, 65, 100, 127, 128, 129, 200, 255, 257, 400]


@pytest.mark.parametrize("heads", [1, 3, 8, 12, 32, 64, 65, 96, 127, 128])
def test_absorbed_decode(heads):
    w = Paged(heads, LENGTHS, [1] * len(LENGTHS), seed=heads)
    got = w.run(decode=True)
    assert pkv.kv_last_device_status() == 0
    check(got, *w.expected())
    # the same through the ragged form, and again: the same bits
    assert np.array_equal(w.run(), got) and np.array_equal(w.run(decode=True), got)


@pytest.mark.parametrize("heads,lens,rows", [
    (32, [40, 300, 77, 4], [4, 4, 4, 4]), (8, [70, 500, 33], [70, 3, 1]), (20, [130, 64, 65], [7, 64, 1]),
    (64, [5, 190], [5, 3]), (128, [90, 9, 300], [2, 9, 1]), (1, [300, 129], [300, 128]), (40, [100], [3]),
    (96, [66, 2], [3, 2])])
def test_absorbed_rows(heads, lens, rows):
    w = Paged(heads, lens, rows, seed=heads + len(lens))
    got = w.run()
    assert pkv.kv_last_device_status() == 0
    check(got, *w.expected())


@pytest.mark.parametrize("heads,lens,rows", [(8, [20000], [1]), (128, [9000], [1]), (16, [3, 7000, 64, 2500], [1, 3, 2, 1]),
                                             (64, [5000, 5001], [2, 1])])
def test_absorbed_long(heads, lens, rows):
    w = Paged(heads, lens, rows, seed=5, v_mean=0.1)
    got = w.run()
    assert pkv.kv_last_device_status() == 0
    check(got, *w.expected())


def test_absorbed_many_sequences():
    rng = np.random.default_rng(11)
    lens = rng.integers(1, 90, 700).tolist()
    rows = [min(int(n), int(r)) for n, r in zip(lens, rng.integers(0, 3, 700))]
    w = Paged(4, lens, rows, seed=12)
    got = w.run()
    assert pkv.kv_last_device_status() == 0
    check(got, *w.expected())


def test_absorbed_sharp_and_flat_scores():
    for k_std in (0.0, 0.02, 6.0):
        w = Paged(16, [1, 50, 333], [1, 2, 1], seed=3, k_std=k_std, v_mean=1.0)
        check(w.run(), *w.expected())


def test_absorbed_scales():
    w = Paged(16, [150], [2], seed=4)
    for scale in (1e-30, 0.01, 1.0):
        check(w.run(scale=scale), *w.expected(scale))


def test_absorbed_growing_scores():
    """Each block's scores exceed the one before by far: the running maximum moves in every tile."""
    w = Paged(8, [700], [1], seed=9)
    x = w.small[w.tables[0, :44]].reshape(-1, 576)[:700]
    q = f64(w.q)[0]
    x += np.linspace(0, 40, 700)[:, None] * q.sum(0)[None, :] / (q.sum(0) ** 2).sum() / SCALE
    t = np.arange(700)
    w.small[w.tables[0, t // 16], t % 16] = x
    w.cache.copy_(bf(w.small))
    w.small = f64(w.cache)
    check(w.run(), *w.expected())


# rows x heads at most 64 an average sequence: another kernel than for more
@pytest.mark.parametrize("heads,lens,rows", [
    (1, [300, 70, 129], [64, 60, 65]), (5, [100, 90, 13, 64], [12, 13, 12, 13]), (33, [100, 64, 40, 7], [1, 1, 1, 4]),
    (17, [500, 65, 2], [3, 5, 2]), (64, [700, 64, 1], [1, 1, 1]), (8, [900, 10, 9, 8, 7, 6], [40, 1, 1, 1, 1, 1]),
    (8, [30000, 5], [9, 1]), (2, [64, 65, 0, 1], [33, 31, 1, 1]), (49, [3000], [1])])
def test_absorbed_units_of_64_rows(heads, lens, rows):
    assert sum(rows) * heads <= 64 * len(rows)
    w = Paged(heads, lens, rows, seed=heads, extra_rows=2)
    got = w.run()
    assert pkv.kv_last_device_status() == 0
    check(got, *w.expected())
    assert np.isnan(got[int(w.cu[-1]):]).all()
    assert np.array_equal(w.run(), got, equal_nan=True)


@pytest.mark.parametrize("heads,rows", [(8, 1), (64, 1), (4, 3), (128, 1), (16, 20)])
@pytest.mark.parametrize("top", [200, 3000])
def test_absorbed_scores_that_keep_growing(heads, rows, top):
    """One head's scores grow past any reference tile after tile; the others' do not."""
    w = Paged(heads, [1000], [rows], seed=heads)
    x = w.small[w.tables[0, :63]].reshape(-1, 576)[:1000]
    q = f64(w.q)[-1, heads // 2]
    x += np.linspace(0, top, 1000)[:, None] * q[None, :] / (q ** 2).sum() / SCALE
    t = np.arange(1000)
    w.small[w.tables[0, t // 16], t % 16] = x
    w.cache.copy_(bf(w.small))
    w.small = f64(w.cache)
    check(w.run(), *w.expected())
    assert pkv.kv_last_device_status() == 0


def test_absorbed_padded_batch():
    """Entries without keys give zeros, entries without rows nothing, and rows of no sequence stay as they were."""
    w = Paged(12, [0, 30, 0, 17, 5], [1, 2, 0, 0, 1], seed=6, extra_rows=3)
    got = w.run()
    assert pkv.kv_last_device_status() == 0
    ref, tol = w.expected()
    assert (got[0] == 0).all() and np.isnan(got[4:]).all()
    check(got, ref, tol)


def test_absorbed_bad_lengths_leave_the_others():
    w = Paged(8, [30, 20, 64, 40], [1, 1, 2, 1], seed=8)
    ref, tol = w.expected()
    for bad in ([30, -1, 64, 40], [30, 20, 1, 40], [30, 20, 64, w.width * 16 + 1]):
        w.lens = bad
        got = w.run()
        assert pkv.kv_last_device_status() == 5 and pkv.kv_last_device_status_flags() == 4
        ok = [i for i in range(4) if bad[i] == [30, 20, 64, 40][i]]
        for i in range(4):
            a, b = w.cu[i], w.cu[i + 1]
            if i in ok:
                check(got[a:b], ref[a:b], tol[a:b])
            else:
                assert np.isnan(got[a:b]).all()
    # rows past the query tensor
    w.lens = [30, 20, 64, 40]
    cu = i32([0, 1, 2, 4, 6])
    got = w.run(cu_q_lens=cu)
    assert pkv.kv_last_device_status() == 5 and pkv.kv_last_device_status_flags() == 4
    check(got[:4], ref[:4], tol[:4])
    assert np.isnan(got[4:]).all()


def test_absorbed_bad_blocks_leave_the_others():
    w = Paged(8, [300, 200, 64], [1, 1, 1], seed=8)
    ref, tol = w.expected()
    for bad in (-1, w.cache.shape[0], 2 ** 31 - 1):
        for at in (0, 5, 12):
            keep = int(w.tables[1, at])
            w.tables[1, at] = bad
            got = w.run()
            assert pkv.kv_last_device_status() == 5 and pkv.kv_last_device_status_flags() == 1
            check(got[[0, 2]], ref[[0, 2]], tol[[0, 2]])
            w.tables[1, at] = keep
    check(w.run(), ref, tol)


def test_absorbed_placement_does_not_change_bits():
    a = Paged(32, [500, 77], [1, 4], seed=21)
    got = a.run()
    perm = torch.randperm(a.cache.shape[0], device="cuda")
    moved = torch.empty_like(a.cache)
    moved[perm] = a.cache
    valid = (a.tables >= 0) & (a.tables < a.cache.shape[0])
    tables = np.where(valid, perm.cpu().numpy()[np.where(valid, a.tables, 0)], a.tables)
    assert np.array_equal(a.run(cache=moved, block_tables=i32(tables)), got)


def test_absorbed_far_blocks():
    """Block offsets past 2^32 bytes (and elements past 2^31)."""
    w = Paged(8, [100, 333], [1, 2], seed=13, first_block=(2 ** 31) // (16 * 576) + 5)
    got = w.run()
    assert pkv.kv_last_device_status() == 0
    check(got, *w.expected())


def test_absorbed_on_other_streams_and_in_graphs():
    a, b = Paged(16, [900, 50], [1, 1], seed=1), Paged(128, [40, 2000], [3, 1], seed=2)
    ra, rb = a.run(), b.run()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        assert np.array_equal(a.run(), ra)
    # two captured calls with a workspace each, replayed side by side
    graphs, works = [], [(a, torch.cuda.Stream()), (b, torch.cuda.Stream())]
    for w, _ in works:
        args = w.args()
        need = pkv.paged_latent_attention_workspace_size(len(w.lens), w.q.shape[0], w.heads, w.width)
        args["workspace"] = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pkv.paged_latent_attention(**args)
        graphs.append((g, args))
    for w, _ in works:
        w.out.fill_(float("nan"))
    torch.cuda.synchronize()
    for _ in range(20):
        for (g, _), (_, st) in zip(graphs, works):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(f64(a.out), ra) and np.array_equal(f64(b.out), rb)
    # new lengths in the same graph
    graphs[0][1]["context_lens"].copy_(i32([300, 49]))
    graphs[0][0].replay()
    torch.cuda.synchronize()
    a.lens = [300, 49]
    check(f64(a.out), *a.expected())
    assert pkv.kv_last_device_status() == 0


def test_scratch_of_a_call_on_another_stream():
    """A call without a workspace on a given stream: its scratch is not handed to the
    current stream's next allocation while the call still runs."""
    a, b = Paged(16, [9000, 50], [1, 1], seed=3), Prompt(8, [300] * 40, [300] * 40, seed=4)
    ra, rb = a.run(), b.run()
    side = torch.cuda.Stream()
    args, held = a.args(), (i32(b.cu_q), i32(b.cu_k))
    sizes = [pkv.paged_latent_attention_workspace_size(2, 2, 16, a.width),
             pkv.latent_prefill_attention_workspace_size(40, b.q.shape[0], 8)]
    torch.cuda.synchronize()
    for _ in range(10):
        a.out.fill_(float("nan"))
        b.out.fill_(float("nan"))
        side.wait_stream(torch.cuda.current_stream())
        pkv.paged_latent_attention(**args, stream=side)
        pkv.latent_prefill_attention(b.out, b.q, b.kv, b.rope, *held, scale=SCALE, stream=side)
        junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes]
        torch.cuda.synchronize()
        assert np.array_equal(f64(a.out), ra) and np.array_equal(f64(b.out), rb)
        del junk
    assert pkv.kv_last_device_status() == 0


# ----------------------------------------------------------------- expanded form
class Prompt:
    def __init__(self, heads, nq, nk, seed=0, extra_q=0, extra_k=0, std=1.0):
        rng = np.random.default_rng(seed)
        self.cu_q, self.cu_k, self.heads = cu_of(nq), cu_of(nk), heads
        Rq, Rk = int(self.cu_q[-1]) + extra_q, int(self.cu_k[-1]) + extra_k
        self.q = bf(rng.normal(size=(Rq, heads, 192)) * std)
        kv = rng.normal(size=(Rk, heads, 256))
        rope = rng.normal(size=(Rk, 576))
        # keys of no sequence are NaN
        kv[int(self.cu_k[-1]):] = np.nan
        rope[int(self.cu_k[-1]):] = np.nan
        self.kv, self.rope = bf(kv), bf(rope)[:, 512:]
        self.out = torch.empty(Rq, heads, 128, dtype=torch.bfloat16, device="cuda")

    def run(self, **kw):
        self.out.fill_(float("nan"))
        args = dict(out=self.out, q=self.q, kv=self.kv, k_rope=self.rope, cu_q_lens=i32(self.cu_q),
                    cu_k_lens=i32(self.cu_k), scale=SCALE)
        pkv.latent_prefill_attention(**{**args, **kw})
        return f64(self.out)

    def expected(self, scale=SCALE):
        return ol.expanded(f64(self.q), f64(self.kv), f64(self.rope), self.cu_q, self.cu_k, scale)


@pytest.mark.parametrize("heads,nq,nk", [
    (4, [1, 2, 15, 16, 17, 63, 64, 65], None), (3, [127, 128, 129], None), (2, [255, 256, 257, 300], None),
    (1, [700], None), (5, [1, 40, 130], [1, 90, 500]), (8, [3, 1, 200], [70, 64, 201]), (128, [9], None),
    (16, [128, 1, 1], [128, 700, 1]), (2, [513], [1030]),
    (100, [513, 40, 700, 129], [513, 41, 700, 300])])
def test_expanded(heads, nq, nk):
    w = Prompt(heads, nq, nk or nq, seed=heads)
    got = w.run()
    assert pkv.kv_last_device_status() == 0
    check(got, *w.expected())
    assert np.array_equal(w.run(), got)


def test_expanded_many_sequences():
    rng = np.random.default_rng(31)
    nq = rng.integers(0, 60, 600)
    w = Prompt(2, nq, nq + rng.integers(0, 40, 600), seed=32, extra_q=5, extra_k=9)
    got = w.run()
    assert pkv.kv_last_device_status() == 0
    ref, tol = w.expected()
    check(got, ref, tol)
    assert np.isnan(got[int(w.cu_q[-1]):]).all()


def test_expanded_rows_that_see_nothing():
    w = Prompt(3, [300, 5, 7, 140], [20, 0, 7, 2], seed=33)
    got = w.run()
    assert pkv.kv_last_device_status() == 0
    ref, tol = w.expected()
    check(got, ref, tol)
    assert (got[:280] == 0).all() and (got[300:305] == 0).all()


def test_expanded_without_any_key():
    w = Prompt(3, [5, 2], [0, 0], seed=34)
    assert (w.run() == 0).all() and pkv.kv_last_device_status() == 0


def test_expanded_sharp_scores_and_scales():
    for std, scale in ((8.0, SCALE), (0.0, SCALE), (1.0, 1e-30), (1.0, 1.0)):
        w = Prompt(2, [150], [400], seed=35, std=std)
        check(w.run(scale=scale), *w.expected(scale))


def test_expanded_bad_offsets_leave_the_others():
    w = Prompt(2, [30, 40, 50], [30, 40, 50], seed=36)
    ref, tol = w.expected()
    # keys past the tensor, a negative count, rows past the tensor
    for cu_q, cu_k, ok in (([0, 30, 70, 120], [0, 30, 70, 121], [0, 1]), ([0, 30, 70, 120], [0, 30, 20, 120], [0]),
                           ([0, 30, 70, 121], [0, 30, 70, 120], [0, 1])):
        got = w.run(cu_q_lens=i32(cu_q), cu_k_lens=i32(cu_k))
        assert pkv.kv_last_device_status() == 5 and pkv.kv_last_device_status_flags() == 4
        for i in ok:
            a, b = w.cu_q[i], w.cu_q[i + 1]
            check(got[a:b], ref[a:b], tol[a:b])
    assert np.isnan(w.run(cu_q_lens=i32([0, 30, 70, 121]))[70:]).all()
    assert pkv.kv_last_device_status() == 5


def test_expanded_on_other_streams_and_in_graphs():
    a, b = Prompt(4, [200, 33], [200, 90], seed=1), Prompt(16, [40, 300], [40, 300], seed=2)
    ra, rb = a.run(), b.run()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        assert np.array_equal(a.run(), ra)
    graphs = []
    for w in (a, b):
        need = pkv.latent_prefill_attention_workspace_size(2, w.q.shape[0], w.heads)
        keep = (i32(w.cu_q), i32(w.cu_k), torch.empty(max(need, 1), dtype=torch.uint8, device="cuda"))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pkv.latent_prefill_attention(w.out, w.q, w.kv, w.rope, keep[0], keep[1], scale=SCALE, workspace=keep[2])
        graphs.append((g, keep, torch.cuda.Stream()))
        w.out.fill_(float("nan"))
    torch.cuda.synchronize()
    for _ in range(20):
        for g, _, st in graphs:
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(f64(a.out), ra) and np.array_equal(f64(b.out), rb)
    assert pkv.kv_last_device_status() == 0


# ----------------------------------------------------------------- together
def test_a_server_step_with_a_latent_cache():
    """Prompts through the expanded form, then drafts and single tokens through the
    absorbed one, with tables, slots and lengths that stay on the device; every
    step against attention over the whole history in 64 bits."""
    rng = np.random.default_rng(41)
    H, B, width, nb = 8, 5, 12, 80
    wk, wv = rng.normal(size=(H, 128, 512)) / 22, rng.normal(size=(H, 128, 512)) / 22
    pool = pkv.KVPool(nb, rng.permutation(nb))
    cache = torch.full((nb, 16, 576), float("nan"), dtype=torch.bfloat16, device="cuda")
    tables = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    history = [np.zeros((0, 576))] * B
    for new in ([40, 1, 17, 100, 64], [1, 1, 1, 1, 1], [3, 0, 4, 1, 2], [1, 20, 1, 0, 1]):
        R, cap = sum(new), 240
        reserve = pool.alloc(20)
        out = {k: torch.empty(n, dtype=t, device="cuda") for k, n, t in (
            ("cu", B + 1, torch.int32), ("total", B, torch.int32), ("slots", cap, torch.int64),
            ("pos", cap, torch.int32), ("totals", 2, torch.int32))}
        pkv.kv_build_step_tables(tables, lens, i32(new), i32(reserve), nb, out["cu"], out["total"], out["slots"],
                                 out["pos"], out["totals"])
        down = bf(rng.normal(size=(cap, 576)))       # padded to the step's capacity
        pkv.reshape_and_cache_latent(down[:, :512], down[:, 512:], cache, out["slots"])
        q = bf(rng.normal(size=(cap, H, 192)))
        x, cu = f64(down), cu_of(new)
        first = all(len(h) == 0 for h in history)
        for s in range(B):
            history[s] = np.concatenate([history[s], x[cu[s]:cu[s + 1]]])
        if first:
            kv = bf(np.concatenate([np.einsum("hdl,tl->thd", wk, x[:, :512]), np.einsum("hdl,tl->thd", wv, x[:, :512])], -1))
            got = torch.full((cap, H, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
            pkv.latent_prefill_attention(got, q, kv, down[:, 512:], out["cu"], out["cu"])
            ref, tol = ol.expanded(f64(q), f64(kv), x[:, 512:], cu, cu, SCALE)
        else:
            qa = bf(np.concatenate([np.einsum("rhd,hdl->rhl", f64(q)[..., :128], wk), f64(q)[..., 128:]], -1))
            got = torch.full((cap, H, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
            pkv.paged_latent_attention(got, qa, cache, tables, out["total"], cu_q_lens=out["cu"])
            ref, tol = np.full((cap, H, 512), np.nan), np.zeros((cap, H, 512))
            for s in range(B):
                a, b = cu[s], cu[s + 1]
                if a == b:
                    continue
                h = history[s]
                ref[a:b], tol[a:b] = ol.attend(f64(qa)[a:b], h, h[:, :512], SCALE,
                                               np.arange(len(h) - (b - a) + 1, len(h) + 1))
        assert pkv.kv_last_device_status() == 0
        check(f64(got), ref, tol)
        assert np.isnan(f64(got)[R:]).all()
        lens.copy_(out["total"])
        used = int(out["totals"][1])
        pool.free(reserve[used:][::-1])              # what the step did not take, back in its order
    assert pool.stats()["live"] == sum(-(-len(h) // 16) for h in history)
    assert np.array_equal(lens.cpu().numpy(), [len(h) for h in history])
