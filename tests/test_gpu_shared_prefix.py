"""Parity of attention over shared prefixes with its fp64 reference.  The tolerances
are the reference's own bounds, per output element (see oracle/shared_prefix.py)."""
import numpy as np
import pytest
import torch

import paged_kv_cache_263_gb300 as pkv
from oracle import shared_prefix as osp
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu
D, BS = 128, 16


@pytest.fixture(scope="module", autouse=True)
def gpu():
    require_gpu()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


class Batch:
    """A batch with its caches: sizes [sequences per group], prefix lengths, tails
    (tokens behind the whole blocks of the prefix), rows a sequence."""

    def __init__(self, sizes, prefix, tails, rows=1, hq=8, hkv=2, fp8=False, seed=0, loose=0, before=0, width=None, spread=1.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.B = B = before + sum(sizes) + loose
        n = np.broadcast_to(rows, (B,)) if np.ndim(rows) else np.full(B, rows)
        self.cu = np.concatenate([[0], np.cumsum(n)])
        self.groups = before + np.concatenate([[0], np.cumsum(sizes)])
        self.prefix = np.asarray(prefix)
        held = np.zeros(B, int)
        for i, s in enumerate(sizes):
            held[self.groups[i]:self.groups[i] + s] = prefix[i] // BS
        self.lens = held * BS + np.asarray(tails)
        self.width = width or max(1, int((-(-self.lens // BS)).max()))
        need = [max(0, -(-int(x) // BS) - int(h)) for x, h in zip(self.lens, held)]
        shared = [int(p) // BS for p in prefix]
        self.nb = nb = sum(need) + sum(shared) + 3
        ids = rng.permutation(nb - 1)
        # what a row must not read holds a block of NaN or an id outside the pool
        self.poison = nb - 1
        self.tables = np.where(rng.random((B, self.width)) < 0.5, -7, self.poison)
        at = sum(shared)
        for i, s in enumerate(sizes):
            p0 = sum(shared[:i])
            if s:
                self.tables[self.groups[i], :shared[i]] = ids[p0:p0 + shared[i]]
        for s in range(B):
            self.tables[s, held[s]:held[s] + need[s]] = ids[at:at + need[s]]
            at += need[s]
        self.k, self.v = (torch.randn(nb, hkv, BS, D, generator=g, device="cuda") for _ in range(2))
        self.q = (spread * torch.randn(int(self.cu[-1]), hq, D, generator=g, device="cuda")).to(torch.bfloat16)
        self.fp8, self.hq, self.hkv, self.rows = fp8, hq, hkv, n
        self.ks = self.vs = None
        if fp8:
            self.ks, self.vs = (torch.rand(hkv, generator=g, device="cuda") * 0.02 + 0.01 for _ in range(2))
            self.k, self.v = ((x / s[:, None, None]).clamp(-448, 448).to(torch.float8_e4m3fn) for x, s in
                              ((self.k, self.ks), (self.v, self.vs)))
            self.k64, self.v64 = f64(self.k) * f64(self.ks)[:, None, None], f64(self.v) * f64(self.vs)[:, None, None]
            self.k, self.v = self.k.view(torch.uint8), self.v.view(torch.uint8)
            nan = 0x7F
        else:
            self.k, self.v = self.k.to(torch.bfloat16), self.v.to(torch.bfloat16)
            self.k64, self.v64 = f64(self.k), f64(self.v)
            nan = float("nan")
        # keys past every context, and the block that nobody owns, are not numbers
        for x in (self.k, self.v):
            x[self.poison] = nan
            for s in range(B):
                if self.lens[s] % BS and need[s] and self.lens[s] > held[s] * BS:
                    x[self.tables[s, (self.lens[s] - 1) // BS], :, self.lens[s] % BS:] = nan
        self.scale = D ** -0.5

    def call(self, out=None, pad=0, **kw):
        """pad: entries without rows or context behind the batch."""
        if out is None:
            out = torch.full(self.q.shape, 77.0, dtype=torch.bfloat16, device="cuda")
        cu, lens = np.append(self.cu, [self.cu[-1]] * pad), np.append(self.lens, [0] * pad)
        tables = np.concatenate([self.tables.reshape(self.B, self.width), np.full((pad, self.width), -7)])
        args = dict(cu_q_lens=None if pad == 0 and (self.rows == 1).all() else i32(cu), max_q_len=int(max(self.rows.max(), 1)),
                    scale=self.scale, k_scale=self.ks, v_scale=self.vs, max_prefix_len=int(max([0, *self.prefix])),
                    max_tail_len=self.width * BS)
        args.update(kw)
        pkv.paged_attention_shared_prefix(out, self.q, self.k, self.v, i32(tables), i32(lens), i32(self.groups),
                                          i32(self.prefix), **args)
        return out

    def reference(self, **kw):
        return osp.shared(f64(self.q), self.k64, self.v64, self.tables, self.lens, self.groups, self.prefix, self.scale,
                          cu=self.cu, fp8=self.fp8, **kw)

    def ways(self, rows=None):
        """Bounds and padding with which the call goes each of its ways."""
        return ways_of(self.B, len(self.q), rows or int(max(self.rows.max(), 1)), len(self.prefix), self.hq, self.hkv,
                       int(max([0, *self.prefix])), self.width * BS, self.fp8)

    def apart(self):
        """Bounds with which a kernel of its own attends the prefixes."""
        return self.ways()[1]

    def check(self, flags=0, got=None, ref=None, **kw):
        exp, tol, f = ref or self.reference()
        assert f == flags
        if got is None and "max_prefix_len" not in kw and "max_tail_len" not in kw:
            for bounds in self.ways(kw.get("max_q_len")).values():
                self.check(flags, ref=(exp, tol, f), **bounds, **kw)
        got = self.call(**kw) if got is None else got
        assert pkv.kv_last_device_status() == (5 if flags else 0)
        assert pkv.kv_last_device_status_flags() == flags
        compare(f64(got), exp, tol)
        return got


def ways_of(B, R, n, groups, hq, hkv, prefix, tail, fp8):
    found = {}
    for pad in (0, 60, 600):
        for t in (tail, 1 << 15, 1 << 18):
            for p in (prefix, 1 << 12, 1 << 14, 1 << 16, 1 << 18):
                sizes = (B + pad, R, n, groups, hq, hkv, max(p, prefix), max(t, tail))
                if pkv.paged_attention_shared_prefix_workspace_size(*sizes) < 1 << 30:
                    found.setdefault(pkv.paged_attention_shared_prefix_way(*sizes, fp8),
                                     dict(max_prefix_len=sizes[6], max_tail_len=sizes[7], **({"pad": pad} if pad else {})))
    return found


def compare(got, exp, tol):
    kept = np.isnan(exp)
    assert (got[kept] == 77.0).all()
    assert np.isfinite(got[~kept]).all()
    off = np.abs(got - exp)[~kept] - tol[~kept]
    assert off.size == 0 or off.max() <= 0, (off.max(), np.abs(got - exp)[~kept].max())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 8), (4, 2), (8, 2), (16, 2), (16, 1), (64, 8)])
def test_head_layouts(hq, hkv, fp8):
    Batch([3, 5], [100, 33], [7, 1, 16, 17, 40, 2, 31, 90], hq=hq, hkv=hkv, fp8=fp8, seed=hq + hkv).check()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("p", [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 144, 255, 640, 1000, 2048, 5000])
def test_prefix_lengths(p, fp8):
    Batch([4], [p], [1, 16, 33, 250], hq=16, hkv=2, fp8=fp8, seed=p).check()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("tail", [1, 2, 15, 16, 17, 64, 65, 333, 1024, 1025, 4100])
def test_tail_lengths(tail, fp8):
    Batch([5, 3], [48, 200], [tail, 5, tail, 1, 16, 40, tail, 9], hq=8, hkv=1, fp8=fp8, seed=tail).check()


@pytest.mark.parametrize("size", [1, 2, 7, 8, 15, 16, 17, 31, 33, 64, 130, 300])
def test_group_sizes(size):
    """Up to several query tiles a group, whole and partly filled."""
    rng = np.random.default_rng(size)
    Batch([size], [300], rng.integers(1, 60, size), hq=16, hkv=2, seed=size).check()


@pytest.mark.parametrize("fp8", [False, True])
def test_many_groups_of_all_sizes(fp8):
    rng = np.random.default_rng(5)
    sizes = [0, 1, 9, 0, 0, 40, 2, 17, 1, 1, 3, 0] + [5] * 40
    n = sum(sizes) + 4
    Batch(sizes, rng.integers(0, 700, len(sizes)), rng.integers(1, 90, n), hq=8, hkv=2, fp8=fp8, loose=3, before=1).check()


@pytest.mark.parametrize("ng", [31, 32, 33, 100, 1025])
def test_numbers_of_groups(ng):
    rng = np.random.default_rng(ng)
    sizes = rng.integers(1, 9, ng)
    sizes[ng // 2] = 0
    Batch(list(sizes), rng.integers(0, 100, ng), rng.integers(1, 20, int(sizes.sum()) + 1), hq=2, hkv=1, loose=1).check()


@pytest.mark.parametrize("rows", [1, 5])
@pytest.mark.parametrize("empty", [31, 32, 33, 64, 1000, 65533])
def test_many_empty_groups(empty, rows):
    """As a graph has them that is captured for many groups: behind the last, between two or in front, and
    sequences of no group behind.  They are not gone through one by one."""
    for sizes, at in (([50], 0), ([20, 30], 1), ([20, 30], 2), ([50], 1)):
        b = Batch(sizes, [130, 70][:len(sizes)], np.random.default_rng(empty).integers(rows, 60, 55), rows=rows, hq=8, hkv=1,
                  loose=5, seed=empty)
        ref = b.reference()
        b.groups = np.insert(b.groups, at, [b.groups[at]] * empty)
        b.prefix = np.insert(b.prefix, at, [100] * empty)
        for bounds in (dict(max_prefix_len=130), dict(max_prefix_len=1 << 14, max_tail_len=64)):
            b.check(ref=ref, **bounds)
    out, put = torch.empty_like(b.q), (i32(b.tables), i32(b.lens), i32(b.groups), i32(b.prefix))
    took = []
    for _ in range(5):
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        pkv.paged_attention_shared_prefix(out, b.q, b.k, b.v, *put, cu_q_lens=i32(b.cu), max_q_len=rows, max_prefix_len=130,
                                          max_tail_len=64)
        end.record()
        torch.cuda.synchronize()
        took.append(start.elapsed_time(end))
    assert min(took) < 1      # ms


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("rows", [2, 3, 4, 8, 20])
@pytest.mark.parametrize("hq,hkv", [(2, 2), (8, 2), (16, 1)])
def test_drafts(rows, hq, hkv, fp8):
    """Several rows a sequence, causal among themselves, all of them behind the prefix."""
    Batch([3, 4], [130, 500], [rows, rows + 1, 40, 17 + rows, 64, 33, 200], rows=rows, hq=hq, hkv=hkv, fp8=fp8, loose=0,
          seed=rows).check()


def test_rows_of_all_lengths():
    """Ragged rows, sequences without any among them."""
    rows = [0, 1, 5, 2, 0, 7, 1, 3]
    Batch([4, 3], [95, 260], [9, 1, 5, 20, 30, 77, 1, 4], rows=rows, hq=8, hkv=2, loose=1).check()
    Batch([4, 3], [95, 260], [9, 1, 5, 20, 30, 77, 1, 4], rows=rows, hq=8, hkv=2, loose=1, fp8=True).check(max_q_len=9)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("rows,hq,hkv", [(1, 8, 2), (3, 16, 2), (5, 16, 1)])
def test_rows_bound_far_above_their_number(rows, hq, hkv, fp8):
    """max_q_len as loose as the number of all rows."""
    tails = np.random.default_rng(rows).integers(rows, 400, 150)
    b = Batch([60, 0, 70], [330, 40, 97], tails, rows=rows, hq=hq, hkv=hkv, fp8=fp8, loose=20, seed=rows)
    b.lens[[5, 70, 149]] = 0
    b.check(cu_q_lens=i32(b.cu), max_q_len=150 * rows, max_prefix_len=330, max_tail_len=b.width * BS)
    b.check(max_q_len=40 * rows) if rows > 1 else None


def test_every_way_is_gone():
    """The batches of the tests above reach whole contexts, prefixes apart, and both joined."""
    for fp8 in (False, True):
        for hq, hkv in ((1, 1), (8, 8), (16, 1), (64, 8)):
            assert set(ways_of(8, 8, 1, 2, hq, hkv, 100, 208, fp8)) == {0, 1}
        for n, hq, hkv in ((20, 8, 2), (3, 16, 1)):
            assert set(ways_of(7, 7 * n, n, 2, hq, hkv, 500, 700, fp8)) == {0, 1, 2}


def test_long_prefix_of_many_parts():
    b = Batch([20], [40000], np.arange(1, 21), hq=8, hkv=1, seed=3)
    b.check()
    b.check(max_prefix_len=65536)
    Batch([1, 20], [40000, 9000], np.arange(1, 22), hq=16, hkv=2, seed=4).check()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hq,hkv,rows", [(8, 4, 1), (32, 2, 1), (16, 4, 4), (16, 4, 3), (16, 2, 5)])
def test_many_items_a_cta(hq, hkv, rows, fp8):
    """Hundreds of sequences and parts: every CTA goes through many items, some of one block."""
    rng = np.random.default_rng(hq + rows)
    n = 330 // rows
    tails = rng.integers(rows, 1100, n)
    tails[::7] = rows
    b = Batch([n // 3, 0, n - n // 3 - 2], [330, 40, 97], tails, rows=rows, hq=hq, hkv=hkv, fp8=fp8, loose=2, seed=rows)
    ref = b.reference()
    for bounds in b.ways().values():
        first = b.check(ref=ref, **bounds).view(torch.int16).clone()
        for _ in range(3):
            assert torch.equal(b.call(**bounds).view(torch.int16), first)


def test_more_parts_than_lanes():
    """A prefix and a tail of more parts than the merge's warp has lanes."""
    b = Batch([12], [30000], [4000, 70000, 3] + [20] * 9, hq=4, hkv=1, seed=12)
    b.check()
    b = Batch([1], [30000], [900], hq=4, hkv=1, seed=13)
    assert 0 in b.ways()
    b.check()


def test_caches_past_four_gigabytes():
    """Blocks at the end of caches of 4.6 GB."""
    b = Batch([4, 3], [600, 90], [20, 30, 400, 5, 7, 9, 11], hq=16, hkv=8)
    ref, nb = b.reference(), 140000
    for name in ("k", "v"):
        small, big = getattr(b, name), torch.empty(nb, 8, BS, D, dtype=torch.bfloat16, device="cuda")
        big[-small.shape[0]:] = small
        setattr(b, name, big)
    b.tables = np.where(b.tables >= 0, b.tables + nb - b.nb, b.tables)
    b.nb = nb
    b.check(ref=ref, max_prefix_len=600)
    b.check(ref=ref, **b.apart())


def test_sharp_scores():
    """Scores spread so far that the running maximum moves often and most weights vanish."""
    Batch([6, 6], [700, 320], [3, 90, 200, 16, 1, 33] * 2, hq=16, hkv=2, spread=30.0).check()


def test_default_bounds():
    b = Batch([3], [77], [20, 9, 1])
    b.check(max_prefix_len=None, max_tail_len=None)
    b.check(got=b.call(cu_q_lens=i32(b.cu), max_q_len=None))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("rows,hq,hkv", [(1, 8, 2), (1, 16, 1), (2, 8, 1), (5, 16, 1), (20, 8, 1), (40, 16, 2)])
def test_without_groups(rows, hq, hkv, fp8):
    """Nothing shared: one part a sequence, written by the only kernel, or several; padded entries."""
    for tails in ([rows, 2 * rows, 40, 41, 130, 250], [rows, 40, 700, 1500, 9000, 41]):
        b = Batch([], [], tails, before=6, rows=rows, hq=hq, hkv=hkv, fp8=fp8, seed=rows)
        b.lens[2] = 0
        b.check(max_tail_len=max(tails))
        b.check()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("rows,hq,hkv", [(1, 8, 2), (2, 8, 1), (3, 16, 2), (9, 8, 1)])
def test_many_padded_entries(rows, hq, hkv, fp8):
    """Every third of 200 sequences without a context: zeros, whichever CTA comes upon it."""
    tails = np.random.default_rng(rows).integers(rows, 300, 200)
    for groups in (([], []), ([50, 60], [40, 100])):
        b = Batch(*groups, tails, before=200 - sum(groups[0]), rows=rows, hq=hq, hkv=hkv, fp8=fp8, seed=rows)
        b.lens[::3] = 0
        b.check()


def test_padded_and_bad_sequences():
    """L = 0 gives zeros; sequences that break a rule are left as they were."""
    b = Batch([4, 4, 3], [100, 64, 33], [5, 6, 7, 8, 20, 21, 22, 23, 40, 41, 42], hq=8, hkv=2)
    b.lens[1] = 0
    b.check()
    for what, value in (("short", 97), ("equal", 96), ("negative", -3), ("wide", 16 * b.width + 1)):
        lens, old = b.lens.copy(), b.lens
        lens[2] = value
        b.lens = lens
        ok = what == "short"           # one key behind the prefix's 96
        b.check(flags=0 if ok else 4)
        b.lens = old
    prefix = b.prefix
    b.prefix = np.array([100, -1, 33])
    b.check(flags=4, max_prefix_len=100)
    b.prefix = prefix
    # bounds that the batch breaks
    b.check(flags=4, max_prefix_len=95, ref=b.reference(max_prefix=95))
    b.check(flags=4, max_tail_len=30, ref=b.reference(max_tail=30))
    groups = b.groups
    for bad in ([0, 4, 8, 12], [-1, 4, 8, 11], [0, 4, 99, 11]):
        b.groups = np.array(bad)
        for bounds in b.ways().values():
            got = b.call(**bounds)
            assert pkv.kv_last_device_status() == 5 and pkv.kv_last_device_status_flags() == 4
            assert np.isfinite(f64(got)).all()
    b.groups = groups
    b.check()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("rows,hq,hkv", [(1, 8, 2), (3, 16, 2), (5, 16, 1)])
def test_padded_groups(rows, hq, hkv, fp8):
    """A group of padded entries reads nothing, whatever its prefix length and table rows hold; one entry that
    is not padded, wherever it is, attends its group's prefix."""
    sizes = [5, 200, 40, 3, 150, 1] if rows > 1 else [5, 1100, 40, 3, 700, 1]
    n = sum(sizes)
    b = Batch(sizes, [130, 500, 77, 90, 260, 400], np.random.default_rng(rows).integers(rows, 90, n), rows=rows, hq=hq, hkv=hkv,
              fp8=fp8, seed=rows)
    lens, tables = b.lens, b.tables
    for alive in ((2, 3), (0, 5), (1,), (4,), ()):
        for kept in ("last", "all", "middle"):
            b.lens, b.tables = np.zeros_like(lens), np.full_like(tables, -1)
            for g in alive:
                a, e = b.groups[g], b.groups[g + 1]
                on = {"last": [e - 1], "all": range(a, e), "middle": [(a + e) // 2]}[kept]
                b.lens[on] = lens[on]
                b.tables[on] = tables[on]
                b.tables[a, :b.prefix[g] // BS] = tables[a, :b.prefix[g] // BS]
            b.check()
    # a group of sequences that break a rule: flagged and left as they were, the others as ever
    # (its prefix may be read, and its blocks be flagged)
    b.lens, b.tables = lens.copy(), tables.copy()
    b.lens[b.groups[1]:b.groups[2]] = 7
    b.tables[b.groups[1]:b.groups[2]] = -1
    exp, tol, f = b.reference()
    assert f == 4
    for bounds in b.ways().values():
        got = b.call(**bounds)
        assert pkv.kv_last_device_status() == 5 and pkv.kv_last_device_status_flags() in (4, 5)
        compare(f64(got), exp, tol)


@pytest.mark.parametrize("n", [700, 1024, 1025, 2100])
def test_bad_groups_in_large_batches(n):
    """Groups outside the batch are flagged, and no length is read for them; the others are as ever."""
    b = Batch([10, n - 10], [130, 500], np.random.default_rng(n).integers(1, 90, n), hq=8, hkv=2, seed=n)
    b.tables[:10, :8], b.tables[10:, :31] = b.tables[0, :8], b.tables[10, :31]
    b.lens[20:] = 0        # (padded entries, so that the walk goes on)
    groups, prefix = b.groups, b.prefix
    far = 2 ** 31 - 1
    for bad in ([0, 10, far, n], [0, 10, -5, far, 20, n], [-far, far, 10, n, n + 1], [0, 10, n, far, -1, -1, n, n + 7]):
        b.groups, b.prefix = np.array(bad), np.full(len(bad) - 1, 130)
        for bounds in b.ways().values():
            got = b.call(**bounds)
            assert pkv.kv_last_device_status() == 5 and pkv.kv_last_device_status_flags() in (4, 5)
            assert np.isfinite(f64(got)).all()
    b.groups, b.prefix = groups, prefix
    b.check()


def test_more_rows_than_announced():
    b = Batch([2, 2], [40, 50], [9, 9, 9, 9], rows=[3, 1, 2, 3], hq=4, hkv=1)
    b.check(flags=4, max_q_len=2, ref=b.reference(max_q=2))


def test_rows_out_of_order():
    """Offsets of rows that go back and forth: flagged, and the rows of a sequence that keeps the rules are right."""
    rows, n = 4, 7
    b = Batch([4, 3], [95, 260], [40, 33, 64, 29, 50, 31, 77], rows=rows, hq=8, hkv=2)
    exp, tol, _ = b.reference()
    back = b.cu.copy()
    back[3] = back[2] - 2          # sequence 2 has -2 rows, sequence 3 six of which two are sequence 1's
    claim = np.array([0, n * rows] * (n // 2 + 1))[:n + 1]
    for cu, kept in ((back, range(0, rows)), (claim, ())):
        for bounds in b.ways(n * rows).values():
            if "pad" in bounds:
                continue
            got = f64(b.call(cu_q_lens=i32(cu), max_q_len=n * rows, **bounds))
            assert pkv.kv_last_device_status() == 5 and pkv.kv_last_device_status_flags() == 4
            for r in kept:
                compare(got[r], exp[r], tol[r])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("rows", [1, 3])
def test_groups_that_claim_the_same_rows(rows, fp8):
    """Offsets of groups that go back and forth, so that 33 groups of 65 have all rows: flagged, and no more is
    done than a batch of so many groups and rows can need."""
    n, ng = 300, 65
    b = Batch([n], [330], np.random.default_rng(rows).integers(rows, 90, n), rows=rows, hq=64, hkv=4, fp8=fp8, seed=rows)
    b.tables[:, :20] = b.tables[0, :20]      # (whichever group a sequence is taken for, its row holds the prefix)
    groups, prefix = b.groups, b.prefix
    b.groups, b.prefix = np.array([0, n] * (ng // 2 + 1)), np.full(ng, 330)
    ways = b.ways()
    assert 1 in ways or rows > 1 and 2 in ways
    for way in (1, 2):
        if way in ways:
            got = b.call(**ways[way])
            assert pkv.kv_last_device_status() == 5 and pkv.kv_last_device_status_flags() == 4
            assert np.isfinite(f64(got)).all()
    b.groups, b.prefix = groups, prefix
    b.check()


def test_blocks_outside_the_pool():
    """Flagged and not read; the other groups' rows are as ever."""
    for where in ("prefix", "tail"):
        b = Batch([3, 3], [200, 150], [20, 30, 40, 50, 60, 70], hq=8, hkv=2)
        exp, tol, _ = b.reference()
        b.tables[0, 3 if where == "prefix" else 13] = b.nb + 5
        for bounds in b.ways().values():
            got = b.call(**bounds)
            assert pkv.kv_last_device_status() == 5 and pkv.kv_last_device_status_flags() == 1
            first = 3 if where == "prefix" else 1
            compare(f64(got)[first:], exp[first:], tol[first:])


@pytest.mark.parametrize("where", [0, 5])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_queries_that_are_not_finite(bad, where):
    """They make their own row of that head NaN, and no other."""
    b = Batch([4, 3], [200, 90], [20, 30, 40, 5, 7, 9, 11], hq=8, hkv=2)
    exp, tol, _ = b.reference()
    b.q[where, 3, 17] = bad
    for bounds in b.ways().values():
        got = f64(b.call(**bounds))
        assert pkv.kv_last_device_status() == 0
        assert np.isnan(got[where, 3]).all()
        got[where, 3] = exp[where, 3]
        compare(got, exp, tol)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("rows", [1, 5])
@pytest.mark.parametrize("groups", [True, False])
def test_scores_that_are_all_minus_infinity(rows, groups, fp8):
    """Their softmax is NaN, in their own row of that head; where one key has another score, it is a softmax as any."""
    b = Batch(*(([4, 3], [200, 90]) if groups else ([], [])), [20, 30, 40, 5, 7, 9, 11], before=0 if groups else 7, rows=rows,
              hq=8, hkv=2, fp8=fp8)
    if fp8:
        b.k[..., 17] = b.k[..., 17] & 0x7F | 1
        b.k64[..., 17] = f64(b.k.view(torch.float8_e4m3fn))[..., 17] * f64(b.ks)[:, None]
    else:
        b.k[..., 17] = b.k[..., 17].abs() + 0.5
        b.k64 = f64(b.k)
    exp, tol, _ = b.reference()
    some = [0, rows + rows // 2, 6 * rows]
    b.q[some, 3, 17] = -float("inf")
    for bounds in b.ways().values():
        got = f64(b.call(**bounds))
        assert pkv.kv_last_device_status() == 0
        assert np.isnan(got[some, 3]).all()
        got[some, 3] = exp[some, 3]
        compare(got, exp, tol)


def test_any_placement_and_workspace_gives_the_same_bits():
    args = dict(sizes=[20, 7], prefix=[3000, 800], tails=np.arange(1, 28) * 11, hq=16, hkv=4)
    b = Batch(**args, width=300)
    need = pkv.paged_attention_shared_prefix_workspace_size(b.B, b.B, 1, 2, 16, 4, 3000, b.width * BS)
    ws = torch.full((need + 512,), 0xFF, dtype=torch.uint8, device="cuda")
    ws = ws[-ws.data_ptr() % 256:][:need]
    assert need > 0
    exact = dict(max_prefix_len=3000)
    first = b.check(workspace=ws, **exact).view(torch.int16).clone()
    ws.fill_(0x7F)
    assert torch.equal(b.call(workspace=ws, **exact).view(torch.int16), first)
    # another order of the blocks
    perm = np.random.default_rng(8).permutation(b.nb)
    inv = torch.tensor(np.argsort(perm), device="cuda")
    b.k, b.v = b.k[inv].contiguous(), b.v[inv].contiguous()
    b.tables = np.where(b.tables >= 0, perm[b.tables.clip(0)], b.tables)
    assert torch.equal(b.call(**exact).view(torch.int16), first)
    assert pkv.kv_last_device_status() == 0


@pytest.mark.parametrize("rows", [1, 3])
def test_one_workspace_for_smaller_batches_and_bounds(rows):
    """Kept from call to call, as a server does: asked for once, for the largest batch and the loosest bounds."""
    most = (256, 256 * rows, rows, 4, 64, 8, 4096, 4096)
    ws = torch.full((pkv.paged_attention_shared_prefix_workspace_size(*most),), 0xFF, dtype=torch.uint8, device="cuda")
    for n in (38, 32, 16, 5, 1):
        b = Batch([n], [4000 - n], np.random.default_rng(n).integers(rows, 500, n), rows=rows, hq=64, hkv=8, width=300, seed=n)
        ref = b.reference()
        for bounds in (dict(max_prefix_len=4096, max_tail_len=4096), dict(max_prefix_len=4000, max_tail_len=500),
                       dict(max_prefix_len=4000, max_tail_len=4096), dict(max_prefix_len=4096, max_tail_len=600)):
            b.check(ref=ref, workspace=ws, **bounds)


@pytest.mark.parametrize("rows,fp8", [(1, False), (1, True), (3, False)])
def test_fewer_parts_where_the_workspace_ends(rows, fp8):
    """Bounds so far above the lengths that parts by them alone would not fit what partial results may take."""
    tails = np.random.default_rng(5).integers(rows, 60, 40)
    tails[7] = 9000
    b = Batch([40], [2000], tails, rows=rows, hq=128, hkv=8, fp8=fp8, seed=5)
    ref = b.reference()
    for tail in (1 << 14, 1 << 18, 1 << 22):
        for prefix in (2000, 1 << 18):
            b.check(ref=ref, max_prefix_len=prefix, max_tail_len=tail)


def test_agrees_with_decode_over_the_whole_context():
    """The same rows through paged_attention_decode with the prefix in every table row."""
    b = Batch([16, 9], [2000, 512], np.arange(1, 26) * 13, hq=16, hkv=2)
    exp, tol, _ = b.reference()
    tables = b.tables.copy()
    for i in range(2):
        a, e, n = b.groups[i], b.groups[i + 1], b.prefix[i] // BS
        tables[a:e, :n] = tables[a, :n]
    out = torch.empty(b.B, 16, D, device="cuda")
    pkv.paged_attention_decode(out, b.q, b.k, b.v, i32(tables), i32(b.lens), b.scale)
    got = b.check()
    assert (np.abs(f64(got) - f64(out)) <= 2 * tol).all()


def test_on_another_stream_and_twice_at_once():
    b, c = Batch([9], [900], np.arange(1, 10) * 30, seed=1), Batch([5, 5], [300, 2000], np.arange(1, 11), seed=2)
    far = b.apart()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(s1):
            x = b.call(**far)
        with torch.cuda.stream(s2):
            y = c.call(**c.apart())
            y2 = c.call()
        z = b.call(stream=s2, out=torch.full(b.q.shape, 77.0, dtype=torch.bfloat16, device="cuda"), **far)
        torch.cuda.synchronize()
        c.check(got=y2)
        b.check(got=x)
        c.check(got=y)
        b.check(got=z)


@pytest.mark.parametrize("bound", [1024, 20000])
def test_captured_and_replayed_with_other_lengths(bound):
    """One graph, padded to its size, replayed over batches with other groups, prefixes and tails."""
    big = Batch([8, 8, 4], [900, 400, 200], np.arange(1, 21) * 9, hq=8, hkv=2, loose=0)
    tables, lens = i32(big.tables), i32(big.lens)
    groups, prefix, q = i32(big.groups), i32(big.prefix), big.q.clone()
    out = torch.full(q.shape, 77.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(pkv.paged_attention_shared_prefix_workspace_size(20, 20, 1, 3, 8, 2, bound, 256), dtype=torch.uint8,
                     device="cuda")

    def call():
        pkv.paged_attention_shared_prefix(out, q, big.k, big.v, tables, lens, groups, prefix, max_prefix_len=bound,
                                          max_tail_len=256, scale=big.scale, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    full = big.lens
    for cut, sizes in ((0, [8, 8, 4]), (3, [8, 8, 4]), (0, [8, 8, 0])):
        # (at least one key behind the whole blocks of each prefix)
        big.lens = np.maximum(full - cut, np.repeat([897, 401, 193], [8, 8, 4]))
        big.groups = np.concatenate([[0], np.cumsum(sizes)])
        if sizes[2] == 0:
            big.lens[16:] = 0              # padding
        lens.copy_(i32(big.lens))
        groups.copy_(i32(big.groups))
        out.fill_(77.0)
        graph.replay()
        big.check(got=out)
