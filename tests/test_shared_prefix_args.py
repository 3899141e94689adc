"""Shared-prefix attention, block copies, forks and compaction without a GPU: the
refusals of the C calls and of the binding, and the pool and the prefix cache
against their models.  (The addresses below are never read.)"""
import ctypes
import sys
import sysconfig

import numpy as np
import pytest
import torch

import paged_kv_cache_263_gb300 as pkv
from oracle import shared_prefix as osp
from oracle.allocator import PoolModel
from oracle.prefix_cache import PrefixCacheModel
from paged_kv_cache_263_gb300 import build as pkv_build

A = 1 << 20     # any 256-byte aligned address
OK, INVALID, UNSUPPORTED = 0, 1, 3
BIG = 2 ** 31 - 1


@pytest.fixture(scope="module", autouse=True)
def built():
    pkv_build.build()


def _call(name, base, **change):
    return getattr(pkv.lib(), name)(*dict(base, **change).values())


ATT = dict(out=A, q=2 * A, cu=3 * A, lens=4 * A, B=4, R=8, nq=2, groups=5 * A, prefix=6 * A, G=2, mp=640, mt=4096,
           k=7 * A, v=8 * A, tables=9 * A, mb=300, hq=32, hkv=8, nb=64, scale=0.1, dt=0, ks=None, vs=None, ws=10 * A,
           nbytes=1 << 40, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(B=-1), INVALID), (dict(R=-1), INVALID), (dict(nq=0), INVALID), (dict(G=-1), INVALID), (dict(mp=-1), INVALID),
    (dict(mt=-1), INVALID), (dict(hq=0), INVALID), (dict(hkv=0), INVALID), (dict(nb=0), INVALID), (dict(mb=0), INVALID),
    (dict(hq=30), INVALID), (dict(hq=24), UNSUPPORTED), (dict(hq=256), UNSUPPORTED), (dict(dt=2), UNSUPPORTED),
    (dict(dt=1), INVALID), (dict(dt=1, ks=A), INVALID), (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(cu=None), INVALID),
    (dict(cu=None, R=4), INVALID), (dict(B=65536), INVALID), (dict(G=65536), INVALID), (dict(mb=1 << 28), UNSUPPORTED), (dict(mb=(1 << 27) - 15), UNSUPPORTED),
    (dict(hq=16 * 65535, hkv=65535), UNSUPPORTED), (dict(nb=1 << 27), UNSUPPORTED), (dict(out=None), INVALID), (dict(q=None), INVALID), (dict(lens=None), INVALID),
    (dict(groups=None), INVALID), (dict(prefix=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(tables=None), INVALID), (dict(out=A + 8), INVALID), (dict(q=2 * A + 4), INVALID), (dict(k=7 * A + 8), INVALID),
    (dict(v=8 * A + 2), INVALID), (dict(cu=3 * A + 1), INVALID), (dict(lens=4 * A + 2), INVALID),
    (dict(groups=5 * A + 2), INVALID), (dict(prefix=6 * A + 1), INVALID), (dict(tables=9 * A + 3), INVALID)])
def test_attention_refuses(change, status):
    assert _call("paged_attention_shared_prefix", ATT, **change) == status


@pytest.mark.parametrize("change", [dict(ws=None), dict(ws=10 * A + 128), dict(nbytes=-1), dict(nbytes=0)])
def test_attention_refuses_a_workspace(change):
    need = pkv.paged_attention_shared_prefix_workspace_size(4, 8, 2, 2, 32, 8, 640, 4096)
    assert need > 0
    change = dict(change, nbytes=need - 1) if change.get("nbytes") == -1 else change
    assert _call("paged_attention_shared_prefix", ATT, **change) == INVALID


@pytest.mark.parametrize("fp8", [0, 1])
@pytest.mark.parametrize("nq", [1, 2, 3, 17, 4000])
@pytest.mark.parametrize("mp,mt", [(0, 0), (15, 1), (640, 4096), (BIG, BIG), (BIG, 0), (5, BIG)])
def test_attention_sizes_its_workspace_for_any_bounds(mp, mt, nq, fp8):
    """No bound makes the call ask for more than the size that it was told, or for less than nothing."""
    need = pkv.paged_attention_shared_prefix_workspace_size(4, 4 * nq, nq, 2, 32, 8, mp, mt)
    assert 0 <= need < 1 << 45
    if need:
        st = _call("paged_attention_shared_prefix", ATT, mp=mp, mt=mt, nq=nq, R=4 * nq, dt=fp8, ks=A, vs=A, nbytes=0)
        assert st == INVALID
    assert pkv.paged_attention_shared_prefix_workspace_size(4, 4 * nq, nq, 2, 24, 7, mp, mt) == 0


def test_a_workspace_serves_every_smaller_call():
    """The size grows with every argument, so that the one for the largest batch and bounds can be kept."""
    size = pkv.paged_attention_shared_prefix_workspace_size
    falling = [size(n, n, 1, 1, 64, 8, 4096, 4096) for n in (256, 128, 64, 38, 32, 16, 8, 1)]
    assert falling == sorted(falling, reverse=True) and falling[-1] > 0
    rng = np.random.default_rng(3)
    for _ in range(4000):
        kv, per, rows = rng.choice([1, 2, 8, 16]), rng.choice([1, 2, 4, 8, 16]), rng.choice([1, 1, 2, 4, 7, 30])
        seqs = int(np.exp(rng.uniform(0, 9)))
        heads = [int(kv * per), int(kv)]
        large = [seqs, seqs * int(rows), int(rows), int(rng.integers(0, seqs + 1)), *(int(np.exp(rng.uniform(0, 13))) for _ in range(2))]
        small = [max(1, int(x * rng.choice([1, 1, rng.random()]))) for x in large[:3]] + [
            int(x * rng.choice([1, 1, rng.random()])) for x in large[3:]]
        assert size(*small[:4], *heads, *small[4:]) <= size(*large[:4], *heads, *large[4:]), (small, large, heads)


@pytest.mark.parametrize("sizes,fp8,way", [
    ((4, 4, 1, 1, 8, 2, 256, 64), False, 0), ((64, 64, 1, 1, 64, 8, 32768, 1000), False, 1),
    ((64, 64, 1, 1, 64, 8, 32768, 1000), True, 1), ((52, 364, 7, 1, 16, 2, 29, 11260), False, 2),
    ((152, 608, 4, 2, 32, 4, 38, 210), False, 0), ((6, 6, 1, 0, 8, 2, 4096, 4096), False, 0), ((6, 6, 1, 2, 8, 2, 15, BIG), True, 0),
    ((65535, BIG, BIG, 65535, 16, 1, BIG, BIG), False, None), ((0, 4, 1, 1, 8, 2, 256, 64), False, -1),
    ((4, 4, 0, 1, 8, 2, 256, 64), False, -1), ((4, 4, 1, 1, 9, 2, 256, 64), False, -1), ((4, 4, 1, 1, 8, 2, -1, 64), False, -1),
    ((4, 4, 1, 1, 34, 2, 256, 64), False, -1)])
def test_way(sizes, fp8, way):
    got = pkv.paged_attention_shared_prefix_way(*sizes, fp8)
    assert got == way if way is not None else got in (0, 1, 2)


def test_way_refuses_a_type():
    assert pkv.lib().paged_attention_shared_prefix_way(4, 4, 1, 1, 8, 2, 256, 64, 2) == -1


@pytest.mark.parametrize("fp8", [0, 1])
@pytest.mark.parametrize("hq,hkv,mp,mt", [(64, 8, 20000, 2000), (64, 8, 30000, 9000), (8, 8, 30000, 100), (16, 1, 30000, 16384)])
def test_rows_bound_far_above_their_number(hq, hkv, mp, mt, fp8):
    """max_q_len as loose as the number of all rows is no reason to refuse a batch."""
    # (a prefix and a tail: at least two parts, so that a workspace is asked for)
    assert pkv.paged_attention_shared_prefix_way(4096, 8192, 8192, 64, hq, hkv, mp, mt, fp8) in (1, 2)
    st = _call("paged_attention_shared_prefix", ATT, B=4096, R=8192, nq=8192, G=64, hq=hq, hkv=hkv, mp=mp, mt=mt, mb=2000, nb=4096,
               dt=fp8, ks=A, vs=A, ws=A + 16)
    assert st == INVALID       # (the workspace's alignment)


@pytest.mark.parametrize("change", [dict(B=0), dict(R=0)])
def test_attention_of_nothing(change):
    assert _call("paged_attention_shared_prefix", ATT, **change) == OK


COPY = dict(caches=None, count=2, bytes=4096, nb=64, src=A, dst=2 * A, n=3, stream=None)


@pytest.mark.parametrize("change", [
    dict(count=-1), dict(n=-1), dict(nb=0), dict(bytes=0), dict(bytes=4104), dict(bytes=-16), dict(src=None),
    dict(dst=None), dict(src=A + 2), dict(dst=2 * A + 1), dict(bytes=1 << 62), dict(caches=None),
    dict(caches=(ctypes.c_void_p * 2)(A, None)), dict(caches=(ctypes.c_void_p * 2)(A, 2 * A + 8))])
def test_copy_refuses(change):
    assert _call("kv_copy_blocks", dict(COPY, caches=(ctypes.c_void_p * 2)(A, 2 * A)), **change) == INVALID


def test_copy_of_nothing():
    assert _call("kv_copy_blocks", COPY, n=0) == OK
    assert _call("kv_copy_blocks", COPY, count=0) == OK


FORK = dict(tables=A, mb=4, lens=2 * A, P=8, parents=3 * A, C=8, keep=1, free=4 * A, nfree=8, ctables=5 * A, clens=6 * A,
            src=7 * A, dst=8 * A, taken=9 * A, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(P=-1), INVALID), (dict(C=-1), INVALID), (dict(nfree=-1), INVALID), (dict(mb=0), INVALID),
    (dict(mb=1 << 28), INVALID), (dict(P=16385), UNSUPPORTED), (dict(C=16385), UNSUPPORTED), (dict(tables=None), INVALID),
    (dict(lens=None), INVALID), (dict(parents=None), INVALID), (dict(free=None), INVALID), (dict(ctables=None), INVALID),
    (dict(clens=None), INVALID), (dict(src=None), INVALID), (dict(dst=None), INVALID), (dict(taken=None), INVALID),
    (dict(clens=6 * A + 2), INVALID),
    # overlaps: in place, an output over an input's tail, two outputs
    (dict(ctables=A), INVALID), (dict(ctables=A + 124), INVALID), (dict(clens=2 * A), INVALID), (dict(src=8 * A + 28), INVALID),
    (dict(taken=4 * A + 4), INVALID)])
def test_fork_refuses(change, status):
    assert _call("kv_fork_tables", FORK, **change) == status


REMAP = dict(tables=A, mb=4, lens=2 * A, B=8, src=3 * A, dst=4 * A, n=5, stream=None)


@pytest.mark.parametrize("change", [
    dict(B=-1), dict(n=-1), dict(mb=0), dict(mb=1 << 28), dict(tables=None), dict(lens=None), dict(src=None),
    dict(dst=None), dict(tables=A + 2), dict(src=3 * A + 2), dict(lens=A + 64), dict(src=A - 16), dict(dst=A)])
def test_remap_refuses(change):
    assert _call("kv_remap_tables", REMAP, **change) == INVALID


def test_remap_of_nothing():
    assert _call("kv_remap_tables", REMAP, n=0) == OK
    assert _call("kv_remap_tables", REMAP, B=0) == OK


@pytest.mark.parametrize("name", ["kv_copy_blocks", "kv_fork_tables", "kv_remap_tables", "paged_attention_shared_prefix"])
def test_binding_refuses_cpu_tensors(name):
    t = torch.zeros(4, 4, dtype=torch.int32)
    args = {"kv_copy_blocks": ([t], t[0], t[1]), "kv_fork_tables": (t,) + (t[0],) * 8, "kv_remap_tables": (t, t[0], t[0], t[0]),
            "paged_attention_shared_prefix": (t,) * 8}[name]
    with pytest.raises(ValueError, match="CUDA tensor"):
        getattr(pkv, name)(*args)


DIRECT = {"paged_attention_shared_prefix": ATT, "kv_copy_blocks": dict(COPY, caches=[A, 2 * A], count=None),
          "kv_fork_tables": FORK, "kv_remap_tables": REMAP}
SIZES = dict(B=4, R=8, nq=2, G=2, hq=32, hkv=8, mp=640, mt=4096)


def _direct(name, **change):
    return getattr(pkv._fast(), name)(*[v for k, v in dict(DIRECT[name], **change).items() if k != "count"])


@pytest.mark.parametrize("name,change,status", [
    ("paged_attention_shared_prefix", dict(nq=0), INVALID), ("paged_attention_shared_prefix", dict(hq=24), UNSUPPORTED),
    ("paged_attention_shared_prefix", dict(dt=1), INVALID), ("paged_attention_shared_prefix", dict(scale=-1.0), INVALID),
    ("paged_attention_shared_prefix", dict(scale=float("nan")), INVALID), ("paged_attention_shared_prefix", dict(nbytes=0), INVALID),
    ("paged_attention_shared_prefix", dict(tables=9 * A + 3), INVALID), ("paged_attention_shared_prefix", dict(B=0), OK),
    ("paged_attention_shared_prefix", dict(v=None), INVALID), ("paged_attention_shared_prefix", dict(nb=1 << 27), UNSUPPORTED),
    ("kv_copy_blocks", dict(bytes=4104), INVALID), ("kv_copy_blocks", dict(caches=[A, None]), INVALID),
    ("kv_copy_blocks", dict(caches=[A] * 129 + [A + 8]), INVALID), ("kv_copy_blocks", dict(caches=[]), OK),
    ("kv_copy_blocks", dict(dst=None), INVALID), ("kv_copy_blocks", dict(n=0), OK),
    ("kv_fork_tables", dict(taken=4 * A + 4), INVALID), ("kv_fork_tables", dict(C=16385), UNSUPPORTED),
    ("kv_fork_tables", dict(free=None), INVALID), ("kv_remap_tables", dict(dst=A), INVALID),
    ("kv_remap_tables", dict(lens=A + 64), INVALID), ("kv_remap_tables", dict(B=0), OK)])
def test_direct_entries_refuse_alike(name, change, status):
    assert _direct(name, **change) == status


@pytest.mark.parametrize("name", DIRECT)
def test_direct_entries_check_their_arguments(name):
    values = [v for k, v in DIRECT[name].items() if k != "count"]
    entry = getattr(pkv._fast(), name)
    for wrong in (values[:-1], values + [0], []):
        with pytest.raises(TypeError, match="arguments"):
            entry(*wrong)
    for i, v in enumerate(values):
        with pytest.raises(TypeError):
            entry(*values[:i], "1", *values[i + 1:])
    for key, v in DIRECT[name].items():
        if key in ("B", "R", "mb", "nb", "n", "P", "C", "nfree", "hq"):
            for far in (1 << 31, -(1 << 31) - 1, 1 << 80):
                with pytest.raises(OverflowError):
                    _direct(name, **{key: far})
    with pytest.raises(TypeError):
        pkv._fast().kv_copy_blocks((A, 2 * A), *[v for k, v in COPY.items() if k not in ("caches", "count")])
    with pytest.raises(TypeError):
        pkv._fast().kv_copy_blocks([A, "2"], *[v for k, v in COPY.items() if k not in ("caches", "count")])


@pytest.mark.parametrize("change", [dict(), dict(B=0), dict(nq=17), dict(hq=24, hkv=7), dict(mp=BIG, mt=BIG), dict(G=0), dict(mt=-1)])
def test_direct_size_agrees(change):
    args = list(dict(SIZES, **change).values())
    assert pkv._fast().paged_attention_shared_prefix_workspace_size(*args) == \
        pkv.lib().paged_attention_shared_prefix_workspace_size(*args)


# ------------------------------------------------- without the module of direct entries
@pytest.fixture
def no_module(monkeypatch):
    monkeypatch.setitem(sys.modules, "paged_kv_cache_263_gb300._fastcall", None)     # (its import fails)
    monkeypatch.setattr(pkv, "_fast_module", None)


@pytest.mark.parametrize("name,change,status", [
    ("paged_attention_shared_prefix", dict(nq=0), INVALID), ("paged_attention_shared_prefix", dict(hq=24), UNSUPPORTED),
    ("paged_attention_shared_prefix", dict(nbytes=0), INVALID), ("paged_attention_shared_prefix", dict(B=0), OK),
    ("kv_copy_blocks", dict(bytes=4104), INVALID), ("kv_copy_blocks", dict(caches=[A, None]), INVALID),
    ("kv_copy_blocks", dict(caches=[A] * 129 + [A + 8]), INVALID), ("kv_copy_blocks", dict(caches=[]), OK),
    ("kv_fork_tables", dict(taken=4 * A + 4), INVALID), ("kv_fork_tables", dict(C=16385), UNSUPPORTED),
    ("kv_remap_tables", dict(dst=A), INVALID), ("kv_remap_tables", dict(B=0), OK)])
def test_calls_without_the_module(no_module, name, change, status):
    """It takes Python's headers to build, and is one interpreter's: the calls do without it."""
    assert _direct(name, **change) == status
    assert not hasattr(pkv._fast(), "__file__")


def test_size_without_the_module(no_module):
    assert pkv.paged_attention_shared_prefix_workspace_size(*SIZES.values()) > 0


def test_build_without_python_headers(monkeypatch, tmp_path):
    """The library is complete, and nothing is built again at the next call."""
    monkeypatch.setattr(pkv_build, "FAST", str(tmp_path / "none.so"))
    monkeypatch.setattr(pkv_build.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    monkeypatch.setattr(pkv_build.subprocess, "run", lambda *a, **k: pytest.fail("compiles"))
    assert pkv_build.build() == pkv.library_path
    assert not list(tmp_path.iterdir())


def test_the_module_is_one_interpreters():
    tag = sysconfig.get_config_var("EXT_SUFFIX")
    assert tag.count(".") > 1 and pkv._fast().__file__.endswith(tag)


# ------------------------------------------------------------------ compaction
def _busy_pool(seed, nb):
    rng = np.random.default_rng(seed)
    order = rng.permutation(nb)
    pool, model = pkv.KVPool(nb, order), PoolModel(nb, order)
    held = []
    for _ in range(60):
        n = int(rng.integers(0, max(2, nb // 8)))
        if rng.random() < 0.6 and n <= model.free_blocks:
            ids = pool.alloc(n).tolist()
            assert ids == model.alloc(n)
            held += ids
        elif held:
            some = [held[i] for i in sorted(set(rng.integers(0, len(held), size=n).tolist()))]
            if rng.random() < 0.3:
                pool.share(some)
                model.share(some)
                held += some
            else:
                for b in some:
                    held.remove(b)
                pool.free(some)
                model.free(some)
    return pool, model, held


@pytest.mark.parametrize("seed,nb,most", [(0, 1, None), (1, 40, None), (2, 200, None), (3, 200, 5), (4, 200, 0), (5, 333, 1)])
def test_pool_compaction_matches_the_model(seed, nb, most):
    pool, model, held = _busy_pool(seed, nb)
    want = osp.compact(model.ref, model.free_list(), nb if most is None else most)
    src, dst = pool.compact(most)
    assert (src.tolist(), dst.tolist()) == (want[0], want[1])
    assert [pool.refcount(b) for b in range(nb)] == want[2]
    if most is None:
        live = pool.stats()["live"]
        assert all(r > 0 for r in want[2][:live]) and not any(want[2][live:])
    # what is allocated next, and that the moved references can be dropped
    free = pool.stats()["free"]
    assert pool.alloc(free).tolist() == want[3]
    to = dict(zip(want[0], want[1]))
    pool.free([to.get(b, b) for b in held])
    assert pool.stats()["live"] == free


def test_pool_compaction_refuses():
    pool = pkv.KVPool(4)
    L, n = pkv.lib(), ctypes.c_int32(7)
    a = np.zeros(4, dtype=np.int32)
    p = a.ctypes.data_as(ctypes.c_void_p)
    assert L.kv_pool_compact(None, 4, p, p, ctypes.byref(n)) == INVALID
    assert L.kv_pool_compact(pool._p, -1, p, p, ctypes.byref(n)) == INVALID
    assert L.kv_pool_compact(pool._p, 4, None, p, ctypes.byref(n)) == INVALID
    assert L.kv_pool_compact(pool._p, 4, p, p, None) == INVALID
    assert L.kv_pool_compact(pool._p, 0, None, None, ctypes.byref(n)) == OK and n.value == 0


def test_prefix_cache_follows_a_compaction():
    nb = 64
    order = np.random.default_rng(9).permutation(nb)
    pool, model = pkv.KVPool(nb, order), PrefixCacheModel(PoolModel(nb, order))
    cache = pkv.PrefixCache(pool)
    rng = np.random.default_rng(10)
    prompts = [rng.integers(0, 9000, size=int(n)).tolist() for n in (40, 100, 64, 17, 160)]
    prompts.append(prompts[1][:50] + prompts[2])
    for i, t in enumerate(prompts):
        got = cache.match(t).tolist()
        assert got == model.match(t, 0)
        own = pool.alloc(-(-len(t) // 16) - len(got)).tolist()
        assert own == model.pool.alloc(len(own))
        cache.insert(t, got + own)
        model.insert(t, got + own, 0)
        if i % 2 == 0:
            pool.free(got + own)
            model.pool.free(got + own)
    before = cache.stats()
    src, dst = pool.compact()
    assert len(src) > 3
    cache.remap(src, dst)
    assert cache.stats() == before
    to = dict(zip(src.tolist(), dst.tolist()))
    for t in prompts:
        assert cache.match(t).tolist() == [to.get(b, b) for b in model.match(t, 0)]
    with pytest.raises(pkv.KVError):
        cache.remap([3, 3], [1, 2])
    with pytest.raises(pkv.KVError):
        cache.remap([3, 2], [1, 4])
    for bad in (-1, nb):
        with pytest.raises(pkv.KVError):
            cache.remap([3, 5], [1, bad])
    with pytest.raises(ValueError):
        cache.remap([3], [1, 4])
    assert [cache.match(t).tolist() for t in prompts] == [[to.get(b, b) for b in model.match(t, 0)] for t in prompts]
    # everything can be given back under the new ids
    free = pool.stats()["free"]
    evicted = cache.evict(nb)
    assert pool.stats()["free"] == free + len(evicted)


# ------------------------------------------------------------- the reference itself
def test_reference_joins_prefix_and_tail_like_one_context():
    """The definition in its two parts: log-sum-exp of prefix and tail is the softmax over both."""
    rng = np.random.default_rng(3)
    q, k, v = rng.standard_normal((1, 4, 8)), rng.standard_normal((48, 2, 8)), rng.standard_normal((48, 2, 8))
    out, tol = osp.attend(q, k, v, 0.3, [40])
    assert (tol > 0).all()
    for h in range(4):
        s = 0.3 * (k[:40, h // 2] @ q[0, h])
        parts = []
        for a, b in ((0, 32), (32, 40)):
            m = s[a:b].max()
            e = np.exp(s[a:b] - m)
            parts.append((m, e.sum(), e @ v[a:b, h // 2]))
        m = max(x[0] for x in parts)
        w = [np.exp(x[0] - m) for x in parts]
        o = sum(f * x[2] for f, x in zip(w, parts)) / sum(f * x[1] for f, x in zip(w, parts))
        assert np.abs(o - out[0, h]).max() < 1e-12


def test_reference_forks_by_hand():
    tables = [[5, 6, 7], [1, 2, 3]]
    child = np.full((4, 3), -9)
    out, lens, src, dst, taken, flags = osp.fork(tables, [33, 32], [0, 1, 0, 0], [10, 11, 12], True, child)
    assert out.tolist() == [[5, 6, 7], [1, 2, -9], [5, 6, 10], [5, 6, 11]]
    assert lens.tolist() == [33, 32, 33, 33] and src.tolist() == [-1, -1, 7, 7] and dst.tolist() == [-1, -1, 10, 11]
    assert taken == 2 and flags == 0
    out, lens, src, dst, taken, flags = osp.fork(tables, [33, 32], [0, 5, 0], [10], False, child[:3])
    assert lens.tolist() == [33, 0, 0] and taken == 1 and flags == osp.BAD_LEN | osp.NO_BLOCKS
    assert osp.remap([[4, 9, 9], [9, 4, 4]], [32, 17], [4, 9], [0, 1])[0].tolist() == [[0, 1, 9], [1, 0, 4]]
