"""Block copies, forks and table rewriting against their models, exactly."""
import sys

import numpy as np
import pytest
import torch

import paged_kv_cache_263_gb300 as pkv
from oracle import shared_prefix as osp
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu
BS = 16


@pytest.fixture(scope="module", autouse=True)
def gpu():
    require_gpu()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def status(flags=0):
    assert pkv.kv_last_device_status() == (5 if flags else 0)
    assert pkv.kv_last_device_status_flags() == flags


# ---------------------------------------------------------------------- copies
@pytest.mark.parametrize("shape,dtype", [((1, 16, 128), torch.uint8), ((2, 16, 128), torch.bfloat16),
                                         ((8, 16, 128), torch.bfloat16), ((16, 576), torch.bfloat16), ((8,), torch.bfloat16),
                                         ((3, 16, 128), torch.float8_e4m3fn), ((5000,), torch.float32)])
@pytest.mark.parametrize("caches,n", [(1, 1), (2, 7), (5, 130), (160, 3)])
def test_copies(shape, dtype, caches, n):
    rng = np.random.default_rng(n)
    nb = 2 * n + 3
    pool = torch.randint(0, 256, (caches, nb, int(np.prod(shape)) * dtype.itemsize), dtype=torch.uint8, device="cuda")
    ids = rng.permutation(nb)
    src, dst = rng.choice(ids[:n + 1], n), ids[n + 1:2 * n + 1]
    exp = pool.clone()
    exp[:, torch.tensor(dst, device="cuda")] = pool[:, torch.tensor(src, device="cuda")]
    pkv.kv_copy_blocks([x.view(dtype).view(nb, *shape) for x in pool], i32(src), i32(dst))
    status()
    assert torch.equal(pool, exp)


def test_copies_that_are_skipped():
    pool = torch.randn(9, 4, 16, 128, device="cuda").to(torch.bfloat16)
    exp = pool.clone()
    exp[3] = pool[1]
    pkv.kv_copy_blocks([pool], i32([-1, 1, 5, -3]), i32([-1, 3, 5, -8]))
    status()
    assert torch.equal(pool, exp)
    pkv.kv_copy_blocks([pool], i32([1, 9, -1, 2, 2]), i32([4, 2, 2, 9, -2]))
    exp[4] = pool[1]
    status(1)
    assert torch.equal(pool, exp)
    pkv.kv_copy_blocks([], i32([1]), i32([2]))
    pkv.kv_copy_blocks([pool], i32([]), i32([]))
    status()
    assert torch.equal(pool, exp)


def test_copies_refused():
    pool = torch.zeros(9, 4, 16, 128, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        pkv.kv_copy_blocks([pool, pool[:8]], i32([1]), i32([2]))
    with pytest.raises(ValueError):
        pkv.kv_copy_blocks([pool, pool.float()], i32([1]), i32([2]))
    with pytest.raises(ValueError):
        pkv.kv_copy_blocks([pool.transpose(1, 2)], i32([1]), i32([2]))
    with pytest.raises(ValueError):
        pkv.kv_copy_blocks([pool], i32([1]), i32([2, 3]))
    with pytest.raises(pkv.KVError):
        pkv.kv_copy_blocks([torch.zeros(4, 3, device="cuda")], i32([1]), i32([2]))


def test_copies_past_four_gigabytes():
    """A cache larger than 2^32 bytes: ids near its end."""
    nb = 140000
    pool = torch.empty(nb, 8, 16, 128, dtype=torch.bfloat16, device="cuda")
    pool[nb - 2:] = 3.0
    pool[0] = 5.0
    pool[70000] = 6.0
    pkv.kv_copy_blocks([pool], i32([nb - 1, 0, 70000]), i32([1, nb - 2, 139000]))
    status()
    assert (pool[1] == 3).all() and (pool[nb - 2] == 5).all() and (pool[139000] == 6).all() and (pool[nb - 1] == 3).all()


# ----------------------------------------------------------------------- forks
def run_fork(tables, lens, parents, free, keep, seed=0):
    rng = np.random.default_rng(seed)
    C, width = len(parents), tables.shape[1]
    child = rng.integers(-50, 0, (C, width))
    got = [i32(child).reshape(C, width)] + [torch.full((C,), -9, dtype=torch.int32, device="cuda") for _ in range(3)]
    taken = torch.full((1,), -9, dtype=torch.int32, device="cuda")
    pkv.kv_fork_tables(i32(tables).reshape(len(lens), width), i32(lens), i32(parents), i32(free), *got, taken,
                       first_keeps=keep)
    exp = osp.fork(tables, lens, parents, free, keep, child)
    status(exp[5])
    for a, b in zip(got, exp[:4]):
        assert np.array_equal(a.cpu().numpy(), b)
    assert taken.item() == exp[4]
    return got, taken


@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("P,C,width", [(1, 1, 1), (1, 16, 64), (4, 3, 7), (300, 513, 20), (1000, 1025, 33), (16384, 16384, 2),
                                       (5, 0, 3)])
def test_forks(P, C, width, keep):
    rng = np.random.default_rng(P + C)
    lens = rng.integers(0, width * BS + 1, P)
    run_fork(rng.integers(0, 1 << 30, (P, width)), lens, rng.integers(0, P, C), rng.integers(0, 1 << 30, C + 1), keep)


@pytest.mark.parametrize("keep", [False, True])
def test_forks_refused(keep):
    rng = np.random.default_rng(1)
    lens = rng.integers(0, 160, 40)
    lens[[3, 5]] = -1, 161
    parents = rng.integers(0, 40, 90)
    parents[[0, 7, 50, 51, 52]] = 40, -1, 3, 5, 2 ** 31 - 1
    run_fork(rng.integers(0, 999, (40, 10)), lens, parents, rng.integers(0, 999, 90), keep)
    run_fork(rng.integers(0, 999, (40, 10)), lens, parents, rng.integers(0, 999, 20), keep)
    run_fork(rng.integers(0, 999, (40, 10)), lens, parents, [], keep)


# ------------------------------------------------------------- table rewriting
def run_remap(tables, lens, src, dst):
    t = i32(tables).reshape(tables.shape)
    pkv.kv_remap_tables(t, i32(lens), i32(src), i32(dst))
    exp, flags = osp.remap(tables, lens, src, dst)
    status(flags)
    assert np.array_equal(t.cpu().numpy(), exp)


@pytest.mark.parametrize("B,width,n,ids", [(1, 1, 1, 2), (3, 5, 2, 20), (16, 256, 9, 4000), (100, 33, 777, 3000),
                                           (700, 64, 5000, 9000), (64, 2048, 8192, 70000), (9, 100, 40000, 90000)])
def test_remap(B, width, n, ids):
    rng = np.random.default_rng(n)
    lens = rng.integers(0, width * BS + 1, B)
    src = np.sort(rng.choice(ids, n, replace=False))
    run_remap(rng.integers(-1, ids, (B, width)), lens, src, rng.integers(0, ids, n))


def test_remap_of_bad_rows():
    rng = np.random.default_rng(4)
    lens = rng.integers(0, 81, 30)
    lens[[0, 4, 29]] = -1, 81, 2 ** 31 - 1
    run_remap(rng.integers(0, 60, (30, 5)), lens, np.arange(20, 60), np.arange(40))
    run_remap(rng.integers(0, 60, (30, 5)), lens, [2 ** 31 - 1], [0])


def test_remap_with_ids_in_both_lists():
    """A chain 1 -> 2 -> 3 moves each entry once."""
    run_remap(np.array([[1, 2, 3, 4], [4, 3, 2, 1]]), [64, 49], [1, 2, 3], [2, 3, 9])


def test_calls_without_the_module_of_direct_entries(monkeypatch):
    """As where Python's headers were missing: the same calls through ctypes."""
    monkeypatch.setitem(sys.modules, "paged_kv_cache_263_gb300._fastcall", None)
    monkeypatch.setattr(pkv, "_fast_module", None)
    test_copies((2, 16, 128), torch.bfloat16, 160, 3)
    test_copies_that_are_skipped()
    test_forks(300, 513, 20, True)
    test_remap(16, 256, 9, 4000)
    test_a_prompt_sampled_searched_and_compacted(False)
    assert not hasattr(pkv._fast(), "__file__")


# ---------------------------------------------------------------------- in use
@pytest.mark.parametrize("fp8", [False, True])
def test_a_prompt_sampled_searched_and_compacted(fp8):
    """One prompt forked into samples, their blocks copied in two layers, a step of
    beam search among them, the pool compacted under them: attention over the shared
    prefix gives what it gave, and the host's references come out even."""
    hq, hkv, D, width, n0, steps = 8, 2, 128, 40, 9, 20
    L0 = 333
    pool = pkv.KVPool(300, np.random.default_rng(2).permutation(300))
    pool.alloc(100)                                     # blocks of others, freed below
    g = torch.Generator(device="cuda").manual_seed(4)

    def cache():
        x = torch.randn(300, hkv, BS, D, generator=g, device="cuda")
        return (x * 90).to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else x.to(torch.bfloat16)

    layers = [(cache(), cache()) for _ in range(2)]
    scales = torch.full((hkv,), 1 / 90, device="cuda") if fp8 else None
    prompt = pool.alloc(-(-L0 // BS))
    table = np.full((1, width), -1)
    table[0, :len(prompt)] = prompt
    i = lambda n, *s: torch.full((n, *s), -1, dtype=torch.int32, device="cuda")  # noqa: E731

    def forked(tables, lens, parents, keep):
        C = len(parents)
        free = pool.alloc(C)
        child, clens, src, dst, taken = i(C, width), i(C), i(C), i(C), i(1)
        pkv.kv_fork_tables(tables, lens, i32(parents), i32(free), child, clens, src, dst, taken, first_keeps=keep)
        pkv.kv_copy_blocks([c for kv in layers for c in kv], src, dst)
        status()
        t = int(taken.item())
        if t < C:
            pool.free(free[t:])
        old, new = tables.cpu().numpy(), child.cpu().numpy()
        for c, n in enumerate(clens.tolist()):
            k = -(-n // BS)
            same = [b for b in new[c, :k].tolist() if b in set(old[parents[c]].tolist())]
            pool.share(same) if same else None
        for p, n in enumerate(lens.tolist()):
            pool.free(old[p, :-(-n // BS)])
        return child, clens

    tables, lens = forked(i32(table), i32([L0]), [0] * n0, False)
    assert (lens == L0).all()

    def grow(tables, lens, upto):
        """Every sequence gets its own tokens up to `upto`, in blocks of its own."""
        t = tables.cpu().numpy()
        for s, n in enumerate(lens.tolist()):
            for j in range(-(-n // BS), -(-upto // BS)):
                t[s, j] = pool.alloc(1)[0]
            slots = i32([t[s, x // BS] * BS + x % BS for x in range(n, upto)]).long()
            for k, v in layers:
                a, b = (torch.randn(upto - n, hkv, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
                pkv.reshape_and_cache(a, b, k, v, slots, scales, scales)
        return i32(t), torch.full_like(lens, upto)

    tables, lens = grow(tables, lens, L0 + steps)
    beams = [4, 4, 0, 8, 8, 8, 1, 7, 2]
    tables, lens = forked(tables, lens, beams, True)
    tables, lens = grow(tables, lens, L0 + steps + 3)
    q = torch.randn(n0, hq, D, generator=g, device="cuda").to(torch.bfloat16)

    def attend(layer):
        k, v = layers[layer]
        out = torch.empty(n0, hq, D, dtype=torch.bfloat16, device="cuda")
        pkv.paged_attention_shared_prefix(out, q, k, v, tables, lens, i32([0, n0]), i32([L0]), max_prefix_len=L0,
                                          max_tail_len=64, k_scale=scales, v_scale=scales)
        status()
        return out

    def reference(layer):
        k, v = (x.view(torch.float8_e4m3fn).float() / 90 if fp8 else x.float() for x in layers[layer])
        f = lambda x: x.cpu().numpy().astype(np.float64)  # noqa: E731
        return osp.shared(f(q.float()), f(k), f(v), tables.cpu().numpy(), lens.tolist(), [0, n0], [L0], D ** -0.5, fp8=fp8)

    before = [attend(0), attend(1)]
    for layer in range(2):
        exp, tol, _ = reference(layer)
        assert (np.abs(before[layer].float().cpu().numpy() - exp) <= tol).all()
    # the others leave; the pool is compacted under the samples
    others = [b for b in range(300) if pool.refcount(b) and b not in set(tables.cpu().numpy().ravel().tolist())]
    assert len(others) == 100
    pool.free(others)
    src, dst = pool.compact()
    assert len(src) > 5
    pkv.kv_copy_blocks([c for kv in layers for c in kv], i32(src), i32(dst))
    pkv.kv_remap_tables(tables, lens, i32(src), i32(dst))
    status()
    live = pool.stats()["live"]
    t = tables.cpu().numpy()
    assert t[:, :-(-(L0 + steps + 3) // BS)].max() == live - 1
    for layer in range(2):
        for x in layers[layer]:
            x[live:] = 0x7F if fp8 else float("nan")
        assert torch.equal(attend(layer).view(torch.int16), before[layer].view(torch.int16))
    for row, n in zip(t, lens.tolist()):
        pool.free(row[:-(-n // BS)])
    assert pool.stats()["live"] == 0
