"""Absorbed latent attention at work: batches of several hundred key tiles, where
every worker runs its ring of stages and exchange slots many times over."""
import numpy as np
import pytest
import torch

import paged_kv_cache_263_gb300 as pkv
from oracle import latent as ol
from tests.gpu_util import require_gpu
from tests.test_gpu_latent import SCALE, Paged, Prompt, bf, check, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    require_gpu()


@pytest.mark.parametrize("heads,lens,rows", [
    (48, [500, 900, 1300, 130, 64, 700], [90, 70, 20, 90, 64, 5]), (128, [2000, 300, 1500], [9, 20, 1])])
def test_absorbed_masked_tiles_repeat_exactly(heads, lens, rows):
    """Chunks whose rows see different numbers of keys: the tiles at their ends are masked,
    and the exchange slots that carry them are used again at once."""
    w = Paged(heads, lens, rows, seed=heads)
    got = w.run()
    check(got, *w.expected())
    args, first = w.args(), w.out.clone().view(torch.int16)
    for _ in range(30):
        w.out.fill_(float("nan"))
        pkv.paged_latent_attention(**args)
        assert torch.equal(w.out.view(torch.int16), first)
    assert pkv.kv_last_device_status() == 0


@pytest.mark.parametrize("heads", [8, 128])
@pytest.mark.parametrize("short", [0, 5])
def test_absorbed_longest_context(heads, short):
    """2^31 - 64 keys, all in two blocks: the first block's score 0 and hold 1 in dim 0,
    the last one's score 30 (to base 2) and hold 1 in dim 1.  Every number in the sums is
    exact, so only the quotient and its rounding to bf16 are off."""
    blocks = 2 ** 27 - 4
    L = 16 * blocks - short
    tables = torch.zeros(1, blocks, dtype=torch.int32, device="cuda")
    tables[0, -1] = 1
    cache = torch.zeros(2, 16, 576, dtype=torch.bfloat16, device="cuda")
    cache[0, :, 0], cache[1, :, 1], cache[1, :, 512] = 1.0, 1.0, 30.0
    if short:
        cache[1, 16 - short:] = float("nan")
    q = torch.zeros(1, heads, 576, dtype=torch.bfloat16, device="cuda")
    q[:, :, 512] = 1.0
    out = torch.full((1, heads, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
    pkv.paged_latent_attention(out, q, cache, tables, torch.tensor([L], dtype=torch.int32, device="cuda"),
                               scale=float(np.log(2.0)))
    assert pkv.kv_last_device_status() == 0
    got, last = f64(out)[0], 2.0 ** 30 * (16 - short)
    exp = np.array([16.0 * (blocks - 1), last]) / (16.0 * (blocks - 1) + last)
    # (30 x scale x log2(e) in fp32 is 30 up to 2^-18, the exponential's weight up to as much)
    assert (np.abs(got[:, :2] - exp) <= exp * (2.0 ** -8 + 2.0 ** -16)).all(), (got[0, :2], exp)
    assert (got[:, 2:] == 0).all()


# ----------------------------------------------------------------- known shares
FACTORS = np.array([-1.0, 0.0, 1.0])


def shares(lens, rows, weight, tile, dims):
    """Every key of tile i weighs 2^(a weight[s][i]) for a head of factor a and holds 1 in dim
    i mod `dims`, so the output holds each tile's share of the weights: [R][factor][dims] of
    it for rows that see the first L - n + 1, .. keys."""
    out = np.zeros((int(sum(rows)), len(FACTORS), dims))
    r = 0
    for s, (L, n) in enumerate(zip(lens, rows)):
        at = np.arange(-(-L // tile))
        for i in range(n):
            seen = np.clip(L - n + 1 + i - tile * at, 0, tile)
            w = seen[None, :] * 2.0 ** (FACTORS[:, None] * weight[s][at][None, :])
            if L > 0:
                np.add.at(out[r], (slice(None), at % dims), w / w.sum(axis=1, keepdims=True))
            r += 1
    return out


# Scores are whole numbers (the scale is ln 2), so that the weights are powers of two: exact in
# bf16, as are the values.  The exponent, in fp32, is off by at most 2^-18 of its size (below 64
# here: 2^-17), sums by less; the output's rounding is 2^-8.
KNOWN = 2.0 ** -8 + 2.0 ** -15


def check_shares(got, exp, a):
    for i, f in enumerate(FACTORS):
        off = np.abs(got[:, a == f] - exp[:, i, None]) - KNOWN * exp[:, i, None]
        assert off.size == 0 or off.max() <= 0, (f, off.max(), np.argwhere(off > 0)[:5])


class Marked(Paged):
    """Paged, with known shares: a tile that is lost, taken twice or weighed wrongly, and a row
    that sees a key more or less, changes them by at least a 64th of a tile's share."""

    def __init__(self, heads, lens, rows, kind, seed=0, **kw):
        super().__init__(1, lens, rows, seed=seed, **kw)
        rng = np.random.default_rng(seed)
        self.heads = heads
        most = max(1, -(-max(lens) // 64))
        self.weight = [np.zeros(most) if kind == "even" else rng.integers(-6, 7, most) if kind == "uneven"
                       else np.minimum(np.arange(most) * 5, 60) for _ in lens]
        self.a = rng.choice(FACTORS, heads)
        self.small[~np.isnan(self.small)] = 0.0
        for s, L in enumerate(lens):
            t = np.arange(L)
            block, at = self.tables[s, t // 16], t % 16
            self.small[block, at, (t // 64) % 512] = 1.0
            self.small[block, at, 512] = self.weight[s][t // 64]
        self.cache = bf(self.small)
        self.q = torch.zeros(len(self.q), heads, 576, dtype=torch.bfloat16, device="cuda")
        self.q[:, :, 512] = bf(self.a)
        self.out = torch.empty(len(self.q), heads, 512, dtype=torch.bfloat16, device="cuda")

    def args(self, decode=False):
        return {**super().args(decode), "scale": float(np.log(2.0))}

    def check(self, got):
        check_shares(got, shares(self.lens, self.rows, self.weight, 64, 512), self.a)


RAGGED = [200 + (i * 911) % 2300 for i in range(40)]
BATCHES = {
    # pairs of CTAs: decode, chunks of tens of rows, one long chunk, drafts, one long context
    "decode": (128, RAGGED, [1] * 40),
    "chunks": (96, [500 + (i * 577) % 1500 for i in range(12)], [70] * 12),
    "chunk": (32, [3000], [500]),
    "drafts": (32, [300 + (i * 1777) % 5700 for i in range(48)], [4] * 48),
    "long": (128, [60000], [1]),
    # a CTA each: decode, one long chunk among short entries, one long context, few rows
    "small-decode": (16, [17 + (i * 911) % 4000 for i in range(150)], [1] * 150),
    "small-chunk": (8, [20] * 30 + [3000] + [90] * 25, [1] * 30 + [300] + [1] * 25),
    "small-long": (64, [60000], [1]),
    "small-rows": (5, [(i * 333) % 1500 + 70 for i in range(60)], [(i * 7) % 13 for i in range(60)]),
}


@pytest.mark.parametrize("kind", ["even", "uneven", "growing"])
@pytest.mark.parametrize("name", list(BATCHES))
def test_absorbed_known_shares(name, kind):
    heads, lens, rows = BATCHES[name]
    assert (sum(rows) * heads <= 64 * len(rows)) == name.startswith("small")
    w = Marked(heads, lens, rows, kind, seed=len(name))
    got = w.run()
    assert pkv.kv_last_device_status() == 0
    w.check(got)
    assert np.array_equal(w.run(), got)


@pytest.mark.parametrize("heads,n", [(2, 5000), (65, 3300)])
def test_absorbed_thousands_of_sequences(heads, n):
    """Ranges of more sequences than a worker tables."""
    rng = np.random.default_rng(heads)
    lens = rng.integers(1, 41, n)
    w = Marked(heads, lens.tolist(), [1] * n, "even", seed=heads)
    w.check(w.run(decode=True))
    assert pkv.kv_last_device_status() == 0


@pytest.mark.parametrize("heads", [8, 128])
def test_absorbed_hundreds_of_entries_without_rows(heads):
    lens = [700] + [30] * 400 + [500] + [0] * 300 + [900]
    rows = [3] + [0] * 400 + [2] + [0] * 300 + [1]
    w = Marked(heads, lens, rows, "uneven", seed=heads)
    w.check(w.run())
    assert pkv.kv_last_device_status() == 0


@pytest.mark.parametrize("heads", [8, 128])
def test_absorbed_sequences_that_share_blocks(heads):
    """A beginning of 40 blocks that all sequences' tables name, and ends of their own."""
    lens, rows = [640 + 16 * i + 3 for i in range(9)], [1, 2, 1, 4, 1, 1, 3, 1, 1]
    w = Paged(heads, lens, rows, seed=heads)
    w.tables[:, :40] = w.tables[0, :40]
    got = w.run()
    assert pkv.kv_last_device_status() == 0
    check(got, *w.expected())
    assert np.array_equal(w.run(), got)


# ----------------------------------------------------------------- error of a row
def row_limit(q, k, v, scale, limit):
    """Twice the root mean square, over a row's dims, of the roundings that the kernels make:
    (out, limit) of attend()'s arguments, k and v [T][d], [T][e].  Half a step of bf16 at most
    each, and taken as evenly spread and independent: u = 2^-8 / sqrt(3) of every probability,
    of their sum (which adds them unrounded) and of the output.  (512 dims: the mean square of
    their errors is within a tenth of its expectation, and the limit is four times that.)"""
    out, allowed = np.zeros(q.shape[:2] + (v.shape[1],)), np.zeros(q.shape[:2])
    u2 = (2.0 ** -8) ** 2 / 3
    for h in range(q.shape[1]):
        s = np.where(np.arange(len(k))[None, :] < np.asarray(limit)[:, None], scale * (q[:, h] @ k.T), -np.inf)
        p = np.exp(s - s.max(axis=1, keepdims=True))
        p /= p.sum(axis=1, keepdims=True)
        o = p @ v
        out[:, h] = o
        o2, p2 = (o ** 2).mean(axis=1), p ** 2
        allowed[:, h] = 2 * np.sqrt(u2 * (o2 * (1 + p2.sum(axis=1)) + p2 @ (v ** 2).mean(axis=1)))
    return out, allowed


@pytest.mark.parametrize("heads,lens,rows", [(8, [20000], [1]), (8, [30000, 5], [3, 1]), (49, [3000], [1]),
                                             (128, [9000], [1]), (64, [5000, 5001], [2, 1])])
def test_absorbed_error_of_a_row(heads, lens, rows):
    w = Paged(heads, lens, rows, seed=heads, v_mean=0.1)
    got = w.run()
    for s, L in enumerate(lens):
        a, b = w.cu[s], w.cu[s + 1]
        x = ol.gather(w.small, w.tables[s], L)
        out, allowed = row_limit(f64(w.q)[a:b], x, x[:, :512], SCALE, np.arange(L - (b - a) + 1, L + 1))
        rms = np.sqrt(((got[a:b] - out) ** 2).mean(axis=-1))
        assert (rms <= allowed).all(), (rms / allowed).max()


# ----------------------------------------------------------------- expanded form
class MarkedPrompt(Prompt):
    def __init__(self, heads, nq, nk, kind, seed=0):
        super().__init__(heads, nq, nk, seed=seed)
        rng = np.random.default_rng(seed)
        self.nq, self.nk = list(nq), list(nk)
        most = max(1, -(-int(max(nk)) // 128))
        self.weight = [np.zeros(most) if kind == "even" else rng.integers(-6, 7, most) if kind == "uneven"
                       else np.minimum(np.arange(most) * 9, 60) for _ in nk]
        self.a = rng.choice(FACTORS, heads)
        kv, rope = np.zeros((sum(nk), 256)), np.zeros((sum(nk), 64))
        for s, n in enumerate(self.nk):
            t, at = np.arange(n), int(self.cu_k[s])
            kv[at + t, 128 + (t // 128) % 128] = 1.0
            rope[at + t, 0] = self.weight[s][t // 128]
        self.kv = bf(kv)[:, None, :].expand(-1, heads, -1).contiguous()
        self.rope = bf(rope)
        self.q.zero_()
        self.q[:, :, 128] = bf(self.a)

    def check(self, got):
        check_shares(got, shares(self.nk, self.nq, self.weight, 128, 128), self.a)


@pytest.mark.parametrize("kind", ["even", "uneven", "growing"])
@pytest.mark.parametrize("heads,nq,nk", [
    (24, [333 + 343 * i for i in range(6)], [450 + 343 * i + 117 * i for i in range(6)]), (128, [2000], [2000]),
    (3, [1500, 1, 129], [6000, 3000, 1290])])
def test_expanded_known_shares(heads, nq, nk, kind):
    w = MarkedPrompt(heads, nq, nk, kind, seed=heads)
    got = w.run(scale=float(np.log(2.0)))
    assert pkv.kv_last_device_status() == 0
    w.check(got)


def test_expanded_thousands_of_sequences():
    """A list of more sequences than the threads that build it."""
    rng = np.random.default_rng(5)
    nq = rng.integers(1, 4, 2500)
    nk = nq + rng.integers(0, 300, 2500)
    w = MarkedPrompt(3, nq.tolist(), nk.tolist(), "uneven", seed=5)
    got = w.run(scale=float(np.log(2.0)))
    assert pkv.kv_last_device_status() == 0
    w.check(got)


# ----------------------------------------------------------------- cache write
@pytest.mark.parametrize("T,pad", [(1, 0), (64, 0), (333, 7)])
def test_latent_write_of_one_row_to_every_slot(T, pad):
    """Broadcast rows (stride 0), a slot outside the pool, and nothing else touched."""
    g = torch.Generator(device="cuda").manual_seed(T)
    nb = -(-T // 16) + 2
    wide = torch.randn(2, 704, generator=g, device="cuda").to(torch.bfloat16)
    lat, rope = wide[:1, 8:520].expand(T + pad, -1), wide[1:, 600:664].expand(T + pad, -1)
    cache = torch.randn(nb, 16, 576, generator=g, device="cuda").to(torch.bfloat16)
    slots = torch.full((T + pad,), -1, dtype=torch.int64, device="cuda")
    slots[:T] = torch.randperm(nb * 16, generator=g, device="cuda")[:T]
    slots[0] = nb * 16
    exp = cache.clone().view(-1, 576)
    exp[slots[1:T]] = torch.cat([lat[:1], rope[:1]], dim=1)
    pkv.reshape_and_cache_latent(lat, rope, cache, slots)
    assert pkv.kv_last_device_status() == 5 and pkv.kv_last_device_status_flags() == 2
    assert torch.equal(cache.view(-1, 576).view(torch.int16), exp.view(torch.int16))
