"""fp64 reference of attention over shared prefixes, of the forks of sequences and
of what happens to tables and pools when blocks move (numpy; independent of the
library's code).

attend() also returns, per output element, how far a correct kernel may be off.
Scores, softmax statistics, sums and partial outputs are held in fp32,
probabilities are rounded to 16 bits for the second product, and the output is
rounded to bf16.  With u16 = 2^-8 (bf16, half a step) and u = 2^-24 (fp32):
 - a score is a sum of d products, exact in fp32, added in some order: it is off
   by at most scale * sum|q_i k_i| * d * 2u (2u: the adder may truncate); over an
   fp8 cache each q_i is rounded to f16 first, 2^-11 of it; a weight's numerator and
   the normaliser are each off by that factor, 2 delta;
 - a probability's rounding is at most u16 of it (2^-11 in f16), the exponential,
   the sums and the joining of parts stay below 2^-15 together, so
   sum_t p_t |v_t| (u16 + 2 delta + 2^-15);
 - the last rounding adds u16 of the value reached.
"""
from __future__ import annotations

import numpy as np

BS = 16
U16, U32, UF16 = 2.0 ** -8, 2.0 ** -24, 2.0 ** -11
BAD_BLOCK, BAD_LEN, NO_BLOCKS = 1, 4, 16


def gather(cache, table, n):
    """Keys (or values) 0 .. n-1 of a sequence: cache [blocks][Hkv][16][128] -> [n][Hkv][128]."""
    t = np.arange(n)
    return cache[np.asarray(table)[t // BS], :, t % BS]


def attend(q, k, v, scale, limit, fp8=False):
    """q [R][Hq][d], k and v [T][Hkv][d] (head h reads h // (Hq / Hkv)); row r sees the
    keys t < limit[r].  Returns (out, allowed error), [R][Hq][d] each."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    R, H, d = q.shape
    per = H // k.shape[1]
    out, tol = np.zeros((R, H, d)), np.zeros((R, H, d))
    seen = np.arange(k.shape[0])[None, :] < np.asarray(limit)[:, None]
    for h in range(H):
        kh, vh = k[:, h // per], v[:, h // per]
        s = np.where(seen, scale * (q[:, h] @ kh.T), -np.inf)
        size = np.where(seen, scale * (np.abs(q[:, h]) @ np.abs(kh).T), 0.0).max(axis=1, keepdims=True)
        e = np.exp(s - s.max(axis=1, keepdims=True))
        p = e / e.sum(axis=1, keepdims=True)
        delta = size * (d * 2 * U32 + (UF16 if fp8 else 0.0))
        out[:, h] = p @ vh
        off = (p @ np.abs(vh)) * ((UF16 if fp8 else U16) + 2 * delta + 2.0 ** -15)
        tol[:, h] = off + U16 * (np.abs(out[:, h]) + off)
    return out, tol


def shared(q, k, v, tables, lens, cu_groups, prefix, scale, cu=None, fp8=False, max_q=None, max_prefix=1 << 30,
           max_tail=1 << 30):
    """The call: (out, allowed error, flags).  NaN in rows that are left as they were."""
    q = np.asarray(q, dtype=np.float64)
    B, width = np.asarray(tables).shape
    cu = np.arange(B + 1) if cu is None else np.asarray(cu)
    R = q.shape[0]
    out, tol = np.full(q.shape, np.nan), np.zeros(q.shape)
    flags = 0
    for s in range(B):
        a, b, L = int(cu[s]), int(cu[s + 1]), int(lens[s])
        P, first, ok = 0, s, True
        for g in range(len(prefix)):
            s0, s1 = int(cu_groups[g]), int(cu_groups[g + 1])
            if s0 <= s < s1:
                P, first = int(prefix[g]) // BS * BS, s0
                ok = 0 <= s0 and s1 <= B and prefix[g] >= 0 and P <= max_prefix // BS * BS
                ok = ok and 0 <= int(cu[s0]) <= int(cu[s1]) <= R
        n = b - a
        if a < 0 or n < 0 or b > R or n > (R if max_q is None else max_q):
            flags |= BAD_LEN
            continue
        if L == 0:
            out[a:b] = 0.0
            continue
        if not ok or L < 0 or L > width * BS or L - n < P or L - P > max_tail:
            flags |= BAD_LEN
            continue
        if n == 0:
            continue
        row = np.concatenate([np.asarray(tables[first])[:P // BS], np.asarray(tables[s])[P // BS:]])
        out[a:b], tol[a:b] = attend(q[a:b], gather(k, row, L), gather(v, row, L), scale, np.arange(L - n, L) + 1, fp8)
    return out, tol, flags


def fork(tables, lens, parents, free, first_keeps, child_tables):
    """(child tables, child lengths, copy sources, copy destinations, taken, flags)."""
    tables, out = np.asarray(tables), np.array(child_tables)
    C, width = out.shape
    clens, src, dst = np.zeros(C, int), np.full(C, -1), np.full(C, -1)
    kept, taken, flags = set(), 0, 0
    for c, a in enumerate(parents):
        a = int(a)
        if a < 0 or a >= len(lens) or not 0 <= int(lens[a]) <= width * BS:
            flags |= BAD_LEN
            continue
        L = int(lens[a])
        n = -(-L // BS)
        fresh = L % BS != 0 and not (first_keeps and a not in kept)
        kept.add(a)
        if fresh:
            if taken >= len(free):
                flags |= NO_BLOCKS
                continue
            src[c], dst[c] = tables[a, n - 1], free[taken]
            taken += 1
        out[c, :n] = tables[a, :n]
        if fresh:
            out[c, n - 1] = dst[c]
        clens[c] = L
    return out, clens, src, dst, taken, flags


def remap(tables, lens, src, dst):
    """(tables, flags)."""
    out, flags = np.array(tables), 0
    to = dict(zip((int(x) for x in src), (int(x) for x in dst)))
    for s, L in enumerate(lens):
        if not 0 <= int(L) <= out.shape[1] * BS:
            flags |= BAD_LEN
            continue
        for j in range(-(-int(L) // BS)):
            out[s, j] = to.get(int(out[s, j]), out[s, j])
    return out, flags


def compact(ref, free_list, max_moves):
    """A pool's refcounts and its order of allocation after a compaction:
    (src, dst, refcounts, order)."""
    ref, live = list(ref), sum(r > 0 for r in ref)
    high = [b for b in range(live, len(ref)) if ref[b] > 0][::-1][:max_moves][::-1]
    low = [b for b in range(live) if ref[b] == 0][:len(high)]
    for a, b in zip(high, low):
        ref[a], ref[b] = 0, ref[a]
    to = dict(zip(low, high))
    return high, low, ref, [to.get(b, b) for b in free_list]
