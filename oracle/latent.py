"""fp64 reference of the latent-attention operators and of the step tables
(numpy; independent of the library's code).

attend() also returns, per output element, how far a correct kernel may be off:
scores, softmax statistics and sums are held in fp32, probabilities are rounded
to bf16 for the second product, and the output is rounded to bf16.  With
u16 = 2^-8 (bf16, half a step) and u = 2^-24 (fp32):
 - a score is a sum of d products, exact in fp32, added in some order: it is off
   by at most scale * sum|q_i x_i| * d * 2u (2u: the adder may truncate), so a
   weight's numerator and the normaliser are each off by that factor, 2 delta;
 - a probability's rounding is at most u16 of it, the exponential and the sums
   stay below 2^-16 together, so sum_t p_t |v_t| (u16 + 2 delta + 2^-16);
 - the last rounding adds u16 of the value (of the value reached, so also of the
   error above).
"""
from __future__ import annotations

import numpy as np

BS = 16
U16, U32 = 2.0 ** -8, 2.0 ** -24


def attend(q, k, v, scale, limit):
    """q [R][H][d], k [T][d] or [T][H][d], v [T][e] or [T][H][e]; row r sees the
    keys t < limit[r].  Returns (out, allowed error), [R][H][e] each."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    R, H, d = q.shape
    T = k.shape[0]
    if k.ndim == 2:
        k = np.broadcast_to(k[:, None], (T, H, d))
    if v.ndim == 2:
        v = np.broadcast_to(v[:, None], (T, H, v.shape[-1]))
    out = np.zeros((R, H, v.shape[-1]))
    tol = np.zeros_like(out)
    limit = np.minimum(np.asarray(limit), T)
    seen = np.arange(T)[None, :] < limit[:, None]
    some = limit > 0
    if not some.any():
        return out, tol
    for h in range(H):
        s = np.where(seen, scale * (q[:, h] @ k[:, h].T), -np.inf)[some]
        size = np.where(seen, scale * (np.abs(q[:, h]) @ np.abs(k[:, h]).T), 0.0)[some]
        e = np.exp(s - s.max(axis=1, keepdims=True))
        p = e / e.sum(axis=1, keepdims=True)
        delta = size.max(axis=1, keepdims=True) * d * 2 * U32
        o = p @ v[:, h]
        off = (p @ np.abs(v[:, h])) * (U16 + 2 * delta + 2.0 ** -16)
        out[some, h] = o
        tol[some, h] = off + U16 * (np.abs(o) + off)
    return out, tol


def gather(cache, table, length):
    """The rows of a sequence's keys from the paged latent cache [blocks][16][576]."""
    t = np.arange(length)
    return cache[table[t // BS], t % BS]


def absorbed(q, cache, tables, lens, cu, scale):
    """(out, allowed error) of the absorbed form; rows of no sequence are NaN."""
    out = np.full(q.shape[:2] + (512,), np.nan)
    tol = np.zeros_like(out)
    for s, L in enumerate(lens):
        a, b = int(cu[s]), int(cu[s + 1])
        n, L = b - a, int(L)
        if n == 0:
            continue
        x = gather(cache, tables[s], L)
        out[a:b], tol[a:b] = attend(q[a:b], x, x[:, :512], scale, np.arange(L - n + 1, L + 1) if L else np.zeros(n))
    return out, tol


def expanded(q, kv, rope, cu_q, cu_k, scale):
    """(out, allowed error) of the expanded form; rows of no sequence are NaN."""
    H = q.shape[1]
    out = np.full(q.shape[:2] + (128,), np.nan)
    tol = np.zeros_like(out)
    for s in range(len(cu_q) - 1):
        a, b, c, d = int(cu_q[s]), int(cu_q[s + 1]), int(cu_k[s]), int(cu_k[s + 1])
        n, nk = b - a, d - c
        if n == 0:
            continue
        if nk == 0:
            out[a:b] = 0.0
            continue
        k = np.concatenate([kv[c:d, :, :128], np.repeat(rope[c:d, None], H, axis=1)], axis=-1)
        out[a:b], tol[a:b] = attend(q[a:b], k, kv[c:d, :, 128:], scale, np.arange(nk - n + 1, nk + 1))
    return out, tol


def step_tables(tables, ctx, new, free, num_blocks, max_tokens):
    """Sequence by sequence: (tables, cu, lens, slots, positions, (rows, taken), flags)."""
    tables = np.array(tables, dtype=np.int64)
    width = tables.shape[1]
    cu, lens, slots, pos, flags = [0], [], [], [], 0
    all_rows = all_need = taken = 0
    for s, (c, n) in enumerate(zip(map(int, ctx), map(int, new))):
        if c < 0 or n < 0 or c + n > width * BS:
            flags |= 4
            cu.append(cu[-1])
            lens.append(c)
            continue
        need, start = -(-(c + n) // BS) - -(-c // BS), all_need
        all_rows, all_need = all_rows + n, all_need + need
        ok = True
        if n and all_rows > max_tokens:
            ok, flags = False, flags | 4
        if need and all_need > len(free):
            ok, flags = False, flags | 16
        if ok:
            have = -(-c // BS)
            tables[s, have:have + need] = free[start:start + need]
            taken = max(taken, all_need) if need else taken
            for t in range(c, c + n):
                b = int(tables[s, t // BS])
                inside = 0 <= b < num_blocks
                flags |= 0 if inside else 1
                slots.append(b * BS + t % BS if inside else -1)
                pos.append(t)
        cu.append(cu[-1] + (n if ok else 0))
        lens.append(c + (n if ok else 0))
    rows = cu[-1]
    slots += [-1] * (max_tokens - rows)
    pos += [0] * (max_tokens - rows)
    return tables, np.array(cu), np.array(lens), np.array(slots), np.array(pos), (rows, taken), flags
