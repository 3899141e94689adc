"""Cases that measure the latent-attention operators: block tables and slot
numbers built on the device, the latent cache write, attention over the paged
latent cache (absorbed form) and prompt attention over expanded keys and values.

A latent cache keeps one vector of 512 + 64 values a token: a latent that every
head's keys and values are linear functions of, and a rotary key that all heads
share.  The absorbed form folds the expansion into the queries (576 wide) and
attends the cached vectors themselves; the expanded form attends keys of
128 + 64 and values of 128 per head.

``run`` computes an operator in plain torch operations (32-bit arithmetic, one
rounding at the end) or, with ``own`` set, through the library's calls.
``exact`` gives the same results in 64 bits, sequence by sequence.
"""
import math

import torch

own = False

LAT, ROPE, NOPE, VD, BS = 512, 64, 128, 128, 16
KD = LAT + ROPE
SCALE = (NOPE + ROPE) ** -0.5
DEV = "cuda"


# ------------------------------------------------------------------- the cases
def listed():
    return [
        # every sequence of a small serving batch gains one token: the call before each decode step
        {"name": "tables-decode", "op": "tables", "seqs": 64, "lo": 1, "hi": 4096, "new_lo": 1, "new_hi": 1},
        # a large batch that mixes one-token steps with prompt chunks
        {"name": "tables-mixed", "op": "tables", "seqs": 4096, "lo": 0, "hi": 8192, "new_lo": 0, "new_hi": 33},
        # the new tokens of a decode step
        {"name": "write-decode", "op": "write", "tokens": 64, "pad": 0},
        # a prompt batch, padded to a captured graph's size
        {"name": "write-prompt", "op": "write", "tokens": 16384, "pad": 37},
        # one short conversation: latency
        {"name": "absorbed-one", "op": "absorbed", "seqs": 1, "heads": 128, "lo": 1000, "hi": 1000, "q": 1},
        # one very long context: split over its length and joined
        {"name": "absorbed-long", "op": "absorbed", "seqs": 1, "heads": 64, "lo": 131072, "hi": 131072, "q": 1},
        # an ordinary decode batch with ragged lengths
        {"name": "absorbed-batch", "op": "absorbed", "seqs": 64, "heads": 128, "lo": 1500, "hi": 8200, "q": 1},
        # many sequences and few heads, as on one of several ranks
        {"name": "absorbed-few-heads", "op": "absorbed", "seqs": 256, "heads": 8, "lo": 17, "hi": 4096, "q": 1},
        # speculative drafts: several query rows a sequence, causal among themselves
        {"name": "absorbed-drafts", "op": "absorbed", "seqs": 48, "heads": 32, "lo": 300, "hi": 6000, "q": 4},
        # short prompts
        {"name": "prompt-short", "op": "expanded", "seqs": 8, "heads": 32, "lo": 40, "hi": 300, "before": 0},
        # one long prompt, all heads
        {"name": "prompt-long", "op": "expanded", "seqs": 1, "heads": 128, "lo": 4096, "hi": 4096, "before": 0},
        # ragged prompt chunks that also see keys before them
        {"name": "prompt-chunks", "op": "expanded", "seqs": 6, "heads": 64, "lo": 333, "hi": 2048, "before": 700},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "write", "absorbed", "absorbed", "expanded", "expanded"])
    if op == "tables":
        hi = _log(rng, 16, 8192)
        return {"op": op, "seqs": _log(rng, 1, 4096), "lo": rng.randint(0, hi), "hi": hi, "new_lo": rng.randint(0, 1),
                "new_hi": _log(rng, 1, 33)}
    if op == "write":
        return {"op": op, "tokens": _log(rng, 1, 16384), "pad": rng.randint(0, 40)}
    if op == "absorbed":
        heads, q = rng.choice([1, 4, 8, 12, 20, 32, 40, 64, 96, 128]), rng.choice([1, 1, 1, 2, 3, 5, 8, 70])
        seqs = _log(rng, 1, 256)
        most = max(q, min(131072, 360000 // (seqs * max(1, heads * q // 128))))
        hi = _log(rng, q, most)
        return {"op": op, "seqs": seqs, "heads": heads, "lo": rng.randint(q, hi), "hi": hi, "q": q}
    heads, seqs = rng.choice([1, 3, 8, 16, 32, 48, 64, 128]), _log(rng, 1, 16)
    hi = _log(rng, 1, min(4096, int((2.0e9 / (seqs * heads)) ** 0.5)))
    before = rng.choice([0, 0, _log(rng, 1, 1000)])
    while before and seqs * heads * hi * (hi + before) > 2.1e9:
        before //= 2
    return {"op": op, "seqs": seqs, "heads": heads, "lo": rng.randint(1, hi), "hi": hi, "before": before}


def _spread(n, lo, hi, step=7):
    """n lengths between lo and hi, both reached where n > 1, in no order."""
    return [hi if n == 1 else lo + (hi - lo) * ((i * step + n // 2) % n) // (n - 1) for i in range(n)]


def _lens(c):
    """(context or key lengths, query rows) of each sequence."""
    n = c["seqs"]
    if c["op"] == "tables":
        return _spread(n, c["lo"], c["hi"]), _spread(n, c["new_lo"], c["new_hi"], 13)
    if c["op"] == "absorbed":
        return _spread(n, c["lo"], c["hi"]), [c["q"]] * n
    q = _spread(n, c["lo"], c["hi"])
    return [x + (c["before"] * (i + 1)) // n for i, x in enumerate(q)], q


def work(case):
    c = case
    if c["op"] == "write":
        return {"bytes": c["tokens"] * (2 * KD * 2 + 8) + c["pad"] * 8, "flops": 0}
    lens, new = _lens(c)
    if c["op"] == "tables":
        blocks = sum(-(-(a + b) // BS) - -(-a // BS) for a, b in zip(lens, new))
        return {"bytes": 4 * (4 * len(lens) + 2 * blocks + len(lens)) + sum(new) * 12, "flops": 0}
    seen = sum(n * (k - n) + n * (n + 1) // 2 for k, n in zip(lens, new))
    h, rows = c["heads"], sum(new)
    if c["op"] == "absorbed":
        return {"bytes": sum(lens) * KD * 2 + rows * h * (KD + LAT) * 2 + 4 * sum(-(-k // BS) for k in lens),
                "flops": 2 * h * (KD + LAT) * seen}
    return {"bytes": rows * h * (NOPE + ROPE + VD) * 2 + sum(lens) * (h * (NOPE + VD) + ROPE) * 2,
            "flops": 2 * h * (NOPE + ROPE + VD) * seen}


# ------------------------------------------------------------------- the inputs
def _cu(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device=DEV)


def _tables(blocks, width, order):
    """Block tables [n][width]: each sequence's blocks in turn from `order`, the rest -1."""
    b = torch.tensor(blocks, device=DEV)
    at = torch.arange(width, device=DEV)[None, :]
    inside = at < b[:, None]
    idx = (b.cumsum(0) - b)[:, None] + at
    return torch.where(inside, order[idx.clamp(max=order.numel() - 1)], -1).to(torch.int32).contiguous()


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).to(torch.bfloat16)

    st = {"op": c["op"]}
    if c["op"] == "write":
        # the projection's output holds the latent and the rotary key side by side: two views of its rows
        T, nb = c["tokens"], -(-c["tokens"] // BS) + 3
        down = normal(T + c["pad"], KD)
        slots = torch.full((T + c["pad"],), -1, dtype=torch.int64, device=DEV)
        slots[:T] = torch.randperm(nb * BS, generator=g, device=DEV)[:T]
        st |= {"latent": down[:, :LAT], "rope": down[:, LAT:], "cache": normal(nb, BS, KD), "slots": slots}
        return st
    lens, new = _lens(c)
    n = c["seqs"]
    if c["op"] == "tables":
        have = [-(-x // BS) for x in lens]
        need = [-(-(x + y) // BS) - b for x, y, b in zip(lens, new, have)]
        nb = sum(have) + sum(need) + 5
        order = torch.randperm(nb, generator=g, device=DEV)
        rows = sum(new)
        cap = rows + 3
        st |= {"tables": _tables(have, max(1, max(a + b for a, b in zip(have, need))), order[:max(1, sum(have))]),
               "lens": torch.tensor(lens, dtype=torch.int32, device=DEV),
               "new": torch.tensor(new, dtype=torch.int32, device=DEV),
               "free": order[sum(have):].to(torch.int32).contiguous(), "blocks": nb,
               "cu": torch.empty(n + 1, dtype=torch.int32, device=DEV),
               "total_lens": torch.empty(n, dtype=torch.int32, device=DEV),
               "slots": torch.empty(cap, dtype=torch.int64, device=DEV),
               "positions": torch.empty(cap, dtype=torch.int32, device=DEV),
               "totals": torch.empty(2, dtype=torch.int32, device=DEV)}
        return st
    h, rows = c["heads"], sum(new)
    st |= {"cu": _cu(new), "longest": max(lens), "most": max(new), "heads": h, "decode": max(new) == min(new) == 1}
    if c["op"] == "absorbed":
        blocks = [-(-x // BS) for x in lens]
        nb = sum(blocks) + 7
        # normalised latents and rotary keys; queries that spread the scores by about 1.7
        st |= {"cache": normal(nb, BS, KD), "q": normal(rows, h, KD),
               "tables": _tables(blocks, max(blocks), torch.randperm(nb, generator=g, device=DEV)),
               "lens": torch.tensor(lens, dtype=torch.int32, device=DEV),
               "out": torch.empty(rows, h, LAT, dtype=torch.bfloat16, device=DEV)}
        return st
    keys = sum(lens)
    st |= {"cu_k": _cu(lens), "q": normal(rows, h, NOPE + ROPE), "kv": normal(keys, h, NOPE + VD),
           "rope": normal(keys, KD)[:, LAT:], "out": torch.empty(rows, h, VD, dtype=torch.bfloat16, device=DEV)}
    return st


# ------------------------------------------------------------------- one pass
def run(state):
    return (_own if own else _plain)[state["op"]](state)


def _out_tables(s):
    return {"tables": s["tables"], "cu": s["cu"], "lens": s["total_lens"], "slots": s["slots"],
            "positions": s["positions"], "totals": s["totals"]}


def _own_tables(s):
    import paged_kv_cache_263_gb300 as pkv
    pkv.kv_build_step_tables(s["tables"], s["lens"], s["new"], s["free"], s["blocks"], s["cu"], s["total_lens"],
                             s["slots"], s["positions"], s["totals"])
    return _out_tables(s)


def _own_write(s):
    import paged_kv_cache_263_gb300 as pkv
    pkv.reshape_and_cache_latent(s["latent"], s["rope"], s["cache"], s["slots"])
    return s["cache"]


def _own_absorbed(s):
    import paged_kv_cache_263_gb300 as pkv
    if "workspace" not in s:   # kept by the program from call to call
        s["workspace"] = torch.empty(pkv.paged_latent_attention_workspace_size(
            s["lens"].numel(), s["q"].shape[0], s["heads"], s["tables"].shape[1]), dtype=torch.uint8, device=DEV)
    return pkv.paged_latent_attention(s["out"], s["q"], s["cache"], s["tables"], s["lens"],
                                      cu_q_lens=None if s["decode"] else s["cu"], scale=SCALE,
                                      workspace=s["workspace"])


def _own_expanded(s):
    import paged_kv_cache_263_gb300 as pkv
    if "workspace" not in s:
        s["workspace"] = torch.empty(pkv.latent_prefill_attention_workspace_size(
            s["cu"].numel() - 1, s["q"].shape[0], s["heads"]), dtype=torch.uint8, device=DEV)
    return pkv.latent_prefill_attention(s["out"], s["q"], s["kv"], s["rope"], s["cu"], s["cu_k"], scale=SCALE,
                                        workspace=s["workspace"])


_own = {"tables": _own_tables, "write": _own_write, "absorbed": _own_absorbed, "expanded": _own_expanded}


def _plain_tables(s):
    lens, new, n, cap = s["lens"], s["new"], s["lens"].numel(), s["slots"].numel()
    s["total_lens"].copy_(lens + new)
    s["cu"][0] = 0
    s["cu"][1:] = new.cumsum(0)
    have, want = (lens + BS - 1) // BS, (lens + new + BS - 1) // BS
    ends = (want - have).cumsum(0)
    starts = ends - (want - have)
    # the free blocks, in their order, to the sequences, in theirs
    at = torch.arange(s["tables"].shape[1], device=DEV)[None, :]
    fresh = (at >= have[:, None]) & (at < want[:, None])
    idx = (starts[:, None] + at - have[:, None]).clamp(0, s["free"].numel() - 1)
    s["tables"].copy_(torch.where(fresh, s["free"][idx], s["tables"]))
    row = torch.arange(cap, device=DEV)
    seq = torch.searchsorted(s["cu"][1:].contiguous(), row.to(torch.int32), right=True)
    real = seq < n
    seq = seq.clamp(max=n - 1)
    pos = torch.where(real, lens[seq] + row - s["cu"][seq], 0)
    s["positions"].copy_(pos)
    s["slots"].copy_(torch.where(real, s["tables"][seq, pos // BS].long() * BS + pos % BS, -1))
    s["totals"][0] = s["cu"][-1]
    s["totals"][1] = ends[-1]
    return _out_tables(s)


def _plain_write(s):
    real = s["slots"] >= 0
    s["cache"].view(-1, KD)[s["slots"][real]] = torch.cat([s["latent"], s["rope"]], dim=1)[real]
    return s["cache"]


def _padded(x, cu, most):
    """Rows of ragged sequences as [sequence][row][...], and which of them are real."""
    at = cu[:-1, None] + torch.arange(most, device=DEV)[None, :]
    real = at < cu[1:, None]
    return x[at.clamp(max=x.shape[0] - 1)].float(), real


def _back(x, cu, rows):
    """The reverse of _padded for `rows` rows: x [sequence][row][...]."""
    row = torch.arange(rows, dtype=torch.int32, device=DEV)
    seq = torch.searchsorted(cu[1:].contiguous(), row, right=True)
    return x[seq, row - cu[seq]]


def _attend(scores, seen, v):
    """softmax over the seen scores (zeros for a row that sees nothing) times v."""
    scores = scores.masked_fill_(~seen, -math.inf)
    m = scores.amax(-1, keepdim=True)
    p = scores.sub_(m.masked_fill(m == -math.inf, 0.0)).exp_()
    total = p.sum(-1, keepdim=True)
    return (p @ v) / total.masked_fill(total == 0, 1.0)


def _plain_absorbed(s):
    lens, longest, most, h = s["lens"], s["longest"], s["most"], s["heads"]
    t = torch.arange(longest, device=DEV)
    slots = s["tables"].clamp(min=0)[:, t // BS].long() * BS + t % BS
    k = s["cache"].view(-1, KD)[slots].float()
    q, _ = _padded(s["q"], s["cu"], most)
    n = s["cu"][1:] - s["cu"][:-1]
    last = lens[:, None] - n[:, None] + torch.arange(most, device=DEV)[None, :]
    seen = (t[None, None, :] <= last[:, :, None]) & (t[None, None, :] < lens[:, None, None])
    seen = seen[:, :, None, :].expand(-1, -1, h, -1).reshape(len(lens), most * h, longest)
    o = _attend((q.flatten(1, 2) * SCALE) @ k.transpose(1, 2), seen, k[..., :LAT])
    return _back(o.view(len(lens), most, h, LAT), s["cu"], s["q"].shape[0]).to(torch.bfloat16)


def _plain_expanded(s):
    longest, most = s["longest"], s["most"]
    q, _ = _padded(s["q"], s["cu"], most)
    kv, there = _padded(s["kv"], s["cu_k"], longest)
    rope, _ = _padded(s["rope"], s["cu_k"], longest)
    k = torch.cat([kv[..., :NOPE], rope[:, :, None, :].expand(-1, -1, s["heads"], -1)], dim=-1)
    n, nk = s["cu"][1:] - s["cu"][:-1], s["cu_k"][1:] - s["cu_k"][:-1]
    last = nk[:, None] - n[:, None] + torch.arange(most, device=DEV)[None, :]
    seen = (torch.arange(longest, device=DEV)[None, None, :] <= last[:, :, None]) & there[:, None, :]
    o = _attend((q.transpose(1, 2) * SCALE) @ k.permute(0, 2, 3, 1), seen[:, None], kv[..., NOPE:].transpose(1, 2))
    return _back(o.transpose(1, 2), s["cu"], s["q"].shape[0]).to(torch.bfloat16)


_plain = {"tables": _plain_tables, "write": _plain_write, "absorbed": _plain_absorbed, "expanded": _plain_expanded}


# ------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    """out[row][head] = sum_t softmax_t(scale q . k_t) v_t over the keys that the row sees, one sequence at a
    time; the written cache is a copy, and the tables are whole numbers."""
    c = case
    if c["op"] == "tables":
        return None
    s = prepare(case, seed)
    if c["op"] == "write":
        t = c["tokens"]
        rows = torch.cat([s["latent"][:t], s["rope"][:t]], dim=1).double()
        return s["cache"].double().view(-1, KD).index_copy(0, s["slots"][:t], rows).view(s["cache"].shape)
    lens, new = _lens(c)
    out, row, key = [], 0, 0
    for i, (n, r) in enumerate(zip(lens, new)):
        limit = torch.arange(n - r, n, device=DEV)
        hidden = (torch.arange(n, device=DEV)[None, :] > limit[:, None])[:, None, :]
        if c["op"] == "absorbed":
            pages = s["tables"][i, :-(-n // BS)].long()
            x = torch.index_select(s["cache"], 0, pages).reshape(-1, KD)[:n].double()
            a = torch.einsum("rhd,nd->rhn", s["q"][row:row + r].double(), x) * SCALE
            w = torch.softmax(a.masked_fill(hidden, -math.inf), dim=-1)
            out.append(torch.einsum("rhn,nd->rhd", w, x[:, :LAT]))
        else:
            # a few heads at a time
            parts, step = [], max(1, int(4e8 / max(1, r * n)))
            both = s["kv"][key:key + n].double()
            shared = s["rope"][key:key + n].double()
            for h0 in range(0, c["heads"], step):
                q = s["q"][row:row + r, h0:h0 + step].double()
                a = torch.einsum("rhd,nhd->rhn", q[..., :NOPE], both[:, h0:h0 + step, :NOPE])
                a = (a + torch.einsum("rhd,nd->rhn", q[..., NOPE:], shared)) * SCALE
                w = torch.softmax(a.masked_fill(hidden, -math.inf), dim=-1)
                parts.append(torch.einsum("rhn,nhd->rhd", w, both[:, h0:h0 + step, NOPE:]))
            out.append(torch.cat(parts, dim=1))
        row, key = row + r, key + n
    return torch.cat(out)
