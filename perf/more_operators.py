"""Cases that measure decode attention over a shared prefix and the calls that make
and keep such prefixes: forks of sequences, copies of blocks, and the rewriting of
block tables after blocks have moved.

Sequences that begin with the same tokens (samples of one prompt, requests behind
one system prompt, questions about one document) hold those tokens' blocks in
common.  The attention call takes the sequences in groups with a prefix each,
attends the prefix once for all rows of its group, each sequence's own tail for
itself, and joins the two by their softmax sums; the result is what decode
attention over each whole context gives.

``run`` computes an operator in plain torch operations (32-bit arithmetic, one
rounding at the end) or, with ``own`` set, through the library's calls.
``exact`` gives the same results in 64 bits, sequence by sequence.
"""
import math

import torch

own = False

D, BS = 128, 16
SCALE = D ** -0.5
DEV = "cuda"


# ------------------------------------------------------------------- the cases
# attention: `seqs` sequences in `groups` groups (`loose` more of them share nothing), `q` rows each; a group's
# prefix has p_lo .. p_hi tokens, and a sequence own_lo .. own_hi of its own behind it
def listed():
    return [
        # four samples of one short prompt: latency
        {"name": "samples-one", "op": "attend", "seqs": 4, "groups": 1, "loose": 0, "kv": 2, "per": 4, "q": 1,
         "p_lo": 300, "p_hi": 300, "own_lo": 5, "own_hi": 90, "fp8": False},
        # the requests of one system prompt, each with a long conversation of its own behind it
        {"name": "system-prompt", "op": "attend", "seqs": 128, "groups": 1, "loose": 0, "kv": 8, "per": 8, "q": 1,
         "p_lo": 2000, "p_hi": 2000, "own_lo": 1024, "own_hi": 16384, "fp8": False},
        # many short questions about one long document
        {"name": "document", "op": "attend", "seqs": 64, "groups": 1, "loose": 0, "kv": 8, "per": 8, "q": 1,
         "p_lo": 32768, "p_hi": 32768, "own_lo": 20, "own_hi": 1000, "fp8": False},
        # prompts with eight samples each, and a few requests that share nothing
        {"name": "samples-many", "op": "attend", "seqs": 128, "groups": 16, "loose": 5, "kv": 8, "per": 4, "q": 1,
         "p_lo": 500, "p_hi": 4001, "own_lo": 10, "own_hi": 500, "fp8": False},
        # two tenants' prompts over an fp8 cache
        {"name": "tenants-fp8", "op": "attend", "seqs": 48, "groups": 2, "loose": 0, "kv": 8, "per": 8, "q": 1,
         "p_lo": 4099, "p_hi": 8192, "own_lo": 100, "own_hi": 2500, "fp8": True},
        # speculative drafts of four tokens behind a shared prompt
        {"name": "drafts", "op": "attend", "seqs": 32, "groups": 2, "loose": 1, "kv": 8, "per": 4, "q": 4,
         "p_lo": 2500, "p_hi": 6000, "own_lo": 200, "own_hi": 2000, "fp8": False},
        # the partial last blocks of a prompt's samples, one layer
        {"name": "copy-layer", "op": "copy", "caches": 2, "blocks": 127, "kv": 8, "from": 1},
        # blocks of every layer, moved in one call
        {"name": "copy-layers", "op": "copy", "caches": 32, "blocks": 512, "kv": 8, "from": 512},
        # one prompt, sampled
        {"name": "fork-prompt", "op": "fork", "parents": 1, "children": 16, "width": 64, "lo": 1000, "hi": 1000, "keep": False},
        # a step of beam search over a large batch
        {"name": "fork-beams", "op": "fork", "parents": 1024, "children": 1024, "width": 512, "lo": 5, "hi": 8192, "keep": True},
        # a few blocks moved under a small batch
        {"name": "remap-few", "op": "remap", "seqs": 16, "width": 256, "lo": 100, "hi": 4096, "moves": 9},
        # a pool compacted under a large batch
        {"name": "remap-pool", "op": "remap", "seqs": 512, "width": 2048, "lo": 1024, "hi": 32768, "moves": 8192},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "attend", "copy", "fork", "remap"])
    if op == "copy":
        kv, caches, blocks = rng.choice([1, 2, 4, 8]), _log(rng, 1, 48), _log(rng, 1, 2048)
        while caches * blocks * kv > 32 * 512 * 8:
            blocks = max(1, blocks // 2)
        return {"op": op, "caches": caches, "blocks": blocks, "kv": kv, "from": rng.choice([1, rng.randint(1, blocks), blocks])}
    if op == "fork":
        width = _log(rng, 1, 512)
        hi = rng.randint(0, width * BS)
        return {"op": op, "parents": _log(rng, 1, 1024), "children": _log(rng, 1, 1024), "width": width,
                "lo": rng.randint(0, hi), "hi": hi, "keep": rng.random() < 0.5}
    if op == "remap":
        width = _log(rng, 1, 2048)
        hi = rng.randint(0, width * BS)
        seqs = _log(rng, 1, 512)
        return {"op": op, "seqs": seqs, "width": width, "lo": rng.randint(0, hi), "hi": hi,
                "moves": _log(rng, 1, max(1, min(8192, seqs * hi // 32)))}
    kv, per, q = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8, 8, 16]), rng.choice([1, 1, 1, 2, 4, 7])
    seqs = _log(rng, 1, 256)
    groups = min(seqs, _log(rng, 1, 32))
    loose = rng.choice([0, 0, rng.randint(0, 8)])
    # (no more keys, counted for each sequence, and no more operations than the largest listed case)
    room = min(128 * 18384 * 8 // ((seqs + loose) * kv), 128 * 18384 * 64 // ((seqs + loose) * kv * per * q), 32768 + 1000)
    p_hi = min(32768, rng.choice([_log(rng, 1, room), room // 2, rng.randint(0, 40)]))
    own_hi = _log(rng, q, max(q, min(16384, room - p_hi)))
    return {"op": op, "seqs": seqs, "groups": groups, "loose": loose, "kv": kv, "per": per, "q": q,
            "p_lo": rng.randint(p_hi // 4, p_hi), "p_hi": p_hi, "own_lo": rng.randint(q, own_hi), "own_hi": own_hi,
            "fp8": rng.random() < 0.3}


def _spread(n, lo, hi, step=7):
    """n numbers between lo and hi, both reached where n > 1, in no order."""
    return [hi if n == 1 else lo + (hi - lo) * ((i * step + n // 2) % n) // (n - 1) for i in range(n)]


def _groups(c):
    """Sequences before each group's end, each group's prefix, and each sequence's (group, prefix, context)."""
    n, ng = c["seqs"], c["groups"]
    ends = [n * (i + 1) // ng for i in range(ng)]
    pre = _spread(ng, c["p_lo"], c["p_hi"], 5)
    tails = _spread(n + c["loose"], c["own_lo"], c["own_hi"])
    seqs, g = [], 0
    for i in range(n):
        while i >= ends[g]:
            g += 1
        seqs.append((g, pre[g], pre[g] + tails[i]))
    return ends, pre, seqs + [(-1, 0, t) for t in tails[n:]]


def work(case):
    c = case
    if c["op"] == "copy":
        block = c["kv"] * BS * D * 2
        return {"bytes": c["caches"] * (c["blocks"] + c["from"]) * block + 8 * c["blocks"], "flops": 0}
    if c["op"] == "fork":
        lens = _parent_lens(c)
        moved = sum(-(-lens[p] // BS) for p in _parents(c))
        read = sum(-(-lens[p] // BS) for p in set(_parents(c)))
        return {"bytes": 4 * (moved + read + 5 * c["children"] + c["parents"]), "flops": 0}
    if c["op"] == "remap":
        lens = _spread(c["seqs"], c["lo"], c["hi"])
        return {"bytes": 4 * (sum(-(-x // BS) for x in lens) + c["seqs"] + 3 * c["moves"]), "flops": 0}
    ends, pre, seqs = _groups(c)
    q, h = c["q"], c["kv"] * c["per"]
    tokens = sum(p // BS * BS for p in pre) + sum(n - p // BS * BS for _, p, n in seqs)
    seen = sum((n - q) * q + q * (q + 1) // 2 for _, _, n in seqs)
    return {"bytes": tokens * c["kv"] * D * 2 * (1 if c["fp8"] else 2) + len(seqs) * q * h * D * 4 + 4 * tokens // BS,
            "flops": 4 * h * D * seen}


# ------------------------------------------------------------------- the inputs
def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _parent_lens(c):
    return _spread(c["parents"], c["lo"], c["hi"])


def _parents(c):
    """Each child's parent: in beam search some sequences go on more than once, and some not at all."""
    n = c["parents"]
    return [(i * i // 3 + i) % n for i in range(c["children"])]


def _some_tables(lens, width, blocks, g):
    """Rows of distinct blocks, as many as each length needs, and -1 behind them."""
    need = torch.tensor([-(-x // BS) for x in lens], device=DEV)
    at = torch.arange(width, device=DEV)[None, :]
    ids = torch.randperm(blocks, generator=g, device=DEV)
    idx = (need.cumsum(0) - need)[:, None] + at
    return torch.where(at < need[:, None], ids[idx.clamp(max=blocks - 1)], -1).to(torch.int32).contiguous()


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    st = {"op": c["op"]}
    if c["op"] == "copy":
        nb = c["blocks"] + c["from"] + 5
        pool = torch.randn(c["caches"], nb, c["kv"], BS, D, generator=g, device=DEV, dtype=torch.bfloat16)
        ids = torch.randperm(nb, generator=g, device=DEV).to(torch.int32)
        at = torch.arange(c["blocks"], device=DEV) % c["from"]
        st |= {"pool": pool, "caches": list(pool.unbind(0)), "src": ids[:c["from"]][at].contiguous(),
               "dst": ids[c["from"]:c["from"] + c["blocks"]].contiguous()}
        return st
    if c["op"] == "fork":
        lens, n, w = _parent_lens(c), c["children"], c["width"]
        used = sum(-(-x // BS) for x in lens)
        nb = used + n + 3
        ids = torch.randperm(nb, generator=g, device=DEV).to(torch.int32)
        tables = _some_tables(lens, w, max(1, used), g)
        st |= {"tables": torch.where(tables >= 0, ids[tables.clamp(min=0).long()], -1).contiguous(), "lens": _i32(lens),
               "parents": _i32(_parents(c)), "free": ids[used:].contiguous(), "keep": c["keep"],
               "child_tables": torch.full((n, w), -1, dtype=torch.int32, device=DEV),
               "child_lens": torch.empty(n, dtype=torch.int32, device=DEV),
               "src": torch.empty(n, dtype=torch.int32, device=DEV), "dst": torch.empty(n, dtype=torch.int32, device=DEV),
               "taken": torch.empty(1, dtype=torch.int32, device=DEV)}
        return st
    if c["op"] == "remap":
        lens = _spread(c["seqs"], c["lo"], c["hi"])
        used = max(1, sum(-(-x // BS) for x in lens))
        moves = min(c["moves"], used)
        # the blocks of the pool's upper end move to holes at its lower end
        st |= {"tables": _some_tables(lens, c["width"], used, g), "lens": _i32(lens), "blocks": used + moves,
               "src": torch.arange(used - moves, used, dtype=torch.int32, device=DEV) + moves,
               "dst": torch.randperm(moves, generator=g, device=DEV).to(torch.int32)}
        st["tables"] += torch.where(st["tables"] >= 0, moves, 0).to(torch.int32)
        return st
    ends, pre, seqs = _groups(c)
    n, q, kv, h = len(seqs), c["q"], c["kv"], c["kv"] * c["per"]
    width = max(-(-x // BS) for _, _, x in seqs)
    # the prefix's whole blocks once a group, in every sharer's row, then each sequence's own
    shared = [p // BS for p in pre]
    starts = [sum(shared[:i]) for i in range(len(shared))]
    of = torch.tensor([max(0, s[0]) for s in seqs], device=DEV)
    held = torch.tensor([s[1] // BS for s in seqs], device=DEV)
    need = torch.tensor([-(-s[2] // BS) for s in seqs], device=DEV)
    at = torch.arange(width, device=DEV)[None, :]
    mine = need - held
    idx = sum(shared) + (mine.cumsum(0) - mine - held)[:, None] + at
    idx = torch.where(at < held[:, None], torch.tensor(starts, device=DEV)[of][:, None] + at, idx)
    nb = sum(shared) + int(mine.sum()) + 5
    order = torch.randperm(nb, generator=g, device=DEV)
    tables = torch.where(at < need[:, None], order[idx.clamp(0, nb - 1)], -1).to(torch.int32).contiguous()
    k, v = (torch.randn(nb, kv, BS, D, generator=g, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    st |= {"q": torch.randn(n * q, h, D, generator=g, device=DEV, dtype=torch.float32).to(torch.bfloat16),
           "tables": tables, "lens": _i32([s[2] for s in seqs]), "cu_groups": _i32([0] + ends), "prefix": _i32(pre),
           "cu": _i32([i * q for i in range(n + 1)]) if q > 1 else None, "rows": q, "kv": kv,
           "longest": max(s[2] for s in seqs), "most_shared": max(pre), "most_own": max(s[2] - s[1] // BS * BS for s in seqs),
           "out": torch.empty(n * q, h, D, dtype=torch.bfloat16, device=DEV), "k_scale": None, "v_scale": None}
    if c["fp8"]:
        for name, x in (("k", k), ("v", v)):
            scale = x.abs().amax(dim=(0, 2, 3)).float() / 448 * (0.5 + torch.rand(kv, generator=g, device=DEV))
            st[name + "_scale"] = scale.contiguous()
            st[name] = (x.float() / scale[None, :, None, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        st |= {"k": k, "v": v}
    return st


# ------------------------------------------------------------------- one pass
def run(state):
    return (_own if own else _plain)[state["op"]](state)


def _out_fork(s):
    return {"tables": s["child_tables"], "lens": s["child_lens"], "src": s["src"], "dst": s["dst"], "taken": s["taken"]}


def _own_copy(s):
    import paged_kv_cache_263_gb300 as pkv
    pkv.kv_copy_blocks(s["caches"], s["src"], s["dst"])
    return s["pool"]


def _own_fork(s):
    import paged_kv_cache_263_gb300 as pkv
    pkv.kv_fork_tables(s["tables"], s["lens"], s["parents"], s["free"], s["child_tables"], s["child_lens"], s["src"],
                       s["dst"], s["taken"], first_keeps=s["keep"])
    return _out_fork(s)


def _own_remap(s):
    import paged_kv_cache_263_gb300 as pkv
    pkv.kv_remap_tables(s["tables"], s["lens"], s["src"], s["dst"])
    return s["tables"]


def _own_attend(s):
    import paged_kv_cache_263_gb300 as pkv
    # (the program knows how long its prefixes and tails may get: they size the grids and the workspace)
    longest = {"max_prefix_len": s["most_shared"], "max_tail_len": s["most_own"]}
    if "workspace" not in s:   # kept by the program from call to call
        s["workspace"] = torch.empty(pkv.paged_attention_shared_prefix_workspace_size(
            s["lens"].numel(), s["q"].shape[0], s["rows"], s["prefix"].numel(), s["q"].shape[1], s["kv"],
            s["most_shared"], s["most_own"]), dtype=torch.uint8, device=DEV)
    return pkv.paged_attention_shared_prefix(
        s["out"], s["q"], s["k"], s["v"], s["tables"], s["lens"], s["cu_groups"], s["prefix"], cu_q_lens=s["cu"],
        max_q_len=s["rows"], scale=SCALE, k_scale=s["k_scale"], v_scale=s["v_scale"], workspace=s["workspace"], **longest)


_own = {"copy": _own_copy, "fork": _own_fork, "remap": _own_remap, "attend": _own_attend}


def _plain_copy(s):
    s["pool"][:, s["dst"].long()] = s["pool"][:, s["src"].long()]
    return s["pool"]


def _plain_fork(s):
    par, n = s["parents"].long(), s["parents"].numel()
    lens = s["lens"][par]
    need, partial = (lens + BS - 1) // BS, lens % BS != 0
    child = torch.arange(n, device=DEV)
    first = torch.full((s["lens"].numel(),), n, device=DEV).scatter_reduce(0, par, child, "amin")
    fresh = partial & (first[par] != child) if s["keep"] else partial
    place = fresh.cumsum(0)
    new = s["free"][(place - 1).clamp(min=0)]
    rows = s["tables"][par]
    last = rows.gather(1, (need.long() - 1).clamp(min=0)[:, None])[:, 0]
    at = torch.arange(rows.shape[1], device=DEV)[None, :]
    rows = torch.where(fresh[:, None] & (at == need[:, None] - 1), new[:, None], rows)
    s["child_tables"].copy_(torch.where(at < need[:, None], rows, s["child_tables"]))
    s["child_lens"].copy_(lens)
    s["src"].copy_(torch.where(fresh, last, -1))
    s["dst"].copy_(torch.where(fresh, new, -1))
    s["taken"].copy_(place[-1:])
    return _out_fork(s)


def _plain_remap(s):
    now = torch.arange(s["blocks"], dtype=torch.int32, device=DEV)
    now[s["src"].long()] = s["dst"]
    at = torch.arange(s["tables"].shape[1], device=DEV)[None, :]
    held = at < ((s["lens"] + BS - 1) // BS)[:, None]
    s["tables"].copy_(torch.where(held, now[s["tables"].clamp(min=0).long()], s["tables"]))
    return s["tables"]


def _plain_attend(s):
    lens, q, kv, n = s["lens"], s["rows"], s["kv"], s["lens"].numel()
    t = torch.arange(s["longest"], device=DEV)
    blocks = s["tables"].clamp(min=0)[:, :-(-s["longest"] // BS)].long()

    def keys(cache, scale):
        if scale is not None:
            x = cache.view(torch.float8_e4m3fn)[blocks].float() * scale[:, None, None]
        else:
            x = cache[blocks].float()
        return x.transpose(1, 2).reshape(n, kv, -1, D)[:, :, :s["longest"]]

    rows = s["q"].view(n, q, kv, -1, D).float().permute(0, 2, 1, 3, 4).reshape(n, kv, -1, D)
    a = (rows * SCALE) @ keys(s["k"], s["k_scale"]).transpose(2, 3)
    last = (lens[:, None] - q + torch.arange(q, device=DEV)[None, :]).repeat_interleave(rows.shape[2] // q, dim=1)
    a.masked_fill_((t[None, None, :] > last[:, :, None])[:, None], -math.inf)
    p = a.sub_(a.amax(-1, keepdim=True)).exp_()
    o = (p @ keys(s["v"], s["v_scale"])) / p.sum(-1, keepdim=True)
    s["out"].copy_(o.view(n, kv, q, -1, D).permute(0, 2, 1, 3, 4).reshape(s["out"].shape))
    return s["out"]


_plain = {"copy": _plain_copy, "fork": _plain_fork, "remap": _plain_remap, "attend": _plain_attend}


# ------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    """Copies are copies; out[row][head] = sum_t softmax_t(scale q . k_t) v_t over the keys that the row sees, one
    sequence and a few heads at a time; tables are whole numbers."""
    c = case
    if c["op"] in ("fork", "remap"):
        return None
    s = prepare(case, seed)
    if c["op"] == "copy":
        return s["pool"].double().index_copy(1, s["dst"].long(), torch.index_select(s["pool"], 1, s["src"].long()).double())
    q, kv, per = c["q"], c["kv"], c["per"]
    out = torch.empty(s["out"].shape, dtype=torch.float64, device=DEV)

    def whole(cache, scale, pages, n):
        x = torch.index_select(cache, 0, pages)
        x = x.view(torch.float8_e4m3fn).double() if scale is not None else x.double()
        x = x.transpose(0, 1).reshape(kv, -1, D)[:, :n]
        return x if scale is None else x * scale.double()[:, None, None]

    for i, n in enumerate(s["lens"].tolist()):
        pages = s["tables"][i, :-(-n // BS)].long()
        x = s["q"][i * q:(i + 1) * q].double().view(q, kv, per, D)
        a = torch.einsum("rkgd,knd->krgn", x, whole(s["k"], s["k_scale"], pages, n)) * SCALE
        hidden = torch.arange(n, device=DEV)[None, :] > torch.arange(n - q, n, device=DEV)[:, None]
        w = torch.softmax(a.masked_fill(hidden[None, :, None, :], -math.inf), dim=-1)
        o = torch.einsum("krgn,knd->rkgd", w, whole(s["v"], s["v_scale"], pages, n))
        out[i * q:(i + 1) * q] = o.reshape(q, kv * per, D)
    return out
