"""What is measured of a step of tree speculation over the paged cache: the plan of new tokens
(pages, slots, positions, tree masks) and its trim, the norm + rotation + append at given
positions and slots, the attention of drafted trees, and the acceptance with its move of the
accepted rows.

``run`` computes an operator in elementary torch operations, or, where ``own`` is set, through
the package's public entry points; ``exact`` computes it from its definition in 64 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
LAYER = 0


# ------------------------------------------------------------------- cases


def _plan(name, **kw):
    # shape: how a node finds its parent: "none" (no trees), "chain", "wide" (two children each),
    # "random" (any earlier node)
    case = dict(name=name, kind="plan", batch=8, new_min=8, new_max=8, prefix_min=16, prefix_max=800,
                block=16, shape="wide", words=1, pad=0, lengths=1)
    case.update(kw)
    return case


def _append(name, **kw):
    case = dict(name=name, kind="append", dtype="bf16", heads=32, kv_heads=8, head_dim=128, block=16,
                batch=8, new_min=8, new_max=8, prefix_min=0, prefix_max=1024, shape="wide", pad=0,
                lengths=1, norm=True, rotary=128, interleaved=False, base=10000.0, packed=True)
    case.update(kw)
    return case


def _tree(name, **kw):
    case = dict(name=name, kind="tree", dtype="bf16", heads=32, kv_heads=8, head_dim=128, block=16,
                batch=1, new_min=8, new_max=8, prefix_min=0, prefix_max=1024, shape="wide", words=1,
                blind=0.0, pad=0, lengths=1)
    case.update(kw)
    return case


def _accept(name, **kw):
    case = dict(name=name, kind="accept", dtype="bf16", layers=24, kv_heads=2, head_dim=64, block=16,
                batch=8, new_min=8, new_max=8, prefix_min=16, prefix_max=800, shape="wide",
                max_path=8, vocab=32000, right=0.8, pad=0, lengths=1)
    case.update(kw)
    return case


def listed():
    return [
        # a small batch's drafted trees get their pages and slots, and all are taken back: latency
        _plan("plan_b8x8"),
        # a large batch's trees, ragged, in a batch padded to a fixed number of rows
        _plan("plan_b256x64", batch=256, new_min=33, new_max=64, prefix_min=128, prefix_max=4096,
              shape="random", words=2, pad=200, lengths=2),
        # prompts admitted: the pages and slots of thousands of tokens each
        _plan("plan_prompts_b16", batch=16, new_min=500, new_max=4096, prefix_min=0, prefix_max=64,
              shape="none", words=0, lengths=3),
        # the trees of a batch on their way into the cache, behind contexts of usual lengths
        _append("append_b32x16", batch=32, new_min=5, new_max=16, pad=17, lengths=4),
        # large trees of a large batch at far positions, half of each head rotated, 32 bits
        _append("append_b64x64_f32", dtype="f32", batch=64, new_min=40, new_max=64, prefix_min=60000,
                prefix_max=129000, rotary=64, interleaved=True, base=500000.0, norm=False, block=32,
                packed=False, shape="random", lengths=5),
        # one sequence of a small model, a tree of eight: latency
        _tree("tree_b1x8_d64", heads=16, kv_heads=2, head_dim=64, prefix_min=500, prefix_max=500),
        # a batch's ragged trees over contexts of usual lengths, some rows padding
        _tree("tree_b8x25", batch=8, new_min=9, new_max=25, prefix_min=500, prefix_max=4000, blind=0.1,
              pad=5, lengths=6),
        # large trees of a serving batch: the most work
        _tree("tree_b32x64", batch=32, new_min=64, new_max=64, prefix_min=2000, prefix_max=8000,
              shape="random", words=2, lengths=7),
        # a few drafted tokens over long contexts: few rows, much cache
        _tree("tree_b2x9_long", batch=2, new_min=5, new_max=9, prefix_min=60000, prefix_max=100000,
              block=32, lengths=8),
        # small trees in 32 bits
        _tree("tree_b4x20_f32", dtype="f32", batch=4, heads=8, kv_heads=2, head_dim=64, new_min=0,
              new_max=20, prefix_max=1000, shape="random", lengths=9),
        # the drafts of a small batch decided, their rows moved: latency
        _accept("accept_b8x8"),
        # the same for large trees in a large model's cache
        _accept("accept_b64x64", layers=32, kv_heads=8, head_dim=128, batch=64, new_min=33, new_max=64,
                prefix_max=400, shape="random", max_path=16, right=0.9, pad=11, lengths=10),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        case = _draw(rng)
        w = work(case)
        if w["flops"] <= 1.4e11 and w["bytes"] <= 7.0e8 and _plain_bytes(case) <= 1.6e10:
            return case


def _draw(rng):
    kind = rng.choice(["plan", "append", "tree", "tree", "accept"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    head_dim = rng.choice([64, 128])
    block = rng.choice([16, 32])
    kv = rng.choice([1, 2, 4, 8])
    lengths = rng.randrange(1 << 20)
    shape = rng.choice(["chain", "wide", "random", "random"])
    most = _log_int(rng, 1, 128)
    pad = rng.choice([0, 0, _log_int(rng, 1, 64)])
    if kind == "plan":
        case = _plan("", batch=_log_int(rng, 1, 1024), new_min=rng.randint(0, most), new_max=most,
                     prefix_min=0, prefix_max=_log_int(rng, 1, 20000), block=block, shape=shape,
                     words=(most + 31) // 32, pad=pad, lengths=lengths)
        if rng.random() < 0.3:
            most = _log_int(rng, 1, max(1, 65536 // case["batch"]))
            case.update(shape="none", words=0, new_min=rng.randint(0, most), new_max=most)
    elif kind == "append":
        case = _append("", dtype=dtype, head_dim=head_dim, block=block, kv_heads=kv,
                       heads=kv * rng.choice([1, 2, 3, 4, 7, 8]), batch=_log_int(rng, 1, 128),
                       new_min=rng.randint(0, most), new_max=most,
                       prefix_max=_log_int(rng, 1, 130000), shape=shape, pad=pad, lengths=lengths,
                       norm=rng.random() < 0.6, rotary=16 * rng.randint(1, head_dim // 16),
                       interleaved=rng.random() < 0.5, base=rng.choice([10000.0, 500000.0]),
                       packed=rng.random() < 0.5)
    elif kind == "tree":
        lo = rng.choice([0, _log_int(rng, 1, 30000)])
        case = _tree("", dtype=dtype, head_dim=head_dim, block=block, kv_heads=kv,
                     heads=kv * rng.choice([1, 2, 3, 4, 5, 8, 16]), batch=_log_int(rng, 1, 48),
                     new_min=rng.randint(0, most), new_max=most, prefix_min=lo,
                     prefix_max=lo + _log_int(rng, 1, 4096), shape=shape, words=(most + 31) // 32,
                     blind=rng.choice([0.0, 0.0, 0.2]), pad=pad, lengths=lengths)
    else:
        case = _accept("", dtype=dtype, head_dim=head_dim, block=block, kv_heads=kv,
                       layers=rng.randint(1, 32), batch=_log_int(rng, 1, 96),
                       new_min=rng.randint(0, most), new_max=most, prefix_min=0,
                       prefix_max=_log_int(rng, 1, 800), shape=shape, max_path=rng.randint(1, 24),
                       vocab=rng.choice([8, 32000]), right=rng.choice([0.3, 0.7, 0.95]), pad=pad,
                       lengths=lengths)
    del case["name"]
    return case


# ------------------------------------------------------------------- sizes


def _cdiv(a, b):
    return -(-a // b)


def _new_and_cached(case):
    """New tokens and cached ones of every sequence."""
    r = random.Random(case["lengths"])
    new = [r.randint(case["new_min"], case["new_max"]) for _ in range(case["batch"])]
    cached = [r.randint(case["prefix_min"], case["prefix_max"]) for _ in new]
    if sum(new) == 0:
        new[0] = 1
    return new, cached


def _parents(case, new):
    """Every tree's parents (an index within the tree; -1: the root)."""
    r = random.Random(case["lengths"] + 1)
    if case["shape"] == "chain":
        return [list(range(-1, n - 1)) for n in new]
    if case["shape"] == "wide":
        return [[(i - 1) // 2 if i else -1 for i in range(n)] for n in new]
    return [[r.randrange(i) if i else -1 for i in range(n)] for n in new]


def _masks(case, trees):
    """Every row's mask (bit j: the tree's node j is seen) as a whole number."""
    r, out = random.Random(case["lengths"] + 2), []
    for tree in trees:
        seen = []
        for i, p in enumerate(tree):
            seen.append((seen[p] if p >= 0 else 0) | 1 << i)
        out += [0 if r.random() < case["blind"] else m for m in seen]
    return out


def _depths(tree):
    depth = []
    for p in tree:
        depth.append(depth[p] + 1 if p >= 0 else 0)
    return depth


def _elt(case):
    return 4 if case["dtype"] == "f32" else 2


def _token_bytes(case):
    """K and V of one token in all layers."""
    return 2 * case["layers"] * case["kv_heads"] * case["head_dim"] * _elt(case)


def _blocks(case):
    """Pages of the whole contexts."""
    new, cached = _new_and_cached(case)
    return sum(_cdiv(n + c, case["block"]) for n, c in zip(new, cached))


def _plain_bytes(case):
    """Roughly what the plain form holds at once."""
    new, cached = _new_and_cached(case)
    most = max(n + c for n, c in zip(new, cached))
    if case["kind"] == "tree":
        return case["batch"] * most * (case["heads"] * max(new) * 8 + case["kv_heads"] * case["head_dim"] * 12)
    if case["kind"] == "accept":
        return 3 * _blocks(case) * case["block"] * _token_bytes(case)
    return case["batch"] * _cdiv(most, case["block"]) * 40


def work(case):
    new, cached = _new_and_cached(case)
    tokens, kind, block = sum(new), case["kind"], case["block"]
    if kind == "plan":
        # pages popped and pushed: the stack's entry read and written, the table's written twice
        pages = sum(_cdiv(n + c, block) - _cdiv(c, block) for n, c in zip(new, cached))
        tree = 0 if case["shape"] == "none" else 4 + 4 * case["words"]
        return {"bytes": 16 * pages + 24 * len(new) + (12 + tree) * tokens, "flops": 0}
    if kind == "append":
        moved = tokens * (case["heads"] + 2 * case["kv_heads"]) * case["head_dim"] * _elt(case)
        return {"bytes": 2 * moved + 12 * tokens,
                "flops": tokens * (case["heads"] + case["kv_heads"]) * case["head_dim"] * 7}
    trees = _parents(case, new)
    if kind == "tree":
        row = case["head_dim"] * _elt(case)
        kv = sum(n + c for n, c in zip(new, cached) if n) * case["kv_heads"] * row * 2
        pairs = sum(n * c for n, c in zip(new, cached))
        pairs += sum(bin(m).count("1") for m in _masks(case, trees))
        return {"bytes": 2 * tokens * case["heads"] * row + kv + 4 * case["words"] * tokens,
                "flops": 4 * pairs * case["heads"] * case["head_dim"]}
    # accept: the rows that leave their places, as the tokens of seed 0 have it
    moved = 0
    for tree, (tokens_of, targets) in zip(trees, _drafts(case, trees, 0)):
        moved += sum(p != k for k, p in enumerate(_walk(tree, tokens_of, targets, case["max_path"])))
    return {"bytes": 2 * moved * _token_bytes(case) + 20 * tokens + 16 * len(new), "flops": 0}


# ------------------------------------------------------------------ inputs


def _drafts(case, trees, seed):
    """Every tree's drafted tokens, and the model's choice after each of its nodes: a child's
    token where the draft was right, any token where it was not."""
    r = random.Random(seed)
    out = []
    for tree in trees:
        tokens = [r.randrange(case["vocab"]) for _ in tree]
        children = [[] for _ in tree]
        for i, p in enumerate(tree):
            if p >= 0:
                children[p].append(i)
        targets = [tokens[r.choice(c)] if c and r.random() < case["right"] else r.randrange(case["vocab"])
                   for c in children]
        out.append((tokens, targets))
    return out


def _walk(tree, tokens, targets, most):
    """The accepted nodes: from the root to the first child that the model chose, and on."""
    path, at = [0] if tree else [], 0
    for i in range(1, len(tree)):  # (parents stand before their children)
        if len(path) < most and tree[i] == at and tokens[i] == targets[at]:
            path.append(i)
            at = i
    return path


def _frequencies(case):
    """Radians per position of each rotated pair, in 64 bits (a list)."""
    return [case["base"] ** (-2.0 * i / case["rotary"]) for i in range(case["rotary"] // 2)]


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(shape, dtype, g, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _starts(new):
    s = [0]
    for n in new:
        s.append(s[-1] + n)
    return s


def _flat(lists):
    return [x for row in lists for x in row]


def _tables(nblk, nb, maxb, seed):
    """Distinct random pages for every sequence, -1 past them; and the pages left over."""
    ids = torch.randperm(nb, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    tables, at = torch.full((len(nblk), maxb), -1, dtype=torch.int32), 0
    for row, n in enumerate(nblk):
        tables[row, :n] = ids[at:at + n]
        at += n
    return tables, ids[at:]


def _plan_inputs(case, seed):
    new, cached = _new_and_cached(case)
    block, words, total = case["block"], case["words"], sum(new) + case["pad"]
    nblk = [_cdiv(c, block) for c in cached]
    nb = _blocks(case) + 5
    maxb = max(1, max(_cdiv(n + c, block) for n, c in zip(new, cached)))
    tables, left = _tables(nblk, nb, maxb, seed)
    stack = torch.full((nb + 1,), -1, dtype=torch.int32)
    stack[0] = len(left)
    stack[1:1 + len(left)] = left
    trees = None if case["shape"] == "none" else _parents(case, new)
    parents = None if trees is None else _ints(_flat(trees) + [-1] * case["pad"])
    depth = 0 if trees is None else 1 + max(max(_depths(t), default=0) for t in trees)
    blank = lambda shape, dtype: torch.zeros(shape, dtype=dtype, device="cuda")  # noqa: E731
    return {"case": case, "stack": stack.cuda(), "tables": tables.cuda(), "cached": _ints(cached),
            "new": _ints(new), "parents": parents, "total": total, "depth": depth,
            "lens": blank(len(new), torch.int32), "starts": blank(len(new) + 1, torch.int32),
            "slots": blank(total, torch.int64), "positions": blank(total, torch.int32),
            "masks": blank((total, words), torch.int32) if words else None}


def _append_inputs(case, seed):
    g, dt = _generator(seed), DTYPES[case["dtype"]]
    new, cached = _new_and_cached(case)
    h, kv, d, b = case["heads"], case["kv_heads"], case["head_dim"], case["block"]
    total, tokens = sum(new) + case["pad"], sum(new)
    # pages for the new tokens only, which the slots name
    nblk = [_cdiv(n + c, b) - c // b for n, c in zip(new, cached)]
    nb = sum(nblk) + 4
    tables, _ = _tables(nblk, nb, max(1, max(nblk)), seed)
    rows, slots, positions = tables.tolist(), [], []
    for row, n, c, tree in zip(rows, new, cached, _parents(case, new)):
        slots += [row[p // b - c // b] * b + p % b for p in range(c, c + n)]
        positions += [c + x for x in _depths(tree)]
    pool = _normal((nb, 2, 1, kv, b, d), dt, g)
    if case["packed"]:
        qkv = _normal((total, h + 2 * kv, d), dt, g)
        q, k, v = qkv[:, :h], qkv[:, h:h + kv], qkv[:, h + kv:]
    else:
        q, k, v = (_normal((total, n, d), dt, g) for n in (h, kv, kv))
    weights = [None, None]
    if case["norm"]:
        weights = [(1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dt) for _ in range(2)]
    return {"case": case, "pool": pool, "q": q, "k": k, "v": v, "q_weight": weights[0],
            "k_weight": weights[1], "tokens": tokens,
            "slots": torch.tensor(slots + [-1] * case["pad"], dtype=torch.int64, device="cuda"),
            "positions": _ints(positions + [0] * case["pad"]),
            "out": torch.zeros((total, h, d), dtype=dt, device="cuda"),
            "freq": torch.tensor(_frequencies(case), dtype=torch.float64, device="cuda")}


def _tree_inputs(case, seed):
    g, dt = _generator(seed), DTYPES[case["dtype"]]
    new, cached = _new_and_cached(case)
    h, kv, d, b = case["heads"], case["kv_heads"], case["head_dim"], case["block"]
    total, words = sum(new) + case["pad"], case["words"]
    nblk = [_cdiv(n + c, b) for n, c in zip(new, cached)]
    nb = sum(nblk) + 2
    tables, _ = _tables(nblk, nb, max(1, max(nblk)), seed)
    bits = _masks(case, _parents(case, new)) + [0] * case["pad"]
    words_of = [[(m >> 32 * w) & 0xffffffff for w in range(words)] for m in bits]
    masks = torch.tensor(words_of, dtype=torch.int64).to(torch.int32).cuda()
    pool = _normal((nb, 2, 1, kv, b, d), dt, g)
    # scores spread over a few units, as those of trained heads are
    q = _normal((total, h, d), dt, g, 1.5)
    return {"case": case, "pool": pool, "q": q, "tables": tables.cuda(),
            "lens": _ints([n + c for n, c in zip(new, cached)]), "starts": _ints(_starts(new)),
            "masks": masks, "scale": d ** -0.5, "new_max": max(new), "out": torch.zeros_like(q)}


def _accept_inputs(case, seed):
    g, dt = _generator(seed), DTYPES[case["dtype"]]
    new, cached = _new_and_cached(case)
    b, total = case["block"], sum(new) + case["pad"]
    nblk = [_cdiv(n + c, b) for n, c in zip(new, cached)]
    nb = sum(nblk) + 2
    tables, _ = _tables(nblk, nb, max(1, max(nblk)), seed)
    rows, slots = tables.tolist(), []
    for row, n, c in zip(rows, new, cached):
        slots += [row[p // b] * b + p % b for p in range(c, c + n)]
    trees = _parents(case, new)
    drafts = _drafts(case, trees, seed)
    pad = [-1] * case["pad"]
    blank = lambda *shape: torch.zeros(shape, dtype=torch.int32, device="cuda")  # noqa: E731
    return {"case": case, "slots": torch.tensor(slots + pad, dtype=torch.int64, device="cuda"),
            "pool": _normal((nb, 2, case["layers"], case["kv_heads"], b, case["head_dim"]), dt, g),
            "parents": _ints(_flat(trees) + pad), "tokens": _ints(_flat(t for t, _ in drafts) + pad),
            "targets": _ints(_flat(t for _, t in drafts) + pad),
            "lens": _ints([n + c for n, c in zip(new, cached)]), "starts": _ints(_starts(new)),
            "counts": blank(len(new)), "nodes": blank(len(new), case["max_path"]),
            "next_tokens": blank(len(new)), "next_lens": blank(len(new))}


_INPUTS = {"plan": _plan_inputs, "append": _append_inputs, "tree": _tree_inputs,
           "accept": _accept_inputs}


def prepare(case, seed):
    s = _INPUTS[case["kind"]](case, seed)
    if own:
        from paged_kv_cache_239_gb300.pool import BlockPool
        from paged_kv_cache_239_gb300.rope import Rope

        if case["kind"] == "plan":  # (the plan touches no page: a pool of small ones)
            s["pool"] = torch.zeros((s["stack"].shape[0] - 1, 2, 1, 1, case["block"], 64),
                                    dtype=torch.bfloat16, device="cuda")
        nb, _, layers, kv, block, d = s["pool"].shape
        s["cache"] = BlockPool(nb, block, layers, kv, d, tensor=s["pool"])
        if case["kind"] == "plan":
            s["cache"].device_stack()  # the pages are the device's to give
        if case["kind"] == "append":
            s["rope"] = Rope(case["rotary"], base=case["base"], interleaved=case["interleaved"])
        if case["kind"] == "tree":
            need = s["cache"].tree_workspace_size(s["lens"].shape[0], s["q"].shape[0], case["heads"],
                                                  s["tables"].shape[1])
            s["workspace"] = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    return s


# --------------------------------------------------------------------- run


def run(s):
    kind = s["case"]["kind"]
    return (_RUN_OWN if own else _RUN_PLAIN)[kind](s)


_PLANNED = ("lens", "starts", "slots", "positions", "masks", "tables", "stack")
_ACCEPTED = ("counts", "nodes", "next_tokens", "next_lens", "pool")


def _named(s, names):
    return {n: s[n] for n in names if s[n] is not None}


def _own_plan(s):
    s["cache"].device_plan_tokens(s["stack"], s["tables"], s["cached"], s["new"], s["total"],
                                  parents=s["parents"], context_lens=s["lens"],
                                  query_starts=s["starts"], slots=s["slots"],
                                  positions=s["positions"], tree_masks=s["masks"])
    # every draft is refused: the pages go back
    s["cache"].device_trim_sequences(s["stack"], s["tables"], s["lens"], s["cached"])
    return _named(s, _PLANNED)


def _own_append(s):
    s["cache"].norm_rope_write_kv_slots(LAYER, s["q"], s["k"], s["v"], s["positions"], s["slots"],
                                        rope=s["rope"], q_weight=s["q_weight"],
                                        k_weight=s["k_weight"], eps=EPS, out=s["out"])
    return {"q": s["out"], "pool": s["pool"]}


def _own_tree(s):
    return s["cache"].tree_attention(s["q"], LAYER, s["tables"], s["lens"], s["starts"], s["masks"],
                                     s["scale"], out=s["out"], workspace=s["workspace"])


def _own_accept(s):
    s["cache"].device_accept_tree(s["slots"], s["parents"], s["tokens"], s["targets"], s["lens"],
                                  s["starts"], s["case"]["max_path"], counts=s["counts"],
                                  nodes=s["nodes"], next_tokens=s["next_tokens"],
                                  next_lens=s["next_lens"])
    return _named(s, _ACCEPTED)


def _places(starts, total):
    """Sequence of every row (the batch's size for rows behind the last one), and its index."""
    t = torch.arange(total, device=starts.device)
    seq = torch.searchsorted(starts[1:].contiguous(), t, right=True)
    return seq, t - torch.cat((starts, starts[-1:]))[seq]


def _plain_plan(s):
    block, stack, tables, total = s["case"]["block"], s["stack"], s["tables"], s["total"]
    cached, new = s["cached"].long(), s["new"].long()
    batch, maxb = tables.shape
    lens = cached + new
    s["lens"].copy_(lens)
    starts = torch.cat((new.new_zeros(1), new.cumsum(0)))
    s["starts"].copy_(starts)
    # pages from the stack's top, in increasing order of sequence and block
    first, last = (cached + block - 1) // block, (lens + block - 1) // block
    base = (last - first).cumsum(0) - (last - first)
    j = torch.arange(maxb, device=tables.device)
    taken = (j >= first[:, None]) & (j < last[:, None])
    rank = base[:, None] + j - first[:, None]
    ids = stack[(stack[0] - rank).clamp(min=0, max=stack.shape[0] - 1)]
    tables.copy_(torch.where(taken, ids, tables))
    stack[0] -= taken.sum()
    # where every token goes
    seq, i = _places(starts, total)
    there = seq < batch
    seq = seq.clamp(max=batch - 1)
    at = cached[seq] + i
    page = tables[seq, (at // block).clamp(max=maxb - 1)].long()
    s["slots"].copy_(torch.where(there, page * block + at % block, -1))
    if s["parents"] is None:
        s["positions"].copy_(torch.where(there, at, 0))
    else:
        # the ancestors of all rows, a generation at a time
        words = s["masks"].shape[1]
        masks = torch.zeros((total, words), dtype=torch.int64, device=tables.device)
        node, depth = torch.where(there, i, -1), torch.zeros_like(i)
        for _ in range(s["depth"]):
            up = node >= 0
            bit = torch.where(up, torch.ones_like(node) << node.clamp(min=0) % 32, 0)
            masks.scatter_add_(1, (node.clamp(min=0) // 32)[:, None], bit[:, None])
            node = torch.where(up, s["parents"][(starts[seq] + node).clamp(min=0)].long(), -1)
            depth += node >= 0
        s["masks"].copy_(masks.to(torch.int32))
        s["positions"].copy_(torch.where(there, cached[seq] + depth, 0))
    # the trim: the pages past the cached tokens go back, the last one taken first
    push = torch.where(taken, stack[0] + (last - first).sum() - rank, stack.shape[0])
    grown = torch.cat((stack, stack.new_zeros(1)))
    grown[push.view(-1)] = tables.view(-1)
    stack.copy_(grown[:-1])
    stack[0] += taken.sum()
    tables.masked_fill_(taken, -1)
    return _named(s, _PLANNED)


def _norm_rotate(x, weight, cos, sin, rotary, interleaved):
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()
    rot, rest = x[..., :rotary], x[..., rotary:]
    if interleaved:
        a, b = rot[..., 0::2], rot[..., 1::2]
        rot = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = rot[..., :rotary // 2], rot[..., rotary // 2:]
        rot = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((rot, rest), -1)


def _plain_append(s):
    case, pool, n = s["case"], s["pool"], s["tokens"]
    angle = s["positions"][:n].double()[:, None, None] * s["freq"]
    args = (angle.cos().float(), angle.sin().float(), case["rotary"], case["interleaved"])
    s["out"][:n] = _norm_rotate(s["q"][:n], s["q_weight"], *args).to(pool.dtype)
    k = _norm_rotate(s["k"][:n], s["k_weight"], *args).to(pool.dtype)
    page, row = s["slots"][:n] // case["block"], s["slots"][:n] % case["block"]
    pool[:, 0, LAYER][page, :, row] = k
    pool[:, 1, LAYER][page, :, row] = s["v"][:n]
    return {"q": s["out"], "pool": pool}


def _plain_tree(s):
    case, q = s["case"], s["q"]
    kv, d, new_max = case["kv_heads"], case["head_dim"], s["new_max"]
    group, batch = case["heads"] // kv, s["lens"].shape[0]
    lens, starts = s["lens"].long(), s["starts"].long()
    pages = s["pool"][s["tables"].long().clamp(min=0), :, LAYER]  # [b, blocks, 2, kv, B, d]
    pages = pages.permute(2, 0, 3, 1, 4, 5).flatten(3, 4).float()
    i = torch.arange(new_max, device=q.device)
    cached = lens - (starts[1:] - starts[:-1])
    token = (starts[:-1, None] + i).clamp(max=q.shape[0] - 1)
    x = q[token].float().view(batch, new_max, kv, group, d).permute(0, 2, 3, 1, 4)
    scores = torch.matmul(x.reshape(batch, kv, group * new_max, d), pages[0].transpose(-1, -2))
    scores = scores.mul_(s["scale"]).view(batch, kv, group, new_max, -1)
    # a row sees the cached tokens and the nodes of its mask
    t = torch.arange(scores.shape[-1], device=q.device)
    node = (t - cached[:, None]).clamp(min=0, max=32 * case["words"] - 1)          # [b, t]
    word = s["masks"][token].gather(2, (node // 32)[:, None].expand(-1, new_max, -1))
    bit = (word >> (node % 32)[:, None].to(torch.int32)) & 1
    inside = (t < lens[:, None])[:, None]
    seen = ((t < cached[:, None])[:, None] | (bit != 0)) & inside
    scores.masked_fill_(~seen[:, None, None], float("-inf"))
    top = scores.amax(-1, keepdim=True).clamp(min=-1e30)
    p = scores.sub_(top).exp_()
    sums = p.sum(-1, keepdim=True)
    v = pages[1].masked_fill((t >= lens[:, None])[:, None, :, None], 0.0)
    o = torch.matmul(p.view(batch, kv, group * new_max, -1), v).view(batch, kv, group, new_max, d)
    o = (o / sums.clamp(min=1e-30)).permute(0, 3, 1, 2, 4).reshape(batch, new_max, -1, d)
    seq, at = _places(starts, q.shape[0])
    there = seq < batch
    rows = o[seq.clamp(max=batch - 1), at.clamp(max=new_max - 1)].to(q.dtype)
    return s["out"].copy_(torch.where(there[:, None, None], rows, s["out"]))


def _plain_accept(s):
    case, pool, parents = s["case"], s["pool"], s["parents"].long()
    block, most = case["block"], case["max_path"]
    starts, batch, total = s["starts"].long(), s["lens"].shape[0], s["parents"].shape[0]
    seq, i = _places(starts, total)
    there = (seq < batch) & (i > 0) & (parents >= 0)
    seq = seq.clamp(max=batch - 1)
    up = (starts[seq] + parents).clamp(min=0, max=total - 1)
    match = there & (s["tokens"] == s["targets"][up])
    new = starts[1:] - starts[:-1]
    node = torch.where(new > 0, 0, -1)
    path, last = [node], node
    for _ in range(most - 1):
        step = match & (parents == node[seq])
        found = torch.full((batch,), total, dtype=torch.long, device=seq.device)
        found = found.scatter_reduce(0, seq, torch.where(step, i, total), "amin")
        node = torch.where((found < total) & (node >= 0), found, -1)
        last = torch.where(node >= 0, node, last)
        path.append(node)
    nodes = torch.stack(path, 1)
    count = (nodes >= 0).sum(1)
    s["nodes"].copy_(nodes)
    s["counts"].copy_(count)
    after = s["targets"][(starts[:-1] + last).clamp(min=0, max=total - 1)]
    s["next_tokens"].copy_(torch.where(new > 0, after, -1))
    s["next_lens"].copy_(s["lens"] - new + count)
    # the accepted rows close up behind the cached ones
    k = torch.arange(most, device=nodes.device).expand(batch, -1)
    moves = nodes > k
    first = starts[:-1, None].expand(-1, most)[moves]
    src, dst = s["slots"][first + nodes[moves]], s["slots"][first + k[moves]]
    pool[dst // block, :, :, :, dst % block] = pool[src // block, :, :, :, src % block]
    return _named(s, _ACCEPTED)


_RUN_PLAIN = {"plan": _plain_plan, "append": _plain_append, "tree": _plain_tree,
              "accept": _plain_accept}
_RUN_OWN = {"plan": _own_plan, "append": _own_append, "tree": _own_tree, "accept": _own_accept}


# ------------------------------------------------------------------- exact


def exact(case, seed):
    s = _INPUTS[case["kind"]](case, seed)
    return {"plan": _exact_plan, "append": _exact_append, "tree": _exact_tree,
            "accept": _exact_accept}[case["kind"]](case, s)


def _exact_plan(case, s):
    """The allocator's own steps: one page after another from the end of a list."""
    (new, cached), block = _new_and_cached(case), case["block"]
    tables, stack = s["tables"].tolist(), s["stack"].tolist()
    free = stack[1:1 + stack[0]]
    slots, positions, masks = [], [], []
    trees = [None] * len(new) if s["parents"] is None else _parents(case, new)
    for row, n, c, tree in zip(tables, new, cached, trees):
        for at in range(c, c + n):
            if at % block == 0:
                row[at // block] = free.pop()
            slots.append(row[at // block] * block + at % block)
        positions += range(c, c + n) if tree is None else [c + x for x in _depths(tree)]
        for i in range(n if tree is not None else 0):
            up, bits = i, 0
            while up >= 0:
                bits, up = bits | 1 << up, tree[up]
            masks.append([(bits >> 32 * w) & 0xffffffff for w in range(case["words"])])
    pad, blank = case["pad"], [[0] * case["words"]] * case["pad"]
    out = {"lens": _ints([n + c for n, c in zip(new, cached)]), "starts": _ints(_starts(new)),
           "slots": torch.tensor(slots + [-1] * pad, dtype=torch.int64, device="cuda"),
           "positions": _ints(positions + [0] * pad), "tables": s["tables"], "stack": s["stack"]}
    if s["masks"] is not None:
        out["masks"] = torch.tensor(masks + blank, dtype=torch.int64).to(torch.int32).cuda()
    return out


def _exact_append(case, s):
    """Each pair a complex number, turned by e^(i p f), token by token into its slot."""
    n, r = s["tokens"], case["rotary"]
    q_out, pool = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda"), s["pool"].double()
    angle = s["positions"][:n].double()[:, None, None] * s["freq"]
    turn = torch.polar(torch.ones_like(angle), angle)
    done = []
    for x, w in ((s["q"][:n], s["q_weight"]), (s["k"][:n], s["k_weight"])):
        x = x.double()
        if w is not None:
            x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w.double()
        if case["interleaved"]:
            z = torch.view_as_complex(x[..., :r].reshape(*x.shape[:2], r // 2, 2).contiguous())
            x[..., :r] = torch.view_as_real(z * turn).reshape(*x.shape[:2], r)
        else:
            z = torch.complex(x[..., :r // 2], x[..., r // 2:r]) * turn
            x[..., :r // 2], x[..., r // 2:r] = z.real, z.imag
        done.append(x)
    q_out[:n] = done[0]
    for t, slot in enumerate(s["slots"][:n].tolist()):
        page = pool[slot // case["block"], :, LAYER, :, slot % case["block"]]
        page[0], page[1] = done[1][t], s["v"][t].double()
    return {"q": q_out, "pool": pool}


def _exact_tree(case, s):
    """Head by head over the gathered keys, softmax by its definition."""
    new, cached = _new_and_cached(case)
    group = case["heads"] // case["kv_heads"]
    bits = _masks(case, _parents(case, new))
    out, start = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda"), 0
    for b, (n, c) in enumerate(zip(new, cached)):
        if n == 0:
            continue
        pages = s["tables"][b, :_cdiv(n + c, case["block"])].long()
        see = torch.tensor([[(m >> j) & 1 for j in range(n)] for m in bits[start:start + n]],
                           dtype=torch.bool, device="cuda")
        see = torch.cat((torch.ones((n, c), dtype=torch.bool, device="cuda"), see), 1)
        none = ~see.any(1)
        for kvh in range(case["kv_heads"]):
            kv = s["pool"][pages, :, LAYER, kvh].double()
            keys, values = (kv[:, x].reshape(-1, case["head_dim"])[:n + c] for x in range(2))
            x = s["q"][start:start + n, kvh * group:(kvh + 1) * group].double()
            z = torch.einsum("ngd,td->ngt", x, keys) * s["scale"]
            z = torch.where(see[:, None], z, float("-inf"))
            p = torch.where(none[:, None, None], 0.0, torch.softmax(z, -1))
            out[start:start + n, kvh * group:(kvh + 1) * group] = torch.einsum("ngt,td->ngd", p, values)
        start += n
    return out


def _exact_accept(case, s):
    """Tree by tree: the walk, and each accepted row in turn to its place."""
    new, cached = _new_and_cached(case)
    pool, block = s["pool"].double(), case["block"]
    slots, tokens, targets = (s[n].tolist() for n in ("slots", "tokens", "targets"))
    counts, nodes, after, lens, start = [], [], [], [], 0
    for n, c, tree in zip(new, cached, _parents(case, new)):
        path = _walk(tree, tokens[start:start + n], targets[start:start + n], case["max_path"])
        for k, p in enumerate(path):
            a, z = slots[start + p], slots[start + k]
            if a != z:
                pool[z // block, :, :, :, z % block] = pool[a // block, :, :, :, a % block]
        counts.append(len(path))
        nodes.append(path + [-1] * (case["max_path"] - len(path)))
        after.append(targets[start + path[-1]] if path else -1)
        lens.append(c + len(path))
        start += n
    return {"counts": _ints(counts), "nodes": _ints(nodes), "next_tokens": _ints(after),
            "next_lens": _ints(lens), "pool": pool}
