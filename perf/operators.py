"""What is measured of the serving operators around the paged cache: the norm + rotation +
append of new tokens, the attention of several new tokens per sequence over the cache, and
the page operations (copy, fork and free of shared pages, compaction).

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


def _append(name, **kw):
    case = dict(name=name, kind="append", dtype="bf16", heads=32, kv_heads=8, head_dim=128, block=16,
                batch=8, new_min=1, new_max=1, prefix_min=0, prefix_max=1024, lengths=1, norm=True,
                rotary=128, interleaved=False, base=10000.0, scaling="none", factor=1.0,
                original=4096, packed=True)
    case.update(kw)
    return case


def _prefill(name, **kw):
    case = dict(name=name, kind="prefill", dtype="bf16", heads=32, kv_heads=8, head_dim=128, block=16,
                batch=1, new_min=128, new_max=128, prefix_min=0, prefix_max=0, lengths=1)
    case.update(kw)
    return case


def _copy(name, **kw):
    case = dict(name=name, kind="copy", dtype="bf16", layers=8, kv_heads=8, head_dim=128, block=16,
                pairs=16)
    case.update(kw)
    return case


def _beam(name, **kw):
    case = dict(name=name, kind="beam", dtype="bf16", layers=8, kv_heads=8, head_dim=128, block=16,
                parents=8, width=3, len_min=16, len_max=800, lengths=1)
    case.update(kw)
    return case


def _compact(name, **kw):
    case = dict(name=name, kind="compact", dtype="bf16", layers=8, kv_heads=8, head_dim=128, block=16,
                batch=32, len_min=16, len_max=800, lengths=1, free_share=0.5)
    case.update(kw)
    return case


def listed():
    return [
        # one decode step of a small model's batch: a token per sequence, latency
        _append("append_decode_b32_d64", batch=32, heads=16, kv_heads=2, head_dim=64, rotary=64,
                prefix_min=15, prefix_max=799),
        # the prompts of a long-context batch: many tokens at far positions, half of each head
        # rotated in interleaved pairs with frequencies stretched by parts
        _append("append_prompt_8k_far", batch=8, new_min=700, new_max=1345, prefix_min=60000,
                prefix_max=129000, rotary=64, interleaved=True, base=500000.0, scaling="parts",
                factor=8.0, original=8192, block=32, lengths=3),
        # a ragged step in 32 bits without norms: separate q, k and v tensors
        _append("append_ragged_f32", dtype="f32", batch=64, heads=32, kv_heads=32, new_min=0,
                new_max=37, prefix_max=1024, norm=False, scaling="linear", factor=4.0, block=32,
                packed=False, lengths=5),
        # a few speculated tokens checked against long cached contexts: few rows, much cache
        _prefill("verify_5_long", batch=4, new_min=3, new_max=5, prefix_min=32763,
                 prefix_max=131000, block=32, lengths=7),
        # chunks of prompts behind cached prefixes in a small model's batch, odd lengths
        _prefill("chunk_b8_d64", batch=8, heads=16, kv_heads=2, head_dim=64, new_min=1,
                 new_max=513, prefix_min=0, prefix_max=800, lengths=9),
        # a whole prompt of 8192 tokens: the largest
        _prefill("prompt_8192", batch=1, new_min=8192, new_max=8192),
        # a small ragged batch in 32 bits
        _prefill("ragged_f32", dtype="f32", batch=4, heads=8, kv_heads=2, head_dim=64, new_min=0,
                 new_max=130, prefix_max=300, lengths=11),
        # copy-on-write of a handful of small pages: latency
        _copy("copy_16_small", layers=24, kv_heads=2, head_dim=64, pairs=16),
        # a prefix cache's pages duplicated in bulk
        _copy("copy_1024", pairs=1024),
        # a beam step of a small batch: the dropped rows are freed, the kept ones forked
        _beam("beam_8x3", layers=24, kv_heads=2, head_dim=64),
        # the same for 64 prompts with three samples each
        _beam("beam_64x3", parents=64, width=3, len_min=128, len_max=1024, lengths=2),
        # a half-empty pool defragmented
        _compact("compact_half", batch=64, len_min=16, len_max=1024, lengths=4),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        case = _draw(rng)
        w = work(case)
        if w["flops"] <= 5.6e11 and w["bytes"] <= 1.6e9 and _plain_bytes(case) <= 2.0e10:
            return case


def _draw(rng):
    kind = rng.choice(["append", "append", "prefill", "prefill", "copy", "beam", "compact"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    head_dim = rng.choice([64, 128])
    block = rng.choice([16, 32])
    kv = rng.choice([1, 2, 4, 8])
    lengths = rng.randrange(1 << 20)
    if kind == "append":
        decode = rng.random() < 0.5
        case = _append("", dtype=dtype, head_dim=head_dim, block=block, kv_heads=kv,
                       heads=kv * rng.choice([1, 2, 3, 4, 7, 8]), batch=_log_int(rng, 1, 256),
                       lengths=lengths, norm=rng.random() < 0.6,
                       rotary=16 * rng.randint(1, head_dim // 16),
                       interleaved=rng.random() < 0.5,
                       base=rng.choice([10000.0, 500000.0, 1000000.0]),
                       scaling=rng.choice(["none", "linear", "ntk", "parts"]),
                       factor=rng.choice([2.0, 4.0, 8.0, 32.0]), packed=rng.random() < 0.5)
        if not decode:
            hi = _log_int(rng, 1, max(1, 8192 // case["batch"]))
            case.update(new_min=rng.randint(0, hi), new_max=hi)
        lo = rng.choice([0, 0, _log_int(rng, 1, 100000)])
        case.update(prefix_min=lo, prefix_max=lo + _log_int(rng, 1, 4096))
    elif kind == "prefill":
        hi = _log_int(rng, 1, 4096)
        lo = rng.choice([0, _log_int(rng, 1, 30000)])
        case = _prefill("", dtype=dtype, head_dim=head_dim, block=block, kv_heads=kv,
                        heads=kv * rng.choice([1, 2, 3, 4, 5, 8, 16]), batch=_log_int(rng, 1, 32),
                        new_min=rng.randint(0, hi), new_max=hi, prefix_min=lo,
                        prefix_max=lo + _log_int(rng, 1, 2048), lengths=lengths)
    elif kind == "copy":
        case = _copy("", dtype=dtype, head_dim=head_dim, block=block, kv_heads=kv,
                     layers=rng.randint(1, 24), pairs=_log_int(rng, 1, 1024))
    elif kind == "beam":
        lo = rng.randint(0, 64)
        case = _beam("", dtype=dtype, head_dim=head_dim, block=block, kv_heads=kv,
                     layers=rng.randint(1, 12), parents=_log_int(rng, 1, 64),
                     width=rng.randint(1, 4), len_min=lo, len_max=lo + _log_int(rng, 1, 1000),
                     lengths=lengths)
    else:
        lo = rng.randint(0, 64)
        case = _compact("", dtype=dtype, head_dim=head_dim, block=block, kv_heads=kv,
                        layers=rng.randint(1, 12), batch=_log_int(rng, 1, 96), len_min=lo,
                        len_max=lo + _log_int(rng, 1, 1000), lengths=lengths,
                        free_share=rng.choice([0.1, 0.3, 0.5, 0.8]))
    del case["name"]
    return case


# ------------------------------------------------------------------- sizes


def _cdiv(a, b):
    return -(-a // b)


def _new_and_context(case):
    """New tokens and context lengths (the new tokens included) of every sequence."""
    r = random.Random(case["lengths"])
    new = [r.randint(case["new_min"], case["new_max"]) for _ in range(case["batch"])]
    ctx = [n + r.randint(case["prefix_min"], case["prefix_max"]) for n in new]
    if sum(new) == 0:
        new[0], ctx[0] = 1, ctx[0] + 1
    return new, ctx


def _row_lengths(case, count):
    r = random.Random(case["lengths"])
    lens = [r.randint(case["len_min"], case["len_max"]) for _ in range(count)]
    if sum(lens) == 0:
        lens[0] = 1
    return lens


def _elt(case):
    return 4 if case["dtype"] == "f32" else 2


def _block_bytes(case):
    return 2 * case["layers"] * case["kv_heads"] * case["block"] * case["head_dim"] * _elt(case)


def _plain_bytes(case):
    """Roughly what the plain form holds at once."""
    if case["kind"] == "prefill":
        new, ctx = _new_and_context(case)
        return case["batch"] * max(ctx) * (case["heads"] * max(new) * 8 +
                                           case["kv_heads"] * case["head_dim"] * 12)
    if case["kind"] == "append":
        return 0
    return 3 * _pool_blocks(case) * _block_bytes(case)


def _pool_blocks(case):
    if case["kind"] == "copy":
        return 2 * case["pairs"] + 8
    if case["kind"] == "beam":
        used = sum(_cdiv(n, case["block"]) for n in _row_lengths(case, case["parents"]))
        return used + 2 * case["parents"] * case["width"] + 8
    used = sum(_cdiv(n, case["block"]) for n in _row_lengths(case, case["batch"]))
    return max(used + 1, int(used / (1.0 - case["free_share"])))


def work(case):
    kind = case["kind"]
    if kind in ("append", "prefill"):
        new, ctx = _new_and_context(case)
        tokens, row = sum(new), case["head_dim"] * _elt(case)
        if kind == "append":
            moved = tokens * (case["heads"] + 2 * case["kv_heads"]) * row
            flops = tokens * (case["heads"] + case["kv_heads"]) * case["head_dim"] * 7
            return {"bytes": 2 * moved, "flops": flops}
        pairs = sum(n * (c - n) + n * (n + 1) // 2 for n, c in zip(new, ctx))
        kv = sum(c for n, c in zip(new, ctx) if n) * case["kv_heads"] * row * 2
        return {"bytes": 2 * tokens * case["heads"] * row + kv,
                "flops": 4 * pairs * case["heads"] * case["head_dim"]}
    if kind == "copy":
        return {"bytes": 2 * case["pairs"] * _block_bytes(case), "flops": 0}
    if kind == "beam":
        # every child: its parent's last rows copied, its table row freed and written; the
        # parents are drawn per seed, so the mean length stands for each
        lens, children = _row_lengths(case, case["parents"]), case["parents"] * case["width"]
        rows = children * sum(n % case["block"] for n in lens) / len(lens)
        blocks = children * sum(_cdiv(n, case["block"]) for n in lens) / len(lens)
        return {"bytes": 2 * rows * _block_bytes(case) / case["block"] + 24 * blocks, "flops": 0}
    # compact: the expected number of live pages past the live count (the live set is drawn)
    nb = _pool_blocks(case)
    live = sum(_cdiv(n, case["block"]) for n in _row_lengths(case, case["batch"]))
    return {"bytes": 2 * live * (nb - live) / nb * _block_bytes(case) + 16 * nb, "flops": 0}


# ------------------------------------------------------------------ inputs


def _frequencies(case):
    """Radians per position of each rotated pair, in 64 bits (a list)."""
    r, s = case["rotary"], case["factor"]
    base = case["base"] * s ** (r / (r - 2)) if case["scaling"] == "ntk" else case["base"]
    f = [base ** (-2.0 * i / r) for i in range(r // 2)]
    if case["scaling"] == "linear":
        f = [x / s for x in f]
    if case["scaling"] == "parts":
        keep = [min(1.0, max(0.0, (case["original"] * x / (2 * math.pi) - 1.0) / 3.0)) for x in f]
        f = [(1.0 - g) * x / s + g * x for g, x in zip(keep, f)]
    return f


def _amplitude(case):
    return 0.1 * math.log(case["factor"]) + 1.0 if case["scaling"] == "parts" else 1.0


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


def _append_inputs(case, seed):
    g, r, dt = _generator(seed), random.Random(seed), DTYPES[case["dtype"]]
    new, ctx = _new_and_context(case)
    h, kv, d, b, tokens = (case["heads"], case["kv_heads"], case["head_dim"], case["block"], sum(new))
    # pages for the new tokens only; the entries of the cached prefixes name some page of the
    # pool (the append does not read them)
    first = [(c - n) // b for n, c in zip(new, ctx)]
    maxb = max(1, max(_cdiv(c, b) for c in ctx))
    count = sum(_cdiv(c, b) - f for c, f in zip(ctx, first))
    nb = count + 4
    ids = list(range(nb))
    r.shuffle(ids)
    tables = torch.randint(0, nb, (len(new), maxb), generator=torch.Generator().manual_seed(seed),
                           dtype=torch.int32)
    for row, (f, c) in enumerate(zip(first, ctx)):
        for j in range(f, _cdiv(c, b)):
            tables[row, j] = ids.pop()
    pool = _normal((nb, 2, 1, kv, b, d), dt, g)
    if case["packed"]:
        qkv = _normal((tokens, h + 2 * kv, d), dt, g)
        q, k, v = qkv[:, :h], qkv[:, h:h + kv], qkv[:, h + kv:]
    else:
        q, k, v = (_normal((tokens, n, d), dt, g) for n in (h, kv, kv))
    weights = [None, None]
    if case["norm"]:
        weights = [(1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dt) for _ in range(2)]
    decode = case["new_min"] == case["new_max"] == 1
    return {"case": case, "pool": pool, "q": q, "k": k, "v": v, "q_weight": weights[0],
            "k_weight": weights[1], "tables": tables.cuda(), "lens": _ints(ctx),
            "starts": None if decode else _ints(_starts(new)),
            "out": torch.zeros((tokens, h, d), dtype=dt, device="cuda"),
            "freq": torch.tensor(_frequencies(case), dtype=torch.float64, device="cuda")}


def _prefill_inputs(case, seed):
    g, dt = _generator(seed), DTYPES[case["dtype"]]
    new, ctx = _new_and_context(case)
    h, kv, d, b, tokens = (case["heads"], case["kv_heads"], case["head_dim"], case["block"], sum(new))
    nblk = [_cdiv(c, b) for c in ctx]
    nb, maxb = sum(nblk) + 2, max(1, max(nblk))
    ids = torch.randperm(nb, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    tables, at = torch.full((len(new), maxb), -1, dtype=torch.int32), 0
    for row, n in enumerate(nblk):
        tables[row, :n] = ids[at:at + n]
        at += n
    pool = _normal((nb, 2, 1, kv, b, d), dt, g)
    # scores spread over a few units, as those of trained heads are
    q = _normal((tokens, h, d), dt, g, 1.5)
    return {"case": case, "pool": pool, "q": q, "tables": tables.cuda(), "lens": _ints(ctx),
            "starts": _ints(_starts(new)), "scale": d ** -0.5, "new_max": max(new),
            "out": torch.zeros_like(q)}


def _pool(case, nb, g):
    return _normal((nb, 2, case["layers"], case["kv_heads"], case["block"], case["head_dim"]),
                   DTYPES[case["dtype"]], g)


def _copy_inputs(case, seed):
    nb, n = _pool_blocks(case), case["pairs"]
    ids = torch.randperm(nb, generator=torch.Generator().manual_seed(seed)).to(torch.int32).cuda()
    return {"case": case, "pool": _pool(case, nb, _generator(seed)), "src": ids[:n].contiguous(),
            "dst": ids[n:2 * n].contiguous()}


def _stack_of(ids, nb):
    """The device free stack: height, then the ids from the bottom up."""
    stack = torch.full((nb + 1,), -1, dtype=torch.int32)
    stack[0] = len(ids)
    stack[1:1 + len(ids)] = torch.tensor(ids, dtype=torch.int32)
    return stack.cuda()


def _beam_inputs(case, seed):
    r, b, p = random.Random(seed), case["block"], case["parents"]
    lens, children, nb = _row_lengths(case, p), p * case["width"], _pool_blocks(case)
    ids = list(range(nb))
    r.shuffle(ids)
    # after a step, a row's owner has its own last block: room for every child's
    maxb = max(1, max(_cdiv(n, b) for n in lens)) + 1
    rows, shares, own_len = [], [0] * nb, list(lens)
    for n in lens:
        rows.append([ids.pop() for _ in range(_cdiv(n, b))])
    for c in range(children):  # the previous step's forks
        n, row = lens[c % p], list(rows[c % p])
        for j in range(n // b):
            shares[row[j]] += 1
        if n % b:
            row[n // b] = ids.pop()
        rows.append(row)
        own_len.append(n)
    tables = torch.full((p + children, maxb), -1, dtype=torch.int32)
    for i, row in enumerate(rows):
        tables[i, :len(row)] = torch.tensor(row, dtype=torch.int32)
    return {"case": case, "pool": _pool(case, nb, _generator(seed)), "tables": tables.cuda(),
            "lens": _ints(own_len), "shares": _ints(shares), "stack": _stack_of(ids, nb),
            "finished": torch.tensor([0] * p + [1] * children, dtype=torch.uint8, device="cuda"),
            "parents": _ints([r.randrange(p) for _ in range(children)]),
            "children": _ints(list(range(p, p + children)))}


def _compact_inputs(case, seed):
    r, b, nb = random.Random(seed), case["block"], _pool_blocks(case)
    lens = _row_lengths(case, case["batch"])
    ids = list(range(nb))
    r.shuffle(ids)
    nblk = [_cdiv(n, b) for n in lens]
    tables, at = torch.full((len(lens), max(1, max(nblk)) + 1), -1, dtype=torch.int32), 0
    for i, n in enumerate(nblk):
        tables[i, :n] = torch.tensor(ids[at:at + n], dtype=torch.int32)
        at += n
    shares = torch.zeros(nb, dtype=torch.int32)
    shares[torch.tensor(ids[:at:7], dtype=torch.long)] = 1  # held a second time elsewhere
    new = lambda like: torch.full_like(like, -1)  # noqa: E731
    tables, shares, stack = tables.cuda(), shares.cuda(), _stack_of(ids[at:], nb)
    return {"case": case, "pool": _pool(case, nb, _generator(seed)), "tables": tables,
            "lens": _ints(lens), "shares": shares, "stack": stack, "new_tables": new(tables),
            "new_shares": new(shares), "new_stack": new(stack), "remap": new(shares)}


_INPUTS = {"append": _append_inputs, "prefill": _prefill_inputs, "copy": _copy_inputs,
           "beam": _beam_inputs, "compact": _compact_inputs}


def prepare(case, seed):
    s = _INPUTS[case["kind"]](case, seed)
    if own:
        from paged_kv_cache_239_gb300.pool import BlockPool
        from paged_kv_cache_239_gb300.rope import Rope

        nb, _, layers, kv, block, d = s["pool"].shape
        s["cache"] = BlockPool(nb, block, layers, kv, d, tensor=s["pool"])
        if case["kind"] == "append":
            s["rope"] = Rope(case["rotary"], base=case["base"], interleaved=case["interleaved"],
                             scaling=case["scaling"], factor=case["factor"],
                             original_len=case["original"], low=1.0, high=4.0,
                             amplitude=_amplitude(case))
        need = 0
        if case["kind"] == "prefill":
            need = s["cache"].prefill_workspace_size(s["lens"].shape[0], s["q"].shape[0],
                                                     case["heads"], s["tables"].shape[1])
        if case["kind"] == "compact":
            need = s["cache"].compact_workspace_size()
        s["workspace"] = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    return s


# --------------------------------------------------------------------- run


def run(s):
    kind = s["case"]["kind"]
    return (_RUN_OWN if own else _RUN_PLAIN)[kind](s)


def _own_append(s):
    s["cache"].norm_rope_write_kv(LAYER, s["q"], s["k"], s["v"], s["tables"], s["lens"],
                                  rope=s["rope"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                                  eps=EPS, query_starts=s["starts"], out=s["out"])
    return {"q": s["out"], "pool": s["pool"]}


def _own_prefill(s):
    return s["cache"].prefill_attention(s["q"], LAYER, s["tables"], s["lens"], s["starts"],
                                        s["scale"], out=s["out"], workspace=s["workspace"])


def _own_copy(s):
    s["cache"].copy_blocks(s["src"], s["dst"])
    return s["pool"]


def _own_beam(s):
    s["cache"].device_free_shared(s["stack"], s["shares"], s["tables"], s["lens"], s["finished"])
    s["cache"].device_fork_sequences(s["stack"], s["shares"], s["tables"], s["lens"], s["parents"],
                                     s["children"])
    return {n: s[n] for n in ("pool", "tables", "lens", "shares", "stack")}


def _own_compact(s):
    s["cache"].device_compact_blocks(s["stack"], s["tables"], s["lens"], shares=s["shares"],
                                     out_stack=s["new_stack"], out_tables=s["new_tables"],
                                     out_shares=s["new_shares"], remap=s["remap"],
                                     workspace=s["workspace"])
    return {n: s[n] for n in ("pool", "new_tables", "new_shares", "new_stack", "remap")}


def _token_places(s, tokens):
    """Sequence, index within its new tokens, and position of every new token."""
    lens = s["lens"].long()
    t = torch.arange(tokens, device=lens.device)
    if s["starts"] is None:
        return t, torch.zeros_like(t), lens - 1
    starts = s["starts"].long()
    seq = (t[:, None] >= starts[None, 1:]).sum(1)
    i = t - starts[seq]
    return seq, i, lens[seq] - (starts[seq + 1] - starts[seq]) + i


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
    case, pool, out = s["case"], s["pool"], s["out"]
    seq, _, pos = _token_places(s, out.shape[0])
    angle = pos.double()[:, None, None] * s["freq"]
    amp = _amplitude(case)
    cos, sin = (angle.cos() * amp).float(), (angle.sin() * amp).float()
    args = (cos, sin, case["rotary"], case["interleaved"])
    out.copy_(_norm_rotate(s["q"], s["q_weight"], *args))
    k = _norm_rotate(s["k"], s["k_weight"], *args).to(pool.dtype)
    blk = s["tables"][seq, pos // case["block"]].long()
    row = pos % case["block"]
    pool[:, 0, LAYER][blk, :, row] = k
    pool[:, 1, LAYER][blk, :, row] = s["v"]
    return {"q": out, "pool": pool}


def _plain_prefill(s):
    case, q = s["case"], s["q"]
    kv, d, new_max = case["kv_heads"], case["head_dim"], s["new_max"]
    group, batch = case["heads"] // kv, s["lens"].shape[0]
    lens, starts = s["lens"].long(), s["starts"].long()
    pages = s["pool"][s["tables"].long().clamp(min=0), :, LAYER]  # [b, blocks, 2, kv, B, d]
    pages = pages.permute(2, 0, 3, 1, 4, 5).flatten(3, 4).float()
    i = torch.arange(new_max, device=q.device)
    new = starts[1:] - starts[:-1]
    token = (starts[:-1, None] + i).clamp(max=q.shape[0] - 1)
    x = q[token].float().view(batch, new_max, kv, group, d).permute(0, 2, 3, 1, 4)
    scores = torch.matmul(x.reshape(batch, kv, group * new_max, d), pages[0].transpose(-1, -2))
    scores = scores.mul_(s["scale"]).view(batch, kv, group, new_max, -1)
    t = torch.arange(scores.shape[-1], device=q.device)
    last = (lens - new)[:, None] + i
    hidden = (t > last[..., None]) | (t >= lens[:, None, None])
    scores.masked_fill_(hidden[:, None, None], float("-inf"))
    top = scores.amax(-1, keepdim=True).clamp(min=-1e30)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    v = pages[1].masked_fill((t >= lens[:, None])[:, None, :, None], 0.0)
    o = torch.matmul(p.view(batch, kv, group * new_max, -1), v).view(batch, kv, group, new_max, d)
    o = (o / total.clamp(min=1e-30)).permute(0, 3, 1, 2, 4).reshape(batch, new_max, -1, d)
    seq, at, _ = _token_places(s, q.shape[0])
    return s["out"].copy_(o[seq, at])


def _plain_copy(s):
    s["pool"][s["dst"].long()] = s["pool"][s["src"].long()]
    return s["pool"]


def _plain_beam(s):
    block, pool, stack, tables = s["case"]["block"], s["pool"], s["stack"], s["tables"]
    lens, shares = s["lens"], s["shares"]
    nb, (rows, maxb) = pool.shape[0], tables.shape
    j = torch.arange(maxb, device=tables.device)
    # free: one owner less per entry of a finished row; a page without another owner is pushed
    # by the last of its owners here, in row and table order
    gone = s["finished"].bool()[:, None] & (j < (lens[:, None] + block - 1) // block)
    ids = torch.where(gone, tables, nb).long().view(-1)
    count = torch.zeros(nb + 1, dtype=torch.int32, device=ids.device)
    count.index_add_(0, ids, torch.ones_like(ids, dtype=torch.int32))
    place = torch.arange(ids.shape[0], device=ids.device)
    last = torch.full((nb + 1,), -1, dtype=torch.long, device=ids.device)
    last = last.scatter_reduce(0, ids, place, "amax")
    left = torch.cat((shares, shares.new_zeros(1))) - count
    push = gone.view(-1) & (left[ids] < 0) & (last[ids] == place)
    at = torch.where(push, stack[0].long() + push.cumsum(0), nb + 1)
    grown = torch.cat((stack, stack.new_zeros(1)))
    grown[at] = ids.to(torch.int32)
    height = stack[0] + push.sum().to(torch.int32)
    shares.copy_(left[:nb].clamp(min=0))
    tables.masked_fill_(gone, -1)
    # fork: full pages shared, the last one's rows copied into a page from the stack's top
    par, chi = s["parents"].long(), s["children"].long()
    n = lens[par]
    full, part = n // block, n % block > 0
    rank = part.cumsum(0) - 1
    new = grown[(height - rank).clamp(min=1).long()]
    old = tables[par].gather(1, full.long()[:, None].clamp(max=maxb - 1))[:, 0].clamp(min=0).long()
    row = torch.where(j < full[:, None], tables[par],
                      torch.where((j == full[:, None]) & part[:, None], new[:, None], -1))
    tables[chi] = row.to(torch.int32)
    lens[chi] = n
    held = torch.where(j < full[:, None], row, nb).long().view(-1)
    more = torch.zeros(nb + 1, dtype=torch.int32, device=ids.device)
    more.index_add_(0, held, torch.ones_like(held, dtype=torch.int32))
    shares.add_(more[:nb])
    to = torch.where(part, new.long(), old)
    live = torch.arange(block, device=n.device)[None] < (n % block)[:, None]
    pool[to] = torch.where(live[:, None, None, None, :, None], pool[old], pool[to])
    stack.copy_(grown[:nb + 1])
    stack[0] = height - part.sum().to(torch.int32)
    return {name: s[name] for name in ("pool", "tables", "lens", "shares", "stack")}


def _plain_compact(s):
    pool, stack, tables = s["pool"], s["stack"], s["tables"]
    nb, block = pool.shape[0], s["case"]["block"]
    ids = torch.arange(nb, device=pool.device)
    free = torch.zeros(nb + 1, dtype=torch.bool, device=pool.device)
    free[torch.where(ids < stack[0], stack[1:], nb).long()] = True
    free[nb] = False
    live = ~free[:nb]
    count = live.sum()
    hole, mover = ~live & (ids < count), live & (ids >= count)
    spot = torch.zeros(nb + 1, dtype=torch.long, device=pool.device)
    spot[torch.where(hole, hole.cumsum(0) - 1, nb)] = ids
    remap = torch.where(live, torch.where(mover, spot[(mover.cumsum(0) - 1).clamp(min=0)], ids), -1)
    src = mover.nonzero()[:, 0]
    pool[remap[src]] = pool[src]
    s["remap"].copy_(remap)
    used = torch.arange(tables.shape[1], device=ids.device) < (s["lens"][:, None] + block - 1) // block
    moved = remap[tables.long().clamp(min=0)].to(torch.int32)
    s["new_tables"].copy_(torch.where(used, moved, tables))
    held = torch.zeros(nb + 1, dtype=torch.int32, device=ids.device)
    held[torch.where(live, remap, nb)] = s["shares"]
    s["new_shares"].copy_(held[:nb])
    s["new_stack"][0] = nb - count
    s["new_stack"][1:] = torch.where(ids < nb - count, nb - 1 - ids, -1).to(torch.int32)
    return {n: s[n] for n in ("pool", "new_tables", "new_shares", "new_stack", "remap")}


_RUN_PLAIN = {"append": _plain_append, "prefill": _plain_prefill, "copy": _plain_copy,
              "beam": _plain_beam, "compact": _plain_compact}
_RUN_OWN = {"append": _own_append, "prefill": _own_prefill, "copy": _own_copy,
            "beam": _own_beam, "compact": _own_compact}


# ------------------------------------------------------------------- exact


def exact(case, seed):
    s = _INPUTS[case["kind"]](case, seed)
    return {"append": _exact_append, "prefill": _exact_prefill, "copy": _exact_copy,
            "beam": _exact_beam, "compact": _exact_compact}[case["kind"]](case, s)


def _exact_append(case, s):
    """Each pair a complex number, turned by e^(i p f), sequence by sequence."""
    new, ctx = _new_and_context(case)
    r, block, amp = case["rotary"], case["block"], _amplitude(case)
    q_out, pool = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda"), s["pool"].double()
    tables, start = s["tables"].tolist(), 0
    for b, (n, c) in enumerate(zip(new, ctx)):
        if n == 0:
            continue
        p = torch.arange(c - n, c, dtype=torch.float64, device="cuda")
        turn = torch.polar(torch.full((n, 1, r // 2), amp, dtype=torch.float64, device="cuda"),
                           p[:, None, None] * s["freq"])
        rows = slice(start, start + n)
        done = []
        for x, w in ((s["q"][rows], s["q_weight"]), (s["k"][rows], s["k_weight"])):
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
        q_out[rows] = done[0]
        for j in range((c - n) // block, _cdiv(c, block)):
            lo, hi = max(c - n, j * block), min(c, (j + 1) * block)
            page = pool[tables[b][j], :, LAYER]
            at = slice(lo - (c - n), hi - (c - n))
            page[0, :, lo - j * block:hi - j * block] = done[1][at].transpose(0, 1)
            page[1, :, lo - j * block:hi - j * block] = s["v"][rows][at].double().transpose(0, 1)
        start += n
    return {"q": q_out, "pool": pool}


def _exact_prefill(case, s):
    """Head by head and in strips of queries, softmax by its definition."""
    new, ctx = _new_and_context(case)
    group = case["heads"] // case["kv_heads"]
    out, start = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda"), 0
    for b, (n, c) in enumerate(zip(new, ctx)):
        pages = s["tables"][b, :_cdiv(c, case["block"])].long()
        for kvh in range(case["kv_heads"] if n else 0):
            kv = s["pool"][pages, :, LAYER, kvh].double()
            keys, values = (kv[:, x].reshape(-1, case["head_dim"])[:c] for x in range(2))
            for lo in range(0, n, 1024):
                hi = min(n, lo + 1024)
                x = s["q"][start + lo:start + hi, kvh * group:(kvh + 1) * group].double()
                z = torch.einsum("ngd,td->ngt", x, keys) * s["scale"]
                see = torch.arange(c, device="cuda") <= torch.arange(
                    c - n + lo, c - n + hi, device="cuda")[:, None]
                z = torch.where(see[:, None], z, float("-inf"))
                out[start + lo:start + hi, kvh * group:(kvh + 1) * group] = torch.einsum(
                    "ngt,td->ngd", torch.softmax(z, -1), values)
        start += n
    return out


def _exact_copy(case, s):
    pool = s["pool"].double()
    for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
        pool[b] = pool[a]
    return pool


def _exact_beam(case, s):
    pool, block = s["pool"].double(), case["block"]
    tables, lens, stack = s["tables"].tolist(), s["lens"].tolist(), s["stack"].tolist()
    shares = s["shares"].tolist()
    owners, top = list(shares), stack[0]
    for b, f in enumerate(s["finished"].tolist()):
        for j in range(_cdiv(lens[b], block) if f else 0):
            page = tables[b][j]
            owners[page] -= 1
            if owners[page] < 0:
                owners[page], top = 0, top + 1
                stack[top] = page
    for p, c in zip(s["parents"].tolist(), s["children"].tolist()):
        if lens[p] % block:
            page, top = stack[top], top - 1
            old = tables[p][lens[p] // block]
            pool[page, :, :, :, :lens[p] % block] = pool[old, :, :, :, :lens[p] % block]
    return {"pool": pool, "tables": None, "lens": None, "shares": None, "stack": None}


def _exact_compact(case, s):
    pool, stack = s["pool"].double(), s["stack"].tolist()
    free = set(stack[1:1 + stack[0]])
    count = pool.shape[0] - len(free)
    holes = sorted(i for i in free if i < count)
    movers = [i for i in range(count, pool.shape[0]) if i not in free]
    for a, b in zip(movers, holes):
        pool[b] = pool[a]
    return {"pool": pool, "new_tables": None, "new_shares": None, "new_stack": None, "remap": None}
