"""GPU parity of the operators for drafted trees (plan and trim of pages, append at given slots,
attention under tree masks, acceptance) against plain implementations, at the sizes, masks and
inputs where they can go wrong, and whole steps of them together."""
from types import SimpleNamespace

import numpy as np
import pytest
import torch

import prompt_reference as R
import tree_reference as T
from gpu_helpers import pool_in_layout
from paged_kv_cache_239_gb300 import binding as B
from paged_kv_cache_239_gb300.pool import BlockPool
from paged_kv_cache_239_gb300.rope import Rope

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def ints(x, dev, dtype=torch.int32):
    return torch.tensor(np.asarray(x), dtype=dtype, device=dev)


def randn(shape, dtype, dev, seed, scale=1.0):
    g = torch.Generator(device=dev).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=dev) * scale).to(dtype)


def check(got, want, bound):
    err = (got.double() - want).abs()
    assert bool(torch.isfinite(got).all())
    over = err - bound
    assert bool((over <= 0).all()), f"error {err.max().item():.3g}, over its bound by {over.max().item():.3g}"


def status_is(want):
    assert B.pa_get_status() == want


def small_pool(nb, block, dev):
    return BlockPool(nb, block, 1, 1, 64, tensor=torch.zeros((nb, 2, 1, 1, block, 64), dtype=torch.bfloat16, device=dev))


def stack_tensor(ids, nb, dev):
    s = np.full(nb + 1, -7, np.int32)   # (what lies above the height is no one's)
    s[0], s[1:1 + len(ids)] = len(ids), ids
    return ints(s, dev)


def stack_ids(t):
    s = t.tolist()
    return s[1:1 + s[0]]


# ------------------------------------------------------------------ plan


def plan_case(rng, batch, most, block, shape):
    """Sequences with none, one and many cached and new tokens, full and partial last pages."""
    new = [int(x) for x in rng.integers(0, most + 1, batch)]
    cached = [int(x) for x in rng.integers(0, 5 * block, batch)]
    for b in range(0, batch, 5):
        cached[b] = block * int(rng.integers(0, 3))
    trees = None if shape is None else [T.random_tree(rng, n, shape) for n in new]
    nblk = [R.cdiv(c, block) for c in cached]
    maxb = max(R.cdiv(c + n, block) for c, n in zip(cached, new)) + 2
    nb = sum(R.cdiv(c + n, block) for c, n in zip(cached, new)) + 3
    ids = [int(x) for x in rng.permutation(nb)]
    tables = np.full((batch, maxb), -1, np.int32)
    for b, n in enumerate(nblk):
        for j in range(n):
            tables[b, j] = ids.pop()
    return new, cached, trees, tables, ids, nb


@pytest.mark.parametrize("batch,most,block,shape,words,pad", [
    (1, 1, 16, "chain", 1, 0), (1, 8, 16, "wide", 1, 3), (5, 33, 32, "random", 2, 0),
    (40, 64, 16, "random", 2, 100), (33, 128, 16, "chain", 4, 1), (7, 200, 24, "random", 32, 5),
    (3, 3000, 16, None, 0, 9), (1030, 20, 16, "random", 1, 7), (2100, 3, 32, None, 1, 0),
    (300, 40, 16, "wide", 0, 50),
])
def test_plan_and_trim(cuda_device, batch, most, block, shape, words, pad):
    dev = cuda_device
    rng = np.random.default_rng(batch * 1000 + most)
    new, cached, trees, tables, ids, nb = plan_case(rng, batch, most, block, shape)
    total = sum(new) + pad
    want = T.Plan(block, tables, ids, cached, new, trees, total, words)
    cache = small_pool(nb, block, dev)
    stack, bt = stack_tensor(ids, nb, dev), ints(tables, dev)
    flat = None if trees is None else ints([x for t in trees for x in t] + [5] * pad, dev)
    lens, starts, slots, positions, masks = cache.device_plan_tokens(
        stack, bt, ints(cached, dev), ints(new, dev), total, parents=flat, mask_words=words)
    status_is(0)
    assert lens.tolist() == want.lens and starts.tolist() == want.starts
    assert slots.tolist() == want.slots and positions.tolist() == want.positions
    if words:
        assert np.array_equal(masks.cpu().numpy(), want.masks)
    else:
        assert masks is None
    assert np.array_equal(bt.cpu().numpy(), want.tables) and stack_ids(stack) == want.stack
    # back to some of the new tokens, then to the cached ones, then to none
    keep = [c + int(rng.integers(0, n + 1)) for c, n in zip(cached, new)]
    t, s = T.trim(block, want.tables, want.stack, want.lens, keep)
    cache.device_trim_sequences(stack, bt, lens, ints(keep, dev))
    assert np.array_equal(bt.cpu().numpy(), t) and stack_ids(stack) == s
    cache.device_trim_sequences(stack, bt, ints(keep, dev), ints(cached, dev))
    assert np.array_equal(bt.cpu().numpy(), tables) and sorted(stack_ids(stack)) == sorted(ids)
    cache.device_trim_sequences(stack, bt, ints(cached, dev), ints([0] * batch, dev))
    assert bool((bt == -1).all()) and sorted(stack_ids(stack)) == list(range(nb))
    status_is(0)
    cache.close()


def test_plan_trimmed_back_leaves_the_stack(cuda_device):
    dev, rng = cuda_device, np.random.default_rng(2)
    new, cached, trees, tables, ids, nb = plan_case(rng, 50, 64, 16, "random")
    cache = small_pool(nb, 16, dev)
    stack, bt = stack_tensor(ids, nb, dev), ints(tables, dev)
    before = stack.clone()
    for _ in range(3):
        lens = cache.device_plan_tokens(stack, bt, ints(cached, dev), ints(new, dev), sum(new))[0]
        assert not torch.equal(stack, before)
        cache.device_trim_sequences(stack, bt, lens, ints(cached, dev))
        assert torch.equal(stack, before) and np.array_equal(bt.cpu().numpy(), tables)
    status_is(0)
    cache.close()


def test_plan_of_nothing(cuda_device):
    dev = cuda_device
    cache = small_pool(4, 16, dev)
    stack, bt = stack_tensor([0, 1, 2, 3], 4, dev), torch.full((0, 3), -1, dtype=torch.int32, device=dev)
    lens, starts, slots, positions, masks = cache.device_plan_tokens(
        stack, bt, ints([], dev), ints([], dev), 5, mask_words=2)
    assert lens.numel() == 0 and starts.tolist() == [0] and slots.tolist() == [-1] * 5
    assert positions.tolist() == [0] * 5 and bool((masks == 0).all()) and stack.tolist() == [4, 0, 1, 2, 3]
    bt = torch.full((2, 3), -1, dtype=torch.int32, device=dev)
    lens, starts, slots, _, _ = cache.device_plan_tokens(stack, bt, ints([0, 0], dev), ints([0, 0], dev), 0)
    assert lens.tolist() == [0, 0] and starts.tolist() == [0, 0, 0] and slots.numel() == 0
    status_is(0)
    cache.close()


def test_plan_flags(cuda_device):
    """A dry stack, bad lengths and counts, batches without room, bad parents and bad pages."""
    dev, block = cuda_device, 16
    cache = small_pool(6, block, dev)

    def plan(tables, cached, new, total, ids, parents=None, words=0):
        stack, bt = stack_tensor(ids, 6, dev), ints(tables, dev)
        out = cache.device_plan_tokens(stack, bt, ints(cached, dev), ints(new, dev), total,
                                       parents=None if parents is None else ints(parents, dev), mask_words=words)
        return [None if x is None else x.tolist() for x in out], bt.tolist(), stack_ids(stack)

    # two pages for three: the last sequence's second page is not to be had
    out, bt, left = plan([[-1, -1]] * 2, [0, 0], [16, 17], 33, [4, 2])
    status_is(B.PA_STATUS_NO_FREE_BLOCKS)
    assert bt == [[2, -1], [4, -1]] and left == [] and out[0] == [16, 17]
    assert out[2] == list(range(32, 48)) + list(range(64, 80)) + [-1]
    # a length past the table, one below 0, a count below 0, more than the masks hold
    out, bt, left = plan([[0, 1]] * 5, [33, -1, 3, 3, 3], [1, 1, -1, 33, 2], 9, [5, 4], words=1)
    status_is(B.PA_STATUS_BAD_LENGTH)
    assert out[0] == [0, 0, 3, 3, 5] and out[1] == [0, 0, 0, 0, 0, 2] and left == [5, 4]
    assert out[2] == [3, 4] + [-1] * 7 and out[4] == [[1], [3]] + [[0]] * 7
    # no room for the second sequence: it and what comes after gets nothing
    out, bt, left = plan([[-1, -1]] * 3, [0, 0, 0], [3, 4, 1], 5, [1, 0])
    status_is(B.PA_STATUS_BAD_LENGTH)
    assert out[0] == [3, 0, 0] and out[1] == [0, 3, 3, 3] and out[2] == [0, 1, 2, -1, -1] and left == [1]
    # counts whose sum passes 32 bits
    out, _, _ = plan(np.full((3, 1 << 20), -1), [0, 0, 0], [1 << 24] * 3, 4, [1, 0])
    status_is(B.PA_STATUS_BAD_LENGTH)
    assert out[0] == [0, 0, 0] and out[1] == [0] * 4
    # parents that are not below their children are roots
    out, _, _ = plan([[-1]], [0], [4], 4, [3], parents=[0, 0, 7, -2], words=1)
    status_is(B.PA_STATUS_BAD_LENGTH)
    assert out[3] == [0, 1, 0, 0] and out[4] == [[1], [3], [4], [8]]
    # the cached last page is none; a stack id is none
    out, bt, _ = plan([[9, -1], [-1, -1]], [3, 0], [14, 1], 15, [3, 77])
    status_is(B.PA_STATUS_BAD_BLOCK_ID)
    assert out[2] == [-1] * 13 + [-1, 48] and bt == [[9, -1], [3, -1]]
    # a stack whose height is none
    stack, bt = stack_tensor([1, 2], 6, dev), ints([[-1]], dev)
    stack[0] = 99
    cache.device_plan_tokens(stack, bt, ints([0], dev), ints([1], dev), 1)
    assert B.pa_get_status() & B.PA_STATUS_BAD_LENGTH
    cache.close()


def test_trim_flags(cuda_device):
    dev = cuda_device
    cache = small_pool(8, 16, dev)
    stack = stack_tensor([7], 8, dev)
    bt = ints([[0, 1, 2], [3, 4, -1], [9, 5, -1], [6, -1, -1]], dev)
    # longer than it was, below 0, a page outside the pool, a length past the table
    cache.device_trim_sequences(stack, bt, ints([20, 20, 20, 49], dev), ints([21, -1, 0, 0], dev))
    status_is(B.PA_STATUS_BAD_LENGTH | B.PA_STATUS_BAD_BLOCK_ID)
    assert bt.tolist() == [[0, 1, 2], [3, 4, -1], [-1, -1, -1], [6, -1, -1]] and stack_ids(stack) == [7, 5]
    # more ids than the pool holds (the same page again and again): the height stays in it
    stack, bt = stack_tensor(list(range(8)), 8, dev), ints([[1, 1, 1]], dev)
    cache.device_trim_sequences(stack, bt, ints([48], dev), ints([0], dev))
    assert B.pa_get_status() & B.PA_STATUS_BAD_BLOCK_ID
    assert stack_ids(stack) == list(range(8)) and bt.tolist() == [[-1] * 3]
    cache.close()


# ----------------------------------------------------------- append at slots


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,block,h,hkv", [(64, 16, 16, 2), (128, 32, 3, 3), (128, 16, 10, 2), (64, 32, 1, 1)])
@pytest.mark.parametrize("scaling,interleaved", [("none", False), ("linear", True), (None, False)])
@pytest.mark.parametrize("norm", [True, False])
def test_append_at_slots(cuda_device, dtype, d, block, h, hkv, scaling, interleaved, norm):
    dev, dt = cuda_device, DT[dtype]
    rng = np.random.default_rng(d + h)
    t, nb = 41, 9
    slots = [int(x) for x in rng.permutation(nb * block)[:t]]
    positions = [int(x) for x in rng.integers(0, 200000, t)]
    positions[3], slots[5], slots[17] = 2 ** 31 - 1, -1, -(1 << 40)   # (two rows are no tokens)
    rotary = d if norm else d // 2
    r = None if scaling is None else Rope(rotary, interleaved=interleaved, scaling=scaling, factor=4.0)
    freq = None if scaling is None else R.frequencies(rotary, 10000.0, scaling, 4.0)
    qkv = randn((t, h + 2 * hkv, d), dt, dev, 1)
    q, k, v = qkv[:, :h], qkv[:, h:h + hkv], qkv[:, h + hkv:]
    w = [(randn((d,), torch.float32, dev, 2 + i, 0.3) + 1).to(dt) if norm else None for i in range(2)]
    pool_t = randn((nb, 2, 2, hkv, block, d), dt, dev, 5)
    before = pool_t.clone()
    cache = BlockPool(nb, block, 2, hkv, d, tensor=pool_t)
    out = torch.full((t, h, d), 7.0, dtype=dt, device=dev)
    cache.norm_rope_write_kv_slots(1, q, k, v, ints(positions, dev), ints(slots, dev, torch.int64), rope=r,
                                   q_weight=w[0], k_weight=w[1], eps=1e-5, out=out)
    status_is(0)
    pos = ints(positions, dev, torch.int64)
    want_q, size_q = R.norm_rope(q, pos, freq, interleaved, 1.0, w[0], 1e-5)
    want_k, size_k = R.norm_rope(k, pos, freq, interleaved, 1.0, w[1], 1e-5)
    bq, bk = R.norm_rope_bound(want_q, size_q, dt), R.norm_rope_bound(want_k, size_k, dt)
    for i, s in enumerate(slots):
        if s < 0:
            assert bool((out[i] == 7.0).all())
            continue
        check(out[i], want_q[i], bq[i])
        row = pool_t[s // block, :, 1, :, s % block]
        check(row[0], want_k[i], bk[i])
        assert torch.equal(row[1], v[i])
        pool_t[s // block, :, 1, :, s % block] = before[s // block, :, 1, :, s % block]
    assert torch.equal(pool_t, before)   # nothing else was touched
    cache.close()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_at_planned_slots_is_the_append(cuda_device, dtype):
    """Chains planned on the device: the same bits as norm_rope_write_kv stores."""
    dev, dt, d, block, h, hkv = cuda_device, DT[dtype], 128, 16, 8, 2
    rng = np.random.default_rng(4)
    new, cached, _, tables, ids, nb = plan_case(rng, 9, 40, block, None)
    t = sum(new)
    a_t, b_t = (torch.zeros((nb, 2, 1, hkv, block, d), dtype=dt, device=dev) for _ in range(2))
    a, b = BlockPool(nb, block, 1, hkv, d, tensor=a_t), BlockPool(nb, block, 1, hkv, d, tensor=b_t)
    stack, bt, r = stack_tensor(ids, nb, dev), ints(tables, dev), Rope(d)
    q, k, v = (randn((t, n, d), dt, dev, n) for n in (h, hkv, hkv))
    lens, starts, slots, positions, _ = a.device_plan_tokens(stack, bt, ints(cached, dev), ints(new, dev), t)
    x = a.norm_rope_write_kv_slots(0, q, k, v, positions, slots, rope=r)
    y = b.norm_rope_write_kv(0, q, k, v, bt, lens, rope=r, query_starts=starts)
    assert torch.equal(x, y) and torch.equal(a_t, b_t)
    status_is(0)


def test_append_at_bad_slots(cuda_device):
    dev, d, block = cuda_device, 64, 16
    pool_t = torch.zeros((2, 2, 1, 1, block, d), dtype=torch.bfloat16, device=dev)
    cache = BlockPool(2, block, 1, 1, d, tensor=pool_t)
    x = randn((3, 1, d), torch.bfloat16, dev, 1)
    out = cache.norm_rope_write_kv_slots(0, x, x, x, ints([1, 2, 3], dev), ints([32, 1 << 40, 31], dev, torch.int64))
    status_is(B.PA_STATUS_BAD_BLOCK_ID)
    assert torch.equal(out, x) and torch.equal(pool_t[1, 0, 0, 0, 15], x[2, 0])
    assert int((pool_t != 0).any(-1).sum()) == 2
    pool_t.zero_()
    out = cache.norm_rope_write_kv_slots(0, x, x, x, ints([1, -1, 3], dev), ints([3, 4, 5], dev, torch.int64))
    status_is(B.PA_STATUS_BAD_LENGTH)
    assert bool((out[1] == 0).all()) and int((pool_t != 0).any(-1).sum()) == 4


# ---------------------------------------------------------- tree attention


def tree_case(seed, new, ctx, d, block, h, hkv, dt, dev, shape="random", words=None, pad=0, layers=1, spare=3):
    rng = np.random.default_rng(seed)
    t = sum(new)
    maxb = max(1, max(R.cdiv(c, block) for c in ctx)) + 1
    nb = sum(R.cdiv(c, block) for c in ctx) + spare
    tables = R.random_tables(rng, ctx, block, nb, maxb)
    bits = []
    for n in new:
        if shape == "any":      # no tree: any bits, with rows that see nothing of the new tokens
            bits += [int(rng.integers(0, 2)) * int.from_bytes(rng.bytes(n // 8 + 1), "little") % (1 << n) for _ in range(n)]
        else:
            bits += T.ancestors(T.random_tree(rng, n, shape))
    words = words or max(1, R.cdiv(max(new), 32))
    pool_t = randn((nb, 2, layers, hkv, block, d), dt, dev, seed)
    q = randn((t + pad, h, d), dt, dev, seed + 1, 1.5)
    return dict(tables=tables, bits=bits, pool=pool_t, q=q, nb=nb, starts=ints(R.starts_of(new), dev), bt=ints(tables, dev),
                lens=ints(ctx, dev), masks=ints(T.mask_words(bits + [0] * pad, words), dev))


SHAPES = [  # new tokens, contexts
    ([8], [508]), ([1], [1]), ([1, 1, 1], [1, 16, 300]), ([0, 5, 0, 33, 64], [9, 5, 0, 100, 64 + 128]),
    ([64, 64, 63, 1], [1064, 64, 700, 2000]), ([130, 256], [130, 300]), ([17] * 6, [17, 18, 130, 145, 257, 129]),
    ([3, 5], [9000, 20011]),
]


@pytest.mark.parametrize("dtype,kernel", [("bf16", "mma"), ("bf16", "tcgen05"), ("bf16", "auto"), ("f32", "auto"), ("f32", "mma"),
                                          ("f32", "tcgen05")])
@pytest.mark.parametrize("d,block,h,hkv", [(64, 16, 16, 2), (128, 16, 8, 2), (128, 32, 3, 3), (64, 32, 20, 4), (128, 16, 12, 1)])
@pytest.mark.parametrize("case", range(len(SHAPES)))
@pytest.mark.parametrize("shape", ["random", "chain", "any"])
def test_tree_attention(cuda_device, dtype, kernel, d, block, h, hkv, case, shape):
    dev, dt = cuda_device, DT[dtype]
    new, ctx = SHAPES[case]
    c = tree_case(case + d, new, ctx, d, block, h, hkv, dt, dev, shape, pad=3)
    cache = BlockPool(c["nb"], block, 1, hkv, d, tensor=c["pool"])
    cache.set_prefill_kernel(kernel)
    out = torch.full(c["q"].shape, 7.0, dtype=dt, device=dev)
    cache.tree_attention(c["q"], 0, c["bt"], c["lens"], c["starts"], c["masks"], d ** -0.5, out=out)
    status_is(0)
    t = sum(new)
    want, bound = T.attention(c["pool"], c["q"][:t], c["tables"], ctx, new, c["bits"], d ** -0.5)
    check(out[:t], want, bound)
    assert bool((out[t:] == 7.0).all())
    cache.close()


KERNELS = [("bf16", "mma"), ("bf16", "tcgen05"), ("f32", "auto"), ("f32", "mma"), ("f32", "tcgen05")]


@pytest.mark.parametrize("dtype,kernel", KERNELS)
@pytest.mark.parametrize("d", [64, 128])
def test_tree_rows_that_see_nothing(cuda_device, dtype, kernel, d):
    """Masks without a bit and nothing cached: zeros; bits past the new tokens mean nothing."""
    dev, dt, block, h, hkv = cuda_device, DT[dtype], 16, 8, 2
    new, ctx = [5, 40], [5, 40]
    c = tree_case(3, new, ctx, d, block, h, hkv, dt, dev)
    masks = c["masks"].clone()
    masks[1], masks[20] = 0, 0
    masks[4, 0] |= -32               # bits 5 .. 31 of a sequence of five
    masks[4, 1] = -1
    masks[5:, 1] |= -256             # bits 40 .. 63 of one of forty
    c["bits"][1] = c["bits"][20] = 0
    cache = BlockPool(c["nb"], block, 1, hkv, d, tensor=c["pool"])
    cache.set_prefill_kernel(kernel)
    out = cache.tree_attention(c["q"], 0, c["bt"], c["lens"], c["starts"], masks, d ** -0.5)
    want, bound = T.attention(c["pool"], c["q"], c["tables"], ctx, new, c["bits"], d ** -0.5)
    check(out, want, bound)
    assert bool((out[1] == 0).all()) and bool((out[20] == 0).all())
    status_is(0)


@pytest.mark.parametrize("dtype,kernel", KERNELS)
@pytest.mark.parametrize("d,block", [(64, 32), (128, 16)])
@pytest.mark.parametrize("prefix", [0, 77, 3000])
def test_tree_values_that_are_not_finite(cuda_device, dtype, kernel, d, block, prefix):
    """NaN and infinities in branches that a row does not see do not reach it; in those it
    sees, and in what is cached, they reach their own column."""
    dev, dt, h, hkv = cuda_device, DT[dtype], 8, 2
    n = 20
    tree = T.random_tree(np.random.default_rng(5), n)
    c = tree_case(9, [n], [prefix + n], d, block, h, hkv, dt, dev)
    c["bits"] = T.ancestors(tree)
    c["masks"] = ints(T.mask_words(c["bits"], 1), dev)
    pool_t = c["pool"]
    # everything outside the context
    last = prefix + n
    page = int(c["tables"][0, (last - 1) // block])
    if last % block:
        pool_t[page, :, :, :, last % block:] = float("nan")
    free = set(range(c["nb"])) - set(int(x) for x in c["tables"][0] if x >= 0)
    for x in free:
        pool_t[x] = float("inf")
    clean = pool_t.clone()
    marks = {7: ("nan", 3), 12: ("inf", 4), 13: ("-inf", 4), 19: ("inf", d - 1)}   # node: value, column
    if prefix:
        marks[-5] = ("-inf", 10)   # a cached one: all rows see it
    for node, (value, col) in marks.items():
        at = prefix + node
        p = int(c["tables"][0, at // block])
        pool_t[p, 1, 0, 1, at % block, col] = float(value)
        clean[p, 1, 0, 1, at % block, col] = 0.0
        if node >= 0:                                     # keys that some rows must not see
            pool_t[p, 0, 0, 0, at % block, 0] = float("nan")
            clean[p, 0, 0, 0, at % block, 0] = 0.0
    cache = BlockPool(c["nb"], block, 1, hkv, d, tensor=pool_t)
    cache.set_prefill_kernel(kernel)
    out = cache.tree_attention(c["q"], 0, c["bt"], c["lens"], c["starts"], c["masks"], d ** -0.5)
    status_is(0)
    want, bound = T.attention(clean, c["q"], c["tables"], [last], [n], c["bits"], d ** -0.5)
    group = h // hkv
    for i in range(n):
        seen = [x for x in marks if x < 0 or c["bits"][i] >> x & 1]
        for hh in range(h):
            if hh < group:   # KV head 0: rows that see a NaN key are not looked at further
                if any(x >= 0 for x in seen):
                    continue
                check(out[i, hh], want[i, hh], bound[i, hh])
                continue
            special = {}
            for x in seen:
                special.setdefault(marks[x][1], []).append(float(marks[x][0]))
            for col, values in special.items():
                got, s = float(out[i, hh, col]), sum(values)
                assert got == s or (np.isnan(got) and np.isnan(s)), (i, hh, col, got, values)
            rest = [x for x in range(d) if x not in special]
            check(out[i, hh, rest], want[i, hh, rest], bound[i, hh, rest])


@pytest.mark.parametrize("dtype,kernel", KERNELS)
def test_tree_bad_pages_and_lengths(cuda_device, dtype, kernel):
    dev, dt, d, block, h, hkv = cuda_device, DT[dtype], 64, 16, 8, 2
    new, ctx = [4, 40, 6, 3], [300, 140, 5, 60]      # (the third has more new tokens than context)
    good = [4, 40, 0, 3]
    c = tree_case(2, new, [300, 140, 6, 60], d, block, h, hkv, dt, dev)
    tables = c["tables"].copy()
    tables[0, 3], tables[3, 3] = -1, c["nb"]          # a cached page; the one with the new tokens
    lens = ints(ctx, dev)
    cache = BlockPool(c["nb"], block, 1, hkv, d, tensor=c["pool"])
    cache.set_prefill_kernel(kernel)
    out = cache.tree_attention(c["q"], 0, ints(tables, dev), lens, c["starts"], c["masks"], d ** -0.5)
    status_is(B.PA_STATUS_BAD_BLOCK_ID | B.PA_STATUS_BAD_LENGTH)
    rows = [i for i in range(53) if not 44 <= i < 50]
    bits = [c["bits"][i] for i in rows]
    want, bound = T.attention(c["pool"], c["q"][rows], tables, [300, 140, 0, 60], good, bits, d ** -0.5)
    check(out[rows], want, bound)
    assert bool((out[44:50] == 0).all())
    # more new tokens than the masks have bits for
    out = cache.tree_attention(c["q"], 0, c["bt"], ints([300, 140, 6, 60], dev), c["starts"],
                               c["masks"][:, :1].contiguous(), d ** -0.5)
    status_is(B.PA_STATUS_BAD_LENGTH)
    assert bool((out[4:44] == 0).all()) and bool((out[:4] != 0).any()) and bool((out[44:] != 0).any())


@pytest.mark.parametrize("dtype,kernel", KERNELS)
@pytest.mark.parametrize("layout", ["fused", "separate", "layer_major"])
def test_tree_layouts_and_scales(cuda_device, dtype, kernel, layout):
    dev, dt, d, block, h, hkv = cuda_device, DT[dtype], 128, 16, 8, 4
    new, ctx = [9, 30], [300, 77]
    layers, layer = (1, 0) if layout == "separate" else (2, 1)
    c = tree_case(12, new, ctx, d, block, h, hkv, dt, dev, layers=layers)
    wl = SimpleNamespace(num_blocks=c["nb"], num_layers=layers, num_kv_heads=hkv, block_size=block, head_dim=d)
    keep, handle = pool_in_layout(wl, c["pool"], layout, dev)
    B.pa_pool_set_prefill_kernel(handle, {"auto": 0, "mma": 1, "tcgen05": 2}[kernel])
    t = sum(new)
    need = B.pa_tree_workspace_size(handle, 2, t, h, c["bt"].shape[1])
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    for scale in (0.3, -0.2, 0.0):
        out = torch.empty_like(c["q"])
        B.pa_tree_attention(out, c["q"], handle, layer, c["bt"], c["bt"].shape[1], c["lens"], c["starts"], c["masks"],
                            c["masks"].shape[1], 2, t, h, scale, ws, need)
        want, bound = T.attention(c["pool"], c["q"], c["tables"], ctx, new, c["bits"], scale, layer)
        check(out, want, bound)
    status_is(0)
    del keep
    B.pa_pool_destroy(handle)


@pytest.mark.parametrize("dtype,kernel", KERNELS)
def test_tree_captured_and_on_two_streams(cuda_device, dtype, kernel):
    """Replays see new inputs; two streams with workspaces of their own do not meet."""
    dev, dt, d, block, h, hkv = cuda_device, DT[dtype], 128, 16, 16, 2
    new, ctx = [16, 3, 40], [5000, 900, 3000]
    c = tree_case(21, new, ctx, d, block, h, hkv, dt, dev)
    cache = BlockPool(c["nb"], block, 1, hkv, d, tensor=c["pool"])
    cache.set_prefill_kernel(kernel)
    t = sum(new)
    args = (0, c["bt"], c["lens"], c["starts"], c["masks"], d ** -0.5)
    need = cache.tree_workspace_size(3, t, h, c["bt"].shape[1])
    outs, qs, graphs = [], [], []
    side = [torch.cuda.Stream() for _ in range(2)]
    for s in side:
        q, out = c["q"].clone(), torch.empty_like(c["q"])
        ws = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
        cache.tree_attention(q, *args, out=out, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            cache.tree_attention(q, *args, out=out, workspace=ws)
        graphs.append((g, ws))
        outs.append(out), qs.append(q)
    for i in range(2):
        qs[i].copy_(randn(qs[i].shape, dt, dev, 50 + i))
    torch.cuda.synchronize()
    for _ in range(5):
        for s, (g, _) in zip(side, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for i in range(2):
        want, bound = T.attention(c["pool"], qs[i], c["tables"], ctx, new, c["bits"], d ** -0.5)
        check(outs[i], want, bound)
    status_is(0)


# ---------------------------------------------------------------- accept


def accept_case(rng, new, max_path, vocab, right, shape):
    trees = [T.random_tree(rng, n, shape) for n in new]
    tokens, targets, paths = [], [], []
    for tree in trees:
        tok = [int(x) for x in rng.integers(0, vocab, len(tree))]
        tgt = [int(x) for x in rng.integers(0, vocab, len(tree))]
        for i, p in enumerate(tree):
            if p >= 0 and rng.random() < right:
                tgt[p] = tok[i]
        tokens += tok
        targets += tgt
        paths.append(T.walk(tree, tok, tgt, max_path))
    return trees, tokens, targets, paths


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["fused", "layer_major"])
@pytest.mark.parametrize("new,max_path,vocab,right,shape", [
    ([1], 1, 9, 1.0, "chain"), ([8, 0, 8], 8, 99, 0.7, "wide"), ([64, 33, 2, 0, 40], 16, 5, 0.9, "random"),
    ([300, 5], 300, 50, 1.0, "chain"), ([20] * 70, 3, 3, 0.8, "random"), ([1024], 1024, 2, 1.0, "random"),
])
def test_accept(cuda_device, dtype, layout, new, max_path, vocab, right, shape):
    dev, dt = cuda_device, DT[dtype]
    rng = np.random.default_rng(sum(new) + max_path)
    block, layers, hkv, d = 16, 3, 2, 64
    cached = [int(x) for x in rng.integers(0, 40, len(new))]
    ctx = [c + n for c, n in zip(cached, new)]
    nb = sum(R.cdiv(c, block) for c in ctx) + 2
    tables = R.random_tables(rng, ctx, block, nb, max(1, max(R.cdiv(c, block) for c in ctx)))
    trees, tokens, targets, paths = accept_case(rng, new, max_path, vocab, right, shape)
    slots = [int(tables[b, p // block]) * block + p % block for b, (c, n) in enumerate(zip(cached, new))
             for p in range(c, c + n)]
    fused = randn((nb, 2, layers, hkv, block, d), dt, dev, 1)
    wl = SimpleNamespace(num_blocks=nb, num_layers=layers, num_kv_heads=hkv, block_size=block, head_dim=d)
    want = fused.clone()
    keep, handle = pool_in_layout(wl, fused, layout, dev)
    start, flat = 0, [x for tr in trees for x in tr]
    for n, path in zip(new, paths):
        for k, p in enumerate(path):
            a, z = slots[start + p], slots[start + k]
            want[z // block, :, :, :, z % block] = want[a // block, :, :, :, a % block].clone()
        start += n
    batch, pad = len(new), 4
    outs = [torch.full(s, 77, dtype=torch.int32, device=dev) for s in ((batch,), (batch, max_path), (batch,), (batch,))]
    B.pa_device_accept_tree(handle, ints(slots + [-1] * pad, dev, torch.int64), ints(flat + [3] * pad, dev),
                            ints(tokens + [0] * pad, dev), ints(targets + [0] * pad, dev), ints(ctx, dev),
                            ints(R.starts_of(new), dev), batch, sum(new) + pad, max_path, *outs)
    status_is(0)
    starts = R.starts_of(new)
    assert outs[0].tolist() == [len(p) for p in paths]
    assert outs[1].tolist() == [p + [-1] * (max_path - len(p)) for p in paths]
    assert outs[2].tolist() == [targets[starts[b] + p[-1]] if p else -1 for b, p in enumerate(paths)]
    assert outs[3].tolist() == [c + len(p) for c, p in zip(cached, paths)]
    if layout == "fused":
        assert torch.equal(keep[0], want)
    else:
        assert torch.equal(keep[0], want[:, 0].permute(1, 0, 2, 3, 4))
        assert torch.equal(keep[1], want[:, 1].permute(1, 0, 2, 3, 4))
    B.pa_pool_destroy(handle)


def test_accept_flags(cuda_device):
    dev = cuda_device
    pool_t = randn((4, 2, 1, 1, 16, 64), torch.bfloat16, dev, 1)
    before = pool_t.clone()
    cache = BlockPool(4, 16, 1, 1, 64, tensor=pool_t)

    def accept(slots, parents, tokens, targets, lens, starts, most=4):
        out = cache.device_accept_tree(ints(slots, dev, torch.int64), ints(parents, dev), ints(tokens, dev),
                                       ints(targets, dev), ints(lens, dev), ints(starts, dev), most)
        return [x.tolist() for x in out]

    # parents that are not below their children are accepted by no one; a second root neither
    out = accept([0, 1, 2, 3], [-1, 2, -1, 0], [5, 5, 5, 6], [5, 5, 5, 5], [4], [0, 4])
    status_is(B.PA_STATUS_BAD_LENGTH)
    assert out == [[1], [[0, -1, -1, -1]], [5], [1]] and torch.equal(pool_t, before)
    # starts that are none, more tokens than context
    out = accept([0, 1], [-1, 0], [1, 1], [1, 1], [2, 1, 9], [0, 3, 2, 2])
    status_is(B.PA_STATUS_BAD_LENGTH)
    assert out[0] == [0, 0, 0] and out[3] == [2, 1, 9] and out[2] == [-1] * 3
    # slots that are no page's: counted, not moved
    out = accept([0, 1, 64, 3], [-1, 0, 0, 2], [9, 7, 8, 4], [8, 0, 4, 1], [4], [0, 4])
    status_is(B.PA_STATUS_BAD_BLOCK_ID)
    assert out == [[3], [[0, 2, 3, -1]], [1], [3]]
    assert torch.equal(pool_t[0, :, 0, 0, 1], before[0, :, 0, 0, 1])
    pool_t.copy_(before)
    out = accept([0, -1, 2], [-1, 0, 0], [9, 7, 8], [8, 0, 4], [3], [0, 3])
    status_is(B.PA_STATUS_BAD_BLOCK_ID)
    assert out[1] == [[0, 2, -1, -1]] and torch.equal(pool_t, before)
    cache.close()


# -------------------------------------------------------- steps of all of them


@pytest.mark.parametrize("dtype,kernel", [("bf16", "auto"), ("bf16", "tcgen05"), ("f32", "auto"), ("f32", "tcgen05")])
def test_speculation_steps(cuda_device, dtype, kernel):
    """Steps of plan, append, tree attention, acceptance and trim, captured once and replayed:
    after each, the cache holds what appending the accepted tokens one by one gives, and the
    attention is that of the accepted context."""
    dev, dt = cuda_device, DT[dtype]
    rng = np.random.default_rng(8)
    batch, nodes, most, block, layers, h, hkv, d, vocab = 5, 12, 6, 16, 2, 8, 2, 64, 40
    maxb, nb, total = 20, 60, batch * nodes + 7
    table = {x: randn((layers, vocab, n, d), dt, dev, i) for i, (x, n) in enumerate((("q", h), ("k", hkv), ("v", hkv)))}
    pool_t = torch.zeros((nb, 2, layers, hkv, block, d), dtype=dt, device=dev)
    cache, rope = BlockPool(nb, block, layers, hkv, d, tensor=pool_t), Rope(d)
    cache.set_prefill_kernel(kernel)
    stack = cache.device_stack()
    bt = torch.full((batch, maxb), -1, dtype=torch.int32, device=dev)
    # prompts: planned without trees, appended at their slots
    prompts = [[int(x) for x in rng.integers(0, vocab, n)] for n in (1, 16, 30, 47, 5)]
    new = [len(p) for p in prompts]
    lens, starts, slots, positions, _ = cache.device_plan_tokens(stack, bt, ints([0] * batch, dev), ints(new, dev), sum(new))
    flat = ints([x for p in prompts for x in p], dev).long()
    for layer in range(layers):
        cache.norm_rope_write_kv_slots(layer, *(table[x][layer][flat] for x in "qkv"), positions, slots, rope=rope)
    cached = lens.clone()
    history = [list(p) for p in prompts]

    counts = ints([nodes, nodes, 0, nodes, 3], dev)   # (one waits, one drafts little)
    parents, tokens, targets = (torch.zeros(total, dtype=torch.int32, device=dev) for _ in range(3))
    outs = []

    def step():
        lens, starts, slots, positions, masks = cache.device_plan_tokens(
            stack, bt, cached, counts, total, parents=parents, mask_words=1)
        outs[:] = []
        for layer in range(layers):
            q, k, v = (table[x][layer][tokens.long()] for x in "qkv")
            q = cache.norm_rope_write_kv_slots(layer, q, k, v, positions, slots, rope=rope)
            outs.append(cache.tree_attention(q, layer, bt, lens, starts, masks, d ** -0.5))
        result = cache.device_accept_tree(slots, parents, tokens, targets, lens, starts, most)
        cache.device_trim_sequences(stack, bt, lens, result[3])
        cached.copy_(result[3])
        return result

    step_in = dict(stack=stack.clone(), bt=bt.clone(), cached=cached.clone(), pool=pool_t.clone())
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()                                         # (warm up; undone below)
    status_is(B.PA_STATUS_BAD_LENGTH)                  # (parents that are all 0 are no trees)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        result = step()
    stack.copy_(step_in["stack"]), bt.copy_(step_in["bt"]), cached.copy_(step_in["cached"]), pool_t.copy_(step_in["pool"])

    def sequential():
        """The accepted tokens appended to a cache of its own, in the same pages."""
        other_t = torch.zeros_like(pool_t)
        other = BlockPool(nb, block, layers, hkv, d, tensor=other_t)
        n = [len(x) for x in history]
        ids = ints([x for p in history for x in p], dev).long()
        for layer in range(layers):
            other.norm_rope_write_kv(layer, *(table[x][layer][ids] for x in "qkv"), bt, ints(n, dev), rope=rope,
                                     query_starts=ints(R.starts_of(n), dev))
        return other_t

    n_new = counts.tolist()
    starts_h = R.starts_of(n_new)
    for it in range(6):
        trees, tok, tgt, paths = accept_case(rng, n_new, most, vocab, 0.8, "random")
        fill = lambda x: x + [0] * (total - len(x))  # noqa: E731
        parents.copy_(ints(fill([x for tr in trees for x in tr]), dev))
        tokens.copy_(ints(fill(tok), dev)), targets.copy_(ints(fill(tgt), dev))
        graph.replay()
        torch.cuda.synchronize()
        status_is(0)
        assert result[1].tolist() == [p + [-1] * (most - len(p)) for p in paths]
        before = [len(x) for x in history]
        for b, p in enumerate(paths):
            history[b] += [tok[starts_h[b] + x] for x in p]
        assert cached.tolist() == [len(x) for x in history]
        want = sequential()
        table_h = bt.tolist()
        for b, x in enumerate(history):
            used = [i for i in table_h[b] if i >= 0]
            assert len(used) == R.cdiv(len(x), block)
            for at in range(len(x)):
                page = table_h[b][at // block]
                assert torch.equal(pool_t[page, :, :, :, at % block], want[page, :, :, :, at % block])
        held = [i for row in table_h for i in row if i >= 0]
        assert len(set(held)) == len(held) and sorted(held + stack_ids(stack)) == list(range(nb))
        # the accepted nodes' outputs are those of the accepted context
        for layer in range(layers):
            ids = ints([x for h_, n in zip(history, before) for x in h_[n:]], dev).long()
            pos = torch.cat([torch.arange(n, len(x)) for x, n in zip(history, before)]).to(dev)
            q = cache.norm_rope_write_kv_slots(layer, *(table[x][layer][ids] for x in "qkv"), pos.to(torch.int32),
                                               torch.full_like(pos, nb * block), rope=rope)
            assert B.pa_get_status() == B.PA_STATUS_BAD_BLOCK_ID   # (queries alone: the slots are no page's)
            n = [len(x) - y for x, y in zip(history, before)]
            ref, bound = R.prefill(pool_t, q, bt.cpu().numpy(), [len(x) for x in history], n, d ** -0.5, layer)
            got = torch.cat([outs[layer][starts_h[b] + np.array(p, dtype=np.int64)] for b, p in enumerate(paths) if p])
            check(got, ref, bound)
