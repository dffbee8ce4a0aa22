"""The operators for drafted trees at their limits: many sequences, the largest trees, pages far
into a pool, calls at once on several streams, values of tiny weight, refused calls."""
import threading

import numpy as np
import pytest
import torch

import prompt_reference as R
import tree_reference as T
from paged_kv_cache_239_gb300 import binding as B
from paged_kv_cache_239_gb300.pool import BlockPool
from paged_kv_cache_239_gb300.rope import Rope
from test_tree_ops_gpu import (DT, KERNELS, accept_case, check, ints, plan_case, randn, small_pool,
                               stack_ids, stack_tensor, status_is, tree_case)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,kernel", KERNELS)
@pytest.mark.parametrize("batch,most,extra,h,hkv", [(45, 9, 400, 8, 4), (33, 2, 60, 4, 4), (400, 3, 40, 4, 2), (1000, 2, 20, 2, 1)])
def test_tree_many_sequences(cuda_device, dtype, kernel, batch, most, extra, h, hkv):
    """More sequences than a warp or a CTA looks at in one go, some without new tokens."""
    dev, dt, d, block = cuda_device, DT[dtype], 64, 16
    rng = np.random.default_rng(batch)
    new = [int(x) for x in rng.integers(0, most + 1, batch)]
    ctx = [n + int(x) for n, x in zip(new, rng.integers(0, extra + 1, batch))]
    c = tree_case(batch, new, ctx, d, block, h, hkv, dt, dev, pad=5)
    cache = BlockPool(c["nb"], block, 1, hkv, d, tensor=c["pool"])
    cache.set_prefill_kernel(kernel)
    out = torch.full(c["q"].shape, 7.0, dtype=dt, device=dev)
    cache.tree_attention(c["q"], 0, c["bt"], c["lens"], c["starts"], c["masks"], d ** -0.5, out=out)
    status_is(0)
    t = sum(new)
    want, bound = T.attention(c["pool"], c["q"][:t], c["tables"], ctx, new, c["bits"], d ** -0.5)
    check(out[:t], want, bound)
    assert bool((out[t:] == 7.0).all())


@pytest.mark.parametrize("dtype,kernel", KERNELS)
@pytest.mark.parametrize("new,ctx,h,hkv,d", [([1024], [1500], 2, 2, 64), ([1000, 3], [1000, 40], 4, 1, 128), ([16], [40000], 8, 8, 128),
                                             ([4, 4], [30000, 2], 16, 2, 64)])
def test_tree_largest_and_longest(cuda_device, dtype, kernel, new, ctx, h, hkv, d):
    dev, dt, block = cuda_device, DT[dtype], 32
    c = tree_case(7, new, ctx, d, block, h, hkv, dt, dev)
    cache = BlockPool(c["nb"], block, 1, hkv, d, tensor=c["pool"])
    cache.set_prefill_kernel(kernel)
    out = cache.tree_attention(c["q"], 0, c["bt"], c["lens"], c["starts"], c["masks"], d ** -0.5)
    # a sequence of more new tokens than context is flagged, and its rows are zero
    good = [n if n <= x else 0 for n, x in zip(new, ctx)]
    status_is(0 if good == new else B.PA_STATUS_BAD_LENGTH)
    t = sum(good)
    want, bound = T.attention(c["pool"], c["q"][:t], c["tables"], ctx, good, c["bits"], d ** -0.5)
    check(out[:t], want, bound)
    assert bool((out[t:] == 0).all())


@pytest.mark.parametrize("dtype,kernel", KERNELS)
def test_tree_masks_wider_than_the_trees(cuda_device, dtype, kernel):
    """32 words of mask for trees of a few nodes, in a table far wider than the contexts."""
    dev, dt, d, block, h, hkv = cuda_device, DT[dtype], 64, 16, 8, 2
    new, ctx = [5, 9, 2], [70, 9, 300]
    c = tree_case(31, new, ctx, d, block, h, hkv, dt, dev, words=32)
    wide = torch.full((3, 2000), -1, dtype=torch.int32, device=dev)
    wide[:, :c["bt"].shape[1]] = c["bt"]
    cache = BlockPool(c["nb"], block, 1, hkv, d, tensor=c["pool"])
    cache.set_prefill_kernel(kernel)
    out = cache.tree_attention(c["q"], 0, wide, c["lens"], c["starts"], c["masks"], d ** -0.5)
    want, bound = T.attention(c["pool"], c["q"], c["tables"], ctx, new, c["bits"], d ** -0.5)
    check(out, want, bound)
    status_is(0)


@pytest.mark.parametrize("dtype,kernel", KERNELS)
@pytest.mark.parametrize("prefix", [40, 3000])
def test_tree_infinite_values_of_tiny_weight(cuda_device, dtype, kernel, prefix):
    """Scores so far apart that most weights are below the smallest number: an infinite value
    shows as not finite in every row that sees it, and in no other row or column."""
    dev, dt, d, block, h, hkv, n = cuda_device, DT[dtype], 128, 16, 8, 2, 12
    tree = T.random_tree(np.random.default_rng(3), n)
    c = tree_case(5, [n], [prefix + n], d, block, h, hkv, dt, dev)
    bits = T.ancestors(tree)
    marks = {x: (11 * x) % d for x in (2, 5, 8, 11)}
    for x, col in marks.items():
        at = prefix + x
        c["pool"][int(c["tables"][0, at // block]), 1, 0, :, at % block, col] = float("inf")
    at = prefix // 2
    c["pool"][int(c["tables"][0, at // block]), 1, 0, :, at % block, 127] = -float("inf")
    cache = BlockPool(c["nb"], block, 1, hkv, d, tensor=c["pool"])
    cache.set_prefill_kernel(kernel)
    out = cache.tree_attention(c["q"], 0, c["bt"], c["lens"], c["starts"], ints(T.mask_words(bits, 1), dev), 6.0).float()
    status_is(0)
    for i in range(n):
        cols = sorted({marks[x] for x in marks if bits[i] >> x & 1} | {127})
        rest = [x for x in range(d) if x not in cols]
        assert not bool(torch.isfinite(out[i][:, cols]).any()), i
        assert bool(torch.isfinite(out[i][:, rest]).all()), i


@pytest.mark.parametrize("dtype,kernel", KERNELS)
def test_tree_large_scores(cuda_device, dtype, kernel):
    """Rows whose maximum rises by hundreds along the context and into the tree."""
    dev, dt, d, block, h, hkv = cuda_device, DT[dtype], 128, 16, 4, 1
    new, ctx = [30], [700]
    c = tree_case(8, new, ctx, d, block, h, hkv, dt, dev)
    for j in range(R.cdiv(700, block)):
        c["pool"][int(c["tables"][0, j]), 0] *= 1.0 + 0.25 * j
    cache = BlockPool(c["nb"], block, 1, hkv, d, tensor=c["pool"])
    cache.set_prefill_kernel(kernel)
    out = cache.tree_attention(c["q"], 0, c["bt"], c["lens"], c["starts"], c["masks"], d ** -0.5)
    want, bound = T.attention(c["pool"], c["q"], c["tables"], ctx, new, c["bits"], d ** -0.5)
    check(out, want, bound)


@pytest.mark.parametrize("kernel", ["mma", "tcgen05"])
@pytest.mark.parametrize("d,block", [(64, 16), (128, 32)])
def test_tree_f32_infinite_keys_and_queries(cuda_device, kernel, d, block):
    """A key's infinite component: no weight in rows whose query is negative there (the score is
    -inf), nothing finite in the others; a query's: nothing finite in its row."""
    dev, h, hkv, n, ctx = cuda_device, 2, 2, 20, 300
    tree = T.random_tree(np.random.default_rng(4), n)
    c = tree_case(5, [n], [ctx], d, block, h, hkv, torch.float32, dev)
    bits = T.ancestors(tree)
    for at, value in ((77, float("inf")), (ctx - n + 3, float("inf")), (200, -float("inf"))):
        c["pool"][int(c["tables"][0, at // block]), 0, 0, :, at % block, 9] = value
    bt = c["bt"]
    q = c["q"].clone()
    q[:, :, 9] = -q[:, :, 9].abs()
    q[::3, :, 9] *= -1
    q[10, 0, 4] = float("inf")
    cache = BlockPool(c["nb"], block, 1, hkv, d, tensor=c["pool"])
    cache.set_prefill_kernel(kernel)
    out = cache.tree_attention(q, 0, bt, c["lens"], c["starts"], ints(T.mask_words(bits, 1), dev), d ** -0.5)
    status_is(0)
    # key 200 is infinite in the rows whose queries are negative: those of the others are left
    for i in range(n):
        assert not bool(torch.isfinite(out[i]).any()) if i % 3 else True
    # without key 200 the negative rows lose the infinite keys only
    c["pool"][int(c["tables"][0, 200 // block]), 0, 0, :, 200 % block, 9] = 0.5
    out = cache.tree_attention(q, 0, bt, c["lens"], c["starts"], ints(T.mask_words(bits, 1), dev), d ** -0.5)
    status_is(0)
    plain = c["pool"].clone()
    plain[int(c["tables"][0, 77 // block]), 0, 0, :, 77 % block] = 0.0
    plain[int(c["tables"][0, 77 // block]), 1, 0, :, 77 % block] = 0.0
    at = ctx - n + 3
    plain[int(c["tables"][0, at // block]), 0, 0, :, at % block, 9] = 0.0
    for i in range(n):
        if i % 3 == 0 or i == 10:
            assert not bool(torch.isfinite(out[i, 0]).any()), i
            continue
        # the row by itself: the keys it sees that are finite, in 64 bits
        keys = [j for j in range(ctx - n) if j != 77] + [ctx - n + j for j in range(n) if bits[i] >> j & 1 and j != 3]
        kv = torch.stack([plain[int(c["tables"][0, j // block]), :, 0, :, j % block] for j in keys]).double()
        for head in range(h):
            s = kv[:, 0, head] @ q[i, head].double() * d ** -0.5
            want = torch.softmax(s, 0) @ kv[:, 1, head]
            # a product off by 2^-22, sums of d and of 300 terms off by 2^-24 each time, exponentials by 2^-22
            size = (kv[:, 0, head].abs() @ q[i, head].double().abs()).max() * d ** -0.5
            tol = (2.0 ** -21 * (1 + size) * (1 + d / 4) + 300 * 2.0 ** -24) * kv[:, 1, head].abs().max()
            assert float((out[i, head].double() - want).abs().max()) <= float(tol), (i, head)


@pytest.mark.parametrize("kernel", ["mma", "tcgen05"])
@pytest.mark.parametrize("d,block", [(64, 16), (128, 32)])
def test_tree_f32_values_at_the_end_of_the_range(cuda_device, kernel, d, block):
    """Keys, values and queries that bf16 would round to infinity."""
    dev, h, hkv, n, ctx = cuda_device, 4, 2, 9, 150
    c = tree_case(6, [n], [ctx], d, block, h, hkv, torch.float32, dev)
    huge = 3.395e38
    q = c["q"].clone()
    q[:, :, 5] = 1e-29 * q[:, :, 5].sign()     # (products of about 3e9, times a scale of 1e-9)
    q[2, :, 7] = -huge
    for at in (3, 100, ctx - 2):
        page, row = int(c["tables"][0, at // block]), at % block
        c["pool"][page, 0, 0, :, row, 5] = huge
    c["pool"][:, 0, 0, :, :, 7] = 1e-29
    c["pool"][int(c["tables"][0, 100 // block]), 1, 0, :, 100 % block, 11] = huge   # (one: weights sum to more than 1)
    cache = BlockPool(c["nb"], block, 1, hkv, d, tensor=c["pool"])
    cache.set_prefill_kernel(kernel)
    out = cache.tree_attention(q, 0, c["bt"], c["lens"], c["starts"], c["masks"], 1e-9)
    status_is(0)
    want, bound = T.attention(c["pool"], q, c["tables"], [ctx], [n], c["bits"], 1e-9)
    check(out, want, bound)


def test_far_pages(cuda_device):
    """Pages beyond 2^32 bytes and 2^31 elements of the pool: append at slots, attention on every
    kernel, acceptance."""
    dev, d, block, h, hkv = cuda_device, 128, 32, 8, 8
    nb = (1 << 31) // (2 * hkv * block * d) + 60
    pool_t = torch.empty((nb, 2, 1, hkv, block, d), dtype=torch.bfloat16, device=dev)
    new, ctx = [9, 33], [200, 300]
    rng = np.random.default_rng(6)
    tables = np.full((2, 10), -1, np.int32)
    ids = [nb - 1 - int(x) for x in rng.permutation(50)]
    for b, c in enumerate(ctx):
        for j in range(R.cdiv(c, block)):
            tables[b, j] = ids.pop()
    used = torch.tensor(sorted(int(x) for x in tables.ravel() if x >= 0), device=dev)
    pool_t[used] = randn((len(used), 2, 1, hkv, block, d), torch.bfloat16, dev, 3)
    trees = [T.random_tree(rng, n) for n in new]
    bits = [x for t in trees for x in T.ancestors(t)]
    slots = [int(tables[b, p // block]) * block + p % block for b, (n, c) in enumerate(zip(new, ctx)) for p in range(c - n, c)]
    cache, rope = BlockPool(nb, block, 1, hkv, d, tensor=pool_t), Rope(d)
    t = sum(new)
    q, k, v = (randn((t, n, d), torch.bfloat16, dev, i) for i, n in enumerate((h, hkv, hkv)))
    pos = ints(range(100, 100 + t), dev)
    out = cache.norm_rope_write_kv_slots(0, q, k, v, pos, ints(slots, dev, torch.int64), rope=rope)
    want, size = R.norm_rope(k, pos, R.frequencies(d, 10000.0), False, 1.0, None, 0.0)
    for i, s in enumerate(slots):
        check(pool_t[s // block, 0, 0, :, s % block], want[i], R.norm_rope_bound(want, size, torch.bfloat16)[i])
        assert torch.equal(pool_t[s // block, 1, 0, :, s % block], v[i])
    ref, bound = T.attention(pool_t, out, tables, ctx, new, bits, d ** -0.5)
    for kernel in ("mma", "tcgen05"):
        cache.set_prefill_kernel(kernel)
        got = cache.tree_attention(out, 0, ints(tables, dev), ints(ctx, dev), ints(R.starts_of(new), dev),
                                   ints(T.mask_words(bits, 2), dev), d ** -0.5)
        check(got, ref, bound)
    # every tree's deepest path, by tokens that are the nodes' own numbers
    tokens = [i for n in new for i in range(n)]
    targets, paths = [], []
    for tree in trees:
        at, path = len(tree) - 1, []
        while at >= 0:
            path.insert(0, at)
            at = tree[at]
        target = [-1] * len(tree)
        for a, b in zip(path, path[1:]):
            target[a] = b
        targets += target
        paths.append(path)
    rows = [pool_t[s // block, :, 0, :, s % block].clone() for s in slots]
    counts, nodes, _, _ = cache.device_accept_tree(ints(slots, dev, torch.int64), ints([x for t in trees for x in t], dev),
                                                   ints(tokens, dev), ints(targets, dev), ints(ctx, dev),
                                                   ints(R.starts_of(new), dev), 40)
    status_is(0)
    assert counts.tolist() == [len(p) for p in paths]
    for start, path in zip(R.starts_of(new), paths):
        for i, node in enumerate(path):
            s = slots[start + i]
            assert torch.equal(pool_t[s // block, :, 0, :, s % block], rows[start + node])


def test_append_in_place_and_of_one_token(cuda_device):
    dev, d, block, h, hkv = cuda_device, 128, 16, 8, 2
    pool_t = torch.zeros((3, 2, 1, hkv, block, d), dtype=torch.bfloat16, device=dev)
    cache, rope = BlockPool(3, block, 1, hkv, d, tensor=pool_t), Rope(d)
    for t in (1, 5):
        q, k, v = (randn((t, n, d), torch.bfloat16, dev, n) for n in (h, hkv, hkv))
        args = (k, v, ints(range(t), dev), ints(range(7, 7 + t), dev, torch.int64))
        a = cache.norm_rope_write_kv_slots(0, q, *args, rope=rope)
        b = q.clone()
        assert cache.norm_rope_write_kv_slots(0, b, *args, rope=rope, out=b) is b
        assert torch.equal(a, b)
    empty = cache.norm_rope_write_kv_slots(0, q[:0], k[:0], v[:0], ints([], dev), ints([], dev, torch.int64), rope=rope)
    assert empty.shape == (0, h, d)
    status_is(0)


def test_calls_on_streams_at_once(cuda_device):
    """Two programs' plans, appends, attentions, acceptances and trims on two streams, from two
    host threads: the same as one after the other."""
    dev, d, block, h, hkv, nodes = cuda_device, 64, 16, 8, 2, 20

    class Program:
        def __init__(self, seed):
            self.new, cached, _, tables, ids, nb = plan_case(np.random.default_rng(seed), 6, nodes, block, "random")
            self.new = [nodes] * 6
            nb += 20
            ids = [x for x in range(nb) if x not in set(int(y) for y in tables.ravel() if y >= 0)]
            self.pool = BlockPool(nb, block, 1, hkv, d, tensor=randn((nb, 2, 1, hkv, block, d), torch.bfloat16, dev, seed))
            wide = np.full((6, tables.shape[1] + 4), -1, np.int32)
            wide[:, :tables.shape[1]] = tables
            self.stack, self.bt, self.cached = stack_tensor(ids, nb, dev), ints(wide, dev), ints(cached, dev)
            trees, tok, tgt, _ = accept_case(np.random.default_rng(seed), self.new, 8, 30, 0.8, "random")
            self.parents = ints([x for t in trees for x in t], dev)
            self.tokens, self.targets = ints(tok, dev), ints(tgt, dev)
            self.qkv = randn((6 * nodes, h + 2 * hkv, d), torch.bfloat16, dev, seed + 1)
            self.rope, self.stream = Rope(d), torch.cuda.Stream()

        def step(self):
            p, s = self.pool, self.stream
            n = 6 * nodes
            lens, starts, slots, pos, masks = p.device_plan_tokens(self.stack, self.bt, self.cached, ints(self.new, dev), n,
                                                                   parents=self.parents, mask_words=1, stream=s)
            q = p.norm_rope_write_kv_slots(0, self.qkv[:, :h], self.qkv[:, h:h + hkv], self.qkv[:, h + hkv:], pos, slots,
                                           rope=self.rope, stream=s)
            out = p.tree_attention(q, 0, self.bt, lens, starts, masks, 0.125, stream=s)
            got = p.device_accept_tree(slots, self.parents, self.tokens, self.targets, lens, starts, 8, stream=s)
            p.device_trim_sequences(self.stack, self.bt, lens, got[3], stream=s)
            return [out, *got, slots, masks]

    def run(programs):
        results = [None, None]

        def work(i):
            torch.cuda.set_device(dev)
            with torch.cuda.stream(programs[i].stream):
                results[i] = programs[i].step()

        torch.cuda.synchronize()
        threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        torch.cuda.synchronize()
        return [r + [p.stack, p.bt, p.pool.pool] for r, p in zip(results, programs)]

    alone = []
    for seed in (20, 21):
        p = Program(seed)
        torch.cuda.synchronize()
        with torch.cuda.stream(p.stream):
            r = p.step()
        torch.cuda.synchronize()
        alone.append(r + [p.stack, p.bt, p.pool.pool])
    both = run([Program(20), Program(21)])
    status_is(0)
    for a, b in zip(alone, both):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


def test_refusals_on_the_device(cuda_device):
    dev, d, block, h, hkv = cuda_device, 128, 16, 8, 8
    c = tree_case(1, [4, 4], [9000, 8000], d, block, h, hkv, torch.bfloat16, dev)
    cache = BlockPool(c["nb"], block, 1, hkv, d, tensor=c["pool"])
    cache.set_prefill_kernel("tcgen05")
    args = (0, c["bt"], c["lens"], c["starts"], c["masks"], 0.1)
    need = cache.tree_workspace_size(2, 8, h, c["bt"].shape[1])
    assert need > 0
    for ws in (torch.empty(need - 256, dtype=torch.uint8, device=dev), torch.empty(need + 256, dtype=torch.uint8, device=dev)[1:]):
        with pytest.raises(B.PagedAttnError) as e:
            cache.tree_attention(c["q"], *args, workspace=ws)
        assert e.value.code == B.PA_ERR_WORKSPACE
    with pytest.raises(B.PagedAttnError) as e:
        cache.tree_attention(c["q"], *args, out=c["q"])
    assert e.value.code == B.PA_ERR_INVALID_ARG and "overlaps" in str(e.value)
    with pytest.raises(B.PagedAttnError):
        cache.tree_attention(c["q"], 1, *args[1:])
    # what is on the host, or no tensor at all
    for bad in (c["masks"].cpu(), None, 3, c["masks"].float(), c["masks"][:, :0]):
        with pytest.raises((ValueError, TypeError, AttributeError, B.PagedAttnError)):
            cache.tree_attention(c["q"], *args[:4], bad, 0.1)
    with pytest.raises((ValueError, TypeError)):
        cache.device_trim_sequences(stack_tensor([], c["nb"], dev), c["bt"], c["lens"], c["lens"].long())
    with pytest.raises((ValueError, TypeError)):
        cache.device_plan_tokens(stack_tensor([], c["nb"], dev), c["bt"], c["lens"], c["lens"], 2.5)
    rope = Rope(d)
    rope.close()
    z = torch.zeros((1, h, d), dtype=torch.bfloat16, device=dev)
    with pytest.raises(ValueError):
        cache.norm_rope_write_kv_slots(0, z, z, z, ints([0], dev), ints([0], dev, torch.int64), rope=rope)
    cache.close()
    with pytest.raises(B.PagedAttnError):
        cache.device_trim_sequences(stack_tensor([], c["nb"], dev), c["bt"], c["lens"], c["lens"])
    status_is(0)


def test_calls_need_the_current_device(cuda_device, monkeypatch):
    """A pool on another device than the current one is refused before a launch."""
    dev = cuda_device
    cache = small_pool(4, 16, dev)
    bt, lens = torch.full((1, 2), -1, dtype=torch.int32, device=dev), ints([0], dev)
    monkeypatch.setattr(cache, "_device_index", 1)
    with pytest.raises(ValueError):
        cache.device_trim_sequences(stack_tensor([], 4, dev), bt, lens, lens)


@pytest.mark.parametrize("batch,most,shape,words,pad", [
    (1, 1024, "chain", 32, 0), (1, 5000, "chain", 0, 3), (2, 6000, "random", 0, 0), (60, 1024, "chain", 32, 11), (130, 700, "random", 32, 0),
    (1100, 64, "random", 2, 5), (2000, 40, "chain", 2, 30000), (9000, 9, "wide", 1, 0), (3, 0, "chain", 1, 20),
])
def test_plan_of_many_tokens(cuda_device, batch, most, shape, words, pad):
    """Long chains, trees longer than a mask (no masks written), more rows than a round of the
    launch takes, rows behind the last sequence that take rounds of their own."""
    dev, block = cuda_device, 16
    new, cached, trees, tables, ids, nb = plan_case(np.random.default_rng(batch + most), batch, most, block, shape)
    if batch <= 2:
        new = [most] * batch
        trees = [T.random_tree(np.random.default_rng(b), most, shape) for b in range(batch)]
        cached = [0, 37][:batch]
        tables = np.full((batch, R.cdiv(most + 37, block)), -1, np.int32)
        nb = 2 * tables.size + 9
        ids = [int(x) for x in np.random.default_rng(1).permutation(nb)]
        if batch == 2:
            tables[1, :3] = [ids.pop() for _ in range(3)]
    total = sum(new) + pad
    want = T.Plan(block, tables, ids, cached, new, trees, total, words)
    cache = small_pool(nb, block, dev)
    stack, bt = stack_tensor(ids, nb, dev), ints(tables, dev)
    lens, starts, slots, positions, masks = cache.device_plan_tokens(
        stack, bt, ints(cached, dev), ints(new, dev), total, parents=ints([x for t in trees for x in t] + [5] * pad, dev),
        mask_words=words)
    status_is(0)
    assert lens.tolist() == want.lens and starts.tolist() == want.starts
    assert slots.tolist() == want.slots and positions.tolist() == want.positions
    assert not words or np.array_equal(masks.cpu().numpy(), want.masks)
    assert np.array_equal(bt.cpu().numpy(), want.tables) and stack_ids(stack) == want.stack
    cache.device_trim_sequences(stack, bt, lens, ints(cached, dev))
    assert np.array_equal(bt.cpu().numpy(), tables) and stack_ids(stack) == ids
    status_is(0)


def test_trim_frees_what_a_prompt_took(cuda_device):
    """Thousands of pages in one call, and rows of bad ids between good ones."""
    dev, block = cuda_device, 16
    nb = 6000
    cache = small_pool(nb, block, dev)
    stack = cache.device_stack()
    before = stack.clone()
    bt = torch.full((5, 1400), -1, dtype=torch.int32, device=dev)
    counts = ints([20000, 0, 17, 22000, 21000], dev)
    lens = cache.device_plan_tokens(stack, bt, ints([0] * 5, dev), counts, 63017)[0]
    assert stack_ids(stack) == stack_ids(before)[:nb - sum(R.cdiv(x, block) for x in counts.tolist())]
    cache.device_trim_sequences(stack, bt, lens, ints([0] * 5, dev))
    assert torch.equal(stack, before) and bool((bt == -1).all())
    lens = cache.device_plan_tokens(stack, bt, ints([0] * 5, dev), counts, 63017)[0]
    table = bt.cpu().numpy()
    holes = [(0, 3), (0, 900), (3, 0), (4, 1312)]
    for b, j in holes:
        bt[b, j] = nb + 5
    cache.device_trim_sequences(stack, bt, lens, ints([0] * 5, dev))
    status_is(B.PA_STATUS_BAD_BLOCK_ID)
    lost = {int(table[b, j]) for b, j in holes}
    assert stack_ids(stack) == [x for x in stack_ids(before) if x not in lost]


def test_accept_flags_a_root_with_a_parent(cuda_device):
    """Node 0 is the root whatever its parent says, but a parent that is not below it is flagged, as
    in the plan; the rest of the tree is decided as ever."""
    dev = cuda_device
    pool_t = randn((4, 2, 1, 1, 16, 64), torch.bfloat16, dev, 1)
    before = pool_t.clone()
    cache = BlockPool(4, 16, 1, 1, 64, tensor=pool_t)
    args = (ints([9, 5, 6, 9, 7], dev), ints([6, 0, 3, 7, 2], dev), ints([3, 2], dev), ints([0, 3, 5], dev), 3)
    slots = ints([0, 1, 2, 16, 17], dev, torch.int64)
    want = [[2, 2], [[0, 2, -1], [0, 1, -1]], [3, 2], [2, 2]]
    for root, status in ((-1, 0), (0, B.PA_STATUS_BAD_LENGTH), (5, B.PA_STATUS_BAD_LENGTH), (-2, B.PA_STATUS_BAD_LENGTH)):
        for parents in ([root, 0, 0, -1, 0], [-1, 0, 0, root, 0]):
            pool_t.copy_(before)
            out = cache.device_accept_tree(slots, ints(parents, dev), *args)
            status_is(status)
            assert [x.tolist() for x in out] == want
            assert torch.equal(pool_t[0, :, 0, 0, 1], before[0, :, 0, 0, 2])
            assert torch.equal(pool_t[1], before[1])
    cache.close()


@pytest.mark.parametrize("dtype,kernel", KERNELS)
@pytest.mark.parametrize("new,ctx,h,hkv,d", [([8], [508], 16, 2, 64), ([9, 25, 17, 12], [700, 3000, 1500, 2500], 32, 8, 128),
                                             ([64, 50], [3000, 2000], 8, 2, 128), ([5, 9], [20000, 30011], 8, 2, 64)])
def test_tree_attention_repeats_itself(cuda_device, dtype, kernel, new, ctx, h, hkv, d):
    """Equal calls give equal bits, whatever the workspace and the output held before."""
    dev, dt, block = cuda_device, DT[dtype], 16
    c = tree_case(17, new, ctx, d, block, h, hkv, dt, dev)
    cache = BlockPool(c["nb"], block, 1, hkv, d, tensor=c["pool"])
    cache.set_prefill_kernel(kernel)
    need = cache.tree_workspace_size(len(new), sum(new), h, c["bt"].shape[1])
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    outs = []
    for fill in (0, 255, 127):
        ws.fill_(fill)
        out = torch.full(c["q"].shape, float(fill), dtype=dt, device=dev)
        for _ in range(3):
            cache.tree_attention(c["q"], 0, c["bt"], c["lens"], c["starts"], c["masks"], d ** -0.5, out=out, workspace=ws)
            outs.append(out.clone())
    status_is(0)
    assert all(torch.equal(outs[0], x) for x in outs[1:])
