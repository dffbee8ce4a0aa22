"""Prefill attention on each of its kernels by force, where the call's own choice would
take one of them only: other layouts and layers, far pages, graphs, streams, shared
workspaces; and contexts in which every page, or every key, shows in the output."""
import numpy as np
import pytest
import torch

import prompt_reference as R
import test_prompt_ops_gpu as ops
from gpu_helpers import pool_in_layout
from paged_kv_cache_239_gb300 import binding as B
from paged_kv_cache_239_gb300 import workloads as W
from paged_kv_cache_239_gb300.pool import BlockPool
from paged_kv_cache_239_gb300.rope import Rope

pytestmark = pytest.mark.gpu

KINDS = {"mma": B.PA_PREFILL_MMA, "tcgen05": B.PA_PREFILL_TCGEN05}
BOTH = pytest.mark.parametrize("kernel", ["mma", "tcgen05"])


def ints(x, dev):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)


def randn(shape, dev, seed, scale=1.0):
    g = torch.Generator(device=dev).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=dev) * scale).to(torch.bfloat16)


def check(got, want, bound):
    assert bool(torch.isfinite(got).all())
    over = ((got.double() - want).abs() - bound).max().item()
    assert over <= 0, f"over its bound by {over:.3g}"


def ragged(dev, d, block, h, hkv, new, ctx, seed, layers=1, maxb=None):
    rng = np.random.default_rng(seed)
    nb = sum(R.cdiv(c, block) for c in ctx) + 3
    tables = R.random_tables(rng, ctx, block, nb, maxb or max(R.cdiv(c, block) for c in ctx))
    return randn((nb, 2, layers, hkv, block, d), dev, seed), tables, randn((sum(new), h, d), dev, seed + 1, 1.5)


def forced(pool_t, kernel):
    """A pool over the tensor whose prefill runs on `kernel`: the workspace of a long
    call, which the kernels lay out differently, shows that it does."""
    nb, _, layers, hkv, block, d = pool_t.shape
    cache = BlockPool(nb, block, layers, hkv, d, tensor=pool_t)
    sizes = {}
    for k in KINDS:
        cache.set_prefill_kernel(k)
        sizes[k] = cache.prefill_workspace_size(1, 4, hkv, 4096)
    cache.set_prefill_kernel(kernel)
    other = next(k for k in KINDS if k != kernel)
    assert cache.prefill_workspace_size(1, 4, hkv, 4096) == sizes[kernel] != sizes[other]
    return cache


@BOTH
@pytest.mark.parametrize("d,block,h,hkv", [(128, 16, 8, 2), (64, 32, 6, 3), (128, 32, 3, 1)])
@pytest.mark.parametrize("layout", ["fused", "separate", "layer_major"])
@pytest.mark.parametrize("new,ctx", [([40, 1, 7], [140, 33, 7]), ([300, 2], [700, 3000])])
def test_layouts(cuda_device, kernel, layout, d, block, h, hkv, new, ctx):
    """Every layout and a layer other than the first, with the append before it."""
    dev, layers, layer = cuda_device, *((1, 0) if layout == "separate" else (3, 2))
    pool_t, tables, q = ragged(dev, d, block, h, hkv, new, ctx, 10, layers)
    nb, t, maxb, batch = pool_t.shape[0], sum(new), tables.shape[1], len(new)
    wl = W.Workload("x", "bf16", layers, h, hkv, d, block, np.array(ctx, np.int32), tables, nb, 1.0, 1)
    keep, handle = pool_in_layout(wl, pool_t, layout, dev)
    B.pa_pool_set_prefill_kernel(handle, KINDS[kernel])
    k, v, rope = randn((t, hkv, d), dev, 1), randn((t, hkv, d), dev, 2), Rope(d)
    bt, ln, st = ints(tables, dev), ints(ctx, dev), ints(R.starts_of(new), dev)
    out, qr = torch.empty_like(q), torch.empty_like(q)
    B.pa_norm_rope_write_kv(handle, layer, qr, q, h * d, k, hkv * d, v, hkv * d, rope.handle, None, None,
                            0.0, bt, maxb, ln, st, batch, t, h)
    need = B.pa_prefill_workspace_size(handle, batch, t, h, maxb)
    ws = torch.empty(max(1, need), dtype=torch.uint8, device=dev)
    B.pa_prefill_attention(out, qr, handle, layer, bt, maxb, ln, st, batch, t, h, d ** -0.5, ws, need)
    cache = forced(pool_t, kernel)
    q2 = cache.norm_rope_write_kv(layer, q, k, v, bt, ln, rope=rope, query_starts=st)
    assert torch.equal(q2, qr)
    assert torch.equal(cache.prefill_attention(q2, layer, bt, ln, st, d ** -0.5), out)
    check(out, *R.prefill(pool_t, q2, tables, ctx, new, d ** -0.5, layer))
    assert B.pa_get_status() == 0
    B.pa_pool_destroy(handle)
    cache.close()
    del keep


@BOTH
def test_far_pages(cuda_device, kernel):
    """Pages beyond 2^32 bytes and 2^31 elements of the pool."""
    dev, d, block, h, hkv, new, ctx = cuda_device, 128, 32, 8, 8, [9, 33], [200, 300]
    nb = (1 << 31) // (2 * hkv * block * d) + 40
    pool_t = torch.empty((nb, 2, 1, hkv, block, d), dtype=torch.bfloat16, device=dev)
    tables = np.full((2, 10), -1, np.int32)
    tables[0, :7], tables[1, :10] = nb - 1 - 2 * np.arange(7), nb - 18 - np.arange(10)
    used = torch.as_tensor(tables[tables >= 0].astype(np.int64), device=dev)
    pool_t[used] = randn((len(used),) + tuple(pool_t.shape[1:]), dev, 2)
    q = randn((42, h, d), dev, 3)
    cache = forced(pool_t, kernel)
    got = cache.prefill_attention(q, 0, ints(tables, dev), ints(ctx, dev), ints([0, 9, 42], dev), d ** -0.5)
    assert B.pa_get_status() == 0
    small = np.full_like(tables, -1)
    small[tables >= 0] = np.arange(len(used))
    check(got, *R.prefill(pool_t[used], q, small, ctx, new, d ** -0.5))
    cache.close()


@BOTH
def test_graphs_with_one_workspace(cuda_device, kernel):
    """Two captured calls of different layers that share a workspace, replayed in turns with
    new lengths, queries and row counts in their buffers."""
    dev, d, block, h, hkv = cuda_device, 128, 16, 8, 2
    pool_t, tables, q = ragged(dev, d, block, h, hkv, [5, 3], [3000, 2000], 13, layers=2, maxb=200)
    cache = forced(pool_t, kernel)
    bt, ln, st = ints(tables, dev), ints([3000, 2000], dev), ints([0, 5, 8], dev)
    need = cache.prefill_workspace_size(2, 8, h, 200)
    assert need > 0
    ws, outs, graphs = torch.empty(need, dtype=torch.uint8, device=dev), [], []
    for layer in range(2):
        outs.append(torch.empty_like(q))
        args = (q, layer, bt, ln, st, d ** -0.5, outs[layer], ws)
        cache.prefill_attention(*args)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[layer]):
            cache.prefill_attention(*args)
    for new, ctx in (([5, 3], [3000, 2000]), ([2, 6], [1999, 1500]), ([8, 0], [70, 0]), ([1, 7], [1, 2000]),
                     ([0, 1], [0, 1]), ([4, 4], [3000, 4])):
        ln.copy_(ints(ctx, dev)), st.copy_(ints(R.starts_of(new), dev))
        q.copy_(randn(q.shape, dev, sum(ctx)))
        outs[0].fill_(7.0), outs[1].fill_(7.0)
        for _ in range(3):
            graphs[0].replay(), graphs[1].replay()
        torch.cuda.synchronize()
        t = sum(new)
        for layer in range(2):
            check(outs[layer][:t], *R.prefill(pool_t, q[:t], tables, ctx, new, d ** -0.5, layer))
            assert bool((outs[layer][t:] == 7.0).all())
    assert B.pa_get_status() == 0
    cache.close()


@BOTH
@pytest.mark.parametrize("new,ctx", [([300, 200], [900, 700]), ([3, 5], [3000, 9000])])
def test_streams(cuda_device, kernel, new, ctx):
    """Calls side by side on two streams, each with a workspace of its own (the call's, or
    given), over one pool: the bits of the calls alone."""
    dev, d, h = cuda_device, 128, 8
    pool_t, tables, q = ragged(dev, d, 16, h, 2, new, ctx, 12)
    cache = forced(pool_t, kernel)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    args = [(0, ints(tables[b:b + 1], dev), ints([ctx[b]], dev), ints([0, new[b]], dev), d ** -0.5) for b in range(2)]
    qs = [q[:new[0]].contiguous(), q[new[0]:].contiguous()]
    ws = [torch.empty(max(1, cache.prefill_workspace_size(1, n, h, tables.shape[1])), dtype=torch.uint8, device=dev)
          for n in new]
    outs = [torch.empty_like(x) for x in qs]
    alone = [cache.prefill_attention(x, *a) for x, a in zip(qs, args)]
    check(torch.cat(alone), *R.prefill(pool_t, q, tables, ctx, new, d ** -0.5))
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        got.append([cache.prefill_attention(x, *a, stream=s) for x, a, s in zip(qs, args, streams)])
        for i in range(2):
            cache.prefill_attention(qs[i], *args[i], out=outs[i], workspace=ws[i], stream=streams[i])
    torch.cuda.synchronize()
    assert B.pa_get_status() == 0
    for pair in got + [outs]:
        assert all(torch.equal(x, y) for x, y in zip(pair, alone))
    cache.close()


@BOTH
def test_workspace_refusals(cuda_device, kernel):
    dev = cuda_device
    pool_t, tables, q = ragged(dev, 128, 16, 8, 1, [3], [9000], 14)
    cache = forced(pool_t, kernel)
    need = cache.prefill_workspace_size(1, 3, 8, tables.shape[1])
    assert need > 0
    ws = torch.empty(need + 512, dtype=torch.uint8, device=dev)
    args = (q, 0, ints(tables, dev), ints([9000], dev), ints([0, 3], dev), 0.1)
    for bad in (ws[:need - 1], ws[4:], ws[:0]):
        with pytest.raises(B.PagedAttnError) as e:
            cache.prefill_attention(*args, workspace=bad)
        assert e.value.code == B.PA_ERR_WORKSPACE
    with pytest.raises(B.PagedAttnError):
        cache.prefill_attention(*args, out=q, workspace=ws)
    check(cache.prefill_attention(*args, workspace=ws[:need]), *R.prefill(pool_t, q, tables, [9000], [3], 0.1))
    cache.close()


@pytest.mark.parametrize("kernel", ["mma", "tcgen05", "f32"])
@pytest.mark.parametrize("d,h,hkv", [(128, 8, 2), (64, 16, 1), (64, 3, 3)])
@pytest.mark.parametrize("unit,new,ctx", [
    (16, [4], [20000]), (16, [3, 0, 5, 1], [9000, 0, 33000, 17000]), (16, [300], [9000]), (16, [1] * 9, [8200] * 9),
    (1, [2], [3001]), (1, [130, 7], [1500, 2999]), (1, [1000], [1000]), (1, [5] * 20, [1100] * 20),
])
def test_every_page_or_key_counts(cuda_device, kernel, d, h, hkv, unit, new, ctx):
    """Values that say which unit (a page, or a key) they come from: the key in place s adds
    its weight to column s / unit % d alone, whose share of a context is small enough that
    one unit left out or taken twice is off by more than the bound.  (All values are 0 or 1,
    so the bound is relative to the output: at bf16 2^-8 for the weights, 2^-8 for the output
    and 2^-23 for each key, 1.2 % at 33,000; the scores differ by about 0.04, and a
    column has up to 33,000 / 16 / 64 = 33 pages or 3,000 / 64 = 47 keys.)"""
    dev = cuda_device
    pool_t, tables, q = ragged(dev, d, 16, h, hkv, new, ctx, 20)
    for b, c in enumerate(ctx):
        at = torch.arange(R.cdiv(c, 16) * 16, device=dev)
        code = torch.nn.functional.one_hot(at // unit % d, d).to(pool_t.dtype).view(-1, 1, 16, d)
        pool_t[torch.as_tensor(tables[b, :R.cdiv(c, 16)], device=dev).long(), 1, 0] = code
    pool_t[:, 0] *= 0.25
    if kernel == "f32":
        pool_t, q = pool_t.float(), q.float()
        cache = BlockPool(pool_t.shape[0], 16, 1, hkv, d, tensor=pool_t)
    else:
        cache = forced(pool_t, kernel)
    scale = 0.1 * d ** -0.5
    got = cache.prefill_attention(q, 0, ints(tables, dev), ints(ctx, dev), ints(R.starts_of(new), dev), scale)
    assert B.pa_get_status() == 0
    want, bound = R.prefill(pool_t, q, tables, ctx, new, scale)
    check(got, want, bound)
    # the bound is tight enough: the reference without one unit is outside it
    b = int(np.argmax(ctx))
    row, at = int(R.starts_of(new)[b + 1]) - 1, ctx[b] // 2 // unit * unit
    group, col = h // hkv, at // unit % d
    keys = torch.as_tensor(tables[b, :R.cdiv(ctx[b], 16)], device=dev).long()
    k = pool_t[keys, 0, 0].double().permute(1, 0, 2, 3).reshape(hkv, -1, d)[:, :ctx[b]]
    p = torch.einsum("hgd,htd->hgt", q[row].double().view(hkv, group, d), k).mul(scale).softmax(-1)
    lost = p[:, :, at:at + unit].sum(-1).reshape(h)
    short = (want[row, :, col] - lost) / (1 - lost)
    assert bool(((short - want[row, :, col]).abs() > 2 * bound[row, :, col]).all())
    cache.close()


@BOTH
@pytest.mark.parametrize("d,h,hkv", [(128, 8, 2), (64, 16, 2)])
def test_serving_run(cuda_device, kernel, d, h, hkv, monkeypatch):
    """The run of all calls together, its attention on the one kernel."""

    class Forced(BlockPool):
        def __init__(self, *args, **kw):
            super().__init__(*args, **kw)
            self.set_prefill_kernel(kernel)

    monkeypatch.setattr(ops, "BlockPool", Forced)
    ops.test_serving_run(cuda_device, "bf16", d, h, hkv)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("h,hkv,new,ctx", [(8, 2, [2048], [4096]), (16, 4, [700, 600], [3000, 5000]),
                                           (16, 2, [4], [60000])])
def test_f32_sums_do_not_drift(cuda_device, d, h, hkv, new, ctx):
    """fp32 outputs over thousands of keys are off by what roundings to nearest leave, not by
    a share that grows with the context (a sum kept in the tensor core's accumulator is
    cut toward zero at every step).

    The drift is the mean of error * sign, relative to the mean magnitude: random errors
    leave nothing of it.  Inside one tile of at most 32 keys 12 products are summed in the
    tensor core and each cut by at most 2^-23, half on average: 12 * 2^-24.  Scores are
    cut D / 8 times, on average by 2^-25 of themselves, which moves an output by as much
    for scores of size 1: D / 8 * 2^-25.  Errors of either sign beside it: an addition
    to O per tile, 2^-24 each, grows by its root (at most 16 of them at 4,096 keys unsplit),
    the exponent's rounding and ex2 (2^-22): 2^-20 in all."""
    dev = cuda_device
    pool_t, tables, q = ragged(dev, d, 16, h, hkv, new, ctx, 30)
    pool_t, q = pool_t.float(), q.float() / 1.5
    cache = BlockPool(pool_t.shape[0], 16, 1, hkv, d, tensor=pool_t)
    got = cache.prefill_attention(q, 0, ints(tables, dev), ints(ctx, dev), ints(R.starts_of(new), dev), d ** -0.5)
    want, _ = R.prefill(pool_t, q, tables, ctx, new, d ** -0.5)
    err = got.double() - want
    drift = (err * want.sign()).mean() / want.abs().mean()
    limit = 12 * 2.0 ** -24 + d / 8 * 2.0 ** -25
    assert abs(drift.item()) <= limit, f"drift {drift.item():.2e}, limit {limit:.2e}"
    rms = (err.pow(2).mean() / want.pow(2).mean()).sqrt().item()
    assert rms <= limit + 2.0 ** -20, f"rms {rms:.2e}"
    cache.close()
