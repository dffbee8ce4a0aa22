"""GPU parity of the operators for several new tokens per sequence and of the
page operations against plain 64-bit implementations, at the sizes, masks and
inputs where they can go wrong, and a run of all of them together."""
import numpy as np
import pytest
import torch

import prompt_reference as R
from gpu_helpers import pool_in_layout
from paged_kv_cache_239_gb300 import binding as B
from paged_kv_cache_239_gb300 import workloads as W
from paged_kv_cache_239_gb300.pool import BlockPool
from paged_kv_cache_239_gb300.rope import Rope

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def ints(x, dev):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)


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


# --------------------------------------------------------- norm + rotation

ROPES = [
    ("none", False, None), ("none", True, None), ("linear", False, 4.0), ("parts", True, 8.0),
    ("ntk", False, 2.0), (None, False, None),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,block,h,hkv", [(64, 16, 16, 2), (128, 32, 3, 3), (128, 16, 10, 2), (64, 32, 1, 1)])
@pytest.mark.parametrize("rope", range(len(ROPES)))
@pytest.mark.parametrize("norm", [True, False])
def test_norm_rope(cuda_device, dtype, d, block, h, hkv, rope, norm):
    dev, dt = cuda_device, DT[dtype]
    scaling, interleaved, factor = ROPES[rope]
    rng = np.random.default_rng(7 + d + rope)
    new = [0, 1, 5, 33, 2, 0]
    ctx = [0, 1, 5, 33 + 47, 131072, 9]
    starts = R.starts_of(new)
    t = int(starts[-1])
    maxb = R.cdiv(max(ctx), block)
    nb = 64
    tables = np.full((len(ctx), maxb), -1, np.int32)   # only the new tokens' pages are needed
    ids = [int(x) for x in rng.permutation(nb)]
    for b, (n, c) in enumerate(zip(new, ctx)):
        for j in range((c - n) // block, R.cdiv(c, block) if n else 0):
            tables[b, j] = ids.pop()
    rotary = d if rope % 2 == 0 else d // 2 + 16
    r = freq = None
    if scaling is not None:
        amp = 1.25 if scaling == "parts" else 1.0
        r = Rope(rotary, base=10000.0, interleaved=interleaved, scaling=scaling, factor=factor or 1.0,
                 original_len=4096, amplitude=amp)
        freq = R.frequencies(rotary, 10000.0, scaling, factor or 1.0, 4096.0)
    else:
        amp = 1.0
    pad = 3   # rows behind the last sequence
    qkv = randn((t + pad, h + 2 * hkv, d), dt, dev, 1)
    q, k, v = qkv[:, :h], qkv[:, h:h + hkv], qkv[:, h + hkv:]
    w = [randn((d,), dt, dev, 2 + i, 0.3) + 1 if norm else None for i in range(2)]
    w = [None if x is None else x.to(dt) for x in w]
    pool_t = randn((nb, 2, 2, hkv, block, d), dt, dev, 5)
    before = pool_t.clone()
    cache = BlockPool(nb, block, 2, hkv, d, tensor=pool_t)
    out = torch.full((t + pad, h, d), 7.0, dtype=dt, device=dev)
    cache.norm_rope_write_kv(1, q, k, v, ints(tables, dev), ints(ctx, dev), rope=r, q_weight=w[0],
                             k_weight=w[1], eps=1e-5, query_starts=ints(starts, dev), out=out)
    status_is(0)
    pos = torch.cat([torch.arange(c - n, c) for n, c in zip(new, ctx)]).to(dev)
    want_q, size_q = R.norm_rope(q[:t], pos, freq, interleaved, amp, w[0], 1e-5)
    check(out[:t], want_q, R.norm_rope_bound(want_q, size_q, dt))
    assert bool((out[t:] == 7.0).all())
    want_k, size_k = R.norm_rope(k[:t], pos, freq, interleaved, amp, w[1], 1e-5)
    bound_k = R.norm_rope_bound(want_k, size_k, dt)
    i = 0
    for b, (n, c) in enumerate(zip(new, ctx)):
        for p in range(c - n, c):
            page = int(tables[b, p // block])
            row = pool_t[page, :, 1, :, p % block]
            check(row[0], want_k[i], bound_k[i])
            assert torch.equal(row[1], v[i])
            pool_t[page, :, 1, :, p % block] = before[page, :, 1, :, p % block]
            i += 1
    assert torch.equal(pool_t, before)   # nothing else was touched
    cache.close()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_rope_one_token_each_and_in_place(cuda_device, dtype):
    dev, dt, d, block, h, hkv = cuda_device, DT[dtype], 128, 16, 8, 2
    ctx = [1, 16, 17, 300, 4096]
    rng = np.random.default_rng(3)
    tables = R.random_tables(rng, ctx, block, 300, 257)
    pool_t = torch.zeros((300, 2, 1, hkv, block, d), dtype=dt, device=dev)
    cache, r = BlockPool(300, block, 1, hkv, d, tensor=pool_t), Rope(d)
    q, k, v = (randn((5, n, d), dt, dev, n) for n in (h, hkv, hkv))
    pos = ints(ctx, dev) - 1
    want, size = R.norm_rope(q, pos, R.frequencies(d, 10000.0), False, 1.0, None, 0.0)
    a = cache.norm_rope_write_kv(0, q, k, v, ints(tables, dev), ints(ctx, dev), rope=r)
    check(a, want, R.norm_rope_bound(want, size, dt))
    b = q.clone()
    assert cache.norm_rope_write_kv(0, b, k, v, ints(tables, dev), ints(ctx, dev), rope=r, out=b) is b
    assert torch.equal(a, b)
    # the keys are those of the positions: the same as rotating them as queries
    c = cache.norm_rope_write_kv(0, k.repeat_interleave(h // hkv, 1), k, v, ints(tables, dev),
                                 ints(ctx, dev), rope=r)
    for i, n in enumerate(ctx):
        page = int(tables[i, (n - 1) // block])
        assert torch.equal(pool_t[page, 0, 0, :, (n - 1) % block], c[i, ::h // hkv])
    status_is(0)


def test_norm_rope_far_positions(cuda_device):
    """Positions near 2^31: the angle is as exact as near 0."""
    dev, d, block = cuda_device, 64, 16
    maxb = (1 << 31) // block - 1
    n = maxb * block
    tables = torch.zeros((1, maxb), dtype=torch.int32, device=dev)
    pool_t = torch.zeros((1, 2, 1, 1, block, d), device=dev)
    cache = BlockPool(1, block, 1, 1, d, tensor=pool_t)
    x = randn((1, 1, d), torch.float32, dev, 1)
    freq = R.frequencies(d, 10000.0)
    got = cache.norm_rope_write_kv(0, x, x, x, tables, ints([n], dev), rope=Rope(d))
    want, size = R.norm_rope(x, torch.tensor([n - 1], device=dev), freq, False, 1.0, None, 0.0)
    # the reference's own angle: p f up to 2^31, half a step 2^-22 of 64-bit floats
    check(got, want, R.norm_rope_bound(want, size, torch.float32) + 2.0 ** -22 * size)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope_infinities_stay_in_their_pairs(cuda_device, dtype, interleaved):
    """An infinite element reaches its own pair of its own head, the part that does
    not turn keeps it to itself, and values are copied whatever they are."""
    dev, d, block, dt = cuda_device, 64, 16, DT[dtype]
    cache = BlockPool(2, block, 1, 2, d, tensor=torch.zeros((2, 2, 1, 2, block, d), dtype=dt, device=dev))
    q, k, v = (randn((1, 2, d), dt, dev, i) for i in range(3))
    q[0, 0, 3], q[0, 0, 50], v[0, 1, 7] = float("inf"), -float("inf"), float("nan")
    out = cache.norm_rope_write_kv(0, q, k, v, ints([[1]], dev), ints([3], dev),
                                   rope=Rope(32, interleaved=interleaved))
    pair = [2, 3] if interleaved else [3, 19]
    bad = (~torch.isfinite(out[0])).nonzero().tolist()
    assert bad == [[0, pair[0]], [0, pair[1]], [0, 50]] and float(out[0, 0, 50]) == -float("inf")
    assert torch.equal(out[0, :, 32:50], q[0, :, 32:50])
    assert torch.equal(cache.pool[1, 1, 0, :, 2].nan_to_num(5.0), v[0].nan_to_num(5.0))
    assert torch.equal(cache.norm_rope_write_kv(0, q, k, v, ints([[1]], dev), ints([3], dev)), q)


def test_norm_rope_bad_inputs(cuda_device):
    dev, d, block, dt = cuda_device, 64, 16, torch.bfloat16
    pool_t = torch.zeros((4, 2, 1, 1, block, d), dtype=dt, device=dev)
    cache, r = BlockPool(4, block, 1, 1, d, tensor=pool_t), Rope(d)
    q, k = randn((6, 2, d), dt, dev, 1), randn((6, 1, d), dt, dev, 2)
    # sequence 0: more new tokens than context; 1: longer than its table; 2: a bad page; 3: fine
    starts, ctx = ints([0, 2, 3, 5, 6], dev), ints([1, 33, 2, 1], dev)
    tables = ints([[0, 1], [0, 1], [9, 1], [3, -1]], dev)
    out = cache.norm_rope_write_kv(0, q, k, k, tables, ctx, rope=r, query_starts=starts)
    status_is(B.PA_STATUS_BAD_LENGTH | B.PA_STATUS_BAD_BLOCK_ID)
    assert not out[:3].any() and bool((out[3:] != 0).any(-1).all())
    assert not pool_t[:3].any() and bool(pool_t[3, :, 0, 0, 0].any())
    # lengths below zero, and a block id below zero
    cache.norm_rope_write_kv(0, q[:1], k[:1], k[:1], ints([[-5]], dev), ints([1], dev), rope=r)
    status_is(B.PA_STATUS_BAD_BLOCK_ID)
    cache.norm_rope_write_kv(0, q[:1], k[:1], k[:1], ints([[1]], dev), ints([-1], dev), rope=r)
    status_is(B.PA_STATUS_BAD_LENGTH)


# ----------------------------------------------------------------- prefill


KERNEL = ["auto"]  # what run_prefill asks for on bf16 pools


def pytest_generate_tests(metafunc):
    if metafunc.function.__name__.startswith("test_prefill_"):
        metafunc.parametrize("prefill_kernel", ["auto", "mma", "tcgen05"], indirect=True)


@pytest.fixture(autouse=True)
def prefill_kernel(request):
    KERNEL[0] = getattr(request, "param", "auto")
    params = request.node.callspec.params if hasattr(request.node, "callspec") else {}
    if KERNEL[0] != "auto" and params.get("dtype") == "f32":
        pytest.skip("one kernel serves fp32 pools")
    yield
    KERNEL[0] = "auto"


def prefill_case(dev, dtype, d, block, h, hkv, new, ctx, seed=0, layers=1, layer=0, fill=None, maxb=None):
    """Pool (unused rows `fill`), tables and q of a ragged batch."""
    dt = DT[dtype]
    rng = np.random.default_rng(seed + 17)
    nblk = sum(R.cdiv(c, block) for c in ctx)
    nb = nblk + 3
    maxb = maxb or max(1, max(R.cdiv(c, block) for c in ctx))
    tables = R.random_tables(rng, ctx, block, nb, maxb)
    pool_t = randn((nb, 2, layers, hkv, block, d), dt, dev, seed)
    if fill is not None:
        keep = torch.zeros((nb, block), dtype=torch.bool)
        for b, c in enumerate(ctx):
            for j in range(R.cdiv(c, block)):
                keep[tables[b, j], :min(block, c - j * block)] = True
        pool_t = torch.where(keep.to(dev)[:, None, None, None, :, None], pool_t,
                             torch.tensor(fill, dtype=dt, device=dev))
    q = randn((int(sum(new)), h, d), dt, dev, seed + 1, 1.5)
    return pool_t, tables, q


def run_prefill(dev, pool_t, tables, q, new, ctx, scale=None, layer=0, pad=2):
    nb, _, layers, hkv, block, d = pool_t.shape
    cache = BlockPool(nb, block, layers, hkv, d, tensor=pool_t)
    cache.set_prefill_kernel(KERNEL[0])
    t = q.shape[0]
    qp = torch.cat((q, torch.full((pad,) + q.shape[1:], float("nan"), dtype=q.dtype, device=dev)))
    out = torch.full_like(qp, 7.0)
    scale = d ** -0.5 if scale is None else scale
    cache.prefill_attention(qp, layer, ints(tables, dev), ints(ctx, dev), ints(R.starts_of(new), dev),
                            scale, out=out)
    torch.cuda.synchronize()
    assert bool((out[t:] == 7.0).all()), "rows behind the last sequence were written"
    cache.close()
    return out[:t]


RAGGED = [
    ([1], [1]), ([1], [300]), ([2, 0, 1], [2, 0, 65]), ([7], [7]), ([33, 1, 64], [33, 129, 64]),
    ([127, 128, 129], [127, 140, 500]), ([5, 3], [1029, 2051]), ([257], [1000]), ([0, 0, 31], [5, 0, 31]),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,block,h,hkv", [(64, 16, 16, 2), (128, 16, 32, 8), (128, 32, 4, 4), (64, 32, 5, 1),
                                           (128, 16, 6, 2), (128, 32, 7, 1), (64, 16, 32, 2), (128, 16, 40, 1)])
@pytest.mark.parametrize("case", range(len(RAGGED)))
def test_prefill_ragged(cuda_device, dtype, d, block, h, hkv, case):
    """Lengths from one token up, odd groups, empty sequences; what is not in
    any context is NaN."""
    new, ctx = RAGGED[case]
    pool_t, tables, q = prefill_case(cuda_device, dtype, d, block, h, hkv, new, ctx, seed=case,
                                     fill=float("nan"))
    got = run_prefill(cuda_device, pool_t, tables, q, new, ctx)
    status_is(0)
    check(got, *R.prefill(pool_t, q, tables, ctx, new, d ** -0.5))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,h,hkv,new,ctx", [
    (128, 32, 8, [1500], [1500]), (64, 16, 2, [700, 900], [1000, 900]), (128, 8, 8, [400], [3000]),
    (128, 16, 1, [300, 20], [2000, 9000]), (64, 3, 3, [1025], [1025]),
    (128, 32, 8, [3, 5, 4, 1], [9000, 4097, 20000, 33]), (64, 16, 2, [5] * 20, list(range(40, 840, 40))),
])
def test_prefill_longer(cuda_device, dtype, d, h, hkv, new, ctx):
    pool_t, tables, q = prefill_case(cuda_device, dtype, d, 16, h, hkv, new, ctx, seed=3, fill=float("inf"))
    got = run_prefill(cuda_device, pool_t, tables, q, new, ctx)
    status_is(0)
    check(got, *R.prefill(pool_t, q, tables, ctx, new, d ** -0.5))
    again = run_prefill(cuda_device, pool_t, tables, q, new, ctx)
    assert torch.equal(got, again)   # no order of additions depends on timing


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
def test_prefill_scales(cuda_device, dtype, scale):
    """Uniform weights, reversed ones, and nearly one-hot ones."""
    new, ctx = [70, 9], [170, 200]
    pool_t, tables, q = prefill_case(cuda_device, dtype, 128, 16, 8, 2, new, ctx, seed=5)
    got = run_prefill(cuda_device, pool_t, tables, q, new, ctx, scale=scale)
    check(got, *R.prefill(pool_t, q, tables, ctx, new, scale))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,h,hkv", [(128, 8, 2), (64, 6, 2), (128, 2, 2)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_prefill_future_values_do_not_reach_earlier_rows(cuda_device, dtype, d, h, hkv, bad):
    """K and V of a later new token are not finite: rows before it are as if it
    were not there; rows from it on show it."""
    new, ctx, at = [200, 30], [300, 30], 180   # new token 180 of sequence 0: position 280
    pool_t, tables, q = prefill_case(cuda_device, dtype, d, 16, h, hkv, new, ctx, seed=6)
    clean, bound = R.prefill(pool_t, q, tables, ctx, new, d ** -0.5)
    page, row = int(tables[0, 280 // 16]), 280 % 16
    pool_t[page, 1, 0, :, row, 3] = bad
    got = run_prefill(cuda_device, pool_t, tables, q, new, ctx)
    check(got[:at], clean[:at], bound[:at])
    check(got[200:], clean[200:], bound[200:])
    seen = got[at:200, :, 3]
    assert bool(torch.isnan(seen).all()) if bad != bad else bool((seen == bad).all())
    rest = [c for c in range(d) if c != 3]
    check(got[at:200][..., rest], clean[at:200][..., rest], bound[at:200][..., rest])
    pool_t[page, 0, 0, :, row] = float("nan")   # the key as well
    got = run_prefill(cuda_device, pool_t, tables, q, new, ctx)
    check(got[:at], clean[:at], bound[:at])
    assert bool(torch.isnan(got[at:200]).all())
    check(got[200:], clean[200:], bound[200:])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf")])
def test_prefill_infinite_key(cuda_device, dtype, bad):
    """One infinite element of a cached key: a score of -inf has no weight, one of
    +inf makes its row NaN."""
    new, ctx, d = [40, 3], [140, 50], 64
    pool_t, tables, q = prefill_case(cuda_device, dtype, d, 16, 6, 2, new, ctx, seed=9)
    pool_t[int(tables[0, 2]), 0, 0, :, 5, 7] = bad   # position 37 of sequence 0
    down = (q[:40, :, 7] * bad) < 0                  # rows to which that key is -inf
    got = run_prefill(cuda_device, pool_t, tables, q, new, ctx)
    assert bool(torch.isnan(got[:40][~down]).all()) and bool(down.any()) and not bool(down.all())
    # without that key, in 64 bits; the bound is that of `R.prefill`
    pages = torch.as_tensor(tables[0, :9].astype(np.int64), device=cuda_device)
    k, v = pool_t[pages, :, 0].double().permute(1, 2, 0, 3, 4).reshape(2, 2, -1, d)[:, :, :140]
    k, v = k.repeat_interleave(3, 0).clone(), v.repeat_interleave(3, 0)
    k[:, 37] = 0
    x = q[:40].double()
    see = torch.arange(140, device=cuda_device) <= torch.arange(100, 140, device=cuda_device)[:, None]
    see = see & (torch.arange(140, device=cuda_device) != 37)
    p = torch.softmax((torch.einsum("nhd,htd->nht", x, k) * d ** -0.5)
                      .masked_fill(~see[:, None], -float("inf")), -1)
    size = torch.einsum("nhd,htd->nht", x.abs(), k.abs()).amax(-1, keepdim=True) * d ** -0.5
    rel = 2 * ((d + 4) * R.U * size + 2.0 ** -22) + 2 * 148 * R.U + (2.0 ** -8 if dtype == "bf16" else 0)
    want = torch.einsum("nht,htd->nhd", p, v)
    bound = R.HALF_STEP[DT[dtype]] * want.abs() * (1 + rel) + rel * torch.einsum("nht,htd->nhd", p, v.abs())
    check(got[:40][down], want[down], bound[down])
    clean = prefill_case(cuda_device, dtype, d, 16, 6, 2, new, ctx, seed=9)[0]
    want, bound = R.prefill(clean, q, tables, ctx, new, d ** -0.5)
    check(got[40:], want[40:], bound[40:])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("batch,most,extra", [(40, 70, 300), (130, 3, 2000), (500, 4, 60), (1200, 1, 20)])
def test_prefill_many_sequences(cuda_device, dtype, batch, most, extra):
    """Batches that the schedule takes in one warp, in all warps and in several turns."""
    rng = np.random.default_rng(batch)
    new = [int(x) for x in rng.integers(0, most + 1, batch)]
    ctx = [n + int(rng.integers(0, extra + 1)) for n in new]
    pool_t, tables, q = prefill_case(cuda_device, dtype, 64, 16, 8, 2, new, ctx, seed=batch)
    got = run_prefill(cuda_device, pool_t, tables, q, new, ctx)
    status_is(0)
    check(got, *R.prefill(pool_t, q, tables, ctx, new, 64 ** -0.5))


def test_prefill_two_streams_at_once(cuda_device):
    """Calls side by side on two streams, each with its own workspace, over one pool."""
    dev, cases = cuda_device, []
    pool_t, tables, q = prefill_case(dev, "bf16", 128, 16, 8, 2, [300, 200], [900, 700], seed=12)
    cache = BlockPool(pool_t.shape[0], 16, 1, 2, 128, tensor=pool_t)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    args = [(0, ints(tables[b:b + 1], dev), ints([c], dev), ints([0, n], dev), 128 ** -0.5)
            for b, (n, c) in enumerate([(300, 900), (200, 700)])]
    qs = [q[:300].contiguous(), q[300:].contiguous()]
    alone = [cache.prefill_attention(x, *a) for x, a in zip(qs, args)]
    torch.cuda.synchronize()
    for _ in range(20):
        cases.append([cache.prefill_attention(x, *a, stream=s) for x, a, s in zip(qs, args, streams)])
    torch.cuda.synchronize()
    status_is(0)
    for outs in cases:
        assert all(torch.equal(x, y) for x, y in zip(outs, alone))
    cache.close()


def test_calls_need_the_current_device(cuda_device, monkeypatch):
    cache = BlockPool(4, 16, 1, 2, 64)
    ids = ints([0], cuda_device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="current CUDA device"):
        cache.copy_blocks(ids, ids)
    cache.close()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,h,hkv", [(128, 8, 2), (64, 6, 2), (64, 16, 1)])
def test_prefill_few_rows_long_contexts(cuda_device, dtype, d, h, hkv):
    """Contexts of several key tiles behind a handful of rows: pages that are missing,
    maxima that rise along the context, values that only the last rows see."""
    new, ctx, at = [9, 1, 5, 8], [1200, 513, 777, 2050], 6
    pool_t, tables, q = prefill_case(cuda_device, dtype, d, 16, h, hkv, new, ctx, seed=15, fill=float("nan"))
    for j in range(ctx[0] // 16):
        pool_t[int(tables[0, j]), 0] *= 1 + j / 8
    tables[2, 3], tables[2, 20] = -1, 10 ** 6     # pages of sequence 2 that are not there
    clean, bound = R.prefill(pool_t, q, tables, ctx, new, d ** -0.5)
    got = run_prefill(cuda_device, pool_t, tables, q, new, ctx)
    status_is(B.PA_STATUS_BAD_BLOCK_ID)
    check(got, clean, bound)
    pos = ctx[0] - new[0] + at
    pool_t[int(tables[0, pos // 16]), 1, 0, :, pos % 16, d - 1] = -float("inf")
    got = run_prefill(cuda_device, pool_t, tables, q, new, ctx)
    status_is(B.PA_STATUS_BAD_BLOCK_ID)
    check(got[:at], clean[:at], bound[:at])
    check(got[9:], clean[9:], bound[9:])
    check(got[at:9, :, :d - 1], clean[at:9, :, :d - 1], bound[at:9, :, :d - 1])
    assert not bool(torch.isfinite(got[at:9, :, d - 1]).any())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new,ctx", [([4], [9000]), ([300], [1200]), ([3] * 9, [700] * 9)])
def test_prefill_infinite_values_of_tiny_weight(cuda_device, dtype, new, ctx):
    """Scores so far apart that most weights are below the smallest number, where 0 *
    inf is NaN: a value that is infinite shows as not finite in every row that sees
    it, also where the keys are taken in parts, and in no other column."""
    d = 128
    pool_t, tables, q = prefill_case(cuda_device, dtype, d, 16, 8, 2, new, ctx, seed=13)
    for b, c in enumerate(ctx):
        for i in range(7, c - max(new), 97):
            pool_t[int(tables[b, i // 16]), 1, 0, :, i % 16, i % d] = float("inf")
    got = run_prefill(cuda_device, pool_t, tables, q, new, ctx, scale=4.0).float()
    status_is(0)
    start = 0
    for b, (n, c) in enumerate(zip(new, ctx)):
        cols = sorted({i % d for i in range(7, c - max(new), 97)})
        rest = [x for x in range(d) if x not in cols]
        assert not bool(torch.isfinite(got[start:start + n][..., cols]).any())
        assert bool(torch.isfinite(got[start:start + n][..., rest]).all())
        start += n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefill_large_scores(cuda_device, dtype):
    """Rows whose maximum rises by hundreds along the context."""
    new, ctx, d = [40], [700], 128
    pool_t, tables, q = prefill_case(cuda_device, dtype, d, 16, 4, 1, new, ctx, seed=8)
    for j in range(R.cdiv(700, 16)):
        pool_t[int(tables[0, j]), 0] *= 1.0 + 0.25 * j
    got = run_prefill(cuda_device, pool_t, tables, q, new, ctx)
    check(got, *R.prefill(pool_t, q, tables, ctx, new, d ** -0.5))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,hkv", [(128, 2), (64, 1)])
def test_prefill_bad_pages_and_lengths(cuda_device, dtype, d, hkv):
    """Pages outside the pool have no weight (a row left with none is zero); a
    sequence with a bad length gives zero rows; the others are as ever."""
    new, ctx = [30, 10, 5, 12], [200, 10, 40, 300]
    pool_t, tables, q = prefill_case(cuda_device, dtype, d, 16, 4, hkv, new, ctx, seed=9)
    good, good_bound = R.prefill(pool_t, q, tables, ctx, new, d ** -0.5)
    tables[0, 3], tables[0, 12], tables[1, 0] = pool_t.shape[0], -7, 1 << 30
    got = run_prefill(cuda_device, pool_t, tables, q, new, ctx)
    status_is(B.PA_STATUS_BAD_BLOCK_ID)
    check(got, *R.prefill(pool_t, q, tables, ctx, new, d ** -0.5))
    assert not got[30:40].any()
    for wrong in ([200, 10, 4, 300], [200, 10, 40, 16 * tables.shape[1] + 1], [200, 10, -1, 300]):
        got = run_prefill(cuda_device, pool_t, tables, q, new, wrong)
        assert B.pa_get_status() & B.PA_STATUS_BAD_LENGTH
        zero = slice(40, 45) if wrong[2] != 40 else slice(45, 57)
        assert not got[zero].any()
        same = slice(45, 57) if wrong[2] != 40 else slice(40, 45)
        check(got[same], good[same], good_bound[same])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["fused", "separate", "layer_major"])
def test_prefill_and_append_layouts(cuda_device, dtype, layout):
    """Every pool layout, a layer other than the first, against the fused one."""
    dev, d, block, h, hkv = cuda_device, 128, 16, 8, 2
    layers, layer = (1, 0) if layout == "separate" else (3, 2)
    new, ctx = [40, 1, 7], [140, 33, 7]
    pool_t, tables, q = prefill_case(dev, dtype, d, block, h, hkv, new, ctx, seed=10, layers=layers)
    nb = pool_t.shape[0]
    wl = W.Workload("x", dtype, layers, h, hkv, d, block, np.array(ctx, np.int32), tables, nb, 1.0, 1)
    keep, handle = pool_in_layout(wl, pool_t, layout, dev)
    k, v = randn((48, hkv, d), DT[dtype], dev, 1), randn((48, hkv, d), DT[dtype], dev, 2)
    rope = Rope(d)
    bt, ln, st = ints(tables, dev), ints(ctx, dev), ints(R.starts_of(new), dev)
    out, qr = torch.empty_like(q), torch.empty_like(q)
    B.pa_norm_rope_write_kv(handle, layer, qr, q, h * d, k, hkv * d, v, hkv * d, rope.handle, None, None,
                            0.0, bt, tables.shape[1], ln, st, 3, 48, h)
    need = B.pa_prefill_workspace_size(handle, 3, 48, h, tables.shape[1])
    ws = torch.empty(max(1, need), dtype=torch.uint8, device=dev)
    B.pa_prefill_attention(out, qr, handle, layer, bt, tables.shape[1], ln, st, 3, 48, h, d ** -0.5, ws, need)
    cache = BlockPool(nb, block, layers, hkv, d, tensor=pool_t)
    q2 = cache.norm_rope_write_kv(layer, q, k, v, bt, ln, rope=rope, query_starts=st)
    assert torch.equal(q2, qr)
    assert torch.equal(cache.prefill_attention(q2, layer, bt, ln, st, d ** -0.5), out)
    check(out, *R.prefill(pool_t, q2, tables, ctx, new, d ** -0.5, layer))
    B.pa_pool_destroy(handle)
    del keep


def test_prefill_far_offsets(cuda_device):
    """Pages beyond 2^32 bytes and 2^31 elements of the pool."""
    dev, d, block, h, hkv = cuda_device, 128, 32, 8, 8
    nb = (1 << 31) // (2 * hkv * block * d) + 40
    pool_t = torch.empty((nb, 2, 1, hkv, block, d), dtype=torch.bfloat16, device=dev)
    new, ctx = [9, 33], [200, 300]
    tables = np.full((2, 10), -1, np.int32)
    tables[0, :7], tables[1, :10] = nb - 1 - 2 * np.arange(7), nb - 18 - np.arange(10)
    used = torch.as_tensor(tables[tables >= 0].astype(np.int64), device=dev)
    pool_t[used] = randn((len(used),) + tuple(pool_t.shape[1:]), torch.bfloat16, dev, 2)
    q = randn((42, h, d), torch.bfloat16, dev, 3)
    cache = BlockPool(nb, block, 1, hkv, d, tensor=pool_t)
    k, v = randn((42, hkv, d), torch.bfloat16, dev, 4), randn((42, hkv, d), torch.bfloat16, dev, 5)
    args = (ints(tables, dev), ints(ctx, dev))
    st = ints([0, 9, 42], dev)
    cache.norm_rope_write_kv(0, q, k, v, *args, query_starts=st)
    got = cache.prefill_attention(q, 0, *args, st, d ** -0.5)
    status_is(0)
    small = np.full_like(tables, -1)
    small[tables >= 0] = np.arange(len(used))
    sub = pool_t[used]
    assert torch.equal(sub[small[0, 199 // 32], 1, 0, :, 199 % 32], v[8])
    check(got, *R.prefill(sub, q, small, ctx, new, d ** -0.5))
    cache.copy_blocks(ints([nb - 1], dev), ints([3], dev))
    assert torch.equal(pool_t[3], pool_t[nb - 1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefill_single_tokens_match_decode(cuda_device, dtype):
    """One new token per sequence: the decode of the same cache."""
    dev, d, block, h, hkv = cuda_device, 128, 16, 8, 2
    ctx = [1, 17, 400, 3000]
    pool_t, tables, q = prefill_case(dev, dtype, d, block, h, hkv, [1] * 4, ctx, seed=12)
    got = run_prefill(dev, pool_t, tables, q, [1] * 4, ctx)
    cache = BlockPool(pool_t.shape[0], block, 1, hkv, d, tensor=pool_t)
    one = cache.decode_attention(q, 0, ints(tables, dev), ints(ctx, dev), d ** -0.5)
    want, bound = R.prefill(pool_t, q, tables, ctx, [1] * 4, d ** -0.5)
    check(got, want, bound)
    assert bool(((one.double() - want).abs() <= bound + 1e-5).all())


def test_prefill_graph_and_streams(cuda_device):
    """A captured prefill replays with new lengths, tables and queries in its
    buffers; calls on two streams with workspaces of their own do not meet."""
    dev, d, block, h, hkv = cuda_device, 128, 16, 8, 2
    new, ctx = [5, 3], [3000, 2000]
    pool_t, tables, q = prefill_case(dev, "bf16", d, block, h, hkv, new, ctx, seed=13, maxb=200)
    cache = BlockPool(pool_t.shape[0], block, 1, hkv, d, tensor=pool_t)
    bt, ln, st = ints(tables, dev), ints(ctx, dev), ints(R.starts_of(new), dev)
    need = cache.prefill_workspace_size(2, 8, h, 200)
    ws = [torch.empty(max(1, need), dtype=torch.uint8, device=dev) for _ in range(2)]
    outs = [torch.empty_like(q) for _ in range(2)]
    cache.prefill_attention(q, 0, bt, ln, st, d ** -0.5, out=outs[0], workspace=ws[0])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache.prefill_attention(q, 0, bt, ln, st, d ** -0.5, out=outs[0], workspace=ws[0])
    for new2, ctx2 in (([5, 3], [3000, 2000]), ([2, 6], [1999, 1500]), ([8, 0], [70, 0]), ([1, 7], [1, 2000])):
        ln.copy_(ints(ctx2, dev)), st.copy_(ints(R.starts_of(new2), dev))
        q.copy_(randn(q.shape, q.dtype, dev, sum(ctx2)))
        g.replay()
        torch.cuda.synchronize()
        check(outs[0], *R.prefill(pool_t, q, tables, ctx2, new2, d ** -0.5))
    status_is(0)
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    want = outs[0].clone()
    for _ in range(20):
        for i in range(2):
            cache.prefill_attention(q, 0, bt, ln, st, d ** -0.5, out=outs[i], workspace=ws[i], stream=side[i])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    # allocations of the call itself belong to its stream
    got = cache.prefill_attention(q, 0, bt, ln, st, d ** -0.5, stream=side[0])
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_prefill_workspace_refusal(cuda_device):
    pool_t, tables, q = prefill_case(cuda_device, "bf16", 128, 16, 8, 1, [3], [9000], seed=14)
    cache = BlockPool(pool_t.shape[0], 16, 1, 1, 128, tensor=pool_t)
    need = cache.prefill_workspace_size(1, 3, 8, tables.shape[1])
    assert need > 0
    ws = torch.empty(need + 512, dtype=torch.uint8, device=cuda_device)
    args = (q, 0, ints(tables, cuda_device), ints([9000], cuda_device), ints([0, 3], cuda_device), 0.1)
    for bad in (ws[:need - 1], ws[4:]):
        with pytest.raises(B.PagedAttnError) as e:
            cache.prefill_attention(*args, workspace=bad)
        assert e.value.code == B.PA_ERR_WORKSPACE
    with pytest.raises(B.PagedAttnError):
        B.pa_prefill_attention(q, q, cache.handle, 0, args[2], tables.shape[1], args[3], args[4], 1, 3, 8, 0.1,
                               ws, need)   # in place


# ------------------------------------------------------------------- pages

GEOMS = [("bf16", 2, 2, 16, 64), ("f32", 1, 1, 16, 64), ("bf16", 3, 1, 32, 128), ("bf16", 1, 3, 5, 24),
         ("f32", 2, 1, 1, 4)]


def pages_case(dev, geom, seed, rows, spare, lens):
    dtype, layers, hkv, block, d = geom
    rng = np.random.default_rng(seed)
    nblk = sum(R.cdiv(n, block) for n in lens)
    nb = nblk + spare
    ids = [int(x) for x in rng.permutation(nb)]
    maxb = max(1, max(R.cdiv(n, block) for n in lens)) + 2
    tables = np.full((rows, maxb), -1, np.int32)
    full = np.zeros(rows, np.int32)
    for b, n in enumerate(lens):
        full[b] = n
        for j in range(R.cdiv(n, block)):
            tables[b, j] = ids.pop()
    pool_t = randn((nb, 2, layers, hkv, block, d), DT[dtype], dev, seed)
    cache = BlockPool(nb, block, layers, hkv, d, tensor=pool_t)
    return cache, R.Pages(nb, block, tables, full, ids, pool_t), rng


def device_stack(ids, nb, dev):
    s = np.full(nb + 1, -1, np.int32)
    s[0], s[1:1 + len(ids)] = len(ids), ids
    return ints(s, dev)


def same(cache, ref, stack, tables, lens, shares):
    assert np.array_equal(tables.cpu().numpy(), ref.tables)
    assert np.array_equal(lens.cpu().numpy(), ref.lens)
    assert np.array_equal(shares.cpu().numpy(), ref.shares)
    s = stack.cpu().numpy()
    assert s[0] == len(ref.stack) and list(s[1:1 + s[0]]) == ref.stack
    assert torch.equal(cache.pool, ref.pool)


@pytest.mark.parametrize("geom", range(len(GEOMS)))
@pytest.mark.parametrize("n", [0, 1, 7, 40])
def test_copy_blocks(cuda_device, geom, n):
    cache, ref, rng = pages_case(cuda_device, GEOMS[geom], 1, 1, 100, [3])
    ids = rng.permutation(cache.num_blocks)[:2 * n]
    src, dst = ids[:n].copy(), ids[n:].copy()
    if n > 3:
        src[3] = src[2]          # one page to two places
        dst[1] = src[1]          # onto itself: nothing to do
    for a, b in zip(src, dst):
        ref.pool[int(b)] = ref.pool[int(a)]
    cache.copy_blocks(ints(src, cuda_device), ints(dst, cuda_device))
    assert torch.equal(cache.pool, ref.pool)
    status_is(0)


def test_copy_blocks_bad_ids(cuda_device):
    cache, ref, _ = pages_case(cuda_device, GEOMS[0], 1, 1, 10, [3])
    nb = cache.num_blocks
    ref.pool[4] = ref.pool[2]
    cache.copy_blocks(ints([nb, 0, -1, 2, 1], cuda_device), ints([0, -1, 1, 4, 1 << 30], cuda_device))
    assert torch.equal(cache.pool, ref.pool)
    status_is(B.PA_STATUS_BAD_BLOCK_ID)


@pytest.mark.parametrize("geom", range(len(GEOMS)))
@pytest.mark.parametrize("rows,wide", [(6, 0), (1500, 0), (1500, 150)])
def test_fork_free_compact_steps(cuda_device, geom, rows, wide):
    """Random steps of forks, frees and compactions against the plain model, on
    the device state alone; more rows than one CTA's threads, and tables too large
    for shared memory, too."""
    dev, (_, _, _, block, _) = cuda_device, GEOMS[geom]
    rng = np.random.default_rng(geom)
    first = 3 if rows < 100 else 400
    lens = [int(x) for x in rng.integers(0, 5 * block + 2, first)]
    cache, ref, rng = pages_case(dev, GEOMS[geom], geom, rows, rows + 50, lens)
    ref.tables = np.pad(ref.tables, ((0, 0), (0, wide)), constant_values=-1)
    assert (ref.tables.size > 8 * 24576) == (wide > 0)
    stack, tables = device_stack(ref.stack, cache.num_blocks, dev), ints(ref.tables, dev)
    ln, shares = ints(ref.lens, dev), cache.page_shares()
    used = set(range(first))
    for step in range(8 if rows < 100 else 3):
        free_rows = sorted(set(range(rows)) - used)
        n = int(rng.integers(1, len(free_rows) + 1)) if free_rows else 0
        chi = [int(x) for x in rng.permutation(free_rows)[:n]]
        par = [int(x) for x in rng.choice(sorted(used), n)] if n else []
        ref.fork(par, chi)
        cache.device_fork_sequences(stack, shares, tables, ln, ints(par, dev), ints(chi, dev))
        same(cache, ref, stack, tables, ln, shares)
        used |= set(chi)
        done = np.zeros(rows, np.uint8)
        done[rng.permutation(sorted(used))[:max(1, len(used) // 2)]] = 1
        ref.free(done)
        cache.device_free_shared(stack, shares, tables, ln, torch.from_numpy(done).to(dev))
        same(cache, ref, stack, tables, ln, shares)
        used -= set(np.nonzero(done)[0])
        for b in np.nonzero(done)[0]:
            ref.lens[b] = 0
        ln.copy_(ints(ref.lens, dev))
        remap = ref.compact()
        stack, tables, shares, got = cache.device_compact_blocks(stack, tables, ln, shares=shares)
        assert np.array_equal(got.cpu().numpy(), remap)
        assert bool((stack[1 + len(ref.stack):] == -1).all())
        same(cache, ref, stack, tables, ln, shares)
        if not used:
            break
    status_is(0)


def test_fork_bad_stack_ids(cuda_device):
    """Ids on the stack that are no pages' do not get into a table."""
    dev = cuda_device
    cache, ref, _ = pages_case(dev, GEOMS[0], 2, 8, 2, [20, 21, 5])
    stack, tables = device_stack(ref.stack, cache.num_blocks, dev), ints(ref.tables, dev)
    top = int(stack[0])
    good = int(stack[top - 1])
    stack[top] = cache.num_blocks
    ln, shares = ints(ref.lens, dev), cache.page_shares()
    cache.device_fork_sequences(stack, shares, tables, ln, ints([0, 1], dev), ints([3, 4], dev))
    status_is(B.PA_STATUS_BAD_BLOCK_ID)
    assert int(tables[3, 1]) == -1 and int(tables[4, 1]) == good and int(stack[0]) == top - 2
    assert int(tables[3, 0]) == int(tables[0, 0]) and int(ln[3]) == 20
    cache.close()


def test_fork_runs_dry_and_bad_rows(cuda_device):
    dev, block = cuda_device, 16
    cache, ref, _ = pages_case(dev, GEOMS[0], 2, 8, 2, [20, 16, 5])
    stack, tables = device_stack(ref.stack, cache.num_blocks, dev), ints(ref.tables, dev)
    ln, shares = ints(ref.lens, dev), cache.page_shares()
    ref.fork([0, 1, 2, 0], [3, 4, 5, 6])   # two partial pages to be had, three wanted
    cache.device_fork_sequences(stack, shares, tables, ln, ints([0, 1, 2, 0], dev), ints([3, 4, 5, 6], dev))
    same(cache, ref, stack, tables, ln, shares)
    assert ref.tables[6, 1] == -1
    assert B.pa_get_status() & B.PA_STATUS_NO_FREE_BLOCKS
    before = [x.clone() for x in (stack, tables, ln, shares, cache.pool)]
    ln[2] = 16 * tables.shape[1] + 1
    cache.device_fork_sequences(stack, shares, tables, ln, ints([-1, 8, 0, 1, 2], dev),
                                ints([7, 7, 8, 1, 7], dev))
    status_is(B.PA_STATUS_BAD_LENGTH)
    ln[2] = 5
    for a, b in zip(before, (stack, tables, ln, shares, cache.pool)):
        assert torch.equal(a, b)
    # heights no array can hold, frees of bad entries and of a bad length
    stack[0] = 1 << 30
    cache.device_fork_sequences(stack, shares, tables, ln, ints([1], dev), ints([7], dev))
    status_is(B.PA_STATUS_BAD_LENGTH)
    stack[0] = -4
    tables[7, 0] = 1 << 20
    ln[7] = 16
    cache.device_free_shared(stack, shares, tables, ln, ints([0] * 7 + [1], dev).to(torch.uint8))
    assert B.pa_get_status() == B.PA_STATUS_BAD_LENGTH | B.PA_STATUS_BAD_BLOCK_ID
    assert int(stack[0]) == 0 and int(tables[7, 0]) == -1


def test_free_shared_without_sharing_is_free_blocks(cuda_device):
    dev = cuda_device
    lens = [0, 1, 16, 17, 100, 64]
    a, ref, rng = pages_case(dev, GEOMS[0], 3, 6, 4, lens)
    nb, done = a.num_blocks, torch.tensor([1, 0, 1, 1, 1, 0], dtype=torch.uint8, device=dev)
    s1, s2 = device_stack(ref.stack, nb, dev), device_stack(ref.stack, nb, dev)
    t1, t2, ln, shares = ints(ref.tables, dev), ints(ref.tables, dev), ints(ref.lens, dev), a.page_shares()
    a.device_free_blocks(s1, t1, ln, done)
    a.device_free_shared(s2, shares, t2, ln, done)
    h = int(s1[0])
    assert torch.equal(s1[:1 + h], s2[:1 + h]) and torch.equal(t1, t2) and not shares.any()
    # a page listed by two rows without a share is pushed once
    t = ints([[3, -1], [3, -1]], dev)
    s = device_stack([], nb, dev)
    a.device_free_shared(s, shares, t, ints([4, 4], dev), ints([1, 1], dev).to(torch.uint8))
    assert s[:2].tolist() == [1, 3] and not shares.any() and bool((t == -1).all())
    status_is(0)


def test_compact_bad_entries_and_extremes(cuda_device):
    dev = cuda_device
    cache, ref, _ = pages_case(dev, GEOMS[0], 4, 3, 5, [40, 3, 20])
    nb = cache.num_blocks
    stack, tables, ln = device_stack(ref.stack, nb, dev), ints(ref.tables, dev), ints(ref.lens, dev)
    t = tables.clone()
    t[0, 1], t[1, 0] = nb, ref.stack[0]     # outside the pool; on the stack
    pool0 = cache.pool.clone()
    out = cache.device_compact_blocks(stack, t, ln)
    status_is(B.PA_STATUS_BAD_BLOCK_ID)
    assert int(out[1][0, 1]) == -1 and int(out[1][1, 0]) == -1 and out[2] is None
    cache.pool.copy_(pool0)
    # in place tables; nothing free; everything free
    remap = ref.compact()
    out = cache.device_compact_blocks(stack, tables, ln, out_tables=tables)
    assert out[1] is tables and np.array_equal(tables.cpu().numpy(), ref.tables)
    assert np.array_equal(out[3].cpu().numpy(), remap) and torch.equal(cache.pool, ref.pool)
    none = cache.device_compact_blocks(device_stack([], nb, dev), tables, ln)
    assert int(none[0][0]) == 0 and none[3].tolist() == list(range(nb)) and torch.equal(none[1], tables)
    every = cache.device_compact_blocks(device_stack(list(range(nb)), nb, dev), tables, ints([0, 0, 0], dev))
    assert every[0].tolist() == [nb] + list(range(nb - 1, -1, -1)) and bool((every[3] == -1).all())
    assert torch.equal(cache.pool, ref.pool)
    status_is(0)


@pytest.mark.parametrize("nb", [1, 31, 32, 33, 40000])
def test_compact_many_pages(cuda_device, nb):
    dev = cuda_device
    rng = np.random.default_rng(nb)
    pool_t = torch.arange(nb, device=dev, dtype=torch.float32)[:, None, None, None, None, None].expand(
        nb, 2, 1, 1, 1, 4).contiguous()
    cache = BlockPool(nb, 1, 1, 1, 4, tensor=pool_t)
    ids = rng.permutation(nb)
    live = ids[:(nb + 1) // 2]
    tables = np.ascontiguousarray(live[None, :]).astype(np.int32)
    s = device_stack([int(x) for x in ids[(nb + 1) // 2:]], nb, dev)
    stack, bt, _, remap = cache.device_compact_blocks(s, ints(tables, dev), ints([len(live)], dev))
    new = bt.cpu().numpy()[0]
    assert sorted(new.tolist()) == list(range(len(live)))
    assert torch.equal(pool_t[bt[0].long(), 0, 0, 0, 0, 0].long().cpu(), torch.from_numpy(live))
    holes = sorted(set(range(len(live))) - set(live.tolist()))
    movers = sorted(x for x in live.tolist() if x >= len(live))
    want = {**{int(x): int(x) for x in live}, **dict(zip(movers, holes))}
    assert all(want[int(a)] == int(b) for a, b in zip(live, new))
    status_is(0)


def test_pages_and_append_graphs(cuda_device):
    """Norm + rotation + append, fork and free captured and replayed."""
    dev, d, block, h, hkv = cuda_device, 64, 16, 4, 2
    cache, ref, rng = pages_case(dev, ("bf16", 2, hkv, block, d), 5, 8, 40, [20, 37])
    stack, tables = device_stack(ref.stack, cache.num_blocks, dev), ints(ref.tables, dev)
    ln, shares = ints(ref.lens, dev), cache.page_shares()
    par, chi = ints([0, 1, 0], dev), ints([2, 3, 4], dev)
    done = torch.tensor([0, 0, 1, 1, 1, 0, 0, 0], dtype=torch.uint8, device=dev)
    rope = Rope(d)
    q, k, v = (randn((8, n, d), torch.bfloat16, dev, n) for n in (h, hkv, hkv))
    out = torch.empty_like(q)

    def step():
        cache.device_fork_sequences(stack, shares, tables, ln, par, chi)
        cache.norm_rope_write_kv(1, q, k, v, tables, ln, rope=rope, out=out)
        cache.device_free_shared(stack, shares, tables, ln, done)

    ln[5:] = 0
    step()
    torch.cuda.synchronize()
    status_is(B.PA_STATUS_BAD_LENGTH)   # rows 5 .. 7 hold no token to append
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    height = int(stack[0])
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert int(stack[0]) == height and not shares.any() and bool((tables[2:] == -1).all())
        want, size = R.norm_rope(q[:2], ln[:2] - 1, R.frequencies(d, 10000.0), False, 1.0, None, 0.0)
        check(out[:2], want, R.norm_rope_bound(want, size, torch.bfloat16))
    status_is(B.PA_STATUS_BAD_LENGTH)


# ---------------------------------------------------------------- together


@pytest.mark.parametrize("dtype,d,h,hkv", [("bf16", 128, 8, 2), ("bf16", 64, 16, 2), ("f32", 64, 4, 4)])
def test_serving_run(cuda_device, dtype, d, h, hkv):
    """Prompts in two chunks, forks for three samples each, decode steps, a
    verified run of tokens, frees, a compaction: after each the attention over
    the cache is that of the plain sequences of keys and values."""
    dev, dt, block, layers = cuda_device, DT[dtype], 16, 2
    rows, maxb, nb = 8, 16, 90
    cache = BlockPool(nb, block, layers, hkv, d, dtype=dt, device=dev)
    stack, shares = cache.device_stack(), cache.page_shares()
    tables = torch.full((rows, maxb), -1, dtype=torch.int32, device=dev)
    rope, wq, wk = Rope(d, scaling="linear", factor=2.0), *(randn((d,), dt, dev, i) for i in (1, 2))
    wq, wk = (1 + 0.1 * wq).to(dt), (1 + 0.1 * wk).to(dt)
    freq = R.frequencies(d, 10000.0, "linear", 2.0)
    kept = [[torch.zeros((0, 2, hkv, d), dtype=dt, device=dev) for _ in range(layers)] for _ in range(rows)]
    lens, seed = [0] * rows, [100]

    def feed(new):
        """Appends and attends new[b] tokens of every row."""
        nonlocal stack
        for b, n in enumerate(new):      # pages for the new tokens, one position at a time
            for p in range(lens[b], lens[b] + n):
                if p % block == 0:
                    height = int(stack[0])
                    tables[b, p // block] = stack[height]
                    stack[0] = height - 1
            lens[b] += n
        t, ctx, st = sum(new), ints(lens, dev), ints(R.starts_of(new), dev)
        pos = torch.cat([torch.arange(c - n, c) for n, c in zip(new, lens)]).to(dev)
        for layer in range(layers):
            seed[0] += 1
            qkv = randn((t, h + 2 * hkv, d), dt, dev, seed[0])
            q, k, v = qkv[:, :h], qkv[:, h:h + hkv], qkv[:, h + hkv:]
            y = cache.norm_rope_write_kv(layer, q, k, v, tables, ctx, rope=rope, q_weight=wq, k_weight=wk,
                                         query_starts=st)
            want, size = R.norm_rope(q, pos, freq, False, 1.0, wq, 1e-6)
            check(y, want, R.norm_rope_bound(want, size, dt))
            ky, ksize = R.norm_rope(k, pos, freq, False, 1.0, wk, 1e-6)
            s = R.starts_of(new)
            for b in range(rows):
                at = slice(int(s[b]), int(s[b + 1]))
                pages = tables[b, :R.cdiv(lens[b], block)].long()
                stored = cache.pool[pages, :, layer].permute(0, 3, 1, 2, 4).reshape(-1, 2, hkv, d)[:lens[b]]
                n = lens[b] - new[b]
                assert torch.equal(stored[:n], kept[b][layer])      # what was there
                check(stored[n:, 0], ky[at], R.norm_rope_bound(ky[at], ksize[at], dt))
                assert torch.equal(stored[n:, 1], v[at])
                kept[b][layer] = stored.clone()
            out = cache.prefill_attention(y, layer, tables, ctx, st, d ** -0.5)
            check(out, *R.prefill(cache.pool, y, tables.cpu().numpy(), lens, new, d ** -0.5, layer))
            if max(new) == 1:
                live = [b for b in range(rows) if new[b]]
                one = cache.decode_attention(y, layer, tables[live].contiguous(), ctx[live], d ** -0.5)
                want, bound = R.prefill(cache.pool, y, tables.cpu().numpy(), lens, new, d ** -0.5, layer)
                assert bool(((one.double() - want).abs() <= bound + 1e-5).all())

    feed([37, 20, 0, 0, 0, 0, 0, 0])
    feed([5, 44, 0, 0, 0, 0, 0, 0])
    par, chi = [0, 0, 1, 1], [2, 3, 4, 5]
    ctx = ints(lens, dev)
    cache.device_fork_sequences(stack, shares, tables, ctx, ints(par, dev), ints(chi, dev))
    for p, c in zip(par, chi):
        lens[c], kept[c] = lens[p], [x.clone() for x in kept[p]]
    assert ctx.tolist() == lens and int(shares.sum()) == 2 * (42 // 16) + 2 * (64 // 16)
    for _ in range(20):
        feed([1, 1, 1, 1, 1, 1, 0, 0])
    feed([4, 0, 3, 0, 1, 5, 0, 0])
    done = [1, 0, 0, 1, 0, 1, 0, 0]
    cache.device_free_shared(stack, shares, tables, ints(lens, dev),
                             torch.tensor(done, dtype=torch.uint8, device=dev))
    for b in range(rows):
        if done[b]:
            lens[b], kept[b] = 0, [x[:0] for x in kept[b]]
    assert not shares[tables[2, :2].long()].any()          # row 2 alone holds the first prompt now
    stack, tables, shares, _ = cache.device_compact_blocks(stack, tables, ints(lens, dev), shares=shares)
    used = set(tables[tables >= 0].tolist())
    assert used == set(range(nb - int(stack[0])))
    feed([0, 2, 1, 0, 9, 0, 11, 0])
    status_is(0)
    cache.download_device_stack(stack)
    assert cache.num_free() == int(stack[0])
