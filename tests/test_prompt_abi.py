"""Host checks (no GPU) of the calls for several new tokens per sequence and of
the page operations: frequencies, refusals, workspace rules of bad sizes."""
import math

import numpy as np
import pytest
import torch

import prompt_reference as R

F = 0x7F0000000000  # 16-byte aligned; never dereferenced by host-only calls


@pytest.fixture()
def pool(pa_lib):
    h = pa_lib.pa_pool_create(F, 64, 2, 2, 16, 64, pa_lib.PA_DTYPE_BF16)
    yield h
    pa_lib.pa_pool_destroy(h)


def refused(pa_lib, code, call, *args, **kw):
    with pytest.raises(pa_lib.PagedAttnError) as e:
        call(*args, **kw)
    assert e.value.code == code, str(e.value)
    assert str(e.value)


@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("linear", 4.0), ("ntk", 8.0), ("parts", 8.0)])
@pytest.mark.parametrize("rotary", [16, 48, 128])
def test_frequencies(pa_lib, scaling, factor, rotary):
    from paged_kv_cache_239_gb300.rope import Rope

    r = Rope(rotary, base=500000.0, scaling=scaling, factor=factor, original_len=8192)
    want = R.frequencies(rotary, 500000.0, scaling, factor, 8192.0)
    # a dozen roundings of 2^-53
    assert np.allclose(r.frequencies, want, rtol=1e-14, atol=0)
    r.close()
    r.close()  # twice is fine


def test_parts_keeps_fast_and_divides_slow(pa_lib):
    f = pa_lib.pa_rope_frequencies(64, 10000.0, pa_lib.PA_ROPE_PARTS, 4.0, 8192.0, 1.0, 32.0)
    plain = pa_lib.pa_rope_frequencies(64, 10000.0)
    assert f[0] == plain[0] == 1.0
    assert f[-1] == plain[-1] / 4.0
    assert all(a / 4.0 <= b <= a for a, b in zip(plain, f))


@pytest.mark.parametrize("args", [(0, 1e4), (24, 1e4), (-16, 1e4), (64, 1.0), (64, math.inf), (64, 1e4, 9),
                                  (64, 1e4, 1, 0.0), (64, 1e4, 1, math.nan), (64, 1e4, 3, 2.0, 0.0, 1.0, 4.0),
                                  (64, 1e4, 3, 2.0, 4096.0, 4.0, 4.0)])
def test_frequencies_refusals(pa_lib, args):
    refused(pa_lib, pa_lib.PA_ERR_INVALID_ARG, pa_lib.pa_rope_frequencies, *args)


def test_rope_refusals(pa_lib):
    bad = pa_lib.PA_ERR_INVALID_ARG
    refused(pa_lib, bad, pa_lib.pa_rope_create, 144, False, [0.1] * 72)
    refused(pa_lib, bad, pa_lib.pa_rope_create, 8, False, [0.1] * 4)
    refused(pa_lib, bad, pa_lib.pa_rope_create, 16, False, [0.1] * 7 + [2 * math.pi])
    refused(pa_lib, bad, pa_lib.pa_rope_create, 16, False, [0.1] * 7 + [-0.1])
    refused(pa_lib, bad, pa_lib.pa_rope_create, 16, False, [0.1] * 7 + [math.nan])
    refused(pa_lib, bad, pa_lib.pa_rope_create, 16, False, [0.1] * 8, math.inf)
    with pytest.raises(ValueError):
        pa_lib.pa_rope_create(16, False, [0.1] * 7)
    pa_lib.pa_rope_destroy(None)


def test_norm_rope_refusals(pa_lib, pool):
    B, bad = pa_lib, pa_lib.PA_ERR_INVALID_ARG
    rope = B.pa_rope_create(64, False, [0.1] * 32)
    wide = B.pa_rope_create(128, False, [0.1] * 64)

    def call(**kw):
        a = dict(pool=pool, layer=0, q_out=F, q=F + (1 << 20), q_stride=256, k=F + (2 << 20),
                 k_stride=128, v=F + (3 << 20), v_stride=128, rope=rope, q_weight=F + (4 << 20),
                 k_weight=F + (4 << 20), eps=1e-6, block_tables=F, max_blocks_per_seq=4,
                 context_lens=F, query_starts=F, batch=2, num_tokens=5, num_heads=4)
        a.update(kw)
        B.pa_norm_rope_write_kv(**a)

    try:
        for kw in (dict(pool=None), dict(layer=2), dict(layer=-1), dict(batch=-1), dict(num_tokens=-1),
                   dict(num_heads=3), dict(num_heads=0), dict(max_blocks_per_seq=0),
                   dict(max_blocks_per_seq=1 << 28), dict(block_tables=None), dict(context_lens=None),
                   dict(block_tables=F + 2), dict(query_starts=F + 2), dict(query_starts=None),
                   dict(q=None), dict(k=None), dict(v=None), dict(q_out=None), dict(q=F + (1 << 20) + 8),
                   dict(q_weight=None), dict(k_weight=None), dict(q_weight=F + 8), dict(eps=-1.0),
                   dict(eps=math.nan), dict(q_stride=255), dict(q_stride=260), dict(k_stride=64),
                   dict(rope=wide), dict(q=F + 16), dict(k=F + 256), dict(q=F, q_stride=512)):
            refused(B, bad, call, **kw)
        call(batch=0, num_tokens=0, query_starts=None)   # nothing to do
        call(num_tokens=0)
        odd = B.pa_pool_create(F, 4, 1, 2, 16, 32, B.PA_DTYPE_BF16)
        refused(B, B.PA_ERR_UNSUPPORTED, call, pool=odd, rope=None)
        B.pa_pool_destroy(odd)
    finally:
        B.pa_rope_destroy(rope)
        B.pa_rope_destroy(wide)


def test_prefill_refusals(pa_lib, pool):
    B, bad = pa_lib, pa_lib.PA_ERR_INVALID_ARG

    def call(**kw):
        a = dict(out=F, q=F + (1 << 20), pool=pool, layer=0, block_tables=F, max_blocks_per_seq=4,
                 context_lens=F, query_starts=F, batch=2, num_tokens=5, num_heads=4, scale=0.125)
        a.update(kw)
        B.pa_prefill_attention(**a)

    for kw in (dict(pool=None), dict(layer=2), dict(batch=-1), dict(num_tokens=-1), dict(num_heads=5),
               dict(max_blocks_per_seq=0), dict(max_blocks_per_seq=1 << 28), dict(scale=math.inf), dict(scale=3e38),
               dict(block_tables=None), dict(context_lens=F + 1), dict(num_tokens=1 << 30)):
        refused(B, bad, call, **kw)
    call(batch=0, num_tokens=0)
    call(num_tokens=0)
    odd = B.pa_pool_create(F, 4, 1, 2, 8, 64, B.PA_DTYPE_BF16)
    refused(B, B.PA_ERR_UNSUPPORTED, call, pool=odd)
    refused(B, B.PA_ERR_UNSUPPORTED, B.pa_prefill_workspace_size, odd, 1, 1, 2, 4)
    B.pa_pool_destroy(odd)
    assert B.pa_prefill_workspace_size(pool, 0, 0, 4, 4) == 0
    for kind in (-1, 3):
        refused(B, bad, B.pa_pool_set_prefill_kernel, pool, kind)
    refused(B, bad, B.pa_pool_set_prefill_kernel, None, B.PA_PREFILL_AUTO)
    wide = B.pa_pool_create(F, 4, 1, 2, 16, 64, B.PA_DTYPE_F32)
    B.pa_pool_set_prefill_kernel(wide, B.PA_PREFILL_TCGEN05)
    refused(B, B.PA_ERR_UNSUPPORTED, call, pool=wide)
    B.pa_pool_destroy(wide)


def test_page_refusals(pa_lib, pool):
    B, bad = pa_lib, pa_lib.PA_ERR_INVALID_ARG
    refused(B, bad, B.pa_copy_blocks, None, F, F, 1)
    refused(B, bad, B.pa_copy_blocks, pool, F, F, -1)
    refused(B, bad, B.pa_copy_blocks, pool, None, F, 1)
    refused(B, bad, B.pa_copy_blocks, pool, F, F + 2, 1)
    B.pa_copy_blocks(pool, None, None, 0)
    fork = dict(pool=pool, dev_stack=F, shares=F, block_tables=F, max_blocks_per_seq=4,
                context_lens=F, batch=3, parents=F, children=F, n=2)
    for kw in (dict(pool=None), dict(dev_stack=None), dict(shares=None), dict(n=-1), dict(n=4),
               dict(block_tables=None), dict(max_blocks_per_seq=0), dict(parents=F + 1), dict(children=None)):
        refused(B, bad, B.pa_device_fork_sequences, **{**fork, **kw})
    refused(B, bad, B.pa_device_fork_sequences, **{**fork, "batch": 70000, "n": 65537})
    B.pa_device_fork_sequences(**{**fork, "n": 0})
    free = dict(pool=pool, dev_stack=F, shares=F, block_tables=F, max_blocks_per_seq=4,
                context_lens=F, finished=F, batch=3)
    for kw in (dict(pool=None), dict(dev_stack=F + 1), dict(shares=F + 1), dict(finished=None),
               dict(batch=-1), dict(batch=1 << 20, max_blocks_per_seq=1 << 20)):
        refused(B, bad, B.pa_device_free_shared, **{**free, **kw})
    B.pa_device_free_shared(**{**free, "batch": 0})
    M = 1 << 20
    compact = dict(pool=pool, dev_stack=F, shares=F + M, block_tables=F + 2 * M, max_blocks_per_seq=4,
                   context_lens=F + 3 * M, batch=3, out_stack=F + 4 * M, out_shares=F + 5 * M,
                   out_tables=F + 6 * M, remap=F + 7 * M, workspace=F + 8 * M,
                   workspace_bytes=B.pa_compact_workspace_size(pool))
    for kw in (dict(out_stack=F), dict(out_shares=F + M), dict(remap=F + M), dict(out_tables=F + 2 * M + 4),
               dict(remap=F + 4 * M + 8), dict(out_shares=None), dict(shares=None), dict(remap=None),
               dict(out_tables=None), dict(dev_stack=None), dict(max_blocks_per_seq=-1)):
        refused(B, bad, B.pa_device_compact_blocks, **{**compact, **kw})
    for kw in (dict(workspace=None), dict(workspace_bytes=8), dict(workspace=F + 8 * M + 4)):
        refused(B, B.PA_ERR_WORKSPACE, B.pa_device_compact_blocks, **{**compact, **kw})
    big = B.pa_pool_create(F, 786433, 1, 1, 16, 64, B.PA_DTYPE_BF16)
    refused(B, B.PA_ERR_UNSUPPORTED, B.pa_device_compact_blocks, **{**compact, "pool": big})
    B.pa_pool_destroy(big)


def test_wrapper_refusals(pa_lib):
    """What only the tensors know: shapes, types, strides, devices."""
    from paged_kv_cache_239_gb300.pool import BlockPool

    pool = BlockPool(4, 16, 1, 2, 64, device="cpu")
    bt, ln = torch.zeros((2, 3), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    st = torch.zeros(3, dtype=torch.int32)
    q = torch.zeros((5, 4, 64), dtype=torch.bfloat16)
    kv = torch.zeros((5, 2, 64), dtype=torch.bfloat16)
    one = torch.zeros(1, dtype=torch.int32)
    stack, shares = torch.zeros(5, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    calls = [
        lambda: pool.prefill_attention(q.float(), 0, bt, ln, st, 0.1),
        lambda: pool.prefill_attention(q[:, ::2], 0, bt, ln, st, 0.1),
        lambda: pool.prefill_attention(q, 0, bt, ln, st[:2], 0.1),
        lambda: pool.prefill_attention(q, 0, bt.long(), ln, st, 0.1),
        lambda: pool.prefill_attention(q, 0, bt[0], ln, st, 0.1),
        lambda: pool.prefill_attention(q, 0, bt, ln, st, 0.1, out=q.float()),
        lambda: pool.norm_rope_write_kv(0, q, kv, kv[:4], bt, ln, query_starts=st),
        lambda: pool.norm_rope_write_kv(0, q.transpose(0, 1).contiguous().transpose(0, 1), kv, kv, bt, ln,
                                        query_starts=st),
        lambda: pool.norm_rope_write_kv(0, q, kv, kv, bt, ln, q_weight=one, k_weight=one, query_starts=st),
        lambda: pool.norm_rope_write_kv(0, q, kv, kv, bt, ln.long(), query_starts=st),
        lambda: pool.copy_blocks(one, one.long()),
        lambda: pool.copy_blocks(one, stack),
        lambda: pool.device_fork_sequences(stack[:4], shares, bt, ln, one, one),
        lambda: pool.device_fork_sequences(stack, shares[:3], bt, ln, one, one),
        lambda: pool.device_fork_sequences(stack, shares, bt, ln, one, ln),
        lambda: pool.device_free_shared(stack, shares, bt, ln, one),
        lambda: pool.device_compact_blocks(stack, bt, ln, out_tables=bt[:1]),
        lambda: pool.device_compact_blocks(stack, bt, ln, remap=stack),
    ]
    for call in calls:
        with pytest.raises(ValueError):
            call()
    # tensors that fit, but the pool is not on the current CUDA device
    kid, fin = ln[:1] + 1, torch.zeros(2, dtype=torch.bool)
    for call in [lambda: pool.prefill_attention(q, 0, bt, ln, st, 0.1),
                 lambda: pool.norm_rope_write_kv(0, q, kv, kv, bt, ln, query_starts=st),
                 lambda: pool.copy_blocks(one, one + 1),
                 lambda: pool.device_fork_sequences(stack, shares, bt, ln, one, kid),
                 lambda: pool.device_free_shared(stack, shares, bt, ln, fin),
                 lambda: pool.device_compact_blocks(stack, bt, ln)]:
        with pytest.raises(ValueError, match="current CUDA device"):
            call()
    pool.close()


def test_closed_rope_is_refused(pa_lib):
    """A closed Rope is not taken for "no rotation"."""
    from paged_kv_cache_239_gb300.pool import BlockPool
    from paged_kv_cache_239_gb300.rope import Rope

    pool, rope = BlockPool(4, 16, 1, 2, 64, device="cpu"), Rope(64)
    rope.close()
    q, kv = torch.zeros((1, 4, 64), dtype=torch.bfloat16), torch.zeros((1, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="closed"):
        pool.norm_rope_write_kv(0, q, kv, kv, torch.zeros((1, 1), dtype=torch.int32),
                                torch.ones(1, dtype=torch.int32), rope=rope)
    pool.close()
