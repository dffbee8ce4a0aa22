"""The calls for drafted trees on the host (no GPU): argument checks return the documented
codes, and the Python layer's checks refuse what only tensors know, before a device is touched."""
import numpy as np
import pytest
import torch

import tree_reference as T

P = 0x7F0000000000  # aligned; never dereferenced by host-only calls
MB = 1 << 20


@pytest.fixture
def pool(pa_lib):
    h = pa_lib.pa_pool_create(P, 8, 2, 2, 16, 64, 1)
    yield h
    pa_lib.pa_pool_destroy(h)


def refused(pa_lib, code, call):
    with pytest.raises(pa_lib.PagedAttnError) as e:
        call()
    assert e.value.code == code, str(e.value)
    return str(e.value)


PLAN = dict(dev_stack=P, block_tables=P + MB, max_blocks_per_seq=4, cached_lens=P + 2 * MB, new_counts=P + 3 * MB,
            parents=P + 4 * MB, batch=3, num_tokens=9, context_lens=P + 5 * MB, query_starts=P + 6 * MB, slots=P + 7 * MB,
            positions=P + 8 * MB, tree_masks=P + 9 * MB, mask_words=1)


@pytest.mark.parametrize("change", [
    dict(batch=-1), dict(num_tokens=-1), dict(max_blocks_per_seq=0), dict(max_blocks_per_seq=1 << 28), dict(mask_words=0),
    dict(num_tokens=(1 << 30) + 1), dict(mask_words=33), dict(dev_stack=None), dict(dev_stack=P + 2), dict(block_tables=None), dict(cached_lens=None),
    dict(new_counts=None), dict(context_lens=None), dict(query_starts=None), dict(slots=None), dict(positions=None),
    dict(slots=P + 7 * MB + 4), dict(positions=P + 8 * MB + 1), dict(tree_masks=P + 9 * MB + 2), dict(parents=P + 2),
    # an output over an input, or over another
    dict(context_lens=P + 2 * MB), dict(context_lens=P + 2 * MB + 8), dict(query_starts=P + 3 * MB - 12),
    dict(slots=P + 4 * MB), dict(positions=P + 7 * MB + 64), dict(tree_masks=P + 8 * MB + 32), dict(positions=P + 32),
    dict(slots=P + MB + 40), dict(parents=P + MB),
])
def test_plan_refusals(pa_lib, pool, change):
    refused(pa_lib, pa_lib.PA_ERR_INVALID_ARG, lambda: pa_lib.pa_device_plan_tokens(pool, **{**PLAN, **change}, stream=0))


TRIM = dict(dev_stack=P, block_tables=P + MB, max_blocks_per_seq=4, context_lens=P + 2 * MB, new_lens=P + 3 * MB, batch=3)


@pytest.mark.parametrize("change", [dict(batch=-1), dict(max_blocks_per_seq=0), dict(dev_stack=None), dict(block_tables=None),
                                    dict(context_lens=None), dict(new_lens=None), dict(new_lens=P + 2),
                                    dict(batch=16, max_blocks_per_seq=(1 << 26) + 1)])
def test_trim_refusals(pa_lib, pool, change):
    refused(pa_lib, pa_lib.PA_ERR_INVALID_ARG, lambda: pa_lib.pa_device_trim_sequences(pool, **{**TRIM, **change}, stream=0))
    pa_lib.pa_device_trim_sequences(pool, **{**TRIM, "batch": 0}, stream=0)   # (nothing to do)


ACCEPT = dict(slots=P, parents=P + MB, tokens=P + 2 * MB, targets=P + 3 * MB, context_lens=P + 4 * MB, query_starts=P + 5 * MB,
              batch=3, num_tokens=9, max_path=4, accepted_counts=P + 6 * MB, accepted_nodes=P + 7 * MB, next_tokens=P + 8 * MB,
              next_lens=P + 9 * MB)


@pytest.mark.parametrize("change", [
    dict(batch=-1), dict(num_tokens=-1), dict(max_path=0), dict(max_path=1025), dict(slots=None), dict(slots=P + 4),
    dict(parents=None), dict(tokens=None), dict(targets=P + 1), dict(context_lens=None), dict(query_starts=None),
    dict(accepted_counts=None), dict(accepted_nodes=None), dict(next_tokens=None), dict(next_lens=None),
    dict(next_lens=P + 4 * MB), dict(accepted_nodes=P + 3 * MB - 40), dict(next_tokens=P + 7 * MB + 44), dict(next_lens=P + 64),
])
def test_accept_refusals(pa_lib, pool, change):
    refused(pa_lib, pa_lib.PA_ERR_INVALID_ARG, lambda: pa_lib.pa_device_accept_tree(pool, **{**ACCEPT, **change}, stream=0))
    pa_lib.pa_device_accept_tree(pool, **{**ACCEPT, "batch": 0}, stream=0)


TREE = dict(out=P, q=P + MB, layer=0, block_tables=P + 2 * MB, max_blocks_per_seq=4, context_lens=P + 3 * MB,
            query_starts=P + 4 * MB, tree_masks=P + 5 * MB, mask_words=1, batch=3, num_tokens=0, num_heads=4, scale=0.1)


@pytest.mark.parametrize("change", [
    dict(batch=-1), dict(num_tokens=-1), dict(layer=2), dict(layer=-1), dict(num_heads=3), dict(num_heads=0), dict(mask_words=0),
    dict(mask_words=33), dict(max_blocks_per_seq=0), dict(context_lens=None), dict(block_tables=P + 2),
    dict(scale=float("inf")), dict(scale=float("nan")), dict(tree_masks=None, num_tokens=5), dict(tree_masks=P + 2, num_tokens=5),
])
def test_tree_attention_refusals(pa_lib, pool, change):
    args = {**TREE, **change}
    refused(pa_lib, pa_lib.PA_ERR_INVALID_ARG,
            lambda: pa_lib.pa_tree_attention(args.pop("out"), args.pop("q"), pool, **args, stream=0))


def test_tree_attention_of_nothing(pa_lib, pool):
    args = dict(TREE)
    pa_lib.pa_tree_attention(args.pop("out"), args.pop("q"), pool, **args, stream=0)
    assert pa_lib.pa_tree_workspace_size(pool, 0, 0, 4, 4) == 0


SLOTS = dict(layer=0, q_out=P, q=P + MB, q_stride=256, k=P + 2 * MB, k_stride=128, v=P + 3 * MB, v_stride=128, rope=None,
             q_weight=None, k_weight=None, eps=1e-6, positions=P + 4 * MB, slots=P + 5 * MB, num_tokens=5, num_heads=4)


@pytest.mark.parametrize("change", [
    dict(layer=2), dict(num_tokens=-1), dict(num_heads=3), dict(positions=None), dict(slots=None), dict(slots=P + 5 * MB + 4),
    dict(positions=P + 4 * MB + 2), dict(q=None), dict(q_out=P + 8), dict(q_stride=248), dict(k_stride=132), dict(k=P),
    dict(q_weight=P + 6 * MB), dict(q_weight=P + 6 * MB, k_weight=P + 6 * MB, eps=-1.0),
])
def test_append_at_slots_refusals(pa_lib, pool, change):
    refused(pa_lib, pa_lib.PA_ERR_INVALID_ARG,
            lambda: pa_lib.pa_norm_rope_write_kv_slots(pool, **{**SLOTS, **change}, stream=0))


def test_append_at_slots_needs_a_built_head_dim(pa_lib):
    h = pa_lib.pa_pool_create(P, 8, 2, 2, 16, 32, 1)
    refused(pa_lib, pa_lib.PA_ERR_UNSUPPORTED, lambda: pa_lib.pa_norm_rope_write_kv_slots(h, **SLOTS, stream=0))
    pa_lib.pa_pool_destroy(h)


def test_python_checks(pa_lib):
    """The wrappers look at shapes, types and devices before the library sees an address."""
    from paged_kv_cache_239_gb300.pool import BlockPool

    cache = BlockPool(4, 16, 1, 2, 64, tensor=torch.zeros((4, 2, 1, 2, 16, 64), dtype=torch.bfloat16))
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    q, kv = torch.zeros((3, 4, 64), dtype=torch.bfloat16), torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    bt, lens, starts, stack = i32(2, 4), i32(2), i32(3), i32(5)
    slots = torch.zeros(3, dtype=torch.int64)
    for call in (
        lambda: cache.device_plan_tokens(stack, bt, lens, i32(3), 3),
        lambda: cache.device_plan_tokens(i32(4), bt, lens, lens, 3),
        lambda: cache.device_plan_tokens(stack, bt, lens, lens, 3, parents=i32(2)),
        lambda: cache.device_plan_tokens(stack, bt, lens, lens, 3, slots=i32(3)),
        lambda: cache.device_plan_tokens(stack, bt, lens, lens, 3, tree_masks=i32(3, 2), mask_words=1),
        lambda: cache.device_trim_sequences(stack, bt, lens, i32(3)),
        lambda: cache.tree_attention(q, 0, bt, lens, starts, i32(2, 1), 1.0),
        lambda: cache.tree_attention(q, 0, bt, lens, starts, i32(3, 2).t().contiguous().t(), 1.0),
        lambda: cache.tree_attention(q.float(), 0, bt, lens, starts, i32(3, 1), 1.0),
        lambda: cache.norm_rope_write_kv_slots(0, q, kv, kv, i32(3), i32(3)),
        lambda: cache.norm_rope_write_kv_slots(0, q, kv, kv, i32(2), slots),
        lambda: cache.norm_rope_write_kv_slots(0, q, kv, kv[:2], i32(3), slots),
        lambda: cache.device_accept_tree(slots, i32(3), i32(3), i32(2), lens, starts, 2),
        lambda: cache.device_accept_tree(slots, i32(3), i32(3), i32(3), lens, lens, 2),
        lambda: cache.device_accept_tree(slots, i32(3), i32(3), i32(3), lens, starts, 2, nodes=i32(2, 3)),
        # all in order, but not on the GPU
        lambda: cache.device_trim_sequences(stack, bt, lens, lens),
    ):
        with pytest.raises(ValueError):
            call()


def test_reference_masks_and_plan():
    """The plain implementations themselves, on a tree worked by hand."""
    tree = [-1, 0, 0, 1, 3]
    assert T.ancestors(tree) == [0b1, 0b11, 0b101, 0b1011, 0b11011] and T.depths(tree) == [0, 1, 1, 2, 3]
    assert T.walk(tree, [9, 5, 6, 7, 8], [5, 7, 0, 8, 1], 9) == [0, 1, 3, 4]
    assert T.walk(tree, [9, 5, 5, 7, 8], [5, 0, 0, 8, 1], 9) == [0, 1]
    p = T.Plan(4, np.full((2, 3), -1, np.int32), [7, 8, 9], [0, 0], [5, 1], [tree, [-1]], 7, 1)
    assert p.slots == [36, 37, 38, 39, 32, 28, -1] and p.positions == [0, 1, 1, 2, 3, 0, 0]
    tables, stack = T.trim(4, p.tables, p.stack, [5, 1], [2, 0])
    assert stack == [7, 8] and tables.tolist() == [[9, -1, -1], [-1, -1, -1]]


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("kernel", [0, 1, 2])
@pytest.mark.parametrize("masks", [None, P + 5 * MB])
@pytest.mark.parametrize("nothing", [dict(num_tokens=0), dict(batch=0), dict(batch=0, num_tokens=0)])
def test_trees_of_nothing_on_every_kernel(pa_lib, dtype, kernel, masks, nothing):
    """An empty tensor's address is NULL: a call without tokens is still a call of trees."""
    h = pa_lib.pa_pool_create(P, 8, 2, 2, 16, 64, dtype)
    pa_lib.pa_pool_set_prefill_kernel(h, kernel)
    args = {**TREE, "tree_masks": masks, **nothing}
    pa_lib.pa_tree_attention(args.pop("out"), args.pop("q"), h, **args, stream=0)
    assert pa_lib.pa_tree_workspace_size(h, args["batch"], args["num_tokens"], 4, 4) == 0
    pa_lib.pa_pool_destroy(h)


def test_refused_numbers_are_named(pa_lib):
    """A number of the wrong type, or one that the call's 32 bits do not hold, is named."""
    from paged_kv_cache_239_gb300.pool import BlockPool

    cache = BlockPool(4, 16, 1, 2, 64, tensor=torch.zeros((4, 2, 1, 2, 16, 64), dtype=torch.bfloat16))
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    q, kv = torch.zeros((3, 4, 64), dtype=torch.bfloat16), torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    bt, lens, starts, stack, slots = i32(2, 4), i32(2), i32(3), i32(5), torch.zeros(3, dtype=torch.int64)
    ws = torch.zeros(1, dtype=torch.uint8)
    plan = dict(context_lens=i32(2), query_starts=starts, slots=slots, positions=i32(3))
    for name, call in (
        ("layer", lambda: cache.tree_attention(q, "0", bt, lens, starts, i32(3, 1), 1.0, workspace=ws)),
        ("layer", lambda: cache.tree_attention(q, 1 << 40, bt, lens, starts, i32(3, 1), 1.0, workspace=ws)),
        ("scale", lambda: cache.tree_attention(q, 0, bt, lens, starts, i32(3, 1), None, workspace=ws)),
        ("layer", lambda: cache.norm_rope_write_kv_slots(0.5, q, kv, kv, i32(3), slots)),
        ("eps", lambda: cache.norm_rope_write_kv_slots(0, q, kv, kv, i32(3), slots, eps="small")),
        ("num_tokens", lambda: cache.device_plan_tokens(stack, bt, lens, lens, 3.0, **plan)),
        ("mask_words", lambda: cache.device_plan_tokens(stack, bt, lens, lens, 3, tree_masks=i32(3, 1), mask_words=1.0, **plan)),
        ("max_path", lambda: cache.device_accept_tree(slots, i32(3), i32(3), i32(3), lens, starts, 2.0, nodes=i32(2, 2))),
    ):
        with pytest.raises((TypeError, ValueError), match=name):
            call()
