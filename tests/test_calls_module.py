"""The module of the speculation calls (``pa_calls.cpp``) on the host (no GPU): who needs it, when
it is built again, and what is built where it cannot be."""
import pytest
import torch


def cpu_pool():
    from paged_kv_cache_239_gb300.pool import BlockPool

    return BlockPool(4, 16, 1, 2, 64, tensor=torch.zeros((4, 2, 1, 2, 16, 64), dtype=torch.bfloat16))


def test_only_the_speculation_calls_need_the_module(pa_lib, monkeypatch):
    """Where the module cannot be loaded a pool does all that goes without it; the calls that
    need it say why they cannot."""
    def calls():
        raise RuntimeError("built for another torch")

    monkeypatch.setattr(pa_lib, "calls", calls)
    cache = cpu_pool()
    ids = [cache.allocate_block() for _ in range(4)]
    assert sorted(ids) == [0, 1, 2, 3] and cache.num_free() == 0
    cache.free_block(ids[0])
    cache.set_prefill_kernel("mma")
    assert cache.prefill_workspace_size(0, 0, 4, 4) == 0 and cache.tree_workspace_size(0, 0, 4, 4) == 0
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(RuntimeError, match="another torch"):
        cache.device_trim_sequences(i32(5), i32(2, 4), i32(2), i32(2))
    # and once it can be loaded, the same pool takes them
    monkeypatch.undo()
    with pytest.raises(ValueError, match="device"):
        cache.device_trim_sequences(i32(5), i32(2, 4), i32(2), i32(2))
    cache.close()
