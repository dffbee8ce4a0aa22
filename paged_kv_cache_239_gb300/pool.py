"""``BlockPool``: a torch-owned pool tensor plus its library handle.

Mirrors the mini-infer BlockPool interface ("Paged KV-Cache Memory Management",
section "Python Implementation: Physical Block Pool": ``allocate_block``,
``free_block``, the [num_blocks, 2, num_layers, num_kv_heads, block_size,
head_dim] tensor) on top of the C ABI.  Marshalling only: torch allocates the
device memory, every operation runs in libpagedattn's kernels.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import binding as B


_DECODE_KERNELS = {"auto": B.PA_DECODE_AUTO, "cuda_cores": B.PA_DECODE_CUDA_CORES,
                   "tensor_cores": B.PA_DECODE_TENSOR_CORES, "tcgen05": B.PA_DECODE_TCGEN05}
_PREFILL_KERNELS = {"auto": B.PA_PREFILL_AUTO, "mma": B.PA_PREFILL_MMA, "tcgen05": B.PA_PREFILL_TCGEN05}


class BlockPool:
    def __init__(self, num_blocks: int, block_size: int = 16, num_layers: int = 24,
                 num_kv_heads: int = 2, head_dim: int = 64, dtype=torch.bfloat16,
                 device="cuda", tensor: Optional[torch.Tensor] = None):
        shape = (num_blocks, 2, num_layers, num_kv_heads, block_size, head_dim)
        if tensor is None:
            tensor = torch.zeros(shape, dtype=dtype, device=device)
        if tuple(tensor.shape) != shape or not tensor.is_contiguous():
            raise ValueError(f"pool tensor must be contiguous with shape {shape}")
        self.pool = tensor
        self.num_blocks, self.block_size, self.num_layers = num_blocks, block_size, num_layers
        self.num_kv_heads, self.head_dim = num_kv_heads, head_dim
        self.dtype = tensor.dtype
        self._device_index = tensor.get_device()
        self.handle = B.pa_pool_create(tensor, num_blocks, num_layers, num_kv_heads, block_size,
                                       head_dim, tensor.dtype)

    # -- allocator ---------------------------------------------------------
    def allocate_block(self) -> int:
        return B.pa_alloc_block(self.handle)

    def free_block(self, block_id: int) -> None:
        B.pa_free_block(self.handle, block_id)

    def num_free(self) -> int:
        return B.pa_num_free(self.handle)

    def seed_free_stack(self, order) -> None:
        B.pa_pool_seed_free_stack(self.handle, order)

    def block_bytes(self) -> int:
        return B.pa_pool_block_bytes(self.handle)

    # -- the same free stack on the device (one launch per batch) -----------
    def device_stack(self, stream=None) -> torch.Tensor:
        """Moves the free stack into a new device tensor; the host allocator
        refuses until download_device_stack brings it back."""
        n = B.pa_device_stack_bytes(self.handle) // 4
        stack = torch.empty(n, dtype=torch.int32, device=self.pool.device)
        B.pa_device_stack_upload(self.handle, stack, stream)
        return stack

    def download_device_stack(self, stack: torch.Tensor, stream=None) -> None:
        B.pa_device_stack_download(self.handle, stack, stream)

    def device_allocate_blocks(self, stack: torch.Tensor, block_tables: torch.Tensor,
                               positions: torch.Tensor, stream=None) -> None:
        """Every sequence whose position starts a new block pops one from the
        device stack into its table (the order repeated host calls give)."""
        B.pa_device_alloc_blocks(self.handle, stack, block_tables, block_tables.shape[1],
                                 positions, positions.shape[0], stream)

    def device_allocate_blocks_step(self, stack: torch.Tensor, block_tables: torch.Tensor,
                                    positions: torch.Tensor, next_lens: torch.Tensor,
                                    stream=None) -> None:
        """device_allocate_blocks, and next_lens = positions + 1 in the same
        launch (the context lengths once this step's tokens are appended)."""
        B.pa_device_alloc_blocks_step(self.handle, stack, block_tables, block_tables.shape[1],
                                      positions, next_lens, positions.shape[0], stream)

    def device_free_blocks(self, stack: torch.Tensor, block_tables: torch.Tensor,
                           context_lens: torch.Tensor, finished: torch.Tensor,
                           stream=None) -> None:
        """Finished sequences push their blocks back and their table rows become -1."""
        B.pa_device_free_blocks(self.handle, stack, block_tables, block_tables.shape[1],
                                context_lens, finished, context_lens.shape[0], stream)

    def set_decode_kernel(self, kind: str) -> None:
        """'auto' (default), 'cuda_cores', 'tensor_cores' (mma.sync) or 'tcgen05'."""
        B.pa_pool_set_decode_kernel(self.handle, _DECODE_KERNELS[kind])

    # -- kernels -----------------------------------------------------------
    def write_kv(self, layer: int, k: torch.Tensor, v: torch.Tensor, block_tables: torch.Tensor,
                 positions: torch.Tensor, stream=None) -> None:
        B.pa_write_kv(self.handle, layer, k, v, block_tables, block_tables.shape[1], positions,
                      positions.shape[0], stream)

    def workspace_size(self, batch: int, num_heads: int, max_blocks_per_seq: int,
                       partition_blocks: int = 0) -> int:
        return B.pa_decode_workspace_size(self.handle, batch, num_heads, max_blocks_per_seq,
                                          partition_blocks)

    def decode_attention(self, q: torch.Tensor, layer: int, block_tables: torch.Tensor,
                         context_lens: torch.Tensor, scale: float,
                         out: Optional[torch.Tensor] = None, partition_blocks: int = 0,
                         workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        batch, num_heads, head_dim = q.shape
        maxb = block_tables.shape[1]
        if out is None:
            out = torch.empty((batch, num_heads, head_dim), dtype=torch.float32, device=q.device)
        need = self.workspace_size(batch, num_heads, maxb, partition_blocks)
        if need and (workspace is None or workspace.numel() * workspace.element_size() < need):
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
        B.pa_decode_attention_partitioned(out, q, self.handle, layer, block_tables, maxb,
                                          context_lens, batch, self.block_size, num_heads,
                                          self.num_kv_heads, head_dim, scale, partition_blocks,
                                          workspace, wbytes, stream)
        return out

    def write_kv_and_decode(self, q: torch.Tensor, layer: int, k: torch.Tensor, v: torch.Tensor,
                            positions: torch.Tensor, block_tables: torch.Tensor,
                            context_lens: torch.Tensor, scale: float,
                            out: Optional[torch.Tensor] = None, partition_blocks: int = 0,
                            workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """write_kv then decode_attention in one launch (context_lens normally
        include the new token)."""
        batch, num_heads, head_dim = q.shape
        maxb = block_tables.shape[1]
        if out is None:
            out = torch.empty((batch, num_heads, head_dim), dtype=torch.float32, device=q.device)
        need = self.workspace_size(batch, num_heads, maxb, partition_blocks)
        if need and (workspace is None or workspace.numel() * workspace.element_size() < need):
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
        B.pa_write_kv_and_decode(out, q, self.handle, layer, k, v, positions, block_tables, maxb,
                                 context_lens, batch, self.block_size, num_heads,
                                 self.num_kv_heads, head_dim, scale, partition_blocks, workspace,
                                 wbytes, stream)
        return out

    def gather_kv(self, layer: int, block_tables: torch.Tensor, context_lens: torch.Tensor,
                  max_len: int, stream=None):
        batch = context_lens.shape[0]
        shape = (batch, max_len, self.num_kv_heads, self.head_dim)
        k = torch.empty(shape, dtype=self.dtype, device=self.pool.device)
        v = torch.empty(shape, dtype=self.dtype, device=self.pool.device)
        mask = torch.empty((batch, max_len), dtype=torch.uint8, device=self.pool.device)
        B.pa_gather_kv(k, v, mask, self.handle, layer, block_tables, block_tables.shape[1],
                       context_lens, batch, max_len, stream)
        return k, v, mask.bool()

    # -- several new tokens per sequence ------------------------------------
    def norm_rope_write_kv(self, layer: int, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                           block_tables: torch.Tensor, context_lens: torch.Tensor,
                           rope=None, q_weight: Optional[torch.Tensor] = None,
                           k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                           query_starts: Optional[torch.Tensor] = None,
                           out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """RMS norm of query and key heads (with weights), rotation (with a
        ``Rope``) and append of the new tokens: returns the queries, stores the
        keys and values.  q, k, v: [tokens, heads, head_dim], any stride between
        tokens (slices of one packed projection); context_lens include the new
        tokens; query_starts [batch + 1] says which rows are whose (None: one
        token per sequence).  ``out`` may be q itself when q is contiguous."""
        tokens, num_heads = q.shape[0], q.shape[1]
        q_stride = self._check_rows(q, tokens, num_heads, "q")
        k_stride = self._check_rows(k, tokens, self.num_kv_heads, "k")
        v_stride = self._check_rows(v, tokens, self.num_kv_heads, "v")
        if q_weight is not None:
            self._check_dense(q_weight, (self.head_dim,), self.dtype, "q_weight")
        if k_weight is not None:
            self._check_dense(k_weight, (self.head_dim,), self.dtype, "k_weight")
        batch, maxb = self._check_batch(block_tables, context_lens, query_starts)
        if out is None:
            out = self._empty(q.shape, self.dtype, stream)
        else:
            self._check_dense(out, (tokens, num_heads, self.head_dim), self.dtype, "out")
        if rope is not None and rope.handle is None:  # (NULL would mean no rotation)
            raise ValueError("the Rope is closed")
        self._check_current()
        B.pa_norm_rope_write_kv(self.handle, layer, out, q, q_stride, k, k_stride, v, v_stride,
                                None if rope is None else rope.handle, q_weight, k_weight, eps,
                                block_tables, maxb, context_lens, query_starts, batch, tokens,
                                num_heads, stream)
        return out

    def set_prefill_kernel(self, kind: str) -> None:
        """'auto' (default), 'mma' or 'tcgen05' (bf16 pools)."""
        B.pa_pool_set_prefill_kernel(self.handle, _PREFILL_KERNELS[kind])

    def prefill_workspace_size(self, batch: int, num_tokens: int, num_heads: int,
                               max_blocks_per_seq: int) -> int:
        return B.pa_prefill_workspace_size(self.handle, batch, num_tokens, num_heads,
                                           max_blocks_per_seq)

    def prefill_attention(self, q: torch.Tensor, layer: int, block_tables: torch.Tensor,
                          context_lens: torch.Tensor, query_starts: torch.Tensor, scale: float,
                          out: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """Causal attention of the new tokens (rows query_starts[b] ..
        query_starts[b + 1] of q, the last of sequence b's context_lens[b]) over
        the cache, which holds them already.  q and out: [tokens, num_heads,
        head_dim], contiguous, the pool's dtype."""
        tokens, num_heads = q.shape[0], q.shape[1]
        shape = (tokens, num_heads, self.head_dim)
        self._check_dense(q, shape, self.dtype, "q")
        batch, maxb = self._check_batch(block_tables, context_lens, query_starts)
        if out is None:
            out = self._empty(shape, self.dtype, stream)
        else:
            self._check_dense(out, shape, self.dtype, "out")
        self._check_current()
        if workspace is None:  # (the call checks one that is given)
            need = self.prefill_workspace_size(batch, tokens, num_heads, maxb)
            if need:
                workspace = self._empty((need,), torch.uint8, stream)
        wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
        B.pa_prefill_attention(out, q, self.handle, layer, block_tables, maxb, context_lens,
                               query_starts, batch, tokens, num_heads, scale, workspace, wbytes,
                               stream)
        return out

    # -- pages --------------------------------------------------------------
    def copy_blocks(self, src_ids: torch.Tensor, dst_ids: torch.Tensor, stream=None) -> None:
        """Page src_ids[i] to page dst_ids[i] (int32), all layers."""
        n = src_ids.shape[0]
        self._check_dense(src_ids, (n,), torch.int32, "src_ids")
        self._check_dense(dst_ids, (n,), torch.int32, "dst_ids")
        self._check_current()
        B.pa_copy_blocks(self.handle, src_ids, dst_ids, n, stream)

    def page_shares(self) -> torch.Tensor:
        """A new array of page shares (owners beyond the first): nothing shared."""
        return torch.zeros(self.num_blocks, dtype=torch.int32, device=self.pool.device)

    def device_fork_sequences(self, stack: torch.Tensor, shares: torch.Tensor,
                              block_tables: torch.Tensor, context_lens: torch.Tensor,
                              parents: torch.Tensor, children: torch.Tensor, stream=None) -> None:
        """Rows children[i] continue rows parents[i]: full pages shared, the
        partial last page copied into one from the device stack."""
        n = parents.shape[0]
        batch, maxb = self._check_batch(block_tables, context_lens)
        self._check_pages(stack, shares)
        self._check_dense(parents, (n,), torch.int32, "parents")
        self._check_dense(children, (n,), torch.int32, "children")
        self._check_current()
        B.pa_device_fork_sequences(self.handle, stack, shares, block_tables, maxb, context_lens,
                                   batch, parents, children, n, stream)

    def device_free_shared(self, stack: torch.Tensor, shares: torch.Tensor,
                           block_tables: torch.Tensor, context_lens: torch.Tensor,
                           finished: torch.Tensor, stream=None) -> None:
        """device_free_blocks for rows that may share pages."""
        batch, maxb = self._check_batch(block_tables, context_lens)
        self._check_pages(stack, shares)
        self._check_dense(finished, (batch,),
                          torch.bool if finished.dtype is torch.bool else torch.uint8, "finished")
        self._check_current()
        B.pa_device_free_shared(self.handle, stack, shares, block_tables, maxb, context_lens,
                                finished, batch, stream)

    def compact_workspace_size(self) -> int:
        return B.pa_compact_workspace_size(self.handle)

    def device_compact_blocks(self, stack: torch.Tensor, block_tables: torch.Tensor,
                              context_lens: torch.Tensor, shares: Optional[torch.Tensor] = None,
                              out_stack: Optional[torch.Tensor] = None,
                              out_tables: Optional[torch.Tensor] = None,
                              out_shares: Optional[torch.Tensor] = None,
                              remap: Optional[torch.Tensor] = None,
                              workspace: Optional[torch.Tensor] = None, stream=None):
        """Moves the pages in use to the lowest ids.  Returns the new (stack,
        tables, shares, remap); remap[old id] is a page's new id."""
        batch, maxb = self._check_batch(block_tables, context_lens)
        self._check_pages(stack, shares)
        new = lambda like: self._empty(like.shape, torch.int32, stream)  # noqa: E731
        out_stack = new(stack) if out_stack is None else out_stack
        out_tables = new(block_tables) if out_tables is None else out_tables
        if shares is not None and out_shares is None:
            out_shares = new(shares)
        remap = self._empty((self.num_blocks,), torch.int32, stream) if remap is None else remap
        self._check_pages(out_stack, out_shares)
        self._check_dense(out_tables, tuple(block_tables.shape), torch.int32, "out_tables")
        self._check_dense(remap, (self.num_blocks,), torch.int32, "remap")
        self._check_current()
        if workspace is None:
            workspace = self._empty((self.compact_workspace_size(),), torch.uint8, stream)
        B.pa_device_compact_blocks(self.handle, stack, shares, block_tables, maxb, context_lens,
                                   batch, out_stack, out_shares, out_tables, remap, workspace,
                                   workspace.numel() * workspace.element_size(), stream)
        return out_stack, out_tables, out_shares, remap

    # -- checks of what only the tensors know --------------------------------
    def _empty(self, shape, dtype, stream) -> torch.Tensor:
        """A tensor that `stream` may write at once (torch reuses memory in the
        order of the stream it was allocated on)."""
        if stream is None:
            return torch.empty(shape, dtype=dtype, device=self.pool.device)
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=self.pool.device)
        with torch.cuda.stream(stream):
            return torch.empty(shape, dtype=dtype, device=self.pool.device)

    def _check_current(self) -> None:
        """The calls launch on torch's current device; its kernels could not reach
        a pool elsewhere."""
        if self._device_index < 0 or torch.cuda.current_device() != self._device_index:
            raise ValueError(f"the pool is on {self.pool.device}, which is not the current CUDA device")

    def _check_dense(self, t: torch.Tensor, shape, dtype, name: str) -> None:
        if (t.shape == shape and t.dtype is dtype and t.get_device() == self._device_index
                and t.is_contiguous()):
            return
        if t.dtype != dtype:
            raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
        if t.get_device() != self._device_index:
            raise ValueError(f"{name} is on {t.device}, the pool on {self.pool.device}")
        raise ValueError(f"{name} must be contiguous with shape {tuple(shape)}, "
                         f"not {tuple(t.shape)}")

    def _check_rows(self, t: torch.Tensor, tokens: int, heads: int, name: str) -> int:
        """The stride between the tokens of [tokens, heads, head_dim] rows."""
        d = self.head_dim
        if t.shape != (tokens, heads, d) or t.dtype is not self.dtype:
            raise ValueError(f"{name} must be {self.dtype} [{tokens}, {heads}, {d}], "
                             f"not {t.dtype} {tuple(t.shape)}")
        if t.get_device() != self._device_index:
            raise ValueError(f"{name} is on {t.device}, the pool on {self.pool.device}")
        stride = t.stride()
        if tokens and (stride[2] != 1 or (heads > 1 and stride[1] != d)):
            raise ValueError(f"{name}: the heads of a token must be contiguous")
        return stride[0] if tokens > 1 else heads * d

    def _check_batch(self, block_tables, context_lens, query_starts=None):
        batch, maxb = block_tables.shape  # (two dimensions, or a ValueError)
        self._check_dense(block_tables, (batch, maxb), torch.int32, "block_tables")
        self._check_dense(context_lens, (batch,), torch.int32, "context_lens")
        if query_starts is not None:
            self._check_dense(query_starts, (batch + 1,), torch.int32, "query_starts")
        return batch, maxb

    def _check_pages(self, stack, shares) -> None:
        self._check_dense(stack, (self.num_blocks + 1,), torch.int32, "stack")
        if shares is not None:
            self._check_dense(shares, (self.num_blocks,), torch.int32, "shares")

    def close(self) -> None:
        if getattr(self, "handle", None):
            B.pa_pool_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
