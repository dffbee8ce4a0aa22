"""Plain implementations of the operators for drafted trees: Python lists for pages, slots,
masks and paths, 64-bit torch for the attention, with the bound its kernels are held to."""
import numpy as np
import torch

import prompt_reference as R


def random_tree(rng, n, shape="random"):
    """Parents of n nodes, each before its children; -1 for the root."""
    if shape == "chain":
        return list(range(-1, n - 1))
    if shape == "wide":
        return [(i - 1) // 2 if i else -1 for i in range(n)]
    return [int(rng.integers(0, i)) if i else -1 for i in range(n)]


def ancestors(tree):
    """Row i: the nodes on the way from i to its root, as a whole number of bits."""
    seen = []
    for i, p in enumerate(tree):
        seen.append((seen[p] if p >= 0 else 0) | 1 << i)
    return seen


def depths(tree):
    d = []
    for p in tree:
        d.append(d[p] + 1 if p >= 0 else 0)
    return d


def mask_words(bits, words):
    """Whole numbers as int32 [rows, words]."""
    out = np.zeros((len(bits), words), np.uint32)
    for i, m in enumerate(bits):
        for w in range(words):
            out[i, w] = (m >> (32 * w)) & 0xFFFFFFFF
    return out.view(np.int32)


class Plan:
    """Pages, slots, positions and masks of a batch's new tokens, one token at a time."""

    def __init__(self, block, tables, stack, cached, new, trees, num_tokens, words):
        self.tables, self.stack = tables.copy(), list(stack)   # stack: ids from the bottom up
        self.lens = [c + n for c, n in zip(cached, new)]
        self.starts = [0]
        self.slots, self.positions, masks = [], [], []
        for b, (c, n) in enumerate(zip(cached, new)):
            tree = None if trees is None else trees[b]
            tree = random_tree(None, n, "chain") if tree is None else tree
            for at in range(c, c + n):
                if at % block == 0:
                    self.tables[b, at // block] = self.stack.pop() if self.stack else -1
                page = int(self.tables[b, at // block])
                self.slots.append(page * block + at % block if page >= 0 else -1)
            self.positions += [c + d for d in depths(tree)]
            masks += ancestors(tree)
            self.starts.append(self.starts[-1] + n)
        pad = num_tokens - self.starts[-1]
        self.slots += [-1] * pad
        self.positions += [0] * pad
        self.masks = mask_words(masks + [0] * pad, words) if words else None


def trim(block, tables, stack, lens, new_lens):
    tables, stack = tables.copy(), list(stack)
    for b in reversed(range(len(lens))):
        for j in reversed(range(R.cdiv(int(new_lens[b]), block), R.cdiv(int(lens[b]), block))):
            stack.append(int(tables[b, j]))
            tables[b, j] = -1
    return tables, stack


def walk(tree, tokens, targets, most):
    path, at = [0] if tree else [], 0
    while path and len(path) < most:
        after = [i for i in range(1, len(tree)) if tree[i] == at and tokens[i] == targets[at]]
        if not after:
            break
        at = after[0]
        path.append(at)
    return path


def attention(pool, q, tables, ctx, new, bits, scale, layer=0):
    """(out, bound) of prompt_reference.prefill with rows that see the keys before the
    sequence's new tokens and the new tokens in `bits` (a whole number per row)."""
    nb, _, _, hkv, block, d = pool.shape
    t, heads = q.shape[0], q.shape[1]
    group = heads // hkv
    out = torch.zeros((t, heads, d), dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(out)
    start = 0
    for b, (n, c) in enumerate(zip(new, ctx)):
        if n == 0:
            continue
        rows = slice(start, start + n)
        pages = torch.as_tensor(np.ascontiguousarray(tables[b, :R.cdiv(c, block)]), device=q.device).long()
        ok = (pages >= 0) & (pages < nb)
        kv = pool[pages.clamp(0, nb - 1), :, layer].double()
        kv = kv.permute(1, 2, 0, 3, 4).reshape(2, hkv, -1, d)[:, :, :c]
        has = ok.repeat_interleave(block)[:c]
        own = torch.tensor([[bits[start + i] >> j & 1 for j in range(n)] for i in range(n)],
                           dtype=torch.bool, device=q.device)
        see = torch.cat((torch.ones((n, c - n), dtype=torch.bool, device=q.device), own), 1) & has
        start += n
        kv = torch.where(see.any(0)[None, None, :, None], kv, 0.0)
        x = q[rows].double().view(n, hkv, group, d)
        s = torch.einsum("nhgd,htd->nhgt", x, kv[0]) * scale
        size = torch.einsum("nhgd,htd->nhgt", x.abs(), kv[0].abs()) * abs(scale)
        s = torch.where(see[:, None, None], s, float("-inf"))
        top = s.amax(-1, keepdim=True)
        e = torch.exp(s - torch.where(torch.isfinite(top), top, 0.0))
        e = torch.where(see[:, None, None], e, 0.0)
        p = e / e.sum(-1, keepdim=True).clamp(min=1e-300)
        o = torch.einsum("nhgt,htd->nhgd", p, kv[1])
        mag = torch.einsum("nhgt,htd->nhgd", p, kv[1].abs())
        a = torch.where(see[:, None, None], size, 0.0).amax(-1, keepdim=True)
        # (as derived at prompt_reference.prefill: the same products and sums)
        rel = 2 * ((d + 4) * R.U * a + 2.0 ** -22) + 2 * (c + 8) * R.U
        if q.dtype == torch.bfloat16:
            rel = rel + 2.0 ** -8
        out[rows] = o.reshape(n, heads, d)
        bound[rows] = (R.HALF_STEP[q.dtype] * o.abs() * (1 + rel) + rel * mag).reshape(n, heads, d)
    return out, bound
