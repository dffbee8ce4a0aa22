"""Plain 64-bit implementations of the operators for several new tokens per
sequence and of the page operations, in torch on any device and plain Python,
with the error bounds their kernels are held to."""
import math

import numpy as np
import torch

HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
U = 2.0 ** -24  # one fp32 rounding


def cdiv(a, b):
    return -(-a // b)


def random_tables(rng, ctx, block, num_blocks, max_blocks):
    """Distinct random pages for every sequence, -1 past them."""
    ids = [int(x) for x in rng.permutation(num_blocks)]
    t = np.full((len(ctx), max_blocks), -1, np.int32)
    for b, c in enumerate(ctx):
        for j in range(cdiv(c, block)):
            t[b, j] = ids.pop()
    return t


def starts_of(new):
    return np.concatenate(([0], np.cumsum(new))).astype(np.int32)


# ------------------------------------------------------ norm + rotation


def frequencies(rotary, base, scaling="none", factor=1.0, original=4096.0, low=1.0, high=4.0):
    j = np.arange(rotary // 2, dtype=np.float64)
    if scaling == "ntk":
        base = base * factor ** (rotary / (rotary - 2))
    f = np.power(float(base), -2.0 * j / rotary)
    if scaling == "linear":
        f = f / factor
    if scaling == "parts":
        g = np.clip((original * f / (2 * math.pi) - low) / (high - low), 0.0, 1.0)
        f = (1 - g) * f / factor + g * f
    return f


def norm_rope(x, pos, freq, interleaved, amplitude, weight, eps):
    """x [T, heads, D] (any float type), pos [T]: (result, size of each rotated
    element's pair) in 64 bits."""
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.double()
    if freq is None:
        return x, x.abs()
    r = 2 * len(freq)
    angle = pos.double()[:, None, None] * torch.as_tensor(freq, device=x.device)
    cos, sin = angle.cos() * amplitude, angle.sin() * amplitude
    y, size = x.clone(), x.abs()
    if interleaved:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y[..., 0:r:2], y[..., 1:r:2] = a * cos - b * sin, a * sin + b * cos
        size[..., 0:r:2] = size[..., 1:r:2] = (a.abs() + b.abs()) * abs(amplitude)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y[..., :r // 2], y[..., r // 2:r] = a * cos - b * sin, a * sin + b * cos
        size[..., :r // 2] = size[..., r // 2:r] = (a.abs() + b.abs()) * abs(amplitude)
    return y, size


def norm_rope_bound(y, size, dtype):
    """Half a step of the stored type, and the fp32 work in between: the norm's
    sum (13 additions at most in a chain, halved by the root: 7 U), the root (2
    ulp, 4 U), two products (2 U); the angle (2^-25 half turns: 2 U), its sine (2
    ulp: 4 U) and amplitude (1 U); two products and an addition (3 U): 23 U, taken
    as 32 U."""
    return HALF_STEP[dtype] * y.abs() + 32 * U * size


# ------------------------------------------------------------ attention


def prefill(pool, q, tables, ctx, new, scale, layer=0):
    """(out, bound): out [T, H, D] in 64 bits for a fused pool [nb, 2, L, Hkv,
    B, D]; table entries outside the pool have no weight.

    The bound on a row: half a step of the output type; the weights' error
    times sum p |v|.  A score is D products summed in fp32 (each partial sum off
    by U of at most A = sum |q k| scale) and scaled: (D + 4) U A, which is its
    weight's relative error; so is the sum's, once more, with a rounding for each
    of its terms (n U; they all have one sign) and the exponential's 2^-22 twice.
    Products with v: n more.  bf16 pools round the weights to bf16 (2^-8)."""
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
        start += n
        pages = torch.as_tensor(np.ascontiguousarray(tables[b, :cdiv(c, block)]), device=q.device).long()
        ok = (pages >= 0) & (pages < nb)
        kv = pool[pages.clamp(0, nb - 1), :, layer].double()      # [blocks, 2, Hkv, B, D]
        kv = kv.permute(1, 2, 0, 3, 4).reshape(2, hkv, -1, d)[:, :, :c]
        has = ok.repeat_interleave(block)[:c]
        kv = torch.where(has[None, None, :, None], kv, 0.0)
        x = q[rows].double().view(n, hkv, group, d)
        see = (torch.arange(c, device=q.device) <= torch.arange(c - n, c, device=q.device)[:, None]) & has
        s = torch.einsum("nhgd,htd->nhgt", x, kv[0]) * scale
        size = torch.einsum("nhgd,htd->nhgt", x.abs(), kv[0].abs()) * abs(scale)
        s = torch.where(see[:, None, None], s, float("-inf"))
        top = s.amax(-1, keepdim=True)
        e = torch.exp(s - torch.where(torch.isfinite(top), top, 0.0))
        e = torch.where(see[:, None, None], e, 0.0)
        p = e / e.sum(-1, keepdim=True).clamp(min=1e-300)
        # 0 * (a value no row may see) must not matter: sum where p > 0 only
        v = torch.where(torch.isfinite(kv[1]), kv[1], 0.0)
        o = torch.einsum("nhgt,htd->nhgd", p, v)
        mag = torch.einsum("nhgt,htd->nhgd", p, v.abs())
        a = torch.where(see[:, None, None], size, 0.0).amax(-1, keepdim=True)
        rel = 2 * ((d + 4) * U * a + 2.0 ** -22) + 2 * (c + 8) * U
        if q.dtype == torch.bfloat16:
            rel = rel + 2.0 ** -8
        out[rows] = o.reshape(n, heads, d)
        bound[rows] = (HALF_STEP[q.dtype] * o.abs() * (1 + rel) + rel * mag).reshape(n, heads, d)
    return out, bound


# ---------------------------------------------------------------- pages


class Pages:
    """Owners, tables, stack and page contents, one step at a time."""

    def __init__(self, num_blocks, block, tables, lens, stack, pool):
        self.nb, self.block = num_blocks, block
        self.tables, self.lens = tables.copy(), lens.copy()
        self.stack, self.pool = list(stack), pool.clone()   # stack: ids from the bottom up
        self.shares = np.zeros(num_blocks, np.int32)

    def fork(self, parents, children):
        for p, c in zip(parents, children):
            n = int(self.lens[p])
            row = np.full(self.tables.shape[1], -1, np.int32)
            for j in range(n // self.block):
                row[j] = self.tables[p, j]
                self.shares[row[j]] += 1
            if n % self.block:
                j = n // self.block
                if self.stack:
                    row[j] = self.stack.pop()
                    old = int(self.tables[p, j])
                    self.pool[row[j], :, :, :, :n % self.block] = \
                        self.pool[old, :, :, :, :n % self.block]
            self.tables[c], self.lens[c] = row, n

    def free(self, finished):
        owners = {}
        for b in range(len(self.lens)):
            if finished[b]:
                for j in range(cdiv(int(self.lens[b]), self.block)):
                    page = int(self.tables[b, j])
                    owners[page] = owners.get(page, int(self.shares[page]) + 1) - 1
                    if owners[page] == 0:
                        self.stack.append(page)
                    self.shares[page] = max(owners[page] - 1, 0)
                    self.tables[b, j] = -1

    def compact(self):
        free = set(self.stack)
        live = [i for i in range(self.nb) if i not in free]
        holes = [i for i in range(len(live)) if i in free]
        movers = [i for i in live if i >= len(live)]
        remap = np.full(self.nb, -1, np.int32)
        for i in live:
            remap[i] = i
        for a, b in zip(movers, holes):
            remap[a] = b
            self.pool[b] = self.pool[a]
        shares = np.zeros(self.nb, np.int32)
        for i in live:
            shares[remap[i]] = self.shares[i]
        for b in range(len(self.lens)):
            for j in range(cdiv(int(self.lens[b]), self.block)):
                self.tables[b, j] = remap[self.tables[b, j]]
        self.shares, self.stack = shares, list(range(self.nb - 1, len(live) - 1, -1))
        return remap
