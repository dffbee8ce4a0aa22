"""Page operations at their edges: forks of rows whose partial page is missing,
shared frees at the sizes where the shared-memory limit turns, compactions of pools
of different sizes side by side."""
import ctypes
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import prompt_reference as R
from paged_kv_cache_239_gb300 import binding as B
from paged_kv_cache_239_gb300.pool import BlockPool

pytestmark = pytest.mark.gpu

REPO = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def ints(x, dev):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)


def stack_of(ids, nb, dev):
    s = np.full(nb + 1, -1, np.int32)
    s[0], s[1:1 + len(ids)] = len(ids), ids
    return ints(s, dev)


# --------------------------------------------------------------------- fork


def fork_state(dev, nb, free, tables, lens):
    pool_t = torch.randn((nb, 2, 2, 1, 16, 8), generator=torch.Generator(device=dev).manual_seed(5), device=dev)
    cache = BlockPool(nb, 16, 2, 1, 8, tensor=pool_t)
    return cache, stack_of(free, nb, dev), cache.page_shares(), ints(tables, dev), ints(lens, dev)


@pytest.mark.parametrize("bad", [-1, -7, 12, 1 << 30])
def test_fork_of_a_missing_partial_page(cuda_device, bad):
    """A parent whose partial page is no page has nothing to copy: its child's entry is
    -1, not the id of a page that was never written for it, and no page is taken."""
    dev = cuda_device
    tables = np.full((8, 3), -1, np.int32)
    tables[0, :2], tables[1, :2], tables[2, 0] = (3, bad), (4, 5), bad
    cache, stack, shares, bt, ln = fork_state(dev, 12, [9, 10, 11], tables, [20, 30, 5, 0, 0, 0, 0, 0])
    before = cache.pool.clone()
    cache.device_fork_sequences(stack, shares, bt, ln, ints([0, 1, 2, 1], dev), ints([3, 4, 5, 6], dev))
    assert B.pa_get_status() == B.PA_STATUS_BAD_BLOCK_ID
    want = tables.copy()
    want[3, 0], want[4, :2], want[6, :2] = 3, (4, 11), (4, 10)   # the good pairs take 11 and 10
    assert np.array_equal(bt.cpu().numpy(), want)
    assert ln.tolist() == [20, 30, 5, 20, 30, 5, 30, 0]
    assert stack[:2].tolist() == [1, 9]
    assert shares.tolist() == [0, 0, 0, 1, 2] + [0] * 7
    before[11, ..., :14, :] = before[5, ..., :14, :]
    before[10, ..., :14, :] = before[5, ..., :14, :]
    assert torch.equal(cache.pool, before)
    cache.close()


def test_fork_of_a_fork_that_ran_dry(cuda_device):
    """What a dry stack left without a page stays without one in the forks of it, also
    when there are free pages again."""
    dev = cuda_device
    tables = np.full((4, 2), -1, np.int32)
    tables[0] = 1, 2
    cache, stack, shares, bt, ln = fork_state(dev, 8, [], tables, [20, 0, 0, 0])
    cache.device_fork_sequences(stack, shares, bt, ln, ints([0], dev), ints([1], dev))
    assert B.pa_get_status() == B.PA_STATUS_NO_FREE_BLOCKS and bt[1].tolist() == [1, -1]
    stack = stack_of([6, 7], 8, dev)
    cache.device_fork_sequences(stack, shares, bt, ln, ints([1], dev), ints([2], dev))
    assert B.pa_get_status() == B.PA_STATUS_BAD_BLOCK_ID
    assert bt[2].tolist() == [1, -1] and stack[:3].tolist() == [2, 6, 7] and int(ln[2]) == 20
    cache.close()


@pytest.mark.parametrize("n", [257, 8192])
def test_fork_many_children(cuda_device, n):
    """Children whose pages are counted in several steps, bad partial pages among their parents'."""
    dev, block, parents = cuda_device, 4, 64
    rng = np.random.default_rng(n)
    rows, nb = parents + n, parents * 3 + n + 5
    lens = np.zeros(rows, np.int32)
    lens[:parents] = rng.integers(0, 3 * block + 1, parents)
    tables = np.full((rows, 3), -1, np.int32)
    for b in range(parents):
        for j in range(R.cdiv(int(lens[b]), block)):
            tables[b, j] = 3 * b + j
        if b % 9 == 0 and lens[b] % block:
            tables[b, lens[b] // block] = -1
    free = [int(x) for x in rng.permutation(np.arange(parents * 3, nb))]
    pool_t = torch.randn((nb, 2, 1, 1, block, 4), device=dev)
    cache = BlockPool(nb, block, 1, 1, 4, tensor=pool_t)
    par, chi = rng.integers(0, parents, n), parents + rng.permutation(n)
    want_t, want_p, left = tables.copy(), pool_t.clone(), list(free)
    want_s = np.zeros(nb, np.int32)
    for p, c in zip(par, chi):
        full, part = divmod(int(lens[p]), block)
        want_t[c, :full] = tables[p, :full]
        want_s[tables[p, :full]] += 1
        if part and tables[p, full] >= 0:
            want_t[c, full] = left.pop()
            want_p[want_t[c, full], ..., :part, :] = want_p[int(tables[p, full]), ..., :part, :]
    bt, ln, stack, shares = ints(tables, dev), ints(lens, dev), stack_of(free, nb, dev), cache.page_shares()
    cache.device_fork_sequences(stack, shares, bt, ln, ints(par, dev), ints(chi, dev))
    assert B.pa_get_status() == B.PA_STATUS_BAD_BLOCK_ID
    assert np.array_equal(bt.cpu().numpy(), want_t) and np.array_equal(shares.cpu().numpy(), want_s)
    assert int(stack[0]) == len(left) and torch.equal(cache.pool, want_p)
    cache.close()


# -------------------------------------------------------------- shared free

FREE_ALONE = """
import sys
sys.path.insert(0, {repo!r})
import torch
from paged_kv_cache_239_gb300 import binding as B
from paged_kv_cache_239_gb300.pool import BlockPool
rows, width = {rows}, {width}
cache = BlockPool(rows, 1, 1, 1, 4, dtype=torch.float32)
i32 = dict(dtype=torch.int32, device="cuda")
tables = torch.full((rows, width), -1, **i32)
tables[:, 0] = torch.arange(rows, **i32)
stack = torch.full((rows + 1,), -1, **i32)
stack[0] = 0
done = torch.ones(rows, dtype=torch.uint8, device="cuda")
cache.device_free_shared(stack, cache.page_shares(), tables, torch.ones(rows, **i32), done)
assert stack.tolist() == [rows] + list(range(rows)), stack
assert bool((tables == -1).all()) and B.pa_get_status() == 0
print("freed")
"""


@pytest.mark.parametrize("rows,width", [(256, 375), (64, 1523), (128, 758), (256, 376), (128, 768)])
def test_free_shared_as_the_first_call(cuda_device, rows, width):
    """Tables whose places take about 48 KiB of shared memory, which is what a kernel gets
    without asking for more: in a process of their own, so that no call asked before."""
    run = subprocess.run([sys.executable, "-c", FREE_ALONE.format(repo=REPO, rows=rows, width=width)],
                         capture_output=True, text=True, timeout=300, cwd=REPO)
    assert run.returncode == 0 and "freed" in run.stdout, run.stderr[-2000:]


# ------------------------------------------------------------------ compact


def test_compact_pools_of_two_sizes_side_by_side(cuda_device, tmp_path):
    """Two host threads compact pools whose maps take little and much shared memory: the
    one's launch does not take the other's limit away."""
    dev, n, results, start = cuda_device, 20000, {}, threading.Barrier(2)
    so = tmp_path / "loop.so"
    subprocess.run(["gcc", "-std=c11", "-O2", "-shared", "-fPIC", "-I", os.path.join(REPO, "include"),
                    os.path.join(REPO, "tests", "c_abi", "pa_compact_loop.c"), "-o", str(so)], check=True)
    loop = ctypes.CDLL(str(so)).compact_loop
    call = ctypes.cast(B.lib().pa_device_compact_blocks, ctypes.c_void_p)
    p = ctypes.c_void_p

    def work(nb):
        torch.cuda.set_device(dev)
        cache = BlockPool(nb, 1, 1, 1, 4, tensor=torch.zeros((nb, 2, 1, 1, 1, 4), device=dev))
        stack, bt, ln = stack_of([nb - 1], nb, dev), ints([[0]], dev), ints([1], dev)
        out_stack, out_bt, _, remap = cache.device_compact_blocks(stack, bt, ln)
        ws = torch.empty(cache.compact_workspace_size(), dtype=torch.uint8, device=dev)
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        start.wait(60)
        results[nb] = loop(call, n, p(cache.handle), *(p(t.data_ptr()) for t in (stack, bt, ln, out_stack, out_bt,
                                                                                  remap, ws)),
                           ctypes.c_size_t(ws.numel()), p(side.cuda_stream))
        side.synchronize()
        cache.close()

    threads = [threading.Thread(target=work, args=(nb,)) for nb in (4, 200000)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert results == {4: B.PA_OK, 200000: B.PA_OK}
    assert B.pa_get_status() == 0
