// pa_pages.cu -- operations on whole pages (physical blocks): copies, forks of
// sequences that share pages, frees of shared pages, and compaction.
//
// A page is 2 * L * Hkv tiles of B x D contiguous elements.  The copies move
// tiles (or, for a fork's last page, the live first rows of each tile) in
// 16-byte chunks, a warp to a tile with four chunks per lane in flight; they are
// bound by bytes: 1024 pages of 512 KiB take 166 us, 6.5 TB/s read and written (97 % of
// a plain copy's rate), 16 pages of 192 KiB 2.6 us.  What decides which pages to
// copy runs on the device too, from the free stack, the tables and the lengths, so
// that no call waits for the host.
//
// Sharing: shares[id] counts the owners of page id beyond the first, so an
// array of zeros describes a pool in which nothing is shared, and the calls
// that do not know of sharing keep their meaning.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kCopyThreads = 256;

// Tile `i` of a page: its K or V base and its element offset within the page.
__device__ __forceinline__ unsigned char* tile_base(const PageGeom& g, int i, long long* off) {
    const int h = i % g.Hkv;
    i /= g.Hkv;
    const int layer = i % g.L;
    *off = ((long long)layer * g.s_layer + (long long)h * g.s_head) * g.elt;
    return static_cast<unsigned char*>(i / g.L ? g.v_base : g.k_base);
}

// The warp copies the first `chunks` 16-byte chunks of tile `i` of page src
// to page dst.
__device__ __forceinline__ void warp_copy_tile(const PageGeom& g, int i, int src, int dst,
                                               int chunks, int lane) {
    long long off;
    unsigned char* base = tile_base(g, i, &off);
    const uint4* a = reinterpret_cast<const uint4*>(base + off + (long long)src * g.s_blk * g.elt);
    uint4* b = reinterpret_cast<uint4*>(base + off + (long long)dst * g.s_blk * g.elt);
    int c = lane;
    for (; c + 96 < chunks; c += 128) {
        const uint4 v0 = ld_dep(a + c), v1 = ld_dep(a + c + 32), v2 = ld_dep(a + c + 64),
                    v3 = ld_dep(a + c + 96);
        b[c] = v0, b[c + 32] = v1, b[c + 64] = v2, b[c + 96] = v3;
    }
    for (; c < chunks; c += 32) b[c] = ld_dep(a + c);
}

// The stack's height, held to what the array can hold (flagged if it was not).
__device__ __forceinline__ int stack_height(const int* stack, long long num_blocks,
                                            unsigned* status) {
    const int h = ld_dep(stack);
    if (h >= 0 && h <= num_blocks) return h;
    if (threadIdx.x == 0) atomicOr(status, kStatusBadLength);
    return h < 0 ? 0 : (int)num_blocks;
}

// Exclusive prefix sum of `v` over the CTA; `total` receives the sum.
__device__ __forceinline__ int cta_exclusive_scan(int v, int* s_warp, int& total) {
    const int lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(kFullMask, incl, o);
        if (lane >= o) incl += t;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        int w = lane < (blockDim.x >> 5) ? s_warp[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(kFullMask, w, o);
            if (lane >= o) w += t;
        }
        s_warp[lane] = w;
    }
    __syncthreads();
    const int before = warp > 0 ? s_warp[warp - 1] : 0;
    total = s_warp[(blockDim.x >> 5) - 1];
    __syncthreads();
    return before + incl - v;
}

// ------------------------------------------------------------------- copies

__global__ void __launch_bounds__(kCopyThreads)
pa_copy_blocks_kernel(const PageGeom g, const int* src, const int* dst, const int* count, int n_max) {
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int tiles = 2 * g.L * g.Hkv;
    const int chunks = g.tile_bytes / 16;
    const int n = count != nullptr ? ld_dep(count) : n_max;
    const long long total = (long long)n * tiles;
    const long long warps = (long long)gridDim.x * (kCopyThreads / 32);
    for (long long w = (long long)blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5); w < total;
         w += warps) {
        const int pair = (int)(w / tiles), tile = (int)(w % tiles);
        const int a = ld_dep(src + pair), b = ld_dep(dst + pair);
        if (a < 0 || a >= g.num_blocks || b < 0 || b >= g.num_blocks) {
            if (tile == 0 && lane == 0) atomicOr(g.status, kStatusBadBlock);
            continue;
        }
        if (a != b) warp_copy_tile(g, tile, a, b, chunks, lane);
    }
}

// --------------------------------------------------------------------- fork

// A pair of a fork: the parent's row, length and partial last page (-1 where it has
// none, or one that is no page and so holds nothing to copy), or par = -1 where the
// pair is to be skipped (both flagged by `report`).
struct ForkPair {
    int par, chi, len, old;
};
__device__ __forceinline__ ForkPair fork_pair(const ForkParams& p, int i, bool report) {
    ForkPair f{ld_dep(p.parents + i), ld_dep(p.children + i), 0, -1};
    bool good = f.par >= 0 && f.par < p.batch && f.chi >= 0 && f.chi < p.batch && f.par != f.chi;
    if (good) {
        f.len = ld_dep(p.lens + f.par);
        good = f.len >= 0 && f.len <= p.maxb * p.g.B;
    }
    if (!good) {
        f.par = -1;
        if (report) atomicOr(p.g.status, kStatusBadLength);
    } else if (f.len % p.g.B) {
        f.old = ld_dep(p.bt + (long long)f.par * p.maxb + f.len / p.g.B);
        if (f.old < 0 || f.old >= p.g.num_blocks) {
            f.old = -1;
            if (report) atomicOr(p.g.status, kStatusBadBlock);
        }
    }
    return f;
}

// How many of the pairs before `n` take a page (the CTA counts together).
__device__ __forceinline__ int fork_pages_before(const ForkParams& p, int n) {
    int mine = 0;
    for (int i0 = 0; i0 < n; i0 += blockDim.x) {
        const int i = i0 + threadIdx.x;
        mine += __syncthreads_count(i < n && fork_pair(p, i, false).old >= 0);
    }
    return mine;
}

// Child blockIdx.x takes its parent's table: full pages by reference, the
// partial last page (if any) as a page of its own from the stack's top, in
// increasing order of the children.  Each CTA counts the pages that the
// children before its own take, so that the rows and the copies run side by side and
// no launch comes before them: n / 256 steps at most per CTA, n^2 / 512 in the grid, which
// is nothing for a batch's children and all there is to it for tens of thousands
// (pages of 4 KiB: 128 children 6.0 us, 1,024 12.4, 8,192 137, 65,536 7.0 ms).  CTAs (x,
// 0) write the rows, all of them copy the tiles of the last page.  The stack's
// height is set by the kernel after this one, since every CTA reads it here.
__global__ void __launch_bounds__(kCopyThreads) pa_fork_kernel(const ForkParams p) {
    pdl_trigger();
    pdl_wait();
    const int i = blockIdx.x;
    const bool first = blockIdx.y == 0;
    const int lane = threadIdx.x & 31;
    const int height = stack_height(p.stack, p.g.num_blocks, p.g.status);
    const ForkPair f = fork_pair(p, i, first && threadIdx.x == 0);
    const int rank = fork_pages_before(p, i);
    if (f.par < 0) return;
    const int full = f.len / p.g.B, rows = f.len % p.g.B;
    int id = -1;
    if (f.old >= 0) {
        if (rank < height) {
            id = ld_dep(p.stack + height - rank);
            if (id < 0 || id >= p.g.num_blocks) {
                id = -1;
                if (first && threadIdx.x == 0) atomicOr(p.g.status, kStatusBadBlock);
            }
        } else if (first && threadIdx.x == 0) {
            atomicOr(p.g.status, kStatusNoFreeBlocks);
        }
    }
    const int* from = p.bt + (long long)f.par * p.maxb;
    if (first) {
        int* to = p.bt + (long long)f.chi * p.maxb;
        for (int j = threadIdx.x; j < p.maxb; j += kCopyThreads) {
            int e = -1;
            if (j < full) {
                e = ld_dep(from + j);
                if (e < 0 || e >= p.g.num_blocks) {
                    e = -1;
                    atomicOr(p.g.status, kStatusBadBlock);
                } else {
                    atomicAdd(p.shares + e, 1);
                }
            } else if (j == full) {
                e = id;
            }
            to[j] = e;
        }
        if (threadIdx.x == 0) p.lens[f.chi] = f.len;
    }
    if (id == -1) return;
    // the live rows of the partial last page
    const int tiles = 2 * p.g.L * p.g.Hkv;
    const int chunks = rows * (p.g.tile_bytes / p.g.B / 16);
    for (int t = blockIdx.y * (kCopyThreads / 32) + (threadIdx.x >> 5); t < tiles;
         t += gridDim.y * (kCopyThreads / 32))
        if (f.old != id) warp_copy_tile(p.g, t, f.old, id, chunks, lane);
}

__global__ void __launch_bounds__(kCopyThreads) pa_fork_height_kernel(const ForkParams p) {
    pdl_trigger();
    pdl_wait();
    const int height = stack_height(p.stack, p.g.num_blocks, p.g.status);
    const int taken = fork_pages_before(p, p.n);
    if (threadIdx.x == 0) p.stack[0] = taken < height ? height - taken : 0;
}

// --------------------------------------------------------------- shared free

// Each entry of a finished row gives up one ownership; a page without another
// owner is pushed by the last of the owners that gave it up in this call, in
// row and table order, so the stack does not depend on the threads' timing.
//  1  shares[id] -= 1 for every such entry: < 0 where no owner is left;
//  2  the owners of those pages bid with their place in the order; the lowest
//     code (the last place) stays in shares[id];
//  3  the winning entries are counted, a scan gives them their slots, and they
//     push and put shares[id] back to 0.
// The steps wait for one another.  A cluster of CTAs takes an equal share of the
// entries each and keeps their ids in shared memory between the steps: what
// bounds it is the scattered accesses to `shares`, about one per cycle and SM
// (64 finished groups of 3, 6,900 entries: one CTA 17 us).  Tables too large for
// that are read again in every step, by one CTA.
constexpr int kFreeCluster = 8;
constexpr int kFreeRows = 8192;                    // rows whose places fit
constexpr int kFreeEntries = kFreeCluster * 24576;  // entries whose ids fit

// Pages of row b that are given up (0 for a row that is not finished).
__device__ __forceinline__ int free_row_blocks(const FreeSharedParams& p, int b, bool report) {
    if (b >= p.batch || !p.finished[b]) return 0;
    const int n = ld_dep(p.lens + b);
    if (n < 0 || n > p.maxb * p.B) {
        if (report) atomicOr(p.status, kStatusBadLength);
        return 0;
    }
    return (n + p.B - 1) / p.B;
}
// The code of a place < 2^30: below every count that `shares` can hold.
__device__ __forceinline__ int free_bid(long long place) {
    return (int)(0x80000000u + (0x40000000u - (unsigned)place));
}
__device__ __forceinline__ void free_push(const FreeSharedParams& p, int slot, int id) {
    if (slot < p.num_blocks)
        p.stack[1 + slot] = id;
    else
        atomicOr(p.status, kStatusBadBlock);  // more ids than the pool holds
    p.shares[id] = 0;
}
__device__ __forceinline__ void free_height(const FreeSharedParams& p, int height, int pushed) {
    const long long h = (long long)height + pushed;
    p.stack[0] = (int)(h < p.num_blocks ? h : p.num_blocks);
}

__global__ void __launch_bounds__(kPlanThreads) pa_free_shared_kernel(const FreeSharedParams p) {
    pdl_trigger();
    pdl_wait();
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    extern __shared__ int s_start[];       // [batch + 1] places of the rows, then ids
    int* s_ids = s_start + p.batch + 1;
    __shared__ int s_warp[32], s_wins[kFreeCluster];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
    const int height = stack_height(p.stack, p.num_blocks, p.status);
    int count = 0;
    for (int at = 0; at < p.batch; at += kPlanThreads) {
        const int nblk = free_row_blocks(p, at + threadIdx.x, rank == 0);
        int total = 0;
        const int start = count + cta_exclusive_scan(nblk, s_warp, total);
        if (at + threadIdx.x < p.batch) s_start[at + threadIdx.x] = start;
        count += total;
    }
    if (threadIdx.x == 0) s_start[p.batch] = count;
    __syncthreads();
    // this CTA's entries: places [lo, hi)
    const int each = (count + ctas - 1) / ctas;
    const int lo = min(rank * each, count), hi = min(lo + each, count);
    for (int k = warp; k < p.batch; k += kPlanThreads / 32) {
        const int start = s_start[k];
        const int j1 = min(s_start[k + 1], hi) - start;
        int* row = p.bt + (long long)k * p.maxb;
#pragma unroll 4
        for (int j = max(lo - start, 0) + lane; j < j1; j += 32) {
            int id = ld_dep(row + j);
            row[j] = -1;
            if (id < 0 || id >= p.num_blocks) {
                id = -1;
                atomicOr(p.status, kStatusBadBlock);
            } else {
                atomicSub(p.shares + id, 1);
            }
            s_ids[start + j - lo] = id;
        }
    }
    __threadfence();
    cluster.sync();
    for (int e = lo + threadIdx.x; e < hi; e += kPlanThreads) {
        const int id = s_ids[e - lo];
        if (id >= 0 && __ldcg(p.shares + id) < 0) atomicMin(p.shares + id, free_bid(e));
    }
    __threadfence();
    cluster.sync();
    // a thread's entries are neighbours (an odd number of them: no two lanes on one
    // bank), so that one scan orders all
    const int mine_n = (hi - lo + kPlanThreads - 1) / kPlanThreads | 1;
    const int e0 = min(lo + (int)threadIdx.x * mine_n, hi), e1 = min(e0 + mine_n, hi);
    int mine = 0;
#pragma unroll 4
    for (int e = e0; e < e1; ++e) {
        const int id = s_ids[e - lo];
        const bool win = id >= 0 && __ldcg(p.shares + id) == free_bid(e);
        if (!win) s_ids[e - lo] = -1;
        mine += win;
    }
    int wins = 0;
    int slot = height + cta_exclusive_scan(mine, s_warp, wins);
    if (threadIdx.x < ctas) cluster.map_shared_rank(s_wins, threadIdx.x)[rank] = wins;
    cluster.sync();  // (and no CTA resets `shares` before all have compared)
    int pushed = 0;
    for (int r = 0; r < ctas; ++r) {
        if (r < rank) slot += s_wins[r];
        pushed += s_wins[r];
    }
    for (int e = e0; e < e1; ++e) {
        const int id = s_ids[e - lo];
        if (id >= 0) free_push(p, slot++, id);
    }
    if (rank == 0 && threadIdx.x == 0) free_height(p, height, pushed);
}

__global__ void __launch_bounds__(kPlanThreads) pa_free_shared_large_kernel(const FreeSharedParams p) {
    pdl_trigger();
    pdl_wait();
    __shared__ int s_warp[32];
    __shared__ int s_nblk[kPlanThreads], s_slot[kPlanThreads];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int height = stack_height(p.stack, p.num_blocks, p.status);
    auto good = [&](int id) { return id >= 0 && id < p.num_blocks; };
    int pushed = 0;
    for (int pass = 0; pass < 2; ++pass) {
        for (int at = 0; at < p.batch; at += kPlanThreads) {
            s_nblk[threadIdx.x] = free_row_blocks(p, at + threadIdx.x, pass == 0);
            __syncthreads();
            const int here = min(kPlanThreads, p.batch - at);
            for (int k = warp; k < here; k += kPlanThreads / 32) {
                const int* row = p.bt + (long long)(at + k) * p.maxb;
                for (int j = lane; j < s_nblk[k]; j += 32) {
                    const int id = row[j];
                    if (!good(id)) {
                        if (pass == 0) atomicOr(p.status, kStatusBadBlock);
                    } else if (pass == 0) {
                        atomicSub(p.shares + id, 1);
                    } else if (__ldcg(p.shares + id) < 0) {
                        atomicMin(p.shares + id, free_bid((long long)(at + k) * p.maxb + j));
                    }
                }
            }
            __syncthreads();
        }
        __threadfence();
        __syncthreads();
    }
    for (int at = 0; at < p.batch; at += kPlanThreads) {
        s_nblk[threadIdx.x] = free_row_blocks(p, at + threadIdx.x, false);
        s_slot[threadIdx.x] = 0;
        __syncthreads();
        const int here = min(kPlanThreads, p.batch - at);
        for (int k = warp; k < here; k += kPlanThreads / 32) {
            const int* row = p.bt + (long long)(at + k) * p.maxb;
            int mine = 0;
            for (int j = lane; j < s_nblk[k]; j += 32) {
                const int id = row[j];
                mine += good(id) && __ldcg(p.shares + id) == free_bid((long long)(at + k) * p.maxb + j);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(kFullMask, mine, o);
            if (lane == 0) s_slot[k] = mine;
        }
        __syncthreads();
        int total = 0;
        const int slot0 = cta_exclusive_scan(s_slot[threadIdx.x], s_warp, total);
        s_slot[threadIdx.x] = height + pushed + slot0;
        pushed += total;
        __syncthreads();
        for (int k = warp; k < here; k += kPlanThreads / 32) {
            int* row = p.bt + (long long)(at + k) * p.maxb;
            int slot = s_slot[k];
            for (int j0 = 0; j0 < s_nblk[k]; j0 += 32) {
                const int j = j0 + lane;
                int id = -1;
                if (j < s_nblk[k]) {
                    id = row[j];
                    row[j] = -1;
                }
                const bool win =
                    good(id) && __ldcg(p.shares + id) == free_bid((long long)(at + k) * p.maxb + j);
                const unsigned wins = __ballot_sync(kFullMask, win);
                if (win) free_push(p, slot + __popc(wins & ((1u << lane) - 1u)), id);
                slot += __popc(wins);
            }
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) free_height(p, height, pushed);
}

// ------------------------------------------------------------------ compact

// With `live` pages in use, the i-th smallest live id >= live moves to the
// i-th smallest free id < live.  Every CTA builds the bitmap of the free ids
// and its running counts in shared memory (the same in each, from the stack),
// then writes its share of the results: no CTA waits for another.
struct FreeMap {
    const unsigned* bits;   // 1 = free
    const int* before;      // free ids in the words before
    int nb, words, live;
    __device__ __forceinline__ bool free(int id) const { return (bits[id >> 5] >> (id & 31)) & 1u; }
    __device__ __forceinline__ int free_before(int id) const {
        return before[id >> 5] + __popc(bits[id >> 5] & ((1u << (id & 31)) - 1u));
    }
    // the r-th free id
    __device__ __forceinline__ int nth_free(int r) const {
        int lo = 0, hi = words - 1;  // the last word with before <= r
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (before[mid] <= r) lo = mid; else hi = mid - 1;
        }
        return lo * 32 + nth_bit(bits[lo], r - before[lo]);
    }
    // the r-th live id
    __device__ __forceinline__ int nth_live(int r) const {
        int lo = 0, hi = words - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (mid * 32 - before[mid] <= r) lo = mid; else hi = mid - 1;
        }
        return lo * 32 + nth_bit(~bits[lo], r - (lo * 32 - before[lo]));
    }
    static __device__ __forceinline__ int nth_bit(unsigned w, int r) {
        for (; r > 0; --r) w &= w - 1u;
        return __ffs(w) - 1;
    }
    // where live page id ends up
    __device__ __forceinline__ int place(int id) const {
        if (id < live) return id;
        const int live_before_id = id - free_before(id);
        // live ids in [0, live): live - holes; holes = free ids below live
        const int holes = free_before(live);
        return nth_free(live_before_id - (live - holes));
    }
};

__global__ void __launch_bounds__(kPlanThreads) pa_compact_plan_kernel(const CompactParams p) {
    pdl_trigger();
    pdl_wait();
    extern __shared__ unsigned s_mem[];
    __shared__ int s_warp[32];
    const int nb = (int)p.g.num_blocks;
    const int words = nb / 32 + 1;  // (one more than the ids need: `live` may be nb)
    unsigned* bits = s_mem;
    int* before = reinterpret_cast<int*>(s_mem + words);
    for (int i = threadIdx.x; i < words; i += kPlanThreads) bits[i] = 0u;
    __syncthreads();
    const int height = stack_height(p.stack, nb, p.g.status);
    for (int i = threadIdx.x; i < height; i += kPlanThreads) {
        const int id = ld_dep(p.stack + 1 + i);
        if (id < 0 || id >= nb) {
            if (blockIdx.x == 0) atomicOr(p.g.status, kStatusBadBlock);
        } else {
            atomicOr(bits + (id >> 5), 1u << (id & 31));
        }
    }
    __syncthreads();
    int done = 0;
    for (int at = 0; at < words; at += kPlanThreads) {
        const int i = at + threadIdx.x;
        int total = 0;
        const int r = cta_exclusive_scan(i < words ? __popc(bits[i]) : 0, s_warp, total);
        if (i < words) before[i] = done + r;
        done += total;
    }
    __syncthreads();
    FreeMap m{bits, before, nb, words, nb - done};
    const int free_count = done;
    const int step = gridDim.x * kPlanThreads;
    const int me = blockIdx.x * kPlanThreads + threadIdx.x;
    // pages: where each goes, the list of moves, the shares by new id, the stack
    const int stay = m.live - m.free_before(m.live);  // live ids that keep their place
    for (int id = me; id < nb; id += step) {
        const bool live = !m.free(id);
        const int to = live ? m.place(id) : -1;
        p.remap[id] = to;
        if (live && to != id) {
            const int r = id - m.free_before(id) - stay;
            p.move_src[r] = id, p.move_dst[r] = to;
        }
        if (p.shares != nullptr) {
            int from = -1;  // the page that ends up at id
            if (id < m.live) from = live ? id : m.nth_live(stay + m.free_before(id));
            p.out_shares[id] = from >= 0 ? ld_dep(p.shares + from) : 0;
        }
        p.out_stack[1 + id] = id < free_count ? nb - 1 - id : -1;
    }
    if (me == 0) {
        p.out_stack[0] = free_count;
        *p.move_count = m.live - stay;
    }
    // tables
    const long long entries = (long long)p.batch * p.maxb;
    for (long long x = me; x < entries; x += step) {
        const int b = (int)(x / p.maxb), j = (int)(x % p.maxb);
        const int n = ld_dep(p.lens + b);
        int e = ld_dep(p.bt + x);
        if (n < 0 || n > p.maxb * p.g.B) {
            if (j == 0) atomicOr(p.g.status, kStatusBadLength);
        } else if (j < (n + p.g.B - 1) / p.g.B) {
            if (e < 0 || e >= nb || m.free(e)) {
                atomicOr(p.g.status, kStatusBadBlock);
                e = -1;
            } else {
                e = m.place(e);
            }
        }
        p.out_bt[x] = e;
    }
}

int copy_grid(long long tiles, int num_sms) {
    const long long blocks = (tiles + kCopyThreads / 32 - 1) / (kCopyThreads / 32);
    const long long cap = (long long)num_sms * 8;
    return (int)(blocks < cap ? blocks : cap);
}

}  // namespace

cudaError_t launch_copy_blocks(const PageGeom& g, const int* src, const int* dst, int n,
                               int num_sms, cudaStream_t s) {
    if (n <= 0) return cudaSuccess;
    return launch_pdl(pa_copy_blocks_kernel, dim3(copy_grid(2LL * g.L * g.Hkv * n, num_sms)),
                      dim3(kCopyThreads), 0, s, g, src, dst, (const int*)nullptr, n);
}

cudaError_t launch_fork(const ForkParams& p, int num_sms, cudaStream_t s) {
    if (p.n <= 0) return cudaSuccess;
    // CTAs per child: enough to fill the GPU with few children, no more than a
    // page has tiles for
    const long long tiles = 2LL * p.g.L * p.g.Hkv;
    long long parts = (8LL * num_sms + p.n - 1) / p.n;
    const long long most = (tiles + kCopyThreads / 32 - 1) / (kCopyThreads / 32);
    if (parts > most) parts = most;
    if (parts > 65535) parts = 65535;
    cudaError_t e = launch_pdl(pa_fork_kernel, dim3((unsigned)p.n, (unsigned)parts),
                               dim3(kCopyThreads), 0, s, p);
    if (e != cudaSuccess) return e;
    return launch_pdl(pa_fork_height_kernel, dim3(1), dim3(kCopyThreads), 0, s, p);
}

cudaError_t launch_free_shared(const FreeSharedParams& p, cudaStream_t s) {
    if (p.batch <= 0) return cudaSuccess;
    const long long entries = (long long)p.batch * p.maxb;
    if (p.batch > kFreeRows || entries > kFreeEntries)
        return launch_pdl(pa_free_shared_large_kernel, dim3(1), dim3(kPlanThreads), 0, s, p);
    // (a cluster's barriers cost about 1 us more than a CTA's: 24 finished rows of
    // a 32-row table with 1,664 entries take 5.7 us in one CTA and 6.7 in eight)
    const int ctas = entries <= 4096 ? 1 : kFreeCluster;
    const long long ids = (entries + ctas - 1) / ctas;
    const size_t smem = (size_t)(p.batch + 1 + ids) * sizeof(int);
    // (always, and the same for all calls: the kernel's static shared memory counts toward the
    // 48 KiB that go without it, and the limit is the function's, not the call's)
    const cudaError_t e = cudaFuncSetAttribute(
        pa_free_shared_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
        (kFreeRows + 1 + kFreeEntries / kFreeCluster) * (int)sizeof(int));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, pa_free_shared_kernel, p);
}

constexpr size_t compact_smem_bytes(long long num_blocks) {
    return (size_t)(num_blocks / 32 + 1) * 8;
}
static_assert(compact_smem_bytes(kCompactMaxBlocks) + 1024 <= 232448, "shared memory");

cudaError_t launch_compact(const CompactParams& p, int num_sms, cudaStream_t s) {
    const long long nb = p.g.num_blocks;
    const size_t smem = compact_smem_bytes(nb);
    // (the same for all calls: the limit is the function's, and another thread's call with a
    // smaller pool may come between this one's limit and its launch)
    cudaError_t e = cudaFuncSetAttribute(pa_compact_plan_kernel,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)compact_smem_bytes(kCompactMaxBlocks));
    if (e != cudaSuccess) return e;
    const long long items = nb > (long long)p.batch * p.maxb ? nb : (long long)p.batch * p.maxb;
    long long grid = (items + kPlanThreads - 1) / kPlanThreads;
    if (grid > num_sms) grid = num_sms;
    e = launch_pdl(pa_compact_plan_kernel, dim3((unsigned)grid), dim3(kPlanThreads), smem, s, p);
    if (e != cudaSuccess) return e;
    // the moves are counted on the device: at most half the pages
    return launch_pdl(pa_copy_blocks_kernel, dim3(copy_grid(2LL * p.g.L * p.g.Hkv * ((nb + 1) / 2), num_sms)),
                      dim3(kCopyThreads), 0, s, p.g, (const int*)p.move_src,
                      (const int*)p.move_dst, (const int*)p.move_count, 0);
}

}  // namespace pa
