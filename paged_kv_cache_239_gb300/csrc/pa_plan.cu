// pa_plan.cu -- a batch's new tokens planned on the device: the pages they need, where each
// goes and stands, what each node of a drafted tree sees; and pages given back.
//
// Sequence b holds c_b tokens and gets n_b.  With first_b = ceil(c_b / B) it takes the pages of
// blocks first_b .. ceil((c_b + n_b) / B) - 1 from the stack's top, all sequences in increasing
// order, so the rank of block j is base_b + j - first_b with base the prefix sums of the counts,
// and the rank alone names the stack's entry: no page waits for another.  Token i of sequence b
// is token starts_b + i of the batch (starts: the prefix sums of n) at slot
// page((c_b + i) / B) * B + (c_b + i) % B.
//
// Every CTA of the cluster scans the sequences by itself (a thread each), so that no CTA waits for
// another but for the stack's height, which is read before it is written; then the tokens are dealt
// out: a binary search in the starts names the sequence, and four tokens of a thread have their
// pages on their way at once.  What bounds it is never the bytes (256 trees of 64 nodes: 0.05 us):
// small batches wait for a launch and four dependent loads, 2 to 3 us each of plan and trim; many
// tokens keep the one cluster's eight SMs at work, of whose cycles 53 % issue (256 trees of up to
// 64), with searches, the ancestors' walks and scattered stores.  On the device, plan / trim: 8
// trees of 8 nodes 3.1 / 2.5 us, 256 trees of up to 64 7.7 / 3.4, 16 prompts of 500 to 4,096 tokens
// 7.2 / 4.8; both together 5.3, 11.1 and 12.0 (7.0, 11.9 and 13.5 with one token on its way, a scan
// each for pages and tokens, and the height read first).
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_stack.cuh"

namespace pa {

namespace {

namespace cg = cooperative_groups;

constexpr int kPlanThreads = 1024;
constexpr int kPlanCluster = 8;

// Exclusive prefix sums of two values over the CTA, and their totals.  (Within 32 sequences a
// warp knows by itself; the others need not wait for one another.)
struct Two {
    long long a;
    int b;
};
__device__ __forceinline__ Two warp_inclusive(Two v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long a = __shfl_up_sync(kFullMask, v.a, o);
        const int b = __shfl_up_sync(kFullMask, v.b, o);
        if (lane >= o) v.a += a, v.b += b;
    }
    return v;
}
__device__ __forceinline__ Two cta_exclusive_scan2(Two v, long long* s_a, int* s_b, Two& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const Two incl = warp_inclusive(v, lane);
    if (lane == 31) s_a[warp] = incl.a, s_b[warp] = incl.b;
    __syncthreads();
    // (every warp sums the warps' totals by itself)
    const Two sums = warp_inclusive(lane < warps ? Two{s_a[lane], s_b[lane]} : Two{0, 0}, lane);
    total = Two{__shfl_sync(kFullMask, sums.a, warps - 1), __shfl_sync(kFullMask, sums.b, warps - 1)};
    const long long a = __shfl_sync(kFullMask, sums.a, (warp + 31) & 31);
    const int b = __shfl_sync(kFullMask, sums.b, (warp + 31) & 31);
    return Two{(warp ? a : 0) + incl.a - v.a, (warp ? b : 0) + incl.b - v.b};
}

__device__ __forceinline__ int blocks_of(int tokens, int B) { return tokens / B + (tokens % B != 0); }

// The last x in [0, n) with at[x] <= v (at[0] <= v, increasing).
__device__ __forceinline__ int last_not_above(const int* at, int n, int v) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (at[mid] <= v) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// Depth of a node below its root and, word by word from the last, the bits of its ancestors and
// itself (parents come before their children); up: the sequence's parents, or null (a chain).
// Every step waits for the one before it, by loads that L1 answers (a chain of 1,024 nodes takes
// 58 us, 64 chains of 256 44; with the parents brought to shared memory 90 and 62).
__device__ __forceinline__ int plan_ancestors(const PlanParams& p, const int* up, int node, long long row) {
    int depth = -1;
    bool bad = false;
    for (int w = p.masks != nullptr ? p.words - 1 : 0; w >= 0; --w) {
        unsigned bits = 0;
        while (node >= 32 * w) {
            bits |= 1u << (node & 31);
            ++depth;
            int q = node - 1;
            if (up != nullptr) {
                q = ld_dep(up + node);
                const bool below = (unsigned)(q + 1) <= (unsigned)node;  // -1 .. node - 1
                bad |= !below;
                q = below ? q : -1;
            }
            node = q;
        }
        if (p.masks != nullptr) p.masks[row * p.words + w] = bits;
    }
    if (bad) atomicOr(p.status, kStatusBadLength);
    return depth;
}

__global__ void __launch_bounds__(kPlanThreads) pa_plan_kernel(const PlanParams p) {
    pdl_trigger();
    pdl_wait();
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
    __shared__ int s_start[kPlanThreads], s_base[kPlanThreads], s_cached[kPlanThreads];
    __shared__ int s_warp[32];
    __shared__ long long s_warp64[32];
    const int tid = threadIdx.x, threads = blockDim.x;
    const int step = ctas * threads, me = rank * threads + tid;
    int c0 = 0, n0 = 0;        // (on their way before the height is looked at)
    if (tid < p.batch) c0 = ld_dep(p.cached + tid), n0 = ld_dep(p.counts + tid);
    const int height = stack_height(p.stack, p.num_blocks, p.status);
    cluster.barrier_arrive();  // (this CTA has read the height)
    long long asked = 0;       // tokens of the sequences before, as asked for
    int given = 0, taken = 0;  // and as planned; pages taken
    for (int b0 = 0; b0 < p.batch; b0 += threads) {
        const int b = b0 + tid, here = min(threads, p.batch - b0);
        int c = 0, n = 0;
        bool bad = false;
        if (b < p.batch) {
            c = b0 ? ld_dep(p.cached + b) : c0, n = b0 ? ld_dep(p.counts + b) : n0;
            if (c < 0 || c > p.maxb * p.B) bad = true, c = n = 0;
            if (n < 0 || n > p.maxb * p.B - c || (p.masks != nullptr && n > 32 * p.words)) bad = true, n = 0;
        }
        const int first = blocks_of(c, p.B);
        Two sum;
        Two at = cta_exclusive_scan2(Two{n, blocks_of(c + n, p.B) - first}, s_warp64, s_warp, sum);
        if (asked + sum.a > p.num_tokens) {  // the first that does not fit, and all after it, get none
            if (n > 0 && asked + at.a + n > p.num_tokens) bad = true, n = 0;
            asked += sum.a;
            __syncthreads();
            at = cta_exclusive_scan2(Two{n, blocks_of(c + n, p.B) - first}, s_warp64, s_warp, sum);
        } else {
            asked += sum.a;
        }
        if (bad && rank == 0) atomicOr(p.status, kStatusBadLength);
        const int start = given + (int)at.a, tokens = (int)sum.a;
        if (b < p.batch) {
            s_start[tid] = start, s_base[tid] = taken + at.b - first, s_cached[tid] = c;
            if (rank == 0) p.lens[b] = c + n, p.starts[b] = start;
        }
        __syncthreads();
        constexpr int U = 4;  // tokens whose pages are on their way at once
        for (int t0 = given + me; t0 < given + tokens; t0 += U * step) {
            int seq[U], id[U], row[U], kind[U];
            int* entry[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int t = t0 + u * step;
                kind[u] = -1;
                if (t >= given + tokens) continue;
                const int x = seq[u] = last_not_above(s_start, here, t);
                const int pos = s_cached[x] + t - s_start[x], j = pos / p.B;
                row[u] = pos - j * p.B;
                entry[u] = p.bt + (long long)(b0 + x) * p.maxb + j;
                // the cached tokens' last page, or the rank-th from the stack's top
                const int r = s_base[x] + j;
                kind[u] = j * p.B < s_cached[x] ? 0 : r < height ? 1 : 2;
                id[u] = kind[u] == 2 ? -1 : ld_dep(kind[u] ? p.stack + height - r : entry[u]);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int t = t0 + u * step;
                if (kind[u] < 0) continue;
                const int x = seq[u], i = t - s_start[x];
                const int depth = p.parents == nullptr && p.masks == nullptr
                                      ? i
                                      : plan_ancestors(p, p.parents ? p.parents + s_start[x] : nullptr, i, t);
                p.positions[t] = s_cached[x] + depth;
                if (id[u] < 0 || id[u] >= p.num_blocks) {
                    atomicOr(p.status, kind[u] == 2 ? kStatusNoFreeBlocks : kStatusBadBlock);
                    id[u] = -1;
                }
                if (kind[u] && row[u] == 0) *entry[u] = id[u];
                p.slots[t] = id[u] < 0 ? -1 : (long long)id[u] * p.B + row[u];
            }
        }
        given += tokens, taken += sum.b;
        __syncthreads();  // (before the places are written again)
    }
    // rows behind the last sequence
    for (int t = given + me; t < p.num_tokens; t += step) {
        p.slots[t] = -1;
        p.positions[t] = 0;
        if (p.masks != nullptr)
            for (int w = 0; w < p.words; ++w) p.masks[(long long)t * p.words + w] = 0;
    }
    cluster.barrier_wait();    // (all have)
    if (rank == 0 && tid == 0) {
        p.starts[p.batch] = given;
        p.stack[0] = taken < height ? height - taken : 0;
    }
}

// Pages of blocks ceil(m / B) .. ceil(n / B) - 1 of every sequence go back, the last block of
// the last sequence first: the reverse of the order they are taken in, so a plan that is
// trimmed back leaves the stack as it was.
__global__ void __launch_bounds__(kPlanThreads) pa_trim_kernel(const TrimParams p) {
    pdl_trigger();
    pdl_wait();
    __shared__ int s_start[kPlanThreads], s_last[kPlanThreads];
    __shared__ int s_warp[32];
    __shared__ long long s_warp64[32];
    const int tid = threadIdx.x, threads = blockDim.x;
    int n0 = 0, m0 = 0;        // (on their way before the height is looked at)
    if (tid < p.batch) n0 = ld_dep(p.lens + p.batch - 1 - tid), m0 = ld_dep(p.new_lens + p.batch - 1 - tid);
    const int height = stack_height(p.stack, p.num_blocks, p.status);
    int pushed = 0;
    for (int x0 = 0; x0 < p.batch; x0 += threads) {
        const int b = p.batch - 1 - (x0 + tid), here = min(threads, p.batch - x0);
        int count = 0, last = 0;
        if (b >= 0) {
            const int n = x0 ? ld_dep(p.lens + b) : n0, m = x0 ? ld_dep(p.new_lens + b) : m0;
            if (n < 0 || n > p.maxb * p.B || m < 0 || m > n) {
                atomicOr(p.status, kStatusBadLength);
            } else {
                last = blocks_of(n, p.B);
                count = last - blocks_of(m, p.B);
            }
        }
        Two sum;
        s_start[tid] = cta_exclusive_scan2(Two{0, count}, s_warp64, s_warp, sum).b;
        s_last[tid] = last - 1;
        const int total = sum.b;
        __syncthreads();
        constexpr int U = 4;  // entries of a thread on their way at once
        for (int e0 = 0; e0 < total; e0 += U * threads) {
            int id[U];
            bool odd = false;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int e = e0 + u * threads + tid;
                id[u] = -1;
                if (e >= total) continue;
                const int x = last_not_above(s_start, here, e);
                int* entry = p.bt + (long long)(p.batch - 1 - (x0 + x)) * p.maxb + s_last[x] - (e - s_start[x]);
                id[u] = ld_dep(entry);
                *entry = -1;
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (e0 + u * threads + tid < total && (id[u] < 0 || id[u] >= p.num_blocks)) odd = true, id[u] = -1;
            if (odd) atomicOr(p.status, kStatusBadBlock);
            // (a place for every entry, unless one is no page)
            odd = __syncthreads_or(odd);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                int slot = height + pushed + tid, ids = min(threads, max(total - e0 - u * threads, 0));
                if (odd) {
                    slot = height + pushed + cta_exclusive_scan2(Two{0, id[u] >= 0}, s_warp64, s_warp, sum).b;
                    ids = sum.b;
                    __syncthreads();
                }
                if (id[u] >= 0) {
                    if (slot < p.num_blocks)
                        p.stack[1 + slot] = id[u];
                    else
                        atomicOr(p.status, kStatusBadBlock);  // more ids than the pool holds
                }
                pushed += ids;
            }
        }
        __syncthreads();
    }
    if (tid == 0) {
        const long long h = (long long)height + pushed;
        p.stack[0] = (int)(h < p.num_blocks ? h : p.num_blocks);
    }
}

}  // namespace

cudaError_t launch_plan(const PlanParams& p, cudaStream_t s) {
    // a thread per token and per sequence, in CTAs of 128 to 1024
    const int items = p.num_tokens > p.batch ? p.num_tokens : p.batch;
    int threads = 128, ctas = 1;
    while (threads < kPlanThreads && threads < p.batch) threads *= 2;
    while (threads < kPlanThreads && (long long)threads * kPlanCluster < items) threads *= 2;
    while (ctas < kPlanCluster && (long long)ctas * threads < items) ctas *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(threads);
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
    return cudaLaunchKernelEx(&cfg, pa_plan_kernel, p);
}

cudaError_t launch_trim(const TrimParams& p, cudaStream_t s) {
    if (p.batch <= 0) return cudaSuccess;
    // (four entries to a thread; more threads wait longer for one another)
    const int threads = p.batch <= 512 ? 512 : kPlanThreads;
    return launch_pdl(pa_trim_kernel, dim3(1), dim3(threads), 0, s, p);
}

}  // namespace pa
