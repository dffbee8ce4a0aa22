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
// What bounds it: latency.  Every CTA of the cluster scans the sequences by itself (a thread each,
// 1024 at a time), then the tokens are dealt out, a thread each: a binary search in the starts
// names the sequence.
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

__device__ __forceinline__ long long cta_exclusive_scan64(long long v, long long* s_warp, long long& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long t = __shfl_up_sync(kFullMask, incl, o);
        if (lane >= o) incl += t;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        long long w = lane < (blockDim.x >> 5) ? s_warp[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long t = __shfl_up_sync(kFullMask, w, o);
            if (lane >= o) w += t;
        }
        s_warp[lane] = w;
    }
    __syncthreads();
    const long long before = warp > 0 ? s_warp[warp - 1] : 0;
    total = s_warp[(blockDim.x >> 5) - 1];
    __syncthreads();
    return before + incl - v;
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

__global__ void __launch_bounds__(kPlanThreads) pa_plan_kernel(const PlanParams p) {
    pdl_trigger();
    pdl_wait();
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
    __shared__ int s_start[kPlanThreads + 1], s_base[kPlanThreads], s_cached[kPlanThreads];
    __shared__ int s_warp[32];
    __shared__ long long s_warp64[32];
    const int tid = threadIdx.x;
    const int height = stack_height(p.stack, p.num_blocks, p.status);
    long long asked = 0;       // tokens of the sequences before, as asked for
    int given = 0, taken = 0;  // and as planned; pages taken
    for (int b0 = 0; b0 < p.batch; b0 += kPlanThreads) {
        const int b = b0 + tid, here = min(kPlanThreads, p.batch - b0);
        int c = 0, n = 0;
        bool bad = false;
        if (b < p.batch) {
            c = ld_dep(p.cached + b), n = ld_dep(p.counts + b);
            if (c < 0 || c > p.maxb * p.B) bad = true, c = n = 0;
            if (n < 0 || n > p.maxb * p.B - c || (p.masks != nullptr && n > 32 * p.words)) bad = true, n = 0;
        }
        long long sum;
        const long long before = asked + cta_exclusive_scan64(n, s_warp64, sum);
        asked += sum;
        if (n > 0 && before + n > p.num_tokens) bad = true, n = 0;  // (and all after it)
        if (bad && rank == 0) atomicOr(p.status, kStatusBadLength);
        int tokens, pages;
        const int start = given + cta_exclusive_scan(n, s_warp, tokens);
        const int first = blocks_of(c, p.B);
        const int base = taken + cta_exclusive_scan(blocks_of(c + n, p.B) - first, s_warp, pages);
        if (b < p.batch) {
            s_start[tid] = start, s_base[tid] = base - first, s_cached[tid] = c;
            if (rank == 0) p.lens[b] = c + n, p.starts[b] = start;
        }
        __syncthreads();
        for (int t = given + rank * kPlanThreads + tid; t < given + tokens; t += ctas * kPlanThreads) {
            const int x = last_not_above(s_start, here, t);
            const int i = t - s_start[x], at = s_cached[x] + i, j = at / p.B, row = at - j * p.B;
            const int r = s_base[x] + j;  // the page's rank, if it is new
            int* entry = p.bt + (long long)(b0 + x) * p.maxb + j;
            int id = -1;
            if (j * p.B < s_cached[x]) {  // the cached tokens' last page
                id = ld_dep(entry);
                if (id < 0 || id >= p.num_blocks) id = -1, atomicOr(p.status, kStatusBadBlock);
            } else {
                if (r < height) {
                    id = ld_dep(p.stack + height - r);
                    if (id < 0 || id >= p.num_blocks) id = -1, atomicOr(p.status, kStatusBadBlock);
                } else {
                    atomicOr(p.status, kStatusNoFreeBlocks);
                }
                if (row == 0) *entry = id;
            }
            p.slots[t] = id < 0 ? -1 : (long long)id * p.B + row;
            int depth = i;
            if (p.parents != nullptr || p.masks != nullptr) {
                // up to the root: its bits by words from the last, since parents come first
                const int* up = p.parents != nullptr ? p.parents + s_start[x] : nullptr;
                int node = i;
                depth = -1;
                for (int w = p.masks != nullptr ? p.words - 1 : 0; w >= 0; --w) {
                    unsigned bits = 0;
                    while (node >= 32 * w) {
                        bits |= 1u << (node & 31);
                        ++depth;
                        int q = node - 1;
                        if (up != nullptr) {
                            q = ld_dep(up + node);
                            if (q < -1 || q >= node) q = -1, atomicOr(p.status, kStatusBadLength);
                        }
                        node = q;
                        if (node < 0) break;
                    }
                    if (p.masks != nullptr) p.masks[(long long)t * p.words + w] = bits;
                }
            }
            p.positions[t] = s_cached[x] + depth;
        }
        given += tokens, taken += pages;
        __syncthreads();  // (before the places are written again)
    }
    // rows behind the last sequence
    for (int t = given + rank * kPlanThreads + tid; t < p.num_tokens; t += ctas * kPlanThreads) {
        p.slots[t] = -1;
        p.positions[t] = 0;
        if (p.masks != nullptr)
            for (int w = 0; w < p.words; ++w) p.masks[(long long)t * p.words + w] = 0;
    }
    cluster.sync();  // (all have read the height)
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
    const int tid = threadIdx.x;
    const int height = stack_height(p.stack, p.num_blocks, p.status);
    int pushed = 0;
    for (int x0 = 0; x0 < p.batch; x0 += kPlanThreads) {
        const int b = p.batch - 1 - (x0 + tid), here = min(kPlanThreads, p.batch - x0);
        int count = 0, last = 0;
        if (b >= 0) {
            const int n = ld_dep(p.lens + b), m = ld_dep(p.new_lens + b);
            if (n < 0 || n > p.maxb * p.B || m < 0 || m > n) {
                atomicOr(p.status, kStatusBadLength);
            } else {
                last = blocks_of(n, p.B);
                count = last - blocks_of(m, p.B);
            }
        }
        int total;
        s_start[tid] = cta_exclusive_scan(count, s_warp, total);
        s_last[tid] = last - 1;
        __syncthreads();
        for (int e0 = 0; e0 < total; e0 += kPlanThreads) {
            const int e = e0 + tid;
            int id = -1;
            if (e < total) {
                const int x = last_not_above(s_start, here, e);
                int* entry = p.bt + (long long)(p.batch - 1 - (x0 + x)) * p.maxb + s_last[x] - (e - s_start[x]);
                id = ld_dep(entry);
                *entry = -1;
                if (id < 0 || id >= p.num_blocks) id = -1, atomicOr(p.status, kStatusBadBlock);
            }
            int ids;
            const int slot = height + pushed + cta_exclusive_scan(id >= 0, s_warp, ids);
            if (id >= 0) {
                if (slot < p.num_blocks)
                    p.stack[1 + slot] = id;
                else
                    atomicOr(p.status, kStatusBadBlock);  // more ids than the pool holds
            }
            pushed += ids;
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
    const int want = (p.num_tokens + kPlanThreads - 1) / kPlanThreads;
    const int ctas = want < 1 ? 1 : want < kPlanCluster ? want : kPlanCluster;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kPlanThreads);
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
    return launch_pdl(pa_trim_kernel, dim3(1), dim3(kPlanThreads), 0, s, p);
}

}  // namespace pa
