// pa_accept.cu -- drafted trees decided: the path from the root along the nodes that the model chose
// itself, and the K and V of its tokens moved up behind the cached ones.
//
// A node is accepted where its parent is and its token is the model's choice after the parent
// (the lowest such node where there are several, whose path need not be the longest).  Every node bids for its parent's link with an
// atomic minimum in shared memory, so the link does not depend on the threads' timing; the path is
// then one thread's walk from the root.
//
// The k-th node of the path, p_k, moves from its slot to that of node k.  The path increases,
// so p_k >= k, and a destination k is no source of a later move (p_j >= j > k): a thread that
// takes its 16 bytes of the rows in increasing k, all loads of a group before its stores, needs
// no other order.  The threads deal out the 16-byte columns of a token's K and V in all layers
// among themselves, several CTAs to a sequence, each of which walks by itself.
//
// What bounds it: for small batches the chain of dependent loads (starts, the tree, rows): 8 trees
// of 8 nodes 3.1 us on the device.  64 trees of 64 nodes whose paths move 26 MB in and out: 8.1 us
// against 3.9 for the bytes alone; before the first row moves there are the launch, the dependent loads and the
// walk by one thread.  (Four rows in flight and up to eight CTAs per SM: eight and 16 rows, or 1
// to 32 CTAs, were no faster.)
#include <cuda_runtime.h>
#include <stdint.h>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

constexpr int kAcceptThreads = 256;

__global__ void __launch_bounds__(kAcceptThreads) pa_accept_kernel(const AcceptParams p) {
    pdl_trigger();
    pdl_wait();
    extern __shared__ long long s_moves[];  // [max_path] sources, destinations; then the path
    __shared__ int s_child[kMaxTreeNodes], s_target[kMaxTreeNodes];
    __shared__ long long s_slot[kMaxTreeNodes];
    __shared__ int s_count;
    long long *s_src = s_moves, *s_dst = s_moves + p.max_path;
    int* s_path = reinterpret_cast<int*>(s_moves + 2 * p.max_path);
    const int tid = threadIdx.x;
    const int b = blockIdx.x / p.parts, part = blockIdx.x % p.parts;
    const int start = ld_dep(p.starts + b), end = ld_dep(p.starts + b + 1), len = ld_dep(p.lens + b);
    const int n = end - start;
    const bool good = start >= 0 && end >= start && end <= p.num_tokens && n <= kMaxTreeNodes && n <= len;
    const int nodes = good ? n : 0;
    if (!good && part == 0 && tid == 0) atomicOr(p.g.status, kStatusBadLength);
    // (all of the tree in one round of loads)
    for (int i0 = 0; i0 < nodes; i0 += kAcceptThreads) {
        const int i = i0 + tid;
        int up = -1, token = 0;
        if (i < nodes) {
            up = ld_dep(p.parents + start + i), token = ld_dep(p.tokens + start + i);
            s_target[i] = ld_dep(p.targets + start + i);
            s_slot[i] = ld_dep(p.slots + start + i);
            s_child[i] = kMaxTreeNodes;
        }
        __syncthreads();
        if (i < nodes) {
            if (up < -1 || up >= i) {  // (node 0 is the root all the same)
                if (part == 0) atomicOr(p.g.status, kStatusBadLength);
            } else if (up >= 0 && token == s_target[up]) {
                atomicMin(s_child + up, i);
            }
        }
    }
    __syncthreads();
    if (tid == 0) {
        int k = 0;
        for (int at = 0; at < nodes && k < p.max_path; at = s_child[at]) s_path[k++] = at;
        s_count = k;
    }
    __syncthreads();
    const int count = s_count;
    if (part == 0) {
        for (int k = tid; k < p.max_path; k += kAcceptThreads)
            p.nodes[(long long)b * p.max_path + k] = k < count ? s_path[k] : -1;
        if (tid == 0) {
            p.counts[b] = count;
            p.next_tokens[b] = count > 0 ? s_target[s_path[count - 1]] : -1;
            p.next_lens[b] = good ? len - n + count : len;
        }
    }
    // the moves, as offsets in elements (-1: none)
    for (int k = tid; k < count; k += kAcceptThreads) {
        long long from = -1, to = -1;
        if (s_path[k] != k) {
            const long long a = s_slot[s_path[k]], z = s_slot[k];
            const long long most = p.g.num_blocks * p.g.B;
            if (a >= 0 && a < most && z >= 0 && z < most) {
                const int row = p.g.tile_bytes / p.g.B;
                from = a / p.g.B * p.g.s_blk * p.g.elt + a % p.g.B * row;
                to = z / p.g.B * p.g.s_blk * p.g.elt + z % p.g.B * row;
            } else if (part == 0) {
                atomicOr(p.g.status, kStatusBadBlock);
            }
        }
        s_src[k] = from, s_dst[k] = to;
    }
    __syncthreads();
    int k0 = 0;
    while (k0 < count && s_path[k0] == k0) ++k0;  // (no gap comes after one that closed up)
    if (k0 == count) return;
    const int chunks = p.g.tile_bytes / p.g.B / 16;  // of a row
    const int all = 2 * p.g.L * p.g.Hkv * chunks;
    for (int x = part * kAcceptThreads + tid; x < all; x += p.parts * kAcceptThreads) {
        int tile = x / chunks;
        const int c = x - tile * chunks;
        const int h = tile % p.g.Hkv;
        tile /= p.g.Hkv;
        const int layer = tile % p.g.L;
        unsigned char* base = static_cast<unsigned char*>(tile / p.g.L ? p.g.v_base : p.g.k_base) +
                              ((long long)layer * p.g.s_layer + (long long)h * p.g.s_head) * p.g.elt + 16 * c;
        constexpr int U = 4;
        for (int k = k0; k < count; k += U) {
            uint4 v[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (k + u < count && s_src[k + u] >= 0)
                    v[u] = ld_dep(reinterpret_cast<const uint4*>(base + s_src[k + u]));
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (k + u < count && s_src[k + u] >= 0) *reinterpret_cast<uint4*>(base + s_dst[k + u]) = v[u];
        }
    }
}

}  // namespace

cudaError_t launch_accept(const AcceptParams& p_in, int num_sms, cudaStream_t s) {
    AcceptParams p = p_in;
    if (p.batch <= 0) return cudaSuccess;
    // CTAs per sequence: enough to fill the GPU, no more than a token has 16-byte columns for
    const long long all = 2LL * p.g.L * p.g.Hkv * (p.g.tile_bytes / p.g.B / 16);
    long long parts = (8LL * num_sms + p.batch - 1) / p.batch;
    const long long most = (all + kAcceptThreads - 1) / kAcceptThreads;
    if (parts > most) parts = most;
    p.parts = (int)parts;
    const long long grid = parts * p.batch;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    return launch_pdl(pa_accept_kernel, dim3((unsigned)grid), dim3(kAcceptThreads),
                      (size_t)p.max_path * 20, s, p);
}

}  // namespace pa
