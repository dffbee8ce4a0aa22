// pa_tree_mask.cuh -- the masks of drafted trees: token i of a sequence's new ones sees all
// cached tokens and the new tokens j whose bits are set in its mask (bit j % 32 of word
// j / 32), so a tree's branches stand side by side in the cache and do not see one another.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

// Bit k: whether a row sees key j + k, keys counted from the first new token (those before
// it are cached and seen; those past the last of n_new are not there).
__device__ __forceinline__ uint32_t tree_bits(const unsigned* mask, int words, int j, int n_new) {
    const int w = j >> 5;
    auto word = [&](int x) { return x < 0 ? 0xffffffffu : x < words ? ld_dep(mask + x) : 0u; };
    const uint32_t v = (j & 31) ? __funnelshift_r(word(w), word(w + 1), j & 31) : word(w);
    const int left = n_new - j;
    return left >= 32 ? v : left <= 0 ? 0u : v & ((1u << left) - 1u);
}

// The same for keys j .. j + 127, out of line: a tile that reaches the new tokens is rare.
static __device__ __noinline__ uint4 tree_bits128(const unsigned* mask, int words, int j, int n_new) {
    return make_uint4(tree_bits(mask, words, j, n_new), tree_bits(mask, words, j + 32, n_new),
                      tree_bits(mask, words, j + 64, n_new), tree_bits(mask, words, j + 96, n_new));
}

// A row's mask on its way to L1, long before its tile comes.
__device__ __forceinline__ void tree_prefetch(const unsigned* mask) {
    asm volatile("prefetch.global.L1 [%0];" ::"l"(mask));
}

// Adds the values that are not finite of the new tokens that a row sees, among keys [lo, hi),
// to its columns c0, c0 + step, ... < c1: add(column, value).  For rows whose products took
// them as zeros.  v_rows: the pool's V of the layer and KV head; table: the sequence's
// row.  Out of line, all arguments by value: it is rare, and nothing of the caller's shall
// live in memory for it.
template <class T, int D, class Add>
__device__ __noinline__ void tree_odd_values(const T* v_rows, long long s_blk, long long num_blocks,
                                             const int* table, const unsigned* mask, int first_pos,
                                             int n_new, int B, int lo, int hi, int c0, int step, int c1,
                                             Add add) {
    for (int j = max(lo - first_pos, 0); j < min(hi - first_pos, n_new); ++j) {
        if (!(ld_dep(mask + (j >> 5)) >> (j & 31) & 1u)) continue;
        const int key = first_pos + j;
        const int blk = ld_dep(table + key / B);
        if (blk < 0 || blk >= num_blocks) continue;
        const T* row = v_rows + (long long)blk * s_blk + key % B * D;
        for (int c = c0; c < c1; c += step) {
            const float v = static_cast<float>(ld_dep(row + c));
            if (!isfinite(v)) add(c, v);
        }
    }
}

}  // namespace pa
