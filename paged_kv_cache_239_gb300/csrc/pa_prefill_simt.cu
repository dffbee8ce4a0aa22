// pa_prefill_simt.cu -- attention of several new tokens per sequence over the
// fp32 paged cache, on the CUDA cores.
//
//   out_t = sum_{s <= p_t} softmax_s(scale q_t . k_s) v_s,
//   p_t = context_lens[b] - n_b + i for the i-th of sequence b's n_b new tokens.
//
// The query heads of a KV head's group share its keys, so the rows of a tile
// are (token, head of the group) in that order, flattened: row r is token r / G,
// head r % G, and a tile takes BM consecutive rows whatever G is.  A CTA holds
// the tile's q in shared memory and streams 64 keys and values at a time; each
// thread accumulates 4 x 4 scores and 4 rows x D / 16 outputs in registers,
// with the running maximum and sum of each row (one pass over the keys).
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

constexpr int BM = 64, BN = 64, kThreads = 256;

template <int D>
struct SimtCfg {
    static constexpr int LD = D + 4;   // row stride of q, k and v (floats)
    static constexpr int LP = BN + 4;  // row stride of p
    static constexpr int SMEM = (3 * 64 * LD + BM * LP) * 4 + BN * 4;
};

__device__ __forceinline__ float4 load4(const float* p) {
    return ld_dep(reinterpret_cast<const float4*>(p));
}
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }

template <int D, int B>
__global__ void __launch_bounds__(kThreads) pa_prefill_simt_kernel(const PrefillParams p) {
    pdl_trigger();
    pdl_wait();
    using C = SimtCfg<D>;
    extern __shared__ float smem[];
    float* sq = smem;
    float* sk = sq + 64 * C::LD;
    float* sv = sk + 64 * C::LD;
    float* sp = sv + 64 * C::LD;
    int* slot = reinterpret_cast<int*>(sp + BM * C::LP);  // page of each key, -1: no weight
    __shared__ int s_at[2];
    const int tid = threadIdx.x, lane = tid & 31;

    // ---- the tile: sequence and first row of tile blockIdx.x ----
    if (tid < 32) {
        int left = blockIdx.x, found = -1, row0 = 0;
        for (int b0 = 0; b0 < p.batch && found < 0; b0 += 32) {
            const int b = b0 + lane;
            int tiles = 0;
            if (b < p.batch) {
                const int s0 = ld_dep(p.starts + b), s1 = ld_dep(p.starts + b + 1);
                const int n = ld_dep(p.lens + b);
                if (s0 < 0 || s1 < s0 || s1 > p.num_tokens || n < 0 || n > p.maxb * B) {
                    if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0)
                        atomicOr(p.status, kStatusBadLength);
                }
                if (s0 >= 0 && s1 > s0 && s1 <= p.num_tokens)
                    tiles = (int)(((long long)(s1 - s0) * p.G + BM - 1) / BM);
            }
            int incl = tiles;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(kFullMask, incl, o);
                if (lane >= o) incl += v;
            }
            const unsigned hit = __ballot_sync(kFullMask, left >= incl - tiles && left < incl);
            if (hit) {
                const int f = __ffs(hit) - 1;
                found = b0 + f;
                row0 = (left - (__shfl_sync(kFullMask, incl, f) - __shfl_sync(kFullMask, tiles, f))) * BM;
            }
            left -= __shfl_sync(kFullMask, incl, 31);
        }
        if (lane == 0) s_at[0] = found, s_at[1] = row0;
    }
    __syncthreads();
    const int b = s_at[0], row0 = s_at[1];
    if (b < 0) return;
    const int kvh = blockIdx.y;
    const int start = ld_dep(p.starts + b);
    const int n_new = ld_dep(p.starts + b + 1) - start;
    int n = ld_dep(p.lens + b);
    if (n < n_new || n > p.maxb * B) {
        if (tid == 0) atomicOr(p.status, kStatusBadLength);
        n = 0;
    }
    const int rows = (int)min((long long)BM, (long long)n_new * p.G - row0);
    const int first_pos = n - n_new;  // position of token 0
    // keys: [k0, k1) of the tile's [0, last visible + 1), by split
    const int see = n > 0 ? first_pos + (row0 + rows - 1) / p.G + 1 : 0;
    const int key_tiles = (see + BN - 1) / BN;
    const int per = (key_tiles + p.splits - 1) / p.splits;
    const int kt0 = min((int)blockIdx.z * per, key_tiles), kt1 = min(kt0 + per, key_tiles);

    const float* q = static_cast<const float*>(p.q);
    for (int x = tid; x < BM * (D / 4); x += kThreads) {
        const int r = x / (D / 4), c = (x % (D / 4)) * 4;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < rows) {
            const int f = row0 + r;
            v = load4(q + ((long long)(start + f / p.G) * p.H + kvh * p.G + f % p.G) * D + c);
        }
        *reinterpret_cast<float4*>(sq + r * C::LD + c) = v;
    }
    const int ty = tid / 16, tx = tid % 16;   // rows 4 ty + i; keys tx + 16 j; columns 4 tx + 64 j
    int pos[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        pos[i] = 4 * ty + i < rows ? first_pos + (row0 + 4 * ty + i) / p.G : -1;
    float m[4], l[4], o[4][D / 16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY, l[i] = 0.f;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) o[i][j] = 0.f;
    }
    const float* kb = static_cast<const float*>(p.k_base) + p.tile_off + (long long)kvh * p.s_head;
    const float* vb = static_cast<const float*>(p.v_base) + p.tile_off + (long long)kvh * p.s_head;

    for (int kt = kt0; kt < kt1; ++kt) {
        const int t0 = kt * BN;
        __syncthreads();  // the previous tile's k, v and p have been read
        if (tid < BN) {
            int blk = -1;
            if (t0 + tid < see) {
                blk = ld_dep(p.bt + (long long)b * p.maxb + (t0 + tid) / B);
                if (blk < 0 || blk >= p.num_blocks) {
                    atomicOr(p.status, kStatusBadBlock);
                    blk = -1;
                }
            }
            slot[tid] = blk;
        }
        __syncthreads();
        for (int x = tid; x < BN * (D / 4); x += kThreads) {
            const int r = x / (D / 4), c = (x % (D / 4)) * 4;
            float4 kv = make_float4(0.f, 0.f, 0.f, 0.f), vv = kv;
            const int blk = slot[r];
            if (blk >= 0) {
                const long long off = (long long)blk * p.s_blk + (long long)((t0 + r) % B) * D + c;
                kv = load4(kb + off), vv = load4(vb + off);
            }
            *reinterpret_cast<float4*>(sk + r * C::LD + c) = kv;
            *reinterpret_cast<float4*>(sv + r * C::LD + c) = vv;
        }
        __syncthreads();
        float s[4][4] = {};
        for (int d = 0; d < D; d += 4) {
            float4 a[4], c[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4*>(sq + (4 * ty + i) * C::LD + d);
#pragma unroll
            for (int j = 0; j < 4; ++j) c[j] = *reinterpret_cast<const float4*>(sk + (tx + 16 * j) * C::LD + d);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[i][j] = fmaf(a[i].x, c[j].x, s[i][j]);
                    s[i][j] = fmaf(a[i].y, c[j].y, s[i][j]);
                    s[i][j] = fmaf(a[i].z, c[j].z, s[i][j]);
                    s[i][j] = fmaf(a[i].w, c[j].w, s[i][j]);
                }
        }
        // a key without weight for a row is marked by p = -1, and skipped below:
        // its value may be anything
        bool hidden = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float mt = -INFINITY;
            bool see_it[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int key = tx + 16 * j;
                see_it[j] = t0 + key <= pos[i] && slot[key] >= 0;
                hidden = hidden || !see_it[j];
                s[i][j] *= p.qscale;
                if (see_it[j]) mt = fmaxf(mt, s[i][j]);
            }
#pragma unroll
            for (int x = 8; x > 0; x >>= 1) mt = fmaxf(mt, __shfl_xor_sync(kFullMask, mt, x));
            const float mn = fmaxf(fmaxf(m[i], mt), -3.0e38f);  // finite: a row may see no key
            const float alpha = exp2f(m[i] - mn);
            m[i] = mn;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float e = see_it[j] ? exp2f(s[i][j] - mn) : -1.f;
                if (see_it[j]) sum += e;
                sp[(4 * ty + i) * C::LP + tx + 16 * j] = e;
            }
            l[i] = l[i] * alpha + sum;  // this thread's share of the row's sum
#pragma unroll
            for (int j = 0; j < D / 16; ++j) o[i][j] *= alpha;
        }
        const bool any_hidden = __syncthreads_or(hidden);
        if (any_hidden) {
            for (int key = 0; key < BN; ++key) {
                float4 v[D / 64];
#pragma unroll
                for (int j = 0; j < D / 64; ++j) v[j] = *reinterpret_cast<const float4*>(sv + key * C::LD + 4 * tx + 64 * j);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float e = sp[(4 * ty + i) * C::LP + key];
                    if (e < 0.f) continue;
#pragma unroll
                    for (int j = 0; j < D / 64; ++j) {
                        o[i][4 * j] = fmaf(e, v[j].x, o[i][4 * j]);
                        o[i][4 * j + 1] = fmaf(e, v[j].y, o[i][4 * j + 1]);
                        o[i][4 * j + 2] = fmaf(e, v[j].z, o[i][4 * j + 2]);
                        o[i][4 * j + 3] = fmaf(e, v[j].w, o[i][4 * j + 3]);
                    }
                }
            }
        } else {
#pragma unroll 4
            for (int key = 0; key < BN; ++key) {
                float4 v[D / 64];
#pragma unroll
                for (int j = 0; j < D / 64; ++j) v[j] = *reinterpret_cast<const float4*>(sv + key * C::LD + 4 * tx + 64 * j);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float e = sp[(4 * ty + i) * C::LP + key];
#pragma unroll
                    for (int j = 0; j < D / 64; ++j) {
                        o[i][4 * j] = fmaf(e, v[j].x, o[i][4 * j]);
                        o[i][4 * j + 1] = fmaf(e, v[j].y, o[i][4 * j + 1]);
                        o[i][4 * j + 2] = fmaf(e, v[j].z, o[i][4 * j + 2]);
                        o[i][4 * j + 3] = fmaf(e, v[j].w, o[i][4 * j + 3]);
                    }
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int x = 8; x > 0; x >>= 1) l[i] += __shfl_xor_sync(kFullMask, l[i], x);
        const int r = 4 * ty + i;
        if (r >= rows) continue;
        const int f = row0 + r;
        const long long orow = (long long)(start + f / p.G) * p.H + kvh * p.G + f % p.G;
        if (p.splits == 1) {
            const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
#pragma unroll
            for (int j = 0; j < D / 64; ++j)
                store4(static_cast<float*>(p.out) + orow * D + 4 * tx + 64 * j,
                       make_float4(o[i][4 * j] * inv, o[i][4 * j + 1] * inv, o[i][4 * j + 2] * inv,
                                   o[i][4 * j + 3] * inv));
        } else {
            const long long prow = (long long)blockIdx.z * p.num_tokens * p.H + orow;
#pragma unroll
            for (int j = 0; j < D / 64; ++j)
                store4(p.part_o + prow * D + 4 * tx + 64 * j,
                       make_float4(o[i][4 * j], o[i][4 * j + 1], o[i][4 * j + 2], o[i][4 * j + 3]));
            if (tx == 0) p.part_ml[2 * prow] = m[i], p.part_ml[2 * prow + 1] = l[i];
        }
    }
}

// Joins the splits of every row before the last sequence's end: a warp a row.
template <int D>
__global__ void __launch_bounds__(kThreads) pa_prefill_join_kernel(const PrefillParams p) {
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const long long all = (long long)p.num_tokens * p.H;
    if (row >= all || row / p.H < ld_dep(p.starts) || row / p.H >= ld_dep(p.starts + p.batch)) return;
    float m = -INFINITY;
    for (int z = 0; z < p.splits; ++z) m = fmaxf(m, ld_dep(p.part_ml + 2 * (z * all + row)));
    float l = 0.f, o[D / 32] = {};
    for (int z = 0; z < p.splits; ++z) {
        const float lz = ld_dep(p.part_ml + 2 * (z * all + row) + 1);
        if (lz == 0.f) continue;
        const float w = exp2f(ld_dep(p.part_ml + 2 * (z * all + row)) - m);
        l += w * lz;
#pragma unroll
        for (int j = 0; j < D / 32; ++j)
            o[j] = fmaf(w, ld_dep(p.part_o + (z * all + row) * D + lane * (D / 32) + j), o[j]);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    float* out = static_cast<float*>(p.out) + row * D + lane * (D / 32);
#pragma unroll
    for (int j = 0; j < D / 32; ++j) out[j] = o[j] * inv;
}

template <int D, int B>
cudaError_t launch_simt(const PrefillParams& p, cudaStream_t s) {
    auto kern = pa_prefill_simt_kernel<D, B>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         SimtCfg<D>::SMEM);
    if (e != cudaSuccess) return e;
    const long long tiles = (long long)p.num_tokens * p.G / BM + p.batch;
    if (tiles > 0x7fffffffLL || p.Hkv > 65535) return cudaErrorInvalidConfiguration;
    e = launch_pdl(kern, dim3((unsigned)tiles, p.Hkv, p.splits), dim3(kThreads), SimtCfg<D>::SMEM,
                   s, p);
    if (e != cudaSuccess || p.splits == 1) return e;
    const long long rows = (long long)p.num_tokens * p.H;
    return launch_pdl(pa_prefill_join_kernel<D>, dim3((unsigned)((rows + 7) / 8)), dim3(kThreads),
                      0, s, p);
}

}  // namespace

bool prefill_supported(int dtype, int D, int B) {
    return (dtype == 0 || dtype == 1) && (D == 64 || D == 128) && (B == 16 || B == 32);
}

int prefill_simt_splits(int G, int Hkv, int batch, int num_tokens, int maxb, int B, int num_sms) {
    const long long tiles = ((long long)num_tokens * G / BM + batch) * Hkv;
    const long long want = 2LL * num_sms / (tiles > 0 ? tiles : 1);
    const long long most = ((long long)maxb * B + 255) / 256;  // four key tiles at least
    long long n = want < most ? want : most;
    return (int)(n < 1 ? 1 : n > 64 ? 64 : n);
}

cudaError_t launch_prefill_simt(const PrefillParams& p, int D, int B, cudaStream_t s) {
    if (D == 64 && B == 16) return launch_simt<64, 16>(p, s);
    if (D == 64 && B == 32) return launch_simt<64, 32>(p, s);
    if (D == 128 && B == 16) return launch_simt<128, 16>(p, s);
    if (D == 128 && B == 32) return launch_simt<128, 32>(p, s);
    return cudaErrorNotSupported;
}

}  // namespace pa
