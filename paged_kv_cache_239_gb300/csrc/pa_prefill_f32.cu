// pa_prefill_f32.cu -- attention of several new tokens per sequence over an fp32
// paged cache: mma.sync on TF32 with every operand split in two.
//
//   out_t = sum_{s <= p_t} softmax_s(scale q_t . k_s) v_s,
//   p_t = context_lens[b] - n_b + i for the i-th of sequence b's n_b new tokens.
//
// The query heads of a KV head's group share its keys, so the rows of a tile
// are (token, head of the group) in that order, flattened: row r is token r / G,
// head r % G, and a tile takes 64 consecutive rows whatever G is, 16 to a warp.
// Keys and values come 32 at a time (head_dim 128: 16), by cp.async in two stages:
// what leaves room for three CTAs on an SM.
//
// TF32 keeps 11 bits of a product's factors, so x = hi + lo with hi = x rounded to
// TF32 and lo = x - hi (exact; 12 bits, of which TF32 keeps 11): hi hi' + hi lo' +
// lo hi' misses x x' by about 2^-22, as an fp32 product does by 2^-24, and the
// sums are fp32.  Three m16n8k8 products take 24 cycles of a scheduler's tensor pipe
// for 1024 multiply-adds; fused multiply-adds take 32, and two operands from shared
// memory for each sixteenth of them.
//
// What bounds it: five in six instructions are not products (splits, operand loads,
// the softmax), and the pipe is busy about 62 % of the time.  A prompt of
// 4096 with 32 heads on 8: head_dim 64 1.13 ms, 128 2.23 ms (2.38 with tiles of 32
// keys and two CTAs per SM), 61 TFLOP/s of the formula; with fused multiply-adds
// it ran at 12.
//
// Few row tiles: each is split over the keys, up to eight ways in a cluster that
// joins its parts through distributed shared memory (a prompt of 128: 8.7 us; the
// same joined by a second launch 12.5), and beyond that in several clusters, whose
// parts a second launch joins (4 tokens over 30,000 keys 26 us; all 64 parts joined
// by the launch, 52).
//
// The order of the summed index is free in a product, so it is chosen to suit the
// fragments: a thread's four neighbouring elements of q and k are its columns of
// two steps, a thread's scores of neighbouring keys are its columns of P, and its
// four neighbouring columns of v belong to four tiles of O.  Every operand is
// read as float4, with strides that keep eight lanes on 32 banks.
//
// inf * 0 and inf - inf would make NaN of what a row sees as an infinite value, or
// does not see at all.  Values that are not finite are zeroed in shared memory and
// remembered by column and position, and put into the rows that see them at the
// end; a warp whose scores come out not finite sums that tile's plainly.  (What
// TF32 would round to infinity, the last 2^-12 of the range, is taken the same
// way; such a value is cut by as much.)
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

namespace cg = cooperative_groups;

constexpr int BM = 64, kThreads = 128;
constexpr int key_tile(int D) { return D == 128 ? 16 : 32; }  // keys per tile

template <int D>
struct F32Cfg {
    static constexpr int BN = key_tile(D);
    static constexpr int LQ = D + 16, LV = D + 4;   // row strides (floats) of q and k; v
    static constexpr int STAGE = BN * (LQ + LV);    // floats
    static constexpr int SMEM = (BM * LQ + 2 * STAGE) * 4 + 3 * D * 4;
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(valid ? 16 : 0)
                 : "memory");
}

// x = hi + lo, both to be read as TF32 (which ignores the low 13 bits).
__device__ __forceinline__ void split(float x, uint32_t& hi, uint32_t& lo) {
    hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
    lo = __float_as_uint(x - __uint_as_float(hi));
}

__device__ __forceinline__ void mma8(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float4 lds4(const float* p) { return *reinterpret_cast<const float4*>(p); }

// The largest magnitude that rounds to a finite TF32 value.
constexpr float kTop = 0x1.ffdffep127f;
__device__ __forceinline__ float max_nan(float x, float y) {  // (NaN if one is)
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(x) : "f"(y));
    return x;
}
__device__ __forceinline__ float top4(const float* p) {
    const float4 x = lds4(p);
    return max_nan(max_nan(fabsf(x.x), fabsf(x.y)), max_nan(fabsf(x.z), fabsf(x.w)));
}

// Four columns of a row joined from parts of the keys: maximum (in powers of two), sum, sums of values.
struct Joined {
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    __device__ __forceinline__ void add(float2 ml, float4 x) {
        if (ml.y == 0.f) return;  // (the part saw no key of the row)
        const float mn = fmaxf(m, ml.x);
        const float keep = ex2_approx(m - mn), w = ex2_approx(ml.x - mn);
        m = mn;
        l = fmaf(l, keep, w * ml.y);
        o.x = fmaf(o.x, keep, w * x.x), o.y = fmaf(o.y, keep, w * x.y);
        o.z = fmaf(o.z, keep, w * x.z), o.w = fmaf(o.w, keep, w * x.w);
    }
    __device__ __forceinline__ float4 out() const {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        return make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
    }
};

template <int D, int B>
__global__ void __launch_bounds__(kThreads, 3) pa_prefill_f32_kernel(const PrefillParams p) {
    pdl_trigger();
    pdl_wait();
    using C = F32Cfg<D>;
    constexpr int BN = C::BN;
    extern __shared__ __align__(16) float smem[];
    float* sq = smem;
    float* ring = sq + BM * C::LQ;
    int* marks = reinterpret_cast<int*>(ring + 2 * C::STAGE);  // first NaN, +inf, -inf per column
    __shared__ int s_at[5];  // sequence, first row, first token, new tokens, context
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    auto token = [&](int row) {  // row / G (the host's multiplier, for rows below 2^31)
        return (int)(((unsigned long long)(unsigned)row * p.div_mul) >> p.div_shift);
    };

    // ---- the tile: sequence and first row; the last tiles first, of all KV heads (a
    // prompt's last rows see most: what starts late is short) ----
    const int kvh = blockIdx.x % p.Hkv;
    if (warp == 0) {
        int left = gridDim.x / p.Hkv - 1 - blockIdx.x / p.Hkv, found = -1, row0 = 0;
        for (int b0 = 0; b0 < p.batch && found < 0; b0 += 32) {
            const int b = b0 + lane;
            int tiles = 0, s0 = 0, s1 = 0, n = 0;
            if (b < p.batch) {
                s0 = ld_dep(p.starts + b), s1 = ld_dep(p.starts + b + 1);
                n = ld_dep(p.lens + b);
                const bool good = s0 >= 0 && s1 >= s0 && s1 <= p.num_tokens;
                if ((!good || n < 0 || n > p.maxb * B) && blockIdx.x == 0 && blockIdx.y == 0)
                    atomicOr(p.status, kStatusBadLength);
                if (good) tiles = (int)(((long long)(s1 - s0) * p.G + BM - 1) / BM);
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
                if (lane == f) s_at[2] = s0, s_at[3] = s1 - s0, s_at[4] = n;
            }
            left -= __shfl_sync(kFullMask, incl, 31);
        }
        if (lane == 0) s_at[0] = found, s_at[1] = row0;
    }
    for (int x = tid; x < 3 * D; x += kThreads) marks[x] = INT_MAX;
    __syncthreads();
    const int b = s_at[0], row0 = s_at[1];
    if (b < 0) return;
    const int start = s_at[2], n_new = s_at[3];
    int n = s_at[4];
    if (n < n_new || n > p.maxb * B) {
        if (tid == 0) atomicOr(p.status, kStatusBadLength);
        n = 0;
    }
    const int rows = (int)min((long long)BM, (long long)n_new * p.G - row0);
    const int first_pos = n - n_new;
    // keys: this split's part of the tile's [0, last visible + 1)
    const int see = n > 0 ? first_pos + token(row0 + rows - 1) + 1 : 0;
    const int key_tiles = (see + BN - 1) / BN;
    const int per = (key_tiles + p.splits - 1) / p.splits;
    const int kt0 = min((int)blockIdx.y * per, key_tiles), kt1 = min(kt0 + per, key_tiles);

    // ---- copies: q once; k and v a tile ahead, thread = 16-byte chunk of rows ----
    constexpr int CPR = D / 4, RPP = kThreads / CPR;  // chunks per row, rows per pass
    const int cc = tid % CPR, cr = tid / CPR;
    const uint32_t q_at = smem_addr(sq) + (uint32_t)(cr * C::LQ + 4 * cc) * 4;
    const float* q = static_cast<const float*>(p.q);
    const float* kb = static_cast<const float*>(p.k_base) + p.tile_off + (long long)kvh * p.s_head + 4 * cc;
    const float* vb = static_cast<const float*>(p.v_base) + p.tile_off + (long long)kvh * p.s_head + 4 * cc;
    constexpr int PAGES = BN > B ? BN / B : 1;  // 1 or 2 per tile
    int page[2], ids[2];           // the next tile's pages (-1: none); ids as read, one tile ahead
    auto look_up = [&](int kt) {
#pragma unroll
        for (int u = 0; u < PAGES; ++u) {
            const int tok = kt * BN + u * B;
            ids[u] = 0;
            if (kt < kt1 && tok < see) ids[u] = ld_dep(p.bt + (long long)b * p.maxb + tok / B);
        }
    };
    auto copy = [&](int kt) {  // copies tile kt, whose ids have been read
#pragma unroll
        for (int u = 0; u < PAGES; ++u) {
            const bool in = kt < kt1 && kt * BN + u * B < see;
            const bool good = ids[u] >= 0 && ids[u] < p.num_blocks;
            if (in && !good && tid == 0) atomicOr(p.status, kStatusBadBlock);
            page[u] = in && good ? ids[u] : -1;
        }
        look_up(kt + 1);
        if (kt < kt1) {
            float* st = ring + (kt & 1) * C::STAGE;
            const uint32_t k_at = smem_addr(st) + (uint32_t)(cr * C::LQ + 4 * cc) * 4;
            const uint32_t v_at = smem_addr(st + BN * C::LQ) + (uint32_t)(cr * C::LV + 4 * cc) * 4;
#pragma unroll
            for (int r = 0; r < BN; r += RPP) {
                const int key = r + cr, blk = PAGES == 1 || key < B ? page[0] : page[1];
                const bool in = blk >= 0 && kt * BN + key < n;
                const int row = (BN < B ? kt * BN + key : key) % B;
                const long long off = in ? (long long)blk * p.s_blk + row * D : 0;
                cp16(k_at + r * C::LQ * 4, kb + off, in);
                cp16(v_at + r * C::LV * 4, vb + off, in);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    look_up(kt0);  // (under the addresses of q)
    for (int r = 0; r < BM; r += RPP) {
        const int f = row0 + r + cr;
        const bool live = r + cr < rows;
        const int tok = live ? token(f) : 0;
        cp16(q_at + r * C::LQ * 4,
             live ? q + ((long long)(start + tok) * p.H + kvh * p.G + f - tok * p.G) * D + 4 * cc : q, live);
    }
    copy(kt0);

    // this thread's rows: g and g + 8 of the warp's 16
    int pos[2];
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int r = 16 * warp + g + 8 * h;
        pos[h] = r < rows ? first_pos + token(row0 + r) : -1;
    }
    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[i][k] = 0.f;
    const int tile_pos = first_pos + token(row0);  // the tile's first row's position
    const float* qw = sq + (16 * warp + g) * C::LQ + 4 * t;

    for (int kt = kt0; kt < kt1; ++kt) {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        const float* sk = ring + (kt & 1) * C::STAGE;
        float* sv = ring + (kt & 1) * C::STAGE + BN * C::LQ;
        const int t0 = kt * BN;
        // the largest value of what this thread copied
        float top = 0.f;
#pragma unroll
        for (int r = 0; r < BN; r += RPP) top = max_nan(top, top4(sv + (r + cr) * C::LV + 4 * cc));
        // tile kt is in for all, and the other stage has been read
        const bool odd = !(top <= kTop);
        const bool any_odd = __syncthreads_or(odd);
        const bool there0 = page[0] >= 0, there1 = PAGES == 1 ? there0 : page[1] >= 0;
        copy(kt + 1);
        if (any_odd) {
            if (odd)
                for (int r = 0; r < BN; r += RPP)
                    for (int e = 0; e < 4; ++e) {
                        float& x = sv[(r + cr) * C::LV + 4 * cc + e];
                        if (isfinite(x)) {
                            x = fminf(fmaxf(x, -kTop), kTop);
                            continue;
                        }
                        atomicMin(marks + (x != x ? 0 : x > 0.f ? D : 2 * D) + 4 * cc + e, t0 + r + cr);
                        x = 0.f;
                    }
            __syncthreads();
        }
        if (16 * warp >= rows) continue;  // (none of the warp's rows are there)

        // S = Q K^T
        float s[BN / 8][4];
#pragma unroll
        for (int i = 0; i < BN / 8; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) s[i][k] = 0.f;
#pragma unroll 2
        for (int d = 0; d < D; d += 16) {
            uint32_t ah[2][4], al[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float4 x = lds4(qw + h * 8 * C::LQ + d);
                split(x.x, ah[0][h], al[0][h]), split(x.y, ah[0][2 + h], al[0][2 + h]);
                split(x.z, ah[1][h], al[1][h]), split(x.w, ah[1][2 + h], al[1][2 + h]);
            }
            uint32_t bh[BN / 8][4], bl[BN / 8][4];
#pragma unroll
            for (int i = 0; i < BN / 8; ++i) {
                const float4 x = lds4(sk + (8 * i + g) * C::LQ + 4 * t + d);
                split(x.x, bh[i][0], bl[i][0]), split(x.y, bh[i][1], bl[i][1]);
                split(x.z, bh[i][2], bl[i][2]), split(x.w, bh[i][3], bl[i][3]);
            }
            // (four sums in turn: a product waits for the one before on its sum)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
#pragma unroll
                for (int i = 0; i < BN / 8; ++i) mma8(s[i], al[u], bh[i][2 * u], bh[i][2 * u + 1]);
#pragma unroll
                for (int i = 0; i < BN / 8; ++i) mma8(s[i], ah[u], bl[i][2 * u], bl[i][2 * u + 1]);
#pragma unroll
                for (int i = 0; i < BN / 8; ++i) mma8(s[i], ah[u], bh[i][2 * u], bh[i][2 * u + 1]);
            }
        }
        // x - hi is NaN for an infinite x: scores that are not finite are summed plainly
        float z = 0.f;
#pragma unroll
        for (int i = 0; i < BN / 8; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) z = fmaf(s[i][k], 0.f, z);
        if (__any_sync(kFullMask, z != 0.f)) {
#pragma unroll
            for (int i = 0; i < BN / 8; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) s[i][k] = 0.f;
            for (int d = 0; d < D; ++d) {
                const float q0 = qw[d - 4 * t], q1 = qw[8 * C::LQ + d - 4 * t];
#pragma unroll
                for (int i = 0; i < BN / 8; ++i)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const float x = sk[(8 * i + 2 * t + c) * C::LQ + d];
                        s[i][c] = fmaf(q0, x, s[i][c]), s[i][2 + c] = fmaf(q1, x, s[i][2 + c]);
                    }
            }
        }
        // weights: the keys of s[i][2 h + c] are t0 + 8 i + 2 t + c, its row pos[h]
        const bool masked = t0 + BN - 1 > tile_pos || !there0 || !there1 || rows < BM;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float mt = -INFINITY;
#pragma unroll
            for (int i = 0; i < BN / 8; ++i)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float& x = s[i][2 * h + c];
                    x *= p.qscale;
                    if (masked) {
                        const int key = 8 * i + 2 * t + c;
                        const bool in = t0 + key <= pos[h] && (PAGES == 1 || key < B ? there0 : there1);
                        if (!in) x = -INFINITY;
                    }
                    mt = fmaxf(mt, x);
                }
            mt = fmaxf(mt, __shfl_xor_sync(kFullMask, mt, 1));
            mt = fmaxf(mt, __shfl_xor_sync(kFullMask, mt, 2));
            const float mn = fmaxf(fmaxf(m[h], mt), -3.0e38f);  // finite: a row may see no key
            const float alpha = ex2_approx(m[h] - mn);
            m[h] = mn;
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < BN / 8; ++i)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float& x = s[i][2 * h + c];
                    x = ex2_approx(x - mn);
                    sum += x;
                }
            l[h] = l[h] * alpha + sum;  // (this thread's share)
            if (__any_sync(kFullMask, alpha != 1.f))
#pragma unroll
                for (int i = 0; i < D / 8; ++i) o[i][2 * h] *= alpha, o[i][2 * h + 1] *= alpha;
        }
        // O += P V: step i sums over keys 8 i + (2 t, 2 t + 1)
#pragma unroll
        for (int i = 0; i < BN / 8; ++i) {
            uint32_t ah[4], al[4];
            split(s[i][0], ah[0], al[0]), split(s[i][2], ah[1], al[1]);
            split(s[i][1], ah[2], al[2]), split(s[i][3], ah[3], al[3]);
            const float* v0 = sv + (8 * i + 2 * t) * C::LV + 4 * g;
#pragma unroll
            for (int d = 0; d < D; d += 32) {
                const float4 x = lds4(v0 + d), y = lds4(v0 + C::LV + d);
                const float xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
                uint32_t bh[4][2], bl[4][2];
#pragma unroll
                for (int e = 0; e < 4; ++e) split(xs[e], bh[e][0], bl[e][0]), split(ys[e], bh[e][1], bl[e][1]);
#pragma unroll
                for (int e = 0; e < 4; ++e) mma8(o[d / 8 + e], al, bh[e][0], bh[e][1]);
#pragma unroll
                for (int e = 0; e < 4; ++e) mma8(o[d / 8 + e], ah, bl[e][0], bl[e][1]);
#pragma unroll
                for (int e = 0; e < 4; ++e) mma8(o[d / 8 + e], ah, bh[e][0], bh[e][1]);
            }
        }
    }
    __syncthreads();  // the marks; and the ring is free
    constexpr int LO = D + 4;
    float* part = ring;  // this CTA's O, if others have parts of it
    float2* part_ml = reinterpret_cast<float2*>(ring + BM * LO);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        l[h] += __shfl_xor_sync(kFullMask, l[h], 1);
        l[h] += __shfl_xor_sync(kFullMask, l[h], 2);
        const int r = 16 * warp + g + 8 * h;
        if (r >= rows) continue;
        const int f = row0 + r, tok = token(f);
        const float inv = p.cluster > 1 ? 1.f : l[h] == 0.f ? 0.f : 1.f / l[h];
        float* out = p.cluster > 1
                         ? part + r * LO
                         : static_cast<float*>(p.out) +
                               ((long long)(start + tok) * p.H + kvh * p.G + f - tok * p.G) * D;
#pragma unroll
        for (int d = 0; d < D; d += 32)
#pragma unroll
            for (int c = 0; c < 2; ++c) {  // columns d + 8 t + 4 c + (0 .. 3)
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int* mk = marks + d + 8 * t + 4 * c + e;
                    const bool nan = mk[0] <= pos[h], up = mk[D] <= pos[h], down = mk[2 * D] <= pos[h];
                    v[e] = o[d / 8 + e][2 * h + c] * inv +
                           (nan || (up && down) ? NAN : up ? INFINITY : down ? -INFINITY : 0.f);
                }
                *reinterpret_cast<float4*>(out + d + 8 * t + 4 * c) = make_float4(v[0], v[1], v[2], v[3]);
            }
        if (p.cluster > 1 && t == 0) part_ml[r] = make_float2(m[h], l[h]);
    }
    if (p.cluster == 1) return;

    // ---- the cluster's parts: each CTA joins its share of the rows ----
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    const int rank = (int)cluster.block_rank();
    const int groups = p.splits / p.cluster;
    for (int x = rank * (kThreads / CPR) + cr; x < rows; x += p.cluster * (kThreads / CPR)) {
        const int f = row0 + x, tok = token(f);
        const long long orow = (long long)(start + tok) * p.H + kvh * p.G + f - tok * p.G;
        Joined j;
        float2 ml[8];
        float4 v[8];
#pragma unroll
        for (int z = 0; z < 8; ++z) {
            if (z >= p.cluster) break;
            ml[z] = *cluster.map_shared_rank(part_ml + x, z);
            v[z] = *cluster.map_shared_rank(reinterpret_cast<float4*>(part + x * LO) + cc, z);
        }
#pragma unroll
        for (int z = 0; z < 8; ++z)
            if (z < p.cluster) j.add(ml[z], v[z]);
        if (groups == 1) {
            reinterpret_cast<float4*>(p.out)[orow * CPR + cc] = j.out();
        } else {
            const long long prow = (long long)(blockIdx.y / p.cluster) * p.num_tokens * p.H + orow;
            reinterpret_cast<float4*>(p.part_o)[prow * CPR + cc] = j.o;
            if (cc == 0) reinterpret_cast<float2*>(p.part_ml)[prow] = make_float2(j.m, j.l);
        }
    }
    cluster.sync();  // (no CTA leaves while others read its part)
}

// Joins the clusters' parts of every row of a sequence: D / 4 lanes a row, up to
// eight parts in flight.
constexpr int kJoinThreads = 128;
template <int D>
__global__ void __launch_bounds__(kJoinThreads) pa_prefill_f32_join_kernel(const PrefillParams p) {
    pdl_trigger();
    pdl_wait();
    constexpr int LPR = D / 4;
    const int lane = threadIdx.x % LPR;
    const long long row = (long long)blockIdx.x * (kJoinThreads / LPR) + threadIdx.x / LPR;
    const long long all = (long long)p.num_tokens * p.H;
    if (row >= all || row < (long long)ld_dep(p.starts) * p.H ||
        row >= (long long)ld_dep(p.starts + p.batch) * p.H)
        return;
    const int groups = p.splits / p.cluster;
    Joined j;
    for (int z0 = 0; z0 < groups; z0 += 8) {
        float2 ml[8];
        float4 x[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const long long at = min(z0 + u, groups - 1) * all + row;
            ml[u] = ld_dep(reinterpret_cast<const float2*>(p.part_ml) + at);
            x[u] = ld_dep(reinterpret_cast<const float4*>(p.part_o) + at * LPR + lane);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (z0 + u < groups) j.add(ml[u], x[u]);
    }
    reinterpret_cast<float4*>(p.out)[row * LPR + lane] = j.out();
}

template <int D, int B>
cudaError_t launch_inst(const PrefillParams& p, cudaStream_t s) {
    auto kern = pa_prefill_f32_kernel<D, B>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         F32Cfg<D>::SMEM);
    if (e != cudaSuccess) return e;
    const long long ctas = ((long long)p.num_tokens * p.G / BM + p.batch) * p.Hkv;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas, p.splits);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = F32Cfg<D>::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = attr[1].val.clusterDim.z = 1;
    attr[1].val.clusterDim.y = p.cluster;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, kern, p);
    if (e != cudaSuccess || p.splits == p.cluster) return e;
    const long long rows = (long long)p.num_tokens * p.H;
    constexpr int RPC = kJoinThreads / (D / 4);
    return launch_pdl(pa_prefill_f32_join_kernel<D>, dim3((unsigned)((rows + RPC - 1) / RPC)),
                      dim3(kJoinThreads), 0, s, p);
}

}  // namespace

bool prefill_supported(int dtype, int D, int B) {
    return (dtype == 0 || dtype == 1) && (D == 64 || D == 128) && (B == 16 || B == 32);
}

// Parts of each context (the host knows the tables' width, not the lengths).  Up to
// eight are a cluster, which joins them by itself: as many as give every SM a CTA,
// and up to eight CTAs where each part keeps three key tiles, since a prompt's row
// tiles see few or many keys and short parts even that out (500 tokens of 16 heads
// behind 7,300: 1 part 1250 us, 2 936, 4 670, 8 607); parts of less than three
// tiles do not pay for the join once they share an SM (4 sequences of up to 130
// tokens: 4 parts 20.7 us, 8 25.8).  More than eight take a second launch: where
// two CTAs per SM ask for 16 and each has a tile (4 tokens over 30,000 keys: 152
// parts 26 us, 256 33).
int prefill_f32_splits(int G, int Hkv, int batch, int num_tokens, int maxb, int D, int B,
                       int num_sms, int* cluster) {
    const long long tiles = ((long long)num_tokens * G / BM + batch) * Hkv;
    const long long keys = ((long long)maxb * B + key_tile(D) - 1) / key_tile(D);  // tiles
    if (tiles <= 0) return *cluster = 1;
    const long long one = num_sms / tiles;  // parts that get an SM each
    const long long wide = std::min({2 * num_sms / tiles, keys, 256LL});
    if (wide >= 16) {
        *cluster = 8;
        return (int)wide / 8 * 8;
    }
    const long long n = std::min({8 * num_sms / tiles, keys, std::max(one, keys / 3)});
    return *cluster = n >= 8 ? 8 : n >= 4 ? 4 : n >= 2 ? 2 : 1;
}

cudaError_t launch_prefill_f32(const PrefillParams& p, int D, int B, cudaStream_t s) {
    if (D == 64 && B == 16) return launch_inst<64, 16>(p, s);
    if (D == 64 && B == 32) return launch_inst<64, 32>(p, s);
    if (D == 128 && B == 16) return launch_inst<128, 16>(p, s);
    if (D == 128 && B == 32) return launch_inst<128, 32>(p, s);
    return cudaErrorNotSupported;
}

}  // namespace pa
