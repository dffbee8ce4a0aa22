// pa_prefill_mma.cu -- attention of several new tokens per sequence over the paged
// cache on mma.sync: fp32 pools, and the calls on bf16 pools that are too short for
// the tcgen05 kernel's start to pay.
//
//   out_t = sum_{s <= p_t} softmax_s(scale q_t . k_s) v_s,
//   p_t = context_lens[b] - n_b + i for the i-th of sequence b's n_b new tokens.
//
// The query heads of a KV head's group share its keys, so the rows of a tile
// are (token, head of the group) in that order, flattened: row r is token r / G,
// head r % G, and a tile takes 64 consecutive rows whatever G is, 16 to a warp.
// Keys and values come a tile at a time by cp.async in two stages, scores, weights
// and outputs stay in registers, one pass over the keys with the running maximum and
// sum of each row.
//
// fp32 (tiles of 32 keys, 16 at head_dim 128: what leaves room for three CTAs on an
// SM).  TF32 keeps 11 bits of a product's factors, so x = hi + lo with hi = x
// rounded to TF32 and lo = x - hi (exact; 12 bits, of which TF32 keeps 11): hi hi' +
// hi lo' + lo hi' misses x x' by 2^-22 at most, with either sign.  The tensor core's sums
// are fp32, but cut off toward zero: a sum that runs through it loses the same way at
// every step.  So none runs long there: the small products of a score have a sum of their
// own, and P V of a tile starts from zero and is added to O by ordinary, rounded additions.
// (A prompt of 4096 is off by 4.4e-7 of its output's size at head_dim 128, 3.8e-7 at 64,
// plain fp32 products and exp by 5.4e-7 and 4.9e-7; with O as the products' running sum
// 4.3e-6, all of it one-sided and growing with the context, for 7 % less time at 128, 1 %
// at 64.  The product lo lo', or rounding lo, changes none of these figures.)  Three
// m16n8k8 products take 24 cycles of a scheduler's tensor pipe for 1024 multiply-adds;
// fused multiply-adds take 32, and two operands from shared memory for each sixteenth
// of them.  The order of the summed index is free in a product, so it is chosen to suit
// the fragments: a thread's four neighbouring elements of q and k are its columns of two
// steps, a thread's scores of neighbouring keys are its columns of P, and its four
// neighbouring columns of v belong to four tiles of O.  Every operand is read as float4,
// with strides that keep eight lanes on 32 banks.
//   Five in six instructions are not products (splits, operand loads, the softmax),
// and the pipe is busy 56 % of the time: a prompt of 4096 with 32 heads on 8
// takes 1.12 ms at head_dim 64 and 2.30 ms at 128, 61 and 60 TFLOP/s of the formula; with
// fused multiply-adds it ran at 12.
//
// bf16 (tiles of 64 keys, 32 at head_dim 128): operands by ldmatrix from rows whose
// 16-byte chunks are permuted by the row, so that no two lanes share a bank.  P is
// rounded to bf16 (2^-9 relative on average over many keys: the size of the output's
// own rounding); the sum takes the weights before that.  Eleven instructions to a
// product, latencies between them: it is the short start that counts here (one token
// over 100 keys: 5.0 us, the launch, four dependent loads and two tiles).
//
// Few row tiles: each is split over the keys, up to eight ways in a cluster that
// joins its parts through distributed shared memory (fp32, a prompt of 128 with 16 heads on 2
// of 64: 8.1 us, where a second launch for the join took 5 more), and beyond that in several
// clusters, whose parts a second launch joins (4 tokens over 30,000 keys 30 us; 49 with
// 64 parts).
//
// inf * 0 and inf - inf would make NaN of what a row sees as an infinite value, or
// does not see at all.  Values that are not finite (bf16: in tiles that some row does
// not see whole) are zeroed in shared memory and remembered by column and position,
// and put into the rows that see them at the end; a warp whose fp32 scores come out
// not finite sums that tile's plainly.  (What TF32 would round to infinity, the last
// 2^-12 of the range, is taken the same way; such a value is cut by as much.)
#include <cooperative_groups.h>
#include <cuda_bf16.h>
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

// fp32 operands: where the chunks of a row stand, and the two products.
template <int D>
struct CoreF32 {
    using T = float;
    static constexpr int BN = D == 128 ? 16 : 32;         // keys per tile
    static constexpr int CTAS = 3;                        // per SM
    static constexpr int LQ = D + 16, LV = D + 4;         // row strides (floats) of q and k; v
    static constexpr int QS = 4 * LQ, VS = 4 * LV;        // (bytes)
    static constexpr bool LOOK_ALL = true;                // every tile's V is looked over
    static __device__ __forceinline__ int q_at(int row, int chunk) { return row * QS + 16 * chunk; }
    static __device__ __forceinline__ int v_at(int row, int chunk) { return row * VS + 16 * chunk; }
    // column of O's register (i, c) of thread t
    static __device__ __forceinline__ int column(int i, int c, int t) {
        return i / 4 * 32 + 8 * t + 4 * c + i % 4;
    }
    static __device__ __forceinline__ bool odd(const void* chunk) {
        return !(top4(static_cast<const float*>(chunk)) <= kTop);
    }
    static __device__ __forceinline__ void clamp(float& x) { x = fminf(fmaxf(x, -kTop), kTop); }

    // S = Q K^T: s[i] the 8 keys from 8 i, this warp's 16 rows.  The small products have a
    // sum of their own: cut off at its last bit they lose 2^-12 of what they lose at s's.
    static __device__ __forceinline__ void scores(float (&s)[BN / 8][4], const unsigned char* sq,
                                                  const unsigned char* k, int warp, int lane) {
        const int g = lane >> 2, t = lane & 3;
        const float* qw = reinterpret_cast<const float*>(sq) + (16 * warp + g) * LQ + 4 * t;
        const float* sk = reinterpret_cast<const float*>(k);
        float small[BN / 8][4] = {};
#pragma unroll 4
        for (int d = 0; d < D; d += 16) {
            uint32_t ah[2][4], al[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float4 x = lds4(qw + h * 8 * LQ + d);
                split(x.x, ah[0][h], al[0][h]), split(x.y, ah[0][2 + h], al[0][2 + h]);
                split(x.z, ah[1][h], al[1][h]), split(x.w, ah[1][2 + h], al[1][2 + h]);
            }
            uint32_t bh[BN / 8][4], bl[BN / 8][4];
#pragma unroll
            for (int i = 0; i < BN / 8; ++i) {
                const float4 x = lds4(sk + (8 * i + g) * LQ + 4 * t + d);
                split(x.x, bh[i][0], bl[i][0]), split(x.y, bh[i][1], bl[i][1]);
                split(x.z, bh[i][2], bl[i][2]), split(x.w, bh[i][3], bl[i][3]);
            }
            // (four sums in turn: a product waits for the one before on its sum)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
#pragma unroll
                for (int i = 0; i < BN / 8; ++i) mma8(small[i], al[u], bh[i][2 * u], bh[i][2 * u + 1]);
#pragma unroll
                for (int i = 0; i < BN / 8; ++i) mma8(small[i], ah[u], bl[i][2 * u], bl[i][2 * u + 1]);
#pragma unroll
                for (int i = 0; i < BN / 8; ++i) mma8(s[i], ah[u], bh[i][2 * u], bh[i][2 * u + 1]);
            }
        }
#pragma unroll
        for (int i = 0; i < BN / 8; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) s[i][k] += small[i][k];
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
                const float q0 = qw[d - 4 * t], q1 = qw[8 * LQ + d - 4 * t];
#pragma unroll
                for (int i = 0; i < BN / 8; ++i)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const float x = sk[(8 * i + 2 * t + c) * LQ + d];
                        s[i][c] = fmaf(q0, x, s[i][c]), s[i][2 + c] = fmaf(q1, x, s[i][2 + c]);
                    }
            }
        }
    }

    // O += P V: step i sums over keys 8 i + (2 t, 2 t + 1); the tile's sum starts from zero
    static __device__ __forceinline__ void values(float (&o)[D / 8][4], const float (&s)[BN / 8][4],
                                                  const unsigned char* v, int lane) {
        const int g = lane >> 2, t = lane & 3;
        const float* sv = reinterpret_cast<const float*>(v);
        uint32_t ah[BN / 8][4], al[BN / 8][4];
#pragma unroll
        for (int i = 0; i < BN / 8; ++i) {
            split(s[i][0], ah[i][0], al[i][0]), split(s[i][2], ah[i][1], al[i][1]);
            split(s[i][1], ah[i][2], al[i][2]), split(s[i][3], ah[i][3], al[i][3]);
        }
#pragma unroll
        for (int d = 0; d < D; d += 32) {
            float part[4][4] = {};
#pragma unroll
            for (int i = 0; i < BN / 8; ++i) {
                const float* v0 = sv + (8 * i + 2 * t) * LV + 4 * g;
                const float4 x = lds4(v0 + d), y = lds4(v0 + LV + d);
                const float xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
                uint32_t bh[4][2], bl[4][2];
#pragma unroll
                for (int e = 0; e < 4; ++e) split(xs[e], bh[e][0], bl[e][0]), split(ys[e], bh[e][1], bl[e][1]);
#pragma unroll
                for (int e = 0; e < 4; ++e) mma8(part[e], al[i], bh[e][0], bh[e][1]);
#pragma unroll
                for (int e = 0; e < 4; ++e) mma8(part[e], ah[i], bl[e][0], bl[e][1]);
#pragma unroll
                for (int e = 0; e < 4; ++e) mma8(part[e], ah[i], bh[e][0], bh[e][1]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int k = 0; k < 4; ++k) o[d / 8 + e][k] += part[e][k];
        }
    }
};

// bf16 operands.
template <int D>
struct CoreBf16 {
    using T = __nv_bfloat16;
    static constexpr int BN = D == 128 ? 32 : 64;
    static constexpr int CTAS = 3;
    static constexpr int QS = 2 * D, VS = 2 * D;
    static constexpr bool LOOK_ALL = false;
    static __device__ __forceinline__ int q_at(int row, int chunk) {
        return row * QS + 16 * (chunk ^ (row & 7));
    }
    static __device__ __forceinline__ int v_at(int row, int chunk) { return q_at(row, chunk); }
    static __device__ __forceinline__ int column(int i, int c, int t) { return 8 * i + 2 * t + c; }
    static __device__ __forceinline__ bool odd(const void* chunk) {
        // 0 * x summed up is NaN as soon as one x is not finite
        const uint4 v = *static_cast<const uint4*>(chunk);
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
        const __nv_bfloat162 zero = __floats2bfloat162_rn(0.f, 0.f);
        __nv_bfloat162 z = zero;
#pragma unroll
        for (int e = 0; e < 4; ++e) z = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&u[e]), zero, z);
        const float2 f = __bfloat1622float2(z);
        return f.x + f.y != 0.f;
    }
    static __device__ __forceinline__ void clamp(__nv_bfloat16&) {}

    static __device__ __forceinline__ void scores(float (&s)[BN / 8][4], const unsigned char* sq,
                                                  const unsigned char* k, int warp, int lane) {
        const uint32_t qa = smem_addr(sq), ka = smem_addr(k);
#pragma unroll
        for (int d = 0; d < D / 16; ++d) {
            uint32_t a[4];
            ldmatrix_x4(qa + q_at(16 * warp + (lane & 15), 2 * d + (lane >> 4)), a[0], a[1], a[2], a[3]);
            uint32_t b[BN / 16][4];  // (all on their way before the first product waits)
#pragma unroll
            for (int i = 0; i < BN / 16; ++i)
                ldmatrix_x4(ka + q_at(8 * (2 * i + (lane >> 4)) + (lane & 7), 2 * d + ((lane >> 3) & 1)), b[i][0],
                            b[i][1], b[i][2], b[i][3]);
#pragma unroll
            for (int i = 0; i < BN / 16; ++i) {
                mma_bf16_16816(s[2 * i], a[0], a[1], a[2], a[3], b[i][0], b[i][1]);
                mma_bf16_16816(s[2 * i + 1], a[0], a[1], a[2], a[3], b[i][2], b[i][3]);
            }
        }
    }

    static __device__ __forceinline__ void values(float (&o)[D / 8][4], const float (&s)[BN / 8][4],
                                                  const unsigned char* v, int lane) {
        const uint32_t va = smem_addr(v);
#pragma unroll
        for (int k = 0; k < BN / 16; ++k) {
            const uint32_t a[4] = {pack(s[2 * k][0], s[2 * k][1]), pack(s[2 * k][2], s[2 * k][3]),
                                   pack(s[2 * k + 1][0], s[2 * k + 1][1]), pack(s[2 * k + 1][2], s[2 * k + 1][3])};
#pragma unroll
            for (int d = 0; d < D / 8; d += 8) {
                uint32_t b[4][4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    ldmatrix_x4_trans(va + v_at(16 * k + (lane & 15), d + 2 * i + (lane >> 4)), b[i][0], b[i][1],
                                      b[i][2], b[i][3]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    mma_bf16_16816(o[d + 2 * i], a[0], a[1], a[2], a[3], b[i][0], b[i][1]);
                    mma_bf16_16816(o[d + 2 * i + 1], a[0], a[1], a[2], a[3], b[i][2], b[i][3]);
                }
            }
        }
    }
    static __device__ __forceinline__ uint32_t pack(float x, float y) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
};

template <class C, int D>
struct Cfg {
    static constexpr int STAGE = C::BN * (C::QS + C::VS);  // k, then v
    static constexpr int LO = D + 4;                       // row stride (floats) of a part of O
    static constexpr int WORK = BM * C::QS + 2 * STAGE, PART = BM * LO * 4 + BM * 8;
    static constexpr int MARKS = WORK > PART ? WORK : PART;  // (the part replaces q and the stages)
    static constexpr int SMEM = MARKS + 3 * D * 4;
};

__device__ __forceinline__ void store4(float* at, float4 v) { *reinterpret_cast<float4*>(at) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* at, float4 v) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(at) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

template <class C, int D, int B>
__global__ void __launch_bounds__(kThreads, C::CTAS) pa_prefill_mma_kernel(const PrefillParams p) {
    pdl_trigger();
    pdl_wait();
    using T = typename C::T;
    using L = Cfg<C, D>;
    constexpr int BN = C::BN;
    extern __shared__ __align__(128) unsigned char smem[];
    unsigned char* sq = smem;
    unsigned char* ring = sq + BM * C::QS;
    int* marks = reinterpret_cast<int*>(smem + L::MARKS);  // first NaN, +inf, -inf per column
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
    constexpr int E = 16 / sizeof(T), CPR = D / E, RPP = kThreads / CPR;  // chunks per row, rows per pass
    const int cc = tid % CPR, cr = tid / CPR;
    const uint32_t sq_at = smem_addr(sq), ring_at = smem_addr(ring);
    const T* q = static_cast<const T*>(p.q);
    const T* kb = static_cast<const T*>(p.k_base) + p.tile_off + (long long)kvh * p.s_head + E * cc;
    const T* vb = static_cast<const T*>(p.v_base) + p.tile_off + (long long)kvh * p.s_head + E * cc;
    constexpr int PAGES = BN > B ? BN / B : 1;
    int page[PAGES], ids[PAGES];   // the next tile's pages (-1: none); ids as read, one tile ahead
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
            const uint32_t st = ring_at + (kt & 1) * L::STAGE;
#pragma unroll
            for (int r = 0; r < BN; r += RPP) {
                const int key = r + cr, blk = page[BN > B ? r / B : 0];  // (RPP divides B)
                const bool in = blk >= 0 && kt * BN + key < n;
                const int row = (BN < B ? kt * BN + key : key) % B;
                const long long off = in ? (long long)blk * p.s_blk + row * D : 0;
                cp16(st + C::q_at(key, cc), kb + off, in);
                cp16(st + BN * C::QS + C::v_at(key, cc), vb + off, in);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    look_up(kt0);  // (under the addresses of q)
    for (int r = cr; r < BM; r += RPP) {
        const int f = row0 + r;
        const bool live = r < rows;
        const int tok = live ? token(f) : 0;
        cp16(sq_at + C::q_at(r, cc),
             live ? q + ((long long)(start + tok) * p.H + kvh * p.G + f - tok * p.G) * D + E * cc : q, live);
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
    bool marked = false;  // (for the whole CTA)
    const int tile_pos = first_pos + token(row0);  // the tile's first row's position

    for (int kt = kt0; kt < kt1; ++kt) {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        unsigned char* sk = ring + (kt & 1) * L::STAGE;
        unsigned char* sv = sk + BN * C::QS;
        const int t0 = kt * BN;
        // (some row of the tile does not see all of it)
        const bool partly = t0 + BN - 1 > tile_pos;
        bool odd = false, any_odd = false;
        if (C::LOOK_ALL || partly) {
            // values that are not finite, in what this thread copied
#pragma unroll
            for (int r = 0; r < BN; r += RPP) odd |= C::odd(sv + C::v_at(r + cr, cc));
            any_odd = __syncthreads_or(odd);
        } else {
            __syncthreads();
        }
        // (tile kt is in for all, and the other stage has been read)
        bool there[PAGES], all_there = true;
#pragma unroll
        for (int u = 0; u < PAGES; ++u) there[u] = page[u] >= 0, all_there = all_there && there[u];
        copy(kt + 1);
        if (any_odd) {
            marked = true;
            if (odd)
                for (int r = cr; r < BN; r += RPP)
                    for (int e = 0; e < E; ++e) {
                        T& x = reinterpret_cast<T*>(sv + C::v_at(r, cc))[e];
                        const float v = static_cast<float>(x);
                        if (isfinite(v)) {
                            C::clamp(x);
                            continue;
                        }
                        atomicMin(marks + (v != v ? 0 : v > 0.f ? D : 2 * D) + E * cc + e, t0 + r);
                        x = T(0.f);
                    }
            __syncthreads();
        }
        if (16 * warp >= rows) continue;  // (none of the warp's rows are there)

        float s[BN / 8][4];
#pragma unroll
        for (int i = 0; i < BN / 8; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) s[i][k] = 0.f;
        C::scores(s, sq, sk, warp, lane);
        // weights: the keys of s[i][2 h + c] are t0 + 8 i + 2 t + c, its row pos[h]
#pragma unroll
        for (int i = 0; i < BN / 8; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) s[i][k] *= p.qscale;
        if (partly || !all_there) {
#pragma unroll
            for (int i = 0; i < BN / 8; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (t0 + 8 * i + 2 * t + (k & 1) > pos[k >> 1] || !there[BN > B ? 8 * i / B : 0])
                        s[i][k] = -INFINITY;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float mt = -INFINITY;
#pragma unroll
            for (int i = 0; i < BN / 8; ++i) mt = fmaxf(mt, fmaxf(s[i][2 * h], s[i][2 * h + 1]));
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
        C::values(o, s, sv, lane);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();  // the marks; and q and the stages are free
    float* part = reinterpret_cast<float*>(smem);  // this CTA's part of O
    float2* part_ml = reinterpret_cast<float2*>(part + BM * L::LO);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        l[h] += __shfl_xor_sync(kFullMask, l[h], 1);
        l[h] += __shfl_xor_sync(kFullMask, l[h], 2);
        const int r = 16 * warp + g + 8 * h;  // (rows that are not there: into their own places)
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
#pragma unroll
            for (int c = 0; c < 2; ++c) part[r * L::LO + C::column(i, c, t)] = o[i][2 * h + c];
        if (marked) {
            __syncwarp();  // (column t of all, by the four threads of the row)
            for (int col = t; col < D; col += 4) {
                const bool nan = marks[col] <= pos[h], up = marks[D + col] <= pos[h],
                           down = marks[2 * D + col] <= pos[h];
                if (nan || up || down)
                    part[r * L::LO + col] = nan || (up && down) ? NAN : up ? INFINITY : -INFINITY;
            }
        }
        if (t == 0) part_ml[r] = make_float2(m[h], l[h]);
    }

    // ---- the cluster's parts: each CTA joins its share of the rows ----
    cg::cluster_group cluster = cg::this_cluster();
    if (p.cluster > 1)
        cluster.sync();
    else
        __syncthreads();
    const int rank = p.cluster > 1 ? (int)cluster.block_rank() : 0;
    const int groups = p.splits / p.cluster;
    constexpr int LPR = D / 4, ROWS = kThreads / LPR;  // lanes per row, rows per pass
    const int c4 = tid % LPR;
    for (int x = rank * ROWS + tid / LPR; x < rows; x += p.cluster * ROWS) {
        const int f = row0 + x, tok = token(f);
        const long long orow = (long long)(start + tok) * p.H + kvh * p.G + f - tok * p.G;
        Joined j;
        float2 ml[8];
        float4 v[8];
#pragma unroll
        for (int z = 0; z < 8; ++z) {
            if (z >= p.cluster) break;
            ml[z] = p.cluster > 1 ? *cluster.map_shared_rank(part_ml + x, z) : part_ml[x];
            const float4* at = reinterpret_cast<const float4*>(part + x * L::LO) + c4;
            v[z] = p.cluster > 1 ? *cluster.map_shared_rank(at, z) : *at;
        }
#pragma unroll
        for (int z = 0; z < 8; ++z)
            if (z < p.cluster) j.add(ml[z], v[z]);
        if (groups == 1) {
            store4(static_cast<T*>(p.out) + orow * D + 4 * c4, j.out());
        } else {
            const long long prow = (long long)(blockIdx.y / p.cluster) * p.num_tokens * p.H + orow;
            reinterpret_cast<float4*>(p.part_o)[prow * LPR + c4] = j.o;
            if (c4 == 0) reinterpret_cast<float2*>(p.part_ml)[prow] = make_float2(j.m, j.l);
        }
    }
    if (p.cluster > 1) cluster.sync();  // (no CTA leaves while others read its part)
}

// Joins the clusters' parts of every row of a sequence: D / 4 lanes a row, up to
// eight parts in flight.
constexpr int kJoinThreads = 128;
template <class T, int D>
__global__ void __launch_bounds__(kJoinThreads) pa_prefill_mma_join_kernel(const PrefillParams p) {
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
    store4(static_cast<T*>(p.out) + row * D + 4 * lane, j.out());
}

template <class C, int D, int B>
cudaError_t launch_inst(const PrefillParams& p, cudaStream_t s) {
    auto kern = pa_prefill_mma_kernel<C, D, B>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         Cfg<C, D>::SMEM);
    if (e != cudaSuccess) return e;
    const long long ctas = ((long long)p.num_tokens * p.G / BM + p.batch) * p.Hkv;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas, p.splits);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Cfg<C, D>::SMEM;
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
    return launch_pdl(pa_prefill_mma_join_kernel<typename C::T, D>, dim3((unsigned)((rows + RPC - 1) / RPC)),
                      dim3(kJoinThreads), 0, s, p);
}

}  // namespace

bool prefill_supported(int dtype, int D, int B) {
    return (dtype == 0 || dtype == 1) && (D == 64 || D == 128) && (B == 16 || B == 32);
}

// Whether a call on a bf16 pool takes this kernel: the shorter of both estimates, in
// us.  This one starts in 4 and takes 0.75 us of an SM for 64 rows x 64 keys of
// head_dim 64 (1.7 of 128); the tcgen05 kernel and its join take 9 (12 where
// every 256 rows' keys are cut among SMs), and 1.45 us for 256 rows x 128 keys (0.95
// for up to 128 rows of 64), three such more per 256 rows.  (Measured, this / tcgen05: one token
// over 100 keys, 16 heads on 2 of 64, 4.8 / 8.9; a prompt of 128 6.6 / 9.7, of 512 11.9
// / 14.3, of 1,024 19.0 / 17.9; 32 sequences of 5 tokens over 2,000 18.7 / 21.6; 32
// heads on 8 of 128: 8 sequences of one token over 1,000 13.1 / 19.6, a prompt of 128
// 10.1 / 12.0, of 512 22.1 / 20.7, 8 of 128 24.1 / 14.8.)
//   The lengths are on the device, so the tables' width stands for them here and in the
// splits below.  In a table of 8,192 blocks, far wider than the contexts, short calls
// take tcgen05 where this kernel is the faster: one token over 100 keys 8.2 / 11.1 (of
// 128: 7.9 / 13.0), 8 of one token over 1,000 8.6 / 13.8 (17.3 / 18.6), a prompt of 128 7.8
// / 12.3 (but 17.0 / 13.2); fp32, cut finer than its keys ask for, 9.3 in place of 6.0.
bool prefill_mma_preferred(int G, int Hkv, int batch, int num_tokens, int maxb, int D, int B,
                           int num_sms) {
    const double keys = (double)maxb * B, rows = (double)num_tokens * G;
    const double here = 4 + (rows / 64 + batch) * Hkv * (keys / 64) * (D == 64 ? 0.75 : 1.7) / num_sms;
    const double pairs = (rows / 256 + batch) * Hkv;
    const double tile = D == 64 && rows <= 128.0 * batch ? 0.95 : 1.45;
    const double there = (pairs < num_sms ? 12 : 9) + pairs * (3 + keys / 128) * tile / num_sms;
    return here < there;
}

// Parts of each context (the host knows the tables' width, not the lengths).  Up to
// eight are a cluster, which joins them by itself: of 1, 2, 4 and 8 the one with the
// shortest estimate.  A part takes its key tiles and 2.5 more (start, join); an SM's
// share of them takes 0.62 of their times' sum, for three run at once, and half a part
// more until all have ended.  (fp32, 1 / 2 / 4 / 8 parts: 500 tokens of 16 heads of 128
// behind 7,300, 125 row tiles, 1460 / 954 / 707 / 677 us; 4 sequences of up to 130 tokens, 38
// row tiles of 14 key tiles, 29.0 / 22.6 / 18.6 / 21.6; 24 of up to 212 behind 2,000 - 2,800, 672
// row tiles, 917 / 781 / 779 / 843.)  More than eight take a second launch: where two
// CTAs per SM ask for 16 and each has a tile (4 tokens over 30,000 keys: 152 parts 30
// us, 256 33).
int prefill_mma_splits(int dtype, int G, int Hkv, int batch, int num_tokens, int maxb, int D, int B,
                       int num_sms, int* cluster) {
    const int BN = dtype == 1 ? (D == 64 ? CoreBf16<64>::BN : CoreBf16<128>::BN)
                              : (D == 64 ? CoreF32<64>::BN : CoreF32<128>::BN);
    const long long tiles = ((long long)num_tokens * G / BM + batch) * Hkv;
    const long long keys = ((long long)maxb * B + BN - 1) / BN;  // tiles
    if (tiles <= 0) return *cluster = 1;
    const long long wide = std::min({2 * num_sms / tiles, keys, 256LL});
    if (wide >= 16) {
        *cluster = 8;
        return (int)wide / 8 * 8;
    }
    double best = 0;
    for (int n = 1; n <= 8 && n <= keys; n *= 2) {
        const double share = (double)tiles * n / num_sms;
        const double time = ((double)keys / n + 2.5) * std::max(1.0, 0.62 * share + 0.5);
        if (n == 1 || time < best) best = time, *cluster = n;
    }
    return *cluster;
}

cudaError_t launch_prefill_mma(const PrefillParams& p, int dtype, int D, int B, cudaStream_t s) {
    if (dtype == 1) {
        if (D == 64 && B == 16) return launch_inst<CoreBf16<64>, 64, 16>(p, s);
        if (D == 64 && B == 32) return launch_inst<CoreBf16<64>, 64, 32>(p, s);
        if (D == 128 && B == 16) return launch_inst<CoreBf16<128>, 128, 16>(p, s);
        if (D == 128 && B == 32) return launch_inst<CoreBf16<128>, 128, 32>(p, s);
    } else {
        if (D == 64 && B == 16) return launch_inst<CoreF32<64>, 64, 16>(p, s);
        if (D == 64 && B == 32) return launch_inst<CoreF32<64>, 64, 32>(p, s);
        if (D == 128 && B == 16) return launch_inst<CoreF32<128>, 128, 16>(p, s);
        if (D == 128 && B == 32) return launch_inst<CoreF32<128>, 128, 32>(p, s);
    }
    return cudaErrorNotSupported;
}

}  // namespace pa
