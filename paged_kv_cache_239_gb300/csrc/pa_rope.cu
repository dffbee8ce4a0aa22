// pa_rope.cu -- new tokens on their way into the cache: per-head RMS norm of
// queries and keys, rotary position embedding, and the append of K and V, in
// one pass over the projections' output.
//
// Token t of sequence b (n_b new ones, this the i-th) stands at position
// p = context_lens[b] - n_b + i.  For a query or key head x of D elements
//   y_d = x_d * rsqrt(mean(x^2) + eps) * w_d                  (w given; else y = x)
//   (y_a, y_b) -> A (y_a cos(p f_j) - y_b sin(p f_j), y_a sin(p f_j) + y_b cos(p f_j))
// for the pairs j < r/2 of the first r elements: (a, b) = (2j, 2j + 1) when
// interleaved, (j, j + r/2) in halves.  Everything is fp32 from the load to the
// one rounding at the store.
//
// The angle: p f_j / 2 pi in turns is only needed modulo 1, so f_j / 2 pi is
// kept as a 64-bit binary fraction and multiplied by p in wrapping integer
// arithmetic: exact modulo 1 up to p * 2^-64 turns plus the fraction's own
// rounding, where an fp32 product would be off by p f_j 2^-24 radians (0.008 at
// p = 131072).  The top 32 bits, as a signed fraction of half a turn, go to
// sincospif.
//
// What bounds it: bytes, (H + 2 Hkv) rows read and written per token, and close
// behind them the instructions (about 100 for a lane's 32 bytes).  A row stays in
// registers; a lane holds two 16-byte chunks of it, the two that its pairs lie in,
// so that only the norm's sum is exchanged (with one chunk per lane and the partner
// elements by shuffle the times below were 45.0 and 18.0 us).  A warp serves one
// token and a share of its rows: it finds the token's place and computes its lanes'
// sines once for all of them, with the first rows' loads under way.  Two passes are
// worked on while two are loaded (one each: 48.6 and 20.7 us; four: 51.7 and 20.3,
// registers); CTAs of 32, 64 and 128 threads are within 2 %.
//
// 9,260 bf16 tokens of 8 prompts with 32 + 2 x 8 heads of 128: 41.7 us, 5.4 TB/s of
// the bytes it cannot do without (82 % of a plain copy's rate); 1,027 fp32 tokens of
// 64 sequences with 32 + 2 x 32 heads of 128, no norm, 101 MB: 18.3 us on cold caches (82
// %), 16.4 again and again on the same data, of which L2 holds a part; one token each
// of 32 sequences: 2.5 us, the latency of a launch and three dependent loads.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

constexpr int kRopeThreads = 64;

template <typename T>
struct Chunk;  // 16 bytes of a row as floats

template <>
struct Chunk<float> {
    static constexpr int E = 4;
    static __device__ __forceinline__ void unpack(const uint4& w, float* x) {
        x[0] = __uint_as_float(w.x), x[1] = __uint_as_float(w.y);
        x[2] = __uint_as_float(w.z), x[3] = __uint_as_float(w.w);
    }
    static __device__ __forceinline__ uint4 pack(const float* x) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                          __float_as_uint(x[3]));
    }
};

template <>
struct Chunk<__nv_bfloat16> {
    static constexpr int E = 8;
    static __device__ __forceinline__ void unpack(const uint4& w, float* x) {
        const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 f = bf16x2_to_float2(v[k]);
            x[2 * k] = f.x, x[2 * k + 1] = f.y;
        }
    }
    static __device__ __forceinline__ uint4 pack(const float* x) {
        uint32_t v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * k], x[2 * k + 1]);
            v[k] = *reinterpret_cast<const uint32_t*>(&h);
        }
        return make_uint4(v[0], v[1], v[2], v[3]);
    }
};

// The number of starts[1 .. batch] that are <= t: the sequence of token t
// (batch for a token behind the last sequence).  The whole warp counts, each
// lane a 32nd of the array.
__device__ __forceinline__ int find_sequence(const int* starts, int batch, int t, int lane) {
    int n = 0;
    for (int b = lane; b < batch; b += 32) n += ld_dep(starts + 1 + b) <= t ? 1 : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(kFullMask, n, o);
    return n;
}

template <typename T, int D, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads) pa_norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
    pdl_trigger();
    pdl_wait();
    using C = Chunk<T>;
    constexpr int E = C::E;
    constexpr int LPR = D / E / 2;   // lanes per row, two chunks each
    constexpr int RPW = 32 / LPR;    // rows per warp and pass
    constexpr int U = 2;             // passes in flight
    const int lane = threadIdx.x & 31;
    const unsigned w = blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
    const int t = (int)(w / (unsigned)p.splits);
    const int split = (int)(w % (unsigned)p.splits);
    if (t >= p.num_tokens) return;
    // this lane's chunks of its row: a pair's elements lie both in them, and its angles
    // are l E .. l E + E - 1 (what does not turn is dealt out behind what does)
    const int l = lane % LPR, sub = lane / LPR;
    const int half = p.rotary / E / 2;
    const bool turns = l < half;
    const int c0 = INTERLEAVED ? 2 * l : turns ? l : 2 * l;
    const int c1 = INTERLEAVED || !turns ? c0 + 1 : l + half;
    const int rows = p.H + 2 * p.Hkv;
    const int step = p.splits * RPW;

    // This lane's chunks of row r (queries, keys, values in that order).
    auto load = [&](int r, uint4 (&to)[2]) {
        to[0] = to[1] = make_uint4(0, 0, 0, 0);
        if (r >= rows) return;
        const bool is_q = r < p.H, is_k = !is_q && r < p.H + p.Hkv;
        const T* src = is_q ? static_cast<const T*>(p.q) + (long long)t * p.q_stride + (long long)r * D
                       : is_k ? static_cast<const T*>(p.k) + (long long)t * p.k_stride +
                                    (long long)(r - p.H) * D
                              : static_cast<const T*>(p.v) + (long long)t * p.v_stride +
                                    (long long)(r - p.H - p.Hkv) * D;
        to[0] = ld_dep(reinterpret_cast<const uint4*>(src) + c0);
        to[1] = ld_dep(reinterpret_cast<const uint4*>(src) + c1);
    };
    // the first rows are on their way while the token's place is looked up
    uint4 raw[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u) load(split * RPW + sub + u * step, raw[u]);

    // ---- where the token stands ----
    int b = t, s0 = t, n_new = 1;
    if (p.starts != nullptr) {
        b = find_sequence(p.starts, p.batch, t, lane);
        if (b >= p.batch) return;    // behind the last sequence: left as it is
        s0 = ld_dep(p.starts + b);
        n_new = ld_dep(p.starts + b + 1) - s0;
    }
    const int n = ld_dep(p.lens + b);
    const int i = t - s0;
    const bool good = n >= 0 && n <= p.maxb * p.B && i >= 0 && i < n_new && n_new <= n;
    if (!good && split == 0 && lane == 0) atomicOr(p.status, kStatusBadLength);
    const int pos = good ? n - n_new + i : 0;
    int blk = good ? ld_dep(p.bt + (long long)b * p.maxb + pos / p.B) : -1;
    if (good && (blk < 0 || blk >= p.num_blocks)) {
        if (split == 0 && lane == 0) atomicOr(p.status, kStatusBadBlock);
        blk = -1;
    }
    const long long slot = (long long)blk * p.s_blk + p.tile_off + (long long)(pos % p.B) * D;
    const bool norm = p.q_weight != nullptr;
    uint4 wq[2], wk[2];
    wq[0] = wq[1] = wk[0] = wk[1] = make_uint4(0, 0, 0, 0);
    if (norm) {
        wq[0] = ld_dep(static_cast<const uint4*>(p.q_weight) + c0);
        wq[1] = ld_dep(static_cast<const uint4*>(p.q_weight) + c1);
        wk[0] = ld_dep(static_cast<const uint4*>(p.k_weight) + c0);
        wk[1] = ld_dep(static_cast<const uint4*>(p.k_weight) + c1);
    }

    // ---- this lane's sines ----
    float cs[E], sn[E];
    if (turns) {
#pragma unroll
        for (int k = 0; k < E; ++k) {
            const unsigned long long x = (unsigned long long)pos * p.freq[l * E + k];
            const float half_turns = (float)(int)(x >> 32) * 4.656612873077393e-10f;  // 2^-31
            sincospif(half_turns, &sn[k], &cs[k]);
            sn[k] *= p.amplitude, cs[k] *= p.amplitude;
        }
    }

    for (int r0 = split * RPW; r0 < rows; r0 += U * step) {
        uint4 next[U][2];
#pragma unroll
        for (int u = 0; u < U; ++u) load(r0 + sub + (U + u) * step, next[u]);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = r0 + sub + u * step;
            if (r0 + u * step >= rows) break;  // (the whole warp)
            const bool is_q = r < p.H, is_k = !is_q && r < p.H + p.Hkv;
            float x[2][E];
            C::unpack(raw[u][0], x[0]);
            C::unpack(raw[u][1], x[1]);
            if (norm) {
                float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int k = 0; k < E; k += 2) {
                        const float2 v = make_float2(x[h][k], x[h][k + 1]);
                        s2 = fma2(v, v, s2);
                    }
                float ss = s2.x + s2.y;
#pragma unroll
                for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(kFullMask, ss, o);
                const float rs = rsqrtf(fmaf(ss, 1.f / D, p.eps));
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float wv[E];
                    C::unpack(is_q ? wq[h] : wk[h], wv);
#pragma unroll
                    for (int k = 0; k < E; k += 2) {
                        const float2 v = mul2(mul2(make_float2(x[h][k], x[h][k + 1]), make_float2(rs, rs)),
                                              make_float2(wv[k], wv[k + 1]));
                        x[h][k] = v.x, x[h][k + 1] = v.y;
                    }
                }
            }
            if (turns) {  // (the rest passes as it is, be it infinite)
                if constexpr (INTERLEAVED) {
#pragma unroll
                    for (int k = 0; k < E; ++k) {
                        float &a = x[2 * k / E][2 * k % E], &d = x[2 * k / E][2 * k % E + 1];
                        const float y = a * cs[k] - d * sn[k];
                        d = a * sn[k] + d * cs[k];
                        a = y;
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < E; k += 2) {
                        const float2 a = make_float2(x[0][k], x[0][k + 1]), d = make_float2(x[1][k], x[1][k + 1]);
                        const float2 c = make_float2(cs[k], cs[k + 1]), s = make_float2(sn[k], sn[k + 1]);
                        const float2 y = fma2(mul2(d, s), make_float2(-1.f, -1.f), mul2(a, c));
                        const float2 z = fma2(d, c, mul2(a, s));
                        x[0][k] = y.x, x[0][k + 1] = y.y, x[1][k] = z.x, x[1][k + 1] = z.y;
                    }
                }
            }
            if (r >= rows) continue;
            if (is_q) {
                uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(p.q_out) + ((long long)t * p.H + r) * D);
                dst[c0] = good ? C::pack(x[0]) : make_uint4(0, 0, 0, 0);
                dst[c1] = good ? C::pack(x[1]) : make_uint4(0, 0, 0, 0);
            } else if (blk >= 0) {
                const int h = is_k ? r - p.H : r - p.H - p.Hkv;
                uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(is_k ? p.k_base : p.v_base) + slot +
                                                      (long long)h * p.s_head);
                dst[c0] = is_k ? C::pack(x[0]) : raw[u][0];
                dst[c1] = is_k ? C::pack(x[1]) : raw[u][1];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) raw[u][0] = next[u][0], raw[u][1] = next[u][1];
    }
}

template <typename T, int D>
cudaError_t launch_d(const NormRopeParams& p, int grid, cudaStream_t s) {
    return p.interleaved
               ? launch_pdl(pa_norm_rope_kernel<T, D, true>, dim3(grid), dim3(kRopeThreads), 0, s, p)
               : launch_pdl(pa_norm_rope_kernel<T, D, false>, dim3(grid), dim3(kRopeThreads), 0, s, p);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams& p_in, int dtype, int D, int num_sms,
                             cudaStream_t s) {
    NormRopeParams p = p_in;
    const int elt = dtype == 1 ? 2 : 4;
    const int rpw = 64 / (D * elt / 16);
    const long long groups = (p.H + 2LL * p.Hkv + rpw - 1) / rpw;
    // warps per token: one, unless that leaves SMs without eight warps
    long long splits = (8LL * num_sms + p.num_tokens - 1) / p.num_tokens;
    if (splits > groups) splits = groups;
    p.splits = (int)splits;
    const long long warps = splits * p.num_tokens;
    const long long grid = (warps + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
    if (warps > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    if (dtype == 1 && D == 64) return launch_d<__nv_bfloat16, 64>(p, (int)grid, s);
    if (dtype == 1 && D == 128) return launch_d<__nv_bfloat16, 128>(p, (int)grid, s);
    if (dtype == 0 && D == 64) return launch_d<float, 64>(p, (int)grid, s);
    if (dtype == 0 && D == 128) return launch_d<float, 128>(p, (int)grid, s);
    return cudaErrorNotSupported;
}

}  // namespace pa
