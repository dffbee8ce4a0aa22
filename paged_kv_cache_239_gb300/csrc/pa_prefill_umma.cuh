// pa_prefill_umma.cuh -- attention of several new tokens per sequence over a
// bf16 paged cache on the 5th-generation tensor cores: the calls that are not short.
//
//   out_t = sum_{s <= p_t} softmax_s(scale q_t . k_s) v_s,
//   p_t = context_lens[b] - n_b + i for the i-th of sequence b's n_b new tokens;
// TREE: over the s < context_lens[b] - n_b and the new tokens whose bits are set in the
// token's mask.
//
// The query heads of a KV head's group share its keys, so the rows of a tile
// are (token, head of the group) in that order, flattened: row r is token r / G,
// head r % G, whatever G is.  A pair is 256 consecutive rows of one (sequence,
// KV head): two row tiles of 128, the M of tcgen05.mma, that run against the
// same stream of 128-key tiles.
//
// Schedule: the work is all pairs' key tiles in order of sequence, KV head and
// rows (a pair is charged kPairUnits more for its fixed cost), and each of the
// persistent CTAs, one per SM, takes an equal contiguous share of it.  Prompts
// of any mix of lengths and a few rows over a long context alike fill the GPU;
// a pair that the shares cut leaves unnormalised partials that the join kernel
// merges.
//
// Roles, connected by mbarriers:
//  * warps 0 and 3: K and V tiles into one ring of stages, K(0) V(0) K(1) V(1)
//    ..., in 16-row boxes by 5-D tensor-map TMA, pages from the block table;
//  * warp 1: tensor memory, and one thread issuing for each key tile i and row
//    tile j  O_j += P_j(i) V(i), then S_j(i + 1) = Q_j K(i + 1)^T: the softmax of
//    one row tile runs under the products of the other;
//  * warp 2: Q of the next pair, by tensor map or row by row (cp.async), and the
//    look over V (below);
//  * warps 4-7 and 8-11: softmax of row tile 0 and 1, one row per thread, so no
//    exchange between threads: S from tensor memory, running maximum (raised,
//    and O rescaled, only when a score exceeds it by more than 2^8: any
//    reference point gives the same normalised result), P as bf16 over S's own
//    columns, sums in fp32, and at the end of a piece O / l to the output.  A pair
//    with one row tile and several key tiles is served by both groups in turns, each
//    with an S and an O of its own: the chain S, softmax, P V of one tile, which is
//    longer than its K and V take to arrive, runs under the other group's; at the end
//    both groups learn the other's sums, and each joins half of the columns.
// P in bf16: its rounding (2^-9 relative on average over many keys) is of the
// size of the output's own; the sum l takes the weights before that rounding.
//
// What a row does not see must not reach it even through 0 * NaN: in tiles that
// reach past the pair's first row, the context's end or a bad page, the rows of
// V outside the context are zeroed in shared memory, and values that are not
// finite are zeroed and remembered by column and position, to be put back into
// the rows that see them at the output.
//
// What bounds it.  Long prompts: a pair's tile is 4 x 8 MMAs of 128 x 128 x 16, 2048
// cycles of the tensor pipe, and takes about 2700, since S(i + 1) waits for the
// softmax of S(i) to leave the columns that P stands in, with 512 columns for two
// row tiles' S and O (the exponentials, 2048 cycles of the special-function units,
// run beside).  A prompt of 8192 with 32 heads on 8 of 128: 353 - 358 us in a graph of
// such calls on warm caches, 1.54 PFLOP/s of the causal half (80 % of a large library
// product's burst rate); 382 - 386, 1.43 PFLOP/s, as a call among others.  Measured and
// slower, at a time when this form took 400: two threads to a row 450; two issuing
// threads 480; P handed over in halves 409.  Without the exponentials it took 383.
// Many keys, few rows: bytes; 3 - 5 tokens over 4 contexts of 32,768 to 131,000: 150
// us, 6.3 TB/s (94 % of a plain copy's rate; 167 us without turns), in shares cut to
// the tile.  Short calls:
// latency (pa_prefill_mma.cuh takes the shortest); one token over 100 keys takes 8.7 us,
// of which 2.5 go to the schedule (its code is fetched by every SM), 2.5 to the first
// K tile and its scores, and 2.5 to the join's launch; 8 chunks of up to 513 tokens
// with 16 heads on 2 of 64: 25 us, of which 9 are five to seven tiles.
//
// The shares charge a pair kPairUnits tiles: a tile costs about 2,930 cycles and a
// pair 9,500 more (Q, the first scores, the output).  With 2 the last CTA of a batch
// of short prompts ends after 802,000 cycles, with 3 after 728,000.
#pragma once

#include <cfloat>
#include <climits>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_tcgen05.cuh"
#include "pa_tree_mask.cuh"

namespace pa {

template <int D_, int B_>
struct PrefillCfg {
    static constexpr int D = D_, B = B_;
    static constexpr int TT = 128;                 // keys per tile
    static constexpr int ROWS = 256;               // rows per pair (two tiles of 128)
    static constexpr int NH = D / 64;              // 64-column halves
    static constexpr int HALF = 128 * 128;         // one half of a 128-row tile (bytes)
    static constexpr int TILE = NH * HALF;
    static constexpr int NS = D == 128 ? 5 : 8;   // K/V stages
    static constexpr int OFF_Q = NS * TILE;
    static constexpr int OFF_CTRL = OFF_Q + 2 * TILE;
    // ctrl (bytes): barriers | TMEM address, abort, mark_piece, done[2] | box bits
    // of eight tiles | schedule (72 bytes) | the producers' page ids | pieces [NP] | marks [3][D]
    // (the schedule's scratch before)
    static constexpr int NP = 4;
    static constexpr int TMEM_SLOT = 384, ABORT = 388, MARK_PIECE = 392, DONE = 396, BITS = 404,
                         SCHED = 448, BLOCKS = 528, PIECES = 592, MARKS = 832, SCAN = MARKS;
    // (TREE has no marks: there the groups that serve a row tile in turns exchange their sums)
    static constexpr int SMEM_BYTES = OFF_CTRL + MARKS + 2 * 128 * 8;
    static_assert(3 * 128 * 4 <= 2 * 128 * 8, "marks");
    static constexpr int THREADS = 384;
    // TMEM: S_0, S_1 (P in their first 64 columns), O_0, O_1
    static constexpr int O_COL = 256;
    static constexpr int TMEM_COLS = 512;
    // barriers
    static constexpr int KV_FULL = 0, KV_EMPTY = NS, Q_FULL = 2 * NS, Q_EMPTY = Q_FULL + 2,
                         S_FULL = Q_FULL + 4, P_FULL = Q_FULL + 6,  // three parts, [part][row tile]
                         PV_DONE = Q_FULL + 12, FINAL = Q_FULL + 14,
                         V_LOOK = Q_FULL + 15, V_CLEAN = Q_FULL + 17,  // two each, in turns
                         PC_FULL = Q_FULL + 19, PC_EMPTY = PC_FULL + NP,
                         X_SUMS = PC_EMPTY + NP, X_READ = X_SUMS + 1, NBAR = X_READ + 1;
    static_assert(NBAR * 8 <= TMEM_SLOT && NS <= 11, "ctrl layout");
    static_assert(SMEM_BYTES <= 232448, "shared memory");
};

constexpr int kPairUnits = 3;  // (see above)

// A sequence as the schedule sees it.
struct PfSeq {
    int start, n_new, n, first_pos, rows, tiles;
};

template <int B, bool TREE>
__device__ __forceinline__ PfSeq pf_sequence(const PrefillParams& p, int b, bool* bad) {
    PfSeq s{0, 0, 0, 0, 0, 0};
    *bad = false;
    if (b >= p.batch) return s;
    const int s0 = ld_dep(p.starts + b), s1 = ld_dep(p.starts + b + 1);
    const int n = ld_dep(p.lens + b);
    if (s0 < 0 || s1 < s0 || s1 > p.num_tokens) {
        *bad = true;
        return s;
    }
    s.start = s0, s.n_new = s1 - s0, s.n = n;
    if (n < s.n_new || n > p.maxb * B || n < 0 || (TREE && s.n_new > 32 * p.words)) {
        *bad = true;
        s.n = 0;  // no key is seen: zero rows
    }
    s.first_pos = s.n - s.n_new;
    s.rows = s.n_new * p.G;
    s.tiles = (s.rows + 255) / 256;
    return s;
}

// A sequence in shared memory (16-byte aligned, 24 bytes).
__device__ __forceinline__ void pf_keep(const PfSeq& s, unsigned char* at) {
    *reinterpret_cast<int4*>(at) = make_int4(s.start, s.n_new, s.n, s.first_pos);
    *reinterpret_cast<int2*>(at + 16) = make_int2(s.rows, s.tiles);
}
__device__ __forceinline__ PfSeq pf_kept(const unsigned char* at) {
    const int4 a = *reinterpret_cast<const int4*>(at);
    const int2 b = *reinterpret_cast<const int2*>(at + 16);
    return PfSeq{a.x, a.y, a.z, a.w, b.x, b.y};
}

// x / G for 0 <= x < 2^31 (the host's multiplier: a 32-bit division costs ~30
// instructions, and the set-up runs many).
__device__ __forceinline__ int pf_div(const PrefillParams& p, int x) {
    return (int)(((unsigned long long)(unsigned)x * p.div_mul) >> p.div_shift);
}

// Key tiles of pair i of a sequence (at least one: the pair owes its output).
template <bool TREE>
__device__ __forceinline__ int pf_key_tiles(const PrefillParams& p, const PfSeq& s, int i) {
    const int last = min(s.rows, 256 * (i + 1)) - 1;
    const int see = TREE ? s.n : s.first_pos + pf_div(p, last) + 1;
    return see > 128 ? (see + 127) >> 7 : 1;
}

// a / b, in 32 bits where both fit; out of line (see pf_wait_call).
static __device__ __noinline__ long long pf_div64(long long a, long long b) {
    if ((unsigned long long)(a | b) >> 32) return a / b;
    return (unsigned)a / (unsigned)b;
}

// A piece: key tiles [kt0, kt1) of one pair, as its roles see it.  The K
// producer walks the CTA's share and hands the pieces to the others in a small
// ring in shared memory.
struct alignas(16) PfPiece {
    int kvh, kt0, kt1, nj;   // KV head, key tiles, row tiles (1 or 2; 0: no more pieces)
    int row0, rows, start, first_pos;  // first row of the pair; the sequence's rows, token, position
    int n, pair_pos, b, flags;  // context; position of the pair's first row; sequence
    __device__ __forceinline__ bool whole() const { return flags & 1; }
    __device__ __forceinline__ bool first() const { return flags & 2; }
    // one row tile and several key tiles: both softmax groups serve it in turns
    __device__ __forceinline__ bool turns() const { return nj == 1 && kt1 - kt0 >= 4; }
};

struct PfWalk {
    int b, kvh, i, count;
    long long left, off, gpos;
    PfSeq s;
};

// Units of sequence b0 + lane (all lanes of the warp take part).
template <int B, bool TREE>
__device__ __forceinline__ long long pf_seq_units(const PrefillParams& p, int b, int lane,
                                                  bool report, PfSeq& s) {
    bool bad;
    s = pf_sequence<B, TREE>(p, b, &bad);
    if (bad && report) atomicOr(p.status, kStatusBadLength);
    long long u = 0;
    if constexpr (TREE)  // (all pairs of a sequence see the same keys)
        return s.tiles ? (long long)s.tiles * (kPairUnits + pf_key_tiles<TREE>(p, s, 0)) : 0;
    // (a sequence taken by the whole warp costs what about 32 pairs cost one lane)
    const int lim = 32 * max(1, __popc(__ballot_sync(kFullMask, s.tiles > 16)));
    if (s.tiles <= lim) {
        int v = s.tiles * kPairUnits;
#pragma unroll 1
        for (int i = 0; i < s.tiles; ++i) v += pf_key_tiles<TREE>(p, s, i);
        u = v;
    }
    unsigned big = __ballot_sync(kFullMask, s.tiles > lim);
    while (big) {
        const int f = __ffs(big) - 1;
        big &= big - 1;
        PfSeq o;
        o.n = __shfl_sync(kFullMask, s.n, f);
        o.first_pos = __shfl_sync(kFullMask, s.first_pos, f);
        o.rows = __shfl_sync(kFullMask, s.rows, f);
        o.tiles = __shfl_sync(kFullMask, s.tiles, f);
        long long v = 0;
#pragma unroll 1
        for (int i = lane; i < o.tiles; i += 32) v += kPairUnits + pf_key_tiles<TREE>(p, o, i);
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) v += __shfl_xor_sync(kFullMask, v, x);
        if (lane == f) u = v;
    }
    return u;
}

// The CTA's range of the T units, into `sched`: [0] T, [8] first unit, [16]
// units, [24] offset within the pair, [32] b, [36] KV head, [40] pair, [48] the
// sequence, all for warp 0.  Up to 32 sequences are that warp's, without barriers in
// between.
template <typename C, bool TREE>
__device__ __forceinline__ void pf_schedule(const PrefillParams& p, unsigned char* ctrl) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int nw = p.batch <= 32 ? 1 : C::THREADS / 32;  // warps that take part
    long long* sums = reinterpret_cast<long long*>(ctrl + C::SCAN);
    long long* out = reinterpret_cast<long long*>(ctrl + C::SCHED);
    int* outi = reinterpret_cast<int*>(ctrl + C::SCHED + 32);
    if (warp >= nw) return;
    long long u = 0, mine = 0;
    PfSeq s{0, 0, 0, 0, 0, 0};
#pragma unroll 1
    for (int b0 = 0; b0 < p.batch; b0 += nw * 32) {
        u = pf_seq_units<C::B, TREE>(p, b0 + threadIdx.x, lane, blockIdx.x == 0, s);
        mine += u;
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) mine += __shfl_xor_sync(kFullMask, mine, x);
    long long T = mine;
    if (nw > 1) {
        if (lane == 0) sums[warp] = mine;
        __syncthreads();
        T = 0;
#pragma unroll 1
        for (int w = 0; w < nw; ++w) T += sums[w];
    }
    T *= p.Hkv;
    // (no more shares than units: an empty one inside a cut pair would be taken
    // for a part of it)
    const long long grid = min((long long)gridDim.x, T);
    const long long j = blockIdx.x;
    long long lo = 0, hi = 0;
    if (j < grid) {
        const long long x = pf_div64((j + (lane & 1)) * T + grid - 1, grid);
        lo = __shfl_sync(kFullMask, x, 0), hi = __shfl_sync(kFullMask, x, 1);
    }
    long long before = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < p.batch; b0 += nw * 32) {
        if (p.batch > nw * 32) u = pf_seq_units<C::B, TREE>(p, b0 + threadIdx.x, lane, false, s);
        long long incl = u * p.Hkv;
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) {
            const long long v = __shfl_up_sync(kFullMask, incl, x);
            if (lane >= x) incl += v;
        }
        long long base = before;
        if (nw > 1) {
            __syncthreads();
            if (lane == 31) sums[warp] = incl;
            __syncthreads();
#pragma unroll 1
            for (int w = 0; w < nw; ++w) {
                if (w < warp) base += sums[w];
                before += sums[w];
            }
        }
        const long long at = base + incl - u * p.Hkv;
        if (lo >= at && lo < at + u * p.Hkv && hi > lo) {
            outi[0] = b0 + threadIdx.x;
            const long long h = pf_div64(lo - at, u);
            outi[1] = (int)h;
            out[3] = lo - at - h * u;
            pf_keep(s, ctrl + C::SCHED + 48);
        }
    }
    if (nw > 1)
        __syncthreads();
    else
        __syncwarp();
    if (warp == 0 && hi > lo) {
        // the pair within the sequence and KV head
        s = pf_kept(ctrl + C::SCHED + 48);
        long long off = out[3];
        int i = 0;
        if constexpr (TREE) {
            const int c = kPairUnits + pf_key_tiles<TREE>(p, s, 0);
            i = (int)pf_div64(off, c);
            off -= (long long)i * c;
        }
#pragma unroll 1
        for (int i0 = 0; i0 < s.tiles && !TREE; i0 += 32) {
            const int c = i0 + lane < s.tiles ? kPairUnits + pf_key_tiles<TREE>(p, s, i0 + lane) : 0;
            long long incl = c;
#pragma unroll
            for (int x = 1; x < 32; x <<= 1) {
                const long long v = __shfl_up_sync(kFullMask, incl, x);
                if (lane >= x) incl += v;
            }
            const unsigned hit = __ballot_sync(kFullMask, off >= incl - c && off < incl);
            if (hit) {
                const int f = __ffs(hit) - 1;
                i = i0 + f;
                off -= __shfl_sync(kFullMask, incl, f) - __shfl_sync(kFullMask, c, f);
                break;
            }
            off -= __shfl_sync(kFullMask, incl, 31);
        }
        __syncwarp();
        if (lane == 0) out[3] = off, outi[2] = i;
    }
    if (threadIdx.x == 0) out[0] = T, out[1] = lo, out[2] = hi - lo;
    __syncwarp();
}

// The same for up to 32 sequences of trees, by one warp: all pairs of a sequence cost the
// same, so that its lane knows where they stand.
template <typename C>
__device__ __forceinline__ void tree_schedule(const PrefillParams& p, unsigned char* ctrl) {
    const int lane = threadIdx.x & 31;
    bool bad;
    const PfSeq s = pf_sequence<C::B, true>(p, lane, &bad);
    if (bad && blockIdx.x == 0) atomicOr(p.status, kStatusBadLength);
    const int c = kPairUnits + pf_key_tiles<true>(p, s, 0);
    const long long u = (long long)s.tiles * p.Hkv * c;
    long long incl = u;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
        const long long v = __shfl_up_sync(kFullMask, incl, x);
        if (lane >= x) incl += v;
    }
    const long long T = __shfl_sync(kFullMask, incl, 31);
    const long long grid = min((long long)gridDim.x, T), j = blockIdx.x;
    long long* out = reinterpret_cast<long long*>(ctrl + C::SCHED);
    int* outi = reinterpret_cast<int*>(ctrl + C::SCHED + 32);
    long long x = 0;
    if (j < grid) x = pf_div64((j + (lane & 1)) * T + grid - 1, grid);
    const long long lo = __shfl_sync(kFullMask, x, 0), hi = __shfl_sync(kFullMask, x, 1);
    if (lane == 0) out[0] = T, out[1] = lo, out[2] = hi - lo;
    const long long at = lo - (incl - u);  // within the lane's sequence, if it is this one's
    if (at >= 0 && at < u && hi > lo) {
        const int pair = (int)pf_div64(at, c), h = pair / s.tiles;
        outi[0] = lane, outi[1] = h, outi[2] = pair - h * s.tiles;
        out[3] = at - (long long)pair * c;
        pf_keep(s, ctrl + C::SCHED + 48);
    }
    __syncwarp();
}

template <typename C>
__device__ __forceinline__ void pf_walk_begin(const PrefillParams& p, const unsigned char* ctrl,
                                              PfWalk& w) {
    const long long* in = reinterpret_cast<const long long*>(ctrl + C::SCHED);
    const int* ini = reinterpret_cast<const int*>(ctrl + C::SCHED + 32);
    w.left = in[2], w.count = 0;
    if (w.left <= 0) return;
    w.off = in[3], w.gpos = in[1] - in[3];
    w.b = ini[0], w.kvh = ini[1], w.i = ini[2];
    w.s = pf_kept(ctrl + C::SCHED + 48);
}

// The next piece with work; kvt: the pair's key tiles, gpos: the global unit of
// its first one.
template <typename C, bool TREE>
__device__ __forceinline__ bool pf_walk_next(const PrefillParams& p, PfWalk& w, PfPiece& pc,
                                             int& kvt, long long& gpos) {
    while (w.left > 0) {
        kvt = pf_key_tiles<TREE>(p, w.s, w.i);
        const long long c = kPairUnits + kvt;
        const long long take = min(c - w.off, w.left);
        const int u0 = (int)max(w.off - kPairUnits, 0LL), u1 = (int)(w.off + take - kPairUnits);
        gpos = w.gpos + kPairUnits;
        pc.kvh = w.kvh, pc.kt0 = u0, pc.kt1 = u1;
        pc.row0 = 256 * w.i, pc.rows = w.s.rows, pc.start = w.s.start;
        pc.nj = pc.rows - pc.row0 > 128 ? 2 : 1;
        pc.first_pos = w.s.first_pos, pc.n = w.s.n, pc.b = w.b;
        // (TREE: the last position that all rows see)
        pc.pair_pos = TREE ? pc.first_pos - 1 : pc.first_pos + pf_div(p, pc.row0);
        pc.flags = (u0 == 0 && u1 == kvt ? 1 : 0) | (w.count == 0 ? 2 : 0);
        w.left -= take;
        if (w.off + take == c) {  // on to the next pair
            w.off = 0, w.gpos += c;
            if (++w.i == w.s.tiles) {
                w.i = 0;
                if (++w.kvh == p.Hkv) {
                    w.kvh = 0;
                    while (w.left > 0 && ++w.b < p.batch) {
                        bool bad;
                        w.s = pf_sequence<C::B, TREE>(p, w.b, &bad);
                        if (w.s.tiles > 0) break;
                    }
                    if (w.b >= p.batch) w.left = 0;
                }
            }
        } else {
            w.off += take;
        }
        if (u1 > u0) {
            ++w.count;
            return true;
        }
    }
    pc.nj = 0;
    return false;
}

// 32 consecutive columns of this thread's lane; the values may be used after
// tmem_loaded32 (which names them, so that no use is moved ahead of the wait).
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]),
          "=f"(r[7]), "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]),
          "=f"(r[14]), "=f"(r[15]), "=f"(r[16]), "=f"(r[17]), "=f"(r[18]), "=f"(r[19]),
          "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]), "=f"(r[25]),
          "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_loaded32(float (&r)[32]) {
    asm volatile(""
                 : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]),
                   "+f"(r[6]), "+f"(r[7]), "+f"(r[8]), "+f"(r[9]), "+f"(r[10]), "+f"(r[11]),
                   "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15]), "+f"(r[16]), "+f"(r[17]),
                   "+f"(r[18]), "+f"(r[19]), "+f"(r[20]), "+f"(r[21]), "+f"(r[22]), "+f"(r[23]),
                   "+f"(r[24]), "+f"(r[25]), "+f"(r[26]), "+f"(r[27]), "+f"(r[28]), "+f"(r[29]),
                   "+f"(r[30]), "+f"(r[31]));
}

// True in one thread of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(r));
    return r != 0;
}

// cp.async of one 16-byte chunk (zeros when !valid).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(valid ? 16 : 0)
                 : "memory");
}

template <int N>
__device__ __forceinline__ void regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// umma_wait for waits on the critical path: the timer and the abort flag are
// looked at once in 64 tries.  pf_wait_call is the same out of line, for the
// roles that wait in many places (code competes for the instruction cache).
__device__ __forceinline__ bool pf_wait(uint32_t bar, uint32_t parity, volatile int* abort_all,
                                        unsigned* status) {
#pragma unroll 1
    for (int it = 0; it < 64; ++it)
        if (mbar_try_wait(bar, parity)) return true;
    const unsigned long long t0 = globaltimer_ns();
#pragma unroll 1
    for (uint32_t it = 0; it < (1u << 30); ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((it & 63) != 63) continue;
        if (*abort_all) return false;
        if (globaltimer_ns() - t0 > kWaitLimitNs) break;
    }
    *abort_all = 1;
    atomicOr(status, kStatusTimeout);
    return false;
}
static __device__ __noinline__ bool pf_wait_call(uint32_t bar, uint32_t parity, volatile int* abort_all,
                                          unsigned* status) {
    return pf_wait(bar, parity, abort_all, status);
}

// 32 bytes to a 32-byte aligned address.
__device__ __forceinline__ void store32(void* at, const uint32_t (&v)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// One row's part of a key tile: reads S (128 columns at s_col), writes P over
// S's first 64 columns and adds its sum to l2; ready(k) follows the first two
// quarters of P (k = 0), the third (1) and the last (2).  The first quarters'
// exponentials are taken at the reference point m as it stands, under the
// search for the tile's maximum; raise(max) settles m, and where it had to move
// (true) they are taken again.  With `masked`, only the keys whose bits are set
// in vis (32 to a word) have weight: the others' scores become -inf and their
// weights 0 (qs > 0, and m is never -inf).  False: stop.
template <typename Raise, typename Ready>
__device__ __forceinline__ bool pf_softmax_tile(uint32_t s_col, float qs, bool masked,
                                                const uint32_t (&vis)[4], const float& m, float2& l2,
                                                Raise raise, Ready ready) {
    // (a load of 32 columns takes 600 - 1300 cycles beside the MMAs, four in
    // flight little more: the second half's are under the first's exponentials)
    float x[4][32];
    tmem_ld32(s_col, x[0]);
    tmem_ld32(s_col + 32, x[1]);
    tmem_wait_ld();
    tmem_loaded32(x[0]);
    tmem_loaded32(x[1]);
    tmem_ld32(s_col + 64, x[2]);
    tmem_ld32(s_col + 96, x[3]);
    auto mask = [&](int c) {
#pragma unroll
        for (int k = 0; k < 32; ++k)
            if (!((vis[c] >> k) & 1u)) x[c][k] = -INFINITY;
    };
    if (masked) mask(0), mask(1);
    const float2 qq = make_float2(qs, qs);
    float2 sum = make_float2(0.f, 0.f), mm = make_float2(-m, -m);
    auto quarter = [&](int c) {
        uint32_t pk[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const float2 e = fma2(make_float2(x[c][2 * k], x[c][2 * k + 1]), qq, mm);
            const float2 pv = make_float2(ex2_approx(e.x), ex2_approx(e.y));
            sum = add2(sum, pv);
            pk[k] = pack_bf16x2(pv.x, pv.y);
        }
        tmem_st16(s_col + 16 * c, pk);
    };
    auto max32 = [&](int c) {
        float a[4];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            a[h] = x[c][8 * h];
#pragma unroll
            for (int k = 1; k < 8; ++k) a[h] = fmaxf(a[h], x[c][8 * h + k]);
        }
        return fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3]));
    };
    quarter(0);
    quarter(1);
    float mx = fmaxf(max32(0), max32(1));
    tmem_wait_ld();
    tmem_loaded32(x[2]);
    tmem_loaded32(x[3]);
    if (masked) mask(2), mask(3);
    mx = fmaxf(mx, fmaxf(max32(2), max32(3)));
    // (no key seen: the finite floor)
    const int moved = raise(fmaxf(mx * qs, -FLT_MAX));
    if (moved < 0) return false;
    if (moved > 0) {
        sum = make_float2(0.f, 0.f), mm = make_float2(-m, -m);
        quarter(0);
        quarter(1);
    }
    ready(0);
    quarter(2);
    ready(1);
    quarter(3);
    ready(2);
    l2 = add2(l2, sum);
    return true;
}

// Whether tile kt of a piece reaches past the pair's first row: its V holds
// values that some row must not see, and is looked over before use.
__device__ __forceinline__ bool pf_unclean(const PfPiece& pc, int kt) {
    return 128 * (kt + 1) - 1 > pc.pair_pos;
}

// Where column d of row `row` of the partials is: 32 rows' 8 columns lie together,
// so that a warp (one row per lane) stores whole lines (a pair's part of 64 columns:
// 4,200 cycles row by row).
__device__ __forceinline__ long long pf_part_at(long long row, int D, int d) {
    return (row >> 5) * 32 * D + (d >> 3) * 256 + ((int)row & 31) * 8 + (d & 7);
}

// What a column's remembered values (first positions of a NaN, +inf, -inf) add
// to the output of a row at `pos`.
__device__ __forceinline__ float poison(const int* marks, int D, int d, int pos) {
    const bool n = marks[d] <= pos, a = marks[D + d] <= pos, b = marks[2 * D + d] <= pos;
    return n || (a && b) ? NAN : a ? INFINITY : b ? -INFINITY : 0.f;
}

template <int D, int B, bool TURNS, bool TREE>
__global__ void __launch_bounds__(384, 1)
    pa_prefill_umma_kernel(const PrefillParams p, const __grid_constant__ CUtensorMap tmk,
                           const __grid_constant__ CUtensorMap tmv,
                           const __grid_constant__ CUtensorMap tmq) {
    pdl_trigger();
    using C = PrefillCfg<D, B>;
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t sbase = smem_addr(smem);
    if (sbase & 1023u) {  // (the swizzled tiles need it; there is no other shared memory)
        if (threadIdx.x == 0) atomicOr(p.status, kStatusTimeout);
        return;
    }
    unsigned char* ctrl = smem + C::OFF_CTRL;
    const uint32_t bar0 = sbase + C::OFF_CTRL;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ctrl + C::TMEM_SLOT);
    volatile int* abort_all = reinterpret_cast<volatile int*>(ctrl + C::ABORT);
    PfPiece* pieces = reinterpret_cast<PfPiece*>(ctrl + C::PIECES);
    volatile int* mark_piece = reinterpret_cast<volatile int*>(ctrl + C::MARK_PIECE);
    volatile int* done = reinterpret_cast<volatile int*>(ctrl + C::DONE);  // pieces, per softmax group's warp
    volatile int* box_bits = reinterpret_cast<volatile int*>(ctrl + C::BITS);
    int* marks = reinterpret_cast<int*>(ctrl + C::MARKS);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    static_assert(C::NBAR <= 64, "barriers");
    if (warp == 2 || warp == 3) {  // (a barrier to a lane)
        const int i = threadIdx.x - 64;
        const bool p_full = i >= C::P_FULL && i < C::P_FULL + 6;
        const bool pc_empty = i >= C::PC_EMPTY && i < C::PC_EMPTY + C::NP;
        if (i < C::NBAR) mbar_init(bar0 + 8 * i, p_full ? 4 : pc_empty ? 11 : i >= C::X_SUMS ? 8 : 1);
        if (i == 0) *abort_all = 0, *mark_piece = -1, done[0] = 0, done[1] = 0;
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc(smem_addr(tmem_slot), C::TMEM_COLS);
    // (the schedule of up to 32 trees is warp 0's alone, and runs beside all this)
    const bool early = TREE && p.batch <= 32;
    if (early && warp == 0) {
        pdl_wait();
        tree_schedule<C>(p, ctrl);
    }
    if (warp == 0 && lane == 0) {
        prefetch_tensormap(&tmk);
        prefetch_tensormap(&tmv);
        prefetch_tensormap(&tmq);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();
    // (the K producer alone needs the schedule: with few sequences the other warps are
    // at their first wait, their code fetched, when it hands out the first piece)
    if (!early) pf_schedule<C, TREE>(p, ctrl);
    auto wait = [&](int bar, uint32_t parity) {
        return pf_wait(bar0 + 8 * bar, parity, abort_all, p.status);
    };
    PfPiece pc;
    int np = 0;  // pieces so far (every warp's own count)

    if (warp < 4) {
        regs_dec<104>();
        auto wait = [&](int bar, uint32_t parity) {
            const uint32_t at = bar0 + 8 * bar;
            return mbar_try_wait(at, parity) || pf_wait_call(at, parity, abort_all, p.status);
        };
        // the next piece, by the whole warp
        auto next_piece = [&] {
            const int slot = np % C::NP;
            if (!__all_sync(kFullMask, wait(C::PC_FULL + slot, (np / C::NP) & 1))) return false;
            pc = pieces[slot];
            __syncwarp();
            if (lane == 0) mbar_arrive(bar0 + 8 * (C::PC_EMPTY + slot));
            ++np;
            return pc.nj > 0;
        };
        if (warp == 0 || warp == 3) {
            // ====================================== K tiles (warp 0), V tiles (warp 3)
            const int kv = warp == 0 ? 0 : 1;
            const CUtensorMap* tm = kv ? &tmv : &tmk;
            int* blocks = reinterpret_cast<int*>(ctrl + C::BLOCKS) + 8 * kv;
            int seq = kv;  // the next stage of the ring (K the even, V the odd ones)
            bool aborted = false;
            const uint64_t pol_normal = l2_policy_evict_normal(), pol_first = l2_policy_evict_first();
            if (kv == 0 && lane == 0 && p.cut != nullptr)
                p.cut[2 * blockIdx.x + 1] = make_int4(0, 0, 0, 0);  // (no cut pair yet)
            PfWalk w;
            if (kv == 0) pf_walk_begin<C>(p, ctrl, w);
            while (!aborted) {
                if (kv == 0) {
                    int kvt;
                    long long gpos;
                    const bool more = pf_walk_next<C, TREE>(p, w, pc, kvt, gpos);
                    const int slot = np % C::NP;
                    if (np >= C::NP &&
                        !__all_sync(kFullMask, wait(C::PC_EMPTY + slot, (np / C::NP - 1) & 1)))
                        break;
                    ++np;
                    if (lane == 0) {
                        pieces[slot] = pc;
                        mbar_arrive(bar0 + 8 * (C::PC_FULL + slot));
                        if (more && p.cut != nullptr && !pc.whole() && pc.kt0 == 0) {
                            // this CTA holds the first part of a pair that others go on with
                            const long long T = *reinterpret_cast<const long long*>(ctrl + C::SCHED);
                            const long long last =
                                pf_div64((gpos + kvt - 1) * min((long long)gridDim.x, T), T);
                            p.cut[2 * blockIdx.x] = make_int4(pc.b, pc.kvh, pc.row0, pc.start);
                            p.cut[2 * blockIdx.x + 1] =
                                make_int4((int)(last - blockIdx.x) + 1, pc.first() ? 0 : 1, pc.rows, 0);
                        }
                    }
                    __syncwarp();
                    if (!more) break;
                    if constexpr (TREE) {
                        // Q on its way to L2 while the tiles before it are worked on (from
                        // DRAM it held up a piece's first scores for 1.6 - 3.6 us)
                        const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q);
#pragma unroll 1
                        for (int x = lane; x < min(256, pc.rows - pc.row0) * C::NH; x += 32) {
                            const int f = pc.row0 + x / C::NH, tok = pf_div(p, f);
                            asm volatile("prefetch.global.L2 [%0];" ::"l"(
                                q + ((long long)(pc.start + tok) * p.H + pc.kvh * p.G + f - tok * p.G) * D +
                                64 * (x % C::NH)));
                        }
                    }
                } else if (!next_piece()) {
                    break;
                }
                auto box_block = [&](int kt) {
                    const int tok = kt * C::TT + 16 * lane;
                    return (kt < pc.kt1 && lane < 8 && tok < pc.n)
                               ? ld_dep(p.bt + (long long)pc.b * p.maxb + tok / B)
                               : -1;
                };
                int blk_next = box_block(pc.kt0);
                // (a tree's keys are read once, unless it has several pairs; 32 trees of 16 nodes: 63.6
                // us for 67.0)
                const uint64_t pol = TREE && pc.rows <= C::ROWS ? pol_first : pol_normal;
#pragma unroll 1
                for (int kt = pc.kt0; kt < pc.kt1; ++kt, seq += 2) {
                    const int tok = kt * C::TT + 16 * lane;
                    const int blk = blk_next;
                    blk_next = box_block(kt + 1);
                    const bool inside = lane < 8 && tok < pc.n;
                    const bool valid = inside && blk >= 0 && blk < p.num_blocks;
                    const unsigned vmask = __ballot_sync(kFullMask, valid);
                    if (kv && inside && !valid) atomicOr(p.status, kStatusBadBlock);
                    const int stage = seq % C::NS;
                    if (lane < 8) blocks[lane] = blk;
                    if (seq >= C::NS &&
                        !__all_sync(kFullMask, wait(C::KV_EMPTY + stage, (seq / C::NS - 1) & 1))) {
                        aborted = true;
                        break;
                    }
                    __syncwarp();
                    if (kv && vmask != 0xffu) {  // missing boxes of V are zero: 0 * stale is not
#pragma unroll 1
                        for (int x = lane; x < 8 * 128 * C::NH; x += 32) {
                            const int box = (x >> 7) & 7;
                            if (!((vmask >> box) & 1u))
                                *reinterpret_cast<uint4*>(smem + stage * C::TILE + (x >> 10) * C::HALF +
                                                          (x & 1023) * 16) = make_uint4(0, 0, 0, 0);
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                    // (one thread issues all boxes: eight lanes taking turns at it
                    // cost the warp several times the instructions)
                    if (elect_one()) {
                        const uint32_t fb = bar0 + 8 * (C::KV_FULL + stage);
                        if (!kv) box_bits[(seq >> 1) & 7] = (int)vmask;
                        mbar_arrive_expect_tx(fb, (uint32_t)__popc(vmask) * C::NH * 2048u);
                        const int4 lo = *reinterpret_cast<const int4*>(blocks);
                        const int4 hi = *reinterpret_cast<const int4*>(blocks + 4);
                        const int id[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
                        const uint32_t dst = sbase + stage * C::TILE;
#pragma unroll
                        for (int r = 0; r < 8; ++r) {
                            if (!((vmask >> r) & 1u)) continue;
                            const int row0 = (16 * r) % B;
                            const int o2 = p.slot_blk == 2 ? id[r] : (p.slot_layer == 2 ? p.layer : pc.kvh);
                            const int o3 = p.slot_blk == 3 ? id[r] : (p.slot_layer == 3 ? p.layer : pc.kvh);
                            const int o4 = p.slot_blk == 4 ? id[r] : (p.slot_layer == 4 ? p.layer : pc.kvh);
#pragma unroll
                            for (int h = 0; h < C::NH; ++h)
                                tma_load_5d(dst + r * 2048 + h * C::HALF, tm, fb, 64 * h, row0, o2, o3, o4, pol);
                        }
                    }
                    __syncwarp();
                }
            }
            if (aborted || *abort_all)  // copies in flight land before the CTA can exit
                for (int k = seq - 2; k >= 0 && k >= seq - C::NS; k -= 2)
                    (void)mbar_wait_bounded(bar0 + 8 * (C::KV_FULL + k % C::NS), (k / C::NS) & 1);
            __syncwarp();
        } else if (warp == 1) {
            // ======================================================= MMA issuer
            // (elect.sync, not lane == 0: ptxas then knows that one thread runs the
            // region and keeps the descriptors in uniform registers.  Beside warps
            // that fill the issue slots a 128 x 128 x 16 MMA is issued every 66
            // cycles, 64 being the pipe's rate; under lane == 0 every 242.)
            if (elect_one()) {
                constexpr uint32_t IDS = umma_idesc_bf16(128, C::TT, 0, 0);
                constexpr uint32_t IDV = umma_idesc_bf16(128, D, 0, 1);
                const uint64_t dK = umma_desc_sw128(sbase, 0, 1024);
                const uint64_t dV = umma_desc_sw128(sbase, C::HALF, 1024);
                const uint64_t dQ = umma_desc_sw128(sbase + C::OFF_Q, 0, 1024);
                int seq = 0, npj[2] = {0, 0}, nqj[2] = {0, 0}, nclean = 0, nlook = 0;
                bool ok = true;
                // asks for the look over V of tile i; up to two are asked for before the
                // first is waited for, and V's stage held K(i - 2) or what came before it
                auto look = [&](int i) {
                    if (i < pc.kt1 - pc.kt0 && pf_unclean(pc, pc.kt0 + i))
                        mbar_arrive(bar0 + 8 * (C::V_LOOK + (nlook++ & 1)));
                };
                auto stage_full = [&](int s) { return wait(C::KV_FULL + s % C::NS, (s / C::NS) & 1); };
                auto score = [&](int j, int q, int s) {  // S_j = Q_q K^T, K in stage s
                    const uint64_t a = dQ + (uint64_t)((q * C::TILE) >> 4);
                    const uint64_t b = dK + (uint64_t)(((s % C::NS) * C::TILE) >> 4);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint64_t o = (uint64_t)(((k >> 2) * C::HALF + (k & 3) * 32) >> 4);
                        umma_bf16(tmem + j * 128, a + o, b + o, IDS, k > 0 ? 1u : 0u);
                    }
                    umma_commit(bar0 + 8 * (C::S_FULL + j));
                };
                while (ok) {
                    const int slot = np % C::NP;
                    if (!(ok = wait(C::PC_FULL + slot, (np / C::NP) & 1))) break;
                    pc = pieces[slot];
                    mbar_arrive(bar0 + 8 * (C::PC_EMPTY + slot));
                    ++np;
                    if (pc.nj == 0) break;
                    const int nk = pc.kt1 - pc.kt0;
                    // in turns, tile i is group i % 2's, and S runs two tiles ahead
                    const bool turns = TURNS && pc.turns();
                    const int ahead = turns ? 2 : 1;
#pragma unroll 1
                    for (int i = 0; i < ahead && ok; ++i) {
                        if (!(ok = stage_full(seq + 2 * i))) break;
                        tc_fence_after();
                        if (i == 0) look(0), look(1);
#pragma unroll 1
                        for (int j = 0; j < pc.nj; ++j) {
                            if (i == 0) {
                                if (!(ok = wait(C::Q_FULL + j, nqj[j] & 1))) break;
                                ++nqj[j];
                                tc_fence_after();
                            }
                            score(turns ? i : j, j, seq + 2 * i);
                            if (nk == 1) umma_commit(bar0 + 8 * (C::Q_EMPTY + j));
                        }
                        if (!ok) break;
                        umma_commit(bar0 + 8 * (C::KV_EMPTY + (seq + 2 * i) % C::NS));
                    }
#pragma unroll 1
                    for (int i = 0; i < nk && ok; ++i, seq += 2) {
                        const uint64_t v = dV + (uint64_t)((((seq + 1) % C::NS) * C::TILE) >> 4);
#pragma unroll 1
                        for (int j = 0; j < pc.nj && ok; ++j) {
                            const int g = turns ? i & 1 : j;
                            // by the parts of P as they come: the exponentials of
                            // the rest are still under way
                            if (j == 0) {
                                ok = stage_full(seq + 1);
                                if (ok && pf_unclean(pc, pc.kt0 + i))
                                    ok = wait(C::V_CLEAN + (nclean & 1), (nclean >> 1) & 1), ++nclean;
                            }
#pragma unroll
                            for (int part = 0; part < 3; ++part) {
                                if (!ok || !(ok = wait(C::P_FULL + 2 * part + g, npj[g] & 1))) break;
                                tc_fence_after();
#pragma unroll
                                for (int k = part ? 2 + 2 * part : 0; k < 4 + 2 * part; ++k)
                                    umma_bf16_ts(tmem + C::O_COL + g * D, tmem + g * 128 + k * 8,
                                                 v + (uint64_t)(k * (2048 >> 4)), IDV,
                                                 (i >= ahead || k > 0) ? 1u : 0u);
                            }
                            if (!ok) break;
                            ++npj[g];
                            umma_commit(bar0 + 8 * (C::PV_DONE + g));
                            if (j == pc.nj - 1)
                                umma_commit(bar0 + 8 * (C::KV_EMPTY + (seq + 1) % C::NS));
                            if (j == 0) look(i + 2);
                            if (i + ahead < nk) {
                                const int ks = seq + 2 * ahead;
                                if (j == 0 && !(ok = stage_full(ks))) break;
                                tc_fence_after();
                                score(g, j, ks);
                                if (i + ahead + 1 == nk) umma_commit(bar0 + 8 * (C::Q_EMPTY + j));
                                if (j == pc.nj - 1) umma_commit(bar0 + 8 * (C::KV_EMPTY + ks % C::NS));
                            }
                        }
                    }
                }
                // every MMA issued so far completes before TMEM is released
                umma_commit(bar0 + 8 * C::FINAL);
                (void)mbar_wait_bounded(bar0 + 8 * C::FINAL, 0);
            }
            __syncwarp();
        } else {
            // ============================================== Q rows (warp 2)
            // Groups that divide 128: a tile is 128 / G tokens' heads, one box of
            // the 3-D tensor map (columns, heads, tokens) per half; what it holds
            // past the sequence belongs to rows that are not written.  Other groups of
            // up to 64: one box per token that lies whole in the tile (the swizzle goes
            // by the address, so a box may start at any row), the rest row by row.
            constexpr int CPR = D / 8;               // 16-byte chunks per row
            constexpr int RPI = 32 / CPR;            // rows per pass
            const int c = lane % CPR;
            const bool boxes = 128 % p.G == 0;
            const bool tokens = p.G <= 64 && p.qscale >= 0.f;  // (at least one whole in a tile)
            int nqj[2] = {0, 0}, vseq = 1, nlook = 0, piece = 0, mark_at = -1;
            bool ok = true;
            const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q);
            while (ok && next_piece()) {
#pragma unroll 1
                for (int j = 0; j < pc.nj && ok; ++j) {
                    if (nqj[j] > 0)
                        ok = __all_sync(kFullMask, wait(C::Q_EMPTY + j, (nqj[j] - 1) & 1));
                    if (!ok) break;
                    ++nqj[j];
                    const uint32_t fb = bar0 + 8 * (C::Q_FULL + j);
                    const uint32_t tile = sbase + C::OFF_Q + j * C::TILE;
                    const int f0 = pc.row0 + 128 * j;
                    if (boxes && p.qscale >= 0.f) {
                        if (elect_one()) {
                            mbar_arrive_expect_tx(fb, (uint32_t)C::TILE);
                            for (int h = 0; h < C::NH; ++h)
                                tma_load_3d(tile + h * C::HALF, &tmq, fb, 64 * h, pc.kvh * p.G,
                                            pc.start + pf_div(p, f0));
                        }
                        __syncwarp();
                        continue;
                    }
                    const uint32_t dst = tile + (c >> 3) * C::HALF;
                    // the tile's whole tokens, from row r0 to r1, as boxes
                    const int tok0 = pf_div(p, f0 + p.G - 1);
                    const int r0 = tokens ? tok0 * p.G - f0 : 128;
                    const int whole = tokens ? pf_div(p, 128 - r0) : 0, r1 = r0 + whole * p.G;
#pragma unroll 4
                    for (int x = lane / CPR; x < r0 + 128 - r1; x += RPI) {
                        const int r = x < r0 ? x : x + r1 - r0;
                        const bool live = f0 + r < pc.rows;
                        const int tok = pf_div(p, f0 + r), g = f0 + r - tok * p.G;
                        cp_async16(dst + sw128(r, c),
                                   live ? q + ((long long)(pc.start + tok) * p.H + pc.kvh * p.G + g) * D + 8 * c
                                        : q,
                                   live);
                    }
                    asm volatile("cp.async.wait_all;" ::: "memory");
                    if (p.qscale < 0.f) {  // S = -Q K^T, and the softmax scales by |scale|
#pragma unroll 1
                        for (int r = lane / CPR; r < 128; r += RPI) {
                            uint4* at = reinterpret_cast<uint4*>(smem + C::OFF_Q + j * C::TILE +
                                                                 (c >> 3) * C::HALF + sw128(r, c));
                            uint4 v = *at;
                            v.x ^= 0x80008000u, v.y ^= 0x80008000u, v.z ^= 0x80008000u, v.w ^= 0x80008000u;
                            *at = v;
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (elect_one()) {
                        mbar_arrive_expect_tx(fb, (uint32_t)(whole * p.G) * D * 2u);
#pragma unroll 1
                        for (int t = 0; t < whole; ++t)
#pragma unroll
                            for (int h = 0; h < C::NH; ++h)
                                tma_load_3d(tile + h * C::HALF + (r0 + t * p.G) * 128, &tmq, fb, 64 * h,
                                            pc.kvh * p.G, pc.start + tok0 + t);
                    }
                    __syncwarp();
                }
                // V of the piece's last tiles: rows that none of the pair's see are zeroed,
                // of the others the values that are not finite, which are remembered.  (Asked
                // for two tiles ahead: it takes 2000 cycles and more beside the softmax, and
                // asked for one ahead the last product waited 2000 - 4400 for it.)
                ++piece;
                const int last =
                    TREE ? pc.n - 1 : pc.first_pos + pf_div(p, min(pc.rows, pc.row0 + 256) - 1);
#pragma unroll 1
                for (int kt = pc.kt0; kt < pc.kt1 && ok; ++kt, vseq += 2) {
                    if (!pf_unclean(pc, kt)) continue;
                    const int t0 = kt * C::TT, stage = vseq % C::NS;
                    // (not before it is asked for: a wait may be no more than one phase
                    // ahead of its barrier)
                    ok = __all_sync(kFullMask, wait(C::V_LOOK + (nlook & 1), (nlook >> 1) & 1) &&
                                                   wait(C::KV_FULL + stage, (vseq / C::NS) & 1));
                    if (!ok) break;
                    const int clean = C::V_CLEAN + (nlook++ & 1);
                    uint32_t odd = 0;
#pragma unroll 1
                    for (int r = lane; r < 128; r += 32) {
                        unsigned char* vrow = smem + stage * C::TILE + r * 128;
                        if (t0 + r <= pc.pair_pos) continue;
                        if (t0 + r > last) {
#pragma unroll
                            for (int h = 0; h < C::NH; ++h)
#pragma unroll
                                for (int k = 0; k < 8; ++k)
                                    *reinterpret_cast<uint4*>(vrow + h * C::HALF + ((k + r) & 7) * 16) =
                                        make_uint4(0, 0, 0, 0);
                            continue;
                        }
                        // 0 * x summed up is NaN as soon as one x is not finite
                        __nv_bfloat162 z[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) z[k] = __floats2bfloat162_rn(0.f, 0.f);
                        const __nv_bfloat162 zero = z[0];
#pragma unroll
                        for (int h = 0; h < C::NH; ++h)
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                const uint4 v =
                                    *reinterpret_cast<const uint4*>(vrow + h * C::HALF + ((k + r) & 7) * 16);
                                const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    z[e] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&u[e]), zero, z[e]);
                            }
                        const float2 f = __bfloat1622float2(__hadd2(__hadd2(z[0], z[1]), __hadd2(z[2], z[3])));
                        if (f.x + f.y != 0.f) odd |= 1u << (r >> 5);
                    }
                    if (__any_sync(kFullMask, odd != 0)) {
                        if (mark_at != piece) {
                            // (the softmax warps may still be reading the last marks)
#pragma unroll 1
                            for (int n = 0; (done[0] < 4 * (piece - 1) || done[1] < 4 * (piece - 1)) && !*abort_all &&
                                            n < (1 << 24); ++n)
                                __nanosleep(100);
#pragma unroll 1
                            for (int k = lane; k < 3 * D && !TREE; k += 32) marks[k] = INT_MAX;
                            mark_at = piece;
                            if (lane == 0) *mark_piece = piece;
                            __syncwarp();
                        }
#pragma unroll 1
                        for (int q4 = 0; q4 < 4; ++q4) {
                            if (!((odd >> q4) & 1u)) continue;
                            const int r = 32 * q4 + lane;
#pragma unroll 1
                            for (int x = 0; x < 64 * C::NH; ++x) {
                                __nv_bfloat16* at = reinterpret_cast<__nv_bfloat16*>(
                                    smem + stage * C::TILE + r * 128 + (x >> 6) * C::HALF) + (x & 63);
                                const float v = __bfloat162float(*at);
                                if (isfinite(v)) continue;
                                const int d = (x & ~63) + ((((x >> 3) & 7) ^ (r & 7)) << 3) + (x & 7);
                                // (TREE: which rows see it is looked up at the output)
                                if (!TREE) atomicMin(marks + (v != v ? 0 : v > 0.f ? D : 2 * D) + d, t0 + r);
                                *at = __float2bfloat16(0.f);
                            }
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar0 + 8 * clean);
                }
            }
            if (*abort_all && lane == 0)  // copies in flight land before the CTA can exit
                for (int j = 0; j < 2; ++j)
                    if (nqj[j] > 0) (void)mbar_wait_bounded(bar0 + 8 * (C::Q_FULL + j), (nqj[j] - 1) & 1);
            __syncwarp();
        }
    } else {
        // ============================================================ softmax
        regs_inc<200>();
        const int j = (warp - 4) >> 2;             // row tile
        const int r = threadIdx.x - 128 - 128 * j; // row within it (TMEM lane)
        const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t s_col = trow + j * 128, o_col = trow + C::O_COL + j * D;
        // (a negative scale's sign is in Q; 0 becomes the smallest positive one, so
        // that -inf stays -inf)
        const float qs = fmaxf(fabsf(p.qscale), FLT_MIN);
        const bool out32 = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
        int seq = 0, ns = 0;                       // K stage; tiles of this row tile so far
        int piece = 0, nturns = 0;
        bool ok = true;
        while (ok) {
            const int slot = np % C::NP;
            if (!(ok = __all_sync(kFullMask, wait(C::PC_FULL + slot, (np / C::NP) & 1)))) break;
            pc = pieces[slot];
            __syncwarp();
            if (lane == 0) mbar_arrive(bar0 + 8 * (C::PC_EMPTY + slot));
            ++np;
            if (pc.nj == 0) break;
            ++piece;
            const int nk = pc.kt1 - pc.kt0;
            const bool turns = TURNS && pc.turns();
            if (j >= pc.nj && !turns) {
                seq += 2 * nk;
                if (lane == 0) atomicAdd(const_cast<int*>(done) + j, 1);
                continue;
            }
            const int f = pc.row0 + (turns ? 0 : 128 * j) + r;
            const int i0 = turns ? j : 0, step = turns ? 2 : 1;
            const bool live = f < pc.rows;
            const int tok = pf_div(p, f);
            // the last of the keys that the row sees all of, and TREE: its token's mask
            const int pos = live ? (TREE ? pc.first_pos - 1 : pc.first_pos + tok) : -1;
            const unsigned* mask = TREE ? p.masks + (live ? (long long)(pc.start + tok) * p.words : 0) : nullptr;
            if (TREE && live) tree_prefetch(mask);
            float m = -FLT_MAX;   // reference point of the exponentials (scaled, base 2)
            float2 l2 = make_float2(0.f, 0.f);
#pragma unroll 1
            for (int i = i0; i < nk; i += step, ++ns) {
                const int t0 = (pc.kt0 + i) * C::TT;
                ok = wait(C::S_FULL + j, ns & 1);
                ok = __all_sync(kFullMask, ok);
                if (!ok) break;
                tc_fence_after();
                // (with S, so its K, arrived; eight tiles are kept, the ring holds four)
                const unsigned bits = (unsigned)box_bits[((seq >> 1) + i) & 7] & 0xffu;
                // keys 0 .. lim of the tile are the row's, in pages that are there
                const int lim = pos - t0;
                // (TREE: rows that are not there may see what they like, no one reads them)
                const bool tail = TREE && t0 + C::TT > pc.first_pos;
                const bool masked = (TREE ? tail : __any_sync(kFullMask, lim < 127)) || bits != 0xffu;
                // settles the row's reference point: 0, it stays; 1, raised, the
                // sum and O scaled down; -1, stop
                auto raise = [&](float mt) {
                    if (i == i0) {
                        m = mt;
                        return 1;
                    }
                    if (!__any_sync(kFullMask, mt > m + 8.f)) return 0;
                    const bool up = mt > m + 8.f;
                    const float alpha = up ? ex2_approx(m - mt) : 1.f;
                    if (up) m = mt;
                    l2.x *= alpha, l2.y *= alpha;
                    if (!__all_sync(kFullMask, wait(C::PV_DONE + j, (ns - 1) & 1))) return -1;
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < D; c += 16) {
                        uint32_t o[16];
                        tmem_ld16(o_col + c, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            asm volatile("" : "+r"(o[k]));
                            o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
                        }
                        tmem_st16(o_col + c, o);
                    }
                    return 1;
                };
                uint32_t vis[4];
                if constexpr (TREE) {
                    uint4 seen = make_uint4(0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu);
                    if (tail && live) seen = tree_bits128(mask, p.words, t0 - pc.first_pos, pc.n - pc.first_pos);
                    vis[0] = seen.x, vis[1] = seen.y, vis[2] = seen.z, vis[3] = seen.w;
                }
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int e = lim - 32 * c;  // the last of the word's keys the row sees
                    vis[c] = (TREE ? vis[c] : e >= 31 ? 0xffffffffu : e < 0 ? 0u : (2u << e) - 1u) &
                             (((bits >> (2 * c)) & 1u ? 0xffffu : 0u) |
                              ((bits >> (2 * c + 1)) & 1u ? 0xffff0000u : 0u));
                }
                auto ready = [&](int k) {
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar0 + 8 * (C::P_FULL + 2 * k + j));
                };
                ok = pf_softmax_tile(s_col, qs, masked, vis, m, l2, raise, ready);
                if (!ok) break;
            }
            if (!ok) break;
            seq += 2 * nk;
            // ------------------------------------------------ the piece's output
            ok = __all_sync(kFullMask, wait(C::PV_DONE + j, (ns - 1) & 1));
            if (!ok) break;
            tc_fence_after();
            float l = l2.x + l2.y;
            const long long orow =
                live ? (long long)(pc.start + tok) * p.H + pc.kvh * p.G + (f - tok * p.G) : 0;
            const long long part = ((long long)blockIdx.x * 2 + (pc.first() ? 0 : 1)) * C::ROWS +
                                   (turns ? 0 : 128 * j) + r;
            // In turns, each group has the sums of its own tiles: both learn the other's
            // maxima and sums, through the rows that a second row tile would have in the
            // workspace (TREE: in shared memory), and each joins and writes half of the columns.
            float w0 = 1.f, w1 = 0.f;
            const int col0 = turns ? j * (D / 2) : 0;
            if (turns) {
                float2* ml = reinterpret_cast<float2*>(p.part_ml) + part;
                float2* sums = reinterpret_cast<float2*>(ctrl + C::MARKS) + r;
                if (TREE)
                    sums[128 * j] = make_float2(m, l);
                else
                    __stcg(ml + 128 * j, make_float2(m, l));
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar0 + 8 * C::X_SUMS);
                if (!(ok = __all_sync(kFullMask, wait(C::X_SUMS, nturns & 1)))) break;
                tc_fence_after();
                const float2 other = TREE ? sums[128 * (1 - j)] : __ldcg(ml + 128 * (1 - j));
                const float top = fmaxf(m, other.x);
                const float mine = ex2_approx(m - top), theirs = ex2_approx(other.x - top);
                w0 = j == 0 ? mine : theirs, w1 = j == 0 ? theirs : mine;
                m = top, l = fmaf(l, mine, other.y * theirs);
            }
            const float inv = pc.whole() ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
            w0 *= inv, w1 *= inv;
            float oall[D / 32][32];  // (all loads in flight at once)
            if (turns) {
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    tmem_ld32(trow + C::O_COL + col0 + 32 * c, oall[c]);
                    tmem_ld32(trow + C::O_COL + D + col0 + 32 * c, oall[D / 64 + c]);
                }
            } else {
#pragma unroll
                for (int c = 0; c < D / 32; ++c) tmem_ld32(o_col + 32 * c, oall[c]);
            }
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < D / 32; ++c) tmem_loaded32(oall[c]);
            if (turns) {
                // (the other group's O may be overwritten once both have it)
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar0 + 8 * C::X_READ);
                if (!(ok = __all_sync(kFullMask, wait(C::X_READ, nturns & 1)))) break;
                tc_fence_after();
                ++nturns;
            }
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                float (&o)[32] = oall[c];
                if (c >= D / 64 && turns) break;
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                    o[k] *= w0;
                    if (c < D / 64 && turns) o[k] = fmaf(oall[D / 64 + c % (D / 64)][k], w1, o[k]);
                }
                const int col = col0 + 32 * c;
                if (live && pc.whole()) {
                    // (whole sectors per thread: the rows of a warp lie apart)
                    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + orow * D + col;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t v[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            v[k] = pack_bf16x2(o[16 * h + 2 * k], o[16 * h + 2 * k + 1]);
                        if (out32) {
                            store32(out + 16 * h, v);
                        } else {
                            reinterpret_cast<uint4*>(out)[2 * h] = make_uint4(v[0], v[1], v[2], v[3]);
                            reinterpret_cast<uint4*>(out)[2 * h + 1] = make_uint4(v[4], v[5], v[6], v[7]);
                        }
                    }
                } else if (live) {
                    float* out = p.part_o + pf_part_at(part, D, col);
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        uint32_t v[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) v[k] = __float_as_uint(o[8 * h + k]);
                        store32(out + 256 * h, v);
                    }
                }
            }
            if (TREE && live && *mark_piece == piece) {
                // values that are not finite, into the rows that see them
                const __nv_bfloat16* vb =
                    static_cast<const __nv_bfloat16*>(p.v_base) + p.tile_off + (long long)pc.kvh * p.s_head;
                __nv_bfloat16* to = pc.whole() ? static_cast<__nv_bfloat16*>(p.out) + orow * D : nullptr;
                tree_odd_values<__nv_bfloat16, D>(
                    vb, p.s_blk, p.num_blocks, p.bt + (long long)pc.b * p.maxb, mask, pc.first_pos,
                    pc.n - pc.first_pos, B, pc.kt0 * C::TT, pc.kt1 * C::TT, col0, 1, turns ? col0 + D / 2 : D,
                    [to, part, part_o = p.part_o](int d, float v) {
                        if (to != nullptr)
                            to[d] = __float2bfloat16(__bfloat162float(to[d]) + v);
                        else
                            part_o[pf_part_at(part, D, d)] += v;
                    });
            } else if (live && *mark_piece == piece) {
                // values that are not finite, into the rows that see them
#pragma unroll 1
                for (int d = col0; d < (turns ? col0 + D / 2 : D); ++d) {
                    const float v = poison(marks, D, d, pos);
                    if (v == 0.f) continue;
                    if (pc.whole())
                        static_cast<__nv_bfloat16*>(p.out)[orow * D + d] = __float2bfloat16(v);
                    else
                        p.part_o[pf_part_at(part, D, d)] = v;
                }
            }
            // (in turns, group 0's rows hold its own sums until both have read them)
            if (!pc.whole() && live && !(turns && j == 1))
                p.part_ml[2 * part] = m, p.part_ml[2 * part + 1] = l;
            __syncwarp();  // (all of the warp have read the marks)
            if (lane == 0) atomicAdd(const_cast<int*>(done) + j, 1);
        }
        if (!ok) *abort_all = 1;
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tmem, C::TMEM_COLS);
}

// Joins the parts of the pairs that the CTAs' shares cut: the CTAs (x, *) the
// pair that main CTA x recorded, a warp 8 columns of 32 rows.  Dependent accesses to
// L2 are all it costs, so four parts are in flight at once, and where a pair has few
// rows and many parts up to eight warps take every eighth part each.
constexpr int kJoinParts = 8;  // CTAs per pair
struct PfJoin {
    float m = -FLT_MAX, l = 0.f;
    float o[8] = {};
    __device__ __forceinline__ void add(float2 ml, const float (&x)[8]) {
        if (ml.y == 0.f) return;  // (the part saw no key of the row)
        const float mn = fmaxf(m, ml.x);
        const float keep = ex2_approx(m - mn), w = ex2_approx(ml.x - mn);
        m = mn;
        l = fmaf(l, keep, w * ml.y);
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = fmaf(o[k], keep, w * x[k]);
    }
};
template <int D, bool TREE, int W = 8>  // W warps (TREE: a name of its own in either unit)
__global__ void __launch_bounds__(32 * W) pa_prefill_umma_join_kernel(const PrefillParams p) {
    pdl_trigger();
    pdl_wait();
    __shared__ float s_part[W][10][32];  // per warp: columns, maximum and sum of 32 rows
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int main_cta = blockIdx.x;
    if (TREE && gridDim.x < p.grid) {  // the blockIdx.x-th of the CTAs that recorded a cut pair
        constexpr int K = 5;  // 32 CTAs at a time
        int pieces[K], left = blockIdx.x;
#pragma unroll
        for (int k = 0; k < K; ++k)
            pieces[k] = 32 * k + lane < p.grid ? ld_dep(&p.cut[2 * (32 * k + lane) + 1].x) : 0;
        main_cta = -1;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const unsigned cuts = __ballot_sync(kFullMask, pieces[k] > 1);
            if (left >= 0 && left < __popc(cuts)) main_cta = 32 * k + __fns(cuts, 0, left + 1);
            left -= __popc(cuts);
        }
        if (main_cta < 0) return;
    }
    const int4 a = ld_dep(p.cut + 2 * main_cta);
    const int4 e = ld_dep(p.cut + 2 * main_cta + 1);
    const int pieces = e.x, rows = min(256, e.z - a.z);
    if (pieces <= 1) return;
    const int units = (rows + 31) / 32 * (D / 8), warps = W * gridDim.y;
    int ways = 1;  // warps to a unit; above 1 there is a warp for each
    if (pieces > 4)
        while (ways < 8 && 2 * ways * units <= warps) ways *= 2;
    const int way = warp % ways;
    for (int u = (blockIdx.y * W + warp) / ways; u < units || ways > 1; u += warps) {
        const int r = u / (D / 8) * 32 + lane, d = u % (D / 8) * 8;
        // (rows of part k: CTA x + k's first slot, but for k = 0)
        const long long row0 = (long long)main_cta * 512 + 256 * e.y + r;
        auto row = [&](int k) { return k == 0 ? row0 : (long long)(main_cta + k) * 512 + r; };
        PfJoin j;
        for (int k0 = way; k0 < pieces && r < rows && u < units; k0 += 4 * ways) {
            float2 ml[4];
            float x[4][8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (k0 + k * ways >= pieces) break;
                const long long at = row(k0 + k * ways);
                ml[k] = ld_dep(reinterpret_cast<const float2*>(p.part_ml) + at);
                const float4* o = reinterpret_cast<const float4*>(p.part_o + pf_part_at(at, D, d));
                *reinterpret_cast<float4*>(x[k]) = ld_dep(o);
                *reinterpret_cast<float4*>(x[k] + 4) = ld_dep(o + 1);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (k0 + k * ways < pieces) j.add(ml[k], x[k]);
        }
        if (ways > 1) {
#pragma unroll
            for (int k = 0; k < 8; ++k) s_part[warp][k][lane] = j.o[k];
            s_part[warp][8][lane] = j.m, s_part[warp][9][lane] = j.l;
            __syncthreads();
            if (way != 0) return;
            for (int w = warp + 1; w < warp + ways; ++w) {
                float x[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) x[k] = s_part[w][k][lane];
                j.add(make_float2(s_part[w][8][lane], s_part[w][9][lane]), x);
            }
        }
        if (r < rows && u < units) {
            const float inv = j.l == 0.f ? 0.f : 1.f / j.l;
            const int f = a.z + r, tok = pf_div(p, f);
            const long long orow = (long long)(a.w + tok) * p.H + a.y * p.G + (f - tok * p.G);
            uint32_t v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = pack_bf16x2(j.o[2 * k] * inv, j.o[2 * k + 1] * inv);
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + orow * D + d) =
                make_uint4(v[0], v[1], v[2], v[3]);
        }
        if (ways > 1) return;
    }
}

}  // namespace pa
