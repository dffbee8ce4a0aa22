// Attention of drafted trees over fp32 pools on tcgen05, for trees of many rows.
//
// An fp32 number is three bf16 ones: a = x rounded to bf16, b = x - a rounded, c = x - a - b
// rounded (8 bits each; x - a and x - a - b are exact, c misses x by 2^-26 at most), so
//   x x' = aa' + ab' + ba' + bb' + ac' + ca', off by 2^-24 at most, either sign,
// and both products of the attention are six products of kind::f16.  (Two TF32 parts and three
// products of kind::tf32, at half the rate, would take the same time, but their V has no plain layout.)
// The tensor core's sums are cut off toward zero, so the small products come first, where what is
// cut off is small, and P V of every tile starts from zero and is added to O by ordinary additions
// in registers, as in the mma.sync kernel.
//
// A CTA has a tile of 128 rows (token, head of the group), as there, and a part of the context, in
// tiles of 64 keys.  Four warps each read K and V (fp32) and write their parts, 128-byte swizzled, to
// shared memory, two stages of 48 KB each (head_dim 128); q's parts are in tensor memory (in shared
// memory they took the room of the second stages, and a product of 64 keys reads twice as much of them as
// of K).  Roles: warps 0 - 3 q, then softmax and O (a row to a thread), 4 - 7 K, 8 - 11 V, 12 the
// MMAs.
// Tensor memory: S_0, S_1 (P's parts a and b over them), P's part c twice, P V, q.
//
// What bounds it: latencies.  128 rows x 64 keys of head_dim 128 take 2.8 us of an SM, of which the
// products are 1.5: K and V of a tile are in registers of the warps that split them, so their loads start
// when the tile before has been written (without loads in the loop a quarter less), and a row's softmax, its
// parts and the addition of P V follow one another.  Nor are K and V split once for all: the two row
// tiles of 64 nodes of 4 heads are CTAs of their own, and each splits both.  32 trees of 64 nodes over
// 4,000 keys, 32 heads on 8 of 128: 712 us, 189 TFLOP/s of fp32 products (mma.sync 2,490; elementary fp32
// operations of torch 6,970; the six products alone 428); 8 of 25 over 2,000: 61 us (212; 1,000; 21); one
// of 64 over 1,000: 19 (34); 4 of 8 over 500 - 2,000: 30 (33).  Errors are half of the TF32 kernel's
// (8 of 25: 4.3e-7 of the output's size, 8.8e-7 there, 1.1e-6 in elementary fp32 operations).
//   Other forms: q in shared memory and one stage of K and V, 79 us for the 8 of 25; each chunk's next
// load right after its split, 86 (a warp has few counters for loads, and the waits for old ones take the new ones
// in); the tiles' lines brought to L2 two ahead, 74; P V summed in tensor memory over two tiles, no
// change.  K and V by cp.async into 64 KB of their own, with one stage of V's parts or of both, 58 for the 8
// of 25 and 670 for the 32 of 64, but 21 for the one of 64, and 2 us more where a call takes 10: over
// 62 calls as good on average, at shorter calls worse.
#include "pa_prefill_mma.cuh"
#include "pa_prefill_umma.cuh"

namespace pa {

namespace {

template <int D_>
struct F32Cfg {
    static constexpr int NH = D_ / 64, D = D_, BM = 128, BN = 64;
    static constexpr int KP = NH * 64 * 128, STAGE = 3 * KP;  // bytes of a part, of a tile
    static constexpr int OFF_V = 2 * STAGE, OFF_CTRL = 2 * OFF_V;
    // ctrl: barriers | TMEM address, abort, marked, odd | pages of eight tiles | the row tile |
    // marks [3][D] (first NaN, +inf, -inf per column)
    static constexpr int TMEM_SLOT = 136, ABORT = 140, MARKED = 144, ODD = 148, BITS = 152, AT = 184, MARKS = 208;
    static constexpr int SMEM_BYTES = OFF_CTRL + MARKS + 3 * D * 4;
    // (K, V, S and P: two each, in turns)
    static constexpr int Q_FULL = 0, K_FULL = 1, V_FULL = 3, P_FULL = 5, O_FREE = 7, K_EMPTY = 8, V_EMPTY = 10, S_FULL = 12,
                         O_FULL = 14, FINAL = 15, NBAR = 16;
    static constexpr int THREADS = 512;
    static constexpr int C_COL = 128, O_COL = 192, Q_COL = O_COL + D, TMEM_COLS = 512;
    static_assert(Q_COL + 3 * D / 2 <= TMEM_COLS, "tensor memory");
    static_assert(SMEM_BYTES <= 232448, "shared memory");
};

// Two numbers' parts, the first's in the low halves.  CUT: a cut off instead of rounded (what
// rounds to infinity).  odd: becomes NaN where an a is not finite.
template <bool CUT>
__device__ __forceinline__ void split3(float x, float y, uint32_t& a, uint32_t& b, uint32_t& c, float& odd) {
    a = CUT ? __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632) : pack_bf16x2(x, y);
    const float ax = __uint_as_float(a << 16), ay = __uint_as_float(a & 0xffff0000u);
    const float2 r = add2(make_float2(x, y), make_float2(-ax, -ay));
    b = pack_bf16x2(r.x, r.y);
    const float2 t = add2(r, make_float2(-__uint_as_float(b << 16), -__uint_as_float(b & 0xffff0000u)));
    c = pack_bf16x2(t.x, t.y);
    odd = fmaf(ax, 0.f, fmaf(ay, 0.f, odd));
}

// Scores of a row against 64 keys, summed plainly, into its S columns: where a factor is not
// finite.  k_rows: the pool's K of the layer and KV head; table: the sequence's row.
template <int D>
__device__ __noinline__ void tree_plain_scores(uint32_t s_col, const float* q, const float* k_rows, long long s_blk,
                                               long long num_blocks, const int* table, int B, int t0, int n, bool live) {
#pragma unroll 1
    for (int k = 0; k < 64; ++k) {
        const int key = t0 + k;
        const int blk = key < n ? ld_dep(table + key / B) : -1;
        float s = 0.f;
        if (live && blk >= 0 && blk < num_blocks) {
            const float* row = k_rows + (long long)blk * s_blk + key % B * D;
#pragma unroll 4
            for (int d = 0; d < D; ++d) s = fmaf(ld_dep(q + d), ld_dep(row + d), s);
        }
        __syncwarp();
        asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(s_col + k), "r"(__float_as_uint(s))
                     : "memory");
    }
    tmem_wait_st();
}

template <int D, int B>
__global__ void __launch_bounds__(512, 1) pa_tree_umma_f32_kernel(const PrefillParams p) {
    using C = F32Cfg<D>;
    extern __shared__ __align__(1024) unsigned char tiles[];
    pdl_trigger();
    const uint32_t sbase = smem_addr(tiles);
    if (sbase & 1023u) {  // (the swizzled tiles need it; there is no other shared memory)
        if (threadIdx.x == 0) atomicOr(p.status, kStatusTimeout);
        return;
    }
    unsigned char* ctrl = tiles + C::OFF_CTRL;
    const uint32_t bar0 = sbase + C::OFF_CTRL;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ctrl + C::TMEM_SLOT);
    volatile int* abort_all = reinterpret_cast<volatile int*>(ctrl + C::ABORT);
    volatile int* marked = reinterpret_cast<volatile int*>(ctrl + C::MARKED);
    volatile int* has_odd = reinterpret_cast<volatile int*>(ctrl + C::ODD);
    volatile int* page_bits = reinterpret_cast<volatile int*>(ctrl + C::BITS);
    int* at = reinterpret_cast<int*>(ctrl + C::AT);
    int* marks = reinterpret_cast<int*>(ctrl + C::MARKS);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == 13) {  // (a barrier to a lane)
        if (lane < C::NBAR) mbar_init(bar0 + 8 * lane, lane < C::K_EMPTY ? 4 : 1);
        if (lane == 0) *abort_all = 0, *marked = 0, *has_odd = 0;
        fence_mbar_init();
    }
    if (warp == 12) tmem_alloc(smem_addr(tmem_slot), C::TMEM_COLS);
    for (int x = threadIdx.x; x < 3 * D; x += C::THREADS) marks[x] = INT_MAX;
    pdl_wait();
    if (warp == 0) find_tile<C::BM, B>(p, lane, at);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int b = at[0], row0 = at[1], start = at[2], n_new = at[3];
    int n = b < 0 ? 0 : at[4];
    if (b >= 0 && (n < n_new || n > p.maxb * B || n_new > 32 * p.words)) {
        if (threadIdx.x == 0) atomicOr(p.status, kStatusBadLength);
        n = 0;
    }
    const int kvh = blockIdx.x % p.Hkv;
    const int rows = b < 0 ? 0 : (int)min((long long)C::BM, (long long)n_new * p.G - row0);
    const int first_pos = n - n_new;
    const int key_tiles = (n + C::BN - 1) / C::BN;
    const int per = (key_tiles + p.splits - 1) / p.splits;
    const int kt0 = min((int)blockIdx.y * per, key_tiles), kt1 = min(kt0 + per, key_tiles);
    auto token = [&](int row) { return (int)(((unsigned long long)(unsigned)row * p.div_mul) >> p.div_shift); };
    auto wait = [&](int bar, uint32_t parity) {
        return __all_sync(kFullMask, pf_wait(bar0 + 8 * bar, parity, abort_all, p.status));
    };
    auto arrive = [&](int bar) {  // (by each warp of a role, what its threads wrote before)
        __syncwarp();
        if (lane == 0) mbar_arrive(bar0 + 8 * bar);
    };
    constexpr int CPR = D / 4;                   // 16-byte chunks of an fp32 row
    const int cc = threadIdx.x % CPR;            // this thread's, of the rows it copies
    // where the chunk's 8 bytes of a part stand in row r of a tile whose halves are `half` bytes
    auto place = [&](int r, int half) { return cc / 16 * half + sw128(r, cc % 16 / 2) + 8 * (cc & 1); };
    // writes a chunk's parts
    auto put = [&](auto cut, unsigned char* to, int part, float4 x, float& odd) {
        uint2 v[3];
        split3<decltype(cut)::value>(x.x, x.y, v[0].x, v[1].x, v[2].x, odd);
        split3<decltype(cut)::value>(x.z, x.w, v[0].y, v[1].y, v[2].y, odd);
#pragma unroll
        for (int k = 0; k < 3; ++k) *reinterpret_cast<uint2*>(to + k * part) = v[k];
    };

    if (b >= 0 && warp < 4) {
        // ================================================ q, then softmax and output
        regs_inc<248>();
        const int r = threadIdx.x;               // row of the tile, TMEM lane
        const float* q = static_cast<const float*>(p.q);
        auto q_row = [&](int row) {
            const int tok = token(row0 + row);
            return ((long long)(start + tok) * p.H + kvh * p.G + row0 + row - tok * p.G) * D;
        };
        const bool live = r < rows;
        const uint32_t trow = tmem + ((uint32_t)(warp * 32) << 16);
        bool ok = true;
        if (kt0 < kt1) {
            const float4* from = reinterpret_cast<const float4*>(q + (live ? q_row(r) : 0));
            float4 x[D / 4];
#pragma unroll
            for (int i = 0; i < D / 4; ++i) x[i] = live ? ld_dep(from + i) : make_float4(0, 0, 0, 0);
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                uint32_t v[3][16];
                auto parts = [&](auto cut) {
                    float odd = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 y = x[8 * c + i];
                        split3<decltype(cut)::value>(y.x, y.y, v[0][2 * i], v[1][2 * i], v[2][2 * i], odd);
                        split3<decltype(cut)::value>(y.z, y.w, v[0][2 * i + 1], v[1][2 * i + 1], v[2][2 * i + 1], odd);
                    }
                    return odd == 0.f;
                };
                if (!parts(std::false_type())) parts(std::true_type());
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 3; ++k) tmem_st16(trow + C::Q_COL + k * (D / 2) + 16 * c, v[k]);
            }
            tmem_wait_st();
            tc_fence_before();
            arrive(C::Q_FULL);
        }
        const unsigned* mask = p.masks + (live ? (long long)(start + token(row0 + r)) * p.words : 0);
        if (live) tree_prefetch(mask);
        const int* table = p.bt + (long long)b * p.maxb;
        float o[D], m = -INFINITY, l = 0.f, alpha = 0.f;
#pragma unroll
        for (int d = 0; d < D; ++d) o[d] = 0.f;
        // adds P V of tile i, and O as it was at the maximum before
        auto add_tile = [&](int i, float keep) {
            if (!(ok = wait(C::O_FULL, i & 1))) return;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {  // (64 columns on their way at once)
                float t[2][32];
                tmem_ld32(trow + C::O_COL + 64 * c, t[0]);
                tmem_ld32(trow + C::O_COL + 64 * c + 32, t[1]);
                tmem_wait_ld();
                tmem_loaded32(t[0]);
                tmem_loaded32(t[1]);
#pragma unroll
                for (int k = 0; k < 64; k += 2) {
                    float* at = o + 64 * c + k;
                    const float2 v = fma2(make_float2(at[0], at[1]), make_float2(keep, keep),
                                          make_float2(t[k / 32][k % 32], t[k / 32][k % 32 + 1]));
                    at[0] = v.x, at[1] = v.y;
                }
            }
            tc_fence_before();
        };
        for (int i = 0; i < kt1 - kt0; ++i) {
            const int t0 = (kt0 + i) * C::BN, j = i & 1;
            const uint32_t s_col = trow + 64 * j;
            if (!(ok = wait(C::S_FULL + j, (i >> 1) & 1))) break;
            tc_fence_after();
            // the keys that the row sees, in pages that are there
            const unsigned pages = (unsigned)page_bits[i & 7];
            const bool tail = t0 + C::BN > first_pos;
            uint32_t vis[2];
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                vis[w] = B == 32 ? (pages >> w & 1u ? 0xffffffffu : 0u)
                                 : (pages >> (2 * w) & 1u ? 0xffffu : 0u) | (pages >> (2 * w + 1) & 1u ? 0xffff0000u : 0u);
                if (tail) vis[w] &= live ? tree_bits(mask, p.words, t0 + 32 * w - first_pos, n_new) : 0u;
            }
            const bool masked = __any_sync(kFullMask, (vis[0] & vis[1]) != 0xffffffffu);
            float x[2][32], mn;
            const float before = alpha;
            float2 sum;
            for (int plain = 0;; plain = 1) {
                tmem_ld32(s_col, x[0]);
                tmem_ld32(s_col + 32, x[1]);
                tmem_wait_ld();
                tmem_loaded32(x[0]);
                tmem_loaded32(x[1]);
                float mt = -INFINITY;
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int k = 0; k < 32; k += 2) {
                        const float2 y = fma2(make_float2(x[c][k], x[c][k + 1]), make_float2(p.qscale, p.qscale),
                                              make_float2(0.f, 0.f));
                        x[c][k] = !masked || (vis[c] >> k & 1u) ? y.x : -INFINITY;
                        x[c][k + 1] = !masked || (vis[c] >> (k + 1) & 1u) ? y.y : -INFINITY;
                        mt = fmaxf(mt, fmaxf(x[c][k], x[c][k + 1]));
                    }
                mn = fmaxf(fmaxf(m, mt), -3.0e38f);  // finite: a row may see no key
                sum = make_float2(0.f, 0.f);
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int k = 0; k < 32; k += 2) {
                        const float2 e = add2(make_float2(x[c][k], x[c][k + 1]), make_float2(-mn, -mn));
                        x[c][k] = ex2_approx(e.x), x[c][k + 1] = ex2_approx(e.y);
                        sum = add2(sum, make_float2(x[c][k], x[c][k + 1]));
                    }
                // (a factor that is not finite: its parts make NaN of any score)
                if (plain || !__any_sync(kFullMask, !(sum.x + sum.y < INFINITY))) break;
                tree_plain_scores<D>(s_col, q + (live ? q_row(r) : 0),
                                     static_cast<const float*>(p.k_base) + p.tile_off + (long long)kvh * p.s_head, p.s_blk,
                                     p.num_blocks, table, B, t0, n, live);
            }
            alpha = ex2_approx(m - mn);
            m = mn;
            float odd = 0.f;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t pa[16], pb[16], pc[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) split3<false>(x[c][2 * k], x[c][2 * k + 1], pa[k], pb[k], pc[k], odd);
                tmem_st16(s_col + 16 * c, pa);
                tmem_st16(s_col + 32 + 16 * c, pb);
                tmem_st16(trow + C::C_COL + 32 * j + 16 * c, pc);
            }
            l = l * alpha + (sum.x + sum.y);
            tmem_wait_st();
            tc_fence_before();
            arrive(C::P_FULL + j);
            if (i > 0) {
                add_tile(i - 1, before);
                if (!ok) break;
                arrive(C::O_FREE);
            }
        }
        if (ok && kt0 < kt1) add_tile(kt1 - kt0 - 1, alpha);
        if (!ok) {
            *abort_all = 1;
        } else if (live) {
            // (nothing seen: zeros)
            const long long orow = q_row(r) / D;
            const bool whole = p.splits == 1;
            const long long prow = (long long)blockIdx.y * p.num_tokens * p.H + orow;
            float* to = whole ? static_cast<float*>(p.out) + orow * D : p.part_o + prow * D;
            const float inv = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
#pragma unroll
            for (int d = 0; d < D; d += 4)
                *reinterpret_cast<float4*>(to + d) =
                    make_float4(o[d] * inv, o[d + 1] * inv, o[d + 2] * inv, o[d + 3] * inv);
            if (!whole) reinterpret_cast<float2*>(p.part_ml)[prow] = make_float2(m, l);
            if (*marked)
#pragma unroll 1
                for (int d = 0; d < D; ++d) {
                    const float v = poison(marks, D, d, first_pos - 1);
                    if (v != 0.f) to[d] = v;
                }
            if (*has_odd)
                tree_odd_values<float, D>(static_cast<const float*>(p.v_base) + p.tile_off + (long long)kvh * p.s_head, p.s_blk,
                                          p.num_blocks, table, mask, first_pos, n_new, B, kt0 * C::BN, kt1 * C::BN, 0, 1, D,
                                          [to](int d, float v) { to[d] += v; });
        }
    } else if (b >= 0 && warp < 12) {
        // ============================================== K (warps 4 - 7), V (8 - 11)
        regs_dec<112>();
        constexpr int RPP = 128 / CPR, N = C::BN / RPP, PAGES = C::BN / B;
        const bool is_v = warp >= 8;
        const int tid = threadIdx.x - (is_v ? 256 : 128), cr = tid / CPR;
        const float* base = static_cast<const float*>(is_v ? p.v_base : p.k_base) + p.tile_off + (long long)kvh * p.s_head + 4 * cc;
        unsigned char* dst = tiles + (is_v ? C::OFF_V : 0);
        const int full = is_v ? C::V_FULL : C::K_FULL, empty = is_v ? C::V_EMPTY : C::K_EMPTY;
        const int* table = p.bt + (long long)b * p.maxb;
        int ids[PAGES];                          // of the next tile
        auto look_up = [&](int kt) {
#pragma unroll
            for (int u = 0; u < PAGES; ++u) {
                const int tok = kt * C::BN + u * B;
                ids[u] = kt < kt1 && tok < n ? ld_dep(table + tok / B) : 0;
            }
        };
        float4 x[N];
        unsigned bits = 0;                       // pages of the tile in x
        auto load = [&](int kt) {
            bits = 0;
#pragma unroll
            for (int u = 0; u < PAGES; ++u) {
                const bool in = kt < kt1 && kt * C::BN + u * B < n;
                const bool good = ids[u] >= 0 && ids[u] < p.num_blocks;
                if (in && !good && tid == 0 && is_v) atomicOr(p.status, kStatusBadBlock);
                if (in && good) bits |= 1u << u;
            }
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int key = i * RPP + cr, u = i * RPP / B;  // (RPP divides B)
                const bool in = (bits >> u & 1u) && kt * C::BN + key < n;
                x[i] = in ? ld_dep(reinterpret_cast<const float4*>(base + (long long)ids[u] * p.s_blk + key % B * D))
                          : make_float4(0, 0, 0, 0);
            }
            look_up(kt + 1);
        };
        look_up(kt0);
        load(kt0);
        bool ok = true;
        for (int i = 0; i < kt1 - kt0; ++i) {
            if (i > 1 && !(ok = wait(empty + (i & 1), ((i >> 1) - 1) & 1))) break;
            unsigned char* to = dst + (i & 1) * C::STAGE;
            if (!is_v && tid == 0) page_bits[i & 7] = (int)bits;
            float odd = 0.f;
#pragma unroll
            for (int k = 0; k < N; ++k) put(std::false_type(), to + place(k * RPP + cr, 64 * 128), C::KP, x[k], odd);
            if (!(odd == 0.f)) {
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    if (is_v) {
                        // values that are not finite: kept as marks, zero in the products
                        float v[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
                        const int key = (kt0 + i) * C::BN + k * RPP + cr;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            if (isfinite(v[e])) continue;
                            if (key < first_pos) {
                                *marked = 1;
                                atomicMin(marks + (v[e] != v[e] ? 0 : v[e] > 0.f ? D : 2 * D) + 4 * cc + e, key);
                            } else {
                                *has_odd = 1;
                            }
                            v[e] = 0.f;
                        }
                        x[k] = make_float4(v[0], v[1], v[2], v[3]);
                    }
                    put(std::true_type(), to + place(k * RPP + cr, 64 * 128), C::KP, x[k], odd);
                }
            }
            fence_proxy_async_smem();
            arrive(full + (i & 1));
            load(kt0 + i + 1);
        }
        if (!ok) *abort_all = 1;
    } else if (b >= 0) {
        regs_dec<40>();
        if (warp == 12 && kt0 < kt1) {
            // ======================================================= MMA issuer
            if (elect_one()) {
                auto wait1 = [&](int bar, uint32_t parity) { return pf_wait(bar0 + 8 * bar, parity, abort_all, p.status); };
                constexpr uint32_t IDS = umma_idesc_bf16(128, C::BN, 0, 0);
                constexpr uint32_t IDV = umma_idesc_bf16(128, D, 0, 1);
                const uint64_t dK = umma_desc_sw128(sbase, 0, 1024);
                const uint64_t dV = umma_desc_sw128(sbase + C::OFF_V, 64 * 128, 1024);
                const int tiles_here = kt1 - kt0;
                // Parts of the factors, two bits each, the small products first.  (A loop, not 72
                // products in a row: their descriptors spilled.)
                constexpr unsigned LEFT = 0x052, RIGHT = 0x118;  // 2 0 1 1 0 0, 0 2 1 0 1 0
                auto score = [&](int i) {
                    const uint64_t k0 = dK + (uint64_t)(((i & 1) * C::STAGE) >> 4);
#pragma unroll 1
                    for (int x = 0; x < 6; ++x) {
                        const uint32_t a = tmem + C::Q_COL + (LEFT >> 2 * x & 3u) * (D / 2);
                        const uint64_t b = k0 + (uint64_t)((RIGHT >> 2 * x & 3u) * (C::KP >> 4));
#pragma unroll
                        for (int k = 0; k < D / 16; ++k)
                            umma_bf16_ts(tmem + 64 * (i & 1), a + 8 * k,
                                         b + (uint64_t)(((k >> 2) * 64 * 128 + (k & 3) * 32) >> 4), IDS,
                                         x + k > 0 ? 1u : 0u);
                    }
                    umma_commit(bar0 + 8 * (C::S_FULL + (i & 1)));
                    umma_commit(bar0 + 8 * (C::K_EMPTY + (i & 1)));
                };
                bool ok = wait1(C::Q_FULL, 0) && wait1(C::K_FULL, 0);
                if (ok) {
                    tc_fence_after();
                    score(0);
                }
#pragma unroll 1
                for (int i = 0; i < tiles_here && ok; ++i) {
                    if (i + 1 < tiles_here) {  // (S(i - 1) has been read: P(i - 1) was there)
                        if (!(ok = wait1(C::K_FULL + ((i + 1) & 1), ((i + 1) >> 1) & 1))) break;
                        tc_fence_after();
                        score(i + 1);
                    }
                    if (!(ok = wait1(C::V_FULL + (i & 1), (i >> 1) & 1) && wait1(C::P_FULL + (i & 1), (i >> 1) & 1) &&
                               (i == 0 || wait1(C::O_FREE, (i - 1) & 1))))
                        break;
                    tc_fence_after();
                    const uint64_t v0 = dV + (uint64_t)(((i & 1) * C::STAGE) >> 4);
#pragma unroll 1
                    for (int x = 0; x < 6; ++x) {
                        const uint32_t left = LEFT >> 2 * x & 3u;
                        const uint32_t a = tmem + (left == 2 ? C::C_COL + 32u * (i & 1) : 64u * (i & 1) + 32u * left);
                        const uint64_t v = v0 + (uint64_t)((RIGHT >> 2 * x & 3u) * (C::KP >> 4));
#pragma unroll
                        for (int k = 0; k < C::BN / 16; ++k)
                            umma_bf16_ts(tmem + C::O_COL, a + 8 * k, v + (uint64_t)(k * (2048 >> 4)), IDV,
                                         x + k > 0 ? 1u : 0u);
                    }
                    umma_commit(bar0 + 8 * C::O_FULL);
                    umma_commit(bar0 + 8 * (C::V_EMPTY + (i & 1)));
                }
                // every MMA issued so far completes before TMEM is released
                umma_commit(bar0 + 8 * C::FINAL);
                (void)mbar_wait_bounded(bar0 + 8 * C::FINAL, 0);
            }
            __syncwarp();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 12) tmem_dealloc(tmem, C::TMEM_COLS);
}

template <int D, int B>
cudaError_t launch_f32(const PrefillParams& p, cudaStream_t s) {
    using C = F32Cfg<D>;
    auto kern = pa_tree_umma_f32_kernel<D, B>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    const long long ctas = ((long long)p.num_tokens * p.G / C::BM + p.batch) * p.Hkv;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    e = launch_pdl(kern, dim3((unsigned)ctas, p.splits), dim3(C::THREADS), C::SMEM_BYTES, s, p);
    if (e != cudaSuccess || p.splits == 1) return e;
    const long long rows = (long long)p.num_tokens * p.H;
    constexpr int RPC = kJoinThreads / (D / 4);
    return launch_pdl(pa_prefill_mma_join_kernel<float, D, true>, dim3((unsigned)((rows + RPC - 1) / RPC)),
                      dim3(kJoinThreads), 0, s, p);
}

}  // namespace

cudaError_t launch_tree_umma_f32(const PrefillParams& p, int D, int B, cudaStream_t s) {
    if (D == 64 && B == 16) return launch_f32<64, 16>(p, s);
    if (D == 64 && B == 32) return launch_f32<64, 32>(p, s);
    if (D == 128 && B == 16) return launch_f32<128, 16>(p, s);
    if (D == 128 && B == 32) return launch_f32<128, 32>(p, s);
    return cudaErrorNotSupported;
}

}  // namespace pa
