// Attention of drafted trees: which kernel a call takes, and how it is split.
#include <algorithm>

#include "pa_internal.h"

namespace pa {

namespace {

// The time of a call, in us, whose contexts are split in n parts: 2.5 to start, the join of more
// than eight parts, and the tiles of a part (and k0 more: its start and join) at `tile` each,
// which changes by `fill` of itself from empty to full row tiles, longer by `share` of the CTAs
// that an SM has.  Least squares over 43 calls of 1 to 48 trees at every row tile and n, all in
// tables as wide as the contexts; there the chosen ones take 5 % more than the best of each (fp32;
// tiles of 64 rows alone: 27 %) and 3 % (bf16, the choice of tcgen05 included).  The width stands
// for the lengths, so in wider tables the choice is worse: a tree of 8 nodes over 500 in a table of
// 8,192 blocks takes 9.9 us by choice and 8.7 on mma.sync by force (bf16; 6.3 in a tight table), on
// fp32 pools 13.1 and 11.0 (7.4).
struct TreeTime {
    double tile, k0, share, base, fill, join;
};
constexpr TreeTime kBf16[2] = {{1.14, 2.24, 0.59, 0.00, 0.47, 8.00}, {0.91, 4.80, 0.48, 0.48, 0.75, 2.59}};
constexpr TreeTime kF32[2][3] = {  // head_dim 64, 128; row tiles of 16, 32, 64
    {{1.70, 1.43, 0.68, 0.40, 0.00, 8.00}, {1.95, 1.66, 0.74, 0.53, 0.16, 3.58}, {1.74, 1.75, 0.50, 0.69, 0.54, 1.31}},
    {{1.90, 1.64, 0.63, 0.02, 0.00, 6.61}, {2.29, 1.53, 0.60, 0.04, 0.31, 6.48}, {2.22, 2.02, 0.44, 0.53, 0.68, 4.06}},
};

}  // namespace

double tree_mma_plan(int dtype, int G, int Hkv, int batch, int num_tokens, int maxb, int D, int B, int num_sms,
                     int* row_tile, int* splits, int* cluster) {
    const double rows = (double)num_tokens * G / batch;
    double best = 0;
    for (int rt = dtype == 1 ? 64 : 16, k = 0; rt <= 64; rt *= 2, ++k) {
        const TreeTime& t = dtype == 1 ? kBf16[D == 128] : kF32[D == 128][k];
        const int keys_per_tile = (dtype == 1 ? 64 : 32) / (D / 64) * (rt < 64 ? 2 : 1);
        const double keys = std::max(1.0, (double)maxb * B / keys_per_tile);
        const double tiles = (double)batch * Hkv * std::max(1.0, rows / rt + 0.3);
        const double tile = t.tile * (1 + t.fill * (std::min(rows, (double)rt) / rt - 0.5));
        for (int n = 1; n <= 64 && n <= keys; n *= 2) {
            const double time = 2.5 + (n > 8 ? t.join : 0) +
                                (keys / n + t.k0) * tile * std::max(1.0, t.share * tiles * n / num_sms + t.base);
            if (best == 0 || time < best) best = time, *row_tile = rt, *splits = n, *cluster = std::min(n, 8);
        }
    }
    return best;
}

// The tcgen05 kernel and its join: 9.4 us, the key tiles of each pair and 5.6 more for the pair
// dealt out to the SMs, and the parts of a pair that are joined, by their rows.
double tree_umma_time(int G, int Hkv, int batch, int num_tokens, int maxb, int D, int B, int num_sms) {
    const double rows = (double)num_tokens * G / batch, keys = (double)maxb * B;
    const double pairs = (double)batch * Hkv * std::max(1.0, rows / 256);
    const double parts = std::min(keys / 128 + 1, std::max(1.0, num_sms / pairs));
    return 9.4 + pairs * (5.6 + keys / 128) / num_sms * (D == 64 ? 0.86 : 1.18) +
           parts * std::min(256.0, std::max(32.0, rows)) * D * 2.7e-5;
}

// The same for the tcgen05 kernel on fp32 pools (one CTA per SM): start, the join of n parts by
// their bytes, the key tiles of a part and k0 more, times the rounds that the SMs take: beyond one, at
// least 1.7, for a few CTAs more than there are SMs wait for the others to end.  Least squares over 62
// calls at 1 to 64 parts in tight tables; the better of this and mma.sync by estimate takes 2.5 % more
// than the best (mma.sync for all: 22 %).  Four rounds at most: parts without keys, where the table is wider than
// the contexts, take a microsecond of an SM each (8 trees of 25 nodes over 2,000 keys, 32 heads on 8 of
// 128, in a table of 8,192 blocks: 61 us, 136 without the limit).
double tree_umma_f32_plan(int G, int Hkv, int batch, int num_tokens, int maxb, int D, int B, int num_sms,
                          int* splits) {
    struct Time {
        double start, join, bytes, k0, tile, rest;
    };
    const Time t = D == 64 ? Time{2.25, 1.91, 3.39, 2.66, 1.55, 0.44} : Time{4.93, 1.00, 2.38, 1.70, 2.43, 0.45};
    const double rows = (double)num_tokens * G / batch, keys = (double)maxb * B / 64;
    const double tiles = (double)batch * Hkv * std::max(1.0, rows / 128 + 0.3);
    const double out = 1e-6 * num_tokens * G * Hkv * D;
    double best = 0;
    for (int n = 1; n <= 64 && (n == 1 || (n <= keys && tiles * n <= 4 * num_sms)); ++n) {
        const double x = tiles * n / num_sms, rounds = x > 1 ? std::max(x + t.rest, 1.7) : 1.0;
        const double time = t.start + (n > 1 ? t.join + t.bytes * n * out : 0) + rounds * (keys / n + t.k0) * t.tile;
        if (n == 1 || time < best) best = time, *splits = n;
    }
    return best;
}

}  // namespace pa
