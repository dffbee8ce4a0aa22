// Attention of several new tokens on mma.sync: when a call takes it, how it is split, and
// the causal kernels.
#include <algorithm>

#include "pa_prefill_mma.cuh"

namespace pa {

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
    const long long tiles = ((long long)num_tokens * G / CoreF32<64>::BM + batch) * Hkv;
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
        if (D == 64 && B == 16) return launch_mma_inst<CoreBf16<64>, 64, 16, false>(p, s);
        if (D == 64 && B == 32) return launch_mma_inst<CoreBf16<64>, 64, 32, false>(p, s);
        if (D == 128 && B == 16) return launch_mma_inst<CoreBf16<128>, 128, 16, false>(p, s);
        if (D == 128 && B == 32) return launch_mma_inst<CoreBf16<128>, 128, 32, false>(p, s);
    } else {
        if (D == 64 && B == 16) return launch_mma_inst<CoreF32<64>, 64, 16, false>(p, s);
        if (D == 64 && B == 32) return launch_mma_inst<CoreF32<64>, 64, 32, false>(p, s);
        if (D == 128 && B == 16) return launch_mma_inst<CoreF32<128>, 128, 16, false>(p, s);
        if (D == 128 && B == 32) return launch_mma_inst<CoreF32<128>, 128, 32, false>(p, s);
    }
    return cudaErrorNotSupported;
}

}  // namespace pa
