// Prefill attention on tcgen05: the grid and the causal kernels.
#include "pa_prefill_umma_launch.cuh"

namespace pa {

// One CTA per SM, unless there are fewer (pair, key tile) units than that: a
// sequence of n_b new tokens has at most n_b G / 256 + 1 pairs of 256 rows.
int prefill_umma_grid(int G, int Hkv, int batch, int num_tokens, int maxb, int B, int num_sms) {
    const long long pairs = ((long long)num_tokens * G / 256 + batch) * Hkv;
    const long long tiles = ((long long)maxb * B + 127) / 128;
    const long long units = pairs * tiles;
    return (int)(units < num_sms ? units : num_sms);
}

cudaError_t launch_prefill_umma(const PrefillParams& p, const void* tmaps, int D, int B,
                                cudaStream_t s) {
    return launch_umma<false>(p, tmaps, D, B, s);
}

}  // namespace pa
