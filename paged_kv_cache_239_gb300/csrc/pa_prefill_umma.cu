// Prefill attention on tcgen05: instantiations and launch.
#include <cuda.h>
#include <cuda_runtime.h>

#include <mutex>

#include "pa_prefill_umma.cuh"

namespace pa {

namespace {

template <int D, int B, bool TURNS>
cudaError_t launch_turns(const PrefillParams& p, const CUtensorMap* tm, cudaStream_t s) {
    using C = PrefillCfg<D, B>;
    auto kern = pa_prefill_umma_kernel<D, B, TURNS>;
    static std::mutex mu;
    static unsigned long long done_mask = 0;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    {
        std::lock_guard<std::mutex> lock(mu);
        const unsigned long long bit = 1ull << (dev & 63);
        if (!(done_mask & bit)) {
            e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     C::SMEM_BYTES);
            if (e != cudaSuccess) return e;
            done_mask |= bit;
        }
    }
    CUtensorMap tq{};  // (not used for groups above 64 that do not divide 128)
    if (128 % p.G == 0 || p.G <= 64) {
        e = encode_heads_tmap(&tq, p.q, D, p.H, p.num_tokens, p.G, 128 % p.G == 0 ? 128 / p.G : 1);
        if (e != cudaSuccess) return e;
    }
    e = launch_pdl(kern, dim3((unsigned)p.grid), dim3(C::THREADS), C::SMEM_BYTES, s, p, tm[0], tm[1], tq);
    if (e != cudaSuccess || p.grid == 1) return e;
    return launch_pdl(pa_prefill_umma_join_kernel<D>, dim3((unsigned)p.grid, kJoinParts),
                      dim3(256), 0, s, p);
}

// Calls with 128 rows to a sequence on average, or fewer, take the kernel in which
// both softmax groups serve a single row tile in turns (3 - 5 tokens over 4 long
// contexts: 150 us, 167 without); it has more code, which costs calls of many pairs
// of row tiles 5 - 15 %, so they take the one without.
template <int D, int B>
cudaError_t launch_inst(const PrefillParams& p, const CUtensorMap* tm, cudaStream_t s) {
    return (long long)p.num_tokens * p.G <= 128LL * p.batch ? launch_turns<D, B, true>(p, tm, s)
                                                            : launch_turns<D, B, false>(p, tm, s);
}

}  // namespace

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
    const CUtensorMap* tm = static_cast<const CUtensorMap*>(tmaps);
    if (D == 64 && B == 16) return launch_inst<64, 16>(p, tm, s);
    if (D == 64 && B == 32) return launch_inst<64, 32>(p, tm, s);
    if (D == 128 && B == 16) return launch_inst<128, 16>(p, tm, s);
    if (D == 128 && B == 32) return launch_inst<128, 32>(p, tm, s);
    return cudaErrorNotSupported;
}

}  // namespace pa
