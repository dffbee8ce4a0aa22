// Attention of drafted trees on mma.sync, bf16 pools.
#include "pa_prefill_mma.cuh"

namespace pa {

cudaError_t launch_tree_mma_bf16(const PrefillParams& p, int D, int B, cudaStream_t s) {
    if (D == 64 && B == 16) return launch_mma_inst<CoreBf16<64>, 64, 16, true>(p, s);
    if (D == 64 && B == 32) return launch_mma_inst<CoreBf16<64>, 64, 32, true>(p, s);
    if (D == 128 && B == 16) return launch_mma_inst<CoreBf16<128>, 128, 16, true>(p, s);
    if (D == 128 && B == 32) return launch_mma_inst<CoreBf16<128>, 128, 32, true>(p, s);
    return cudaErrorNotSupported;
}

}  // namespace pa
