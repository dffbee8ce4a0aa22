// Attention of drafted trees on tcgen05: the kernels with a mask for each token.
#include "pa_prefill_umma_launch.cuh"

namespace pa {

cudaError_t launch_tree_umma(const PrefillParams& p, const void* tmaps, int D, int B,
                             cudaStream_t s) {
    return launch_umma<true>(p, tmaps, D, B, s);
}

}  // namespace pa
