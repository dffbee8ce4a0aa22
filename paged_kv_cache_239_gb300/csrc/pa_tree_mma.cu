// Attention of drafted trees on mma.sync: the kernels with a mask for each token.
#include "pa_prefill_mma.cuh"

namespace pa {

cudaError_t launch_tree_mma(const PrefillParams& p, int dtype, int D, int B, cudaStream_t s) {
    return launch_mma<true>(p, dtype, D, B, s);
}

}  // namespace pa
