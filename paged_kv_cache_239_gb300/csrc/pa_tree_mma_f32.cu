// Attention of drafted trees on mma.sync, fp32 pools: by the rows of a tile.
#include "pa_prefill_mma.cuh"

namespace pa {

namespace {

template <int D, int B>
cudaError_t launch_rows(const PrefillParams& p, cudaStream_t s) {
    switch (p.row_tile) {
        case 16: return launch_mma_inst<CoreF32<D, 1>, D, B, true>(p, s);
        case 32: return launch_mma_inst<CoreF32<D, 2>, D, B, true>(p, s);
        default: return launch_mma_inst<CoreF32<D, 4>, D, B, true>(p, s);
    }
}

}  // namespace

cudaError_t launch_tree_mma_f32(const PrefillParams& p, int D, int B, cudaStream_t s) {
    if (D == 64 && B == 16) return launch_rows<64, 16>(p, s);
    if (D == 64 && B == 32) return launch_rows<64, 32>(p, s);
    if (D == 128 && B == 16) return launch_rows<128, 16>(p, s);
    if (D == 128 && B == 32) return launch_rows<128, 32>(p, s);
    return cudaErrorNotSupported;
}

}  // namespace pa
