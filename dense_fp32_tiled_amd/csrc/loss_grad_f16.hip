// loss_grad_f16.hip -- the products of the cross entropy's gradients for fp16 inputs.
#include <hip/hip_runtime.h>

#include "loss_shapes.hpp"

namespace dft {
// dB, or its transpose: dZ and A both run along the output.
hipError_t launch_loss_f16(const LossWordsGradProblem& p, bool, LinearTile tile, uint32_t tiles_m, uint32_t tiles_n,
                           uint32_t slices, int cus, hipStream_t stream) {
    const hipError_t e = launch_loss_layout<kInputF16, false, false>(p, tile, tiles_m, tiles_n, slices, cus, stream);
    return e == hipSuccess ? launch_loss_join<kInputF16>(p, tiles_m, tiles_n, cus, stream) : e;
}
// dA = dZ B^T: B's words, which the contraction runs over, are its rows or its columns.
hipError_t launch_loss_f16(const LossTokensGradProblem& p, bool kmajor, LinearTile tile, uint32_t tiles_m,
                           uint32_t tiles_n, uint32_t slices, int cus, hipStream_t stream) {
    const hipError_t e = kmajor ? launch_loss_layout<kInputF16, true, false>(p, tile, tiles_m, tiles_n, slices, cus, stream)
                                : launch_loss_layout<kInputF16, true, true>(p, tile, tiles_m, tiles_n, slices, cus, stream);
    return e == hipSuccess ? launch_loss_join<kInputF16>(p, tiles_m, tiles_n, cus, stream) : e;
}
}  // namespace dft
