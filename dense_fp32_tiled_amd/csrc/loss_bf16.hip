// loss_bf16.hip -- the cross entropy's logits for bf16 inputs.
#include <hip/hip_runtime.h>

#include "loss_shapes.hpp"

namespace dft {
hipError_t launch_loss_bf16(const LossRowsProblem& p, bool kmajor, LinearTile tile, uint32_t tiles_m, uint32_t tiles_n,
                           uint32_t slices, int cus, hipStream_t stream) {
    return launch_loss_logits<kInputBf16>(p, kmajor, tile, tiles_m, tiles_n, slices, cus, stream);
}
hipError_t launch_loss_bf16(const LossSlopeProblem& p, bool kmajor, LinearTile tile, uint32_t tiles_m, uint32_t tiles_n,
                           uint32_t slices, int cus, hipStream_t stream) {
    return launch_loss_logits<kInputBf16>(p, kmajor, tile, tiles_m, tiles_n, slices, cus, stream);
}
}  // namespace dft
