// linear_bf16.hip -- the products with an epilogue for bf16 inputs.
#include <hip/hip_runtime.h>

#include "linear_shapes.hpp"

namespace dft {
hipError_t launch_linear_bf16(const LinearProblem& p, LinearLayout layout, LinearTile tile, bool direct,
                              uint32_t tiles_m, uint32_t tiles_n, uint32_t grid_y, int cus, hipStream_t stream) {
    return launch_linear<kInputBf16>(p, layout, tile, direct, tiles_m, tiles_n, grid_y, cus, stream);
}
}  // namespace dft
