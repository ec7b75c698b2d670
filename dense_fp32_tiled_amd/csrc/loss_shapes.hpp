// loss_shapes.hpp -- the loss's launches of the tile kernel, compiled once per
// input type.  Every operand has rows of whole 16 bytes (others are packed).
#pragma once

#include "loss_kernels.hpp"

namespace dft {

template <int TYPE, bool AK, bool BK_, class Shape, class Problem>
hipError_t launch_loss_shape(const Problem& p, uint32_t tiles_m, uint32_t tiles_n, uint32_t slices, int cus,
                             hipStream_t stream) {
    Problem problem = p;
    void* args[] = {&problem, &tiles_m, &tiles_n, &slices};
    uint32_t blocks = tiles_m * tiles_n * slices;
    if (Shape::PERSISTENT && blocks > (uint32_t)cus) blocks = (uint32_t)cus;
    return hipLaunchKernel(reinterpret_cast<const void*>(linear_tile_kernel<TYPE, AK, BK_, Shape, true, Problem>),
                           dim3(blocks), dim3(Shape::THREADS), args, 0, stream);
}
template <int TYPE, bool AK, bool BK_, class Problem>
hipError_t launch_loss_layout(const Problem& p, LinearTile tile, uint32_t tiles_m, uint32_t tiles_n, uint32_t slices,
                              int cus, hipStream_t stream) {
    if constexpr (Problem::SHORT)
        if (tile == kTileShort) return launch_loss_shape<TYPE, AK, BK_, ShortShape>(p, tiles_m, tiles_n, slices, cus, stream);
    switch (tile) {
        case kTile256: return launch_loss_shape<TYPE, AK, BK_, ShapeOf<kTile256>::type>(p, tiles_m, tiles_n, slices, cus, stream);
        case kTile128: return launch_loss_shape<TYPE, AK, BK_, ShapeOf<kTile128>::type>(p, tiles_m, tiles_n, slices, cus, stream);
        case kTile64: return launch_loss_shape<TYPE, AK, BK_, ShapeOf<kTile64>::type>(p, tiles_m, tiles_n, slices, cus, stream);
        default: return launch_loss_shape<TYPE, AK, BK_, ShapeOf<kTile32x128>::type>(p, tiles_m, tiles_n, slices, cus, stream);
    }
}

// The logits of a piece: B's words are its rows, or its columns.
template <int TYPE, class Problem>
hipError_t launch_loss_logits(const Problem& p, bool kmajor, LinearTile tile, uint32_t tiles_m, uint32_t tiles_n,
                              uint32_t slices, int cus, hipStream_t stream) {
    return kmajor ? launch_loss_layout<TYPE, true, true>(p, tile, tiles_m, tiles_n, slices, cus, stream)
                  : launch_loss_layout<TYPE, true, false>(p, tile, tiles_m, tiles_n, slices, cus, stream);
}

// What joins the slices of a gradient's product, of all of it or of its last round.
template <int TYPE, class Problem>
hipError_t launch_loss_join(const Problem& p, uint32_t tiles_m, uint32_t tiles_n, int cus, hipStream_t stream) {
    Problem problem = p;
    if (p.tail) {
        uint32_t grid = (uint32_t)cus < tiles_m * tiles_n ? (uint32_t)cus : tiles_m * tiles_n;
        void* args[] = {&problem, &tiles_m, &tiles_n, &grid};
        return hipLaunchKernel(reinterpret_cast<const void*>(linear_tail_kernel<TYPE, 256, 256, Problem>),
                               dim3(grid / 2, 256 / 32), dim3(256), args, 0, stream);
    }
    if (p.splits <= 1) return hipSuccess;
    const int64_t groups = (p.R * ((p.C + 7) / 8) + kJoinGroups - 1) / kJoinGroups;
    void* args[] = {&problem};
    return hipLaunchKernel(reinterpret_cast<const void*>(linear_join_kernel<TYPE, Problem>),
                           dim3((unsigned)(groups < 16384 ? groups : 16384)), dim3(kJoinThreads), args, 0, stream);
}

}  // namespace dft
