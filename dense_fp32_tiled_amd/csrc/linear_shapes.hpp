// linear_shapes.hpp -- the tile kernel's shapes and the launch of one of them,
// shared by the translation units that compile it (one per input type).
#pragma once

#include "linear_kernels.hpp"

namespace dft {

// Workgroup tiles, largest first.  256x256 has eight waves of 128x64 and one
// persistent workgroup per CU (a ring of five 32 KiB places: all 160 KiB of
// LDS); 128x128 four waves of 64x64 and two per CU; 64x64 four of 32x32 with
// four stages.  32x128 is for few rows: its four waves share the 32 rows and
// stream 128 columns of B through four stages, so that two workgroups keep 96
// KiB of copies in flight per CU.  Measured (dA of grouped rows): 8192 rows in
// 8 groups by 1024, 4096 deep: 89 us with 256x256, 98 with 128x128, 128 with
// 64x64; 64 rows in 16 groups by 2048, 2048 deep: 22.6 us with 64x64, 25.9
// with 128x128, 42.7 with 256x256; 500 rows in 16 groups by 1000, 1496 deep:
// 15.3 us with 32x128, 18.8 with 64x64, 38.6 with 256x256.
enum LinearTile { kTile256 = 0, kTile128 = 1, kTile64 = 2, kTile32x128 = 3, kTileCount = 4 };
struct TileSize {
    int bm, bn;
};
constexpr TileSize kTileSizes[kTileCount] = {{256, 256}, {128, 128}, {64, 64}, {32, 128}};
constexpr int kTileDepth = kDepth;  // contraction elements per tile

template <int TILE>
struct ShapeOf;
template <>
struct ShapeOf<kTile256> { using type = LinearShape<256, 256, 128, 64, 2, 2, true>; };
template <>
struct ShapeOf<kTile128> { using type = LinearShape<128, 128, 64, 64, 2, 2>; };
template <>
struct ShapeOf<kTile64> { using type = LinearShape<64, 64, 32, 32, 4, 2>; };
template <>
struct ShapeOf<kTile32x128> { using type = LinearShape<32, 128, 32, 32, 4, 2>; };

// Which operands run along the contraction.
enum LinearLayout { kForward = 0, kGradA = 1, kGradB = 2 };

// Launches the product of `tile`; `direct`: every row and width of both
// operands is a multiple of 16 bytes.  grid_y: groups of the contraction, or
// slices.
template <int TYPE, bool AK, bool BK_, int TILE, bool DIRECT>
hipError_t launch_linear_tile(const LinearProblem& p, uint32_t tiles_m, uint32_t tiles_n, uint32_t grid_y,
                              int cus, hipStream_t stream) {
    using Shape = typename ShapeOf<TILE>::type;
    LinearProblem problem = p;
    void* args[] = {&problem, &tiles_m, &tiles_n, &grid_y};
    uint32_t blocks = tiles_m * tiles_n * grid_y;
    if (Shape::PERSISTENT && DIRECT && blocks > (uint32_t)cus) blocks = (uint32_t)cus;
    return hipLaunchKernel(reinterpret_cast<const void*>(linear_tile_kernel<TYPE, AK, BK_, Shape, DIRECT>),
                           dim3(blocks), dim3(Shape::THREADS), args, 0, stream);
}

template <int TYPE, bool AK, bool BK_>
hipError_t launch_linear_layout(const LinearProblem& p, LinearTile tile, bool direct, uint32_t tiles_m,
                                uint32_t tiles_n, uint32_t grid_y, int cus, hipStream_t stream) {
    switch (tile) {
        // (through registers the 256x256 tile's staged groups would not fit beside its sums: 128x128 is the largest)
        case kTile256: return launch_linear_tile<TYPE, AK, BK_, kTile256, true>(p, tiles_m, tiles_n, grid_y, cus, stream);
        case kTile128:
            return direct ? launch_linear_tile<TYPE, AK, BK_, kTile128, true>(p, tiles_m, tiles_n, grid_y, cus, stream)
                          : launch_linear_tile<TYPE, AK, BK_, kTile128, false>(p, tiles_m, tiles_n, grid_y, cus, stream);
        case kTile64:
            return direct ? launch_linear_tile<TYPE, AK, BK_, kTile64, true>(p, tiles_m, tiles_n, grid_y, cus, stream)
                          : launch_linear_tile<TYPE, AK, BK_, kTile64, false>(p, tiles_m, tiles_n, grid_y, cus, stream);
        default:
            return direct ? launch_linear_tile<TYPE, AK, BK_, kTile32x128, true>(p, tiles_m, tiles_n, grid_y, cus, stream)
                          : launch_linear_tile<TYPE, AK, BK_, kTile32x128, false>(p, tiles_m, tiles_n, grid_y, cus, stream);
    }
}

template <int TYPE>
hipError_t launch_linear(const LinearProblem& p, LinearLayout layout, LinearTile tile, bool direct, uint32_t tiles_m,
                         uint32_t tiles_n, uint32_t grid_y, int cus, hipStream_t stream) {
    switch (layout) {
        case kForward: return launch_linear_layout<TYPE, true, false>(p, tile, direct, tiles_m, tiles_n, grid_y, cus, stream);
        case kGradA: return launch_linear_layout<TYPE, true, true>(p, tile, direct, tiles_m, tiles_n, grid_y, cus, stream);
        default: return launch_linear_layout<TYPE, false, false>(p, tile, direct, tiles_m, tiles_n, grid_y, cus, stream);
    }
}

hipError_t launch_linear_bf16(const LinearProblem&, LinearLayout, LinearTile, bool, uint32_t, uint32_t, uint32_t, int,
                              hipStream_t);
hipError_t launch_linear_f16(const LinearProblem&, LinearLayout, LinearTile, bool, uint32_t, uint32_t, uint32_t, int,
                             hipStream_t);

}  // namespace dft
