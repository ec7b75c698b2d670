// slope_kernels.hpp -- gfx950 kernels of the epilogue's gradient.
//
// dZ = dY act'(Z), rounded to 16 bits for the two products that read it, and
// the column sums of the unrounded values (dbias): each workgroup sums a
// chunk of 16 or 64 rows of one group over 256 columns into
// partial[chunk][column]; linear_bias_join_kernel adds a group's chunks in
// ascending order.  Bound by bytes: dY and Z read once, dZ written once:
// 8192x8192 with silu 98 us (4.1 TB/s of 403 MB), the join 5 us.
#pragma once

#include "linear_kernels.hpp"

namespace dft {

// Rows per chunk: 64, or 16 where 64 would leave fewer workgroups than keep the
// chip's loads in flight (slope_rows).
constexpr int kSlopeRows = 64, kFewSlopeRows = 16;

struct SlopeProblem {
    int64_t M, N;
    const uint16_t* dY;
    int64_t ldy;
    const uint16_t* Z;
    int64_t ldz;
    uint16_t* dZ;                // nullptr: the sums alone (no activation)
    int64_t lddz;
    float* partial;              // nullptr: no sums wanted
    const int32_t* offsets;
    int32_t groups;
    int32_t act;
    int32_t chunk_rows;
    int64_t chunks;              // places in partial
    float* dbias;                // groups x N, rows N apart
};

template <int TYPE>
__global__ __launch_bounds__(256) void linear_slope_kernel(SlopeProblem p) {
    __shared__ float sums[8][256 + 8];
    const int c = threadIdx.x % 32, r = threadIdx.x / 32;
    const int64_t chunk = blockIdx.x, col = (int64_t)blockIdx.y * 256 + c * 8, left = p.N - col;
    int64_t lo = chunk * p.chunk_rows, hi = p.M;
    if (p.offsets) {
        const GroupTile gt = find_group_tile(p.offsets, p.groups, p.M, p.chunk_rows, chunk);
        if (gt.group < 0) return;
        lo = gt.row0;
        hi = gt.row_end;
    }
    if (hi > lo + p.chunk_rows) hi = lo + p.chunk_rows;
    float sum[8] = {};
    auto rows = [&](auto WHOLE_) {  // (columns wholly inside the matrix: no masks)
        const int64_t in = decltype(WHOLE_)::value ? (int64_t)8 : left;
#pragma unroll 4
        for (int64_t row = lo + r; row < hi; row += 8) {
            float d[8];
            load8(p.dY + row * p.ldy + col, in).widen<TYPE>(d);
            if (p.dZ) {
                float z[8];
                load8(p.Z + row * p.ldz + col, in).widen<TYPE>(z);
                act_slopes(z, p.act);
#pragma unroll
                for (int e = 0; e < 8; ++e) d[e] *= z[e];
                store8(p.dZ + row * p.lddz + col, Row8::narrow<TYPE>(d), in);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[e] += d[e];
        }
    };
    if ((int64_t)(blockIdx.y + 1) * 256 <= p.N)
        rows(std::true_type{});
    else if (left > 0)
        rows(std::false_type{});
    if (!p.partial) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) sums[r][c * 8 + e] = sum[e];
    __syncthreads();
    const int64_t at = (int64_t)blockIdx.y * 256 + threadIdx.x;
    if (at < p.N) {
        float total = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) total += sums[k][threadIdx.x];
        p.partial[chunk * p.N + at] = total;
    }
}

// dbias[group][column] over that group's chunks: 64 columns by 4 strides of
// chunks per workgroup.
__global__ __launch_bounds__(256) void linear_bias_join_kernel(SlopeProblem p) {
    __shared__ float sums[4][64];
    const int c = threadIdx.x % 64, r = threadIdx.x / 64;
    const int64_t col = (int64_t)blockIdx.x * 64 + c;
    const int group = blockIdx.y;
    int64_t first = 0, rows = p.M;
    if (p.offsets) {
        // chunks of the groups before this one, by the same rule as find_group_tile
        int64_t before = 0;
        for (int g = c; g < group; g += 64) {
            const RowRange range = group_rows(p.offsets, g, p.M);
            before += (range.hi - range.lo + p.chunk_rows - 1) / p.chunk_rows;
        }
#pragma unroll
        for (int d = 32; d > 0; d /= 2) before += __shfl_xor((int)before, d);
        first = before;
        const RowRange own = group_rows(p.offsets, group, p.M);
        rows = own.hi - own.lo;
    }
    int64_t chunks = (rows + p.chunk_rows - 1) / p.chunk_rows;
    if (chunks > p.chunks - first) chunks = p.chunks - first;  // (groups that overlap have more chunks than places)
    float sum = 0.0f;
    if (col < p.N) {
#pragma unroll 8
        for (int64_t k = r; k < chunks; k += 4) sum += p.partial[(first + k) * p.N + col];
    }
    sums[r][c] = sum;
    __syncthreads();
    if (r == 0 && col < p.N) p.dbias[group * p.N + col] = sums[0][c] + sums[1][c] + sums[2][c] + sums[3][c];
}

}  // namespace dft
