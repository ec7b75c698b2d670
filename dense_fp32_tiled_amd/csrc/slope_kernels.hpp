// slope_kernels.hpp -- gfx950 kernels of the epilogue's gradient, and the copies
// of operands of odd widths.
//
// dZ = dY act'(Z), rounded to 16 bits for the two products that read it, and
// the column sums of the unrounded values (dbias): each workgroup sums a
// chunk of 16 or 64 rows of one group over 256 columns into
// partial[chunk][column]; bias_join adds a group's chunks in a fixed order.  A
// single chunk's sums are dbias itself.  Bound by bytes: dY and Z read once, dZ written once:
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
    float* partial;              // the sums of chunk c at partial + c * N; nullptr: no sums wanted
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
// chunks per workgroup, workgroup (across, group) of ceil(N / 64) x groups.
__device__ inline void bias_join(const SlopeProblem& p, uint32_t across, int group) {
    __shared__ float sums[4][64];
    const int c = threadIdx.x % 64, r = threadIdx.x / 64;
    const int64_t col = (int64_t)across * 64 + c;
    int64_t first = 0, rows = p.M;
    if (p.offsets) {
        // chunks of the groups before this one, by the same rule as find_group_tile: as many as there are places at
        // most, so that the lanes' sums stay inside 32 bits and `first` inside partial
        int64_t own_chunks = 0;
        for (int g = c; g < group; g += 64) own_chunks += group_rows(p.offsets, g, p.M).tiles(p.chunk_rows);
        int before = count_at_most(own_chunks, p.chunks);
#pragma unroll
        for (int d = 32; d > 0; d /= 2) before = count_at_most((int64_t)before + __shfl_xor(before, d), p.chunks);
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
    __syncthreads();  // the sums of the call before have been read
    sums[r][c] = sum;
    __syncthreads();
    if (r == 0 && col < p.N) p.dbias[group * p.N + col] = sums[0][c] + sums[1][c] + sums[2][c] + sums[3][c];
}
__global__ __launch_bounds__(256) void linear_bias_join_kernel(SlopeProblem p) {
    bias_join(p, blockIdx.x, blockIdx.y);
}

// Copies matrices to rows of whole 16 bytes (zeros past their width): what
// lets a product of unaligned operands run on direct copies.  Bound by bytes,
// at small sizes by latency: 6.8 us for 1000x999, 1000x513 and 513x999 at once,
// which the two products that read them win back (64 us without).
struct PackJob {
    const uint16_t* src;
    int64_t rows, cols, ld, copies, copy_stride;
    uint16_t* dst;
    int64_t ldd;  // a multiple of 8; copies lie rows * ldd apart
};
struct PackJobs {
    PackJob job[3];
};
// The row of workgroups after the jobs' joins dbias: a launch less (all
// gradients of 1000x999x513: 33.0 against 35.4 us).
__global__ __launch_bounds__(256) void linear_pack_kernel(PackJobs jobs, int count, SlopeProblem bias) {
    if ((int)blockIdx.y >= count) {
        const uint32_t across = (uint32_t)((bias.N + 63) / 64);
        for (uint64_t block = blockIdx.x; block < (uint64_t)across * bias.groups; block += gridDim.x)
            bias_join(bias, (uint32_t)(block % across), (int)(block / across));
        return;
    }
    const PackJob& j = jobs.job[blockIdx.y];
    const int64_t groups = j.ldd / 8, total = j.copies * j.rows * groups;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t at = i / groups, col = i % groups * 8, copy = at / j.rows, row = at % j.rows;
        const Row8 v = load8(j.src + copy * j.copy_stride + row * j.ld + col, j.cols - col);
        *reinterpret_cast<u32x4*>(j.dst + at * j.ldd + col) = v.w;
    }
}

}  // namespace dft
