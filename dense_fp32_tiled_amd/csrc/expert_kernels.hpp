// expert_kernels.hpp -- gfx950 kernels that sort (token, choice) pairs by
// expert, lay the tokens' rows out in that order, and bring the experts' rows
// back, with their gradients.
//
//   position[t][j] = offsets[e] + (pairs of expert e before pair (t, j)),  e = experts[t][j]
//   rows[position[t][j]] = x[t]
//   out[t] = sum over j of weights[t][j] * y[position[t][j]]
//   dy[position[t][j]] = weights[t][j] * dout[t],   dweights[t][j] = y[position[t][j]] . dout[t]
//
// The sort is stable (pairs of one expert stay in token order) and uses no
// atomics whose order could change a result.  The row kernels are bound by
// bytes: every row is read once and written once; sums are held in fp32.
#pragma once

#include "linear_kernels.hpp"

namespace dft {

constexpr int kSortWaves = 16, kSortThreads = kSortWaves * kWave;
constexpr int kWavePairs = 256, kSortPairs = kSortWaves * kWavePairs;  // pairs per wave and per workgroup
constexpr int kMaxExperts = 1024;

struct SortProblem {
    const int32_t* experts;
    int64_t pairs;
    int32_t num_experts;
    int32_t* offsets;
    int32_t* order;
    int32_t* position;
    int32_t* counts;  // workgroups x num_experts: pairs of each, then the pairs before each
};

// An expert that does not exist drops the pair.
__device__ inline int pair_expert(const SortProblem& p, int64_t pair) {
    if (pair >= p.pairs) return -1;
    const int e = p.experts[pair];
    return e >= 0 && e < p.num_experts ? e : -1;
}

// Lanes of this wave whose pair has the same expert (none for a dropped one).
__device__ inline uint64_t same_expert(int e) {
    uint64_t same = __ballot(e >= 0);
#pragma unroll
    for (int bit = 0; bit < 10; ++bit) {
        const uint64_t set = __ballot((e >> bit) & 1);
        same &= (e >> bit) & 1 ? set : ~set;
    }
    return e >= 0 ? same : 0;
}

// Counts each wave's pairs per expert into `counts` (kSortWaves x experts),
// then turns them into the pairs of the earlier waves; returns through
// `totals` the workgroup's pairs per expert.
__device__ inline void count_by_wave(const SortProblem& p, int64_t first, uint16_t* counts, int32_t* totals) {
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave, E = p.num_experts;
    for (int i = tid; i < kSortWaves * E; i += kSortThreads) counts[i] = 0;
    __syncthreads();
    for (int k = 0; k < kWavePairs && first + wave * kWavePairs + k < p.pairs; k += kWave) {
        const int e = pair_expert(p, first + wave * kWavePairs + k + lane);
        const uint64_t same = same_expert(e);
        if (e >= 0 && lane == __builtin_ctzll(same)) counts[wave * E + e] += (uint16_t)__popcll(same);
        wave_fence();
    }
    __syncthreads();
    for (int e = tid; e < E; e += kSortThreads) {
        int before = 0;
        for (int w = 0; w < kSortWaves; ++w) {
            const int own = counts[w * E + e];
            counts[w * E + e] = (uint16_t)before;
            before += own;
        }
        totals[e] = before;
    }
    __syncthreads();
}

// Exclusive running sum of values[0 .. n) (n <= kSortThreads) by the whole
// workgroup; returns the sum of all.
__device__ inline int running_sum(int32_t* values, int n, int32_t* wave_sums) {
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    const int own = tid < n ? values[tid] : 0;
    int upto = own;
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) {
        const int other = __shfl_up(upto, d);
        if (lane >= d) upto += other;
    }
    if (lane == kWave - 1) wave_sums[wave] = upto;
    __syncthreads();
    int before = 0, all = 0;
    for (int w = 0; w < kSortWaves; ++w) {
        if (w < wave) before += wave_sums[w];
        all += wave_sums[w];
    }
    if (tid < n) values[tid] = before + upto - own;
    __syncthreads();
    return all;
}

// Writes this workgroup's pairs: `start` holds each expert's first slot for them.
__device__ inline void place_pairs(const SortProblem& p, int64_t first, uint16_t* counts, const int32_t* start,
                                   int64_t sorted) {
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave, E = p.num_experts;
    for (int k = 0; k < kWavePairs && first + wave * kWavePairs + k < p.pairs; k += kWave) {
        const int64_t pair = first + wave * kWavePairs + k + lane;
        const int e = pair_expert(p, pair);
        const uint64_t same = same_expert(e);
        int slot = -1;
        if (e >= 0) slot = start[e] + counts[wave * E + e] + __popcll(same & (((uint64_t)1 << lane) - 1));
        wave_fence();
        if (e >= 0 && lane == __builtin_ctzll(same)) counts[wave * E + e] += (uint16_t)__popcll(same);
        wave_fence();
        if (pair < p.pairs) {
            p.position[pair] = slot;
            if (slot >= 0) p.order[slot] = (int32_t)pair;
            if (pair >= sorted) p.order[pair] = -1;  // slots that no pair takes
        }
    }
}

// All pairs in one workgroup: counts, offsets and places in one launch.  Bound
// by the latency of its steps: 3.5 us for 64 pairs, 9 us for 4096.
__global__ __launch_bounds__(kSortThreads) void expert_sort_small_kernel(SortProblem p) {
    __shared__ uint16_t counts[kSortWaves * kMaxExperts];
    __shared__ int32_t start[kMaxExperts];
    __shared__ int32_t wave_sums[kSortWaves];
    count_by_wave(p, 0, counts, start);
    const int sorted = running_sum(start, p.num_experts, wave_sums);
    for (int e = threadIdx.x; e < p.num_experts; e += kSortThreads) p.offsets[e] = start[e];
    if (threadIdx.x == 0) p.offsets[p.num_experts] = sorted;
    place_pairs(p, 0, counts, start, sorted);
}

// The same over several workgroups: counts of each, their running sums, places
// (5 + 6 to 8 + 10 us for 65536 pairs of 64 experts; the pairs' bytes would take 1 us).
__global__ __launch_bounds__(kSortThreads) void expert_count_kernel(SortProblem p) {
    __shared__ int32_t totals[kMaxExperts];
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    for (int e = tid; e < p.num_experts; e += kSortThreads) totals[e] = 0;
    __syncthreads();
    const int64_t first = (int64_t)blockIdx.x * kSortPairs;
    for (int k = 0; k < kWavePairs; k += kWave) {
        const int e = pair_expert(p, first + wave * kWavePairs + k + lane);
        if (e >= 0) atomicAdd(&totals[e], 1);  // (whole numbers: any order gives the same)
    }
    __syncthreads();
    for (int e = tid; e < p.num_experts; e += kSortThreads) p.counts[(int64_t)blockIdx.x * p.num_experts + e] = totals[e];
}

__global__ __launch_bounds__(kSortThreads) void expert_offsets_kernel(SortProblem p, int64_t workgroups) {
    __shared__ int32_t start[kMaxExperts];
    __shared__ int32_t wave_sums[kSortWaves];
    const int e = threadIdx.x, E = p.num_experts;
    if (e < E) {
        int total = 0;
        for (int64_t b = 0; b < workgroups; ++b) total += p.counts[b * E + e];
        start[e] = total;
    }
    __syncthreads();
    const int sorted = running_sum(start, E, wave_sums);
    if (e < E) {
        int before = start[e];
        p.offsets[e] = before;
        for (int64_t b = 0; b < workgroups; ++b) {
            const int own = p.counts[b * E + e];
            p.counts[b * E + e] = before;
            before += own;
        }
    }
    if (e == 0) p.offsets[E] = sorted;
}

__global__ __launch_bounds__(kSortThreads) void expert_place_kernel(SortProblem p) {
    __shared__ uint16_t counts[kSortWaves * kMaxExperts];
    __shared__ int32_t start[kMaxExperts];
    const int64_t first = (int64_t)blockIdx.x * kSortPairs;
    count_by_wave(p, first, counts, start);
    for (int e = threadIdx.x; e < p.num_experts; e += kSortThreads)
        start[e] = p.counts[(int64_t)blockIdx.x * p.num_experts + e];
    __syncthreads();
    place_pairs(p, first, counts, start, p.offsets[p.num_experts]);
}

// ---- rows ---------------------------------------------------------------------------
struct RowsProblem {
    int64_t tokens, rows, cols;  // rows: sorted rows
    int32_t top_k;
    uint32_t parts;              // waves per token: ceil(cols / kRowCols)
    int64_t step;                // tokens that the grid covers at a time
    const int32_t* position;
    const float* weights;        // tokens x top_k, or nullptr (ones)
    const uint16_t* x;           // token rows: the gather's source, the gradient's dout
    int64_t ldx;
    const uint16_t* y;           // sorted rows read
    int64_t ldy;
    uint16_t* out;               // token rows written
    int64_t ldo;
    uint16_t* sorted;            // sorted rows written
    int64_t lds;
    float* dweights;
};
constexpr int kRowCols = kWave * 8;  // columns per wave
constexpr int kRowWaves = 4;

// Position of choice j of a token; -1 (dropped) for any slot outside the sorted rows.
__device__ inline int64_t slot_of(const RowsProblem& p, int64_t token, int j) {
    const int64_t s = p.position[token * p.top_k + j];
    return s >= 0 && s < p.rows ? s : -1;
}

// This wave's first token and its lane's first column: a wave takes 512 columns
// of one token, the waves of a token follow each other (a row's lines are asked
// for together: 147 us for combining 16384 x 4 rows of 4096, 185 with all
// tokens' first columns first).  The token is uniform, so positions and weights
// come through scalar loads.
__device__ inline bool row_place(const RowsProblem& p, int64_t& token, int64_t& col) {
    const uint32_t wave = __builtin_amdgcn_readfirstlane(blockIdx.x * kRowWaves + threadIdx.x / kWave);
    token = wave / p.parts;
    col = (int64_t)(wave % p.parts) * kRowCols + threadIdx.x % kWave * 8;
    return token < p.step && col < p.cols;
}

// The token's columns read once, written to each of its slots: 105 us for
// 16384 tokens, 4 choices, 4096 columns (6.4 TB/s of 671 MB; mostly stores,
// which go faster than a copy's 5.1).
__global__ __launch_bounds__(kRowWaves* kWave) void expert_gather_kernel(RowsProblem p) {
    int64_t token, col;
    if (!row_place(p, token, col)) return;
    const int64_t left = p.cols - col;
    for (; token < p.tokens; token += p.step) {
        const Row8 v = load8(p.x + token * p.ldx + col, left);
        for (int j = 0; j < p.top_k; ++j) {
            const int64_t s = slot_of(p, token, j);
            if (s >= 0) store8(p.sorted + s * p.lds + col, v, left);
        }
    }
}

// Choices summed in ascending order in fp32 and rounded once; four of them at a
// time, so that their positions, then their rows, are on their way together:
// 147 us at the same sizes (4.6 TB/s of 671 MB).
template <int TYPE>
__global__ __launch_bounds__(kRowWaves* kWave) void expert_combine_kernel(RowsProblem p) {
    int64_t token, col;
    if (!row_place(p, token, col)) return;
    const int64_t left = p.cols - col;
    for (; token < p.tokens; token += p.step) {
        float sum[8] = {};
        for (int j0 = 0; j0 < p.top_k; j0 += 4) {
            int64_t slot[4];
            float w[4];
            Row8 row[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bool there = j0 + j < p.top_k;
                const int choice = there ? j0 + j : j0;
                const int64_t s = slot_of(p, token, choice);
                slot[j] = there ? s : -1;
                w[j] = p.weights ? p.weights[token * p.top_k + choice] : 1.0f;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (slot[j] >= 0) row[j] = load8(p.y + slot[j] * p.ldy + col, left);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (slot[j] < 0) continue;
                float v[8];
                row[j].widen<TYPE>(v);
#pragma unroll
                for (int e = 0; e < 8; ++e) sum[e] += w[j] * v[e];
            }
        }
        store8(p.out + token * p.ldo + col, Row8::narrow<TYPE>(sum), left);
    }
}

// dy of each of a token's slots, and each choice's dot product (lane sums, then
// the wave's by halves, then (0+1)+(2+3): one order whatever the grid).  One
// workgroup per token reads dout from HBM once: 240 us at the same sizes (5.0
// TB/s of 1.2 GB).  With fewer tokens than fill the chip, one per choice
// (gridDim.y): 16 tokens 3.5 against 7.7 us, 512 tokens 8.5 against 11.4; from
// four tokens per CU on both take the same.
template <int TYPE>
__global__ __launch_bounds__(kRowWaves* kWave) void expert_combine_grad_kernel(RowsProblem p) {
    __shared__ float sums[kRowWaves];
    for (int64_t token = blockIdx.x; token < p.tokens; token += p.step) {
        for (int j = blockIdx.y; j < p.top_k; j += gridDim.y) {
            const int64_t s = slot_of(p, token, j);  // uniform
            const int64_t pair = token * p.top_k + j;
            float dot = 0.0f;
            if (s >= 0) {
                const float w = p.weights ? p.weights[pair] : 1.0f;
                for (int64_t col = threadIdx.x * 8; col < p.cols; col += kRowWaves * kRowCols) {
                    const int64_t left = p.cols - col;
                    float d[8];
                    load8(p.x + token * p.ldx + col, left).widen<TYPE>(d);
                    if (p.dweights) {
                        float v[8];
                        load8(p.y + s * p.ldy + col, left).widen<TYPE>(v);
#pragma unroll
                        for (int e = 0; e < 8; ++e) dot += d[e] * v[e];
                    }
                    if (p.sorted) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) d[e] *= w;
                        store8(p.sorted + s * p.lds + col, Row8::narrow<TYPE>(d), left);
                    }
                }
            }
            if (!p.dweights) continue;
#pragma unroll
            for (int d = kWave / 2; d > 0; d /= 2) dot += __shfl_xor(dot, d);
            __syncthreads();  // the sums of the choice before have been read
            if (threadIdx.x % kWave == 0) sums[threadIdx.x / kWave] = dot;
            __syncthreads();
            if (threadIdx.x == 0) p.dweights[pair] = (sums[0] + sums[1]) + (sums[2] + sums[3]);
        }
    }
}

}  // namespace dft
