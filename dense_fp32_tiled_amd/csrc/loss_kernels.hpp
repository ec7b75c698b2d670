// loss_kernels.hpp -- gfx950 kernels of the cross entropy of a product over a
// vocabulary, whose logits are never stored, and of its gradients.
//
//   Z = A B  (M tokens by N words),  lse = log sum exp Z,  loss = lse - Z[target]
//   dZ = (exp(Z - lse) - onehot(target)) dloss,  dA = dZ B^T,  dB = A^T dZ
//
// The forward pass runs the tile kernel of linear_kernels.hpp with an epilogue
// that takes each row's maximum and sum of exponentials over a wave's columns
// straight from the matrix instructions' registers, and the target's logit
// where it lies there; loss_join_kernel joins a row's pieces.  The gradients
// take the vocabulary in pieces: the logits of a piece again, turned into dZ
// and rounded to 16 bits in the epilogue (the two products that follow read
// it as 16-bit operands), then dB's piece, then dA's sum over the pieces in
// fp32.  Bound by the matrix cores: 2 M N K operations forward and 6 M N K
// back, of which 2 M N K are the logits again; keeping them instead would take
// M N values of memory.
//
// Measured: 8192 tokens by 131072 words, 4096 deep, bf16, by card: 6.1-6.3 ms
// forward (1.39-1.44 PFLOP/s; the library's plain product of 8192^3 runs at
// 1.39-1.61), 19.1-19.7 ms back in four pieces: logits 1.62-1.66 ms a piece, dB
// 1.63-1.68, dA 1.51-1.54 (1.33-1.36, 1.31-1.35 and 1.43-1.46 PFLOP/s).  24
// tokens: 181-183 us (5.9 TB/s of the weights).
#pragma once

#include "linear_shapes.hpp"

namespace dft {

constexpr float kLog2e = 1.4426950408889634f;

// A row's target as a column of the vocabulary, -1 where it lies outside (and
// where no targets are given).
struct Targets {
    const void* at;
    int32_t wide;  // 64-bit numbers
    __device__ int column(int64_t row, int64_t cols) const {
        if (!at) return -1;
        const int64_t t = wide ? static_cast<const int64_t*>(at)[row] : static_cast<const int32_t*>(at)[row];
        return t >= 0 && t < cols ? (int)t : -1;
    }
};

// ---- forward ----------------------------------------------------------------------------
// What a wave found in its columns of one row.
struct RowPiece {
    float most, sum;  // the largest logit, and the sum of exp(logit - most)
};
// exp(z - most); -infinity has nothing of any sum, also where all are.
__device__ inline float exp_below(float z, float most) {
    return __builtin_amdgcn_exp2f((z - (most == -__builtin_inff() ? 0.0f : most)) * kLog2e);
}
__device__ inline RowPiece join(const RowPiece& a, const RowPiece& b) {
    // (a NaN of either stays: it is in the sums)
    const float most = fmaxf(a.most, b.most);
    return RowPiece{most, a.sum * exp_below(a.most, most) + b.sum * exp_below(b.most, most)};
}

// One value of the four lanes l % 16, 16 + l % 16, ... that hold a row's
// columns, the same in all of them: a swap puts the odd rows of 16 (then the
// upper half) of one copy into the even rows (the lower half) of the other.
template <class Op>
__device__ inline float over_columns(float x, Op op) {
    const uint32_t bits = __builtin_bit_cast(uint32_t, x);
    const auto rows = __builtin_amdgcn_permlane16_swap(bits, bits, false, false);
    // (into variables first: a bit cast of a vector's element takes the vector's first)
    const uint32_t even = rows[0], odd = rows[1];
    const uint32_t two = __builtin_bit_cast(uint32_t, op(__builtin_bit_cast(float, even), __builtin_bit_cast(float, odd)));
    const auto halves = __builtin_amdgcn_permlane32_swap(two, two, false, false);
    const uint32_t low = halves[0], high = halves[1];
    return op(__builtin_bit_cast(float, low), __builtin_bit_cast(float, high));
}

struct LossRowsProblem : LinearProblem {
    static constexpr int EPILOGUE = kEpilogueRows;
    static constexpr bool SHORT = true;  // may take kTileShort
    Targets targets;
    int64_t first, words;  // the piece's first column, and columns in all
    RowPiece* pieces;      // a wave's columns of row r, slot s: pieces[r * row_step + s * slot_step]
    int64_t row_step, slot_step;
    float* at_target;      // the target's logit of each row that has one

    // Block i of a wave's results: row lane % 16, columns 16 j + 4 (lane / 16) + v.  Nothing overlaps this arithmetic
    // (65536 logits a tile: a subtraction, a product, an exp2 and an addition of each), so what is rare stands in
    // branches: masks in tiles at the vocabulary's end, the search for a target where a row has one here.
    template <int MI, int NI>
    __device__ void rows_epilogue(floatx4 (&z)[MI][NI], int64_t row0, int64_t row_end, int64_t col0, int width,
                                  int lane) const {
        const int64_t slot = (first + col0) / width;
        const int left = C - col0 >= 16 * NI ? 16 * NI : C > col0 ? (int)(C - col0) : 0;  // columns inside
        const int c = 4 * (lane / 16);
        int goal[MI];  // the row's target within the wave's columns, if 0 to left - 1
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const int64_t row = row0 + 16 * i + lane % 16;
            const int target = row < row_end ? targets.column(row, words) : -1;
            const int64_t at = target - first - col0;
            goal[i] = target >= 0 && at >= 0 && at < left ? (int)at : -1;
        }
        if (left < 16 * NI) {
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = 0; j < NI; ++j)
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        if (16 * j + c + v >= left) z[i][j][v] = -__builtin_inff();
        }
        // (all blocks' maxima, then all sums: each step has MI independent chains to overlap)
        float most[MI], sum[MI];
        bool any = false;
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            most[i] = z[i][0][0];
#pragma unroll
            for (int j = 0; j < NI; ++j)
#pragma unroll
                for (int v = 0; v < 4; ++v) most[i] = fmaxf(most[i], z[i][j][v]);
            any = any || goal[i] >= 0;
        }
#pragma unroll
        for (int i = 0; i < MI; ++i) most[i] = over_columns(most[i], [](float x, float y) { return fmaxf(x, y); });
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const float from = most[i] == -__builtin_inff() ? 0.0f : most[i];
            float part[4] = {};
#pragma unroll
            for (int j = 0; j < NI; ++j)
#pragma unroll
                for (int v = 0; v < 4; ++v) part[v] += __builtin_amdgcn_exp2f((z[i][j][v] - from) * kLog2e);
            sum[i] = (part[0] + part[1]) + (part[2] + part[3]);
        }
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            sum[i] = over_columns(sum[i], [](float x, float y) { return x + y; });
            const int64_t row = row0 + 16 * i + lane % 16;
            if (row < row_end && lane < 16) pieces[row * row_step + slot * slot_step] = RowPiece{most[i], sum[i]};
        }
        if (__ballot(any)) {
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = 0; j < NI; ++j)
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        if (goal[i] == 16 * j + c + v) at_target[row0 + 16 * i + lane % 16] = z[i][j][v];
        }
    }
};

// lse and loss of `rows` rows (a power of two up to 32) per workgroup: the
// row's slots in strides, each thread's joined in ascending order, then a
// wave's by halves and the waves' in ascending order.  loss = (most - target's logit) + log(sum): the
// difference of two logits and a logarithm of at least one, so that a small
// loss keeps its digits; lse itself is rounded once more.  25 us for 8192 rows
// of 2048 slots (134 MB).
constexpr int kLossJoinThreads = 1024;
__device__ inline void loss_join(const LossRowsProblem& p, int64_t slots, int rows, float* loss, float* lse) {
    __shared__ RowPiece shared[kLossJoinThreads / kWave][32];
    const int r = threadIdx.x & (rows - 1), first = threadIdx.x / rows, strides = kLossJoinThreads / rows;
    const int64_t row = (int64_t)blockIdx.x * rows + r;
    RowPiece all{-__builtin_inff(), 0.0f};
    if (row < p.R) {
        const RowPiece* from = p.pieces + row * p.row_step;
        int64_t s = first;
        for (; s + 3 * strides < slots; s += 4 * strides) {  // four reads under way at a time
            RowPiece four[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) four[k] = from[(s + k * strides) * p.slot_step];
#pragma unroll
            for (int k = 0; k < 4; ++k) all = join(all, four[k]);
        }
        for (; s < slots; s += strides) all = join(all, from[s * p.slot_step]);
    }
    for (int d = rows; d < kWave; d *= 2)
        all = join(all, RowPiece{__shfl_xor(all.most, d), __shfl_xor(all.sum, d)});
    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
    if (lane < rows) shared[wave][lane] = all;
    __syncthreads();
    if (wave == 0 && lane < rows && row < p.R) {
        for (int w = 1; w < kLossJoinThreads / kWave; ++w) all = join(all, shared[w][lane]);
        const float log_sum = logf(all.sum);
        lse[row] = all.most + log_sum;
        if (loss) loss[row] = p.targets.column(row, p.words) < 0 ? 0.0f : (all.most - p.at_target[row]) + log_sum;
    }
}

// ---- gradients ----------------------------------------------------------------------------
// What the gradient's kernels read of each row, and the scale that dZ is held
// at.  An entry of dZ can be as small as a probability times a token's share
// of the mean, 1e-6 times 1e-4, which fp16 does not hold (its least is 6e-8):
// dZ is multiplied by the factor that takes the largest |dloss| just below
// 2^14, and the two gradients' epilogues take it back (both in fp32, 2^-24
// each).  Not a power of two: the largest entries, the targets' of the heaviest
// tokens, weigh most in the results, and 16 bits round what lies just below a
// power of two by half as much as what lies just above (181 tokens of
// weights even between 0 and 1 / 181 = 1.41 * 2^-8: the targets' entries off by
// 1.7e-3 of their norm in bf16 with a power of two, 1.5e-3 so).
//
// In fp16 a token of far less weight would lose its row of dA all the same
// (256 tokens of 131072 words, one in eight 1e8 times as heavy as the others:
// the light ones' rows off by 16 % of their norm, 24 tokens at 1e6 by 1e-3).
// So each row is held at the factor times a power of two of its own, 2^j, that
// takes its |dloss| into [2^13, 2^14) or 2^16 times further up.  dA's rows are
// multiplied by 2^-j in the epilogue.  In dB's sum over the tokens 2^-j goes to
// the row of A, in a copy of its own, and that copy is lifted by one power of
// two, 2^lift, the largest that no row overflows with, 2^15 over the largest |A|
// or more: what fp16 does not hold of a lowered row is below 2^-24 of the largest
// |A|.  A larger 2^j would take digits of dB for those of dA; with 2^16 tokens of
// 1e-9 of the largest weight are as exact as those of 6e-5 are without.  bf16 has
// fp32's range: j = 0.
// It costs fp16 a pass over A and a launch: 1000 tokens x 32001 words x 1000 265
// us against 258, 24 x 4096 x 512 35 against 32.
struct LossRow {
    float lse, scale;  // scale: dloss times the factor and 2^j; without a target infinity and 0, which make zeros
    int32_t target;
    float shrink;      // 2^-j
};
struct LossBack {
    float factor, lift;  // one over each
};
constexpr float kLargestSlope = 16352.0f;  // 2^14 (1 - 2^-9)
constexpr int kMostShift = 16;             // of j
constexpr int kLossBeginThreads = 256, kLossBeginWaves = kLossBeginThreads / kWave;
constexpr int kMostLifts = kLossBeginThreads;
struct LossPrepare {
    int64_t rows, words;
    Targets targets;
    const float *lse, *dloss;
    LossRow* row;
    LossBack* back;
    const uint16_t* A;  // fp16's; nullptr: j = 0 and lift = 0
    int64_t lda, width;
    int32_t* lifts;     // the largest lift of each workgroup's rows
};
__device__ inline float power_of_two(int n) { return __builtin_bit_cast(float, (uint32_t)(127 + n) << 23); }
__device__ inline int exponent_of(float v) { return (int)(__builtin_bit_cast(uint32_t, v) >> 23 & 0xff) - 127; }
// The largest shift of a row whose largest entry is `slope`, from 0 to kMostShift (that for 0 and NaN).
__device__ inline int row_shift(float slope) {
    const int j = exponent_of(kLargestSlope / slope);
    return j < 0 ? 0 : j < kMostShift ? j : kMostShift;
}
// By the first `blocks` workgroups, each of which reads all of dloss; of fp16, a wave reads a row of A.
__device__ inline void loss_prepare(const LossPrepare& p, uint32_t blocks) {
    if (blockIdx.x >= blocks) return;
    __shared__ float most[kLossBeginWaves];
    __shared__ int least[kLossBeginWaves];
    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
    float m = 0.0f;
#pragma unroll 4
    for (int64_t r = threadIdx.x; r < p.rows; r += kLossBeginThreads)
        if (p.targets.column(r, p.words) >= 0) m = fmaxf(m, fabsf(p.dloss[r]));
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) m = fmaxf(m, __shfl_xor(m, d));
    if (lane == 0) most[wave] = m;
    __syncthreads();
    m = 0.0f;
#pragma unroll
    for (int w = 0; w < kLossBeginWaves; ++w) m = fmaxf(m, most[w]);
    float scale = 1.0f;  // (nothing to hold, or nothing that can be held: as it is)
    if (m > 0.0f && m < __builtin_inff()) scale = fminf(kLargestSlope / m, 0x1p126f);
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.back = LossBack{1.0f / scale, 1.0f};
    const LossRow none{__builtin_inff(), 0.0f, -1, 1.0f};
    if (!p.A) {
        for (int64_t r = (int64_t)blockIdx.x * kLossBeginThreads + threadIdx.x; r < p.rows;
             r += (int64_t)blocks * kLossBeginThreads) {
            const int target = p.targets.column(r, p.words);
            p.row[r] = target < 0 ? none : LossRow{p.lse[r], p.dloss[r] * scale, target, 1.0f};
        }
        return;
    }
    int lift = kMostShift;
    for (int64_t r = (int64_t)blockIdx.x * kLossBeginWaves + wave; r < p.rows; r += (int64_t)blocks * kLossBeginWaves) {
        const int target = p.targets.column(r, p.words);
        if (target < 0) {
            if (lane == 0) p.row[r] = none;
            continue;
        }
        int largest = 0;  // of the row's magnitudes, as bits
        for (int64_t col = lane * 8; col < p.width; col += kWave * 8) {
            const Row8 v = load8(p.A + r * p.lda + col, p.width - col);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int low = (int)(v.w[e] & 0x7fffu), high = (int)(v.w[e] >> 16 & 0x7fffu);
                largest = largest > low ? largest : low;
                largest = largest > high ? largest : high;
            }
        }
#pragma unroll
        for (int d = 1; d < kWave; d *= 2) {
            const int other = __shfl_xor(largest, d);
            largest = largest > other ? largest : other;
        }
        const float slope = p.dloss[r] * scale;
        const int j = row_shift(fabsf(slope));
        // (a row of zeros has room for any lift, and one with an infinity or NaN as much as its other values may need)
        const int top = largest < 0x7c00 ? exponent_of((float)__builtin_bit_cast(_Float16, (uint16_t)largest)) : 15;
        lift = lift < j + 15 - top ? lift : j + 15 - top;
        if (lane == 0) p.row[r] = LossRow{p.lse[r], slope * power_of_two(j), target, power_of_two(-j)};
    }
    if (lane == 0) least[wave] = lift;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
        for (int w = 1; w < kLossBeginWaves; ++w) lift = lift < least[w] ? lift : least[w];
        p.lifts[blockIdx.x] = lift;
    }
}
// The lift of all rows, by every thread of a workgroup.
__device__ inline int common_lift(const int32_t* lifts, int count) {
    __shared__ int least[kLossBeginWaves];
    int lift = (int)threadIdx.x < count ? lifts[threadIdx.x] : kMostShift;
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) {
        const int other = __shfl_xor(lift, d);
        lift = lift < other ? lift : other;
    }
    if (threadIdx.x % kWave == 0) least[threadIdx.x / kWave] = lift;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kLossBeginWaves; ++w) lift = lift < least[w] ? lift : least[w];
    return lift;
}

// A piece's dZ: ep.out has rows of whole 16 bytes, zeros past the piece.
//
// Rounded to 16 bits, an entry is off by up to 2^-8 (bf16).  Over many tokens
// that is random and as large as the result's own rounding; of one token it is
// the target's entry alone, and twice the result's error.  Up to
// kSplitTokens tokens dZ is therefore held in two parts, what was rounded off
// in as many rows again: dB's contraction over the tokens has two rows for
// each and still fits one tile of 64, and dA's rows are joined afterwards.
constexpr int kSplitTokens = 32;
struct LossSlopeProblem : LinearProblem {
    static constexpr int EPILOGUE = kEpilogueValues;
    static constexpr bool SHORT = true;
    const LossRow* row;
    int64_t first;  // the piece's first column
    int64_t rest;   // bytes from a value to what was rounded off it; 0: not kept
};
// A wave reads its rows' values once, a row or two per lane, and passes them
// on by lane: loads between the epilogue's stores would wait for them.
template <>
struct EpilogueRows<LossSlopeProblem> {
    LossRow held[2], now;
    int lane;
    __device__ void load(const LossSlopeProblem& p, int64_t row0, int64_t row_end, int rows, int lane_) {
        lane = lane_;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t r = row0 + h * kWave + lane;
            held[h] = LossRow{__builtin_inff(), 0.0f, -1, 1.0f};
            if (h * kWave + lane < rows && r < row_end) held[h] = p.row[r];
        }
    }
    // (m: uniform, a multiple of the rows that r counts, which divide a wave)
    __device__ void of_row(int m, int r) {
        const LossRow& from = m < kWave ? held[0] : held[1];
        const int l = (m + r) % kWave;
        now.lse = __shfl(from.lse, l);
        now.scale = __shfl(from.scale, l);
        now.target = __shfl(from.target, l);
    }
    template <int TYPE>
    __device__ void finish(const LossSlopeProblem& p, const EpilogueBase& base, const EpilogueLane& at, int64_t,
                           int64_t col, int64_t left, float (&z)[8]) const {
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] = __builtin_amdgcn_exp2f((z[e] - now.lse) * kLog2e);
        const int64_t goal = now.target - p.first - col;
        if (now.target >= 0 && goal >= 0 && goal < 8) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (goal == e) z[e] -= 1.0f;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] *= now.scale;
        if (left < 8) {  // what lies past the piece is read by the products
#pragma unroll
            for (int e = 0; e < 8; ++e) z[e] = e < left ? z[e] : 0.0f;
        }
        const Row8 high = Row8::narrow<TYPE>(z);
        store8(reinterpret_cast<uint16_t*>(base.out + at.out), high, 8);
        if (p.rest) {
            float h[8];
            high.widen<TYPE>(h);
#pragma unroll
            for (int e = 0; e < 8; ++e) z[e] -= h[e];
            store8(reinterpret_cast<uint16_t*>(base.out + at.out + p.rest), Row8::narrow<TYPE>(z), 8);
        }
    }
};

// A gradient's product.  dB's piece is whole: scaled back and stored.  dA's is
// added to the sums of the pieces before it (fp32), and scaled back where it
// is the last, by each row's own power of two (fp16) and by the factor.  (Of two types: what the second has beside the first would not
// fit the registers of the first's 256x256 kernel.)
struct LossWordsGradProblem : LinearProblem {
    static constexpr int EPILOGUE = kEpilogueValues;
    static constexpr bool SHORT = true;
    const LossBack* back;
};
struct LossTokensGradProblem : LinearProblem {
    static constexpr int EPILOGUE = kEpilogueValues;
    static constexpr bool SHORT = false;
    const float* before;  // or nullptr; rows before_ld apart
    int64_t before_ld;
    const LossBack* back;  // nullptr: another piece follows
    const LossRow* row;    // nullptr: no powers of the rows' own, or another piece follows
};
template <int TYPE>
__device__ inline void store_gradient(const LinearEpilogue& ep, const EpilogueBase& base, const EpilogueLane& at,
                                      int64_t left, const float (&z)[8]) {
    if (ep.out_f32)
        store8(reinterpret_cast<float*>(base.out + at.out), z, left);
    else
        store8(reinterpret_cast<uint16_t*>(base.out + at.out), Row8::narrow<TYPE>(z), left);
}
template <>
struct EpilogueRows<LossWordsGradProblem> {
    __device__ void load(const LossWordsGradProblem&, int64_t, int64_t, int, int) {}
    __device__ void load_one(const LossWordsGradProblem&, int64_t) {}
    __device__ void of_row(int, int) {}
    template <int TYPE>
    __device__ void finish(const LossWordsGradProblem& p, const EpilogueBase& base, const EpilogueLane& at, int64_t,
                           int64_t, int64_t left, float (&z)[8]) const {
        // (a product by a power of two first: of both factors it might lie below fp32's numbers)
        const LossBack back = *p.back;
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] = z[e] * back.lift * back.factor;
        store_gradient<TYPE>(p.ep, base, at, left, z);
    }
};
// (the rows' powers as LossSlopeProblem has its rows' values)
template <>
struct EpilogueRows<LossTokensGradProblem> {
    float held[2], now = 1.0f;
    bool rows;
    __device__ void load(const LossTokensGradProblem& p, int64_t row0, int64_t row_end, int count, int lane) {
        rows = p.row;
        if (!rows) return;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t r = row0 + h * kWave + lane;
            held[h] = h * kWave + lane < count && r < row_end ? p.row[r].shrink : 1.0f;
        }
    }
    __device__ void load_one(const LossTokensGradProblem& p, int64_t row) {
        if (p.row) now = p.row[row].shrink;
    }
    __device__ void of_row(int m, int r) {
        if (rows) now = __shfl(m < kWave ? held[0] : held[1], (m + r) % kWave);
    }
    template <int TYPE>
    __device__ void finish(const LossTokensGradProblem& p, const EpilogueBase& base, const EpilogueLane& at, int64_t row,
                           int64_t col, int64_t left, float (&z)[8]) const {
        if (p.before) {
            float add[8];
            load8(add, p.before + row * p.before_ld + col, left);
#pragma unroll
            for (int e = 0; e < 8; ++e) z[e] += add[e];
        }
        if (p.back) {
            const float back = p.back->factor;
#pragma unroll
            for (int e = 0; e < 8; ++e) z[e] = z[e] * now * back;
        }
        store_gradient<TYPE>(p.ep, base, at, left, z);
    }
};

// dA from the sums of its rows' two parts.
struct LossFold {
    int64_t rows, cols;
    const float* held;  // 2 rows x cols
    const LossBack* back;
    const LossRow* row;
    void* out;
    int64_t ldo;
    int32_t out_f32;
};
template <int TYPE>
__device__ inline void loss_fold(const LossFold& p) {
    const int64_t groups = (p.cols + 7) / 8, i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= p.rows * groups) return;
    const int64_t row = i / groups, col = i % groups * 8, left = p.cols - col;
    const float back = p.back->factor, shrink = p.row[row].shrink;
    float z[8], rest[8];
    load8(z, p.held + row * p.cols + col, left);
    load8(rest, p.held + (p.rows + row) * p.cols + col, left);
#pragma unroll
    for (int e = 0; e < 8; ++e) z[e] = (z[e] + rest[e]) * shrink * back;
    if (p.out_f32)
        store8(static_cast<float*>(p.out) + row * p.ldo + col, z, left);
    else
        store8(static_cast<uint16_t*>(p.out) + row * p.ldo + col, Row8::narrow<TYPE>(z), left);
}

// Copies a matrix to rows of whole 16 bytes, zeros past their width; with
// targets, rows without one as zeros, so that nothing they hold reaches dB;
// with `row` (fp16), each row times its 2^-j and the lift of all.
struct LossPack {
    const uint16_t* src;
    int64_t rows, cols, ld;
    uint16_t* dst;
    int64_t ldd;
    int32_t copies;   // one below the other, two at most
    Targets targets;  // at == nullptr: every row
    int64_t words;
    const LossRow* row;
    const int32_t* lifts;
    int32_t count;  // of lifts
    LossBack* back;
};
// EACH accesses of a thread, under way together: 513 rows of 32001 odd columns
// and 1000 of 513 take 12 us with four against 15 with one (8: 13); up to
// kBeginBlocks workgroups, which the card holds at once, one (40 rows of 4096:
// the call 2 us longer with four).
constexpr int kPackGroups = 4;
constexpr int64_t kBeginBlocks = 2048;
template <int EACH>
__device__ inline void loss_pack(const LossPack& j) {
    const int64_t groups = j.ldd / 8, total = j.copies * j.rows * groups;
    const int64_t span = (int64_t)kLossBeginThreads * EACH;  // a workgroup's
    float lifted = 1.0f;
    if (j.row) {
        const int lift = common_lift(j.lifts, j.count);
        lifted = power_of_two(lift);
        if (blockIdx.x == 0 && threadIdx.x == 0) j.back->lift = power_of_two(-lift);
    }
    for (int64_t i0 = blockIdx.x * span + threadIdx.x; i0 < total; i0 += gridDim.x * span) {
        Row8 v[EACH];
#pragma unroll
        for (int k = 0; k < EACH; ++k) {
            const int64_t i = i0 + k * kLossBeginThreads;
            v[k] = Row8{};
            if (i >= total) continue;
            // (64-bit divisions would take longer than the bytes)
            const int64_t to = total <= 0x7fffffff ? (int64_t)((uint32_t)i / (uint32_t)groups) : i / groups;
            const int64_t col = (i - to * groups) * 8, row = to < j.rows ? to : to - j.rows;
            v[k] = load8(j.src + row * j.ld + col, j.cols - col);  // (on its way together with the target)
            if (j.targets.at && j.targets.column(row, j.words) < 0) v[k] = Row8{};
            if (j.row) {
                const float by = j.row[row].shrink * lifted;
                float x[8];
                v[k].template widen<kInputF16>(x);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] *= by;
                v[k] = Row8::narrow<kInputF16>(x);
            }
        }
#pragma unroll
        for (int k = 0; k < EACH; ++k) {  // (rows of dst lie one after the other)
            const int64_t i = i0 + k * kLossBeginThreads;
            if (i < total) *reinterpret_cast<u32x4*>(j.dst + i * 8) = v[k].w;
        }
    }
}

// What comes before the products, in one launch (the copy of A for dB in fp16,
// which needs the rows' values, in another): the rows' values, in the
// first row of workgroups so that they do not begin when the copies end, and
// copies.
struct LossBegin {
    LossPack pack[2];
    int32_t packs, each;
    uint32_t prepare_blocks;
    LossPrepare prepare;
};

// One more tile for short contractions: 128x128 with one place of LDS, which
// is copied into when it has been multiplied.  Its operands take 32 KiB, so
// four workgroups fit a CU in place of two, and one's copies, beginning and
// epilogue pass while the others multiply.  Forward against the best of the
// other tiles: 1094 tokens by 75472 words, 224 deep, 69 against 90 us, 5680 by
// 40672, 480 deep, 250 against 283, but 473 by 25184, 728 deep, 36 against 33
// and 7198 by 66880, 1512 deep, 1418 against 1250; never more than 128x128 with
// two places where there are two tiles or more for every CU.  dB of 24 tokens
// by 32768 words, 4096 wide, 58 against 88 us, both gradients of 512 tokens by
// 50000 words, 1024 wide, 209 against 229.
constexpr LinearTile kTileShort = (LinearTile)kTileCount;
using ShortShape = LinearShape<128, 128, 64, 64, 1, 4>;
constexpr TileSize loss_tile_size(LinearTile tile) {
    return tile == kTileShort ? TileSize{ShortShape::BM, ShortShape::BN} : kTileSizes[tile];
}

// ---- launches, one translation unit per type ------------------------------------------------
// `kmajor`: B's words are rows (b_transposed).
#define DFT_LOSS_LAUNCHES(TYPE)                                                                                       \
    hipError_t launch_loss_##TYPE(const LossRowsProblem&, bool kmajor, LinearTile, uint32_t, uint32_t, uint32_t, int, \
                                  hipStream_t);                                                                       \
    hipError_t launch_loss_##TYPE(const LossSlopeProblem&, bool kmajor, LinearTile, uint32_t, uint32_t, uint32_t, int, \
                                  hipStream_t);                                                                       \
    hipError_t launch_loss_##TYPE(const LossWordsGradProblem&, bool kmajor, LinearTile, uint32_t, uint32_t, uint32_t,  \
                                  int, hipStream_t);                                                                  \
    hipError_t launch_loss_##TYPE(const LossTokensGradProblem&, bool kmajor, LinearTile, uint32_t, uint32_t, uint32_t, \
                                  int, hipStream_t);
DFT_LOSS_LAUNCHES(bf16)
DFT_LOSS_LAUNCHES(f16)
#undef DFT_LOSS_LAUNCHES

}  // namespace dft
