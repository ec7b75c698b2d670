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

struct LossRowsProblem : LinearProblem {
    static constexpr int EPILOGUE = kEpilogueRows;
    Targets targets;
    int64_t first, words;  // the piece's first column, and columns in all
    RowPiece* pieces;      // a wave's columns of row r, slot s at pieces + s * R + r: rows of a slot lie together
    float* at_target;      // the target's logit of each row that has one

    // Block i of a wave's results: row lane % 16, columns 16 j + 4 (lane / 16) + v.
    template <int MI, int NI>
    __device__ void rows_epilogue(floatx4 (&z)[MI][NI], int64_t row0, int64_t row_end, int64_t col0, int width,
                                  int lane) const {
        const int64_t slot = (first + col0) / width;
        const int left = C - col0 >= 16 * NI ? 16 * NI : C > col0 ? (int)(C - col0) : 0;  // columns inside
        const int c = 4 * (lane / 16);
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const int64_t row = row0 + 16 * i + lane % 16;
            const bool inside = row < row_end;
            const int target = inside ? targets.column(row, words) : -1;
            const int goal = target < 0 ? -1 : (int)(target - first - col0);  // within the wave's columns, if 0 to left - 1
            if (left < 16 * NI) {
#pragma unroll
                for (int j = 0; j < NI; ++j)
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        if (16 * j + c + v >= left) z[i][j][v] = -__builtin_inff();
            }
            RowPiece p{z[i][0][0], 0.0f};
#pragma unroll
            for (int j = 0; j < NI; ++j)
#pragma unroll
                for (int v = 0; v < 4; ++v) p.most = fmaxf(p.most, z[i][j][v]);
            p.most = fmaxf(p.most, __shfl_xor(p.most, 16));
            p.most = fmaxf(p.most, __shfl_xor(p.most, 32));
            float hit = 0.0f;
            bool found = false;
#pragma unroll
            for (int j = 0; j < NI; ++j)
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    p.sum += exp_below(z[i][j][v], p.most);
                    if (goal == 16 * j + c + v) {
                        hit = z[i][j][v];
                        found = true;
                    }
                }
            p.sum += __shfl_xor(p.sum, 16);
            p.sum += __shfl_xor(p.sum, 32);
            if (inside && lane < 16) pieces[slot * R + row] = p;
            if (found && goal < left) at_target[row] = hit;
        }
    }
};

// lse and loss of `rows` rows (a power of two up to 32) per workgroup: the
// row's slots in strides, each thread's joined in ascending order, the
// threads' by halves.  loss = (most - target's logit) + log(sum): the
// difference of two logits and a logarithm of at least one, so that a small
// loss keeps its digits; lse itself is rounded once more.
constexpr int kLossJoinThreads = 1024;
__device__ inline void loss_join(const LossRowsProblem& p, int64_t slots, int rows, float* loss, float* lse) {
    __shared__ RowPiece shared[kLossJoinThreads];
    const int r = threadIdx.x & (rows - 1), first = threadIdx.x / rows, strides = kLossJoinThreads / rows;
    const int64_t row = (int64_t)blockIdx.x * rows + r;
    RowPiece all{-__builtin_inff(), 0.0f};
    if (row < p.R) {
        const RowPiece* from = p.pieces + row;
        int64_t s = first;
        for (; s + 3 * strides < slots; s += 4 * strides) {  // four reads under way at a time
            RowPiece four[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) four[k] = from[(s + k * strides) * p.R];
#pragma unroll
            for (int k = 0; k < 4; ++k) all = join(all, four[k]);
        }
        for (; s < slots; s += strides) all = join(all, from[s * p.R]);
    }
    for (int half = strides / 2; half > 0; half /= 2) {
        shared[threadIdx.x] = all;
        __syncthreads();
        if (first < half) all = join(all, shared[threadIdx.x + half * rows]);
        __syncthreads();
    }
    if (first == 0 && row < p.R) {
        const float log_sum = logf(all.sum);
        lse[row] = all.most + log_sum;
        if (loss) loss[row] = p.targets.column(row, p.words) < 0 ? 0.0f : (all.most - p.at_target[row]) + log_sum;
    }
}

// ---- gradients ----------------------------------------------------------------------------
// What the gradient's kernels read of each row, and the scale that dZ is held
// at.  An entry of dZ can be as small as a probability times a token's share
// of the mean, 1e-6 times 1e-4, which fp16 does not hold (its least is 6e-8):
// dZ is multiplied by the power of two that takes the largest |dloss| to
// [2^13, 2^14), an exact step that the two gradients' epilogues take back.
struct LossRow {
    float lse, scale;  // scale: dloss times the power of two; 0 without a target
    int32_t target, pad;
};
struct LossPrepare {
    int64_t rows, words;
    Targets targets;
    const float *lse, *dloss;
    LossRow* row;
    float* back;  // one over the power of two
};
constexpr int kLossPrepareThreads = 1024;
__device__ inline void loss_prepare(const LossPrepare& p) {
    __shared__ float most[kLossPrepareThreads / kWave];
    float m = 0.0f;
    for (int64_t r = threadIdx.x; r < p.rows; r += kLossPrepareThreads)
        if (p.targets.column(r, p.words) >= 0) m = fmaxf(m, fabsf(p.dloss[r]));
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) m = fmaxf(m, __shfl_xor(m, d));
    if (threadIdx.x % kWave == 0) most[threadIdx.x / kWave] = m;
    __syncthreads();
    m = 0.0f;
#pragma unroll
    for (int w = 0; w < kLossPrepareThreads / kWave; ++w) m = fmaxf(m, most[w]);
    int up = 0;  // (nothing to hold, or nothing that can be held: as it is)
    if (m > 0.0f && m < __builtin_inff()) {
        int exponent;
        frexpf(m, &exponent);
        up = 14 - exponent;
        up = up > 126 ? 126 : up < -126 ? -126 : up;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.back = ldexpf(1.0f, -up);
    const float scale = ldexpf(1.0f, up);
    for (int64_t r = (int64_t)blockIdx.x * kLossPrepareThreads + threadIdx.x; r < p.rows;
         r += (int64_t)gridDim.x * kLossPrepareThreads) {
        const int target = p.targets.column(r, p.words);
        p.row[r] = LossRow{p.lse[r], target < 0 ? 0.0f : p.dloss[r] * scale, target, 0};
    }
}

// A piece's dZ: ep.out has rows of whole 16 bytes, zeros past the piece.
struct LossSlopeProblem : LinearProblem {
    static constexpr int EPILOGUE = kEpilogueValues;
    const LossRow* row;
    int64_t first;  // the piece's first column
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
            held[h] = LossRow{0.0f, 0.0f, -1, 0};
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
        const int64_t goal = now.target - p.first - col;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float d = __builtin_amdgcn_exp2f((z[e] - now.lse) * kLog2e) - (goal == e ? 1.0f : 0.0f);
            // (a row without target adds nothing, whatever its logits; what lies past the piece is read by the products)
            z[e] = now.target >= 0 && e < left ? d * now.scale : 0.0f;
        }
        store8(reinterpret_cast<uint16_t*>(base.out + at.out), Row8::narrow<TYPE>(z), 8);
    }
};

// A gradient's product.  dB's piece is whole: scaled back and stored.  dA's is
// added to the sums of the pieces before it (fp32), and scaled back where it
// is the last.  (Of two types: what the second has beside the first would not
// fit the registers of the first's 256x256 kernel.)
struct LossWordsGradProblem : LinearProblem {
    static constexpr int EPILOGUE = kEpilogueValues;
    const float* back;
};
struct LossTokensGradProblem : LinearProblem {
    static constexpr int EPILOGUE = kEpilogueValues;
    const float* before;  // or nullptr; rows before_ld apart
    int64_t before_ld;
    const float* back;    // nullptr: another piece follows
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
    __device__ void of_row(int, int) {}
    template <int TYPE>
    __device__ void finish(const LossWordsGradProblem& p, const EpilogueBase& base, const EpilogueLane& at, int64_t,
                           int64_t, int64_t left, float (&z)[8]) const {
        const float back = *p.back;
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] *= back;
        store_gradient<TYPE>(p.ep, base, at, left, z);
    }
};
template <>
struct EpilogueRows<LossTokensGradProblem> {
    __device__ void load(const LossTokensGradProblem&, int64_t, int64_t, int, int) {}
    __device__ void of_row(int, int) {}
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
            const float back = *p.back;
#pragma unroll
            for (int e = 0; e < 8; ++e) z[e] *= back;
        }
        store_gradient<TYPE>(p.ep, base, at, left, z);
    }
};

// Copies a matrix to rows of whole 16 bytes, zeros past their width; with
// `row`, rows without a target as zeros, so that nothing they hold reaches dB.
struct LossPack {
    const uint16_t* src;
    int64_t rows, cols, ld;
    uint16_t* dst;
    int64_t ldd;
    Targets targets;  // at == nullptr: every row
    int64_t words;
};
__device__ inline void loss_pack(const LossPack& j) {
    const int64_t groups = j.ldd / 8, total = j.rows * groups;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t row = i / groups, col = i % groups * 8;
        Row8 v{};
        if (!j.targets.at || j.targets.column(row, j.words) >= 0) v = load8(j.src + row * j.ld + col, j.cols - col);
        *reinterpret_cast<u32x4*>(j.dst + row * j.ldd + col) = v.w;
    }
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
