// norm_kernels.hpp -- gfx950 kernels of the layer norm with the residual
// stream's addition and the dropout before it, of their gradients, and of
// dropout alone.
//
//   total = dropout(x) + residual          rounded to the type: the stream that the next block adds to
//   mean, rstd = of each row of total, rstd = (mean of (total - mean)^2 + eps)^-1/2
//   y = (total - mean) rstd weight + bias
//
//   u = (total - mean) rstd,  g = dy weight
//   dtotal = rstd (g - mean(g) - u mean(g u)) + dstream,   dx = dropout of dtotal with the same mask
//   dweight = sum over the rows of dy u,  dbias = sum over the rows of dy
//
// All are bound by bytes: each row is read once, kept in registers between
// its sums and its results, and written once.  Statistics and sums are fp32;
// the variance is the mean of squared deviations from the mean, taken in a
// second pass over the registers, so a mean far from zero costs no digits.
// The gradient of weight and bias is summed in registers over the rows that a
// workgroup takes, and joined over the workgroups in a fixed order.
//
// Measured with the residual stream, bf16 (a copy of 1 GiB here runs at 5.1
// TB/s, which rows from several streams pass):
// 16384 x 4096 with dropout 97 us (5.5 TB/s of 537 MB), its gradients 132 us
// (5.1 TB/s of 671 MB) and 5 us for the join; 4096 x 16384 99 and 119 us without
// dropout; rows aligned to nothing, 16384 x 4095, 132 and 156 us.  fp32, 8192 x
// 8192: 192 us (5.6 TB/s), its gradients 206 (5.2).
#pragma once

#include "dropout.hpp"
#include "values8.hpp"

namespace dft {

struct NormProblem {
    int64_t rows, cols;
    float eps;
    Dropout dropout;
    const void* x;        // forward; the gradient's `total` is read at `total`
    int64_t ldx;
    const void* residual;  // or nullptr
    int64_t ldr;
    const void *weight, *bias;  // or nullptr
    void* total;           // forward: nullptr when total is x itself
    int64_t ldt;
    void* y;               // forward: written; gradient: dy, read
    int64_t ldy;
    float *mean, *rstd;
    // gradient
    const void* dstream;   // gradient that reaches total by another way, or nullptr
    int64_t lds;
    void* dtotal;          // or nullptr
    int64_t lddt;
    void* dx;              // or nullptr
    int64_t lddx;
    float* partial;        // places x 2 x cols: sums of dy u and of dy; nullptr: not wanted
    int32_t places;
    float *dweight, *dbias;
};

// A row is WAVES waves' work, CHUNKS chunks of eight per lane; waves that
// share no row stand in one workgroup of at least four.  SUMS_IN_LDS: where the
// gradient's kernel keeps the columns' sums, since the registers do not hold
// them beside a row and the next.
template <int WAVES_, int CHUNKS_, bool SUMS_IN_LDS_ = false>
struct NormShape {
    static constexpr int WAVES = WAVES_, CHUNKS = CHUNKS_, COLS = WAVES * kWave * 8 * CHUNKS;
    static constexpr bool SUMS_IN_LDS = SUMS_IN_LDS_;
    static constexpr int ROWS = WAVES >= 4 ? 1 : 4 / WAVES, THREADS = WAVES * ROWS * kWave;
    static constexpr int MIN_WAVES = 4;  // per SIMD: sixteen per CU
};

// Sums of N values over a row's waves, the same in every lane.  `at` alternates
// between the two halves of the array, so that one barrier does: a wave that
// writes a half again has passed the barrier after all reads of it.
template <int WAVES, int N>
__device__ inline void row_sums(float (&v)[N], float (*shared)[WAVES][N], int at) {
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] = wave_sum(v[n]);
    if constexpr (WAVES > 1) {
        const int wave = threadIdx.x / kWave;
        if (threadIdx.x % kWave == 0) {
#pragma unroll
            for (int n = 0; n < N; ++n) shared[at][wave][n] = v[n];
        }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < N; ++n) {
            v[n] = 0.0f;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) v[n] += shared[at][w][n];
        }
    }
}

// A row's statistics from the rounded mean `near` of a first pass, and the
// mean deviation from it and mean squared deviation of a second: what the
// first rounding left out (`shift`) moves mean, variance and deviations.
struct NormStatistics {
    float mean, shift, rstd;
};
// The rounded mean that deviations are taken from.  Of 16-bit values it is cut
// to 16 significant bits, so that values of up to 256 times its size have exact
// deviations: from a full mean those of one exponent are all rounded the same
// way, which put the mean off by up to two units (16 x 4096 bf16: 1.3e-7 of it
// in the 2-norm, 3e-8 so).  The variance loses nothing by the larger shift s:
// values on a grid of step g whose mean lies s from it have a variance of at
// least s (g - s), and g is 64 s or more.
template <int TYPE>
__device__ inline float near_mean(float mean) {
    if constexpr (TYPE == kValueF32) return mean;
    const uint32_t bits = __builtin_bit_cast(uint32_t, mean);
    return __builtin_bit_cast(float, (bits + 0x80u) & ~0xffu);
}
__device__ inline NormStatistics norm_statistics(float near, float shift, float square, float eps) {
    const float variance = square - shift * shift;
    return NormStatistics{near + shift, shift, 1.0f / sqrtf((variance < 0.0f ? 0.0f : variance) + eps)};
}

// One row at a time per Shape::WAVES waves, one workgroup per row or four: the
// rows of the launch, rather than loads ahead, keep the memory busy.
template <int TYPE, class Shape, bool WHOLE>
__global__ __launch_bounds__(Shape::THREADS, Shape::MIN_WAVES) void norm_kernel(NormProblem p) {
    using V = Values8<TYPE>;
    using E = typename V::element;
    constexpr int WAVES = Shape::WAVES, CHUNKS = Shape::CHUNKS;
    __shared__ float shared[2][WAVES][2];
    const int lane = threadIdx.x % (WAVES * kWave), cols = (int)p.cols, chunks = (cols + 7) / 8;
    const int part = __builtin_amdgcn_readfirstlane(threadIdx.x / (WAVES * kWave));
    const uint64_t offset = p.dropout.drop ? dropout_offset(p.dropout) : 0;
    const float n = (float)cols;
    auto column = [&](int c) { return (lane + c * WAVES * kWave) * 8; };
    for (int64_t first = (int64_t)blockIdx.x * Shape::ROWS; first < p.rows; first += (int64_t)gridDim.x * Shape::ROWS) {
        const int64_t row = first + part;
        if (WAVES < 4 && row >= p.rows) break;  // (whole waves: nothing is waited for together)
        V in[CHUNKS], add[CHUNKS], weight[CHUNKS], bias[CHUNKS];
        // (what is not given has values that change nothing: branches in the arithmetic would keep what they choose from
        // in registers, both chunks' at once)
        auto read = [&](V (&to)[CHUNKS], const void* from, int64_t ld, float instead) {
#pragma unroll
            for (int c = 0; c < CHUNKS; ++c) to[c] = all8<V>(instead);
            if (from) {
#pragma unroll
                for (int c = 0; c < CHUNKS; ++c)
                    to[c].template load_at<WHOLE>(static_cast<const E*>(from) + row * ld, column(c), cols);
            }
        };
        read(in, p.x, p.ldx, 0.0f);
        read(add, p.residual, p.ldr, 0.0f);
        read(weight, p.weight, 0, 1.0f);
        read(bias, p.bias, 0, 0.0f);
        float t[CHUNKS][8], sum[2] = {0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) {
            in[c].widen(t[c]);
            if (p.total) {
                if (p.dropout.drop) drop8(p.dropout, offset, (uint64_t)(row * chunks + column(c) / 8), t[c]);
                float r[8];
                add[c].widen(r);
#pragma unroll
                for (int e = 0; e < 8; ++e) t[c][e] += r[e];
                const V kept = V::narrow(t[c]);
                kept.template store_at<WHOLE>(static_cast<E*>(p.total) + row * p.ldt, column(c), cols);
                kept.widen(t[c]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[0] += t[c][e];  // (zeros past the row)
        }
        row_sums<WAVES, 2>(sum, shared, 0);
        const float near = near_mean<TYPE>(sum[0] / n);
        float off[2] = {0.0f, 0.0f};  // sums of the deviations and of their squares
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) {
            const int left = cols - column(c);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                t[c][e] -= near;
                const float d = (WHOLE ? left > 0 : e < left) ? t[c][e] : 0.0f;
                off[0] += d;
                off[1] += d * d;
            }
        }
        row_sums<WAVES, 2>(off, shared, 1);
        const NormStatistics s = norm_statistics(near, off[0] / n, off[1] / n, p.eps);
        if (lane == 0) {
            if (p.mean) p.mean[row] = s.mean;
            if (p.rstd) p.rstd[row] = s.rstd;
        }
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) {
            float w[8], b[8];
            weight[c].widen(w);
            bias[c].widen(b);
#pragma unroll
            for (int e = 0; e < 8; ++e) t[c][e] = (t[c][e] - s.shift) * s.rstd * w[e] + b[e];
            V::narrow(t[c]).template store_at<WHOLE>(static_cast<E*>(p.y) + row * p.ldy, column(c), cols);
        }
    }
}

// Rows too wide for the registers, and those of fewer than eight columns: the
// row is read three times, from the caches after the first.  4096 x 20000 bf16
// with the residual stream 216 us (3.0 TB/s of 655 MB); 2^20 x 4 12.4 ms, a
// workgroup a row.
constexpr int kWideThreads = 1024;
template <int TYPE>
__global__ __launch_bounds__(kWideThreads) void norm_wide_kernel(NormProblem p) {
    using V = Values8<TYPE>;
    using E = typename V::element;
    constexpr int WAVES = kWideThreads / kWave;
    __shared__ float shared[2][WAVES][2];
    const int64_t chunks = (p.cols + 7) / 8;
    const uint64_t offset = p.dropout.drop ? dropout_offset(p.dropout) : 0;
    const float n = (float)p.cols;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const E* x = static_cast<const E*>(p.x) + row * p.ldx;
        const E* residual = p.residual ? static_cast<const E*>(p.residual) + row * p.ldr : nullptr;
        E* total = p.total ? static_cast<E*>(p.total) + row * p.ldt : nullptr;
        float sum[2] = {0.0f, 0.0f}, off[2] = {0.0f, 0.0f}, t[8];
        V v;
        for (int64_t chunk = threadIdx.x; chunk < chunks; chunk += kWideThreads) {
            const int64_t left = p.cols - chunk * 8;
            v.load(x + chunk * 8, left);
            v.widen(t);
            if (p.total) {
                if (p.dropout.drop) drop8(p.dropout, offset, (uint64_t)(row * chunks + chunk), t);
                if (p.residual) {
                    float r[8];
                    v.load(residual + chunk * 8, left);
                    v.widen(r);
#pragma unroll
                    for (int e = 0; e < 8; ++e) t[e] += r[e];
                }
                v = V::narrow(t);
                v.store(total + chunk * 8, left);
                v.widen(t);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[0] += e < left ? t[e] : 0.0f;
        }
        row_sums<WAVES, 2>(sum, shared, 0);
        const float near = near_mean<TYPE>(sum[0] / n);
        const E* kept = p.total ? total : x;  // (each thread reads back what it wrote)
        for (int64_t chunk = threadIdx.x; chunk < chunks; chunk += kWideThreads) {
            const int64_t left = p.cols - chunk * 8;
            v.load(kept + chunk * 8, left);
            v.widen(t);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float d = e < left ? t[e] - near : 0.0f;
                off[0] += d;
                off[1] += d * d;
            }
        }
        row_sums<WAVES, 2>(off, shared, 1);
        const NormStatistics s = norm_statistics(near, off[0] / n, off[1] / n, p.eps);
        if (threadIdx.x == 0) {
            if (p.mean) p.mean[row] = s.mean;
            if (p.rstd) p.rstd[row] = s.rstd;
        }
        for (int64_t chunk = threadIdx.x; chunk < chunks; chunk += kWideThreads) {
            const int64_t left = p.cols - chunk * 8;
            float w[8];
            v.load(kept + chunk * 8, left);
            v.widen(t);
#pragma unroll
            for (int e = 0; e < 8; ++e) t[e] = (t[e] - near - s.shift) * s.rstd;
            if (p.weight) {
                v.load(static_cast<const E*>(p.weight) + chunk * 8, left);
                v.widen(w);
#pragma unroll
                for (int e = 0; e < 8; ++e) t[e] *= w[e];
            }
            if (p.bias) {
                v.load(static_cast<const E*>(p.bias) + chunk * 8, left);
                v.widen(w);
#pragma unroll
                for (int e = 0; e < 8; ++e) t[e] += w[e];
            }
            V::narrow(t).store(static_cast<E*>(p.y) + row * p.ldy + chunk * 8, left);
        }
    }
}

// ---- gradients ------------------------------------------------------------------------
// Eight columns of one row's results: dtotal and, through the mask, dx.
// `store(matrix's row, values)` stores them.
template <int TYPE, class Store>
__device__ inline void norm_grad_store(const NormProblem& p, uint64_t offset, int64_t row, int64_t chunk, float (&d)[8],
                                       Store store) {
    using V = Values8<TYPE>;
    using E = typename V::element;
    if (p.dtotal) store(static_cast<E*>(p.dtotal) + row * p.lddt, V::narrow(d));
    if (p.dx) {
        if (p.dropout.drop) drop8(p.dropout, offset, (uint64_t)(row * ((p.cols + 7) / 8) + chunk), d);
        store(static_cast<E*>(p.dx) + row * p.lddx, V::narrow(d));
    }
}

// A workgroup works through every gridDim.x-th row (sixteen waves per CU) and
// keeps the columns' sums of dy u and dy; 149 us in place of 132 for 16384 x
// 4096 without the next row's loads ahead.
template <int TYPE, class Shape, bool WHOLE>
__global__ __launch_bounds__(Shape::THREADS, Shape::MIN_WAVES) void norm_grad_kernel(NormProblem p) {
    using V = Values8<TYPE>;
    using E = typename V::element;
    constexpr int WAVES = Shape::WAVES, CHUNKS = Shape::CHUNKS;
    __shared__ float shared[2][WAVES][2];
    const int lane = threadIdx.x % (WAVES * kWave), cols = (int)p.cols;
    const int part = __builtin_amdgcn_readfirstlane(threadIdx.x / (WAVES * kWave));
    const uint64_t offset = p.dropout.drop ? dropout_offset(p.dropout) : 0;
    const float each = 1.0f / (float)cols;
    auto column = [&](int c) { return (lane + c * WAVES * kWave) * 8; };
    // (as in norm_kernel, what is not given has values that change nothing)
    V weight[CHUNKS];
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) weight[c] = all8<V>(1.0f);
    if (p.weight) {
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) weight[c].template load_at<WHOLE>(static_cast<const E*>(p.weight), column(c), cols);
    }
    // The columns' sums: a lane's own, in registers or in LDS, four values an access.
    constexpr bool IN_LDS = Shape::SUMS_IN_LDS;
    __shared__ floatx4 held[IN_LDS ? CHUNKS * 4 : 1][IN_LDS ? Shape::THREADS : 1];
    float dweight[CHUNKS][8] = {}, dbias[CHUNKS][8] = {};
    auto keep = [&](int c) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            held[4 * c + h][threadIdx.x] = floatx4{dweight[c][4 * h], dweight[c][4 * h + 1], dweight[c][4 * h + 2], dweight[c][4 * h + 3]};
            held[4 * c + 2 + h][threadIdx.x] = floatx4{dbias[c][4 * h], dbias[c][4 * h + 1], dbias[c][4 * h + 2], dbias[c][4 * h + 3]};
        }
    };
    auto fetch = [&](int c) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const floatx4 w = held[4 * c + h][threadIdx.x], b = held[4 * c + 2 + h][threadIdx.x];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                dweight[c][4 * h + e] = w[e];
                dbias[c][4 * h + e] = b[e];
            }
        }
    };
    if constexpr (IN_LDS) {
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) keep(c);
    }
    const int64_t step = (int64_t)gridDim.x * Shape::ROWS;
    int at = 0;
    struct RowReads {
        V dy[CHUNKS], total[CHUNKS], stream[CHUNKS];
        float mean, rstd;
    };
    auto read = [&](RowReads& r, int64_t row) {
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) {
            r.dy[c].template load_at<WHOLE>(static_cast<const E*>(p.y) + row * p.ldy, column(c), cols);
            r.total[c].template load_at<WHOLE>(static_cast<const E*>(p.total) + row * p.ldt, column(c), cols);
        }
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) r.stream[c] = all8<V>(0.0f);
        if (p.dstream) {
#pragma unroll
            for (int c = 0; c < CHUNKS; ++c)
                r.stream[c].template load_at<WHOLE>(static_cast<const E*>(p.dstream) + row * p.lds, column(c), cols);
        }
        r.mean = p.mean[row];
        r.rstd = p.rstd[row];
    };
    // The next row is read before this one's sums are joined, so that loads are under way throughout.  For the
    // registers' sake a row stays as it was read, and what the sums and the results need of it is computed twice.
    int64_t row = (int64_t)blockIdx.x * Shape::ROWS + part;
    RowReads next;
    if (row < p.rows) read(next, row);
    for (; row < p.rows; row += step) {
        RowReads now = next;
        if (row + step < p.rows) read(next, row + step);
        const float mean = now.mean, rstd = now.rstd;
        float sums[2] = {0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) {
            const int left = cols - column(c);
            float g[8], u[8], w[8];
            now.dy[c].widen(g);
            now.total[c].widen(u);
            weight[c].afresh();
            weight[c].widen(w);
            if constexpr (IN_LDS) fetch(c);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                // (past the row dy is zero, and u finite)
                u[e] = (WHOLE ? left > 0 : e < left) ? (u[e] - mean) * rstd : 0.0f;
                dweight[c][e] += g[e] * u[e];
                dbias[c][e] += g[e];
                g[e] *= w[e];
                sums[0] += g[e];
                sums[1] += g[e] * u[e];
            }
            if constexpr (IN_LDS) keep(c);
        }
        row_sums<WAVES, 2>(sums, shared, at);
        at ^= 1;
        const float m = sums[0] * each, mu = sums[1] * each;
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) {
            float g[8], u[8], w[8], add[8];
            now.dy[c].afresh();
            now.total[c].afresh();
            weight[c].afresh();
            now.dy[c].widen(g);
            now.total[c].widen(u);
            weight[c].widen(w);
            now.stream[c].widen(add);
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] = (g[e] * w[e] - m - (u[e] - mean) * rstd * mu) * rstd + add[e];
            if (column(c) < cols)
                norm_grad_store<TYPE>(p, offset, row, column(c) / 8, g,
                                      [&](E* to, const V& v) { v.template store_at<WHOLE>(to, column(c), cols); });
        }
    }
    if (!p.partial) return;
    // Rows that different waves of the workgroup took are added in the waves' order.
    if constexpr (Shape::ROWS > 1) {
        __shared__ float sums[Shape::ROWS][2][Shape::COLS];
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                sums[part][0][column(c) + e] = dweight[c][e];
                sums[part][1][column(c) + e] = dbias[c][e];
            }
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * Shape::COLS; i += Shape::THREADS) {
            const int which = i / Shape::COLS, col = i % Shape::COLS;
            float v = 0.0f;
#pragma unroll
            for (int r = 0; r < Shape::ROWS; ++r) v += sums[r][which][col];
            if (col < cols) p.partial[((int64_t)which * p.places + blockIdx.x) * p.cols + col] = v;
        }
    } else {
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) {
            const int left = cols - column(c);
            float* to = p.partial + (int64_t)blockIdx.x * p.cols;
            if constexpr (IN_LDS) fetch(c);
            if (left > 0) {
                store8(to + column(c), dweight[c], WHOLE ? 8 : left);
                store8(to + (int64_t)p.places * p.cols + column(c), dbias[c], WHOLE ? 8 : left);
            }
        }
    }
}

// dweight and dbias over the workgroups' sums: 32 columns by 32 strides of
// places per workgroup.  A stride's places are added in eight chains, the
// chains and the strides by halves: fp32 sums of a thousand places are off by
// two thirds of those added one after the other (1000 x 513: 1.5e-7 -> 9e-8
// in the 2-norm).  512 places of 4096 columns 5 us (16 columns by 64 strides
// 7.5: lines half used).
constexpr int kNormJoinCols = 32, kNormJoinStrides = 32;
template <int N>
__device__ inline float sum_by_halves(float (&v)[N]) {
#pragma unroll
    for (int half = N / 2; half > 0; half /= 2)
#pragma unroll
        for (int i = 0; i < half; ++i) v[i] += v[i + half];
    return v[0];
}
__global__ __launch_bounds__(kNormJoinCols * kNormJoinStrides) void norm_join_kernel(NormProblem p) {
    __shared__ float sums[kNormJoinStrides][kNormJoinCols + 1];
    const int c = threadIdx.x % kNormJoinCols, r = threadIdx.x / kNormJoinCols;
    const int64_t col = (int64_t)blockIdx.x * kNormJoinCols + c;
    float* const out = blockIdx.y == 0 ? p.dweight : p.dbias;
    if (!out) return;
    constexpr int CHAINS = 8, STEP = CHAINS * kNormJoinStrides;
    float sum[CHAINS] = {};
    if (col < p.cols) {
        const float* from = p.partial + (int64_t)blockIdx.y * p.places * p.cols + col;
        int k = r;
        for (; k + STEP - kNormJoinStrides < p.places; k += STEP) {
#pragma unroll
            for (int i = 0; i < CHAINS; ++i) sum[i] += from[(k + i * kNormJoinStrides) * p.cols];
        }
        float rest[CHAINS];  // (read from a place that exists, so that all are under way together)
#pragma unroll
        for (int i = 0; i < CHAINS; ++i) {
            const int place = k + i * kNormJoinStrides;
            rest[i] = k < p.places ? from[(place < p.places ? place : k) * p.cols] : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < CHAINS; ++i)
            if (k + i * kNormJoinStrides < p.places) sum[i] += rest[i];
    }
    sums[r][c] = sum_by_halves(sum);
    __syncthreads();
    if (r == 0 && col < p.cols) {
        float v[kNormJoinStrides];
#pragma unroll
        for (int k = 0; k < kNormJoinStrides; ++k) v[k] = sums[k][c];
        out[col] = sum_by_halves(v);
    }
}

// Rows too wide for the registers (or of fewer than eight columns): the row's
// sums and results in two passes, and the columns' sums in a kernel of their
// own.  2048 x 16384 fp32 with the stream's gradient 124 + 53 us and 8 for the join
// (537 MB would take 105), 4096 x 20000 bf16 185 + 73 + 9.
template <int TYPE>
__global__ __launch_bounds__(kWideThreads) void norm_grad_wide_kernel(NormProblem p) {
    using V = Values8<TYPE>;
    using E = typename V::element;
    constexpr int WAVES = kWideThreads / kWave;
    __shared__ float shared[2][WAVES][2];
    const int64_t chunks = (p.cols + 7) / 8;
    const uint64_t offset = p.dropout.drop ? dropout_offset(p.dropout) : 0;
    const float each = 1.0f / (float)p.cols;
    int at = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const float mean = p.mean[row], rstd = p.rstd[row];
        float sums[2] = {0.0f, 0.0f}, g[8], u[8];
        auto read = [&](int64_t chunk, int64_t left) {
            V v;
            v.load(static_cast<const E*>(p.y) + row * p.ldy + chunk * 8, left);
            v.widen(g);
            v.load(static_cast<const E*>(p.total) + row * p.ldt + chunk * 8, left);
            v.widen(u);
#pragma unroll
            for (int e = 0; e < 8; ++e) u[e] = e < left ? (u[e] - mean) * rstd : 0.0f;
            if (p.weight) {
                float w[8];
                v.load(static_cast<const E*>(p.weight) + chunk * 8, left);
                v.widen(w);
#pragma unroll
                for (int e = 0; e < 8; ++e) g[e] *= w[e];
            }
        };
        for (int64_t chunk = threadIdx.x; chunk < chunks; chunk += kWideThreads) {
            read(chunk, p.cols - chunk * 8);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                sums[0] += g[e];
                sums[1] += g[e] * u[e];
            }
        }
        row_sums<WAVES, 2>(sums, shared, at);
        at ^= 1;
        const float m = sums[0] * each, mu = sums[1] * each;
        for (int64_t chunk = threadIdx.x; chunk < chunks; chunk += kWideThreads) {
            const int64_t left = p.cols - chunk * 8;
            read(chunk, left);
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] = (g[e] - m - u[e] * mu) * rstd;
            if (p.dstream) {
                V v;
                float add[8];
                v.load(static_cast<const E*>(p.dstream) + row * p.lds + chunk * 8, left);
                v.widen(add);
#pragma unroll
                for (int e = 0; e < 8; ++e) g[e] += add[e];
            }
            norm_grad_store<TYPE>(p, offset, row, chunk, g, [&](E* to, const V& v) { v.store(to + chunk * 8, left); });
        }
    }
}

// Sums of dy u and of dy over every places-th row, 2048 columns per workgroup.
template <int TYPE>
__global__ __launch_bounds__(256) void norm_columns_kernel(NormProblem p) {
    using V = Values8<TYPE>;
    using E = typename V::element;
    const int64_t chunk = (int64_t)blockIdx.y * 256 + threadIdx.x, left = p.cols - chunk * 8;
    if (left <= 0) return;
    float dweight[8] = {}, dbias[8] = {};
#pragma unroll 2
    for (int64_t row = blockIdx.x; row < p.rows; row += p.places) {
        const float mean = p.mean[row], rstd = p.rstd[row];
        V v;
        float d[8], u[8];
        v.load(static_cast<const E*>(p.y) + row * p.ldy + chunk * 8, left);
        v.widen(d);
        v.load(static_cast<const E*>(p.total) + row * p.ldt + chunk * 8, left);
        v.widen(u);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            dweight[e] += d[e] * ((u[e] - mean) * rstd);
            dbias[e] += d[e];
        }
    }
    float* to = p.partial + (int64_t)blockIdx.x * p.cols + chunk * 8;
    store8(to, dweight, left);
    store8(to + (int64_t)p.places * p.cols, dbias, left);
}

// ---- dropout alone ---------------------------------------------------------------------
struct DropoutProblem {
    int64_t rows, cols;
    Dropout dropout;
    const void* x;
    int64_t ldx;
    const void* residual;  // or nullptr
    int64_t ldr;
    void* y;
    int64_t ldy;
};

// A thread takes a chunk of eight, or every stride-th where a launch does not
// hold them all.  Rows that lie without gaps in whole chunks come as one row:
// their chunks count on from row to row.  8192 x 16384 bf16 96-100 us (5.4-5.6
// TB/s of 537 MB): the generator's ten rounds stay under the bytes.
template <int TYPE, bool WHOLE>
__global__ __launch_bounds__(256) void dropout_kernel(DropoutProblem p) {
    using V = Values8<TYPE>;
    using E = typename V::element;
    const int64_t chunks = (p.cols + 7) / 8, total = p.rows * chunks, stride = (int64_t)gridDim.x * 256;
    const uint64_t offset = p.dropout.drop ? dropout_offset(p.dropout) : 0;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += stride) {
        // (64-bit divisions would take as long as the generator)
        const int64_t row = p.rows == 1 ? 0 : total <= 0xffffffff ? (int64_t)((uint32_t)i / (uint32_t)chunks) : i / chunks;
        const int64_t chunk = i - row * chunks, left = p.cols - chunk * 8;
        V in, add;
        const int64_t inside = WHOLE ? 8 : left;
        in.load(static_cast<const E*>(p.x) + row * p.ldx + chunk * 8, inside);
        if (p.residual) add.load(static_cast<const E*>(p.residual) + row * p.ldr + chunk * 8, inside);
        float v[8];
        in.widen(v);
        if (p.dropout.drop) drop8(p.dropout, offset, (uint64_t)i, v);
        if (p.residual) {
            float r[8];
            add.widen(r);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += r[e];
        }
        V::narrow(v).store(static_cast<E*>(p.y) + row * p.ldy + chunk * 8, inside);
    }
}

}  // namespace dft
