// norm_api.hip -- the C ABI of the layer norm, its gradients and dropout
// (include/dense_fp32_tiled.h): argument checks, the choice of shape, and the
// launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <stdint.h>

#include "dense_fp32_tiled.h"
#include "host_checks.hpp"
#include "norm_kernels.hpp"

namespace {

using namespace dft;

bool known_value(int t) { return t == GEMM_VALUE_BF16 || t == GEMM_VALUE_F16 || t == GEMM_VALUE_F32; }
int64_t value_bytes(int t) { return t == GEMM_VALUE_F32 ? 4 : 2; }

// Of 65536 equally likely numbers, those that drop an element; -1: not a probability.
int drop_count(double p) { return p >= 0 && p <= 1 ? (int)std::floor(p * 65536 + 0.5) : -1; }
Dropout dropout_of(int drop, uint64_t seed, uint64_t offset, const int64_t* step) {
    return Dropout{seed, offset, step, (uint32_t)drop, drop < 65536 ? (float)(65536.0 / (65536 - drop)) : 0.0f};
}

// Rows and columns that the kernels' arithmetic holds, rows of at least one column.
int check_sizes(int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 1 || rows > kMaxDim || cols > kMaxDim) return GEMM_ERR_INVALID_DIM;
    return rows <= kMaxProduct / cols && cols <= (int64_t)1 << 31 ? GEMM_OK : GEMM_ERR_TOO_LARGE;
}

template <class... Args>
int launch(void (*kernel)(Args...), dim3 grid, int threads, hipStream_t stream, Args... values) {
    void* args[] = {&values...};
    return hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, dim3((unsigned)threads), args, 0, stream) ==
                   hipSuccess
               ? GEMM_OK
               : GEMM_ERR_HIP;
}

// A launch has fewer than 2^32 threads: more rows than that take several
// steps of one grid.
constexpr int64_t kMostBlocks = (int64_t)1 << 21;

// ---- shapes ---------------------------------------------------------------------------
// The narrowest shape that holds a row, so that its loads, sums and results
// stay in registers at four waves per SIMD or more.  Forward a wave of its own
// up to 1024 columns (no barriers), then four or eight waves.  Eight waves with
// twice the values per lane lead over sixteen, which leave a CU one workgroup
// (8192 columns of 32 bits, 8192 rows: 191 against 235 us; 16384 of bf16, 4096
// rows: 99 against 126), but for ragged rows of that width they would spill;
// at 4096 columns of 32 bits eight waves lead over four (16384 rows: 196
// against 204).  The gradient's kernel holds a row, the next one and the
// columns' sums: 8 values per lane, and in the widest shapes the sums in LDS.
// Rows of fewer than 8 columns and of more than the widest shape go to the
// kernels that read a row again.
constexpr int64_t kNarrowest = 8, kWidest = 16384;
bool in_registers(int64_t cols) { return cols >= kNarrowest && cols <= kWidest; }
bool grad_in_registers(int type, int64_t cols) {
    return in_registers(cols) && (type != GEMM_VALUE_F32 || cols <= 8192);
}

#define DFT_SHAPE(...)                                                                          \
    if (cols <= NormShape<__VA_ARGS__>::COLS)                                                   \
        return cols % 8 == 0 ? Run<TYPE, NormShape<__VA_ARGS__>, true>::run(args...)            \
                             : Run<TYPE, NormShape<__VA_ARGS__>, false>::run(args...);
template <template <int, class, bool> class Run, int TYPE, class... Args>
int with_shape(int64_t cols, Args... args) {
    constexpr bool WIDE = TYPE == kValueF32;
    DFT_SHAPE(1, 1)
    if constexpr (Run<TYPE, NormShape<1, 1>, true>::GRADIENT) {
        DFT_SHAPE(4, 1)
        DFT_SHAPE(8, 1)
        DFT_SHAPE(16, 1, WIDE)
        if constexpr (!WIDE) { DFT_SHAPE(16, 2, true) }
    } else {
        DFT_SHAPE(1, 2)
        DFT_SHAPE(4, 1)
        if constexpr (WIDE) {
            DFT_SHAPE(8, 1)
        } else {
            DFT_SHAPE(4, 2)
        }
        DFT_SHAPE(8, 2)
        if constexpr (WIDE) {
            DFT_SHAPE(16, 2)
        } else if (cols <= kWidest) {
            return cols % 8 == 0 ? Run<TYPE, NormShape<8, 4>, true>::run(args...)
                                 : Run<TYPE, NormShape<16, 2>, false>::run(args...);
        }
    }
    return GEMM_ERR_TOO_LARGE;  // (not reached)
}
#undef DFT_SHAPE
template <template <int, class, bool> class Run, class... Args>
int with_type(int type, int64_t cols, Args... args) {
    if (type == GEMM_VALUE_BF16) return with_shape<Run, kInputBf16>(cols, args...);
    if (type == GEMM_VALUE_F16) return with_shape<Run, kInputF16>(cols, args...);
    return with_shape<Run, kValueF32>(cols, args...);
}

template <int TYPE, class Shape, bool WHOLE>
struct RunNorm {
    static constexpr bool GRADIENT = false;
    static int run(const NormProblem* p, hipStream_t stream) {
        const int64_t blocks = std::min(ceil_div(p->rows, Shape::ROWS), kMostBlocks);
        return launch(norm_kernel<TYPE, Shape, WHOLE>, dim3((unsigned)blocks), Shape::THREADS, stream, *p);
    }
};

// Workgroups of the gradient's kernel: sixteen waves per CU, each with as
// many rows as it takes, since each leaves a row of sums to join.  That was
// measured for many rows (16384 x 4096); up to some thousand a place has a row or
// two, and its sums outweigh them: 1000 x 513 fp32 8.0 us and 5.9 for the join.
template <int TYPE, class Shape, bool WHOLE>
struct GradPlaces {
    static constexpr bool GRADIENT = true;
    static int run(int64_t rows, int cus) {
        return (int)std::min<int64_t>(ceil_div(rows, Shape::ROWS), (int64_t)cus * (1024 / Shape::THREADS));
    }
};
template <int TYPE, class Shape, bool WHOLE>
struct RunGrad {
    static constexpr bool GRADIENT = true;
    static int run(const NormProblem* p, hipStream_t stream) {
        return launch(norm_grad_kernel<TYPE, Shape, WHOLE>, dim3((unsigned)p->places), Shape::THREADS, stream, *p);
    }
};
int grad_places(int type, int64_t rows, int64_t cols, int cus) {
    // rows that are read again: the columns' sums, a workgroup for every 2048 columns of a place
    if (!grad_in_registers(type, cols)) return (int)std::min<int64_t>(rows, 256);
    return with_type<GradPlaces>(type, cols, rows, cus);
}

int run_norm(const gemm_layer_norm_args& a, hipStream_t stream) {
    if (!known_value(a.value_type) || !(a.eps >= 0) || std::isinf(a.eps)) return GEMM_ERR_UNSUPPORTED;
    const int drop = drop_count(a.p);
    if (drop < 0) return GEMM_ERR_UNSUPPORTED;
    int st = check_sizes(a.rows, a.cols);
    if (st != GEMM_OK) return st;
    const int64_t size = value_bytes(a.value_type);
    const bool joined = a.residual || a.p > 0;
    const Matrix x{a.x, a.rows, a.cols, a.ldx, size}, residual{a.residual, a.rows, a.cols, a.ldr, size};
    const Matrix total{joined ? a.total : nullptr, a.rows, a.cols, a.ldt, size}, y{a.y, a.rows, a.cols, a.ldy, size};
    // total may lie over x or over the residual, whose rows are read before it is written, and is then checked as
    // itself alone
    const bool over_x = total.data && total.same_place(x), over_r = total.data && total.same_place(residual);
    const Matrix none{nullptr, 0, 0, 1, size};
    const auto list = [](const void* p, int64_t n, int64_t elem) { return Matrix{p, 1, n, std::max<int64_t>(n, 1), elem}; };
    const Use uses[] = {{over_x ? none : x, over_x, false}, {over_r ? none : residual, true, false},
                        {list(a.weight, a.cols, size), true, false}, {list(a.bias, a.cols, size), true, false},
                        {total, !joined, true}, {y, false, true}, {list(a.mean, a.rows, 4), true, true},
                        {list(a.rstd, a.rows, 4), true, true}, {list(drop > 0 ? a.step : nullptr, 1, 8), true, false}};
    st = check_matrices(uses, 9);
    if (st != GEMM_OK || a.rows == 0) return st;
    int cus = 0;
    st = current_cus(&cus);
    if (st != GEMM_OK) return st;
    NormProblem p{};
    p.rows = a.rows; p.cols = a.cols; p.eps = a.eps;
    p.dropout = dropout_of(drop, a.seed, a.offset, a.step);
    p.x = a.x; p.ldx = a.ldx;
    p.residual = a.residual; p.ldr = a.ldr;
    p.weight = a.weight; p.bias = a.bias;
    p.total = const_cast<void*>(total.data); p.ldt = a.ldt;
    p.y = a.y; p.ldy = a.ldy;
    p.mean = a.mean; p.rstd = a.rstd;
    if (in_registers(a.cols)) return with_type<RunNorm>(a.value_type, a.cols, (const NormProblem*)&p, stream);
    const dim3 grid((unsigned)std::min(a.rows, kMostBlocks));
    if (a.value_type == GEMM_VALUE_BF16) return launch(norm_wide_kernel<kInputBf16>, grid, kWideThreads, stream, p);
    if (a.value_type == GEMM_VALUE_F16) return launch(norm_wide_kernel<kInputF16>, grid, kWideThreads, stream, p);
    return launch(norm_wide_kernel<kValueF32>, grid, kWideThreads, stream, p);
}

template <int TYPE>
int run_wide_grad(const NormProblem& p, hipStream_t stream) {
    int st = GEMM_OK;
    if (p.dtotal || p.dx)
        st = launch(norm_grad_wide_kernel<TYPE>, dim3((unsigned)std::min(p.rows, kMostBlocks)), kWideThreads, stream, p);
    if (st == GEMM_OK && p.partial)
        st = launch(norm_columns_kernel<TYPE>, dim3((unsigned)p.places, (unsigned)ceil_div(p.cols, 2048)), 256, stream, p);
    return st;
}

// What a gradient call needs of the workspace, or a negative status.
int64_t check_grad(const gemm_layer_norm_grad_args& a, int* drop) {
    if (!known_value(a.value_type)) return GEMM_ERR_UNSUPPORTED;
    *drop = drop_count(a.p);
    if (*drop < 0) return GEMM_ERR_UNSUPPORTED;
    int st = check_sizes(a.rows, a.cols);
    if (st != GEMM_OK) return st;
    if (a.cols > (int64_t)0xffff * 2048) return GEMM_ERR_TOO_LARGE;  // (the columns' grid)
    if (a.workspace_bytes < 0) return GEMM_ERR_WORKSPACE;
    const int64_t size = value_bytes(a.value_type);
    const auto matrix = [&](const void* p, int64_t ld) { return Matrix{p, a.rows, a.cols, ld, size}; };
    const auto list = [](const void* p, int64_t n, int64_t elem) { return Matrix{p, 1, n, std::max<int64_t>(n, 1), elem}; };
    const bool work = a.dtotal || a.dx || a.dweight || a.dbias;
    const Use uses[] = {{matrix(a.dY, a.ldy), !work, false}, {matrix(a.total, a.ldt), !work, false},
                        {list(a.mean, a.rows, 4), !work, false}, {list(a.rstd, a.rows, 4), !work, false},
                        {list(a.weight, a.cols, size), true, false}, {matrix(a.dstream, a.lds), true, false},
                        {matrix(a.dtotal, a.lddt), true, true}, {matrix(a.dx, a.lddx), true, true},
                        {list(a.dweight, a.cols, 4), true, true}, {list(a.dbias, a.cols, 4), true, true},
                        {list(a.workspace, a.workspace_bytes, 1), true, true},
                        {list(*drop > 0 && a.dx ? a.step : nullptr, 1, 8), true, false}};
    return check_matrices(uses, 12);
}
int64_t grad_workspace(const gemm_layer_norm_grad_args& a, int cus) {
    return a.dweight || a.dbias ? (int64_t)grad_places(a.value_type, a.rows, a.cols, cus) * 2 * a.cols * 4 : 0;
}

int run_grad(const gemm_layer_norm_grad_args& a, hipStream_t stream) {
    int drop = 0, cus = 0;
    int st = (int)check_grad(a, &drop);
    if (st != GEMM_OK || (!a.dtotal && !a.dx && !a.dweight && !a.dbias)) return st;
    if (a.rows == 0 && !a.dweight && !a.dbias) return GEMM_OK;
    st = current_cus(&cus);
    if (st != GEMM_OK) return st;
    const int64_t need = grad_workspace(a, cus);
    if (need > 0 && (!a.workspace || a.workspace_bytes < need || ((uintptr_t)a.workspace & 15))) return GEMM_ERR_WORKSPACE;
    NormProblem p{};
    p.rows = a.rows; p.cols = a.cols;
    p.dropout = dropout_of(drop, a.seed, a.offset, a.step);
    p.y = const_cast<void*>(a.dY); p.ldy = a.ldy;
    p.total = const_cast<void*>(a.total); p.ldt = a.ldt;
    p.mean = const_cast<float*>(a.mean); p.rstd = const_cast<float*>(a.rstd);
    p.weight = a.weight;
    p.dstream = a.dstream; p.lds = a.lds;
    p.dtotal = a.dtotal; p.lddt = a.lddt;
    p.dx = a.dx; p.lddx = a.lddx;
    p.dweight = a.dweight; p.dbias = a.dbias;
    p.places = grad_places(a.value_type, a.rows, a.cols, cus);
    p.partial = a.dweight || a.dbias ? static_cast<float*>(a.workspace) : nullptr;
    if (a.rows > 0) {
        if (grad_in_registers(a.value_type, a.cols))
            st = with_type<RunGrad>(a.value_type, a.cols, (const NormProblem*)&p, stream);
        else if (a.value_type == GEMM_VALUE_BF16)
            st = run_wide_grad<kInputBf16>(p, stream);
        else if (a.value_type == GEMM_VALUE_F16)
            st = run_wide_grad<kInputF16>(p, stream);
        else
            st = run_wide_grad<kValueF32>(p, stream);
        if (st != GEMM_OK) return st;
    }
    if (!a.dweight && !a.dbias) return GEMM_OK;
    return launch(norm_join_kernel, dim3((unsigned)ceil_div(a.cols, kNormJoinCols), 2), kNormJoinCols * kNormJoinStrides,
                  stream, p);
}

template <int TYPE>
int run_dropout(const DropoutProblem& p, hipStream_t stream) {
    const int64_t blocks = std::min(ceil_div(p.rows * ceil_div(p.cols, 8), 256), kMostBlocks * 4);
    return p.cols % 8 == 0 ? launch(dropout_kernel<TYPE, true>, dim3((unsigned)blocks), 256, stream, p)
                           : launch(dropout_kernel<TYPE, false>, dim3((unsigned)blocks), 256, stream, p);
}

}  // namespace

// ---- exported C ABI ---------------------------------------------------------------------
extern "C" {

int gemm_layer_norm(const gemm_layer_norm_args* args, void* stream) {
    return args ? run_norm(*args, (hipStream_t)stream) : GEMM_ERR_NULL;
}

int gemm_layer_norm_grad(const gemm_layer_norm_grad_args* args, void* stream) {
    return args ? run_grad(*args, (hipStream_t)stream) : GEMM_ERR_NULL;
}

int64_t gemm_layer_norm_grad_workspace_bytes(const gemm_layer_norm_grad_args* args, int32_t num_cus) {
    if (!args) return GEMM_ERR_NULL;
    if (num_cus < 1) return GEMM_ERR_INVALID_DIM;
    gemm_layer_norm_grad_args a = *args;
    a.workspace = nullptr;
    a.workspace_bytes = 0;
    int drop = 0;
    const int64_t st = check_grad(a, &drop);
    return st != GEMM_OK ? st : grad_workspace(a, num_cus);
}

int gemm_dropout(int value_type, int64_t rows, int64_t cols, double p, uint64_t seed, uint64_t offset,
                 const int64_t* step, const void* X, int64_t ldx, const void* residual, int64_t ldr, void* Y,
                 int64_t ldy, void* stream) {
    if (!known_value(value_type)) return GEMM_ERR_UNSUPPORTED;
    const int drop = drop_count(p);
    if (drop < 0) return GEMM_ERR_UNSUPPORTED;
    if (rows < 0 || cols < 0) return GEMM_ERR_INVALID_DIM;
    int st = check_sizes(rows, std::max<int64_t>(cols, 1));
    if (st != GEMM_OK) return st;
    const int64_t size = value_bytes(value_type);
    const Matrix x{X, rows, cols, ldx, size}, r{residual, rows, cols, ldr, size}, y{Y, rows, cols, ldy, size};
    // Y may lie over X or over the residual: each value is read before it is written
    const bool over_x = y.data && y.same_place(x), over_r = y.data && y.same_place(r);
    const Matrix none{nullptr, 0, 0, 1, size};
    const Use uses[] = {{over_x ? none : x, over_x, false}, {over_r ? none : r, true, false}, {y, false, true},
                        {Matrix{drop > 0 ? step : nullptr, 1, 1, 1, 8}, true, false}};
    st = check_matrices(uses, 4);
    if (st != GEMM_OK || rows == 0 || cols == 0) return st;
    int cus = 0;
    st = current_cus(&cus);
    if (st != GEMM_OK) return st;
    DropoutProblem problem{rows, cols, dropout_of(drop, seed, offset, step), X, ldx, residual, ldr, Y, ldy};
    if (cols % 8 == 0 && (rows == 1 || (ldx == cols && ldy == cols && (!residual || ldr == cols)))) {
        problem.rows = 1;
        problem.cols = rows * cols;
    }
    if (value_type == GEMM_VALUE_BF16) return run_dropout<kInputBf16>(problem, (hipStream_t)stream);
    if (value_type == GEMM_VALUE_F16) return run_dropout<kInputF16>(problem, (hipStream_t)stream);
    return run_dropout<kValueF32>(problem, (hipStream_t)stream);
}

}  // extern "C"
