// linear_api.hip -- the C ABI of the products with an epilogue, their
// gradients and the token sort (include/dense_fp32_tiled.h): what each call
// takes, and the launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <stdint.h>

#include "dense_fp32_tiled.h"
#include "expert_kernels.hpp"
#include "host_checks.hpp"
#include "linear_plan.hpp"
#include "slope_kernels.hpp"

namespace {

using namespace dft;

bool known_act(int a) { return a >= 0 && a < kActCount; }

hipError_t launch(int type, const LinearProblem& p, LinearLayout layout, const Plan& plan, int cus,
                  hipStream_t stream) {
    const TileSize size = kTileSizes[plan.tile];
    const uint32_t tiles_m = (uint32_t)row_tiles(p.R, p.groups, p.axis, size.bm), tiles_n = (uint32_t)ceil_div(p.C, size.bn);
    const uint32_t grid_y = p.axis == kGroupContraction ? (uint32_t)p.groups : (uint32_t)plan.splits;
    if (tiles_m == 0 || tiles_n == 0) return hipSuccess;
    const hipError_t e = type == GEMM_INPUT_BF16
                             ? launch_linear_bf16(p, layout, plan.tile, plan.direct, tiles_m, tiles_n, grid_y, cus, stream)
                             : launch_linear_f16(p, layout, plan.tile, plan.direct, tiles_m, tiles_n, grid_y, cus, stream);
    if (e != hipSuccess) return e;
    LinearProblem problem = p;
    if (p.tail) {
        uint32_t m = tiles_m, n = tiles_n, grid = std::min<uint32_t>((uint32_t)cus, tiles_m * tiles_n);
        void* args[] = {&problem, &m, &n, &grid};
        const void* join = type == GEMM_INPUT_BF16
                               ? reinterpret_cast<const void*>(linear_tail_kernel<kInputBf16, 256, 256>)
                               : reinterpret_cast<const void*>(linear_tail_kernel<kInputF16, 256, 256>);
        return hipLaunchKernel(join, dim3(grid / 2, 256 / 32), dim3(256), args, 0, stream);
    }
    if (plan.splits <= 1) return e;
    const int64_t blocks = std::min<int64_t>(ceil_div(p.R * ceil_div(p.C, 8), kJoinGroups), 16384);
    void* args[] = {&problem};
    const void* join = type == GEMM_INPUT_BF16 ? reinterpret_cast<const void*>(linear_join_kernel<kInputBf16>)
                                               : reinterpret_cast<const void*>(linear_join_kernel<kInputF16>);
    return hipLaunchKernel(join, dim3((unsigned)blocks), dim3(kJoinThreads), args, 0, stream);
}

// ---- gemm_linear ----------------------------------------------------------------------
// `bias`: joined by the same launch; nullptr: nothing to join.
int launch_pack(const Matrix* from, Matrix* to, int n, Space* space, const SlopeProblem* bias, hipStream_t stream) {
    PackJobs jobs{};
    SlopeProblem join = bias ? *bias : SlopeProblem{};
    int64_t most = 1;
    for (int i = 0; i < n; ++i) {
        to[i] = packed(from[i]);
        to[i].data = space->take(packed_bytes(from[i]));
        jobs.job[i] = PackJob{static_cast<const uint16_t*>(from[i].data), from[i].rows, from[i].cols, from[i].ld,
                              from[i].copies, from[i].copy_stride,
                              static_cast<uint16_t*>(const_cast<void*>(to[i].data)), to[i].ld};
        most = std::max(most, from[i].copies * from[i].rows * (to[i].ld / 8));
    }
    void* args[] = {&jobs, &n, &join};
    const int64_t joins = bias ? ceil_div(join.N, 64) * join.groups : 0;
    const unsigned blocks = (unsigned)std::min<int64_t>(std::max(ceil_div(most, 256), joins), 65536);
    return hipLaunchKernel(reinterpret_cast<const void*>(linear_pack_kernel), dim3(blocks, (unsigned)n + (bias ? 1 : 0)),
                           dim3(256), args, 0, stream) == hipSuccess
               ? GEMM_OK
               : GEMM_ERR_HIP;
}

struct LinearCall {
    Matrix A, B, bias, residual, preact, out;
    int64_t groups;
    int axis;
};

int describe(const gemm_linear_args& a, LinearCall* c) {
    if (!known_type(a.input_type) || !known_output(a.output_type) || !known_act(a.activation)) return GEMM_ERR_UNSUPPORTED;
    if (a.variant < 0 || a.variant >= GEMM_LINEAR_COUNT) return GEMM_ERR_UNSUPPORTED;
    if (a.M < 0 || a.N < 0 || a.K < 0 || a.M > kMaxDim || a.N > kMaxDim || a.K > kMaxDim) return GEMM_ERR_INVALID_DIM;
    if (a.groups < 0 || a.groups > GEMM_LINEAR_MAX_GROUPS || a.splits < 0 || a.splits > kMaxSlices) return GEMM_ERR_INVALID_DIM;
    if ((a.groups > 0 && a.M > 0x7fffffff) || !products_ok(a.M, a.N, a.K)) return GEMM_ERR_TOO_LARGE;
    c->groups = a.groups > 0 ? a.groups : 1;
    c->axis = a.groups > 0 ? kGroupRows : kGroupNone;
    const int64_t out = elem_bytes(a.output_type);
    c->A = Matrix{a.A, a.M, a.K, a.lda, 2};
    c->B = Matrix{a.B, a.K, a.N, a.ldb, 2, c->groups, a.b_stride};
    c->bias = Matrix{a.bias, 1, a.N, std::max<int64_t>(a.N, 1), 2, c->groups, a.bias_stride};
    c->residual = Matrix{a.residual, a.M, a.N, a.ldr, out};
    c->preact = Matrix{a.preact, a.M, a.N, a.ldp, 2};
    c->out = Matrix{a.D, a.M, a.N, a.ldd, out};
    const bool in_place = c->residual.data && c->residual.same_place(c->out);
    const Matrix offsets{a.groups > 0 ? a.offsets : nullptr, 1, a.groups + 1, a.groups + 1, 4};
    const Matrix space{a.workspace, 1, a.workspace_bytes, std::max<int64_t>(a.workspace_bytes, 1), 1};
    if (a.workspace_bytes < 0) return GEMM_ERR_WORKSPACE;
    // an empty output: nothing is read
    const bool work = a.M > 0 && a.N > 0;
    const Use uses[] = {{c->A, !work, false}, {c->B, !work, false}, {c->bias, true, false},
                        {in_place ? Matrix{nullptr, 0, 0, 1, 2} : c->residual, true, false}, {c->preact, true, true},
                        {c->out, !work, true}, {offsets, a.groups == 0 || !work, false}, {space, true, true}};
    const int st = check_matrices(uses, 8);
    if (st != GEMM_OK) return st;
    return out_pitch_ok(c->out) && out_pitch_ok(c->residual) && out_pitch_ok(c->preact) ? GEMM_OK : GEMM_ERR_TOO_LARGE;
}

// The operands as they are, or, where their rows are not whole 16 bytes and
// the product is large enough to win the copies' time back, packed.
struct LinearPlan {
    Plan plan;
    bool pack_a, pack_b;
    int64_t workspace;  // bytes
    bool tail;          // slices of the last round
};
int plan_linear(const gemm_linear_args& a, const LinearCall& c, int cus, LinearPlan* plan) {
    LinearPlan& best = *plan;
    best = LinearPlan{choose(a.M, a.N, a.K, c.groups, c.axis, path_of(c.A, true, c.B, false), a.variant, a.splits, cus),
                      false, false, 0, false};
    if (!best.plan.direct && a.K > 0) {
        const bool pack_a = !whole_rows(c.A), pack_b = !whole_rows(c.B);
        const Matrix A = pack_a ? packed(c.A) : c.A, B = pack_b ? packed(c.B) : c.B;
        if (copies_fit(kTile256, A, true, B, false)) {
            const Plan p = choose(a.M, a.N, a.K, c.groups, c.axis, kDirect, a.variant, a.splits, cus);
            const double us = p.us + kPackLaunch + (pack_a ? pack_us(c.A) : 0) + (pack_b ? pack_us(c.B) : 0);
            if (us < best.plan.us) best = LinearPlan{p, pack_a, pack_b, 0, false};
        }
    }
    if (!best.plan.found()) return GEMM_ERR_TOO_LARGE;
    best.tail = tail_bytes(best.plan, a.M, a.N, a.K, c.groups, c.axis, cus) > 0;
    best.workspace = (best.pack_a ? packed_bytes(c.A) : 0) + (best.pack_b ? packed_bytes(c.B) : 0) +
                     partial_bytes(best.plan, a.M, a.N) + tail_bytes(best.plan, a.M, a.N, a.K, c.groups, c.axis, cus);
    return GEMM_OK;
}

int run_linear(const gemm_linear_args& a, hipStream_t stream) {
    LinearCall c;
    int st = describe(a, &c);
    if (st != GEMM_OK) return st;
    if (a.M == 0 || a.N == 0) return GEMM_OK;
    int cus = 0;
    st = current_cus(&cus);
    if (st != GEMM_OK) return st;
    LinearPlan chosen;
    st = plan_linear(a, c, cus, &chosen);
    if (st != GEMM_OK) return st;
    const Plan& plan = chosen.plan;
    if (!workspace_ok(chosen.workspace, a.workspace, a.workspace_bytes)) return GEMM_ERR_WORKSPACE;
    Space space{static_cast<char*>(a.workspace)};
    Matrix A = c.A, B = c.B, from[2], to[2];
    int n = 0;
    if (chosen.pack_a) from[n++] = c.A;
    if (chosen.pack_b) from[n++] = c.B;
    if (n > 0) {
        st = launch_pack(from, to, n, &space, nullptr, stream);
        if (st != GEMM_OK) return st;
        if (chosen.pack_a) A = to[0];
        if (chosen.pack_b) B = to[n - 1];
    }
    LinearProblem p{};
    p.R = a.M; p.C = a.N; p.L = a.K;
    p.A = static_cast<const uint16_t*>(A.data); p.lda = A.ld;
    p.B = static_cast<const uint16_t*>(B.data); p.ldb = B.ld; p.b_group = B.copy_stride;
    p.offsets = a.offsets; p.groups = (int32_t)c.groups; p.axis = c.axis;
    p.splits = plan.splits; p.slice = plan.slice; p.partial = reinterpret_cast<float*>(space.at);
    p.tail = chosen.tail ? reinterpret_cast<float*>(space.at) : nullptr;
    p.ep.bias = static_cast<const uint16_t*>(a.bias); p.ep.bias_group = a.bias_stride;
    p.ep.residual = a.residual; p.ep.ldr = a.ldr;
    p.ep.preact = static_cast<uint16_t*>(a.preact); p.ep.ldp = a.ldp;
    p.ep.out = a.D; p.ep.ldo = a.ldd;
    p.ep.act = a.activation; p.ep.out_f32 = a.output_type == GEMM_OUTPUT_F32;
    return launch(a.input_type, p, kForward, plan, cus, stream) == hipSuccess ? GEMM_OK : GEMM_ERR_HIP;
}

// ---- gemm_linear_grad -------------------------------------------------------------------
struct GradCall {
    Matrix dY, Z, A, B, dZ, dA, dB, dbias;
    int64_t groups;
    int axis;
    Matrix slope() const { return dZ.data ? dZ : dY; }  // what the products read
};

int describe(const gemm_linear_grad_args& a, GradCall* c) {
    if (!known_type(a.input_type) || !known_act(a.activation)) return GEMM_ERR_UNSUPPORTED;
    if (!known_output(a.a_grad_type) || !known_output(a.b_grad_type)) return GEMM_ERR_UNSUPPORTED;
    if (a.M < 0 || a.N < 0 || a.K < 0 || a.M > kMaxDim || a.N > kMaxDim || a.K > kMaxDim) return GEMM_ERR_INVALID_DIM;
    if (a.groups < 0 || a.groups > GEMM_LINEAR_MAX_GROUPS) return GEMM_ERR_INVALID_DIM;
    if ((a.groups > 0 && a.M > 0x7fffffff) || !products_ok(a.M, a.N, a.K)) return GEMM_ERR_TOO_LARGE;
    c->groups = a.groups > 0 ? a.groups : 1;
    c->axis = a.groups > 0 ? kGroupRows : kGroupNone;
    const bool act = a.activation != GEMM_ACT_NONE;
    c->dY = Matrix{a.dY, a.M, a.N, a.ldy, 2};
    c->Z = Matrix{act ? a.Z : nullptr, a.M, a.N, a.ldz, 2};
    c->dZ = Matrix{act ? a.dZ : nullptr, a.M, a.N, a.lddz, 2};
    c->A = Matrix{a.dB ? a.A : nullptr, a.M, a.K, a.lda, 2};
    c->B = Matrix{a.dA ? a.B : nullptr, a.K, a.N, a.ldb, 2, c->groups, a.b_stride};
    c->dA = Matrix{a.dA, a.M, a.K, a.ldda, elem_bytes(a.a_grad_type)};
    c->dB = Matrix{a.dB, a.K, a.N, a.lddb, elem_bytes(a.b_grad_type), c->groups, a.db_stride};
    c->dbias = Matrix{a.dbias, c->groups, a.N, std::max<int64_t>(a.N, 1), 4};
    const Matrix offsets{a.groups > 0 ? a.offsets : nullptr, 1, a.groups + 1, a.groups + 1, 4};
    if (a.workspace_bytes < 0) return GEMM_ERR_WORKSPACE;
    const Matrix space{a.workspace, 1, a.workspace_bytes, std::max<int64_t>(a.workspace_bytes, 1), 1};
    // dZ may overwrite dY, which is then checked as dZ alone: a written matrix
    const bool in_place = c->dZ.data && c->dZ.same_place(c->dY);
    const Use uses[] = {{in_place ? Matrix{nullptr, 0, 0, 1, 2} : c->dY, in_place, false}, {c->Z, !act, false},
                        {c->dZ, !act, true},
                        {c->A, !a.dB, false}, {c->B, !a.dA, false}, {c->dA, true, true}, {c->dB, true, true},
                        {c->dbias, true, true}, {offsets, a.groups == 0, false}, {space, true, true}};
    const int st = check_matrices(uses, 10);
    if (st != GEMM_OK) return st;
    return out_pitch_ok(c->dA) && out_pitch_ok(c->dB) ? GEMM_OK : GEMM_ERR_TOO_LARGE;
}

Plan plan_a(const gemm_linear_grad_args& a, const GradCall& c, Path path, int cus) {
    return choose(a.M, a.K, a.N, c.groups, c.axis, path, GEMM_LINEAR_AUTO, 0, cus);
}
Plan plan_b(const gemm_linear_grad_args& a, const GradCall& c, Path path, int cus) {
    return choose(a.K, a.N, a.M, c.groups, c.axis == kGroupRows ? kGroupContraction : kGroupNone, path,
                  GEMM_LINEAR_AUTO, 0, cus);
}
// Few rows of one matrix: one chunk, whose sums need no join (4096 columns: 1
// row 4.7 against 5.5 us, 17 rows 5.1 against 6.3; 64 rows 9.3 against 6.4).
bool one_chunk(const gemm_linear_grad_args& a) { return a.groups == 0 && a.M > 0 && a.M <= 32; }
int slope_rows(const gemm_linear_grad_args& a) {
    if (one_chunk(a)) return kSlopeRows;
    return ceil_div(a.M, kSlopeRows) * ceil_div(a.N, 256) < 1024 ? kFewSlopeRows : kSlopeRows;
}
int64_t slope_chunks(const gemm_linear_grad_args& a, const GradCall& c) {
    return row_tiles(a.M, c.groups, c.axis, slope_rows(a));
}

// Both products' plans, with dZ, A and B as they are or packed (one choice
// for all that have rows of other than whole 16 bytes, dZ being read by both).
// The workspace holds what is packed, then the column sums' chunks and each
// product's slices, one after the other (the launches run in stream order).
struct GradPlan {
    Plan a, b;
    bool pack_z, pack_a, pack_b;
    int64_t workspace;
    bool tail_a, tail_b;  // slices of the last rounds
};
int plan_grad(const gemm_linear_grad_args& a, const GradCall& c, int cus, GradPlan* plan) {
    // the slope kernel's grid: 256 columns by a chunk of rows per workgroup
    const bool slopes = a.N > 0 && (c.dZ.data || a.dbias);
    if (slopes && (slope_chunks(a, c) > kMaxGrid / 256 || a.N > (int64_t)0xffff * 256)) return GEMM_ERR_TOO_LARGE;
    const Matrix dz = c.slope();
    const bool want_a = a.dA && a.M > 0 && a.K > 0, want_b = a.dB && a.K > 0 && a.N > 0;
    GradPlan& best = *plan;
    best = GradPlan{plan_a(a, c, path_of(dz, true, c.B, true), cus), plan_b(a, c, path_of(c.A, false, dz, false), cus),
                    false, false, false, 0, false, false};
    const bool slow = (want_a && !best.a.direct) || (want_b && !best.b.direct);
    if (slow && a.M > 0 && a.N > 0) {
        const bool z = !whole_rows(dz), pa = want_b && !whole_rows(c.A), pb = want_a && !whole_rows(c.B);
        const Matrix Z = z ? packed(dz) : dz, A = pa ? packed(c.A) : c.A, B = pb ? packed(c.B) : c.B;
        if ((!want_a || copies_fit(kTile256, Z, true, B, true)) && (!want_b || copies_fit(kTile256, A, false, Z, false))) {
            const Plan p = plan_a(a, c, kDirect, cus), q = plan_b(a, c, kDirect, cus);
            const double before = (want_a ? best.a.us : 0) + (want_b ? best.b.us : 0);
            const double after = (want_a ? p.us : 0) + (want_b ? q.us : 0) + kPackLaunch + (z ? pack_us(dz) : 0) +
                                 (pa ? pack_us(c.A) : 0) + (pb ? pack_us(c.B) : 0);
            if (after < before) best = GradPlan{p, q, z, pa, pb, 0, false, false};
        }
    }
    if ((want_a && !best.a.found()) || (want_b && !best.b.found())) return GEMM_ERR_TOO_LARGE;
    int64_t rest = a.dbias && !one_chunk(a) ? slope_chunks(a, c) * a.N * 4 : 0;
    const int axis_b = c.axis == kGroupRows ? kGroupContraction : kGroupNone;
    const int64_t tail_a = want_a ? tail_bytes(best.a, a.M, a.K, a.N, c.groups, c.axis, cus) : 0;
    const int64_t tail_b = want_b ? tail_bytes(best.b, a.K, a.N, a.M, c.groups, axis_b, cus) : 0;
    best.tail_a = tail_a > 0;
    best.tail_b = tail_b > 0;
    if (want_a) rest = std::max({rest, partial_bytes(best.a, a.M, a.K), tail_a});
    if (want_b) rest = std::max({rest, partial_bytes(best.b, a.K, a.N), tail_b});
    best.workspace = (best.pack_z ? packed_bytes(dz) : 0) + (best.pack_a ? packed_bytes(c.A) : 0) +
                     (best.pack_b ? packed_bytes(c.B) : 0) + rest;
    return GEMM_OK;
}

// dZ and the chunks' sums; what is left to join of them.
SlopeProblem slope_problem(const gemm_linear_grad_args& a, const GradCall& c, float* partial) {
    SlopeProblem p{};
    p.M = a.M; p.N = a.N;
    p.dY = static_cast<const uint16_t*>(a.dY); p.ldy = a.ldy;
    p.Z = static_cast<const uint16_t*>(c.Z.data); p.ldz = a.ldz;
    p.dZ = static_cast<uint16_t*>(const_cast<void*>(c.dZ.data)); p.lddz = a.lddz;
    p.partial = !a.dbias ? nullptr : one_chunk(a) ? a.dbias : partial;
    p.offsets = a.groups > 0 ? a.offsets : nullptr; p.groups = (int32_t)c.groups;
    p.act = a.activation; p.dbias = a.dbias; p.chunk_rows = slope_rows(a);
    p.chunks = slope_chunks(a, c);
    return p;
}
int run_slope(int input_type, SlopeProblem p, hipStream_t stream) {
    if ((!p.dZ && !p.partial) || p.chunks == 0 || p.N == 0) return GEMM_OK;
    void* args[] = {&p};
    const void* kernel = input_type == GEMM_INPUT_BF16 ? reinterpret_cast<const void*>(linear_slope_kernel<kInputBf16>)
                                                       : reinterpret_cast<const void*>(linear_slope_kernel<kInputF16>);
    return hipLaunchKernel(kernel, dim3((unsigned)p.chunks, (unsigned)ceil_div(p.N, 256)), dim3(256), args, 0, stream) ==
                   hipSuccess
               ? GEMM_OK
               : GEMM_ERR_HIP;
}
int run_bias_join(SlopeProblem p, hipStream_t stream) {
    void* args[] = {&p};
    return hipLaunchKernel(reinterpret_cast<const void*>(linear_bias_join_kernel), dim3((unsigned)ceil_div(p.N, 64), (unsigned)p.groups),
                           dim3(256), args, 0, stream) == hipSuccess
               ? GEMM_OK
               : GEMM_ERR_HIP;
}

int run_grad(const gemm_linear_grad_args& a, hipStream_t stream) {
    GradCall c;
    int st = describe(a, &c);
    if (st != GEMM_OK) return st;
    int cus = 0;
    st = current_cus(&cus);
    if (st != GEMM_OK) return st;
    GradPlan plan;
    st = plan_grad(a, c, cus, &plan);
    if (st != GEMM_OK) return st;
    if (!workspace_ok(plan.workspace, a.workspace, a.workspace_bytes)) return GEMM_ERR_WORKSPACE;
    const Plan &pa = plan.a, &pb = plan.b;
    const int axis_b = c.axis == kGroupRows ? kGroupContraction : kGroupNone;
    Space space{static_cast<char*>(a.workspace)};
    // places of what is packed, in front of the rest (its kernel runs after dZ's)
    Matrix from[3], to[3], dz = c.slope(), A = c.A, B = c.B;
    int n = 0;
    if (plan.pack_z) from[n++] = dz;
    if (plan.pack_a) from[n++] = c.A;
    if (plan.pack_b) from[n++] = c.B;
    Space rest = space;
    for (int i = 0; i < n; ++i) rest.take(packed_bytes(from[i]));
    const SlopeProblem slope = slope_problem(a, c, reinterpret_cast<float*>(rest.at));
    if ((st = run_slope(a.input_type, slope, stream)) != GEMM_OK) return st;
    const bool join = a.dbias && a.N > 0 && !one_chunk(a);
    if (join && n == 0 && (st = run_bias_join(slope, stream)) != GEMM_OK) return st;
    if (n > 0) {
        st = launch_pack(from, to, n, &space, join ? &slope : nullptr, stream);
        if (st != GEMM_OK) return st;
        int i = 0;
        if (plan.pack_z) dz = to[i++];
        if (plan.pack_a) A = to[i++];
        if (plan.pack_b) B = to[i++];
    }
    LinearProblem p{};
    p.offsets = a.offsets; p.groups = (int32_t)c.groups;
    p.partial = reinterpret_cast<float*>(rest.at);
    if (a.dA && a.M > 0 && a.K > 0) {
        p.R = a.M; p.C = a.K; p.L = a.N; p.axis = c.axis;
        p.A = static_cast<const uint16_t*>(dz.data); p.lda = dz.ld;
        p.B = static_cast<const uint16_t*>(B.data); p.ldb = B.ld; p.b_group = B.copy_stride;
        p.splits = pa.splits; p.slice = pa.slice; p.tail = plan.tail_a ? p.partial : nullptr;
        p.ep = LinearEpilogue{};
        p.ep.out = a.dA; p.ep.ldo = a.ldda; p.ep.out_f32 = a.a_grad_type == GEMM_OUTPUT_F32;
        if (launch(a.input_type, p, kGradA, pa, cus, stream) != hipSuccess) return GEMM_ERR_HIP;
    }
    if (a.dB && a.K > 0 && a.N > 0) {
        p.R = a.K; p.C = a.N; p.L = a.M; p.axis = axis_b;
        p.A = static_cast<const uint16_t*>(A.data); p.lda = A.ld;
        p.B = static_cast<const uint16_t*>(dz.data); p.ldb = dz.ld; p.b_group = 0;
        p.splits = pb.splits; p.slice = pb.slice; p.tail = plan.tail_b ? p.partial : nullptr;
        p.ep = LinearEpilogue{};
        p.ep.out = a.dB; p.ep.ldo = a.lddb; p.ep.out_group = a.db_stride; p.ep.out_f32 = a.b_grad_type == GEMM_OUTPUT_F32;
        if (launch(a.input_type, p, kGradB, pb, cus, stream) != hipSuccess) return GEMM_ERR_HIP;
    }
    return GEMM_OK;
}

// ---- the token sort ---------------------------------------------------------------------
int64_t sort_workgroups(int64_t pairs) { return ceil_div(pairs, kSortPairs); }
int64_t sort_workspace(int64_t pairs, int64_t experts) {
    return sort_workgroups(pairs) > 1 ? sort_workgroups(pairs) * experts * 4 : 0;
}

int launch_sort(const SortProblem& problem, int64_t workgroups, hipStream_t stream) {
    SortProblem p = problem;
    void* args[] = {&p, &workgroups};
    const dim3 one(1), all((unsigned)std::max<int64_t>(workgroups, 1)), threads(kSortThreads);
    hipError_t e;
    if (workgroups <= 1) {
        e = hipLaunchKernel(reinterpret_cast<const void*>(expert_sort_small_kernel), one, threads, args, 0, stream);
    } else {
        e = hipLaunchKernel(reinterpret_cast<const void*>(expert_count_kernel), all, threads, args, 0, stream);
        if (e == hipSuccess)
            e = hipLaunchKernel(reinterpret_cast<const void*>(expert_offsets_kernel), one, threads, args, 0, stream);
        if (e == hipSuccess)
            e = hipLaunchKernel(reinterpret_cast<const void*>(expert_place_kernel), all, threads, args, 0, stream);
    }
    return e == hipSuccess ? GEMM_OK : GEMM_ERR_HIP;
}

// Sizes shared by the row operators; token and sorted rows.
int check_rows(int input_type, int64_t tokens, int64_t rows, int32_t top_k, int64_t cols) {
    if (!known_type(input_type)) return GEMM_ERR_UNSUPPORTED;
    if (tokens < 0 || rows < 0 || cols < 0 || top_k < 1 || top_k > GEMM_EXPERT_MAX_CHOICES) return GEMM_ERR_INVALID_DIM;
    if (tokens > 0x7fffffff / top_k || rows > 0x7fffffff || cols > (int64_t)0xffff * kRowCols) return GEMM_ERR_TOO_LARGE;
    return GEMM_OK;
}

int launch_rows(const void* kernel, const RowsProblem& problem, bool per_token, hipStream_t stream) {
    int cus = 0;
    const int st = current_cus(&cus);
    if (st != GEMM_OK) return st;
    RowsProblem p = problem;
    void* args[] = {&p};
    p.parts = (uint32_t)ceil_div(p.cols, kRowCols);
    // a launch has fewer than 2^32 threads: longer batches take several steps of one grid
    const int64_t waves = per_token ? kRowWaves : p.parts;
    p.step = std::min(p.tokens, std::max<int64_t>((1 << 24) / waves, 1));
    // (per token: a workgroup for each choice where there are fewer than four tokens per CU)
    const dim3 grid((unsigned)ceil_div(p.step * waves, kRowWaves), per_token && p.tokens < 4 * cus ? p.top_k : 1);
    return hipLaunchKernel(kernel, grid, dim3(kRowWaves * kWave), args, 0, stream) == hipSuccess ? GEMM_OK : GEMM_ERR_HIP;
}

}  // namespace

// ---- exported C ABI ---------------------------------------------------------------------
extern "C" {

int gemm_linear(const gemm_linear_args* args, void* stream) {
    return args ? run_linear(*args, (hipStream_t)stream) : GEMM_ERR_NULL;
}

int64_t gemm_linear_workspace_bytes(const gemm_linear_args* args, int32_t num_cus) {
    if (!args) return GEMM_ERR_NULL;
    if (num_cus < 1) return GEMM_ERR_INVALID_DIM;
    gemm_linear_args a = *args;
    a.workspace = nullptr;
    a.workspace_bytes = 0;
    LinearCall c;
    int st = describe(a, &c);
    if (st != GEMM_OK || a.M == 0 || a.N == 0) return st;
    LinearPlan plan;
    st = plan_linear(a, c, num_cus, &plan);
    return st != GEMM_OK ? st : plan.workspace;
}

int gemm_linear_choice(const gemm_linear_args* args, int32_t num_cus, int32_t* variant, int32_t* splits) {
    if (!args || !variant || !splits) return GEMM_ERR_NULL;
    if (num_cus < 1) return GEMM_ERR_INVALID_DIM;
    LinearCall c;
    int st = describe(*args, &c);
    if (st != GEMM_OK) return st;
    LinearPlan plan;
    st = plan_linear(*args, c, num_cus, &plan);
    if (st != GEMM_OK) return st;
    *variant = plan.plan.tile + 1;
    *splits = plan.plan.splits;
    return GEMM_OK;
}

int gemm_linear_grad(const gemm_linear_grad_args* args, void* stream) {
    return args ? run_grad(*args, (hipStream_t)stream) : GEMM_ERR_NULL;
}

int64_t gemm_linear_grad_workspace_bytes(const gemm_linear_grad_args* args, int32_t num_cus) {
    if (!args) return GEMM_ERR_NULL;
    if (num_cus < 1) return GEMM_ERR_INVALID_DIM;
    gemm_linear_grad_args a = *args;
    a.workspace = nullptr;
    a.workspace_bytes = 0;
    GradCall c;
    int st = describe(a, &c);
    if (st != GEMM_OK) return st;
    GradPlan plan;
    st = plan_grad(a, c, num_cus, &plan);
    return st != GEMM_OK ? st : plan.workspace;
}

int64_t gemm_expert_sort_workspace_bytes(int64_t tokens, int32_t top_k, int32_t num_experts) {
    if (tokens < 0 || top_k < 1 || top_k > GEMM_EXPERT_MAX_CHOICES || num_experts < 1 || num_experts > kMaxExperts)
        return GEMM_ERR_INVALID_DIM;
    if (tokens > 0x7fffffff / top_k) return GEMM_ERR_TOO_LARGE;
    return sort_workspace(tokens * top_k, num_experts);
}

int gemm_expert_sort(int64_t tokens, int32_t top_k, int32_t num_experts, const int32_t* experts, int32_t* offsets,
                     int32_t* order, int32_t* position, void* workspace, int64_t workspace_bytes, void* stream) {
    const int64_t need = gemm_expert_sort_workspace_bytes(tokens, top_k, num_experts);
    if (need < 0) return (int)need;
    const int64_t pairs = tokens * top_k;
    if (workspace_bytes < 0) return GEMM_ERR_WORKSPACE;
    const auto list = [](const void* p, int64_t n) { return Matrix{p, 1, n, std::max<int64_t>(n, 1), 4}; };
    const Use uses[] = {{list(experts, pairs), false, false}, {list(offsets, num_experts + 1), false, true},
                        {list(order, pairs), false, true}, {list(position, pairs), false, true},
                        {list(workspace, workspace_bytes / 4), true, true}};
    int st = check_matrices(uses, 5);
    if (st != GEMM_OK) return st;
    if (need > 0 && (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 3))) return GEMM_ERR_WORKSPACE;
    int cus = 0;
    st = current_cus(&cus);
    if (st != GEMM_OK) return st;
    return launch_sort(SortProblem{experts, pairs, num_experts, offsets, order, position, static_cast<int32_t*>(workspace)},
                       sort_workgroups(pairs), (hipStream_t)stream);
}

int gemm_expert_gather(int input_type, int64_t tokens, int64_t rows, int32_t top_k, int64_t cols, const void* X,
                       int64_t ldx, const int32_t* position, void* sorted, int64_t lds, void* stream) {
    int st = check_rows(input_type, tokens, rows, top_k, cols);
    if (st != GEMM_OK) return st;
    const bool work = tokens > 0 && rows > 0 && cols > 0;
    const Use uses[] = {{Matrix{X, tokens, cols, ldx, 2}, !work, false},
                        {Matrix{position, 1, tokens * top_k, std::max<int64_t>(tokens * top_k, 1), 4}, !work, false},
                        {Matrix{sorted, rows, cols, lds, 2}, !work, true}};
    st = check_matrices(uses, 3);
    if (st != GEMM_OK || !work) return st;
    RowsProblem p{};
    p.tokens = tokens; p.rows = rows; p.cols = cols; p.top_k = top_k; p.position = position;
    p.x = static_cast<const uint16_t*>(X); p.ldx = ldx;
    p.sorted = static_cast<uint16_t*>(sorted); p.lds = lds;
    return launch_rows(reinterpret_cast<const void*>(expert_gather_kernel), p, false, (hipStream_t)stream);
}

int gemm_expert_combine(int input_type, int64_t tokens, int64_t rows, int32_t top_k, int64_t cols, const void* Y,
                        int64_t ldy, const int32_t* position, const float* weights, void* out, int64_t ldo,
                        void* stream) {
    int st = check_rows(input_type, tokens, rows, top_k, cols);
    if (st != GEMM_OK) return st;
    const bool work = tokens > 0 && cols > 0;
    const int64_t pairs = tokens * top_k, width = std::max<int64_t>(pairs, 1);
    const Use uses[] = {{Matrix{Y, rows, cols, ldy, 2}, !work, false},
                        {Matrix{position, 1, pairs, width, 4}, !work, false},
                        {Matrix{weights, 1, pairs, width, 4}, true, false},
                        {Matrix{out, tokens, cols, ldo, 2}, !work, true}};
    st = check_matrices(uses, 4);
    if (st != GEMM_OK || !work) return st;
    RowsProblem p{};
    p.tokens = tokens; p.rows = rows; p.cols = cols; p.top_k = top_k; p.position = position; p.weights = weights;
    p.y = static_cast<const uint16_t*>(Y); p.ldy = ldy;
    p.out = static_cast<uint16_t*>(out); p.ldo = ldo;
    return launch_rows(input_type == GEMM_INPUT_BF16 ? reinterpret_cast<const void*>(expert_combine_kernel<kInputBf16>)
                                                     : reinterpret_cast<const void*>(expert_combine_kernel<kInputF16>),
                       p, false, (hipStream_t)stream);
}

int gemm_expert_combine_grad(int input_type, int64_t tokens, int64_t rows, int32_t top_k, int64_t cols,
                             const void* dout, int64_t ldd, const void* Y, int64_t ldy, const int32_t* position,
                             const float* weights, void* dY, int64_t lddy, float* dweights, void* stream) {
    int st = check_rows(input_type, tokens, rows, top_k, cols);
    if (st != GEMM_OK) return st;
    const bool work = tokens > 0;
    const int64_t pairs = tokens * top_k, width = std::max<int64_t>(pairs, 1);
    const Use uses[] = {{Matrix{dout, tokens, cols, ldd, 2}, !work, false},
                        {Matrix{dweights ? Y : nullptr, rows, cols, ldy, 2}, !work || !dweights, false},
                        {Matrix{position, 1, pairs, width, 4}, !work, false},
                        {Matrix{weights, 1, pairs, width, 4}, true, false},
                        {Matrix{dY, rows, cols, lddy, 2}, true, true},
                        {Matrix{dweights, 1, pairs, width, 4}, true, true}};
    st = check_matrices(uses, 6);
    if (st != GEMM_OK || !work || (!dY && !dweights)) return st;
    RowsProblem p{};
    p.tokens = tokens; p.rows = rows; p.cols = cols; p.top_k = top_k; p.position = position; p.weights = weights;
    p.x = static_cast<const uint16_t*>(dout); p.ldx = ldd;
    p.y = static_cast<const uint16_t*>(Y); p.ldy = ldy;
    p.sorted = static_cast<uint16_t*>(dY); p.lds = lddy;
    p.dweights = dweights;
    return launch_rows(input_type == GEMM_INPUT_BF16
                           ? reinterpret_cast<const void*>(expert_combine_grad_kernel<kInputBf16>)
                           : reinterpret_cast<const void*>(expert_combine_grad_kernel<kInputF16>),
                       p, true, (hipStream_t)stream);
}

}  // extern "C"
