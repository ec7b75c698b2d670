// loss_api.hip -- the C ABI of the cross entropy of a product over a
// vocabulary, and of its gradients (include/dense_fp32_tiled.h): argument
// checks, the pieces of the vocabulary, and the launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <stdint.h>

#include "dense_fp32_tiled.h"
#include "host_checks.hpp"
#include "linear_plan.hpp"
#include "loss_kernels.hpp"

namespace {

using namespace dft;

__global__ __launch_bounds__(kLossJoinThreads) void loss_join_kernel(LossRowsProblem p, int64_t slots, int rows,
                                                                     float* loss, float* lse) {
    loss_join(p, slots, rows, loss, lse);
}
// Workgroups for the rows' values: a row to each thread, of fp16 to each wave.
uint32_t prepare_blocks(const LossPrepare& p) {
    const int64_t blocks = p.A ? std::min<int64_t>((p.rows + kLossBeginWaves - 1) / kLossBeginWaves, kMostLifts)
                               : std::min<int64_t>((p.rows + kLossBeginThreads - 1) / kLossBeginThreads, 64);
    return (uint32_t)std::max<int64_t>(blocks, 1);
}
__global__ __launch_bounds__(kLossBeginThreads) void loss_begin_kernel(LossBegin p) {
    const int job = (int)gridDim.y - p.packs;  // 1 with the rows' values, else 0
    if ((int)blockIdx.y < job)
        loss_prepare(p.prepare, p.prepare_blocks);
    else if (p.each == 1)
        loss_pack<1>(p.pack[blockIdx.y - job]);
    else
        loss_pack<kPackGroups>(p.pack[blockIdx.y - job]);
}
template <int TYPE>
__global__ __launch_bounds__(256) void loss_fold_kernel(LossFold p) {
    loss_fold<TYPE>(p);
}

template <class... Args>
int launch(void (*kernel)(Args...), dim3 blocks, int threads, hipStream_t stream, Args... values) {
    void* args[] = {&values...};
    return hipLaunchKernel(reinterpret_cast<const void*>(kernel), blocks, dim3((unsigned)threads), args, 0,
                           stream) == hipSuccess
               ? GEMM_OK
               : GEMM_ERR_HIP;
}
int status(hipError_t e) { return e == hipSuccess ? GEMM_OK : GEMM_ERR_HIP; }

bool known_target(int t) { return t == GEMM_TARGET_I32 || t == GEMM_TARGET_I64; }
int64_t target_bytes(int t) { return t == GEMM_TARGET_I64 ? 8 : 4; }
int64_t round_up(int64_t n, int64_t to) { return ceil_div(n, to) * to; }

// The rows times the width of a vocabulary's matrix as it lies in memory.
Matrix words_matrix(const void* data, bool transposed, int64_t N, int64_t K, int64_t ld, int64_t elem) {
    return transposed ? Matrix{data, N, K, ld, elem} : Matrix{data, K, N, ld, elem};
}
// Its columns [first, first + words) of the vocabulary.
Matrix piece_of(const Matrix& b, bool transposed, int64_t first, int64_t words) {
    Matrix m = b;
    (transposed ? m.rows : m.cols) = words;
    m.data = static_cast<const char*>(b.data) + first * (transposed ? b.ld : 1) * b.elem;
    return m;
}

constexpr int64_t kMostWords = (int64_t)1 << 20;   // of a piece: dZ's pitch, whose offsets within a tile stay below 2^30
constexpr int64_t kPieceStep = 256;                // pieces end where tiles do
constexpr int64_t kPackedPiece = (int64_t)1 << 26;  // values of a packed piece: 128 MiB, read again from the last-level cache

struct LossSizes {
    int32_t input_type, target_type, b_transposed, variant;
    int64_t M, N, K, piece;
};
template <class Args>
LossSizes sizes_of(const Args& a) {
    return LossSizes{a.input_type, a.target_type, a.b_transposed, a.variant, a.M, a.N, a.K, a.piece};
}
int check_sizes(const LossSizes& s) {
    if (!known_type(s.input_type) || !known_target(s.target_type)) return GEMM_ERR_UNSUPPORTED;
    if (s.b_transposed != 0 && s.b_transposed != 1) return GEMM_ERR_UNSUPPORTED;
    if (s.variant < 0 || s.variant >= GEMM_LINEAR_COUNT) return GEMM_ERR_UNSUPPORTED;
    if (s.M < 0 || s.N < 1 || s.K < 0 || s.M > kMaxDim || s.N > kMaxDim || s.K > kMaxDim) return GEMM_ERR_INVALID_DIM;
    if (s.piece < 0 || s.piece % kPieceStep != 0) return GEMM_ERR_INVALID_DIM;
    if (s.N > 0x7fffffff || s.M > 0x7fffffff || !products_ok(s.M, s.N, s.K)) return GEMM_ERR_TOO_LARGE;
    return GEMM_OK;
}

LossPack pack_job(const Matrix& from, const Matrix& to, int32_t copies, const Targets& targets, int64_t words) {
    return LossPack{static_cast<const uint16_t*>(from.data), from.rows, from.cols, from.ld,
                    static_cast<uint16_t*>(const_cast<void*>(to.data)), to.ld, copies, targets, words, nullptr, nullptr,
                    0, nullptr};
}
// Copies, and the rows' values if they are wanted.
int begin(LossBegin& jobs, bool prepare, hipStream_t stream) {
    if (jobs.packs == 0 && !prepare) return GEMM_OK;
    int64_t most = 1;
    for (int i = 0; i < jobs.packs; ++i) most = std::max(most, jobs.pack[i].copies * jobs.pack[i].rows * (jobs.pack[i].ldd / 8));
    if (prepare) {
        jobs.prepare_blocks = prepare_blocks(jobs.prepare);  // (fewer than the grid has, also with kPackGroups)
        most = std::max(most, (int64_t)jobs.prepare_blocks * kLossBeginThreads);
    }
    jobs.each = most <= kBeginBlocks * kLossBeginThreads ? 1 : kPackGroups;
    return launch(loss_begin_kernel, dim3((unsigned)std::min<int64_t>(ceil_div(most, kLossBeginThreads * jobs.each), 65536),
                                          (unsigned)jobs.packs + (prepare ? 1 : 0)),
                  kLossBeginThreads, stream, jobs);
}

// A product's plan, with kTileShort where that leads (loss_kernels.hpp): of one
// contraction tile always, else where every CU has two of its tiles or more, up
// to `depth` and wherever 128x128 with two places is the choice.
constexpr int64_t kShortLogits = 704, kShortRows = 512;
Plan with_short(Plan plan, int64_t R, int64_t C, int64_t L, int64_t depth, int variant, int cus) {
    const int64_t tiles = ceil_div(R, ShortShape::BM) * ceil_div(C, ShortShape::BN);
    if (variant != GEMM_LINEAR_AUTO || R <= 64 || C <= 64 || tiles > kMaxTiles || plan.splits > 1) return plan;
    const bool many = tiles >= 2 * cus && (L <= depth || plan.tile == kTile128);
    if (!many && L > kTileDepth) return plan;
    plan.tile = kTileShort;
    plan.us = 0;  // (found)
    return plan;
}

// The tile of a piece's logits: never sliced, since its epilogue needs whole sums.
Plan logits_plan(const LossSizes& s, int64_t words, int cus) {
    return with_short(choose(s.M, words, s.K, 1, kGroupNone, kDirect, s.variant, 1, cus), s.M, words, s.K, kShortLogits,
                      s.variant, cus);
}

void describe_logits(LinearProblem& p, const LossSizes& s, const Matrix& a, const Matrix& b, int64_t words) {
    p.R = s.M; p.C = words; p.L = s.K;
    p.A = static_cast<const uint16_t*>(a.data); p.lda = a.ld;
    p.B = static_cast<const uint16_t*>(b.data); p.ldb = b.ld;
    p.groups = 1; p.axis = kGroupNone; p.splits = 1; p.slice = s.K;
}
template <class Problem>
int launch_logits(const LossSizes& s, const Problem& p, LinearTile tile, int cus, hipStream_t stream) {
    const TileSize size = loss_tile_size(tile);
    const uint32_t m = (uint32_t)ceil_div(p.R, size.bm), n = (uint32_t)ceil_div(p.C, size.bn);
    const bool k = s.b_transposed != 0;
    return status(s.input_type == GEMM_INPUT_BF16 ? launch_loss_bf16(p, k, tile, m, n, 1, cus, stream)
                                                  : launch_loss_f16(p, k, tile, m, n, 1, cus, stream));
}

// ---- forward ----------------------------------------------------------------------------
// In the workspace, one after the other: A packed, a piece of B packed, the
// rows' pieces, the targets' logits.  Rows have nothing to do with each other:
// so many of them at a time that their pieces stay within some 512 MiB.
constexpr int64_t kRowsAtOnce = 32768;
struct ForwardPlan {
    bool pack_a, pack_b;
    int64_t rows, piece, slots;
    int width;  // columns of a slot: a wave's
    LinearTile tile;
    int64_t a_bytes, b_bytes, pieces_bytes, target_bytes, workspace;
};
int wave_columns(LinearTile tile) { return tile == kTile64 || tile == kTile32x128 ? 32 : 64; }

int plan_forward(const gemm_cross_entropy_args& a, const Matrix& A, const Matrix& B, int cus, ForwardPlan* plan) {
    LossSizes s = sizes_of(a);
    ForwardPlan& f = *plan;
    const bool work = s.K > 0;
    f.rows = std::min(s.M, kRowsAtOnce);
    f.pack_a = work && !whole_rows(A);
    f.pack_b = work && !whole_rows(B);
    // (B as it is: all of it at once)
    f.piece = s.piece > 0 ? s.piece : f.pack_b ? std::max(kPackedPiece / s.K / kPieceStep, (int64_t)1) * kPieceStep : s.N;
    f.piece = std::min(f.piece, s.N);
    const Matrix a_read = f.pack_a ? packed(A) : A;
    const Matrix b_piece = piece_of(B, s.b_transposed, 0, f.piece), b_read = f.pack_b ? packed(b_piece) : b_piece;
    if (!copies_fit(kTile256, a_read, true, b_read, s.b_transposed)) return GEMM_ERR_TOO_LARGE;
    s.M = f.rows;
    const Plan logits = logits_plan(s, f.piece, cus);
    if (!logits.found()) return GEMM_ERR_TOO_LARGE;
    f.tile = logits.tile;
    f.width = wave_columns(f.tile);
    // (whole tiles of columns: the last one's waves past the vocabulary leave empty slots)
    f.slots = round_up(s.N, loss_tile_size(f.tile).bn) / f.width;
    f.a_bytes = f.pack_a ? packed_bytes(A) : 0;
    f.b_bytes = f.pack_b ? packed_bytes(b_piece) : 0;
    f.pieces_bytes = round_up(f.slots * f.rows * (int64_t)sizeof(RowPiece), 256);
    f.target_bytes = round_up(f.rows * 4, 256);
    f.workspace = f.a_bytes + f.b_bytes + f.pieces_bytes + f.target_bytes;
    return GEMM_OK;
}

int check_forward(const gemm_cross_entropy_args& a, Matrix* A, Matrix* B) {
    const int st = check_sizes(sizes_of(a));
    if (st != GEMM_OK) return st;
    if (a.workspace_bytes < 0) return GEMM_ERR_WORKSPACE;
    *A = Matrix{a.A, a.M, a.K, a.lda, 2};
    *B = words_matrix(a.B, a.b_transposed, a.N, a.K, a.ldb, 2);
    const auto list = [](const void* p, int64_t n, int64_t elem) { return Matrix{p, 1, n, std::max<int64_t>(n, 1), elem}; };
    const bool work = a.M > 0;
    const Use uses[] = {{*A, !work, false}, {*B, !work, false},
                        {list(a.targets, a.M, target_bytes(a.target_type)), a.loss == nullptr, false},
                        {list(a.loss, a.M, 4), true, true}, {list(a.lse, a.M, 4), !work, true},
                        {list(a.workspace, a.workspace_bytes, 1), true, true}};
    return check_matrices(uses, 6);
}

// Rows of a join's workgroup.  Up to a row per CU: one, whose pieces lie
// together (24 rows of 4096 pieces each: the call 185 us against 190 with the
// rows of a slot together, where a wave's reads go to 64 lines; 256 of 2048: 74
// against 79).  Else those whose pieces of a slot lie together, as many as leave a
// workgroup for every CU, or four pieces for every thread.
int join_rows(int64_t M, int64_t slots, int cus) {
    int rows = M <= cus ? 1 : 32;
    while (rows > 1 && ceil_div(M, rows) < cus && slots * rows > 4 * kLossJoinThreads) rows /= 2;
    return rows;
}

int run_forward(const gemm_cross_entropy_args& a, hipStream_t stream) {
    Matrix A, B;
    int st = check_forward(a, &A, &B);
    if (st != GEMM_OK || a.M == 0) return st;
    int cus = 0;
    st = current_cus(&cus);
    if (st != GEMM_OK) return st;
    const LossSizes s = sizes_of(a);
    ForwardPlan f;
    st = plan_forward(a, A, B, cus, &f);
    if (st != GEMM_OK) return st;
    if (!workspace_ok(f.workspace, a.workspace, a.workspace_bytes)) return GEMM_ERR_WORKSPACE;
    Space space{static_cast<char*>(a.workspace)};
    void* const a_space = space.take(f.a_bytes);
    void* const b_space = space.take(f.b_bytes);
    LossRowsProblem p{};
    p.pieces = static_cast<RowPiece*>(space.take(f.pieces_bytes));
    p.at_target = static_cast<float*>(space.take(f.target_bytes));
    p.targets.wide = a.target_type == GEMM_TARGET_I64;
    p.words = s.N;
    const Targets every{nullptr, 0};
    LossBegin jobs{};
    if (f.pack_a) {
        Matrix to = packed(A);
        to.data = a_space;
        jobs.pack[jobs.packs++] = pack_job(A, to, 1, every, 0);
        A = to;
    }
    // (a single piece of B is packed once)
    const bool one = f.piece >= s.N;
    Matrix packed_b{};
    for (int64_t row = 0; row < s.M; row += f.rows) {
        LossSizes block = s;
        block.M = std::min(f.rows, s.M - row);
        const int rows = join_rows(block.M, f.slots, cus);
        Matrix x = A;
        x.rows = block.M;
        x.data = static_cast<const char*>(A.data) + row * A.ld * 2;
        p.targets.at = a.loss ? static_cast<const char*>(a.targets) + row * target_bytes(a.target_type) : nullptr;
        for (int64_t first = 0; first < s.N; first += f.piece) {
            const int64_t words = std::min(f.piece, s.N - first);
            Matrix b = piece_of(B, s.b_transposed, first, words);
            if (f.pack_b && (row == 0 || !one)) {
                packed_b = packed(b);
                packed_b.data = b_space;
                jobs.pack[jobs.packs++] = pack_job(b, packed_b, 1, every, 0);
            }
            if (f.pack_b) b = packed_b;
            if ((st = begin(jobs, false, stream)) != GEMM_OK) return st;
            jobs.packs = 0;
            describe_logits(p, block, x, b, words);
            p.first = first;
            p.row_step = rows > 1 ? 1 : f.slots;
            p.slot_step = rows > 1 ? block.M : 1;
            if ((st = launch_logits(block, p, f.tile, cus, stream)) != GEMM_OK) return st;
        }
        st = launch(loss_join_kernel, dim3((unsigned)ceil_div(block.M, rows)), kLossJoinThreads, stream, p, f.slots, rows,
                    a.loss ? a.loss + row : nullptr, a.lse + row);
        if (st != GEMM_OK) return st;
    }
    return GEMM_OK;
}

// ---- gradients ----------------------------------------------------------------------------
// In the workspace: the rows' values, the scale and the lifts, A packed (always:
// rows without a target are zeros in it), in fp16 A's rows times their powers
// for dB, a piece of B packed, a piece's dZ, dA's sums over the pieces, and the
// slices of the product that runs.
struct GradPlan {
    bool pack_b, a_held;
    bool shifted;   // dZ's rows have powers of two of their own (fp16)
    int parts;      // dZ's: 2 for few tokens
    int64_t rows;   // of dZ: tokens times parts
    int64_t piece;
    LinearTile tile;
    Plan a, b;  // the gradients' products of a whole piece
    int64_t rows_bytes, a_bytes, shifted_bytes, b_bytes, slope_bytes, held_bytes, rest_bytes, workspace;
};
constexpr int64_t kLiftBytes = kMostLifts * 4;
// Words of a piece: dZ of 512 MiB, so that a piece is many rounds of tiles and
// dA's sums are read and written again a few times only, and for many tokens
// still 4096 words.  At a depth of 4096: 24 tokens by 131072 words 715 us in one
// piece, 800 to 1490 in pieces that the last-level cache would hold; 8192 tokens
// within 1 % from 8192 to 65536 words.  Contractions of less than some 320 are
// bound by dZ's bytes (6 for each token and word against 6 K operations), at
// any size of piece that is not held by that cache; others were not measured.
constexpr int64_t kSlopeValues = (int64_t)1 << 28, kLeastWords = 4096;
int64_t words_at_once(int64_t M) {
    return std::max(kSlopeValues / std::max<int64_t>(M, 1) / kPieceStep * kPieceStep, kLeastWords);
}

int parts_of(const LossSizes& s) { return s.M <= kSplitTokens ? 2 : 1; }
Plan plan_a(const LossSizes& s, int64_t words, int cus) {
    return choose(parts_of(s) * s.M, s.K, words, 1, kGroupNone, kDirect, s.variant, 0, cus);
}
Plan plan_b(const LossSizes& s, int64_t words, int cus) {
    const int64_t rows = parts_of(s) * s.M, R = s.b_transposed ? words : s.K, C = s.b_transposed ? s.K : words;
    return with_short(choose(R, C, rows, 1, kGroupNone, kDirect, s.variant, 0, cus), R, C, rows, kShortRows, s.variant, cus);
}
// Slices of a product, of all of it or of its last round.
int64_t rest_bytes(const Plan& plan, int64_t R, int64_t C, int64_t L, int cus) {
    return partial_bytes(plan, R, C) + tail_bytes(plan, R, C, L, 1, kGroupNone, cus);
}

int plan_grad(const gemm_cross_entropy_grad_args& a, const Matrix& A, const Matrix& B, int cus, GradPlan* plan) {
    const LossSizes s = sizes_of(a);
    GradPlan& g = *plan;
    g = GradPlan{};
    g.parts = parts_of(s);
    g.rows = g.parts * s.M;
    g.shifted = s.input_type == GEMM_INPUT_F16;
    g.pack_b = s.K > 0 && !whole_rows(B);
    g.piece = s.piece > 0 ? s.piece : words_at_once(s.M);
    if (s.piece == 0 && g.pack_b)  // (what is packed counts too, four times over: it is not used again)
        g.piece = std::min(g.piece, std::max(4 * kPackedPiece / s.K / kPieceStep, (int64_t)1) * kPieceStep);
    g.piece = std::min({g.piece, s.N, kMostWords});
    const Matrix b_piece = piece_of(B, s.b_transposed, 0, g.piece), b_read = g.pack_b ? packed(b_piece) : b_piece;
    Matrix a_read = packed(A);
    a_read.rows = g.rows;
    const Matrix slope{nullptr, g.rows, g.piece, round_up(g.piece, 8), 2};
    const bool kmajor = s.b_transposed != 0;
    if (!copies_fit(kTile256, a_read, true, b_read, kmajor) || !copies_fit(kTile256, slope, true, b_read, !kmajor) ||
        !copies_fit(kTile256, a_read, false, slope, false))
        return GEMM_ERR_TOO_LARGE;
    const Plan logits = logits_plan(s, g.piece, cus);
    g.a = plan_a(s, g.piece, cus);
    g.b = plan_b(s, g.piece, cus);
    if (!logits.found() || !g.a.found() || !g.b.found()) return GEMM_ERR_TOO_LARGE;
    g.tile = logits.tile;
    g.a_held = a.dA && (s.N > g.piece || g.parts > 1);
    g.rows_bytes = round_up(s.M * (int64_t)sizeof(LossRow), 256) + 256 + kLiftBytes;
    g.a_bytes = packed_bytes(g.shifted ? packed(A) : a_read);
    g.shifted_bytes = g.shifted && a.dB ? packed_bytes(a_read) : 0;
    g.b_bytes = g.pack_b ? packed_bytes(b_piece) : 0;
    g.slope_bytes = packed_bytes(slope);
    g.held_bytes = g.a_held ? round_up(g.rows * s.K * 4, 256) : 0;
    // (the last piece, which may be of another size, has a plan of its own)
    const int64_t last = s.N - (s.N - 1) / g.piece * g.piece;
    for (const int64_t words : {g.piece, last}) {
        if (a.dA) g.rest_bytes = std::max(g.rest_bytes, rest_bytes(plan_a(s, words, cus), g.rows, s.K, words, cus));
        if (a.dB) {
            const int64_t R = kmajor ? words : s.K, C = kmajor ? s.K : words;
            g.rest_bytes = std::max(g.rest_bytes, rest_bytes(plan_b(s, words, cus), R, C, g.rows, cus));
        }
    }
    g.workspace = g.rows_bytes + g.a_bytes + g.shifted_bytes + g.b_bytes + g.slope_bytes + g.held_bytes + g.rest_bytes;
    return GEMM_OK;
}

int check_grad(const gemm_cross_entropy_grad_args& a, Matrix* A, Matrix* B, Matrix* dB) {
    const int st = check_sizes(sizes_of(a));
    if (st != GEMM_OK) return st;
    if (!known_output(a.a_grad_type) || !known_output(a.b_grad_type)) return GEMM_ERR_UNSUPPORTED;
    if (a.workspace_bytes < 0) return GEMM_ERR_WORKSPACE;
    *A = Matrix{a.A, a.M, a.K, a.lda, 2};
    *B = words_matrix(a.B, a.b_transposed, a.N, a.K, a.ldb, 2);
    *dB = words_matrix(a.dB, a.b_transposed, a.N, a.K, a.lddb, elem_bytes(a.b_grad_type));
    const Matrix dA{a.dA, a.M, a.K, a.ldda, elem_bytes(a.a_grad_type)};
    const auto list = [](const void* p, int64_t n, int64_t elem) { return Matrix{p, 1, n, std::max<int64_t>(n, 1), elem}; };
    const bool work = a.dA || a.dB;
    const Use uses[] = {{*A, !work, false}, {*B, !work, false},
                        {list(a.targets, a.M, target_bytes(a.target_type)), !work, false},
                        {list(a.lse, a.M, 4), !work, false}, {list(a.dloss, a.M, 4), !work, false}, {dA, true, true},
                        {*dB, true, true}, {list(a.workspace, a.workspace_bytes, 1), true, true}};
    const int bad = check_matrices(uses, 8);
    if (bad != GEMM_OK) return bad;
    return out_pitch_ok(dA) && out_pitch_ok(*dB) ? GEMM_OK : GEMM_ERR_TOO_LARGE;
}

template <class Problem>
int launch_product(const LossSizes& s, Problem& p, const Plan& plan, void* rest, int cus, hipStream_t stream) {
    const TileSize size = loss_tile_size(plan.tile);
    const uint32_t m = (uint32_t)ceil_div(p.R, size.bm), n = (uint32_t)ceil_div(p.C, size.bn);
    p.groups = 1; p.axis = kGroupNone; p.splits = plan.splits; p.slice = plan.slice;
    p.partial = static_cast<float*>(rest);
    p.tail = tail_bytes(plan, p.R, p.C, p.L, 1, kGroupNone, cus) > 0 ? p.partial : nullptr;
    const uint32_t slices = (uint32_t)plan.splits;
    const bool k = s.b_transposed != 0;
    return status(s.input_type == GEMM_INPUT_BF16 ? launch_loss_bf16(p, k, plan.tile, m, n, slices, cus, stream)
                                                  : launch_loss_f16(p, k, plan.tile, m, n, slices, cus, stream));
}

int run_grad(const gemm_cross_entropy_grad_args& a, hipStream_t stream) {
    Matrix A, B, dB;
    int st = check_grad(a, &A, &B, &dB);
    if (st != GEMM_OK || (!a.dA && !a.dB) || a.K == 0 || (a.M == 0 && !a.dB)) return st;
    int cus = 0;
    st = current_cus(&cus);
    if (st != GEMM_OK) return st;
    const LossSizes s = sizes_of(a);
    GradPlan g;
    st = plan_grad(a, A, B, cus, &g);
    if (st != GEMM_OK) return st;
    if (!workspace_ok(g.workspace, a.workspace, a.workspace_bytes)) return GEMM_ERR_WORKSPACE;
    const bool kmajor = s.b_transposed != 0;
    const Targets targets{a.targets, a.target_type == GEMM_TARGET_I64};
    Space space{static_cast<char*>(a.workspace)};
    char* const rows = static_cast<char*>(space.take(g.rows_bytes));
    LossBack* const back = reinterpret_cast<LossBack*>(rows + g.rows_bytes - kLiftBytes - 256);
    int32_t* const lifts = reinterpret_cast<int32_t*>(rows + g.rows_bytes - kLiftBytes);
    const LossRow* const row = reinterpret_cast<const LossRow*>(rows);
    Matrix x = packed(A);
    x.data = space.take(g.a_bytes);
    Matrix by_tokens = x;  // what dB's sum over the tokens reads
    if (g.shifted) by_tokens.data = space.take(g.shifted_bytes);
    void* const b_space = space.take(g.b_bytes);
    void* const slopes = space.take(g.slope_bytes);
    float* const held = static_cast<float*>(space.take(g.held_bytes));
    void* const rest = space.take(g.rest_bytes);
    LossBegin jobs{};
    jobs.prepare = LossPrepare{s.M, s.N, targets, a.lse, a.dloss, reinterpret_cast<LossRow*>(rows), back, nullptr, 0, 0,
                               lifts};
    if (g.shifted) {
        jobs.prepare.A = static_cast<const uint16_t*>(A.data);
        jobs.prepare.lda = A.ld;
        jobs.prepare.width = s.K;
    }
    jobs.pack[jobs.packs++] = pack_job(A, x, g.shifted ? 1 : g.parts, targets, s.N);
    by_tokens.rows = g.rows;
    for (int64_t first = 0; first < s.N; first += g.piece) {
        const int64_t words = std::min(g.piece, s.N - first);
        Matrix b = piece_of(B, kmajor, first, words);
        if (g.pack_b) {
            Matrix to = packed(b);
            to.data = b_space;
            jobs.pack[jobs.packs++] = pack_job(b, to, 1, Targets{nullptr, 0}, 0);
            b = to;
        }
        if ((st = begin(jobs, first == 0, stream)) != GEMM_OK) return st;
        jobs.packs = 0;
        if (first == 0 && g.shifted && a.dB) {
            LossBegin shift{};
            LossPack& job = shift.pack[shift.packs++] = pack_job(A, by_tokens, g.parts, targets, s.N);
            job.row = row;
            job.lifts = lifts;
            job.count = s.M > 0 ? (int32_t)prepare_blocks(jobs.prepare) : 0;
            job.back = back;
            if ((st = begin(shift, false, stream)) != GEMM_OK) return st;
        }
        const Matrix z{slopes, g.rows, words, round_up(words, 8), 2};
        if (s.M > 0) {
            LossSlopeProblem p{};
            describe_logits(p, s, x, b, words);
            p.ep.out = slopes; p.ep.ldo = z.ld;
            p.row = row;
            p.first = first;
            p.rest = g.parts > 1 ? s.M * z.ld * 2 : 0;
            if ((st = launch_logits(s, p, g.tile, cus, stream)) != GEMM_OK) return st;
        }
        if (a.dB) {
            const Matrix out = piece_of(dB, kmajor, first, words);
            LossWordsGradProblem p{};
            const Matrix &left = kmajor ? z : by_tokens, &right = kmajor ? by_tokens : z;
            p.R = kmajor ? words : s.K; p.C = kmajor ? s.K : words; p.L = g.rows;
            p.A = static_cast<const uint16_t*>(left.data); p.lda = left.ld;
            p.B = static_cast<const uint16_t*>(right.data); p.ldb = right.ld;
            p.ep.out = const_cast<void*>(out.data); p.ep.ldo = out.ld; p.ep.out_f32 = a.b_grad_type == GEMM_OUTPUT_F32;
            p.back = back;
            st = launch_product(s, p, plan_b(s, words, cus), rest, cus, stream);
            if (st != GEMM_OK) return st;
        }
        if (a.dA && s.M > 0) {
            const bool last = first + words >= s.N && g.parts == 1;
            LossTokensGradProblem p{};
            p.R = g.rows; p.C = s.K; p.L = words;
            p.A = static_cast<const uint16_t*>(z.data); p.lda = z.ld;
            p.B = static_cast<const uint16_t*>(b.data); p.ldb = b.ld;
            p.before = first > 0 ? held : nullptr; p.before_ld = s.K;
            p.back = last ? back : nullptr;
            p.row = last && g.shifted ? row : nullptr;
            p.ep.out = last ? a.dA : held; p.ep.ldo = last ? a.ldda : s.K;
            p.ep.out_f32 = !last || a.a_grad_type == GEMM_OUTPUT_F32;
            st = launch_product(s, p, plan_a(s, words, cus), rest, cus, stream);
            if (st != GEMM_OK) return st;
        }
    }
    if (!a.dA || s.M == 0 || g.parts == 1) return GEMM_OK;
    const LossFold fold{s.M, s.K, held, back, row, a.dA, a.ldda, a.a_grad_type == GEMM_OUTPUT_F32};
    const dim3 blocks((unsigned)ceil_div(s.M * ceil_div(s.K, 8), 256));
    return s.input_type == GEMM_INPUT_BF16 ? launch(loss_fold_kernel<kInputBf16>, blocks, 256, stream, fold)
                                           : launch(loss_fold_kernel<kInputF16>, blocks, 256, stream, fold);
}

}  // namespace

// ---- exported C ABI ---------------------------------------------------------------------
extern "C" {

int gemm_cross_entropy(const gemm_cross_entropy_args* args, void* stream) {
    return args ? run_forward(*args, (hipStream_t)stream) : GEMM_ERR_NULL;
}

int64_t gemm_cross_entropy_workspace_bytes(const gemm_cross_entropy_args* args, int32_t num_cus) {
    if (!args) return GEMM_ERR_NULL;
    if (num_cus < 1) return GEMM_ERR_INVALID_DIM;
    gemm_cross_entropy_args a = *args;
    a.workspace = nullptr;
    a.workspace_bytes = 0;
    Matrix A, B;
    int st = check_forward(a, &A, &B);
    if (st != GEMM_OK || a.M == 0) return st;
    ForwardPlan f;
    st = plan_forward(a, A, B, num_cus, &f);
    return st != GEMM_OK ? st : f.workspace;
}

int gemm_cross_entropy_grad(const gemm_cross_entropy_grad_args* args, void* stream) {
    return args ? run_grad(*args, (hipStream_t)stream) : GEMM_ERR_NULL;
}

int64_t gemm_cross_entropy_grad_workspace_bytes(const gemm_cross_entropy_grad_args* args, int32_t num_cus) {
    if (!args) return GEMM_ERR_NULL;
    if (num_cus < 1) return GEMM_ERR_INVALID_DIM;
    gemm_cross_entropy_grad_args a = *args;
    a.workspace = nullptr;
    a.workspace_bytes = 0;
    Matrix A, B, dB;
    int st = check_grad(a, &A, &B, &dB);
    if (st != GEMM_OK || (!a.dA && !a.dB) || a.K == 0 || (a.M == 0 && !a.dB)) return st;
    GradPlan g;
    st = plan_grad(a, A, B, num_cus, &g);
    return st != GEMM_OK ? st : g.workspace;
}

}  // extern "C"
