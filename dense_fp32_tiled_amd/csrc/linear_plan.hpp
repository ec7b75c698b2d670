// linear_plan.hpp -- how a product of the tile kernel is run: its tile, its
// slices of the contraction, the operands that are packed first, and the
// workspace they take.
#pragma once

#include <algorithm>
#include <cmath>

#include "host_checks.hpp"
#include "linear_shapes.hpp"

namespace dft {

// ---- the choice of tile and slices ----------------------------------------------------
constexpr double kNoPlan = 1e300;
struct Plan {
    LinearTile tile;
    bool direct;
    int splits;
    int64_t slice;
    double us;  // as estimated

    bool found() const { return us < kNoPlan; }
};

// Times of the tiles in microseconds, fitted to 10000 forward products of
// every tile and slicing, of 1 to 16384 rows by 64 to 8192 columns and 64 to
// 8192 deep, one matrix or up to 32 groups: `once` for the launch, and for a
// round of workgroups `fixed` and, per contraction tile, `alone` with one
// workgroup per CU and `full` with every place taken.  Over those products the
// choice takes 1.4 % more than the best on average (a fit to products of 1024
// columns and depth and more took 6.4 %, most of it on short contractions).
// The register path's, and packing's time, were fitted to 7000 products of odd
// widths run both ways: 2.4 % more than the best on average (11 % before).
struct TileTime {
    int per_cu;
    double once, fixed, alone, full;
};
constexpr TileTime kDirectTimes[kTileCount] = {
    {1, 3.3, 15.3, 0.98, 1.57}, {2, 4.3, 6.7, 0.69, 1.21}, {2, 4.3, 3.1, 0.24, 0.54}, {2, 4.3, 3.3, 0.24, 0.56}};
constexpr TileTime kRegisterTimes[kTileCount] = {
    {1, 0, 0, 0, 0}, {2, 11.6, 0, 2.2, 3.0}, {2, 5.3, 1.5, 1.13, 0.77}, {2, 5.7, 1.2, 1.45, 0.99}};

// How a product reads its operands, and the register path's time per
// contraction tile by which of the two are of odd widths.
struct Path {
    bool direct;
    double slow;
};
constexpr int kMaxSlices = 32;

// Estimated microseconds of a plan: its launch, its rounds (the last one by
// how much of the chip it takes) and its operands' bytes at 4.2 TB/s (2.2
// through registers), the larger of the two counting most (fourth powers), and
// the slices' join.
inline double estimate(int64_t R, int64_t C, int64_t L, int64_t groups, int axis, LinearTile t, Path path, int splits,
                int cus) {
    TileTime time = (path.direct ? kDirectTimes : kRegisterTimes)[t];
    if (time.alone <= 0) return 1e30;
    time.alone *= path.slow;
    time.full *= path.slow;
    const TileSize size = kTileSizes[t];
    double row_tiles = (double)ceil_div(R, size.bm), length = (double)L, copies = 1;
    if (axis == kGroupRows) {
        // half a tile more on average for every group that has rows, and two standard deviations of their sum: a
        // round begun costs more than one left out saves
        copies = (double)std::min<int64_t>(groups, R);
        row_tiles = std::max((double)R / size.bm + 0.5 * copies + 0.6 * std::sqrt(copies), copies);
    }
    double tiles = row_tiles * (double)ceil_div(C, size.bn) * splits;
    if (axis == kGroupContraction) {
        tiles *= (double)groups;
        length = (double)L / (double)groups;
    }
    const double slots = (double)cus * time.per_cu;
    const double depth = (double)ceil_div((int64_t)(length / splits + 0.999), kTileDepth);
    const double whole = (double)(int64_t)(tiles / slots), left = tiles / slots - whole;  // rounds
    double us = whole * (time.fixed + depth * time.full);
    if (left > 0) {
        // from `alone` while there is at most one workgroup per CU (one-per-CU tiles: by the share of CUs) to `full`
        const double busy = time.per_cu == 1 ? left : std::max(0.0, left * time.per_cu - 1) / (time.per_cu - 1);
        const double last = time.fixed + depth * (time.alone + busy * (time.full - time.alone));
        const bool tail = t == kTile256 && path.direct && axis != kGroupContraction && splits == 1 && whole > 0 &&
                          depth >= kTailDepth && left <= 0.5;
        us += tail ? std::min(last, time.fixed + depth * time.full * left + 30) : last;
    }
    const double bytes = 2.0 * ((double)R * (double)L + copies * (double)L * (double)C) +
                         2.0 * (double)R * (double)C * (axis == kGroupContraction ? (double)groups : 1.0);
    const double memory = bytes / (path.direct ? 4.2e6 : 2.2e6), u2 = us * us, m2 = memory * memory;
    us = time.once + std::sqrt(std::sqrt(u2 * u2 + m2 * m2));
    if (splits > 1) us += 2.1 + (splits + 1.0) * (double)R * (double)C * 4.0 / 4.4e6;
    return us;
}

// Row tiles enough for any division of R rows into groups, R of which have
// rows at most (places that no tile takes are not only launched: they leave
// the real tiles to fewer XCDs.  Counted for all groups, 1 row of 32 experts
// of 4096x4096 took 48.7 us, 8 rows 105; so 19.6 and 44.8).
inline int64_t row_tiles(int64_t R, int64_t groups, int axis, int64_t bm) {
    if (axis != kGroupRows) return ceil_div(R, bm);
    return (R + std::min(groups, R) * (bm - 1)) / bm;
}

// Whether a launch holds the tiles (it has fewer than 2^31 threads, of tiles
// with 512 each).
constexpr int64_t kMaxTiles = kMaxGrid / 512;
inline bool grid_fits(int64_t R, int64_t C, int64_t groups, int axis, LinearTile tile, int splits) {
    const TileSize size = kTileSizes[tile];
    const int64_t tiles_m = row_tiles(R, groups, axis, size.bm), tiles_n = ceil_div(C, size.bn);
    return tiles_n == 0 || tiles_m <= kMaxTiles / tiles_n / (axis == kGroupContraction ? groups : splits);
}

// The quickest of the plans that a launch holds; none of them: not found().
inline Plan choose(int64_t R, int64_t C, int64_t L, int64_t groups, int axis, Path path, int variant, int splits, int cus) {
    Plan best{kTile128, path.direct, 1, L, kNoPlan};
    for (int t = 0; t < kTileCount; ++t) {
        if (variant != GEMM_LINEAR_AUTO && t != variant - 1) continue;
        LinearTile tile = (LinearTile)t;
        if (tile == kTile256 && !path.direct) {
            if (variant == GEMM_LINEAR_AUTO) continue;
            tile = kTile128;
        }
        for (int s = 1; s <= kMaxSlices; s *= 2) {
            int use = splits > 0 ? splits : s;
            if (axis != kGroupNone || L == 0) use = 1;
            // slices of whole tiles, none of them empty, at least four deep unless asked for
            const int64_t slice = ceil_div(ceil_div(L, kTileDepth), use) * kTileDepth;
            if (use > 1) {
                if (splits == 0 && slice < 4 * kTileDepth) break;
                use = (int)ceil_div(L, slice);
            }
            if (!grid_fits(R, C, groups, axis, tile, std::max(use, 1))) break;
            double us = estimate(R, C, L, groups, axis, tile, path, use, cus);
            // at equal times the tile whose rows are used, and fewer slices
            if (tile == kTile32x128 && R > 32 * groups) us += 0.3;
            if (us < best.us - 0.2) best = Plan{tile, path.direct, std::max(use, 1), slice, us};
            if (splits > 0 || axis != kGroupNone || L == 0) break;
        }
    }
    return best;
}

inline int64_t partial_bytes(const Plan& plan, int64_t R, int64_t C) { return plan.splits > 1 ? plan.splits * R * C * 4 : 0; }

// The blocks for the slices of a last round (tail_split): one per workgroup
// of a persistent grid, where it has whole rounds before it.
inline int64_t tail_bytes(const Plan& plan, int64_t R, int64_t C, int64_t L, int64_t groups, int axis, int cus) {
    if (plan.tile != kTile256 || !plan.direct || plan.splits > 1 || axis == kGroupContraction) return 0;
    if (ceil_div(L, kTileDepth) < kTailDepth) return 0;
    const int64_t most = row_tiles(R, groups, axis, 256) * ceil_div(C, 256);
    if (most <= cus) return 0;
    if (axis == kGroupNone && (most % cus == 0 || cus / (most % cus) < 2)) return 0;
    return (int64_t)cus * 256 * 256 * 4;
}

// ---- operands ---------------------------------------------------------------------------
inline bool copies_fit(LinearTile tile, const Matrix& a, bool a_kmajor, const Matrix& b, bool b_kmajor) {
    // OperandCopy's offsets: within a tile, k-major within the whole contraction, they stay below 2^30
    const TileSize size = kTileSizes[tile];
    const auto fits = [](int64_t ld, int64_t rows, int64_t cols) { return ld <= 0x3fffffff / (2 * rows) - cols; };
    return fits(a.ld, a_kmajor ? size.bm : kTileDepth, a_kmajor ? kTileDepth : size.bm) &&
           fits(b.ld, b_kmajor ? size.bn : kTileDepth, b_kmajor ? kTileDepth : size.bn);
}

// 16-byte copies of both operands: rows and widths in whole 16 bytes, and
// offsets inside a tile that fit whatever tile is chosen.
inline bool direct_ok(const Matrix& a, bool a_kmajor, const Matrix& b, bool b_kmajor) {
    return a.aligned16() && b.aligned16() && a.cols % 8 == 0 && b.cols % 8 == 0 &&
           copies_fit(kTile256, a, a_kmajor, b, b_kmajor);
}

// An operand as the products read it: itself, or packed to rows of whole 16
// bytes in the workspace.
inline bool whole_rows(const Matrix& m) { return m.aligned16() && m.cols % 8 == 0; }
inline Matrix packed(const Matrix& m) {
    Matrix r = m;
    r.ld = ceil_div(std::max<int64_t>(m.cols, 1), 8) * 8;
    r.copy_stride = m.rows * r.ld;
    r.data = nullptr;  // (placed when the workspace is known)
    return r;
}
inline int64_t packed_bytes(const Matrix& m) { return ceil_div(2 * m.copies * m.rows * packed(m).ld, 256) * 256; }
// Reading and writing every element once at 5.3 TB/s, beside the launch.
constexpr double kPackLaunch = 3.5;
inline double pack_us(const Matrix& m) { return 2.0 * (double)packed_bytes(m) / 5.3e6; }

constexpr Path kDirect{true, 1};
inline Path path_of(const Matrix& a, bool a_kmajor, const Matrix& b, bool b_kmajor) {
    if (direct_ok(a, a_kmajor, b, b_kmajor)) return kDirect;
    const bool whole_a = whole_rows(a), whole_b = whole_rows(b);
    return Path{false, whole_a == whole_b ? 1.0 : whole_b ? 0.55 : 0.94};
}

// Workspace cut into 256-byte pieces from its start.
struct Space {
    char* at;
    void* take(int64_t bytes) {
        void* p = at;
        at += ceil_div(bytes, 256) * 256;
        return p;
    }
};

inline bool workspace_ok(int64_t need, const void* workspace, int64_t bytes) {
    return need == 0 || (workspace && bytes >= need && ((uintptr_t)workspace & 15) == 0);
}

}  // namespace dft
