// linear_kernels.hpp -- gfx950 kernels of the products with an epilogue
// (gemm_linear) and of their gradients (gemm_linear_grad), for one matrix or
// for one matrix per group of rows.
//
//   forward    D[M,N]  = act(A[M,K] B[K,N] + bias) + residual
//   gradients  dA[M,K] = dZ[M,N] B^T,  dB[K,N] = A^T dZ,  dbias = sum of dZ over M
//
// All three products run in one kernel, linear_tile_kernel: an operand whose
// rows run along the contraction ("k-major": A forward, dZ and B for dA) is
// read from LDS 16 bytes per lane; one whose rows run along the output
// (B forward, A and dZ for dB) through the transposing 8-byte reads, so no
// operand is ever transposed in memory.  Products of 16-bit values are exact
// in fp32 and sums are held in fp32; nothing is rounded before the epilogue.
#pragma once

#include "mixed_kernels.hpp"

namespace dft {

// ---- the problem a launch works on --------------------------------------------------
enum LinearAct { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4, kActCount = 5 };

// How `offsets` divides a product: nothing (one matrix), the output rows (one
// B per group), or the contraction (one output per group).
enum GroupAxis { kGroupNone = 0, kGroupRows = 1, kGroupContraction = 2 };

struct LinearEpilogue {
    const uint16_t* bias;        // nullptr: none; group g's at bias + g * bias_group
    int64_t bias_group;
    const void* residual;        // of the output's type, or nullptr
    int64_t ldr;
    uint16_t* preact;            // A B + bias in the inputs' type, or nullptr
    int64_t ldp;
    void* out;
    int64_t ldo;
    int64_t out_group;           // contraction groups: elements between outputs
    int32_t act;
    int32_t out_f32;
};

struct LinearProblem {
    int64_t R, C, L;             // output rows, output columns, contraction length
    const uint16_t* A;           // k-major: R x L; else L x R
    int64_t lda;
    const uint16_t* B;           // k-major: C x L; else L x C; group g's at B + g * b_group (row groups)
    int64_t ldb, b_group;
    const int32_t* offsets;      // groups + 1 row offsets on the device (nullptr: one matrix)
    int32_t groups;
    int32_t axis;                // GroupAxis
    int32_t splits;              // slices of the contraction along gridDim.y (one matrix only)
    int64_t slice;               // contraction elements per slice, a multiple of the tile's
    float* partial;              // splits > 1: packed R x C partial products
    LinearEpilogue ep;
};

// ---- activations --------------------------------------------------------------------
__device__ inline float act_value(float z, int kind) {
    switch (kind) {
        case kActRelu: return z > 0.0f ? z : 0.0f;
        case kActGelu: return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
        // (1 + tanh(u)) / 2 is the logistic function of 2 u
        case kActGeluTanh: return z / (1.0f + expf(-1.5957691216057308f * (z + 0.044715f * z * z * z)));
        case kActSilu: return z / (1.0f + expf(-z));
        default: return z;
    }
}
// The slope at z.  Beyond |z| = 128 every slope has reached its limit in
// fp32; stopping there keeps 0 * infinity out of the products (a NaN z stays).
__device__ inline float act_slope(float z, int kind) {
    if (kind == kActNone) return 1.0f;
    if (kind == kActRelu) return z > 0.0f ? 1.0f : 0.0f;
    z = z > 128.0f ? 128.0f : z < -128.0f ? -128.0f : z;
    if (kind == kActGelu)
        return 0.5f * (1.0f + erff(z * 0.70710678118654752f)) + z * 0.39894228040143268f * expf(-0.5f * z * z);
    float u = z, du = 1.0f;
    if (kind == kActGeluTanh) {
        u = 1.5957691216057308f * (z + 0.044715f * z * z * z);
        du = 1.5957691216057308f * (1.0f + 0.134145f * z * z);
    }
    const float gate = 1.0f / (1.0f + expf(-u));
    return gate + z * gate * (1.0f - gate) * du;
}

// ---- 16-bit values ------------------------------------------------------------------
template <int TYPE>
__device__ inline float widen(uint16_t v) {
    if constexpr (TYPE == kInputBf16)
        return __builtin_bit_cast(float, (uint32_t)v << 16);
    else
        return (float)__builtin_bit_cast(_Float16, v);
}
// Rounds to nearest, ties to even.
template <int TYPE>
__device__ inline uint16_t narrow(float v) {
    if constexpr (TYPE == kInputBf16)
        return __builtin_bit_cast(uint16_t, (__bf16)v);
    else
        return __builtin_bit_cast(uint16_t, (_Float16)v);
}

// Eight consecutive 16-bit values, at any 2-byte alignment: one 16-byte
// access when all are in range, else one access each.
struct Row8 {
    uint16_t v[8];
};
__device__ inline Row8 load8(const uint16_t* p, int64_t in_range) {
    Row8 r;
    if (in_range >= 8) {
        __builtin_memcpy(&r, p, sizeof(r));
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) r.v[e] = e < in_range ? p[e] : (uint16_t)0;
    }
    return r;
}
__device__ inline void store8(uint16_t* p, const Row8& r, int64_t in_range) {
    if (in_range >= 8) {
        __builtin_memcpy(p, &r, sizeof(r));
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < in_range) p[e] = r.v[e];
    }
}
__device__ inline void load8(float (&v)[8], const float* p, int64_t in_range) {
    if (in_range >= 8) {
        __builtin_memcpy(&v, p, sizeof(v));
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = e < in_range ? p[e] : 0.0f;
    }
}
__device__ inline void store8(float* p, const float (&v)[8], int64_t in_range) {
    if (in_range >= 8) {
        __builtin_memcpy(p, &v, sizeof(v));
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < in_range) p[e] = v[e];
    }
}

// The epilogue of eight consecutive columns of one output row: z holds their
// sums; `left` of them lie inside the matrix.
template <int TYPE>
__device__ inline void epilogue8(const LinearEpilogue& ep, int64_t group, int64_t row, int64_t col, int64_t left,
                                 float (&z)[8]) {
    if (ep.bias) {
        const Row8 b = load8(ep.bias + group * ep.bias_group + col, left);
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] += widen<TYPE>(b.v[e]);
    }
    if (ep.preact) {
        Row8 r;
#pragma unroll
        for (int e = 0; e < 8; ++e) r.v[e] = narrow<TYPE>(z[e]);
        store8(ep.preact + row * ep.ldp + col, r, left);
    }
    if (ep.act != kActNone) {
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] = act_value(z[e], ep.act);
    }
    const int64_t at = row * ep.ldo + col + (group * ep.out_group);
    if (ep.out_f32) {
        if (ep.residual) {
            float r[8];
            load8(r, static_cast<const float*>(ep.residual) + row * ep.ldr + col, left);
#pragma unroll
            for (int e = 0; e < 8; ++e) z[e] += r[e];
        }
        store8(static_cast<float*>(ep.out) + at, z, left);
    } else {
        Row8 o;
        if (ep.residual) {
            const Row8 r = load8(static_cast<const uint16_t*>(ep.residual) + row * ep.ldr + col, left);
#pragma unroll
            for (int e = 0; e < 8; ++e) z[e] += widen<TYPE>(r.v[e]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) o.v[e] = narrow<TYPE>(z[e]);
        store8(static_cast<uint16_t*>(ep.out) + at, o, left);
    }
}

// ---- groups of rows -----------------------------------------------------------------
// Group g's rows [lo, hi): offsets outside [0, rows] or not ascending are
// taken as the nearest range inside, so that no access leaves the matrices.
struct RowRange {
    int64_t lo, hi;
};
__device__ inline RowRange group_rows(const int32_t* offsets, int g, int64_t rows) {
    const int64_t a = offsets[g], b = offsets[g + 1];
    const int64_t lo = a < 0 ? 0 : a > rows ? rows : a;
    const int64_t hi = b < lo ? lo : b > rows ? rows : b;
    return RowRange{lo, hi};
}

// The tile-th tile of `tile_rows` rows when every group's rows are tiled from
// the group's own start; group < 0: there is no such tile.  Every wave looks
// it up itself: 64 groups at a time, one per lane.
struct GroupTile {
    int group;
    int64_t row0, row_end;
    int64_t first;  // first tile of that group
};
__device__ inline GroupTile find_group_tile(const int32_t* offsets, int groups, int64_t rows, int tile_rows,
                                            int64_t tile) {
    const int lane = threadIdx.x % kWave;
    int64_t before = 0;
    for (int g0 = 0; g0 < groups; g0 += kWave) {
        const int g = g0 + lane;
        RowRange r{0, 0};
        if (g < groups) r = group_rows(offsets, g, rows);
        const int own = (int)((r.hi - r.lo + tile_rows - 1) / tile_rows);
        int upto = own;  // inclusive running sum over the lanes
#pragma unroll
        for (int d = 1; d < kWave; d *= 2) {
            const int other = __shfl_up(upto, d);
            if (lane >= d) upto += other;
        }
        const bool here = tile >= before + upto - own && tile < before + upto;
        const uint64_t found = __ballot(here);
        if (found) {
            const int l = __builtin_ctzll(found);
            const int64_t first = before + __shfl(upto - own, l);
            const int64_t lo = __shfl((int)r.lo, l), hi = __shfl((int)r.hi, l);
            return GroupTile{g0 + l, lo + (tile - first) * tile_rows, hi, first};
        }
        before += __shfl(upto, kWave - 1);
    }
    return GroupTile{-1, 0, 0, 0};
}

// Orders a wave's own LDS accesses before it and after it: its lanes exchange
// values through LDS without a workgroup barrier.
__device__ inline void wave_fence() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }

// ---- operand tiles ------------------------------------------------------------------
// One operand's tile of OUT output rows (or columns) by DEPTH contraction
// elements, in 4-byte words.  K-major: OUT rows of DEPTH elements, 16-byte
// groups swizzled by (row >> 1) & 7.  Else DEPTH rows of OUT elements, 64-byte
// groups swizzled by the row so that the four rows of a transposing read fall
// on four different quarters of the banks (rows of 64 elements: two rows span
// the banks, so the row's second bit decides; rows of 32: four rows do).
template <bool KMAJOR, int OUT, int DEPTH, int STAGES>
struct OperandTile {
    static_assert(DEPTH == 64 && OUT % 32 == 0, "rows of 128 bytes, k-major");
    static constexpr int unit = KMAJOR ? 4 : OUT >= 64 ? 16 : 0;
    static constexpr int shift = KMAJOR ? 1 : OUT == 64 ? 1 : 0;
    static constexpr int mask = KMAJOR ? 7 : OUT >= 128 ? 3 : OUT == 64 ? 1 : 0;
    using Tile = LdsTile<KMAJOR ? OUT : DEPTH, (KMAJOR ? DEPTH : OUT) / 2, 0, STAGES, unit, shift, mask>;
    static constexpr int row_groups = Tile::cols / 4;  // 16-byte groups per row
};

// One direct global->LDS copy: each lane 16 bytes from byte `offset` of the
// buffer, to LDS byte address lds + 16 * lane.  The buffer's range check
// writes zeros for a lane whose offset is beyond its last byte, which is all
// the masking that whole 16-byte groups need.  A statement of its own, as in
// copy16_to_lds, so that the compiler does not wait for it before LDS reads;
// completion is waited for with wait_vector_memory_at_most.
__device__ inline void copy16_checked(const u32x4& buffer, uint32_t offset, uint32_t lds) {
    asm volatile(
        "s_mov_b32 m0, %2\n\t"
        "s_nop 0\n\t"
        "buffer_load_dwordx4 %0, %1, 0 offen lds"
        :
        : "v"(offset), "s"(buffer), "s"(lds)
        : "memory", "m0");
}

constexpr uint32_t kBeyond = 0x80000000u;  // past every buffer's last byte (buffers stop at 2^31 - 1)

// The copies of one operand's tiles, 16 bytes per lane.  A wave's copies of a
// tile are WAVES pieces of 1 KiB apart, which is a whole number of swizzle
// periods, so one offset per lane and a constant step describe them all.
template <bool KMAJOR, int OUT, int DEPTH, int STAGES, int THREADS>
struct OperandCopy {
    using OT = OperandTile<KMAJOR, OUT, DEPTH, STAGES>;
    using Tile = typename OT::Tile;
    static constexpr int WAVES = THREADS / kWave;
    static constexpr int PIECE_ROWS = kWave / OT::row_groups;
    static constexpr int PER_WAVE = Tile::stage_elems * 4 / 1024 / WAVES;
    static_assert(PER_WAVE * WAVES * 1024 == Tile::stage_elems * 4, "whole pieces per wave");
    static_assert((WAVES * PIECE_ROWS) % ((OT::mask + 1) << OT::shift) == 0, "whole swizzle periods per step");

    const char* base;      // first byte of contraction tile 0 (uniform)
    const char* end;       // past the last byte of the operand's rows (uniform)
    int64_t tile_bytes;    // between contraction tiles
    uint32_t offset;       // this lane's first copy
    uint32_t step;         // between its copies of one tile
    uint32_t depth;        // k-major: contraction index of the lane's 16 bytes within a tile
    uint32_t lds_piece;

    // `origin`: the element at contraction index 0 and the tile's first output row (column); `outs`: output rows
    // (columns) from there; `left`: contraction elements.
    __device__ OperandCopy(const uint16_t* origin, int64_t ld, int64_t outs, int64_t left, int wave, int lane) {
        base = reinterpret_cast<const char*>(origin);
        const int64_t rows = KMAJOR ? outs : left, cols = KMAJOR ? left : outs;
        end = rows > 0 && cols > 0 ? base + 2 * ((rows - 1) * ld + cols) : base;
        tile_bytes = KMAJOR ? 2 * DEPTH : 2 * DEPTH * ld;
        const int row = wave * PIECE_ROWS + lane / OT::row_groups;
        const int word = Swizzle{OT::unit, OT::shift, OT::mask}.apply(row, lane % OT::row_groups * 4);
        offset = (uint32_t)(2 * row * ld) + 4 * word;
        depth = KMAJOR ? 2 * word : 0;
        if (!KMAJOR && 2 * word >= outs) offset = kBeyond;
        step = (uint32_t)(2 * WAVES * PIECE_ROWS * ld);
        lds_piece = wave * 1024;
    }
    // Offsets within a tile stay below 2^31.
    __host__ __device__ static constexpr bool fits(int64_t ld) {
        return ld <= (((int64_t)1 << 31) - 1) / (2 * Tile::rows) - 2 * Tile::cols;
    }
    // Copies of contraction tile t into `stage`; `left`: contraction elements from that tile's first on (a tile
    // past the end fills the stage with zeros).
    __device__ void issue(int64_t t, int64_t left, uint32_t* lds, int stage) const {
        typedef __attribute__((address_space(3))) uint32_t lds_word;
        const char* tile = base + t * tile_bytes;
        int64_t bytes = end - tile;
        bytes = left <= 0 || bytes < 0 ? 0 : bytes > 0x7fffffff ? 0x7fffffff : bytes;
        const uint64_t b = (uint64_t)(uintptr_t)tile;
        const u32x4 buffer{first_lane((uint32_t)b), first_lane((uint32_t)(b >> 32) & 0xffffu),
                           first_lane((uint32_t)bytes), 0x00020000u};
        const uint32_t to = first_lane((uint32_t)(uintptr_t)(lds_word*)lds + stage * (Tile::stage_elems * 4) + lds_piece);
        const uint32_t from = KMAJOR && (int64_t)depth >= left ? kBeyond : offset;
#pragma unroll
        for (int i = 0; i < PER_WAVE; ++i) copy16_checked(buffer, from + i * step, to + i * (WAVES * 1024));
    }
};

// The same tiles through registers, for operands whose rows or widths are
// not multiples of 16 bytes: 16-byte loads at any 2-byte alignment where a
// whole group is in range, masked elements at the edges.
template <bool KMAJOR, int OUT, int DEPTH, int STAGES, int THREADS>
struct OperandLoad {
    using OT = OperandTile<KMAJOR, OUT, DEPTH, STAGES>;
    using Tile = typename OT::Tile;
    static constexpr int GROUPS = Tile::rows * OT::row_groups;
    static constexpr int PER_THREAD = GROUPS / THREADS;
    static_assert(GROUPS % THREADS == 0, "whole groups per thread");

    const uint16_t* origin;
    int64_t ld, outs;
    Row8 held[PER_THREAD];

    __device__ OperandLoad(const uint16_t* origin_, int64_t ld_, int64_t outs_) : origin(origin_), ld(ld_), outs(outs_) {}
    __device__ void load(int64_t t, int64_t left, int tid) {
        const uint16_t* tile = origin + t * (KMAJOR ? (int64_t)DEPTH : DEPTH * ld);
        const int64_t rows = KMAJOR ? outs : left, cols = KMAJOR ? left : outs;
#pragma unroll
        for (int i = 0; i < PER_THREAD; ++i) {
            const int at = tid + i * THREADS, row = at / OT::row_groups, col = at % OT::row_groups * 8;
            held[i] = load8(tile + row * ld + col, row < rows ? cols - col : 0);
        }
    }
    __device__ void store(uint32_t* lds, int stage, int tid) const {
#pragma unroll
        for (int i = 0; i < PER_THREAD; ++i) {
            const int at = tid + i * THREADS, row = at / OT::row_groups, col = at % OT::row_groups * 8;
            *reinterpret_cast<u32x4*>(lds + Tile::offset(stage, row, col / 2)) = __builtin_bit_cast(u32x4, held[i]);
        }
    }
};

// A wave's fragments of one operand: block i (32 output rows or columns) of
// MFMA step st, 8 contraction elements per lane.
template <class OT, bool KMAJOR, int BLOCKS>
struct OperandRead {
    using Tile = typename OT::Tile;
    int at[KMAJOR ? 4 : BLOCKS];  // k-major: by step; else by block

    __device__ OperandRead(int out0, int lane) {
        if constexpr (KMAJOR) {
#pragma unroll
            for (int st = 0; st < 4; ++st) at[st] = Tile::offset(0, out0 + lane % 32, st * 8 + 4 * (lane / 32));
        } else {
            const int row = 8 * (lane / 32) + (lane % 16) / 4, col = 16 * ((lane / 16) % 2) + 4 * (lane % 4);
#pragma unroll
            for (int i = 0; i < BLOCKS; ++i) at[i] = Tile::offset(0, row, (out0 + i * 32 + col) / 2);
        }
    }
    __device__ u32x4 read(const uint32_t* lds, int stage, int st, int i) const {
        if constexpr (KMAJOR) {
            return *reinterpret_cast<const u32x4*>(lds + stage * Tile::stage_elems + at[st] + i * 32 * Tile::row_stride);
        } else {
            typedef __attribute__((address_space(3))) const uint32_t lds_word;
            typedef __attribute__((address_space(3))) shortx4 lds_short4;
            u32x2 half[2];
#pragma unroll
            for (int rr = 0; rr < 2; ++rr) {
                const int word = stage * Tile::stage_elems + at[i] + (st * 16 + 4 * rr) * Tile::row_stride;
                half[rr] = __builtin_bit_cast(u32x2,
                                              __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4*)((lds_word*)lds + word)));
            }
            return u32x4{half[0][0], half[0][1], half[1][0], half[1][1]};
        }
    }
};

// ---- the product --------------------------------------------------------------------
template <int BM_, int BN_, int WM_, int WN_, int STAGES_, int MIN_WAVES_>
struct LinearShape {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, STAGES = STAGES_, MIN_WAVES = MIN_WAVES_;
    static constexpr int BK = 64;
    static constexpr int WAVES_N = BN / WN, THREADS = BM / WM * WAVES_N * kWave;
    static constexpr int MI = WM / 32, NI = WN / 32;
};

// Consecutive tiles on one XCD (workgroups go to the eight XCDs in turn), in
// panels of eight tile rows, so that the tiles an XCD works on at one time
// share their operands' rows and columns in its L2.
struct TilePlace {
    int64_t row, col;
};
__device__ inline TilePlace place_of_block(uint32_t block, uint32_t blocks, uint32_t tiles_m, uint32_t tiles_n) {
    const uint32_t xcd = block % 8, each = blocks / 8, more = blocks % 8;
    const uint32_t id = xcd * each + (xcd < more ? xcd : more) + block / 8;
    const uint32_t panel = 8 * tiles_n, p = id / panel, in = id % panel;
    const uint32_t high = tiles_m - 8 * p < 8 ? tiles_m - 8 * p : 8;
    return TilePlace{8 * p + in % high, in / high};
}

// One workgroup per BM x BN output tile (and slice of the contraction, and
// group).  S LDS stages: during the multiply of contraction tile t the copies
// of tiles t+1 .. t+S-1 are in flight; one barrier per tile.  The fragments of
// an MFMA step are read during the MFMAs of the step before, the first of a
// tile during the last step of the tile before it, after the barrier.
// The MFMAs take B as their row operand, so a lane's four consecutive results
// are four consecutive columns of one output row; each wave passes its
// results through LDS, 32 rows at a time, to give every lane eight columns of
// a row and the epilogue's loads and stores 16 bytes per lane.
template <int TYPE, bool AK, bool BK_, class Shape, bool DIRECT>
__global__ __launch_bounds__(Shape::THREADS, Shape::MIN_WAVES) void linear_tile_kernel(LinearProblem p, uint32_t tiles_m,
                                                                                   uint32_t tiles_n) {
    using Op = Mfma16Op<TYPE, 32>;
    constexpr int BM = Shape::BM, BN = Shape::BN, BK = Shape::BK, S = DIRECT ? Shape::STAGES : 2;
    constexpr int MI = Shape::MI, NI = Shape::NI, THREADS = Shape::THREADS;
    using OA = OperandTile<AK, BM, BK, S>;
    using OB = OperandTile<BK_, BN, BK, S>;
    using TileA = typename OA::Tile;
    using TileB = typename OB::Tile;
    constexpr int STAGE_ROW = Shape::WN + 4;  // words per staged output row
    constexpr int STAGE_WORDS = 32 * STAGE_ROW;
    constexpr int WORDS = TileA::total_elems + TileB::total_elems;
    static_assert(THREADS / kWave * STAGE_WORDS <= WORDS, "the staged rows fit the operand stages");

    __shared__ __attribute__((aligned(16))) uint32_t lds[WORDS];
    poison_lds(lds, WORDS);
    uint32_t* const lds_a = lds;
    uint32_t* const lds_b = lds + TileA::total_elems;

    const int tid = threadIdx.x, lane = tid % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int wm0 = wave / Shape::WAVES_N * Shape::WM, wn0 = wave % Shape::WAVES_N * Shape::WN;

    // This workgroup's tile: rows [m0, m_end) of the output, columns from n0, contraction [l0, l0 + L).
    const TilePlace place = place_of_block(blockIdx.x, gridDim.x, tiles_m, tiles_n);
    int64_t m0 = place.row * BM, m_end = p.R, n0 = place.col * BN, group = 0, L = p.L;
    const uint16_t* A = p.A;
    const uint16_t* B = p.B;
    float* partial = nullptr;
    if (p.axis == kGroupRows) {
        const GroupTile gt = find_group_tile(p.offsets, p.groups, p.R, BM, place.row);
        if (gt.group < 0) return;
        group = gt.group;
        m0 = gt.row0;
        m_end = gt.row_end;
        B += group * p.b_group;
    } else if (p.axis == kGroupContraction) {
        group = blockIdx.y;
        const RowRange r = group_rows(p.offsets, (int)group, p.L);
        A += r.lo * p.lda;
        B += r.lo * p.ldb;
        L = r.hi - r.lo;
    } else if (p.splits > 1) {
        const int64_t l0 = blockIdx.y * p.slice;
        A += AK ? l0 : l0 * p.lda;
        B += BK_ ? l0 : l0 * p.ldb;
        L = L - l0 < p.slice ? L - l0 : p.slice;
        partial = p.partial + blockIdx.y * p.R * p.C;
    }
    const int64_t T = L > 0 ? (L + BK - 1) / BK : 0;
    const uint16_t* a_origin = AK ? A + m0 * p.lda : A + m0;
    const uint16_t* b_origin = BK_ ? B + n0 * p.ldb : B + n0;

    using acc_t = typename Op::acc_t;
    acc_t acc[MI][NI];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j)
#pragma unroll
            for (int v = 0; v < Op::ACC; ++v) acc[i][j][v] = 0.0f;

    const OperandRead<OA, AK, MI> read_a(wm0, lane);
    const OperandRead<OB, BK_, NI> read_b(wn0, lane);
    auto read_fragments = [&](int stage, int st, u32x4 (&af)[MI], u32x4 (&bf)[NI]) {
#pragma unroll
        for (int i = 0; i < MI; ++i) af[i] = read_a.read(lds_a, stage, st, i);
#pragma unroll
        for (int j = 0; j < NI; ++j) bf[j] = read_b.read(lds_b, stage, st, j);
    };
    auto multiply_step = [&](const u32x4 (&af)[MI], const u32x4 (&bf)[NI]) {
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j) acc[i][j] = Op::mma(bf[j], af[i], acc[i][j]);
    };
    u32x4 af[2][MI], bf[2][NI];

    if constexpr (DIRECT) {
        using CA = OperandCopy<AK, BM, BK, S, THREADS>;
        using CB = OperandCopy<BK_, BN, BK, S, THREADS>;
        constexpr int COPIES = CA::PER_WAVE + CB::PER_WAVE;
        const CA copy_a(a_origin, p.lda, m_end - m0, L, wave, lane);
        const CB copy_b(b_origin, p.ldb, p.C - n0, L, wave, lane);
        auto issue = [&](int64_t t, int stage) {
            copy_a.issue(t, L - t * BK, lds_a, stage);
            copy_b.issue(t, L - t * BK, lds_b, stage);
        };
#pragma unroll
        for (int s = 0; s < S - 1; ++s) issue(s, s);
        wait_vector_memory_at_most<(S - 2) * COPIES>();
        __syncthreads();
        int s = 0;  // stage of tile t
        if (T > 0) read_fragments(0, 0, af[0], bf[0]);
        for (int64_t t = 0; t < T; ++t) {
            const int free_stage = s == 0 ? S - 1 : s - 1, next = s + 1 == S ? 0 : s + 1;
            issue(t + S - 1, free_stage);
#pragma unroll
            for (int st = 0; st + 1 < 4; ++st) {
                read_fragments(s, st + 1, af[(st + 1) & 1], bf[(st + 1) & 1]);
                multiply_step(af[st & 1], bf[st & 1]);
                alternate_mfma_and_lds_reads<MI * NI>();
            }
            wait_vector_memory_at_most<(S - 2) * COPIES>();
            __syncthreads();
            read_fragments(next, 0, af[0], bf[0]);  // (of the last tile: zeros)
            multiply_step(af[1], bf[1]);
            alternate_mfma_and_lds_reads<MI * NI>();
            s = next;
        }
        wait_vector_memory();
    } else {
        // Two stages; the loads of tile t+1 are issued before the multiply
        // of tile t and stored to LDS after it.
        OperandLoad<AK, BM, BK, S, THREADS> load_a(a_origin, p.lda, m_end - m0);
        OperandLoad<BK_, BN, BK, S, THREADS> load_b(b_origin, p.ldb, p.C - n0);
        if (T > 0) {
            load_a.load(0, L, tid);
            load_b.load(0, L, tid);
            load_a.store(lds_a, 0, tid);
            load_b.store(lds_b, 0, tid);
        }
        __syncthreads();
        for (int64_t t = 0; t < T; ++t) {
            const int s = (int)(t & 1);
            if (t + 1 < T) {
                load_a.load(t + 1, L - (t + 1) * BK, tid);
                load_b.load(t + 1, L - (t + 1) * BK, tid);
            }
            read_fragments(s, 0, af[0], bf[0]);
#pragma unroll
            for (int st = 0; st < 4; ++st) {
                if (st + 1 < 4) read_fragments(s, st + 1, af[(st + 1) & 1], bf[(st + 1) & 1]);
                multiply_step(af[st & 1], bf[st & 1]);
            }
            if (t + 1 < T) {
                load_a.store(lds_a, s ^ 1, tid);
                load_b.store(lds_b, s ^ 1, tid);
            }
            __syncthreads();
        }
    }
    __syncthreads();  // every read and copy of the operand stages is done

    float* const staged = reinterpret_cast<float*>(lds) + wave * STAGE_WORDS;
    constexpr int ROW_LANES = Shape::WN / 8, ROWS = kWave / ROW_LANES;
    const int r = lane / ROW_LANES, c = lane % ROW_LANES * 8;
    const int64_t col = n0 + wn0 + c, left = p.C - col;
#pragma unroll 1
    for (int i = 0; i < MI; ++i) {
        // (one copy of the epilogue's code for all blocks: only this choice of registers is unrolled)
        static_for<MI>([&](auto I_) {
            constexpr int I = decltype(I_)::value;
            if (i != I) return;
#pragma unroll
            for (int j = 0; j < NI; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const floatx4 x{acc[I][j][4 * q], acc[I][j][4 * q + 1], acc[I][j][4 * q + 2], acc[I][j][4 * q + 3]};
                    *reinterpret_cast<floatx4*>(staged + lane % 32 * STAGE_ROW + j * 32 + 8 * q + 4 * (lane / 32)) = x;
                }
        });
        wave_fence();
#pragma unroll 1
        for (int k = 0; k < 32; k += ROWS) {
            const int64_t row = m0 + wm0 + i * 32 + k + r;
            const float* src = staged + (k + r) * STAGE_ROW + c;
            float z[8];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const floatx4 x = *reinterpret_cast<const floatx4*>(src + 4 * h);
#pragma unroll
                for (int e = 0; e < 4; ++e) z[4 * h + e] = x[e];
            }
            if (row < m_end && left > 0) {
                if (partial)
                    store8(partial + row * p.C + col, z, left);
                else
                    epilogue8<TYPE>(p.ep, group, row, col, left, z);
            }
        }
        wave_fence();
    }
}

// Sums the slices' partial products in ascending order and applies the
// epilogue; eight columns per thread.
template <int TYPE>
__global__ __launch_bounds__(256) void linear_join_kernel(LinearProblem p) {
    const int64_t row_groups = (p.C + 7) / 8, total = p.R * row_groups;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t row = i / row_groups, col = i % row_groups * 8, left = p.C - col;
        const float* src = p.partial + row * p.C + col;
        float z[8];
        load8(z, src, left);
        for (int s = 1; s < p.splits; ++s) {
            float more[8];
            load8(more, src + s * p.R * p.C, left);
#pragma unroll
            for (int e = 0; e < 8; ++e) z[e] += more[e];
        }
        epilogue8<TYPE>(p.ep, 0, row, col, left, z);
    }
}

}  // namespace dft
