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
#include "row_groups.hpp"

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
    float* tail;                 // not nullptr: the tiles past the last whole round are sliced (TailSplit)
    LinearEpilogue ep;
};

// ---- activations --------------------------------------------------------------------
// The epilogue's arithmetic is not small beside its product: 65536 values of
// a 256x256 tile cost a CU 1024 cycles per instruction (4096 for exp2 and
// rcp), so these use the hardware's exp2 and reciprocal (one unit in the last
// place each) and no library functions.

// 1 / (1 + exp(-u)); exp2 overflows to infinity and the reciprocal to 0, the
// limit, for u below -88.7.
__device__ inline float logistic(float u) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * u));
}

// The normal distribution's upper tail at |z| >= 0, erfc(x) / 2 at x = |z| /
// sqrt 2, and its density's exponential exp(-x^2): erfc(x) = exp(-x^2) t P(t)
// with t = 1 / (1 + 0.3 x), P of degree 8 fitted to erfc's own ratio over
// 0 <= x <= 10 for least relative error (2e-8; 5e-7 as evaluated in fp32).
__device__ inline float normal_tail(float z, float* density) {
    const float x = fabsf(z) * 0.70710678118654752f;
    const float t = __builtin_amdgcn_rcpf(1.0f + 0.3f * x);
    float q = -0.1295222492f;
    q = q * t + 0.4855600595f;
    q = q * t - 0.5122715831f;
    q = q * t + 0.5477126241f;
    q = q * t - 0.0946455896f;
    q = q * t + 0.2149238437f;
    q = q * t + 0.1483397484f;
    q = q * t + 0.1707151383f;
    q = q * t + 0.1691880077f;
    *density = __builtin_amdgcn_exp2f(-1.4426950408889634f * (x * x));
    return 0.5f * q * t * *density;
}

__device__ inline float gelu_tanh_argument(float z) { return 1.5957691216057308f * z * (1.0f + 0.044715f * z * z); }

__device__ inline float gelu(float z) {
    float density;
    const float tail = normal_tail(z, &density);
    return z * (z < 0.0f ? tail : 1.0f - tail);
}
// Eight values at a time: one branch on the (uniform) kind for all of them.
__device__ inline void act_values(float (&z)[8], int kind) {
    switch (kind) {
        case kActRelu:
#pragma unroll
            for (int e = 0; e < 8; ++e) z[e] = z[e] < 0.0f ? 0.0f : z[e];
            break;
        case kActGelu:
#pragma unroll
            for (int e = 0; e < 8; ++e) z[e] = gelu(z[e]);
            break;
        case kActGeluTanh:  // (1 + tanh(u)) / 2 is the logistic function of 2 u
#pragma unroll
            for (int e = 0; e < 8; ++e) z[e] *= logistic(gelu_tanh_argument(z[e]));
            break;
        case kActSilu:
#pragma unroll
            for (int e = 0; e < 8; ++e) z[e] *= logistic(z[e]);
            break;
        default: break;
    }
}
// The slope at z.  Beyond |z| = 128 every slope has reached its limit in
// fp32; stopping there keeps 0 * infinity out of the products (a NaN z stays).
__device__ inline void act_slopes(float (&z)[8], int kind) {
#pragma unroll
    for (int e = 0; e < 8; ++e) z[e] = z[e] > 128.0f ? 128.0f : z[e] < -128.0f ? -128.0f : z[e];
    switch (kind) {
        case kActRelu:
#pragma unroll
            for (int e = 0; e < 8; ++e) z[e] = z[e] > 0.0f ? 1.0f : 0.0f;
            break;
        case kActGelu:
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float density;
                const float tail = normal_tail(z[e], &density);
                z[e] = (z[e] < 0.0f ? tail : 1.0f - tail) + z[e] * 0.39894228040143268f * density;
            }
            break;
        case kActGeluTanh:
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float gate = logistic(gelu_tanh_argument(z[e]));
                const float du = 1.5957691216057308f * (1.0f + 0.134145f * z[e] * z[e]);
                z[e] = gate + z[e] * gate * (1.0f - gate) * du;
            }
            break;
        case kActSilu:
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float gate = logistic(z[e]);
                z[e] = gate + z[e] * gate * (1.0f - gate);
            }
            break;
        default:
#pragma unroll
            for (int e = 0; e < 8; ++e) z[e] = 1.0f;
    }
}

// ---- 16-bit values ------------------------------------------------------------------
// Eight consecutive 16-bit values in four words, so that they move as one
// 16-byte access at any 2-byte alignment.
struct Row8 {
    u32x4 w;
    template <int TYPE>
    __device__ void widen(float (&v)[8]) const {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (TYPE == kInputBf16) {
                v[2 * e] = __builtin_bit_cast(float, w[e] << 16);
                v[2 * e + 1] = __builtin_bit_cast(float, w[e] & 0xffff0000u);
            } else {
                v[2 * e] = (float)__builtin_bit_cast(_Float16, (uint16_t)(w[e] & 0xffffu));
                v[2 * e + 1] = (float)__builtin_bit_cast(_Float16, (uint16_t)(w[e] >> 16));
            }
        }
    }
    // Rounded to nearest, ties to even.
    template <int TYPE>
    __device__ static Row8 narrow(const float (&v)[8]) {
        typedef float pair __attribute__((ext_vector_type(2)));
        typedef __bf16 bf16_pair __attribute__((ext_vector_type(2)));
        typedef _Float16 f16_pair __attribute__((ext_vector_type(2)));
        Row8 r;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const pair x{v[2 * e], v[2 * e + 1]};
            if constexpr (TYPE == kInputBf16)
                r.w[e] = __builtin_bit_cast(uint32_t, __builtin_convertvector(x, bf16_pair));
            else
                r.w[e] = __builtin_bit_cast(uint32_t, __builtin_convertvector(x, f16_pair));
        }
        return r;
    }
};
// The first `in_range` of the eight, zeros for the others: one access when all
// are in range, else eight, at the last one in range for those beyond it, so
// that all are on their way together.
__device__ inline Row8 load8(const uint16_t* p, int64_t in_range) {
    Row8 r{};
    if (in_range >= 8) {
        __builtin_memcpy(&r.w, p, sizeof(r.w));
    } else if (in_range > 0) {
        const int last = (int)in_range - 1;
        uint32_t v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = p[e < last ? e : last];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            r.w[e] = (2 * e <= last ? v[2 * e] : 0u) | (2 * e + 1 <= last ? v[2 * e + 1] << 16 : 0u);
    }
    return r;
}
__device__ inline void store8(uint16_t* p, const Row8& r, int64_t in_range) {
    if (in_range >= 8) {
        __builtin_memcpy(p, &r.w, sizeof(r.w));
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < in_range) p[e] = (uint16_t)(r.w[e / 2] >> (e % 2 * 16));
    }
}
__device__ inline void load8(float (&v)[8], const float* p, int64_t in_range) {
    if (in_range >= 8) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            floatx4 x;
            __builtin_memcpy(&x, p + 4 * h, sizeof(x));
#pragma unroll
            for (int e = 0; e < 4; ++e) v[4 * h + e] = x[e];
        }
    } else if (in_range > 0) {
        const int last = (int)in_range - 1;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = p[e < last ? e : last];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = e <= last ? v[e] : 0.0f;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0.0f;
    }
}
__device__ inline void store8(float* p, const float (&v)[8], int64_t in_range) {
    if (in_range >= 8) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const floatx4 x{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
            __builtin_memcpy(p + 4 * h, &x, sizeof(x));
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < in_range) p[e] = v[e];
    }
}

// The epilogue of eight consecutive columns of one output row.  `bias` and
// `residual` (of 16 bits) have been read before; an fp32 residual is read
// here.  Addresses are a uniform base and a lane's byte offset, which the
// loads and stores take as they are; `left` of the columns lie inside the
// matrix.
struct EpilogueBase {
    char *out, *preact;
    const char* residual;
};
struct EpilogueLane {
    uint32_t out, preact, residual;
};
__device__ inline EpilogueBase epilogue_base(const LinearEpilogue& ep, int64_t group, int64_t row, int64_t col) {
    const int64_t bytes = ep.out_f32 ? 4 : 2;
    return EpilogueBase{static_cast<char*>(ep.out) + bytes * (group * ep.out_group + row * ep.ldo + col),
                        reinterpret_cast<char*>(ep.preact) + 2 * (row * ep.ldp + col),
                        static_cast<const char*>(ep.residual) + bytes * (row * ep.ldr + col)};
}
__device__ inline EpilogueLane epilogue_lane(const LinearEpilogue& ep, int row, int col) {
    const uint32_t bytes = ep.out_f32 ? 4 : 2;
    return EpilogueLane{bytes * (row * (uint32_t)ep.ldo + col), 2 * (row * (uint32_t)ep.ldp + col),
                        bytes * (row * (uint32_t)ep.ldr + col)};
}
__device__ inline Row8 bias_reads(const LinearEpilogue& ep, int64_t at, int64_t left) {
    return ep.bias ? load8(ep.bias + at, left) : Row8{};
}
__device__ inline Row8 residual_reads(const LinearEpilogue& ep, const EpilogueBase& base, const EpilogueLane& lane,
                                      int64_t left) {
    if (!ep.residual || ep.out_f32) return Row8{};
    return load8(reinterpret_cast<const uint16_t*>(base.residual + lane.residual), left);
}
// PLAIN (the gradients' products): the sums alone, rounded.
template <int TYPE, bool PLAIN = false>
__device__ inline void epilogue8(const LinearEpilogue& ep, const Row8& bias, const Row8& residual,
                                 const EpilogueBase& base, const EpilogueLane& lane, int64_t left, float (&z)[8]) {
    if constexpr (!PLAIN) {
        float add[8];
        bias.widen<TYPE>(add);  // (zeros without a bias, and so for the residual: an addition is less than a branch)
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] += add[e];
        if (ep.preact) store8(reinterpret_cast<uint16_t*>(base.preact + lane.preact), Row8::narrow<TYPE>(z), left);
        act_values(z, ep.act);
        residual.widen<TYPE>(add);
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] += add[e];
        if (ep.residual && ep.out_f32) {
            load8(add, reinterpret_cast<const float*>(base.residual + lane.residual), left);
#pragma unroll
            for (int e = 0; e < 8; ++e) z[e] += add[e];
        }
    }
    if (ep.out_f32)
        store8(reinterpret_cast<float*>(base.out + lane.out), z, left);
    else
        store8(reinterpret_cast<uint16_t*>(base.out + lane.out), Row8::narrow<TYPE>(z), left);
}

// ---- groups of rows (row_groups.hpp) ------------------------------------------------
// The tile-th tile of `tile_rows` rows when every group's rows are tiled from
// the group's own start; group < 0: there is no such tile.  Every wave looks
// it up itself: 64 groups at a time, one per lane.
struct GroupTile {
    int group;
    int64_t row0, row_end;
};
__device__ inline GroupTile find_group_tile(const int32_t* offsets, int groups, int64_t rows, int tile_rows,
                                            int64_t tile) {
    const int lane = threadIdx.x % kWave;
    int64_t before = 0;
    for (int g0 = 0; g0 < groups; g0 += kWave) {
        const int g = g0 + lane;
        RowRange r{0, 0};
        if (g < groups) r = group_rows(offsets, g, rows);
        const int own = (int)r.tiles(tile_rows);
        int upto = own;  // inclusive running sum over the lanes (a launch has fewer than 2^23 row tiles, so no group more)
#pragma unroll
        for (int d = 1; d < kWave; d *= 2) {
            const int other = __shfl_up(upto, d);
            if (lane >= d) upto += other;
        }
        const bool here = tile >= before + upto - own && tile < before + upto;
        const uint64_t found = __ballot(here);
        if (found) {
            const int l = __builtin_ctzll(found);
            // (lane l's values, uniform: the tile's addresses stay in scalar registers)
            const int64_t first = before + __builtin_amdgcn_readlane(upto - own, l);
            const int64_t lo = __builtin_amdgcn_readlane((int)r.lo, l), hi = __builtin_amdgcn_readlane((int)r.hi, l);
            return GroupTile{g0 + l, lo + (tile - first) * tile_rows, hi};
        }
        before += __builtin_amdgcn_readlane(upto, kWave - 1);
    }
    return GroupTile{-1, 0, 0};
}

// Orders a wave's own LDS accesses before it and after it: its lanes exchange
// values through LDS without a workgroup barrier.
__device__ inline void wave_fence() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }

// ---- operand tiles ------------------------------------------------------------------
// One operand's tile of OUT output rows (or columns) by 64 contraction
// elements in LDS, in 4-byte words.  K-major: OUT rows of 64 elements; else 64
// rows of OUT elements.  16-byte groups are swizzled within a row so that each
// pass of the fragment reads falls on different banks (of 64): a 16-byte read
// takes 16 lanes a pass, four from each of four rows r with r & 1 and (r >> 1)
// & 7 between them telling 16 places apart; an 8-byte transposing read takes
// 32 lanes a pass, eight rows (4 and 4, eight rows apart) of 32 bytes each.
constexpr int kDepth = 64;

template <bool KMAJOR, int OUT, int STAGES>
struct OperandTile {
    static_assert(OUT % 32 == 0, "whole fragments");
    static constexpr int rows = KMAJOR ? OUT : kDepth, cols = (KMAJOR ? kDepth : OUT) / 2;  // words
    static constexpr int stage_words = rows * cols, total_words = STAGES * stage_words;
    static constexpr int row_groups = cols / 4;  // 16-byte groups per row
    static constexpr int period = 16;            // rows after which the swizzle repeats
    __host__ __device__ static constexpr int swizzle(int row) {
        if (KMAJOR) return 4 * ((row >> 1) & 7);
        return 16 * (OUT >= 128 ? row & 3 : OUT == 64 ? (row >> 1) & 1 : 0) + 8 * ((row >> 3) & 1);
    }
    __host__ __device__ static constexpr int at(int row, int col) { return row * cols + (col ^ swizzle(row)); }
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

// The copies of one operand's tiles, 16 bytes per lane, tile after tile.  A
// wave's copies of a tile are WAVES pieces of 1 KiB apart, which is a whole
// number of swizzle periods, so one offset per lane and a constant step
// describe them all.  The next tile is one addition to that offset: the
// buffer stays where it is, except that a contraction along the rows moves it
// on before offsets could pass 2^31.  (Setting up a buffer for every tile
// cost the K loop a tenth: its scalar arithmetic stands between the barriers.)
template <bool KMAJOR, int OUT, int STAGES, int THREADS>
struct OperandCopy {
    using Tile = OperandTile<KMAJOR, OUT, STAGES>;
    static constexpr int WAVES = THREADS / kWave;
    static constexpr int PIECE_ROWS = kWave / Tile::row_groups;
    static constexpr int PER_WAVE = Tile::stage_words * 4 / 1024 / WAVES;
    static_assert(PER_WAVE * WAVES * 1024 == Tile::stage_words * 4, "whole pieces per wave");
    static_assert((WAVES * PIECE_ROWS) % Tile::period == 0, "whole swizzle periods per step");

    const char* base;   // the buffer's first byte (uniform), `size` bytes long
    int64_t size;
    u32x4 buffer;
    uint32_t offset;    // this lane's first copy of the tile, from `base`
    uint32_t step;      // between its copies of one tile
    uint32_t advance;   // between tiles
    int depth, left;    // k-major: contraction index of the lane's 16 bytes in the tile; elements from the tile on
    int until;          // rows along the contraction: tiles before the buffer moves
    int period;
    uint32_t lds_piece;

    // `origin`: the element at contraction index 0 and the tile's first output row (column); `outs`: output rows
    // (columns) from there; `length`: contraction elements.
    __device__ OperandCopy(const uint16_t* origin, int64_t ld, int64_t outs, int64_t length, int wave, int lane) {
        base = reinterpret_cast<const char*>(origin);
        const int64_t rows = KMAJOR ? outs : length, cols = KMAJOR ? length : outs;
        // (widths are multiples of 8, or packed rows padded to them)
        size = rows > 0 && cols > 0 ? 2 * ((rows - 1) * ld + (cols + 7) / 8 * 8) : 0;
        const int row = wave * PIECE_ROWS + lane / Tile::row_groups;
        const int word = (lane % Tile::row_groups * 4) ^ Tile::swizzle(row);
        offset = (uint32_t)(2 * row * ld) + 4 * word;
        step = (uint32_t)(2 * WAVES * PIECE_ROWS * ld);
        advance = KMAJOR ? 2 * kDepth : (uint32_t)(2 * kDepth * ld);
        depth = 2 * word;
        left = KMAJOR ? (int)length : 0;
        if (!KMAJOR && 2 * word >= outs) offset = kBeyond;
        // (a lane past the edge stays beyond: its offset may grow to 2^32 - 1, never past it)
        period = until = KMAJOR ? 0x7fffffff : (int)(0x3fffffff / advance);
        lds_piece = wave * 1024;
        set_buffer();
    }
    __device__ void set_buffer() {
        const uint64_t b = (uint64_t)(uintptr_t)base;
        const int64_t bytes = size < 0 ? 0 : size > 0x7fffffff ? 0x7fffffff : size;
        buffer = u32x4{first_lane((uint32_t)b), first_lane((uint32_t)(b >> 32) & 0xffffu), first_lane((uint32_t)bytes),
                       0x00020000u};
    }
    // Copy i of the tile into `stage` (a tile past the end fills it with zeros).
    struct Issue {
        u32x4 buffer;
        uint32_t from, step, to;
        __device__ void operator()(int i) const { copy16_checked(buffer, from + i * step, to + i * (WAVES * 1024)); }
    };
    __device__ Issue tile(uint32_t* lds, int stage) const {
        typedef __attribute__((address_space(3))) uint32_t lds_word;
        const uint32_t to = first_lane((uint32_t)(uintptr_t)(lds_word*)lds + stage * (Tile::stage_words * 4) + lds_piece);
        return Issue{buffer, KMAJOR && depth >= left ? kBeyond : offset, step, to};
    }
    __device__ void next() {
        offset += advance;
        if constexpr (KMAJOR) {
            left -= kDepth;
        } else if (--until == 0) {
            until = period;
            base += (int64_t)period * advance;
            size -= (int64_t)period * advance;
            offset -= (uint32_t)period * advance;
            set_buffer();
        }
    }
    __device__ void issue(uint32_t* lds, int stage) const {
        const Issue copy = tile(lds, stage);
#pragma unroll
        for (int i = 0; i < PER_WAVE; ++i) copy(i);
    }
};

// The same tiles through registers, for operands whose rows or widths are
// not multiples of 16 bytes: 16-byte loads at any 2-byte alignment where a
// whole group is in range, masked elements at the edges.
template <bool KMAJOR, int OUT, int STAGES, int THREADS>
struct OperandLoad {
    using Tile = OperandTile<KMAJOR, OUT, STAGES>;
    static constexpr int GROUPS = Tile::rows * Tile::row_groups;
    static constexpr int PER_THREAD = GROUPS / THREADS;
    static_assert(GROUPS % THREADS == 0, "whole groups per thread");

    const uint16_t* origin;
    int64_t ld, outs;
    Row8 held[PER_THREAD];

    __device__ OperandLoad(const uint16_t* origin_, int64_t ld_, int64_t outs_) : origin(origin_), ld(ld_), outs(outs_) {}
    __device__ void load(int64_t t, int64_t left, int tid) {
        const uint16_t* tile = origin + t * (KMAJOR ? (int64_t)kDepth : kDepth * ld);
        const int64_t rows = KMAJOR ? outs : left, cols = KMAJOR ? left : outs;
#pragma unroll
        for (int i = 0; i < PER_THREAD; ++i) {
            const int at = tid + i * THREADS, row = at / Tile::row_groups, col = at % Tile::row_groups * 8;
            held[i] = load8(tile + row * ld + col, row < rows ? cols - col : 0);
        }
    }
    __device__ void store(uint32_t* lds, int stage, int tid) const {
#pragma unroll
        for (int i = 0; i < PER_THREAD; ++i) {
            const int at = tid + i * THREADS, row = at / Tile::row_groups, col = at % Tile::row_groups * 8;
            *reinterpret_cast<u32x4*>(lds + stage * Tile::stage_words + Tile::at(row, col / 2)) = held[i].w;
        }
    }
};

// A wave's fragments of one operand: block i (16 output rows or columns) of
// MFMA step st (32 contraction elements), 8 of them per lane.  One place per
// lane: a block along the rows (k-major: a step) is 8 (16) words further on,
// in bits that the swizzle may have flipped but that the wave's first column
// and whole rows leave alone, so it flips the same bits of the place.
template <class Tile, bool KMAJOR, int BLOCKS>
struct OperandRead {
    static_assert(KMAJOR || (BLOCKS & (BLOCKS - 1)) == 0, "a wave's blocks fill an aligned range of columns");
    int from;

    __device__ OperandRead(int out0, int lane) {
        if constexpr (KMAJOR)
            from = Tile::at(out0 + lane % 16, 4 * (lane / 16));
        else
            from = Tile::at(8 * (lane / 16) + (lane % 16) / 4, (out0 + 4 * (lane % 4)) / 2);
    }
    __device__ u32x4 read(const uint32_t* lds, int place, int st, int i) const {
        const int base = place * Tile::stage_words + from;
        if constexpr (KMAJOR) {
            return *reinterpret_cast<const u32x4*>(lds + (base ^ (16 * st)) + i * 16 * Tile::cols);
        } else {
            typedef __attribute__((address_space(3))) const uint32_t lds_word;
            typedef __attribute__((address_space(3))) shortx4 lds_short4;
            u32x2 half[2];
#pragma unroll
            for (int rr = 0; rr < 2; ++rr) {
                const int word = (base ^ (8 * i)) + (st * 32 + 4 * rr) * Tile::cols;
                half[rr] = __builtin_bit_cast(u32x2,
                                              __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4*)((lds_word*)lds + word)));
            }
            return u32x4{half[0][0], half[0][1], half[1][0], half[1][1]};
        }
    }
};

// ---- the product --------------------------------------------------------------------
// PERSISTENT: one workgroup per place on the chip works through many tiles;
// the first copies of the next tile are issued before the epilogue of this
// one, whose rows pass through LDS of their own.
template <int BM_, int BN_, int WM_, int WN_, int STAGES_, int MIN_WAVES_, bool PERSISTENT_ = false>
struct LinearShape {
    static constexpr bool PERSISTENT = PERSISTENT_;
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, STAGES = STAGES_, MIN_WAVES = MIN_WAVES_;
    static constexpr int WAVES_N = BN / WN, THREADS = BM / WM * WAVES_N * kWave;
    static constexpr int MI = WM / 16, NI = WN / 16;
};

// Consecutive tiles on one XCD (workgroups go to the eight XCDs in turn), in
// panels of `high` tile rows, so that the tiles an XCD works on at one time
// share their operands' rows and columns in its L2.
struct TilePlace {
    int64_t row, col;
};
__device__ inline TilePlace place_of_block(uint32_t block, uint32_t blocks, uint32_t tiles_m, uint32_t tiles_n,
                                           uint32_t high) {
    const uint32_t xcd = block % 8, each = blocks / 8, more = blocks % 8;
    const uint32_t id = xcd * each + (xcd < more ? xcd : more) + block / 8;
    const uint32_t panel = high * tiles_n, p = id / panel, in = id % panel;
    const uint32_t rows = tiles_m - high * p < high ? tiles_m - high * p : high;
    return TilePlace{high * p + in % rows, in / rows};
}
// Four tile rows for 256x256 tiles: the XCDs' panels are then more often whole
// ones, which move over B's columns together (8192^3 with bias, activation,
// residual and pre-activation 855 us with panels of 8, 838 with 4, 870 with
// 16).  Eight for grouped rows (each group has a B of its own: 546 against 552
// us for 8 groups of about 2048 rows by 4096, 4096 deep) and for the smaller
// tiles, of which an XCD works on 64 at a time.
template <int BM>
__device__ inline uint32_t panel_rows(const LinearProblem& p) {
    return BM == 256 && p.axis != kGroupRows ? 4 : 8;
}

// Tiles of all groups' rows.
__device__ inline int64_t count_group_tiles(const int32_t* offsets, int groups, int64_t rows, int tile_rows) {
    int64_t all = 0;
    for (int g0 = 0; g0 < groups; g0 += kWave) {
        const int g = g0 + (int)(threadIdx.x % kWave);
        int own = 0;
        if (g < groups) {
            const RowRange r = group_rows(offsets, g, rows);
            own = (int)r.tiles(tile_rows);
        }
#pragma unroll
        for (int d = kWave / 2; d > 0; d /= 2) own += __shfl_xor(own, d);
        all += __builtin_amdgcn_readfirstlane(own);
    }
    return all;
}

// Row tiles there are of the tiles_m that any division of the rows into groups
// has at most (groups that overlap would have more: those are left out).
__device__ inline uint32_t real_row_tiles(const LinearProblem& p, int tile_rows, uint32_t tiles_m) {
    if (p.axis != kGroupRows) return tiles_m;
    const int64_t tiles = count_group_tiles(p.offsets, p.groups, p.R, tile_rows);
    return tiles < (int64_t)tiles_m ? (uint32_t)tiles : tiles_m;
}

// The last round of a persistent grid: `left` tiles for `grid` workgroups.
// Cut along the contraction into `parts` slices each, their partial products
// go to p.tail, one BM x BN block of fp32 per workgroup, and are joined by
// linear_tail_kernel.  A round of whole tiles of 64 contraction tiles takes
// about 100 us; slicing costs the join's launch and twice 64 MiB of traffic,
// about 30 us, so it is asked for from 32 contraction tiles on (by the host)
// and done where each tile gets at least two slices.
constexpr int kTailDepth = 32;
struct TailSplit {
    uint32_t whole, left, parts;  // tiles before the last round (all, if it is not sliced), tiles in it, slices of each
    int64_t slice;                // contraction elements per slice
};
__device__ inline TailSplit tail_split(const LinearProblem& p, uint32_t tiles, uint32_t grid) {
    TailSplit t{tiles, 0, 1, p.L};
    const uint32_t left = tiles % grid, depth = (uint32_t)((p.L + 63) / 64);
    if (!p.tail || left == 0 || grid / left < 2) return t;
    t.left = left;
    t.whole = tiles - left;
    t.parts = grid / left < depth / 8 ? grid / left : depth / 8;
    t.slice = (int64_t)((depth + t.parts - 1) / t.parts) * 64;
    return t;
}

// The kernel's own LinearProblem argument, read again from the argument
// segment (scalar loads).  Kept live from the kernel's start, its fields and
// the K loop's would not fit the scalar registers together, and what does not
// fit is moved to vector registers that the sums need.
__device__ inline LinearProblem problem_again() {
    typedef __attribute__((address_space(4))) const LinearProblem constant_problem;
    auto* at = (constant_problem*)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(at));
    LinearProblem p;
    __builtin_memcpy(&p, at, sizeof(p));
    return p;
}

// The same value, which the compiler may not know to be: what is computed from
// it stays inside the loop over tiles instead of being kept for all of them.
__device__ inline int afresh(int lane) {
    asm volatile("" : "+v"(lane));
    return lane;
}
__device__ inline int afresh_uniform(int wave) {
    asm volatile("" : "+s"(wave));
    return wave;
}

// A uniform value, in scalar registers.
__device__ inline int64_t scalar(int64_t v) {
    const uint64_t lo = first_lane((uint32_t)v), hi = first_lane((uint32_t)((uint64_t)v >> 32));
    return (int64_t)(lo | hi << 32);
}

// A workgroup's share of the work: one output tile of one matrix, group or slice.
struct LinearWork {
    int64_t m0, m_end, n0, group, L;
    const uint16_t* A;  // first element of the operands' rows and contraction
    const uint16_t* B;
    float* partial;     // where the sums go instead of the epilogue: element (row, column) of the output at
    int64_t partial_ld; //   partial + row * partial_ld + column
    bool none;          // past the last group's tiles
};
template <bool AK, bool BK_, int BM, int BN>
__device__ inline LinearWork linear_work(const LinearProblem& p, uint32_t tile, uint32_t tiles_m, uint32_t tiles_n,
                                         uint32_t y) {
    const TilePlace place = place_of_block(tile, tiles_m * tiles_n, tiles_m, tiles_n, panel_rows<BM>(p));
    LinearWork w{place.row * BM, p.R, place.col * BN, 0, p.L, p.A, p.B, nullptr, p.C, false};
    if (p.axis == kGroupRows) {
        const GroupTile gt = find_group_tile(p.offsets, p.groups, p.R, BM, place.row);
        if (gt.group < 0) {
            w.none = true;
            return w;
        }
        w.group = gt.group;
        w.m0 = gt.row0;
        w.m_end = gt.row_end;
        w.B += w.group * p.b_group;
    } else if (p.axis == kGroupContraction) {
        w.group = y;
        const RowRange r = group_rows(p.offsets, (int)y, p.L);
        w.A += r.lo * p.lda;
        w.B += r.lo * p.ldb;
        w.L = r.hi - r.lo;
    } else if (p.splits > 1) {
        const int64_t l0 = y * p.slice;
        w.A += AK ? l0 : l0 * p.lda;
        w.B += BK_ ? l0 : l0 * p.ldb;
        w.L = w.L - l0 < p.slice ? w.L - l0 : p.slice;
        w.partial = p.partial + y * p.R * p.C;
    }
    w.A += AK ? w.m0 * p.lda : w.m0;
    w.B += BK_ ? w.n0 * p.ldb : w.n0;
    return w;
}
// Slice `part` of a tile of the last round, the at-th block of p.tail.
template <bool AK, bool BK_, int BM, int BN>
__device__ inline void slice_work(const LinearProblem& p, const TailSplit& t, LinearWork& w, uint32_t part, uint32_t at) {
    const int64_t l0 = part * t.slice;
    w.A += AK ? l0 : l0 * p.lda;
    w.B += BK_ ? l0 : l0 * p.ldb;
    w.L = w.L - l0 < t.slice ? w.L - l0 : t.slice;
    w.partial = p.tail + (int64_t)at * (BM * BN) - (w.m0 * BN + w.n0);
    w.partial_ld = BN;
}

// One BM x BN output tile (of a slice of the contraction, or of a group) at a
// time, with one barrier per contraction tile: every wave has read all of tile
// t by the barrier inside iteration t, before that iteration's last MFMA step,
// and what is copied into the places it frees is issued between the MFMAs of
// that step.  S LDS stages of both operands: there go the copies of tile t+S.
// Persistent (the operands' tiles are of one size): a ring of five places for
// A 0, B 0, A 1, B 1, A 2, ...; there go B of tile t+2 and A of tile t+3, so
// that A's copies have two tiles' time to land and B's, issued first, one; the
// fifth place serves the epilogue's rows while the next share's first two
// tiles are on their way to the others.
// The fragments of an MFMA step (16x16x32: the same products with 32x32x16
// draw more power and ran at 1.80 against 2.03 PFLOP/s from registers) are
// read between the MFMAs of the step before, the first of a tile between those
// of the last step of the tile before it, after the barrier.
// The MFMAs take B as their row operand, so a lane's four consecutive results
// are four consecutive columns of one output row; each wave passes its
// results through LDS, 16 rows at a time, to give every lane eight columns of
// a row, and the epilogue's loads and stores 16 bytes per lane.
// Bound by the matrix cores at the clock that power leaves them, and per tile
// by the epilogue, which nothing overlaps (8192^2 outputs, four rounds of
// tiles: 9 us a round for storing plain results, 15 with the epilogue's
// branches, 27 with silu, residual and pre-activation): 8192^3 826 us forward
// (1.33 PFLOP/s), 836 with the full epilogue, 745 dA (1.48), 795 dB (1.38).
// Few rows are bound by B's bytes: 24 rows of 4096 by 16384 24.5 us (5.5 TB/s).
template <int TYPE, bool AK, bool BK_, class Shape, bool DIRECT>
__global__ __launch_bounds__(Shape::THREADS, Shape::MIN_WAVES) void linear_tile_kernel(LinearProblem, uint32_t tiles_m,
                                                                                   uint32_t tiles_n, uint32_t grid_y) {
    using Op = Mfma16Op<TYPE, 16>;
    constexpr int BM = Shape::BM, BN = Shape::BN, BK = kDepth, S = DIRECT ? Shape::STAGES : 2;
    constexpr int MI = Shape::MI, NI = Shape::NI, THREADS = Shape::THREADS, STEPS = BK / 32;
    constexpr bool PERSISTENT = Shape::PERSISTENT && DIRECT, PLAIN = !AK || BK_;
    using TileA = OperandTile<AK, BM, S>;
    using TileB = OperandTile<BK_, BN, S>;
    constexpr int RING = 5;
    static_assert(!PERSISTENT || TileA::stage_words == TileB::stage_words, "the ring's places take either operand");
    constexpr int OPERANDS = PERSISTENT ? RING * TileA::stage_words : TileA::total_words + TileB::total_words;
    constexpr int BR = 16;  // rows that a wave stages at a time: one block of results
    constexpr int BLOCK_WORDS = BR * Shape::WN, STAGED = THREADS / kWave * BLOCK_WORDS;
    static_assert(STAGED <= (PERSISTENT ? TileA::stage_words : OPERANDS), "the staged blocks fit");

    __shared__ __attribute__((aligned(16))) uint32_t lds[OPERANDS];
    poison_lds(lds, OPERANDS);
    uint32_t* const lds_a = lds;
    uint32_t* const lds_b = lds + (PERSISTENT ? 0 : TileA::total_words);

    const int tid = threadIdx.x, every_lane = tid % kWave;
    const int every_wave = __builtin_amdgcn_readfirstlane(tid / kWave);

    // Grouped rows: tiles_m is the most that their division may need (row_tiles), and places past the real tiles stay
    // empty.  Counting the real ones first, as the persistent tiles do, spreads them evenly over the XCDs but costs a
    // wave another scan of the offsets before its first copy: 128 rows of 32 experts of 4096x4096 249 -> 201 us, 2048
    // rows 347 -> 288, but dA of 512 rows 248 -> 269, and calls of up to 20 us 0.4 to 2 us more.
    const uint32_t tiles = tiles_m * tiles_n, total = tiles * grid_y;
    auto work_of = [&](uint32_t id) {
        return linear_work<AK, BK_, BM, BN>(problem_again(), id % tiles, tiles_m, tiles_n, id / tiles);
    };
    // The share of tile number id, or the next that exists (grouped rows may need fewer tiles than were counted for
    // them); in the last round, a slice of a tile.
    bool sliced = false;
    auto find_work = [&](uint32_t& id, LinearWork& w) {
        if constexpr (PERSISTENT) {
            const LinearProblem p = problem_again();
            if (p.tail || p.axis == kGroupRows) {
                // (the tiles there are, so that the last ones are the last round)
                const uint32_t real_m = real_row_tiles(p, BM, tiles_m);
                const TailSplit t = tail_split(p, real_m * tiles_n, gridDim.x);
                auto tile_of = [&](uint32_t tile) {
                    return linear_work<AK, BK_, BM, BN>(p, tile, real_m, tiles_n, 0);
                };
                if (id < t.whole) {
                    w = tile_of(id);
                    return true;
                }
                const uint32_t at = blockIdx.x;  // (id is in the last round: id - at == whole)
                if (sliced || at >= t.left * t.parts) return false;
                sliced = true;
                w = tile_of(t.whole + at / t.parts);
                slice_work<AK, BK_, BM, BN>(p, t, w, at % t.parts, at);
                return true;
            }
        }
        for (; id < total; id += gridDim.x) {
            w = work_of(id);
            if (!w.none) return true;
        }
        return false;
    };
    uint32_t id = blockIdx.x;
    LinearWork w;
    if (!find_work(id, w)) return;

    using acc_t = typename Op::acc_t;
    using CA = OperandCopy<AK, BM, S, THREADS>;
    using CB = OperandCopy<BK_, BN, S, THREADS>;
    constexpr int COPIES = CA::PER_WAVE + CB::PER_WAVE;
    // The first copies of a share.
    auto start_copies = [&](const LinearWork& w) {
        if constexpr (DIRECT) {
            const LinearProblem p = problem_again();
            const int lane = afresh(every_lane), wave = afresh_uniform(every_wave);
            CA copy_a(w.A, p.lda, w.m_end - w.m0, w.L, wave, lane);
            CB copy_b(w.B, p.ldb, p.C - w.n0, w.L, wave, lane);
#pragma unroll
            for (int s = 0; s < S; ++s) {
                copy_a.issue(lds_a, PERSISTENT ? 2 * s : s);
                copy_b.issue(lds_b, PERSISTENT ? 2 * s + 1 : s);
                copy_a.next();
                copy_b.next();
            }
        }
    };
    start_copies(w);

    for (;;) {
        const int lane = afresh(every_lane), wave = afresh_uniform(every_wave);
        const int wm0 = wave / Shape::WAVES_N * Shape::WM, wn0 = wave % Shape::WAVES_N * Shape::WN;
        const OperandRead<TileA, AK, MI> read_a(wm0, lane);
        const OperandRead<TileB, BK_, NI> read_b(wn0, lane);
        const int64_t T = w.L > 0 ? (w.L + BK - 1) / BK : 0;
        acc_t acc[MI][NI];
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j)
#pragma unroll
                for (int v = 0; v < Op::ACC; ++v) acc[i][j][v] = 0.0f;
        // Fragments: A's of the step after replace this step's as each has been multiplied, B's alternate.
        u32x4 af[MI], bf[2][NI];
        auto read_first = [&](int place_a, int place_b) {
#pragma unroll
            for (int i = 0; i < MI; ++i) af[i] = read_a.read(lds_a, place_a, 0, i);
#pragma unroll
            for (int j = 0; j < NI; ++j) bf[0][j] = read_b.read(lds_b, place_b, 0, j);
        };

        if constexpr (DIRECT) {
            const LinearProblem p = problem_again();
            CA copy_a(w.A, p.lda, w.m_end - w.m0, w.L, wave, lane);
            CB copy_b(w.B, p.ldb, p.C - w.n0, w.L, wave, lane);
#pragma unroll
            for (int s = 0; s < S; ++s) {  // (issued by start_copies)
                copy_a.next();
                copy_b.next();
            }
            // A persistent workgroup waits for its last epilogue's stores as well: left pending, they would make the
            // compiler wait for all copies inside the K loop.
            if (PERSISTENT)
                wait_vector_memory();
            else
                wait_vector_memory_at_most<(S - 1) * COPIES>();
            __syncthreads();
            int at_a = 0, at_b = PERSISTENT ? 1 : 0;  // places of tile t
            if constexpr (PERSISTENT) {
                copy_a.issue(lds_a, 4);
                copy_a.next();
            }
            if (T > 0) read_first(at_a, at_b);
            for (int64_t t = 0; t < T; ++t) {
                // places of tile t+1
                const int next_a = PERSISTENT ? (at_a >= RING - 2 ? at_a + 2 - RING : at_a + 2) : at_a + 1 == S ? 0 : at_a + 1;
                const int next_b = PERSISTENT ? (at_b >= RING - 2 ? at_b + 2 - RING : at_b + 2) : next_a;
                static_for<STEPS>([&](auto ST_) {
                    constexpr int ST = decltype(ST_)::value, NOW = ST & 1, THEN = NOW ^ 1;
                    constexpr bool LAST = ST + 1 == STEPS;
                    const int from_a = LAST ? next_a : at_a, from_b = LAST ? next_b : at_b;
                    if constexpr (LAST) {
                        wait_vector_memory_at_most<PERSISTENT ? CA::PER_WAVE : (S - 2) * COPIES>();
                        __syncthreads();
                    }
                    const auto issue_b = copy_b.tile(lds_b, PERSISTENT ? at_a : at_b);
                    const auto issue_a = copy_a.tile(lds_a, PERSISTENT ? at_b : at_a);
                    __builtin_amdgcn_sched_barrier(0);
                    static_for<MI>([&](auto I_) {
                        constexpr int I = decltype(I_)::value;
                        static_for<NI>([&](auto J_) {
                            constexpr int J = decltype(J_)::value, Q = I * NI + J;
                            acc[I][J] = Op::mma(bf[NOW][J], af[I], acc[I][J]);
                            if constexpr (Q % 2 == 0 && Q / 2 < NI)
                                bf[THEN][Q / 2] = read_b.read(lds_b, from_b, LAST ? 0 : ST + 1, Q / 2);
                            if constexpr (LAST)
                                static_for<COPIES>([&](auto X_) {
                                    constexpr int X = decltype(X_)::value;
                                    if constexpr (X * MI * NI / COPIES == Q) {
                                        if constexpr (X < CB::PER_WAVE)
                                            issue_b(X);
                                        else
                                            issue_a(X - CB::PER_WAVE);
                                    }
                                });
                            __builtin_amdgcn_sched_barrier(0);
                        });
                        af[I] = read_a.read(lds_a, from_a, LAST ? 0 : ST + 1, I);
                        __builtin_amdgcn_sched_barrier(0);
                    });
                });
                copy_a.next();
                copy_b.next();
                at_a = next_a;
                at_b = next_b;
            }
            wait_vector_memory();  // (copies past the last tile, which write zeros)
        } else {
            // Two stages; the loads of tile t+1 are issued before the
            // multiply of tile t and stored to LDS after it.
            const LinearProblem p = problem_again();
            OperandLoad<AK, BM, S, THREADS> load_a(w.A, p.lda, w.m_end - w.m0);
            OperandLoad<BK_, BN, S, THREADS> load_b(w.B, p.ldb, p.C - w.n0);
            if (T > 0) {
                load_a.load(0, w.L, tid);
                load_b.load(0, w.L, tid);
                load_a.store(lds_a, 0, tid);
                load_b.store(lds_b, 0, tid);
            }
            __syncthreads();
            for (int64_t t = 0; t < T; ++t) {
                const int s = (int)(t & 1);
                if (t + 1 < T) {
                    load_a.load(t + 1, w.L - (t + 1) * BK, tid);
                    load_b.load(t + 1, w.L - (t + 1) * BK, tid);
                }
                read_first(s, s);
                static_for<STEPS>([&](auto ST_) {
                    constexpr int ST = decltype(ST_)::value, NOW = ST & 1, THEN = NOW ^ 1;
                    if constexpr (ST + 1 < STEPS) {
#pragma unroll
                        for (int j = 0; j < NI; ++j) bf[THEN][j] = read_b.read(lds_b, s, ST + 1, j);
                    }
#pragma unroll
                    for (int i = 0; i < MI; ++i) {
#pragma unroll
                        for (int j = 0; j < NI; ++j) acc[i][j] = Op::mma(bf[NOW][j], af[i], acc[i][j]);
                        if constexpr (ST + 1 < STEPS) af[i] = read_a.read(lds_a, s, ST + 1, i);
                    }
                });
                if (t + 1 < T) {
                    load_a.store(lds_a, s ^ 1, tid);
                    load_b.store(lds_b, s ^ 1, tid);
                }
                __syncthreads();
            }
        }
        __syncthreads();  // every read and copy of the operand stages is done

        LinearWork then;
        bool more = false;
        if constexpr (PERSISTENT) {
            id += gridDim.x;
            more = find_work(id, then);
            if (more) start_copies(then);
        }

        // The epilogue, BR rows of a wave's WN columns at a time: a lane has 8 columns of every ROWS-th row, and a
        // row's lanes cover whole 128-byte lines of a 16-bit output (64-byte pieces cost the stores up to a fifth more
        // time).  A tile wholly inside the matrix takes a copy of the
        // code without masks.
        const LinearProblem p = problem_again();
        constexpr int LANES = Shape::WN / 8, ROWS = kWave / LANES, PARTS = BR / ROWS;
        const int out_lane = afresh(every_lane), r = out_lane / LANES, c = out_lane % LANES * 8;
        float* const staged = reinterpret_cast<float*>(lds) + (PERSISTENT ? 4 * TileA::stage_words : 0) + wave * BLOCK_WORDS;
        auto staged_at = [&](int row, int group16) {
            return staged + row * Shape::WN + 4 * (group16 ^ (((row & 1) << 2) | ((row >> 1) & 3)));
        };
        const int64_t tile_row = scalar(w.m0 + wm0), tile_col = scalar(w.n0 + wn0), group = scalar(w.group);
        auto finish = [&](auto WHOLE_) {
            constexpr bool WHOLE = decltype(WHOLE_)::value;
            const int64_t left = WHOLE ? (int64_t)8 : p.C - (tile_col + c);
            // part m: rows r, r + 1, ... of the wave's tile from m * ROWS on
            auto inside = [&](int m) { return WHOLE || (left > 0 && tile_row + m * ROWS + r < w.m_end); };
            auto base = [&](int m) { return epilogue_base(p.ep, group, tile_row + m * ROWS, tile_col); };
            auto read_residual = [&](int m, const EpilogueLane& lane_at) {
                return !w.partial && inside(m) ? residual_reads(p.ep, base(m), lane_at, left) : Row8{};
            };
            Row8 bias{};
            if (!PLAIN && !w.partial && left > 0) bias = bias_reads(p.ep, group * p.ep.bias_group + tile_col + c, left);
            // The residual is read for a group of parts at a time: loads and stores complete in order, so a load
            // waits for every store before it.
            constexpr int ALL = Shape::WM / ROWS, GROUP = WHOLE ? (ALL < 4 ? ALL : 4) : 1;
#pragma unroll 1
            for (int m0 = 0; m0 < ALL; m0 += GROUP) {
                // (the lane's places and the bias afresh for each group: kept across the loop in all the forms they
                // are used in, they would not fit beside the sums)
                const int out_lane = afresh(every_lane), r = out_lane / LANES, c = out_lane % LANES * 8;
                const EpilogueLane lane_at = epilogue_lane(p.ep, r, c);
                asm volatile("" : "+v"(bias.w));
                Row8 residual[GROUP];
#pragma unroll
                for (int u = 0; u < GROUP; ++u) residual[u] = PLAIN ? Row8{} : read_residual(m0 + u, lane_at);
                static_for<GROUP>([&](auto U_) {
                    constexpr int U = decltype(U_)::value;
                    const int m = m0 + U;
                    if (U % PARTS == 0 && (GROUP % PARTS == 0 || m % PARTS == 0)) {
                        const int k = m / PARTS;  // the block of results to stage
                        wave_fence();
                        // Only this choice of registers is unrolled; the comments keep the compiler from merging the
                        // choices into one sequence behind copies of all of a block's registers.
                        static_for<MI>([&](auto I_) {
                            constexpr int I = decltype(I_)::value;
                            if (k != I) return;
#pragma unroll
                            for (int j = 0; j < NI; ++j)
                                *reinterpret_cast<acc_t*>(staged_at(out_lane % 16, 4 * j + out_lane / 16)) = acc[I][j];
                            asm volatile("; rows %0" ::"i"(I) : "memory");
                        });
                        wave_fence();
                    }
                    float z[8];
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        const floatx4 x = *reinterpret_cast<const floatx4*>(staged_at(r + ROWS * (m % PARTS), c / 4 + g));
#pragma unroll
                        for (int e = 0; e < 4; ++e) z[4 * g + e] = x[e];
                    }
                    if (inside(m)) {
                        if (w.partial)
                            store8(w.partial + (tile_row + m * ROWS + r) * w.partial_ld + tile_col + c, z, left);
                        else
                            epilogue8<TYPE, PLAIN>(p.ep, bias, residual[U], base(m), lane_at, left, z);
                    }
                });
            }
        };
        if (w.m0 + BM <= w.m_end && w.n0 + BN <= p.C)
            finish(std::true_type{});
        else
            finish(std::false_type{});
        if (!more) return;
        w = then;
    }
}

// Sums the slices' partial products and applies the epilogue.  Four lanes per
// eight columns: lane l adds slices l, l + 4, ... in ascending order, then the
// four sums are added as (0 + 1) + (2 + 3), so that a few rows of many slices
// are not one long chain of loads.  3.8 us for one row of 4096 columns: a
// launch and two dependent loads.
constexpr int kJoinThreads = 256, kJoinGroups = kJoinThreads / 4;  // column groups per workgroup

template <int TYPE>
__global__ __launch_bounds__(kJoinThreads) void linear_join_kernel(LinearProblem p) {
    const int lane = threadIdx.x % kWave, slice0 = lane / 16;
    const int64_t row_groups = (p.C + 7) / 8, total = p.R * row_groups, stride = p.R * p.C;
    for (int64_t first = (int64_t)blockIdx.x * kJoinGroups + threadIdx.x / kWave * 16; first < total;
         first += (int64_t)gridDim.x * kJoinGroups) {
        const int64_t i = first + lane % 16;
        const bool own = i < total;
        const int64_t row = own ? i / row_groups : 0, col = own ? i % row_groups * 8 : 0, left = own ? p.C - col : 0;
        const float* src = p.partial + row * p.C + col;
        const EpilogueBase base = epilogue_base(p.ep, 0, row, col);
        const EpilogueLane none{0, 0, 0};
        Row8 bias{}, residual{};
        if (slice0 == 0) {
            bias = bias_reads(p.ep, col, left);
            residual = residual_reads(p.ep, base, none, left);
        }
        float z[8] = {};
#pragma unroll 4
        for (int s = slice0; s < p.splits; s += 4) {
            float more[8];
            load8(more, src + s * stride, left);
#pragma unroll
            for (int e = 0; e < 8; ++e) z[e] += more[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            z[e] += __shfl_xor(z[e], 16);
            z[e] += __shfl_xor(z[e], 32);
        }
        if (slice0 == 0 && left > 0) epilogue8<TYPE>(p.ep, bias, residual, base, none, left, z);
    }
}

// Joins the slices of the last round's tiles (tail_split of the same
// arguments) in ascending order: workgroup (j, part) sums 32 rows of its j-th
// tile.  17 us after 16384 rows in 8 groups by 4096 (64 MiB of partial sums,
// most of them still in the last-level cache).
template <int TYPE, int BM, int BN>
__global__ __launch_bounds__(256) void linear_tail_kernel(LinearProblem p, uint32_t tiles_m, uint32_t tiles_n,
                                                          uint32_t grid) {
    const uint32_t real_m = real_row_tiles(p, BM, tiles_m);
    const TailSplit t = tail_split(p, real_m * tiles_n, grid);
    if (blockIdx.x >= t.left) return;
    const LinearWork w = linear_work<true, false, BM, BN>(p, t.whole + blockIdx.x, real_m, tiles_n, 0);
    const float* block = p.tail + (int64_t)blockIdx.x * t.parts * (BM * BN);
#pragma unroll
    for (int k = 0; k < 32 * BN / 8 / 256; ++k) {
        const int i = threadIdx.x + k * 256, r = blockIdx.y * 32 + i / (BN / 8), c = i % (BN / 8) * 8;
        const int64_t row = w.m0 + r, col = w.n0 + c, left = p.C - col;
        if (row >= w.m_end || left <= 0) continue;
        const EpilogueBase base = epilogue_base(p.ep, w.group, row, col);
        const EpilogueLane none{0, 0, 0};
        const Row8 bias = bias_reads(p.ep, w.group * p.ep.bias_group + col, left),
                   residual = residual_reads(p.ep, base, none, left);
        float z[8] = {};
#pragma unroll 4
        for (uint32_t s = 0; s < t.parts; ++s) {
            float more[8];
            load8(more, block + (int64_t)s * (BM * BN) + r * BN + c, left);
#pragma unroll
            for (int e = 0; e < 8; ++e) z[e] += more[e];
        }
        epilogue8<TYPE>(p.ep, bias, residual, base, none, left, z);
    }
}

}  // namespace dft
