// values8.hpp -- eight consecutive values of a row as one lane's access, for
// rows of 16- or 32-bit floats, and sums over a wave or a row's waves.
#pragma once

#include "linear_kernels.hpp"

namespace dft {

constexpr int kValueF32 = 2;  // beside kInputBf16 and kInputF16

// Eight values as they are in memory.  `load` and `store` take `left` of them
// that lie inside the row, at any number.  `load_at` and `store_at` take the
// place `at` in a row of `cols` at `row` (uniform, so that a lane's address is
// one offset): WHOLE, of cols a multiple of 8, and any cols of 8 or more, where
// a row's last values are read with those before them and shifted down, one
// access for all lanes.  What is not inside reads as zeros.
template <int TYPE>
struct Values8 {
    using element = uint16_t;
    Row8 raw;
    __device__ void load(const element* p, int64_t left) { raw = load8(p, left); }
    __device__ void store(element* p, int64_t left) const { store8(p, raw, left); }
    template <bool WHOLE>
    __device__ void load_at(const element* row, int at, int cols) {
        if constexpr (WHOLE) {
            raw = Row8{};
            if (at < cols) __builtin_memcpy(&raw.w, row + at, sizeof(raw.w));
        } else {
            const int from = at < cols - 8 ? at : cols - 8, by = at - from;
            __builtin_memcpy(&raw.w, row + from, sizeof(raw.w));
            if (__ballot(by != 0)) {
                u32x4& w = raw.w;
                if (by & 4) w = u32x4{w[2], w[3], 0, 0};
                if (by & 2) w = u32x4{w[1], w[2], w[3], 0};
                if (by & 1)
                    w = u32x4{w[0] >> 16 | w[1] << 16, w[1] >> 16 | w[2] << 16, w[2] >> 16 | w[3] << 16, w[3] >> 16};
                if (by >= 8) w = u32x4{0, 0, 0, 0};
            }
        }
    }
    template <bool WHOLE>
    __device__ void store_at(element* row, int at, int cols) const {
        if (WHOLE ? at < cols : at + 8 <= cols) {
            __builtin_memcpy(row + at, &raw.w, sizeof(raw.w));
        } else if (!WHOLE && at < cols) {
#pragma unroll
            for (int e = 0; e < 7; ++e)
                if (at + e < cols) row[at + e] = (uint16_t)(raw.w[e / 2] >> (e % 2 * 16));
        }
    }
    // The same values, which the compiler may not know to be: what is computed from them is computed again.
    __device__ void afresh() { asm volatile("" : "+v"(raw.w)); }
    __device__ void widen(float (&v)[8]) const { raw.widen<TYPE>(v); }
    __device__ static Values8 narrow(const float (&v)[8]) { return Values8{Row8::narrow<TYPE>(v)}; }
};
template <>
struct Values8<kValueF32> {
    using element = float;
    float raw[8];
    __device__ void load(const element* p, int64_t left) { load8(raw, p, left); }
    __device__ void store(element* p, int64_t left) const { store8(p, raw, left); }
    template <bool WHOLE>
    __device__ void load_at(const element* row, int at, int cols) {
        if constexpr (WHOLE) {
            load8(raw, row + at, at < cols ? 8 : 0);
        } else {
            const int from = at < cols - 8 ? at : cols - 8, by = at - from;
            load8(raw, row + from, 8);
            if (__ballot(by != 0)) {
#pragma unroll
                for (int step = 4; step > 0; step /= 2)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (by & step) raw[e] = e + step < 8 ? raw[e + step] : 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (by >= 8) raw[e] = 0.0f;
            }
        }
    }
    template <bool WHOLE>
    __device__ void store_at(element* row, int at, int cols) const {
        if (WHOLE ? at < cols : at + 8 <= cols) {
            store8(row + at, raw, 8);
        } else if (!WHOLE && at < cols) {
#pragma unroll
            for (int e = 0; e < 7; ++e)
                if (at + e < cols) row[at + e] = raw[e];
        }
    }
    __device__ void afresh() {
#pragma unroll
        for (int e = 0; e < 8; ++e) asm volatile("" : "+v"(raw[e]));
    }
    __device__ void widen(float (&v)[8]) const {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = raw[e];
    }
    __device__ static Values8 narrow(const float (&v)[8]) {
        Values8 r;
#pragma unroll
        for (int e = 0; e < 8; ++e) r.raw[e] = v[e];
        return r;
    }
};

// Eight times the same value.
template <class V>
__device__ inline V all8(float x) {
    const float v[8] = {x, x, x, x, x, x, x, x};
    return V::narrow(v);
}

__device__ inline float wave_sum(float v) {
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) v += __shfl_xor(v, d);
    return v;
}

}  // namespace dft
