// values8.hpp -- eight consecutive values of a row as one lane's access, for
// rows of 16- or 32-bit floats, and sums over a wave or a row's waves.
#pragma once

#include "linear_kernels.hpp"

namespace dft {

constexpr int kValueF32 = 2;  // beside kInputBf16 and kInputF16

// Eight values as they are in memory, `left` of them inside the row (WHOLE:
// all or none; zeros for what is not inside).
template <int TYPE>
struct Values8 {
    using element = uint16_t;
    Row8 raw;
    template <bool WHOLE>
    __device__ void load(const element* p, int64_t left) {
        if constexpr (WHOLE) {
            raw = Row8{};
            if (left > 0) __builtin_memcpy(&raw.w, p, sizeof(raw.w));
        } else {
            raw = load8(p, left);
        }
    }
    __device__ void widen(float (&v)[8]) const { raw.widen<TYPE>(v); }
    __device__ static Values8 narrow(const float (&v)[8]) { return Values8{Row8::narrow<TYPE>(v)}; }
    template <bool WHOLE>
    __device__ void store(element* p, int64_t left) const {
        if constexpr (WHOLE) {
            if (left > 0) __builtin_memcpy(p, &raw.w, sizeof(raw.w));
        } else {
            store8(p, raw, left);
        }
    }
};
template <>
struct Values8<kValueF32> {
    using element = float;
    float raw[8];
    template <bool WHOLE>
    __device__ void load(const element* p, int64_t left) {
        load8(raw, p, WHOLE ? (left > 0 ? 8 : 0) : left);
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
    template <bool WHOLE>
    __device__ void store(element* p, int64_t left) const {
        if (!WHOLE || left > 0) store8(p, raw, WHOLE ? 8 : left);
    }
};

__device__ inline float wave_sum(float v) {
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) v += __shfl_xor(v, d);
    return v;
}

}  // namespace dft
