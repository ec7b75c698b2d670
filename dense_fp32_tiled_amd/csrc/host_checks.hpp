// host_checks.hpp -- what the library's C entry points check on the host before
// anything is launched: the device, and the sizes, pitches, presence and
// overlaps of matrices.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <mutex>
#include <stdint.h>
#include <string.h>

#include "dense_fp32_tiled.h"

namespace dft {

// ---- the device ---------------------------------------------------------------------
constexpr int kMaxDevices = 64;
inline int g_cus[kMaxDevices];  // 0 unknown, -1 not gfx950, else compute units
inline std::mutex g_cus_mu;

inline int current_cus(int* cus) {
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return GEMM_ERR_HIP;
    if (dev < 0 || dev >= kMaxDevices) return GEMM_ERR_UNSUPPORTED;
    std::lock_guard<std::mutex> lock(g_cus_mu);
    if (g_cus[dev] == 0) {
        hipDeviceProp_t prop;
        if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return GEMM_ERR_HIP;
        g_cus[dev] = strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? prop.multiProcessorCount : -1;
    }
    if (g_cus[dev] < 0) return GEMM_ERR_UNSUPPORTED;
    *cus = g_cus[dev];
    return GEMM_OK;
}

// ---- argument checks ----------------------------------------------------------------
constexpr int64_t kMaxDim = (int64_t)1 << 40;  // products of a size, a pitch and an element's bytes stay inside int64
constexpr int64_t kMaxElements = (int64_t)1 << 59;
constexpr int64_t kMaxProduct = (int64_t)1 << 50;   // M N, M K, K N: 32 fp32 slices of one stay inside int64
constexpr int64_t kMaxOutPitch = (int64_t)1 << 26;  // 16 rows of fp32 stay inside the epilogue's 32-bit lane offsets
constexpr int64_t kMaxGrid = 0x7fffffff;

struct Matrix {
    const void* data;
    int64_t rows, cols, ld, elem, copies = 1, copy_stride = 0;

    bool empty() const { return rows == 0 || cols == 0 || copies == 0; }
    bool pitch_ok() const {
        if (ld < std::max<int64_t>(cols, 1)) return false;
        // (rows too long to count are refused by small_enough)
        return copies <= 1 || rows == 0 || rows > kMaxElements / ld || copy_stride >= (rows - 1) * ld + cols;
    }
    bool small_enough() const {
        return rows <= kMaxElements / ld && (copies <= 1 || copy_stride <= kMaxElements / copies);
    }
    int64_t bytes() const {
        return empty() ? 0 : ((copies - 1) * copy_stride + (rows - 1) * ld + cols) * elem;
    }
    bool overlaps(const Matrix& o) const {
        if (!data || !o.data || empty() || o.empty()) return false;
        const uintptr_t a = (uintptr_t)data, b = (uintptr_t)o.data;
        return a < b + (uintptr_t)o.bytes() && b < a + (uintptr_t)bytes();
    }
    bool same_place(const Matrix& o) const { return data == o.data && ld == o.ld && elem == o.elem; }
    // Every row starts on 16 bytes (and every copy).
    bool aligned16() const {
        return ((uintptr_t)data & 15) == 0 && ld % 8 == 0 && (copies <= 1 || copy_stride % 8 == 0);
    }
};

inline bool products_ok(int64_t m, int64_t n, int64_t k) {
    const auto ok = [](int64_t a, int64_t b) { return b == 0 || a <= kMaxProduct / b; };
    return ok(m, n) && ok(m, k) && ok(k, n);
}
inline bool out_pitch_ok(const Matrix& m) { return !m.data || m.rows <= 1 || m.ld <= kMaxOutPitch; }

// Pitches, sizes and presence of every matrix; an optional one may be NULL.
struct Use {
    Matrix m;
    bool optional, written;
};
inline int check_matrices(const Use* uses, int n) {
    for (int i = 0; i < n; ++i)
        if ((uses[i].m.data || !uses[i].optional) && !uses[i].m.pitch_ok()) return GEMM_ERR_INVALID_LD;
    for (int i = 0; i < n; ++i)
        if ((uses[i].m.data || !uses[i].optional) && !uses[i].m.small_enough()) return GEMM_ERR_TOO_LARGE;
    for (int i = 0; i < n; ++i)
        if (!uses[i].optional && !uses[i].m.empty() && !uses[i].m.data) return GEMM_ERR_NULL;
    for (int i = 0; i < n; ++i)
        for (int j = 0; j < n; ++j)
            if (i != j && uses[i].written && uses[i].m.overlaps(uses[j].m)) return GEMM_ERR_ALIAS;
    return GEMM_OK;
}

inline int64_t elem_bytes(int output_type) { return output_type == GEMM_OUTPUT_F32 ? 4 : 2; }
inline bool known_type(int input_type) { return input_type == GEMM_INPUT_BF16 || input_type == GEMM_INPUT_F16; }
inline bool known_output(int t) { return t == GEMM_OUTPUT_SAME || t == GEMM_OUTPUT_F32; }

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace dft
