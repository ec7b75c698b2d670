// dropout.hpp -- dropout whose mask is a function of a counter and is never
// stored.
//
// Philox4x32-10 (Salmon, Moraes, Dror, Shaw: Parallel random numbers: as easy
// as 1, 2, 3; 2011): ten rounds of two 32 by 32 bit products turn the counter
// (block, offset) under the key `seed` into 128 bits.  A block is eight
// consecutive elements of a row, row * ceil(cols / 8) + column / 8, and each
// element takes 16 of its bits, low halves first: an element is dropped when
// its 16-bit number is below drop = p * 65536 rounded to the nearest, and kept
// ones are scaled by 65536 / (65536 - drop), one over the share that is kept,
// so that the expectation is exact for the p that is drawn with.  16 bits
// rather than 32 halve the products, which would take longer than the bytes:
// 20 wide products per eight elements.
#pragma once

#include <stdint.h>

#include <hip/hip_runtime.h>

namespace dft {

struct Dropout {
    uint64_t seed, offset;
    const int64_t* step;  // added to offset when not nullptr (device)
    uint32_t drop;        // of 65536; 0: nothing is dropped
    float scale;          // of what is kept (0 when nothing is)
};

struct KeepBits {
    uint32_t w[4];
    // Element e of the block's eight.
    __host__ __device__ uint32_t number(int e) const { return e % 2 ? w[e / 2] >> 16 : w[e / 2] & 0xffffu; }
};

__host__ __device__ inline KeepBits philox(uint64_t seed, uint64_t offset, uint64_t block) {
    uint32_t c0 = (uint32_t)block, c1 = (uint32_t)(block >> 32), c2 = (uint32_t)offset, c3 = (uint32_t)(offset >> 32);
    uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
    for (int round = 0; round < 10; ++round) {
        const uint64_t m0 = (uint64_t)c0 * 0xD2511F53u, m1 = (uint64_t)c2 * 0xCD9E8D57u;
        c0 = (uint32_t)(m1 >> 32) ^ c1 ^ k0;
        c2 = (uint32_t)(m0 >> 32) ^ c3 ^ k1;
        c1 = (uint32_t)m1;
        c3 = (uint32_t)m0;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return KeepBits{{c0, c1, c2, c3}};
}

// The counter's offset of this launch.
__device__ inline uint64_t dropout_offset(const Dropout& d) {
    return d.step ? d.offset + (uint64_t)*d.step : d.offset;
}

// Eight elements of a block: zero where dropped, whatever they held.
__device__ inline void drop8(const Dropout& d, uint64_t offset, uint64_t block, float (&v)[8]) {
    const KeepBits bits = philox(d.seed, offset, block);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = bits.number(e) < d.drop ? 0.0f : v[e] * d.scale;
}

}  // namespace dft
