// lm_philox.cuh -- the counter-based generator of the dropout mask.
//
// Philox4x32-10 (J. Salmon, M. Moraes, R. Dror, D. Shaw, "Parallel random
// numbers: as easy as 1, 2, 3", SC 2011): ten rounds of two 32 x 32 -> 64
// products turn a 128-bit counter and a 64-bit key into 128 random bits.  No
// state is kept, so the backward pass makes the same mask again instead of
// reading a stored one.
//
// Element (r, c) of a tensor has 16 of those bits: halfword c % 8 of the block
// at counter {c / 8, r, lo(offset), hi(offset)} under the key `seed`.  It is
// kept where they are at least `drop`, p rounded to a multiple of 2^-16; the
// factor of the kept elements is that of the rounded p, so the expectation is
// exact.  16 bits an element rather than 32 because the wide multiplies would
// else bound the kernel: 2.5 an element now, at the 5.7 elements a clock that an
// SM's share of the memory bandwidth feeds a bf16 tensor read and written.
// The mask depends on (seed, offset, r, c) alone, not on strides or tiling.
#pragma once

#include <stdint.h>

namespace lm {
namespace {

struct Dropout {
    const uint64_t* rng;  // device {seed, offset}
    uint64_t offset;      // added to the offset on the device
    uint32_t drop;        // 0..65536: halfwords below it are dropped
    float scale;          // 65536 / (65536 - drop); 0 where everything is dropped
};

// The key and the offset's halves, read once by each thread.
struct PhiloxKey {
    uint32_t k0, k1, o0, o1;
};

__device__ __forceinline__ PhiloxKey philox_key(const Dropout& d) {
    const uint64_t seed = d.rng[0], off = d.rng[1] + d.offset;
    return {(uint32_t)seed, (uint32_t)(seed >> 32), (uint32_t)off, (uint32_t)(off >> 32)};
}

__device__ __forceinline__ void philox(const PhiloxKey& key, uint32_t c0, uint32_t c1,
                                       uint32_t (&out)[4]) {
    uint32_t c2 = key.o0, c3 = key.o1, k0 = key.k0, k1 = key.k1;
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = (uint64_t)0xD2511F53u * c0, b = (uint64_t)0xCD9E8D57u * c2;
        c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
        c1 = (uint32_t)b;
        c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
        c3 = (uint32_t)a;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    out[0] = c0, out[1] = c1, out[2] = c2, out[3] = c3;
}

// Bit j: whether element j of this lane's chunk stays.  base: the first of the
// warp's 256 columns (a multiple of 256).  Every lane of the warp calls it: without
// VEC each lane makes the bits of columns base + 8 lane .. + 7, and the bits
// that its own elements, base + 32 j + lane, need come from other lanes.
template <bool VEC>
__device__ __forceinline__ uint32_t keep_bits(const PhiloxKey& key, uint32_t drop, int64_t row,
                                              int64_t base, int lane) {
    uint32_t w[4];
    philox(key, (uint32_t)(base >> 3) + lane, (uint32_t)row, w);
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t h = (j & 1) ? w[j >> 1] >> 16 : w[j >> 1] & 0xFFFFu;
        m |= (h >= drop ? 1u : 0u) << j;
    }
    if (VEC) return m;
    uint32_t own = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t g = __shfl_sync(0xFFFFFFFFu, m, 4 * j + (lane >> 3));
        own |= ((g >> (lane & 7)) & 1u) << j;
    }
    return own;
}

}  // namespace
}  // namespace lm
