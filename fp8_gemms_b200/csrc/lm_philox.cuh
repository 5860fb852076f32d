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

#include "lm_chunk.cuh"

namespace lm {
namespace {

struct Dropout {
    const uint64_t* rng;  // device {seed, offset}
    uint64_t offset;      // added to the offset on the device
    // drop = 0..65536: halfwords below it are dropped.  It is held as what the upper half of a
    // word is compared with, min(drop, 65535) << 16, and whether anything is kept (0 for
    // drop = 65536).
    uint32_t least, live;
    float scale;  // 65536 / (65536 - drop); 0 where everything is dropped
};

// The key and the offset's halves, read once by each thread.
struct PhiloxKey {
    uint32_t k0, k1, o0, o1;
};

__device__ __forceinline__ PhiloxKey philox_key(const Dropout& d) {
    const uint64_t seed = d.rng[0], off = d.rng[1] + d.offset;
    return {(uint32_t)seed, (uint32_t)(seed >> 32), (uint32_t)off, (uint32_t)(off >> 32)};
}

// The same key, without what the compiler would keep of it across a loop: the ten
// rounds' keys are made again (two additions a round) instead of held in 20
// registers, for kernels that have none to spare.
__device__ __forceinline__ PhiloxKey renewed(const PhiloxKey& key) {
    PhiloxKey k = key;
    asm volatile("mov.b32 %0, %1;" : "=r"(k.k0) : "r"(key.k0));
    asm volatile("mov.b32 %0, %1;" : "=r"(k.k1) : "r"(key.k1));
    return k;
}

// The ten rounds' keys in registers, for kernels that have 20 to spare: made once a block
// and read from shared memory, or the compiler makes them again for each chunk.
struct PhiloxRounds {
    uint32_t k0[10], k1[10], o0, o1;
    // `keys`: shared, for one block; every thread calls it.
    __device__ __forceinline__ PhiloxRounds(const Dropout& d, uint2 (&keys)[10]) {
        const PhiloxKey key = philox_key(d);
        o0 = key.o0, o1 = key.o1;
        if (threadIdx.x < 10)
            keys[threadIdx.x] = make_uint2(key.k0 + threadIdx.x * 0x9E3779B9u,
                                           key.k1 + threadIdx.x * 0xBB67AE85u);
        __syncthreads();
#pragma unroll
        for (int r = 0; r < 10; ++r)
            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                         : "=r"(k0[r]), "=r"(k1[r])
                         : "r"((uint32_t)__cvta_generic_to_shared(&keys[r])));
    }
};
__device__ __forceinline__ uint32_t round_key0(const PhiloxKey& k, int r) { return k.k0 + r * 0x9E3779B9u; }
__device__ __forceinline__ uint32_t round_key1(const PhiloxKey& k, int r) { return k.k1 + r * 0xBB67AE85u; }
__device__ __forceinline__ uint32_t round_key0(const PhiloxRounds& k, int r) { return k.k0[r]; }
__device__ __forceinline__ uint32_t round_key1(const PhiloxRounds& k, int r) { return k.k1[r]; }

template <typename Key>
__device__ __forceinline__ void philox(const Key& key, uint32_t c0, uint32_t c1, uint32_t (&out)[4]) {
    uint32_t c2 = key.o0, c3 = key.o1;
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = (uint64_t)0xD2511F53u * c0, b = (uint64_t)0xCD9E8D57u * c2;
        c0 = (uint32_t)(b >> 32) ^ c1 ^ round_key0(key, r);
        c1 = (uint32_t)b;
        c2 = (uint32_t)(a >> 32) ^ c3 ^ round_key1(key, r);
        c3 = (uint32_t)a;
    }
    out[0] = c0, out[1] = c1, out[2] = c2, out[3] = c3;
}

// Which elements of this lane's chunk stay.  VEC: the lane's own four words.  Otherwise
// lane l makes the words of columns base + 8 l .. + 7, while its own elements are columns
// base + 32 j + l, whose bits come from other lanes: bit j of `bits`.
template <bool VEC>
struct Keep;
template <>
struct Keep<true> {
    uint32_t w[4];
};
template <>
struct Keep<false> {
    uint32_t bits;
};

// The eight elements of column group `group`: bit j for its column j.
template <typename Key>
__device__ __forceinline__ uint32_t group_bits(const Key& key, const Dropout& d, uint32_t row,
                                               uint32_t group) {
    uint32_t w[4], m = 0;
    philox(key, group, row, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        // the upper half as it is (what is below does not change the comparison), the
        // lower half moved up
        const uint32_t h = (j & 1) ? w[j >> 1] : w[j >> 1] << 16;
        m |= (h >= d.least && d.live ? 1u : 0u) << j;
    }
    return m;
}

// group: the row's eighth column group that this lane makes the words of, base / 8 + lane
// for the warp's 256 columns at `base`.  Every lane calls it.
template <bool VEC, typename Key>
__device__ __forceinline__ Keep<VEC> keep_at(const Key& key, const Dropout& d, uint32_t row,
                                             uint32_t group, int lane) {
    Keep<VEC> k;
    if constexpr (VEC) {
        philox(key, group, row, k.w);
    } else {
        const uint32_t m = group_bits(key, d, row, group);
        k.bits = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t g = __shfl_sync(0xFFFFFFFFu, m, 4 * j + (lane >> 3));
            k.bits |= ((g >> (lane & 7)) & 1u) << j;
        }
    }
    return k;
}

template <bool VEC>
__device__ __forceinline__ Keep<VEC> keep_of(const PhiloxKey& key, const Dropout& d, uint32_t row,
                                             int base, int lane) {
    return keep_at<VEC>(key, d, row, (uint32_t)(base >> 3) + lane, lane);
}

// Elements 2 i and 2 i + 1 of the chunk, zero where dropped.
__device__ __forceinline__ F2 kept(F2 v, const Keep<true>& k, const Dropout& d, int i) {
    return make_f2((k.w[i] << 16) >= d.least && d.live ? lo_of(v) : 0.f,
                   k.w[i] >= d.least && d.live ? hi_of(v) : 0.f);
}
__device__ __forceinline__ F2 kept(F2 v, const Keep<false>& k, const Dropout&, int i) {
    return make_f2((k.bits >> (2 * i)) & 1 ? lo_of(v) : 0.f,
                   (k.bits >> (2 * i + 1)) & 1 ? hi_of(v) : 0.f);
}

}  // namespace
}  // namespace lm
