// lm_chunk.cuh -- how the row operators (layer norm, dropout) read and write a
// row: a warp takes 256 consecutive columns at a time and a lane eight of them,
// a "chunk", held in registers as it is stored (bf16: four words, fp32: eight).
//
//  - VEC: the row starts on a 16-byte (bf16) or 32-byte (fp32) boundary and has
//    a multiple of 8 columns.  Lane l holds columns base + 8 l .. + 7, one
//    16- or 32-byte access.
//  - otherwise (odd widths, rows at any alignment): lane l holds columns
//    base + 32 j + l, j = 0..7, so that each of the eight scalar accesses of a
//    warp is one contiguous run.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace lm {
namespace {

struct bf16_t {};  // tag of a tensor of IEEE bfloat16 bits
struct f32_t {};   // tag of a tensor of fp32

template <typename T>
struct Elem;
template <>
struct Elem<bf16_t> {
    using raw = uint16_t;
    static constexpr int kWords = 4;  // registers of a chunk
};
template <>
struct Elem<f32_t> {
    using raw = uint32_t;
    static constexpr int kWords = 8;
};

constexpr int kChunk = 8;               // columns of a lane
constexpr int kWarpCols = 32 * kChunk;  // columns of a warp's chunks
// Columns are counted in 32 bits; the last chunk's may pass the row's end by
// less than a block's 8192.
constexpr int64_t kMaxCols = int64_t(1) << 30;

template <typename T>
struct Chunk {
    uint32_t w[Elem<T>::kWords];
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// Element j of a chunk as fp32, and eight fp32 values rounded to a chunk (one
// rounding to nearest even for bf16).
__device__ __forceinline__ float get(const Chunk<bf16_t>& c, int j) {
    return __uint_as_float((j & 1) ? c.w[j >> 1] & 0xFFFF0000u : c.w[j >> 1] << 16);
}
__device__ __forceinline__ float get(const Chunk<f32_t>& c, int j) {
    return __uint_as_float(c.w[j]);
}
// Two fp32 in one register pair: the packed instructions do two IEEE operations in one
// issue slot.
struct F2 {
    uint64_t v;
};
__device__ __forceinline__ F2 make_f2(float lo, float hi) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float lo_of(F2 a) { return __uint_as_float((uint32_t)a.v); }
__device__ __forceinline__ float hi_of(F2 a) { return __uint_as_float((uint32_t)(a.v >> 32)); }
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

// Elements 2 i and 2 i + 1 of a chunk, and back.
constexpr int kPairs = kChunk / 2;
__device__ __forceinline__ F2 get2(const Chunk<bf16_t>& c, int i) {
    return make_f2(__uint_as_float(c.w[i] << 16), __uint_as_float(c.w[i] & 0xFFFF0000u));
}
__device__ __forceinline__ F2 get2(const Chunk<f32_t>& c, int i) {
    return make_f2(__uint_as_float(c.w[2 * i]), __uint_as_float(c.w[2 * i + 1]));
}
__device__ __forceinline__ void put2(Chunk<bf16_t>& c, int i, F2 v) {
    c.w[i] = pack_bf16(lo_of(v), hi_of(v));
}
__device__ __forceinline__ void put2(Chunk<f32_t>& c, int i, F2 v) {
    c.w[2 * i] = __float_as_uint(lo_of(v));
    c.w[2 * i + 1] = __float_as_uint(hi_of(v));
}
__device__ __forceinline__ void put(Chunk<bf16_t>& c, const float (&v)[kChunk]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c.w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
}
__device__ __forceinline__ void put(Chunk<f32_t>& c, const float (&v)[kChunk]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) c.w[i] = __float_as_uint(v[i]);
}

__device__ __forceinline__ void ld_vec(Chunk<bf16_t>& c, const void* p) {
    asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(c.w[0]), "=r"(c.w[1]), "=r"(c.w[2]), "=r"(c.w[3])
                 : "l"(p)
                 : "memory");
}
__device__ __forceinline__ void ld_vec(Chunk<f32_t>& c, const void* p) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(c.w[0]), "=r"(c.w[1]), "=r"(c.w[2]), "=r"(c.w[3]), "=r"(c.w[4]),
                   "=r"(c.w[5]), "=r"(c.w[6]), "=r"(c.w[7])
                 : "l"(p)
                 : "memory");
}
__device__ __forceinline__ void st_vec(void* p, const Chunk<bf16_t>& c) {
    asm volatile("st.global.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(c.w[0]), "r"(c.w[1]),
                 "r"(c.w[2]), "r"(c.w[3])
                 : "memory");
}
__device__ __forceinline__ void st_vec(void* p, const Chunk<f32_t>& c) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(c.w[0]),
                 "r"(c.w[1]), "r"(c.w[2]), "r"(c.w[3]), "r"(c.w[4]), "r"(c.w[5]), "r"(c.w[6]),
                 "r"(c.w[7])
                 : "memory");
}

// The column of element j of this lane's chunk.
template <bool VEC>
__device__ __forceinline__ int chunk_col(int base, int lane, int j) {
    return VEC ? base + kChunk * lane + j : base + 32 * j + lane;
}

// Whether this lane has a whole chunk (VEC), or any element of one, in a row
// of `cols` columns.  FULL: every lane has one (known when compiled).
template <bool VEC, bool FULL = false>
__device__ __forceinline__ bool chunk_has(int base, int lane, int cols) {
    return FULL || chunk_col<VEC>(base, lane, 0) < cols;
}

// This lane's chunk of the 256 columns at `base` of a row (nothing is read and
// the elements are zero past `cols`).
template <typename T, bool VEC, bool FULL = false>
__device__ __forceinline__ Chunk<T> load_chunk(const void* row, int base, int lane, int cols) {
    using raw = typename Elem<T>::raw;
    const raw* p = static_cast<const raw*>(row);
    Chunk<T> c;
    if constexpr (FULL) {
        ld_vec(c, p + base + kChunk * lane);
    } else {
#pragma unroll
        for (int i = 0; i < Elem<T>::kWords; ++i) c.w[i] = 0u;
        if constexpr (VEC) {
            if (chunk_has<true>(base, lane, cols)) ld_vec(c, p + base + kChunk * lane);
        } else {
#pragma unroll
            for (int j = 0; j < kChunk; ++j) {
                const int col = base + 32 * j + lane;
                const uint32_t v = col < cols ? (uint32_t)p[col] : 0u;
                if constexpr (sizeof(raw) == 4)
                    c.w[j] = v;
                else
                    c.w[j >> 1] |= v << (16 * (j & 1));
            }
        }
    }
    return c;
}

template <typename T, bool VEC, bool FULL = false>
__device__ __forceinline__ void store_chunk(void* row, int base, int lane, int cols,
                                            const Chunk<T>& c) {
    using raw = typename Elem<T>::raw;
    raw* p = static_cast<raw*>(row);
    if constexpr (VEC) {
        if (chunk_has<true, FULL>(base, lane, cols)) st_vec(p + base + kChunk * lane, c);
    } else {
#pragma unroll
        for (int j = 0; j < kChunk; ++j) {
            const int col = base + 32 * j + lane;
            if (col < cols) {
                if constexpr (sizeof(raw) == 4)
                    p[col] = c.w[j];
                else
                    p[col] = (raw)(c.w[j >> 1] >> (16 * (j & 1)));
            }
        }
    }
}

template <typename T>
__device__ __forceinline__ const void* row_at(const void* base, int64_t row, int64_t ld,
                                              int col = 0) {
    return static_cast<const typename Elem<T>::raw*>(base) + row * ld + col;
}
template <typename T>
__device__ __forceinline__ void* row_at(void* base, int64_t row, int64_t ld) {
    return static_cast<typename Elem<T>::raw*>(base) + row * ld;
}

}  // namespace
}  // namespace lm
