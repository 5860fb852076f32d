// lm_rows.h -- host-side checks shared by the row operators (layer norm,
// dropout): tensors of [rows x cols] with a row stride.
#pragma once

#include <math.h>

#include "lm_chunk.cuh"
#include "lm_internal.h"
#include "lm_philox.cuh"

namespace lm {
namespace {

inline bool aligned_to(const void* p, unsigned bytes) {
    return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

inline bool too_large(int64_t rows, int64_t cols) {
    return rows >= (int64_t(1) << 31) || cols > kMaxCols;
}

struct RowTensor {
    const void* p;  // NULL: absent
    int64_t ld;
    bool matrix;    // false: one row of `cols` elements
};

// Checks the tensors' types, strides and alignment, and whether all of them
// can be accessed a chunk (8 columns) at a time.
inline lm_status row_access(const RowTensor* ts, int n, int64_t rows, int64_t cols,
                            lm_dtype dtype, bool* vec) {
    if (dtype != LM_DTYPE_BF16 && dtype != LM_DTYPE_F32) return LM_ERR_UNSUPPORTED_FORMAT;
    const unsigned size = dtype == LM_DTYPE_BF16 ? 2 : 4;
    bool v = cols % 8 == 0;
    for (int i = 0; i < n; ++i) {
        const RowTensor& t = ts[i];
        if (!t.p) continue;
        if (t.matrix && rows > 1) {
            if (t.ld < cols) return LM_ERR_INVALID_ARG;
            if (t.ld >= (int64_t(1) << 31)) return LM_ERR_UNSUPPORTED_SHAPE;
            v = v && t.ld % 8 == 0;
        }
        if (!aligned_to(t.p, size)) return LM_ERR_ALIGNMENT;
        v = v && aligned_to(t.p, 8 * size);
    }
    *vec = v;
    return LM_OK;
}

// Whether an output may be where an input is: elsewhere, or the same rows.
inline bool in_place_or_apart(const RowTensor& out, const RowTensor& in, int64_t rows) {
    return !out.p || out.p != in.p || rows <= 1 || out.ld == in.ld;
}

// Whether two vectors of n bytes each have any in common (a NULL one has none).
inline bool share_bytes(const void* a, const void* b, int64_t n) {
    const uintptr_t p = reinterpret_cast<uintptr_t>(a), q = reinterpret_cast<uintptr_t>(b);
    return a && b && (p < q ? q - p : p - q) < (uintptr_t)n;
}

// The dropout of probability p: halfwords below round(p 2^16) are dropped.
inline lm_status dropout_args(double p, const uint64_t* rng, uint64_t offset, Dropout* d) {
    if (!(p >= 0.0 && p <= 1.0) || !rng) return LM_ERR_INVALID_ARG;
    if (!aligned_to(rng, 8)) return LM_ERR_ALIGNMENT;
    d->rng = rng;
    d->offset = offset;
    const uint32_t drop = (uint32_t)lrint(p * 65536.0);
    d->least = (drop < 65535u ? drop : 65535u) << 16;
    d->live = drop < 65536u;
    d->scale = drop < 65536u ? (float)(65536.0 / (65536.0 - drop)) : 0.f;
    return LM_OK;
}

}  // namespace
}  // namespace lm
