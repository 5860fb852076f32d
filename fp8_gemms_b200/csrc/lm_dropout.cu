// lm_dropout.cu -- dropout added to a residual stream, and its backward pass:
//
//   Y = residual + (keep ? x scale : 0),   dX = keep ? dY scale : 0
//
// with the mask of lm_philox.cuh, made again in the backward pass and never
// stored.  HBM-bound: x, residual and Y once each.
#include "lm_chunk.cuh"
#include "lm_internal.h"
#include "lm_philox.cuh"
#include "lm_rows.h"

namespace lm {
namespace {

struct DropArgs {
    const void *x, *residual;
    void* y;
    int64_t rows, cols, ldx, ldr, ldy;
    Dropout drop;
};

// A warp takes 256 columns of a row at a time.
template <typename T, bool VEC, bool ADD>
__global__ void __launch_bounds__(256) dropout_kernel(const DropArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t tiles_c = (a.cols + kWarpCols - 1) / kWarpCols;
    const int64_t tiles = a.rows * tiles_c;
    const PhiloxKey key = philox_key(a.drop);
    for (int64_t t = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); t < tiles;
         t += (int64_t)gridDim.x * 8) {
        const int64_t row = t / tiles_c, base = (t - row * tiles_c) * kWarpCols;
        Chunk<T> c = load_chunk<T, VEC>(row_at<T>(a.x, row, a.ldx), base, lane, a.cols), r;
        if (ADD) r = load_chunk<T, VEC>(row_at<T>(a.residual, row, a.ldr), base, lane, a.cols);
        const uint32_t keep = keep_bits<VEC>(key, a.drop.drop, row, base, lane);
        float v[kChunk];
#pragma unroll
        for (int j = 0; j < kChunk; ++j) {
            v[j] = (keep >> j) & 1 ? __fmul_rn(get(c, j), a.drop.scale) : 0.f;
            if (ADD) v[j] = __fadd_rn(get(r, j), v[j]);
        }
        put(c, v);
        store_chunk<T, VEC>(row_at<T>(a.y, row, a.ldy), base, lane, a.cols, c);
    }
}

template <typename T, bool ADD>
lm_status launch(const DropArgs& a, bool vec, cudaStream_t s) {
    const int sms = sm_count();
    if (sms <= 0) return LM_ERR_CUDA;
    const int64_t tiles = a.rows * ((a.cols + kWarpCols - 1) / kWarpCols);
    const int64_t want = (tiles + 7) / 8, most = (int64_t)sms * 8;
    const unsigned grid = (unsigned)(want < most ? want : most);
    timing_mark(s, 'd');
    if (vec)
        dropout_kernel<T, true, ADD><<<grid, 256, 0, s>>>(a);
    else
        dropout_kernel<T, false, ADD><<<grid, 256, 0, s>>>(a);
    return launch_status();
}

lm_status dropout(const DropArgs& a, lm_dtype dtype, lm_stream_t stream) {
    if (a.rows < 0 || a.cols <= 0 || (a.rows > 0 && (!a.x || !a.y))) return LM_ERR_INVALID_ARG;
    if (too_large(a.rows, a.cols)) return LM_ERR_UNSUPPORTED_SHAPE;
    const RowTensor ts[] = {{a.x, a.ldx, true}, {a.residual, a.ldr, true}, {a.y, a.ldy, true}};
    bool vec;
    const lm_status st = row_access(ts, 3, a.rows, a.cols, dtype, &vec);
    if (st != LM_OK || a.rows == 0) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == LM_DTYPE_BF16)
        return a.residual ? launch<bf16_t, true>(a, vec, s) : launch<bf16_t, false>(a, vec, s);
    return a.residual ? launch<f32_t, true>(a, vec, s) : launch<f32_t, false>(a, vec, s);
}

}  // namespace
}  // namespace lm

extern "C" {

lm_status lm_dropout_add_fwd(const void* X, int64_t ldx, const void* residual, int64_t ldr,
                             int64_t rows, int64_t cols, lm_dtype dtype, double p,
                             const uint64_t* rng, uint64_t offset, void* Y, int64_t ldy,
                             lm_stream_t stream) {
    lm::DropArgs a{};
    a.x = X, a.ldx = ldx, a.residual = residual, a.ldr = ldr, a.rows = rows, a.cols = cols;
    a.y = Y, a.ldy = ldy;
    const lm_status st = lm::dropout_args(p, rng, offset, &a.drop);
    return st != LM_OK ? st : lm::dropout(a, dtype, stream);
}

lm_status lm_dropout_add_bwd(const void* dY, int64_t lddy, int64_t rows, int64_t cols,
                             lm_dtype dtype, double p, const uint64_t* rng, uint64_t offset,
                             void* dX, int64_t lddx, lm_stream_t stream) {
    return lm_dropout_add_fwd(dY, lddy, nullptr, 0, rows, cols, dtype, p, rng, offset, dX, lddx,
                              stream);
}

}  // extern "C"
