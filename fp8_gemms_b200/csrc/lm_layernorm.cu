// lm_layernorm.cu -- layer norm, forward and backward, alone or behind dropout
// and a residual add:
//
//   s = residual + dropout(x)               (or s = x), rounded to its type
//   m = mean(s), v = mean((s - m)^2), r = 1 / sqrt(v + eps), h = (s - m) r
//   y = h w + b
//
//   g = dy w;  ds' = r (g - mean(g) - h mean(g h));  dw = sum dy h;  db = sum dy
//   dresidual = ds + ds';  dx = dropout(dresidual), the forward's mask made again
//
// All sums are fp32; the variance is that of the centred values (a second sweep),
// so a large mean costs no digits.  The norm's backward sums over the rows
// go through per-block partial sums in the workspace and a second kernel, in a
// fixed order: no atomics, the same bits from call to call.
#include "lm_chunk.cuh"
#include "lm_internal.h"
#include "lm_philox.cuh"
#include "lm_rows.h"

namespace lm {
namespace {

constexpr int kMaxParts = 296;  // partial sums of the weight gradients, at most

struct FwdArgs {
    const void *x, *residual, *weight, *bias;
    void *s, *y;
    int64_t rows, cols, ldx, ldr, lds, ldy;
    float eps;
    float *mean, *rstd;
    unsigned int* amax;  // fp32 bits, max-reduced; or NULL
    Dropout drop;
};

struct BwdArgs {
    const void *dy, *ds, *s, *weight;
    const float *mean, *rstd;
    void *dx, *dres;
    int64_t rows, cols, lddy, ldds, lds, lddx, lddr;
    Dropout drop;
};

// Sum over the block, the same in every thread.  `buf`: a float per warp.
__device__ __forceinline__ float block_sum(float v, float* buf) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    const int warps = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
    for (int i = 0; i < warps; ++i) v += buf[i];
    __syncthreads();
    return v;
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// One block a row, the row read again for each sweep: for rows that do not fit
// a block's registers.
template <typename T, bool VEC, bool DROP>
__global__ void __launch_bounds__(256) norm_fwd_wide_kernel(const FwdArgs a) {
    __shared__ float buf[8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = blockIdx.x;
    const void* x = row_at<T>(a.x, row, a.ldx);
    const void* s = DROP ? row_at<T>(static_cast<const void*>(a.s), row, a.lds) : x;
    PhiloxKey key{};
    if (DROP) key = philox_key(a.drop);
    float sum = 0.f;
    for (int64_t base = warp * kWarpCols; base < a.cols; base += 8 * kWarpCols) {
        Chunk<T> c = load_chunk<T, VEC>(x, base, lane, a.cols);
        if (DROP) {
            const Chunk<T> r =
                load_chunk<T, VEC>(row_at<T>(a.residual, row, a.ldr), base, lane, a.cols);
            const uint32_t keep = keep_bits<VEC>(key, a.drop.drop, row, base, lane);
            float v[kChunk];
#pragma unroll
            for (int j = 0; j < kChunk; ++j)
                v[j] = __fadd_rn(get(r, j),
                                 (keep >> j) & 1 ? __fmul_rn(get(c, j), a.drop.scale) : 0.f);
            put(c, v);
            store_chunk<T, VEC>(row_at<T>(a.s, row, a.lds), base, lane, a.cols, c);
        }
#pragma unroll
        for (int j = 0; j < kChunk; ++j) sum += get(c, j);
    }
    const float mean = __fdiv_rn(block_sum(sum, buf), (float)a.cols);
    float sq = 0.f;
    for (int64_t base = warp * kWarpCols; base < a.cols; base += 8 * kWarpCols) {
        const Chunk<T> c = load_chunk<T, VEC>(s, base, lane, a.cols);
#pragma unroll
        for (int j = 0; j < kChunk; ++j)
            if (chunk_col<VEC>(base, lane, j) < a.cols) {
                const float d = get(c, j) - mean;
                sq = __fmaf_rn(d, d, sq);
            }
    }
    const float var = __fdiv_rn(block_sum(sq, buf), (float)a.cols);
    const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(var, a.eps)));
    if (threadIdx.x == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
    }
    uint32_t top = 0;
    for (int64_t base = warp * kWarpCols; base < a.cols; base += 8 * kWarpCols) {
        Chunk<T> c = load_chunk<T, VEC>(s, base, lane, a.cols), w, b;
        if (a.weight) w = load_chunk<T, VEC>(a.weight, base, lane, a.cols);
        if (a.bias) b = load_chunk<T, VEC>(a.bias, base, lane, a.cols);
        float v[kChunk];
#pragma unroll
        for (int j = 0; j < kChunk; ++j) {
            v[j] = (get(c, j) - mean) * rstd;
            v[j] = __fmaf_rn(v[j], a.weight ? get(w, j) : 1.f, a.bias ? get(b, j) : 0.f);
        }
        put(c, v);
        if (a.amax) {
#pragma unroll
            for (int j = 0; j < kChunk; ++j)
                if (chunk_col<VEC>(base, lane, j) < a.cols) top = max(top, abs_bits(get(c, j)));
        }
        store_chunk<T, VEC>(row_at<T>(a.y, row, a.ldy), base, lane, a.cols, c);
    }
    if (a.amax) {
        top = __reduce_max_sync(0xFFFFFFFFu, top);
        if (lane == 0 && top) atomicMax(a.amax, top);
    }
}

template <typename T, bool VEC, bool DROP>
__global__ void __launch_bounds__(256) norm_bwd_wide_kernel(const BwdArgs a) {
    __shared__ float buf[8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = blockIdx.x;
    const void* dy = row_at<T>(a.dy, row, a.lddy);
    const void* s = row_at<T>(a.s, row, a.lds);
    const float mean = a.mean[row], rstd = a.rstd[row];
    float c1 = 0.f, c2 = 0.f;
    for (int64_t base = warp * kWarpCols; base < a.cols; base += 8 * kWarpCols) {
        const Chunk<T> d = load_chunk<T, VEC>(dy, base, lane, a.cols);
        const Chunk<T> c = load_chunk<T, VEC>(s, base, lane, a.cols);
        Chunk<T> w;
        if (a.weight) w = load_chunk<T, VEC>(a.weight, base, lane, a.cols);
#pragma unroll
        for (int j = 0; j < kChunk; ++j) {
            const float g = a.weight ? get(d, j) * get(w, j) : get(d, j);
            if (chunk_col<VEC>(base, lane, j) < a.cols) {
                c1 += g;
                c2 = __fmaf_rn(g, (get(c, j) - mean) * rstd, c2);
            }
        }
    }
    c1 = __fdiv_rn(block_sum(c1, buf), (float)a.cols);
    c2 = __fdiv_rn(block_sum(c2, buf), (float)a.cols);
    PhiloxKey key{};
    if (DROP) key = philox_key(a.drop);
    for (int64_t base = warp * kWarpCols; base < a.cols; base += 8 * kWarpCols) {
        const Chunk<T> d = load_chunk<T, VEC>(dy, base, lane, a.cols);
        const Chunk<T> c = load_chunk<T, VEC>(s, base, lane, a.cols);
        Chunk<T> w, up, out;
        if (a.weight) w = load_chunk<T, VEC>(a.weight, base, lane, a.cols);
        if (a.ds) up = load_chunk<T, VEC>(row_at<T>(a.ds, row, a.ldds), base, lane, a.cols);
        float v[kChunk];
#pragma unroll
        for (int j = 0; j < kChunk; ++j) {
            const float g = a.weight ? get(d, j) * get(w, j) : get(d, j);
            const float h = (get(c, j) - mean) * rstd;
            v[j] = (g - c1 - h * c2) * rstd;
            if (a.ds) v[j] = get(up, j) + v[j];
        }
        put(out, v);
        store_chunk<T, VEC>(row_at<T>(a.dres, row, a.lddr), base, lane, a.cols, out);
        if (DROP) {
            const uint32_t keep = keep_bits<VEC>(key, a.drop.drop, row, base, lane);
#pragma unroll
            for (int j = 0; j < kChunk; ++j) v[j] = (keep >> j) & 1 ? v[j] * a.drop.scale : 0.f;
            put(out, v);
            store_chunk<T, VEC>(row_at<T>(a.dx, row, a.lddx), base, lane, a.cols, out);
        }
    }
}

// Partial sums over the rows: block (i, p) sums columns 256 i .. + 255 over the
// rows of part p into part[p][0] (dw) and part[p][1] (db).
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) norm_wgrad_kernel(const BwdArgs a, float* part) {
    __shared__ float sum[2][8][kWarpCols];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t base = (int64_t)blockIdx.x * kWarpCols;
    float dw[kChunk] = {}, db[kChunk] = {};
    for (int64_t row = (int64_t)blockIdx.y * 8 + warp; row < a.rows; row += (int64_t)gridDim.y * 8) {
        const Chunk<T> d = load_chunk<T, VEC>(row_at<T>(a.dy, row, a.lddy), base, lane, a.cols);
        const Chunk<T> c = load_chunk<T, VEC>(row_at<T>(a.s, row, a.lds), base, lane, a.cols);
        const float mean = a.mean[row], rstd = a.rstd[row];
#pragma unroll
        for (int j = 0; j < kChunk; ++j) {
            dw[j] = __fmaf_rn(get(d, j), (get(c, j) - mean) * rstd, dw[j]);
            db[j] += get(d, j);
        }
    }
#pragma unroll
    for (int j = 0; j < kChunk; ++j) {
        const int col = (int)chunk_col<VEC>(0, lane, j);
        sum[0][warp][col] = dw[j];
        sum[1][warp][col] = db[j];
    }
    __syncthreads();
    if (base + threadIdx.x < a.cols) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float t = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) t += sum[k][i][threadIdx.x];
            part[((int64_t)blockIdx.y * 2 + k) * a.cols + base + threadIdx.x] = t;
        }
    }
}

// dw (blockIdx.y 0) and db (1): the parts' sums, eight at a time by the
// eight warps of a block that takes 32 columns.
template <typename T, bool ACCUM>
__global__ void __launch_bounds__(256) norm_wgrad_sum_kernel(const float* part, int parts,
                                                             int64_t cols, void* dweight,
                                                             void* dbias) {
    __shared__ float sum[8][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    void* out = blockIdx.y ? dbias : dweight;
    if (!out) return;
    const int64_t col = (int64_t)blockIdx.x * 32 + lane;
    float t = 0.f;
    if (col < cols)
        for (int p = warp; p < parts; p += 8) t += part[((int64_t)p * 2 + blockIdx.y) * cols + col];
    sum[warp][lane] = t;
    __syncthreads();
    if (warp == 0 && col < cols) {
        t = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) t += sum[i][lane];
        if (ACCUM)
            static_cast<float*>(out)[col] += t;
        else if (sizeof(typename Elem<T>::raw) == 4)
            static_cast<float*>(out)[col] = t;
        else
            static_cast<uint16_t*>(out)[col] = (uint16_t)pack_bf16(t, 0.f);
    }
}

template <typename T, bool VEC, bool DROP>
lm_status launch_fwd(const FwdArgs& a, cudaStream_t s) {
    timing_mark(s, 'n');
    norm_fwd_wide_kernel<T, VEC, DROP><<<(unsigned)a.rows, 256, 0, s>>>(a);
    return launch_status();
}

template <typename T, bool VEC, bool DROP>
lm_status launch_bwd(const BwdArgs& a, void* dweight, void* dbias, bool accum, float* part,
                     cudaStream_t s) {
    int parts = 0;
    if (a.rows > 0) {
        // the weight gradients first: they read dy and s, which dx may overwrite
        if (dweight || dbias) {
            const int64_t tiles = (a.cols + kWarpCols - 1) / kWarpCols;
            parts = (int)((a.rows + 31) / 32 < kMaxParts ? (a.rows + 31) / 32 : kMaxParts);
            timing_mark(s, 'n');
            norm_wgrad_kernel<T, VEC>
                <<<dim3((unsigned)tiles, (unsigned)parts), 256, 0, s>>>(a, part);
            if (launch_status() != LM_OK) return LM_ERR_CUDA;
        }
        timing_mark(s, 'n');
        norm_bwd_wide_kernel<T, VEC, DROP><<<(unsigned)a.rows, 256, 0, s>>>(a);
        if (launch_status() != LM_OK) return LM_ERR_CUDA;
    }
    if (!(dweight || dbias) || (accum && a.rows == 0)) return LM_OK;
    const dim3 grid((unsigned)((a.cols + 31) / 32), 2);
    timing_mark(s, 'n');
    if (accum)
        norm_wgrad_sum_kernel<T, true><<<grid, 256, 0, s>>>(part, parts, a.cols, dweight, dbias);
    else
        norm_wgrad_sum_kernel<T, false><<<grid, 256, 0, s>>>(part, parts, a.cols, dweight, dbias);
    return launch_status();
}

bool bad_sizes(int64_t rows, int64_t cols) { return rows < 0 || cols <= 0; }

size_t ws_bytes_for(int64_t rows, int64_t cols) {
    if (bad_sizes(rows, cols) || too_large(rows, cols)) return 0;
    const int64_t parts = rows < kMaxParts ? (rows ? rows : 1) : kMaxParts;
    return (size_t)parts * 2 * (size_t)cols * sizeof(float);
}

lm_status fwd(FwdArgs a, lm_dtype dtype, bool drop, lm_stream_t stream) {
    if (bad_sizes(a.rows, a.cols) || !(a.eps >= 0.f)) return LM_ERR_INVALID_ARG;
    if (a.rows > 0 && (!a.x || !a.y || (drop && (!a.residual || !a.s)))) return LM_ERR_INVALID_ARG;
    if (too_large(a.rows, a.cols)) return LM_ERR_UNSUPPORTED_SHAPE;
    const RowTensor ts[] = {{a.x, a.ldx, true},      {a.residual, a.ldr, true},
                            {a.s, a.lds, true},      {a.y, a.ldy, true},
                            {a.weight, a.cols, false}, {a.bias, a.cols, false}};
    bool vec;
    lm_status st = row_access(ts, 6, a.rows, a.cols, dtype, &vec);
    if (st != LM_OK) return st;
    if (!aligned_to(a.mean, 4) || !aligned_to(a.rstd, 4) || !aligned_to(a.amax, 4))
        return LM_ERR_ALIGNMENT;
    if (a.rows == 0) return LM_OK;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool bf16 = dtype == LM_DTYPE_BF16;
    if (drop) {
        if (bf16)
            return vec ? launch_fwd<bf16_t, true, true>(a, s) : launch_fwd<bf16_t, false, true>(a, s);
        return vec ? launch_fwd<f32_t, true, true>(a, s) : launch_fwd<f32_t, false, true>(a, s);
    }
    if (bf16)
        return vec ? launch_fwd<bf16_t, true, false>(a, s) : launch_fwd<bf16_t, false, false>(a, s);
    return vec ? launch_fwd<f32_t, true, false>(a, s) : launch_fwd<f32_t, false, false>(a, s);
}

lm_status bwd(BwdArgs a, lm_dtype dtype, bool drop, void* dweight, void* dbias, void* workspace,
              size_t ws_bytes, uint32_t flags, lm_stream_t stream) {
    if (bad_sizes(a.rows, a.cols) || (flags & ~LM_NORM_ACCUMULATE_WGRAD)) return LM_ERR_INVALID_ARG;
    if (a.rows > 0 && (!a.dy || !a.s || !a.mean || !a.rstd || !a.dres || (drop && !a.dx)))
        return LM_ERR_INVALID_ARG;
    if (too_large(a.rows, a.cols)) return LM_ERR_UNSUPPORTED_SHAPE;
    if ((dweight || dbias) &&
        (!workspace || ws_bytes < ws_bytes_for(a.rows, a.cols)))
        return LM_ERR_INVALID_ARG;
    const RowTensor ts[] = {{a.dy, a.lddy, true},   {a.ds, a.ldds, true},
                            {a.s, a.lds, true},     {a.dx, a.lddx, true},
                            {a.dres, a.lddr, true}, {a.weight, a.cols, false}};
    bool vec;
    lm_status st = row_access(ts, 6, a.rows, a.cols, dtype, &vec);
    if (st != LM_OK) return st;
    const bool accum = flags & LM_NORM_ACCUMULATE_WGRAD;
    const unsigned size = accum || dtype == LM_DTYPE_F32 ? 4 : 2;
    if (!aligned_to(dweight, size) || !aligned_to(dbias, size) || !aligned16(workspace) ||
        !aligned_to(a.mean, 4) || !aligned_to(a.rstd, 4))
        return LM_ERR_ALIGNMENT;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    float* part = static_cast<float*>(workspace);
    const bool bf16 = dtype == LM_DTYPE_BF16;
    if (drop) {
        if (bf16)
            return vec ? launch_bwd<bf16_t, true, true>(a, dweight, dbias, accum, part, s)
                       : launch_bwd<bf16_t, false, true>(a, dweight, dbias, accum, part, s);
        return vec ? launch_bwd<f32_t, true, true>(a, dweight, dbias, accum, part, s)
                   : launch_bwd<f32_t, false, true>(a, dweight, dbias, accum, part, s);
    }
    if (bf16)
        return vec ? launch_bwd<bf16_t, true, false>(a, dweight, dbias, accum, part, s)
                   : launch_bwd<bf16_t, false, false>(a, dweight, dbias, accum, part, s);
    return vec ? launch_bwd<f32_t, true, false>(a, dweight, dbias, accum, part, s)
               : launch_bwd<f32_t, false, false>(a, dweight, dbias, accum, part, s);
}

}  // namespace
}  // namespace lm

extern "C" {

lm_status lm_layernorm_fwd(const void* X, int64_t ldx, const void* weight, const void* bias,
                           int64_t rows, int64_t cols, float eps, lm_dtype dtype, void* Y,
                           int64_t ldy, float* mean, float* rstd, float* amax_out,
                           lm_stream_t stream) {
    lm::FwdArgs a{};
    a.x = X, a.ldx = ldx, a.weight = weight, a.bias = bias, a.rows = rows, a.cols = cols;
    a.eps = eps, a.y = Y, a.ldy = ldy, a.mean = mean, a.rstd = rstd;
    a.amax = reinterpret_cast<unsigned int*>(amax_out);
    return lm::fwd(a, dtype, false, stream);
}

lm_status lm_dropout_add_layernorm_fwd(const void* X, int64_t ldx, const void* residual,
                                       int64_t ldr, const void* weight, const void* bias,
                                       int64_t rows, int64_t cols, float eps, lm_dtype dtype,
                                       double p, const uint64_t* rng, uint64_t offset, void* S,
                                       int64_t lds, void* Y, int64_t ldy, float* mean,
                                       float* rstd, float* amax_out, lm_stream_t stream) {
    lm::FwdArgs a{};
    a.x = X, a.ldx = ldx, a.residual = residual, a.ldr = ldr, a.weight = weight, a.bias = bias;
    a.rows = rows, a.cols = cols, a.eps = eps, a.s = S, a.lds = lds, a.y = Y, a.ldy = ldy;
    a.mean = mean, a.rstd = rstd, a.amax = reinterpret_cast<unsigned int*>(amax_out);
    const lm_status st = lm::dropout_args(p, rng, offset, &a.drop);
    return st != LM_OK ? st : lm::fwd(a, dtype, true, stream);
}

size_t lm_layernorm_workspace_size(int64_t rows, int64_t cols) {
    return lm::ws_bytes_for(rows, cols);
}

lm_status lm_layernorm_bwd(const void* dY, int64_t lddy, const void* X, int64_t ldx,
                           const void* weight, const float* mean, const float* rstd, int64_t rows,
                           int64_t cols, lm_dtype dtype, void* dX, int64_t lddx, void* dweight,
                           void* dbias, void* workspace, size_t ws_bytes, uint32_t flags,
                           lm_stream_t stream) {
    lm::BwdArgs a{};
    a.dy = dY, a.lddy = lddy, a.s = X, a.lds = ldx, a.weight = weight, a.mean = mean;
    a.rstd = rstd, a.rows = rows, a.cols = cols, a.dres = dX, a.lddr = lddx;
    return lm::bwd(a, dtype, false, dweight, dbias, workspace, ws_bytes, flags, stream);
}

lm_status lm_dropout_add_layernorm_bwd(const void* dY, int64_t lddy, const void* dS, int64_t ldds,
                                       const void* S, int64_t lds, const void* weight,
                                       const float* mean, const float* rstd, int64_t rows,
                                       int64_t cols, lm_dtype dtype, double p,
                                       const uint64_t* rng, uint64_t offset, void* dX,
                                       int64_t lddx, void* dR, int64_t lddr, void* dweight,
                                       void* dbias, void* workspace, size_t ws_bytes,
                                       uint32_t flags, lm_stream_t stream) {
    lm::BwdArgs a{};
    a.dy = dY, a.lddy = lddy, a.ds = dS, a.ldds = ldds, a.s = S, a.lds = lds, a.weight = weight;
    a.mean = mean, a.rstd = rstd, a.rows = rows, a.cols = cols, a.dx = dX, a.lddx = lddx;
    a.dres = dR, a.lddr = lddr;
    const lm_status st = lm::dropout_args(p, rng, offset, &a.drop);
    return st != LM_OK ? st
                       : lm::bwd(a, dtype, true, dweight, dbias, workspace, ws_bytes, flags, stream);
}

}  // extern "C"
