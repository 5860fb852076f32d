// lm_dropout.cu -- dropout added to a residual stream, and its backward pass:
//
//   Y = residual + (keep ? x scale : 0),   dX = keep ? dY scale : 0
//
// with the mask of lm_philox.cuh, made again in the backward pass and never
// stored.  x, residual and Y move once each, which bounds it (HBM) beside a
// residual; without one the generator and the selections come close (the ALU pipe 65%
// busy, 28.6 M warp instructions for 16384 x 4096 against 43 M before the whole-tile kernel).
// One B200, back to back for some ms, of a copy's 6.46 TB/s: 16384 x 12288 bf16 125 us (100%),
// with a residual 171 us (110%); 8192 x 8192 fp32 78 us (107%).  Odd bf16
// widths, each row at another alignment: 16384 x 4095 69 us (61%; the generator and the bits'
// way to their elements), with a residual 83 us (75%), by 2-byte accesses 119 and 148.
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

// Tiles of a warp: 16 KB of loads a block for either type.
template <typename T>
__host__ __device__ constexpr int tiles_of_warp() {
    return sizeof(typename Elem<T>::raw) == 2 ? 4 : 2;
}

// One chunk: y = (residual +) (keep ? x scale : 0), in place of c.
template <bool ADD, typename T, bool VEC>
__device__ __forceinline__ void drop_chunk(Chunk<T>& c, const Chunk<T>& r, const Keep<VEC>& keep,
                                           const Dropout& d) {
    const F2 scale = make_f2(d.scale, d.scale);
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
        const F2 v = kept(mul2(get2(c, j), scale), keep, d, j);
        put2(c, j, ADD ? add2(get2(r, j), v) : v);
    }
}

// Rows of a whole number of warps' work (kTiles x 256 columns): a warp takes that many
// columns of one row, with no tests and one address.  The generator and the
// selections bound this kernel (the ALU pipe), so every instruction counts.
template <typename T, bool ADD>
__global__ void __launch_bounds__(256) dropout_full_kernel(const DropArgs a, uint32_t across) {
    constexpr int kTiles = tiles_of_warp<T>();
    __shared__ uint2 keys[10];
    const int lane = threadIdx.x & 31;
    const int64_t task = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int64_t row = task >> 32 == 0 ? (uint32_t)task / across : task / across;
    const int first = (int)(task - row * across) * kTiles * kWarpCols;
    const bool in = row < a.rows;
    Chunk<T> c[kTiles], r[kTiles];
    if (in) {
        const void* const x = row_at<T>(a.x, row, a.ldx, first);
        const void* const res = ADD ? row_at<T>(a.residual, row, a.ldr, first) : nullptr;
#pragma unroll
        for (int k = 0; k < kTiles; ++k) {
            c[k] = load_chunk<T, true, true>(x, k * kWarpCols, lane, 0);
            if (ADD) r[k] = load_chunk<T, true, true>(res, k * kWarpCols, lane, 0);
        }
    }
    // beside a residual there are no registers for the rounds' keys
    const auto key = [&] {
        if constexpr (ADD)
            return philox_key(a.drop);
        else
            return PhiloxRounds(a.drop, keys);
    }();
    if (!in) return;
    char* const y = static_cast<char*>(row_at<T>(a.y, row, a.ldy)) +
                    (int64_t)first * sizeof(typename Elem<T>::raw);
#pragma unroll
    for (int k = 0; k < kTiles; ++k) {
        const Keep<true> keep = keep_at<true>(key, a.drop, (uint32_t)row,
                                              (uint32_t)(first >> 3) + 32 * k + lane, lane);
        drop_chunk<ADD>(c[k], r[k], keep, a.drop);
        store_chunk<T, true, true>(y, k * kWarpCols, lane, 0, c[k]);
    }
}

// Any rows.  A tile is 256 columns of a row, or with VEC and rows of at most 128 columns as
// many whole rows as a warp has lanes for.  A warp takes a few tiles that follow one
// another, loads them all, and makes the masks while the loads are on their way.
// `across`: tiles of a row; `rows_in`: rows of a tile.
template <typename T, bool VEC, bool ADD>
__global__ void __launch_bounds__(256) dropout_kernel(const DropArgs a, int across, int rows_in) {
    constexpr int kTiles = tiles_of_warp<T>();
    const int lane = threadIdx.x & 31, cols = (int)a.cols, groups = cols >> 3;
    const int sub = rows_in > 1 ? lane / groups : 0;
    const int group = rows_in > 1 ? lane - sub * groups : lane;
    const int64_t first = ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)) * kTiles;
    int64_t row = first >> 32 == 0 ? (uint32_t)first / (uint32_t)across : first / across;
    int tile = (int)(first - row * across);
    row = row * rows_in + sub;
    Chunk<T> c[kTiles], r[kTiles];
    int64_t at[kTiles];
    int base[kTiles];
    bool has[kTiles];
#pragma unroll
    for (int k = 0; k < kTiles; ++k) {
        at[k] = row;
        base[k] = tile * kWarpCols;
        const bool in = row < a.rows;
        has[k] = VEC ? in && sub < rows_in && base[k] + kChunk * group < cols : in;
        if (VEC) {
            if (has[k]) {
                ld_vec(c[k], row_at<T>(a.x, row, a.ldx, base[k] + kChunk * group));
                if (ADD) ld_vec(r[k], row_at<T>(a.residual, row, a.ldr, base[k] + kChunk * group));
            }
        } else if (in) {
            c[k] = load_chunk<T, VEC>(row_at<T>(a.x, row, a.ldx), base[k], lane, cols);
            if (ADD) r[k] = load_chunk<T, VEC>(row_at<T>(a.residual, row, a.ldr), base[k], lane, cols);
        }
        if (++tile == across) tile = 0, row += rows_in;
    }
    const PhiloxKey key = philox_key(a.drop);
#pragma unroll
    for (int k = 0; k < kTiles; ++k) {
        const Keep<VEC> keep = keep_at<VEC>(key, a.drop, (uint32_t)at[k],
                                            (uint32_t)(base[k] >> 3) + group, lane);
        drop_chunk<ADD>(c[k], r[k], keep, a.drop);
        if (VEC) {
            if (has[k])
                st_vec(static_cast<char*>(row_at<T>(a.y, at[k], a.ldy)) +
                           (int64_t)(base[k] + kChunk * group) * sizeof(typename Elem<T>::raw),
                       c[k]);
        } else if (has[k]) {
            store_chunk<T, VEC>(row_at<T>(a.y, at[k], a.ldy), base[k], lane, cols, c[k]);
        }
    }
}

// The elements of a lane's aligned eight that lie in a row of `cols` columns: one access where
// all do, else one each.  The first is column `col`, which may be before the row.
template <typename T>
__device__ __forceinline__ void load_within(Chunk<T>& c, const void* row, int col, int cols) {
    const typename Elem<T>::raw* p = static_cast<const typename Elem<T>::raw*>(row) + col;
    if (col >= 0 && col + kChunk <= cols) {
        ld_vec(c, p);
        return;
    }
#pragma unroll
    for (int i = 0; i < Elem<T>::kWords; ++i) c.w[i] = 0u;
#pragma unroll
    for (int j = 0; j < kChunk; ++j) {
        const uint32_t v = col + j >= 0 && col + j < cols ? (uint32_t)p[j] : 0u;
        if constexpr (sizeof(*p) == 4)
            c.w[j] = v;
        else
            c.w[j >> 1] |= v << (16 * (j & 1));
    }
}
template <typename T>
__device__ __forceinline__ void store_within(void* row, int col, int cols, const Chunk<T>& c) {
    typename Elem<T>::raw* p = static_cast<typename Elem<T>::raw*>(row) + col;
    if (col >= 0 && col + kChunk <= cols) {
        st_vec(p, c);
        return;
    }
#pragma unroll
    for (int j = 0; j < kChunk; ++j)
        if (col + j >= 0 && col + j < cols) {
            if constexpr (sizeof(*p) == 4)
                p[j] = c.w[j];
            else
                p[j] = (uint16_t)(c.w[j >> 1] >> (16 * (j & 1)));
        }
}

// Rows of any width whose tensors lie alike: row r starts `shift` elements (0..7) past a
// boundary of eight in each of them, as whole tensors of an odd width do.  Aligned
// eight q of a row is its columns 8 q - shift .. + 7; their bits are those of
// column groups q - 1 and q, of which a lane makes q and the lane before it q - 1.  A warp takes
// kTiles x 32 - 1 eights of a row; its first lane starts with a group for the next lane only.
// (The ends of the rows an element a lane, gathered by shuffles, took 80 registers instead of 44
// and 76 us at 16384 x 4095 instead of 69.)
template <typename T, bool ADD>
__global__ void __launch_bounds__(256) dropout_shifted_kernel(const DropArgs a, uint32_t across,
                                                              uint32_t shift0) {
    constexpr int kTiles = tiles_of_warp<T>();
    const int lane = threadIdx.x & 31, cols = (int)a.cols;
    const int64_t task = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int64_t row = task >> 32 == 0 ? (uint32_t)task / across : task / across;
    if (row >= a.rows) return;
    const int q0 = (int)(task - row * across) * (32 * kTiles - 1) - 1;
    const uint32_t shift = (shift0 + (uint32_t)row * (uint32_t)a.ldx) & 7;
    const int first = kChunk * (q0 + lane) - (int)shift;  // this lane's first column
    const void* const x = row_at<T>(a.x, row, a.ldx);
    const void* const res = ADD ? row_at<T>(a.residual, row, a.ldr) : nullptr;
    Chunk<T> c[kTiles], r[kTiles];
#pragma unroll
    for (int k = 0; k < kTiles; ++k) {
        const int col = first + k * kWarpCols;
        if (col < cols && (k > 0 || lane > 0)) {
            load_within(c[k], x, col, cols);
            if (ADD) load_within(r[k], res, col, cols);
        }
    }
    const PhiloxKey key = philox_key(a.drop);
    void* const y = row_at<T>(a.y, row, a.ldy);
    uint32_t last = 0;
#pragma unroll
    for (int k = 0; k < kTiles; ++k) {
        if (kChunk * (q0 + 32 * k) - (int)shift >= cols) break;  // the same for the warp
        const uint32_t m = group_bits(key, a.drop, (uint32_t)row, (uint32_t)(q0 + 32 * k + lane));
        const uint32_t before = __shfl_sync(0xFFFFFFFFu, lane == 31 ? last : m, (lane + 31) & 31);
        last = m;
        const Keep<false> keep = {((m << 8) | before) >> (8 - shift)};
        const int col = first + k * kWarpCols;
        if (col < cols && (k > 0 || lane > 0)) {
            drop_chunk<ADD>(c[k], r[k], keep, a.drop);
            store_within(y, col, cols, c[k]);
        }
    }
}

// Elements past a boundary of eight, of a tensor's first row.
template <typename T>
uint32_t past_eight(const void* p) {
    return (uint32_t)((uintptr_t)p / sizeof(typename Elem<T>::raw)) & 7;
}
template <typename T>
bool lie_alike(const DropArgs& a) {
    const uint32_t shift = past_eight<T>(a.x);
    return past_eight<T>(a.y) == shift && ((a.ldy - a.ldx) & 7) == 0 &&
           (!a.residual || (past_eight<T>(a.residual) == shift && ((a.ldr - a.ldx) & 7) == 0));
}

template <typename T, bool ADD>
lm_status launch(const DropArgs& a, bool vec, cudaStream_t s) {
    constexpr int kTiles = tiles_of_warp<T>();
    if (vec && a.cols % (kTiles * kWarpCols) == 0) {
        const int64_t across = a.cols / (kTiles * kWarpCols), blocks = (a.rows * across + 7) / 8;
        if (blocks >= (int64_t(1) << 31)) return LM_ERR_UNSUPPORTED_SHAPE;
        timing_mark(s, 'd');
        dropout_full_kernel<T, ADD><<<(unsigned)blocks, 256, 0, s>>>(a, (uint32_t)across);
        return launch_status();
    }
    // Up to 256 columns the row's two ends cost more than the wide accesses save (65536 x 250
    // bf16 45 us instead of 34, x 300 42 instead of 52); fp32 beside a residual is at the copy's rate
    // with scalar accesses, and below it here up to a thousand columns.
    if constexpr (sizeof(typename Elem<T>::raw) == 2 || !ADD) {
        if (!vec && a.cols > kWarpCols && lie_alike<T>(a)) {
            // a row's eights where it starts 7 past a boundary
            const int64_t eights = (a.cols + 14) / 8;
            const int64_t across = (eights + 32 * kTiles - 2) / (32 * kTiles - 1);
            const int64_t blocks = (a.rows * across + 7) / 8;
            if (blocks >= (int64_t(1) << 31)) return LM_ERR_UNSUPPORTED_SHAPE;
            timing_mark(s, 'd');
            dropout_shifted_kernel<T, ADD>
                <<<(unsigned)blocks, 256, 0, s>>>(a, (uint32_t)across, past_eight<T>(a.x));
            return launch_status();
        }
    }
    const int across = (int)((a.cols + kWarpCols - 1) / kWarpCols);
    const int rows_in = vec && a.cols <= 128 ? (int)(256 / a.cols) : 1;
    const int64_t tiles = (a.rows + rows_in - 1) / rows_in * across;
    const int64_t blocks = (tiles + 8 * kTiles - 1) / (8 * kTiles);
    if (blocks >= (int64_t(1) << 31)) return LM_ERR_UNSUPPORTED_SHAPE;
    timing_mark(s, 'd');
    if (vec)
        dropout_kernel<T, true, ADD><<<(unsigned)blocks, 256, 0, s>>>(a, across, rows_in);
    else
        dropout_kernel<T, false, ADD><<<(unsigned)blocks, 256, 0, s>>>(a, across, rows_in);
    return launch_status();
}

lm_status dropout(const DropArgs& a, lm_dtype dtype, lm_stream_t stream) {
    if (a.rows < 0 || a.cols <= 0 || (a.rows > 0 && (!a.x || !a.y))) return LM_ERR_INVALID_ARG;
    if (too_large(a.rows, a.cols)) return LM_ERR_UNSUPPORTED_SHAPE;
    const RowTensor ts[] = {{a.x, a.ldx, true}, {a.residual, a.ldr, true}, {a.y, a.ldy, true}};
    bool vec;
    const lm_status st = row_access(ts, 3, a.rows, a.cols, dtype, &vec);
    if (st != LM_OK || a.rows == 0) return st;
    if (!in_place_or_apart(ts[2], ts[0], a.rows) || !in_place_or_apart(ts[2], ts[1], a.rows))
        return LM_ERR_INVALID_ARG;
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
