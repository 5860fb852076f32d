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
// All sums are fp32; the variance is that of the centred values, so a large mean costs
// no digits.  The only roundings to fewer bits are those of bf16 outputs, once
// each, and of s, which the norm is defined on.  The norm's backward sums over the rows
// go through per-block partial sums in the workspace and a second kernel, in a
// fixed order: no atomics, the same bits from call to call.
//
// Bound by HBM: every tensor read and written once, 4 bytes an element of a bf16
// forward, 6 of a backward, 8 and 10 fused with dropout.  What has to be kept
// small for that is the number of instructions (an SM gets 23 bytes a clock: 5.7 elements of
// the forward), hence the packed fp32 pairs, one exchange of sums a row, addresses with
// constant offsets and kernels without tests for whole rows.  One B200, kernels back to
// back for some ms, of the 6.46 TB/s that a copy reaches (in brackets):
//   forward        16384 x 4096 bf16 42.5 us (98%), 8192 x 8192 fp32 81 us (102%)
//   backward       16384 x 4096 bf16 65 us (96%), of which the sum of the parts 4
//   fused forward  8192 x 5120 bf16 52.5 us (99%); fused backward 8192 x 8192 108 (96%)
// These are rows of whole 8-column accesses. Others (odd widths, rows at any alignment) go by
// one element an access, 40 to 50% of a copy: 16384 x 4095 bf16 102 us forward, 148
// backward, 166 and 257 fused. A row is read once up to 32,768 columns forward (others:
// 16,384) and 16,384 backward (fp32 and others: 8,192; others of fp32 with dropout: 4,096); the
// kernels for wider ones read it again for each sweep.
// Over longer times the 1 kW limit lowers the SM clock to 1.6-1.8 GHz and all take 3-12%
// longer, the copy 3%.
#include <type_traits>

#include "lm_chunk.cuh"
#include "lm_device_once.h"
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
    double inv_cols;  // 1 / cols
    double inv_last;  // 1 / the columns of a row's last warp
    float *mean, *rstd;
    unsigned int* amax;  // fp32 bits, max-reduced; or NULL
    Dropout drop;
};

struct BwdArgs {
    const void *dy, *ds, *s, *weight;
    const float *mean, *rstd;
    void *dx, *dres;
    int64_t rows, cols, lddy, ldds, lds, lddx, lddr;
    double inv_cols;  // 1 / cols
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

// A warp's chunks in shared memory, 512 bytes (fp32: 1024) from one to the next, so that
// every access is one register and a constant.  They are filled by asynchronous
// copies of 16 bytes a lane, 512 adjacent ones a warp: of an fp32 chunk a lane
// copies other columns than it reads, so that no 32-byte sector is fetched twice, and
// a warp barrier goes with it.  `swizzled`: the place of the u-th 16 bytes of an fp32
// chunk, such that neither the copies (u = lane, 32 + lane) nor the reads (u = 2 lane,
// 2 lane + 1) have bank conflicts.
template <typename T>
struct Slots {
    static constexpr bool kWide = Elem<T>::kWords == 8;
    static constexpr int kBytes = kWide ? 1024 : 512;  // of a warp's chunk
    uint32_t base;  // shared address of the warp's slot 0
    uint32_t copy0, copy1, read0, read1;

    __device__ __forceinline__ static uint32_t swizzled(uint32_t u) {
        return 16 * (u ^ ((u >> 3) & 1));
    }
    __device__ __forceinline__ Slots(void* smem, int bytes, int lane)
        : base((uint32_t)__cvta_generic_to_shared(smem) + bytes) {
        copy0 = kWide ? swizzled(lane) : 16 * lane;
        copy1 = swizzled(32 + lane);
        read0 = kWide ? swizzled(2 * lane) : 16 * lane;
        read1 = swizzled(2 * lane + 1);
    }
    // The k-th slot `at` bytes on.
    // src: the row's column at 16 lane bytes into the chunk; has: whether it is one, has2: and
    // that 512 bytes on (fp32).
    __device__ __forceinline__ void fill(uint32_t at, int k, const char* src, bool has,
                                         bool has2) const {
        if (has)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(base + at + copy0 +
                                                                          k * kBytes),
                         "l"(src)
                         : "memory");
        if (kWide && has2)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(base + at + copy1 +
                                                                          k * kBytes),
                         "l"(src + 512)
                         : "memory");
    }
    __device__ __forceinline__ void put(uint32_t at, int k, const Chunk<T>& c) const {
#pragma unroll
        for (int p = 0; p < Elem<T>::kWords / 4; ++p)
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                             base + at + (p ? read1 : read0) + k * kBytes),
                         "r"(c.w[4 * p]), "r"(c.w[4 * p + 1]), "r"(c.w[4 * p + 2]),
                         "r"(c.w[4 * p + 3])
                         : "memory");
    }
    __device__ __forceinline__ Chunk<T> take(uint32_t at, int k) const {
        Chunk<T> c;
#pragma unroll
        for (int p = 0; p < Elem<T>::kWords / 4; ++p)
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(c.w[4 * p]), "=r"(c.w[4 * p + 1]), "=r"(c.w[4 * p + 2]),
                           "=r"(c.w[4 * p + 3])
                         : "r"(base + at + (p ? read1 : read0) + k * kBytes)
                         : "memory");
        return c;
    }
};

// Waits until at most `pending` (1 or 2, else 0) of the thread's last groups of copies are
// in flight.
__device__ __forceinline__ void copies_wait(int pending) {
    if (pending == 2)
        asm volatile("cp.async.wait_group 2;" ::: "memory");
    else if (pending == 1)
        asm volatile("cp.async.wait_group 1;" ::: "memory");
    else
        asm volatile("cp.async.wait_group 0;" ::: "memory");
}
__device__ __forceinline__ void copies_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
__device__ __forceinline__ void group_barrier(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

constexpr int kSmemBytes = 226 * 1024;  // dynamic shared memory of a block, at most
// Rows are held two ahead of use where they fit this, else one: beyond it too little of the
// SM's 256 KB is left as cache (16384 x 5120 bf16, 86 us with 130 KB and 92 with 190).
constexpr int kManyBytes = 160 * 1024;

// Mean and sum of centred squares of a row from its warps' own: with n_w columns, sum s_w
// and centred squares q_w in warp w, the row has mean m = sum s_w / n and centred
// squares sum q_w + n_w (s_w / n_w - m)^2, so one exchange does for both.  `buf`: a
// float2 for each warp; exchange(): a barrier of the row's warps.  The mean is a
// product in fp64, so of the sum's value it is rounded once: a constant bf16 row, whose sums
// are exact up to 2^16 columns, has its value for a mean.
template <typename Exchange>
__device__ __forceinline__ void row_moments(int lane, int warp, int warps, float2* buf, int cols,
                                            int each, double inv_cols, float& s, float& q,
                                            Exchange exchange) {
    if (warps == 1) {
        s = (float)(s * inv_cols);
        return;
    }
    if (lane == 0) buf[warp] = make_float2(s, q);
    exchange();
    // the warps' values in a power of two of lanes, again and again
    auto over = [&](auto steps) {
        constexpr int kSpan = 1 << decltype(steps)::value;
        const int w = lane & (kSpan - 1);
        const float2 mine = w < warps ? buf[w] : make_float2(0.f, 0.f);
        float sum = mine.x;
#pragma unroll
        for (int o = kSpan / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        s = (float)(sum * inv_cols);
        const int left = cols - w * each;  // columns of warp w
        const float n = (float)(left < each ? left : each);
        // divided before it is squared: d^2 is up to n times what is added
        const float d = mine.x - n * s;
        q = left > 0 ? __fmaf_rn(__fdividef(d, n), d, mine.y) : 0.f;
#pragma unroll
        for (int o = kSpan / 2; o > 0; o >>= 1) q += __shfl_xor_sync(0xFFFFFFFFu, q, o);
    };
    if (warps <= 4)
        over(std::integral_constant<int, 2>{});
    else if (warps <= 8)
        over(std::integral_constant<int, 3>{});
    else
        over(std::integral_constant<int, 5>{});
}

// Keeps the compiler from holding the fp32 values of bf16 chunks from one sweep to the
// next: they are taken from the words again, which leaves registers to more warps.
template <int NCH>
__device__ __forceinline__ void as_stored(Chunk<bf16_t> (&c)[NCH]) {
#pragma unroll
    for (int i = 0; i < NCH; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) asm volatile("" : "+r"(c[i].w[k]));
}
template <int NCH>
__device__ __forceinline__ void as_stored(Chunk<f32_t> (&)[NCH]) {}

// A warp's sum and centred squares (about its own mean) of its chunks; inv_own: one over
// its number of columns.
template <bool VEC, bool FULL = false, typename T, int NCH>
__device__ __forceinline__ void warp_moments(Chunk<T> (&c)[NCH], int first, int lane, int cols,
                                             double inv_own, float& s, float& q) {
    F2 sum = {}, sq = {};
#pragma unroll
    for (int i = 0; i < NCH; ++i)
#pragma unroll
        for (int j = 0; j < kPairs; ++j) sum = add2(sum, get2(c[i], j));
    s = lo_of(sum) + hi_of(sum);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    const float mean = (float)(s * inv_own);
    as_stored(c);
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const int base = first + i * kWarpCols;
        // past the columns the values are 0 and add nothing
        const float m = chunk_has<VEC, FULL>(base, lane, cols) ? -mean : 0.f;
        const F2 minus_mean = make_f2(m, m);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
            F2 d = add2(get2(c[i], j), minus_mean);
            if (!VEC)
                d = make_f2(chunk_col<false>(base, lane, 2 * j) < cols ? lo_of(d) : 0.f,
                            chunk_col<false>(base, lane, 2 * j + 1) < cols ? hi_of(d) : 0.f);
            sq = fma2(d, d, sq);
        }
    }
    q = lo_of(sq) + hi_of(sq);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) q += __shfl_xor_sync(0xFFFFFFFFu, q, o);
}

// The chunk as S is stored: residual + dropout(x).
template <typename T, bool VEC>
__device__ __forceinline__ Chunk<T> dropped_sum(const Chunk<T>& c, const Chunk<T>& r,
                                                const PhiloxKey& key, const Dropout& d,
                                                int64_t row, int base, int lane) {
    const Keep<VEC> keep = keep_of<VEC>(renewed(key), d, (uint32_t)row, base, lane);
    const F2 scale = make_f2(d.scale, d.scale);
    Chunk<T> s;
#pragma unroll
    for (int i = 0; i < kPairs; ++i)
        put2(s, i, add2(get2(r, i), kept(mul2(get2(c, i), scale), keep, d, i)));
    return s;
}

template <typename T>
__device__ __forceinline__ Chunk<T> ones_chunk() {
    Chunk<T> c;
    const float ones[kChunk] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
    put(c, ones);
    return c;
}

// The largest |element| of a chunk, as fp32 bits (NaN above everything).
template <typename T, bool VEC>
__device__ __forceinline__ uint32_t chunk_top(const Chunk<T>& c, int base, int lane, int cols) {
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < kChunk; ++j)
        if (chunk_col<VEC>(base, lane, j) < cols) top = max(top, abs_bits(get(c, j)));
    return top;
}

constexpr int kFewWarps = 12;
// Registers: with up to kFewWarps warps 56 a thread for bf16 (three blocks of 12 warps an
// SM) and 64 otherwise (two of 16); 64 for one block of 32.
template <typename T, bool VEC, int WARPS>
__host__ __device__ constexpr int fwd_blocks() {
    return WARPS != kFewWarps ? 1 : VEC && sizeof(typename Elem<T>::raw) == 2 ? 3 : 2;
}
template <typename T, bool VEC, int WARPS>
__host__ __device__ constexpr int fwd_bound() {
    return fwd_blocks<T, VEC, WARPS>() == 2 ? 512 : 32 * WARPS;
}

// The row in registers, read once: its warps (blockDim / 32 of them, or with ONE
// one, and blockDim / 32 rows a block) take NCH x 256 columns each.
// FULL: VEC, a multiple of NCH x 256 columns, a weight and a bias, so that nothing is
// tested for each access: 27% fewer instructions for a bf16 row.
// WARPS: the most a block has.
template <typename T, bool VEC, int NCH, int WARPS, bool ONE, bool DROP, bool FULL>
__global__ void __launch_bounds__(fwd_bound<T, VEC, WARPS>(), fwd_blocks<T, VEC, WARPS>())
    norm_fwd_kernel(const FwdArgs a) {
    __shared__ float2 buf[32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const int64_t row = ONE ? (int64_t)blockIdx.x * warps + warp : blockIdx.x;
    if (ONE && row >= a.rows) return;
    const int cols = (int)a.cols, first = ONE ? 0 : warp * NCH * kWarpCols;
    const void* const x = row_at<T>(a.x, row, a.ldx);
    Chunk<T> c[NCH];
#pragma unroll
    for (int i = 0; i < NCH; ++i)
        c[i] = load_chunk<T, VEC, FULL>(x, first + i * kWarpCols, lane, cols);
    if (DROP) {
        const void* const residual = row_at<T>(a.residual, row, a.ldr);
        void* const s = row_at<T>(a.s, row, a.lds);
        Chunk<T> r[NCH];
        if (FULL) {
#pragma unroll
            for (int i = 0; i < NCH; ++i)
                r[i] = load_chunk<T, VEC, FULL>(residual, first + i * kWarpCols, lane, cols);
        }
        const PhiloxKey key = philox_key(a.drop);
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int base = first + i * kWarpCols;
            if (!FULL) r[i] = load_chunk<T, VEC>(residual, base, lane, cols);
            c[i] = dropped_sum<T, VEC>(c[i], r[i], key, a.drop, row, base, lane);
            store_chunk<T, VEC, FULL>(s, base, lane, cols, c[i]);
        }
    }
    float mean, sq;
    const bool whole = FULL || (!ONE && warp < warps - 1);
    const double inv_own = whole ? 1.0 / (NCH * kWarpCols) : a.inv_last;
    warp_moments<VEC, FULL>(c, first, lane, cols, inv_own, mean, sq);
    row_moments(lane, warp, ONE ? 1 : warps, buf, cols, NCH * kWarpCols, a.inv_cols, mean, sq,
                [] { __syncthreads(); });
    const float rstd = rsqrtf(sq * (float)a.inv_cols + a.eps);
    if (lane == 0 && (ONE || warp == 0)) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
    }
    const F2 minus_mean = make_f2(-mean, -mean), r2 = make_f2(rstd, rstd);
    void* const y = row_at<T>(a.y, row, a.ldy);
    as_stored(c);
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const int base = first + i * kWarpCols;
        Chunk<T> w, b;
        if (FULL) {
            w = load_chunk<T, VEC, FULL>(a.weight, base, lane, cols);
            b = load_chunk<T, VEC, FULL>(a.bias, base, lane, cols);
        } else {
            w = a.weight ? load_chunk<T, VEC>(a.weight, base, lane, cols) : ones_chunk<T>();
            b = a.bias ? load_chunk<T, VEC>(a.bias, base, lane, cols) : Chunk<T>{};
        }
#pragma unroll
        for (int j = 0; j < kPairs; ++j)
            put2(c[i], j,
                 fma2(mul2(add2(get2(c[i], j), minus_mean), r2), get2(w, j), get2(b, j)));
        store_chunk<T, VEC, FULL>(y, base, lane, cols, c[i]);
    }
    if (a.amax) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < NCH; ++i)
            top = max(top, chunk_top<T, VEC>(c[i], first + i * kWarpCols, lane, cols));
        top = __reduce_max_sync(0xFFFFFFFFu, top);
        if (lane == 0 && top) atomicMax(a.amax, top);
    }
}

// How a persistent block is laid out: `warps` warps (a group) share a row, and the block's
// groups take different rows, so that one group's exchange of sums is hidden by the
// others' work.  Group g of block b: rows b groups + g, + gridDim groups, ...
struct Group {
    int lane, warps, groups, group, warp;
    __device__ __forceinline__ explicit Group(int w) : lane(threadIdx.x & 31), warps(w) {
        // the same in all lanes, and known to be
        const int bw = __shfl_sync(0xFFFFFFFFu, (int)(threadIdx.x >> 5), 0);
        groups = (int)(blockDim.x >> 5) / w;
        group = bw / w;
        warp = bw - group * w;
    }
};

// Sums of two values over a group of at most 16 warps, the same in every thread.  Lanes
// 0..15 go on with the first value and 16..31 with the second after one exchange.
// `buf`: two floats for each warp of the group, others than the call before used.
__device__ __forceinline__ void group_sum2(const Group& g, float* buf, float& a, float& b) {
    const bool upper = g.lane >= 16;
    const float give = upper ? a : b;
    float v = (upper ? b : a) + __shfl_xor_sync(0xFFFFFFFFu, give, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (g.warps > 1) {
        // the first values of all warps, then the second ones
        if ((g.lane & 15) == 0) buf[(upper ? g.warps : 0) + g.warp] = v;
        group_barrier(g.group + 1, 32 * g.warps);
        const float* const mine = buf + (upper ? g.warps : 0);
        // a path for each: one for both is compiled to a slower kernel (16384 x 4096 bf16 67.1 us
        // instead of 65.3) or one that spills (fused, 8192 x 5120, 82 us instead of 75.7)
        if (g.warps > 8) {
            const int k = g.lane & 15;
            v = k < g.warps ? mine[k] : 0.f;
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
        } else {
            const int k = g.lane & 7;
            v = k < g.warps ? mine[k] : 0.f;
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
        }
    }
    const float other = __shfl_xor_sync(0xFFFFFFFFu, v, 16);
    a = upper ? other : v;
    b = upper ? v : other;
}

// Threads of a backward block, at most: 128 registers each, of which the sums take up to
// 64.
constexpr int kBwdThreads = 512;
static_assert(kBwdThreads <= 16 * 32, "group_sum2 adds up 16 warps");

// The backward pass, every tensor read once for dx and the weight gradients.  A thread
// keeps its NCH chunks' sums over its rows in registers; at the end the block adds its
// groups' sums and writes one part of the partial sums.  With four chunks a thread the
// sums leave no registers for the row and the weight: they are read from shared
// memory again for the second sweep.
// VEC: rows come by asynchronous copies, `stages` - 1 ahead; otherwise by scalar loads into
// registers, one ahead (ds, for which there are none, as it is used).
template <typename T, bool VEC, int NCH, bool DROP, bool FULL>
__global__ void __launch_bounds__(kBwdThreads, 1)
    norm_bwd_kernel(const BwdArgs a, int warps, int stages, float* part) {
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ float buf[2 * 32];
    constexpr int NT = DROP ? 3 : 2;
    constexpr int kSlot = Slots<T>::kBytes, kRow = NT * NCH * kSlot;  // of a warp
    constexpr int kSize = sizeof(typename Elem<T>::raw), kNext = kWarpCols * kSize;
    constexpr bool kAgain = NCH > 2;  // read the row and the weight again for the second sweep
    const int cols = (int)a.cols;
    const Group g(warps);
    const int first = g.warp * NCH * kWarpCols;
    const bool has_ds = DROP && a.ds;
    // the weight's slots, shared by the groups, then each warp's rows
    const Slots<T> ws(smem, g.warp * NCH * kSlot, g.lane);
    const Slots<T> slots(smem, warps * NCH * kSlot + (g.group * warps + g.warp) * stages * kRow,
                         g.lane);
    Chunk<T> w[NCH], d[NCH], c[NCH];
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        w[i] = a.weight ? load_chunk<T, VEC>(a.weight, first + i * kWarpCols, g.lane, cols)
                        : ones_chunk<T>();
        if (kAgain && g.group == 0) ws.put(0, i, w[i]);
    }
    F2 dw[NCH][kPairs] = {}, db[NCH][kPairs] = {};
    PhiloxKey key{};
    if (DROP) key = philox_key(a.drop);
    const uint32_t at0 = (uint32_t)(first + kChunk * g.lane) * kSize;  // VEC: in the outputs' row

    const uint32_t rows = (uint32_t)a.rows, row_step = gridDim.x * g.groups;
    uint32_t row = blockIdx.x * g.groups + g.group;
    // VEC: this lane's place in the row to be fetched next, and in the outputs' row
    const int64_t step = (int64_t)row_step * kSize;
    const int64_t from0 = (int64_t)first * kSize + 16 * g.lane;
    const int from_col = first + 16 / kSize * g.lane;
    const char* dy = static_cast<const char*>(a.dy) + row * a.lddy * kSize + from0;
    const char* s = static_cast<const char*>(a.s) + row * a.lds * kSize + from0;
    const char* ds = static_cast<const char*>(a.ds) + (has_ds ? row * a.ldds * kSize + from0 : 0);
    char* dres = static_cast<char*>(a.dres) + row * a.lddr * kSize + at0;
    char* dx = static_cast<char*>(a.dx) + (DROP ? row * a.lddx * kSize + at0 : 0);
    Chunk<T> next_d[VEC ? 1 : NCH], next_c[VEC ? 1 : NCH];
    auto fetch = [&](uint32_t r, uint32_t to) {
        if (r < rows) {
#pragma unroll
            for (int i = 0; i < NCH; ++i) {
                const int base = first + i * kWarpCols;
                if (VEC) {
                    const bool h1 = FULL || from_col + i * kWarpCols < cols;
                    const bool h2 = FULL || from_col + i * kWarpCols + 128 < cols;
                    slots.fill(to, i, dy + i * kNext, h1, h2);
                    slots.fill(to, NCH + i, s + i * kNext, h1, h2);
                    if (has_ds) slots.fill(to, 2 * NCH + i, ds + i * kNext, h1, h2);
                } else {
                    next_d[i] = load_chunk<T, VEC>(row_at<T>(a.dy, r, a.lddy), base, g.lane, cols);
                    next_c[i] = load_chunk<T, VEC>(row_at<T>(a.s, r, a.lds), base, g.lane, cols);
                }
            }
        }
        if (VEC) {
            dy += step * a.lddy, s += step * a.lds;
            if (DROP) ds += step * a.ldds;
            copies_commit();
        }
    };

    if (VEC) {
        // what no copy fills, past the columns, is zero
        for (int k = 0; k < stages * NT; ++k)
#pragma unroll
            for (int i = 0; i < NCH; ++i)
                if (!chunk_has<true, FULL>(first + i * kWarpCols, g.lane, cols))
                    slots.put(0, k * NCH + i, Chunk<T>{});
        for (int k = 0; k < stages - 1; ++k) fetch(row + k * row_step, k * kRow);
    } else {
        fetch(row, 0);
    }
    // lane l has the mean of the group's row l of 16, lane 16 + l its rstd; `next_stats`: of
    // the 16 rows after them
    float stats = 0.f, next_stats = 0.f;
    auto fetch_stats = [&](uint64_t r) {
        r += (uint64_t)(g.lane & 15) * row_step;
        if (r < rows) next_stats = (g.lane < 16 ? a.mean : a.rstd)[r];
    };
    fetch_stats(row);
    // the kernel that adds the parts may come and wait
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __syncthreads();  // the weight
    // bytes to this row's slots, and to the free ones
    uint32_t at = 0, ahead = (stages - 1) * kRow;
    int mine = 2 * warps * g.group;  // this group's part of one buffer or the other
    for (uint32_t k = 0; row < rows; ++k, row += row_step) {
        if (k % 16 == 0) {
            stats = next_stats;
            fetch_stats((uint64_t)row + 16ull * row_step);
        }
        if (VEC && Slots<T>::kWide) __syncwarp();  // all have read what is overwritten now
        if (VEC) {
            fetch(row + (stages - 1) * row_step, ahead);
            copies_wait(stages - 1);
            if (Slots<T>::kWide) __syncwarp();  // the others' copies
        } else {
#pragma unroll
            for (int i = 0; i < NCH; ++i) d[i] = next_d[i], c[i] = next_c[i];
            fetch(row + row_step, 0);
        }
        const float mean = __shfl_sync(0xFFFFFFFFu, stats, k % 16);
        const float rstd = __shfl_sync(0xFFFFFFFFu, stats, 16 + k % 16);
        const F2 minus_mean = make_f2(-mean, -mean), r2 = make_f2(rstd, rstd);
        F2 s1 = {}, s2 = {};
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            if (NCH > 2 && i == 2) __syncwarp();  // or the compiler loads all four, and spills
            if (VEC) d[i] = slots.take(at, i), c[i] = slots.take(at, NCH + i);
            if (kAgain) w[i] = ws.take(0, i);
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
                // past the columns dy is 0, so the sums get nothing from there
                const F2 y = get2(d[i], j), wj = get2(w[i], j);
                const F2 t = mul2(y, add2(get2(c[i], j), minus_mean));
                s1 = fma2(y, wj, s1);
                s2 = fma2(t, wj, s2);
                dw[i][j] = fma2(t, r2, dw[i][j]);
                db[i][j] = add2(db[i][j], y);
            }
        }
        float c1 = lo_of(s1) + hi_of(s1), c2 = (lo_of(s2) + hi_of(s2)) * rstd;
        group_sum2(g, buf + mine, c1, c2);
        mine ^= 32;
        if (!kAgain) as_stored(d), as_stored(c), as_stored(w);
        // dx = rstd g - rstd c1 - (x - mean) rstd (rstd c2)
        const float per = (float)a.inv_cols * rstd;
        c1 *= per, c2 = c2 * per * rstd;
        const F2 m1 = make_f2(-c1, -c1), m2 = make_f2(-c2, -c2);
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int base = first + i * kWarpCols;
            if (NCH > 2 && i == 2) __syncwarp();  // or the compiler loads all four, and spills
            if (kAgain) {
                d[i] = slots.take(at, i), c[i] = slots.take(at, NCH + i);
                w[i] = ws.take(0, i);
            }
            Chunk<T> up, out;
            if (has_ds)
                up = VEC ? slots.take(at, 2 * NCH + i)
                         : load_chunk<T, VEC>(row_at<T>(a.ds, row, a.ldds), base, g.lane, cols);
            F2 v[kPairs];
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
                v[j] = fma2(mul2(get2(d[i], j), get2(w[i], j)), r2, m1);
                v[j] = fma2(add2(get2(c[i], j), minus_mean), m2, v[j]);
                if (has_ds) v[j] = add2(get2(up, j), v[j]);
                put2(out, j, v[j]);
            }
            if (VEC) {
                if (chunk_has<true, FULL>(base, g.lane, cols)) st_vec(dres + i * kNext, out);
            } else {
                store_chunk<T, VEC>(row_at<T>(a.dres, row, a.lddr), base, g.lane, cols, out);
            }
            if (DROP) {
                const Keep<VEC> keep = keep_of<VEC>(renewed(key), a.drop, row, base, g.lane);
                const F2 scale = make_f2(a.drop.scale, a.drop.scale);
#pragma unroll
                for (int j = 0; j < kPairs; ++j)
                    put2(out, j, kept(mul2(v[j], scale), keep, a.drop, j));
                if (VEC) {
                    if (chunk_has<true, FULL>(base, g.lane, cols)) st_vec(dx + i * kNext, out);
                } else {
                    store_chunk<T, VEC>(row_at<T>(a.dx, row, a.lddx), base, g.lane, cols, out);
                }
            }
        }
        if (VEC) {
            dres += step * a.lddr;
            if (DROP) dx += step * a.lddx;
        }
        ahead = at;
        at = at == (stages - 1) * kRow ? 0 : at + kRow;
    }
    if (!part) return;
    // the last group leaves its sums in shared memory, the others add theirs, group 0 last
    if (g.groups > 1) {
        if (VEC) copies_wait(0);
        __syncthreads();
        const int n = 32 * warps;
        F2* const sum = reinterpret_cast<F2*>(smem) + 32 * g.warp + g.lane;
        for (int k = g.groups - 1; k >= 0; --k) {
            if (g.group == k) {
#pragma unroll
                for (int i = 0; i < NCH; ++i)
#pragma unroll
                    for (int j = 0; j < kPairs; ++j) {
                        F2* const p = sum + (i * kPairs + j) * 2 * n;
                        if (k < g.groups - 1) {
                            dw[i][j] = add2(dw[i][j], p[0]);
                            db[i][j] = add2(db[i][j], p[n]);
                        }
                        if (k > 0) p[0] = dw[i][j], p[n] = db[i][j];
                    }
            }
            __syncthreads();
        }
        if (g.group > 0) return;
    }
    float* const p = part + (int64_t)blockIdx.x * 2 * cols;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const int base = first + i * kWarpCols;
        if (VEC) {
            if (chunk_has<true, FULL>(base, g.lane, cols)) {
                ulonglong2* const q = reinterpret_cast<ulonglong2*>(p + base + kChunk * g.lane);
                ulonglong2* const r =
                    reinterpret_cast<ulonglong2*>(p + cols + base + kChunk * g.lane);
                q[0] = make_ulonglong2(dw[i][0].v, dw[i][1].v);
                q[1] = make_ulonglong2(dw[i][2].v, dw[i][3].v);
                r[0] = make_ulonglong2(db[i][0].v, db[i][1].v);
                r[1] = make_ulonglong2(db[i][2].v, db[i][3].v);
            }
        } else {
#pragma unroll
            for (int j = 0; j < kChunk; ++j) {
                const int col = chunk_col<VEC>(base, g.lane, j);
                const F2 x = dw[i][j >> 1], y = db[i][j >> 1];
                if (col < cols) {
                    p[col] = j & 1 ? hi_of(x) : lo_of(x);
                    p[cols + col] = j & 1 ? hi_of(y) : lo_of(y);
                }
            }
        }
    }
}

// One block a row, the row read again for each sweep: for rows that do not fit
// a block's registers (beyond the widths in launch_fwd and launch_bwd).
template <typename T, bool VEC, bool DROP>
__global__ void __launch_bounds__(256) norm_fwd_wide_kernel(const FwdArgs a) {
    __shared__ float buf[8];
    const int cols = (int)a.cols;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = blockIdx.x;
    const void* x = row_at<T>(a.x, row, a.ldx);
    const void* s = DROP ? row_at<T>(static_cast<const void*>(a.s), row, a.lds) : x;
    PhiloxKey key{};
    if (DROP) key = philox_key(a.drop);
    float sum = 0.f;
    for (int base = warp * kWarpCols; base < cols; base += 8 * kWarpCols) {
        Chunk<T> c = load_chunk<T, VEC>(x, base, lane, cols);
        if (DROP) {
            const Chunk<T> r =
                load_chunk<T, VEC>(row_at<T>(a.residual, row, a.ldr), base, lane, cols);
            c = dropped_sum<T, VEC>(c, r, key, a.drop, row, base, lane);
            store_chunk<T, VEC>(row_at<T>(a.s, row, a.lds), base, lane, cols, c);
        }
#pragma unroll
        for (int j = 0; j < kChunk; ++j) sum += get(c, j);
    }
    const float mean = __fdiv_rn(block_sum(sum, buf), (float)a.cols);
    float sq = 0.f;
    for (int base = warp * kWarpCols; base < cols; base += 8 * kWarpCols) {
        const Chunk<T> c = load_chunk<T, VEC>(s, base, lane, cols);
#pragma unroll
        for (int j = 0; j < kChunk; ++j)
            if (chunk_col<VEC>(base, lane, j) < cols) {
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
    for (int base = warp * kWarpCols; base < cols; base += 8 * kWarpCols) {
        Chunk<T> c = load_chunk<T, VEC>(s, base, lane, cols), w, b;
        if (a.weight) w = load_chunk<T, VEC>(a.weight, base, lane, cols);
        if (a.bias) b = load_chunk<T, VEC>(a.bias, base, lane, cols);
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
                if (chunk_col<VEC>(base, lane, j) < cols) top = max(top, abs_bits(get(c, j)));
        }
        store_chunk<T, VEC>(row_at<T>(a.y, row, a.ldy), base, lane, cols, c);
    }
    if (a.amax) {
        top = __reduce_max_sync(0xFFFFFFFFu, top);
        if (lane == 0 && top) atomicMax(a.amax, top);
    }
}

template <typename T, bool VEC, bool DROP>
__global__ void __launch_bounds__(256) norm_bwd_wide_kernel(const BwdArgs a) {
    __shared__ float buf[8];
    const int cols = (int)a.cols;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = blockIdx.x;
    const void* dy = row_at<T>(a.dy, row, a.lddy);
    const void* s = row_at<T>(a.s, row, a.lds);
    const float mean = a.mean[row], rstd = a.rstd[row];
    float c1 = 0.f, c2 = 0.f;
    for (int base = warp * kWarpCols; base < cols; base += 8 * kWarpCols) {
        const Chunk<T> d = load_chunk<T, VEC>(dy, base, lane, cols);
        const Chunk<T> c = load_chunk<T, VEC>(s, base, lane, cols);
        Chunk<T> w;
        if (a.weight) w = load_chunk<T, VEC>(a.weight, base, lane, cols);
#pragma unroll
        for (int j = 0; j < kChunk; ++j) {
            const float g = a.weight ? get(d, j) * get(w, j) : get(d, j);
            if (chunk_col<VEC>(base, lane, j) < cols) {
                c1 += g;
                c2 = __fmaf_rn(g, (get(c, j) - mean) * rstd, c2);
            }
        }
    }
    c1 = __fdiv_rn(block_sum(c1, buf), (float)a.cols);
    c2 = __fdiv_rn(block_sum(c2, buf), (float)a.cols);
    PhiloxKey key{};
    if (DROP) key = philox_key(a.drop);
    for (int base = warp * kWarpCols; base < cols; base += 8 * kWarpCols) {
        const Chunk<T> d = load_chunk<T, VEC>(dy, base, lane, cols);
        const Chunk<T> c = load_chunk<T, VEC>(s, base, lane, cols);
        Chunk<T> w, up, out;
        if (a.weight) w = load_chunk<T, VEC>(a.weight, base, lane, cols);
        if (a.ds) up = load_chunk<T, VEC>(row_at<T>(a.ds, row, a.ldds), base, lane, cols);
        float v[kChunk];
#pragma unroll
        for (int j = 0; j < kChunk; ++j) {
            const float g = a.weight ? get(d, j) * get(w, j) : get(d, j);
            const float h = (get(c, j) - mean) * rstd;
            v[j] = (g - c1 - h * c2) * rstd;
            if (a.ds) v[j] = get(up, j) + v[j];
        }
        put(out, v);
        store_chunk<T, VEC>(row_at<T>(a.dres, row, a.lddr), base, lane, cols, out);
        if (DROP) {
            const Keep<VEC> keep = keep_of<VEC>(key, a.drop, (uint32_t)row, base, lane);
#pragma unroll
            for (int j = 0; j < kPairs; ++j)
                put2(out, j, kept(mul2(make_f2(v[2 * j], v[2 * j + 1]),
                                       make_f2(a.drop.scale, a.drop.scale)), keep, a.drop, j));
            store_chunk<T, VEC>(row_at<T>(a.dx, row, a.lddx), base, lane, cols, out);
        }
    }
}

// Partial sums over the rows: block (i, p) sums columns 256 i .. + 255 over the
// rows of part p into part[p][0] (dw) and part[p][1] (db).
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) norm_wgrad_kernel(const BwdArgs a, float* part) {
    __shared__ float sum[2][8][kWarpCols];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cols = (int)a.cols;
    const int base = (int)blockIdx.x * kWarpCols;
    float dw[kChunk] = {}, db[kChunk] = {};
    const int64_t step = (int64_t)gridDim.y * 8;
    for (int64_t row = (int64_t)blockIdx.y * 8 + warp; row < a.rows; row += step) {
        const Chunk<T> d = load_chunk<T, VEC>(row_at<T>(a.dy, row, a.lddy), base, lane, cols);
        const Chunk<T> c = load_chunk<T, VEC>(row_at<T>(a.s, row, a.lds), base, lane, cols);
        const float mean = a.mean[row], rstd = a.rstd[row];
#pragma unroll
        for (int j = 0; j < kChunk; ++j) {
            dw[j] = __fmaf_rn(get(d, j), (get(c, j) - mean) * rstd, dw[j]);
            db[j] += get(d, j);
        }
    }
#pragma unroll
    for (int j = 0; j < kChunk; ++j) {
        const int col = chunk_col<VEC>(0, lane, j);
        sum[0][warp][col] = dw[j];
        sum[1][warp][col] = db[j];
    }
    __syncthreads();
    if (base + threadIdx.x < cols) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float t = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) t += sum[k][i][threadIdx.x];
            part[((int64_t)blockIdx.y * 2 + k) * a.cols + base + threadIdx.x] = t;
        }
    }
}

// dw (blockIdx.y 0) and db (1): a block takes 32 columns, its 32 warps every 32nd part
// each, at most ten loads in flight at once.  It may be launched before the kernel that
// writes the parts has ended, and waits for that.
template <typename T, bool ACCUM>
__global__ void __launch_bounds__(1024)
    norm_wgrad_sum_kernel(const float* part, int parts, int cols, void* dweight, void* dbias) {
    __shared__ float sum[32][33];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    void* out = blockIdx.y ? dbias : dweight;
    const int col = (int)blockIdx.x * 32 + lane;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!out) return;
    float t = 0.f;
    if (col < cols) {
        static_assert(kMaxParts <= 32 * 10, "the parts of a warp");
#pragma unroll
        for (int k = 0; k < 10; ++k) {
            const int p = warp + 32 * k;
            t += p < parts ? part[((int64_t)p * 2 + blockIdx.y) * cols + col] : 0.f;
        }
    }
    sum[warp][lane] = t;
    __syncthreads();
    // warp w adds column w's 32 sums
    t = sum[lane][warp];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
    const int at = (int)blockIdx.x * 32 + warp;
    if (lane == 0 && at < cols) {
        if (ACCUM)
            static_cast<float*>(out)[at] += t;
        else if (sizeof(typename Elem<T>::raw) == 4)
            static_cast<float*>(out)[at] = t;
        else
            static_cast<uint16_t*>(out)[at] = (uint16_t)pack_bf16(t, 0.f);
    }
}

template <typename T, bool ACCUM>
lm_status sum_parts(const float* part, int parts, int64_t cols, void* dweight, void* dbias,
                    cudaStream_t s) {
    cudaLaunchConfig_t config{};
    config.gridDim = dim3((unsigned)((cols + 31) / 32), 2);
    config.blockDim = dim3(1024);
    config.stream = s;
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    config.attrs = &early;
    config.numAttrs = 1;
    timing_mark(s, 'n');
    const cudaError_t e = cudaLaunchKernelEx(&config, norm_wgrad_sum_kernel<T, ACCUM>, part, parts,
                                             (int)cols, dweight, dbias);
    return e == cudaSuccess ? launch_status() : LM_ERR_CUDA;
}

template <typename T, bool VEC, int NCH, int WARPS, bool ONE, bool DROP>
void run_fwd(FwdArgs a, int64_t wc, cudaStream_t s) {
    const int warps = (int)((wc + NCH - 1) / NCH);
    const unsigned blocks = (unsigned)(ONE ? (a.rows + 3) / 4 : a.rows);
    const int threads = ONE ? 128 : 32 * warps;
    a.inv_last = 1.0 / (double)(a.cols - (warps - 1) * NCH * kWarpCols);
    if (VEC && a.weight && a.bias && a.cols % (NCH * kWarpCols) == 0)
        norm_fwd_kernel<T, VEC, NCH, WARPS, ONE, DROP, VEC><<<blocks, threads, 0, s>>>(a);
    else
        norm_fwd_kernel<T, VEC, NCH, WARPS, ONE, DROP, false><<<blocks, threads, 0, s>>>(a);
}

// How a persistent block of at most `threads` threads takes `rows` rows: groups of `warps`
// warps, each with `stages` rows (or `few`) of `row` bytes in shared memory, and `shared`
// bytes for all.  groups is 0 where not one fits.
struct Plan {
    int groups, stages, grid, threads, bytes;
};
Plan plan(int64_t rows, int warps, int threads, int sms, int shared, int row, int stages, int few) {
    Plan p{};
    const int64_t share = (rows + sms - 1) / sms;  // rows of an SM
    int groups = threads / (32 * warps);
    if (warps > 1 && groups > 15) groups = 15;  // named barriers
    if (groups > share) groups = (int)share;
    while (groups > 0 && shared + groups * few * row > kSmemBytes) --groups;
    if (groups == 0) return p;
    p.groups = groups;
    p.stages = shared + groups * stages * row > kManyBytes ? few : stages;
    const int64_t need = (rows + groups - 1) / groups;
    p.grid = (int)(need < sms ? need : sms);
    p.threads = 32 * warps * groups;
    p.bytes = shared + groups * p.stages * row;
    return p;
}

// Allows a kernel kSmemBytes of shared memory, once a device.
template <typename K>
bool allow_smem(K kernel, DeviceOnce& once) {
    int dev = -1;
    return cudaGetDevice(&dev) == cudaSuccess && once.run(dev, [&] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    kSmemBytes) == cudaSuccess;
    });
}

// wc: chunks of 256 columns.  A warp takes four, which leaves the least to add up between
// warps; up to 1024 columns that is the whole row.  Without VEC it takes two (a
// chunk's eight scalar accesses need the registers).  Few rows go one chunk a warp, for
// the shortest path: bf16 16 x 1024 in 2.0 us instead of 2.7, 148 x 4096 in 2.5 instead of
// 3.0; fused, 128 x 768 in 2.2 instead of 3.3.
template <typename T, bool VEC, bool DROP>
lm_status launch_fwd(const FwdArgs& a, cudaStream_t s) {
    const int sms = sm_count();
    if (sms <= 0) return LM_ERR_CUDA;
    const int64_t wc = (a.cols + kWarpCols - 1) / kWarpCols;
    constexpr int kNch = VEC ? 4 : 2;
    timing_mark(s, 'n');
    if (wc <= 32 && a.rows * wc <= (int64_t)sms * 32)
        run_fwd<T, VEC, 1, 32, false, DROP>(a, wc, s);
    else if (wc == 1)
        run_fwd<T, VEC, 1, 4, true, DROP>(a, wc, s);
    else if (wc == 2)
        run_fwd<T, VEC, 2, 4, true, DROP>(a, wc, s);
    else if (wc <= 4)
        run_fwd<T, VEC, 4, 4, true, DROP>(a, wc, s);
    else if (wc <= kFewWarps * kNch)
        run_fwd<T, VEC, kNch, kFewWarps, false, DROP>(a, wc, s);
    else if (wc <= 32 * kNch)
        run_fwd<T, VEC, kNch, 32, false, DROP>(a, wc, s);
    else
        norm_fwd_wide_kernel<T, VEC, DROP><<<(unsigned)a.rows, 256, 0, s>>>(a);
    return launch_status();
}

// Launches the backward kernel where it takes the columns; *parts: the partial sums it
// writes, 0 on failure.
template <typename T, bool VEC, int NCH, bool DROP>
bool run_bwd(const BwdArgs& a, int64_t wc, int sms, float* part, cudaStream_t s, int* parts) {
    const int warps = (int)((wc + NCH - 1) / NCH), chunk = warps * NCH * Slots<T>::kBytes;
    Plan p = plan(a.rows, warps, kBwdThreads, sms, chunk, VEC ? (DROP ? 3 : 2) * chunk : 0, 3, 2);
    if (p.groups == 0) return false;
    const int sums = p.groups > 1 ? 32 * warps * NCH * kChunk * 2 * (int)sizeof(float) : 0;
    if (p.bytes < sums) p.bytes = sums;
    *parts = 0;
    static DeviceOnce once[2];
    const bool full = VEC && a.cols % (NCH * kWarpCols) == 0;
    auto kernel = full ? norm_bwd_kernel<T, VEC, NCH, DROP, VEC>
                       : norm_bwd_kernel<T, VEC, NCH, DROP, false>;
    if (!allow_smem(kernel, once[full])) return true;
    kernel<<<p.grid, p.threads, p.bytes, s>>>(a, warps, p.stages, part);
    if (launch_status() == LM_OK) *parts = p.grid;
    return true;
}

template <typename T, bool VEC, bool DROP>
lm_status launch_bwd(const BwdArgs& a, void* dweight, void* dbias, bool accum, float* part,
                     cudaStream_t s) {
    int sms = sm_count();
    if (sms <= 0 && a.rows > 0) return LM_ERR_CUDA;
    if (sms > kMaxParts) sms = kMaxParts;  // a block writes one part
    const bool wgrad = dweight || dbias;
    // Chunks a thread: two up to 4096 columns (two or more groups of up to eight warps), four
    // beyond for bf16 (two groups up to 8192 columns; 16384 x 7168, 113 us, with two chunks
    // and one group of 14 warps 124; at 12288 two chunks and 24 warps are 190 and four 178).
    // But two again where they make one group of 15 or 16 warps (8192 x 8192 with
    // dropout, 108 us, with four chunks and two groups 125).  One where two would spill.
    constexpr bool bf16 = sizeof(typename Elem<T>::raw) == 2;
    constexpr int kTwo = !VEC && DROP && !bf16 ? 1 : 2, kNch = VEC && bf16 ? 4 : kTwo;
    const int64_t wc = (a.cols + kWarpCols - 1) / kWarpCols;
    int parts = 0;
    if (a.rows > 0) {
        float* const p = wgrad ? part : nullptr;
        timing_mark(s, 'n');
        if (wc == 1    ? run_bwd<T, VEC, 1, DROP>(a, wc, sms, p, s, &parts)
            : wc <= 16 || (wc > 28 && wc <= 32 && kTwo == 2)
                ? run_bwd<T, VEC, kTwo, DROP>(a, wc, sms, p, s, &parts)
                : wc <= 16 * kNch && run_bwd<T, VEC, kNch, DROP>(a, wc, sms, p, s, &parts)) {
            if (parts == 0) return LM_ERR_CUDA;
        } else {
            // the weight gradients first: they read dy and s, which dx may overwrite
            if (wgrad) {
                parts = (int)((a.rows + 31) / 32 < kMaxParts ? (a.rows + 31) / 32 : kMaxParts);
                norm_wgrad_kernel<T, VEC>
                    <<<dim3((unsigned)wc, (unsigned)parts), 256, 0, s>>>(a, part);
                if (launch_status() != LM_OK) return LM_ERR_CUDA;
                timing_mark(s, 'n');
            }
            norm_bwd_wide_kernel<T, VEC, DROP><<<(unsigned)a.rows, 256, 0, s>>>(a);
            if (launch_status() != LM_OK) return LM_ERR_CUDA;
        }
    }
    if (!wgrad || (accum && a.rows == 0)) return LM_OK;
    return accum ? sum_parts<T, true>(part, parts, a.cols, dweight, dbias, s)
                 : sum_parts<T, false>(part, parts, a.cols, dweight, dbias, s);
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
    if (a.rows > 0 && a.s == a.y) return LM_ERR_INVALID_ARG;
    for (int out = 2; out < 4; ++out)
        for (int in = 0; in < 2; ++in)
            if (!in_place_or_apart(ts[out], ts[in], a.rows)) return LM_ERR_INVALID_ARG;
    if (!aligned_to(a.mean, 4) || !aligned_to(a.rstd, 4) || !aligned_to(a.amax, 4))
        return LM_ERR_ALIGNMENT;
    if (a.rows == 0) return LM_OK;
    if (share_bytes(a.mean, a.rstd, 4 * a.rows)) return LM_ERR_INVALID_ARG;
    a.inv_cols = 1.0 / (double)a.cols;
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
    if (a.rows > 0 && a.dx == a.dres) return LM_ERR_INVALID_ARG;
    for (int out = 3; out < 5; ++out)
        for (int in = 0; in < 3; ++in)
            if (!in_place_or_apart(ts[out], ts[in], a.rows)) return LM_ERR_INVALID_ARG;
    const bool accum = flags & LM_NORM_ACCUMULATE_WGRAD;
    const unsigned size = accum || dtype == LM_DTYPE_F32 ? 4 : 2;
    if (!aligned_to(dweight, size) || !aligned_to(dbias, size) || !aligned16(workspace) ||
        !aligned_to(a.mean, 4) || !aligned_to(a.rstd, 4))
        return LM_ERR_ALIGNMENT;
    // two blocks would write, or add to, the same elements
    if (a.rows > 0 && share_bytes(dweight, dbias, size * a.cols)) return LM_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    float* part = static_cast<float*>(workspace);
    a.inv_cols = 1.0 / (double)a.cols;
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
