// lm_rope.cu -- rotary positions of up to two tensors (Q and K) in one launch.
//
// Pair i of a head's first `rot_dim` elements is turned by the angle
// a = position * inv_freq[i]:
//
//   (x1, x2) -> m (x1 cos a - x2 sin a, x2 cos a + x1 sin a)
//
// (rotary position embedding: J. Su et al., "RoFormer", 2021); the backward pass
// is the same with the sine negated.  The angle is taken in turns in fp64,
// t = position * inv_freq / 2 pi, with the product's rest, and only t - rint(t) goes to fp32:
// the error does not grow with the position, which is itself held in fp64 (exact to 2^53);
// no table is kept or read.  The other
// head_dim - rot_dim elements are copied (not touched in place).
//
// Bound by HBM: every element read and written once.  A warp keeps a token's cosines and
// sines in registers and takes all heads with them; blocks that shared them through
// shared memory spent their time at barriers and behind 100 registers a thread (16384 tokens, 24 + 8
// heads of 128, bf16: 93 us; now 43.5 us, 96% of what a copy reaches).  One token of 64
// sequences takes 2.5 us: the latency of positions, angles and one access.  Where
// rot_dim / 2 is odd the accesses are scalar (rot_dim 50 of 128: 111 us), where it is no
// multiple of 8 two elements wide (100 of 100: 48 us, 34 of them the bytes; fp32 68 of 68).
#include <type_traits>

#include "lm_chunk.cuh"
#include "lm_internal.h"
#include "lm_rows.h"

namespace lm {
namespace {

struct RopeArgs {
    lm_rope_tensor t[2];
    int64_t batch, seq, tokens;
    int heads0, heads, head_dim, rot_dim;  // heads: of both tensors
    const double* inv_freq;
    const int64_t* positions;
    int64_t start;
    float magnitude, sign;
};

// 1 / 2 pi in two parts.
constexpr double kInvTwoPi = 0.15915494309189533576888376337251;
constexpr double kInvTwoPiLow = -9.8393383375912432e-18;

// cos and sin of position * inv_freq, times the magnitude, the sine with `sign`.  One fp64
// product would be off by 2^-53 of the turns made, 1e-4 of an angle at position 2^40; so
// inv_freq / 2 pi is held in two parts and what the product's rounding leaves is added to
// the reduced turn.  That goes to fp32, to 1e-7 of an angle; fp32 tensors get what the rounding
// leaves too, by cos(a + r) = cos a - r sin a and sin(a + r) = sin a + r cos a.  (bf16, whose
// outputs are rounded to 2^-8, would pay 3% with a head a token: 131072 tokens, 1 + 1 heads of
// 128, 76.2 us instead of 73.8.)
template <typename T>
__device__ __forceinline__ float2 cos_sin(double position, double inv_freq, float magnitude,
                                          float sign) {
    const double f = __dmul_rn(inv_freq, kInvTwoPi);
    const double low = __fma_rn(inv_freq, kInvTwoPiLow, __fma_rn(inv_freq, kInvTwoPi, -f));
    double t = __dmul_rn(position, f);
    const double left = __fma_rn(position, low, __fma_rn(position, f, -t));
    t = (t - rint(t)) + left;
    const double halves = 2.0 * t;
    const float a = (float)halves;
    float c, s;
    sincospif(a, &s, &c);
    if constexpr (sizeof(typename Elem<T>::raw) == 4) {
        const float r = (float)(halves - (double)a) * 3.14159265f, c0 = c;
        c = __fmaf_rn(-s, r, c);
        s = __fmaf_rn(c0, r, s);
    }
    return make_float2(c * magnitude, s * magnitude * sign);
}

// V elements that follow one another: V = 8 is a chunk, 2 a word or two, 1 a scalar.
template <typename T, int V>
struct Run {
    uint32_t w[V == 8 ? Elem<T>::kWords : V == 2 && Elem<T>::kWords == 8 ? 2 : 1];
};
template <typename T, int V>
__device__ __forceinline__ void load_run(Run<T, V>& r, const void* p) {
    if constexpr (V == 8) {
        Chunk<T> c;
        ld_vec(c, p);
#pragma unroll
        for (int i = 0; i < Elem<T>::kWords; ++i) r.w[i] = c.w[i];
    } else if constexpr (V * sizeof(typename Elem<T>::raw) == 8) {
        const uint2 u = *static_cast<const uint2*>(p);
        r.w[0] = u.x, r.w[1] = u.y;
    } else if constexpr (V * sizeof(typename Elem<T>::raw) == 4) {
        r.w[0] = *static_cast<const uint32_t*>(p);
    } else {
        r.w[0] = *static_cast<const uint16_t*>(p);
    }
}
template <typename T, int V>
__device__ __forceinline__ void store_run(void* p, const Run<T, V>& r) {
    if constexpr (V == 8) {
        Chunk<T> c;
#pragma unroll
        for (int i = 0; i < Elem<T>::kWords; ++i) c.w[i] = r.w[i];
        st_vec(p, c);
    } else if constexpr (V * sizeof(typename Elem<T>::raw) == 8) {
        *static_cast<uint2*>(p) = make_uint2(r.w[0], r.w[1]);
    } else if constexpr (V * sizeof(typename Elem<T>::raw) == 4) {
        *static_cast<uint32_t*>(p) = r.w[0];
    } else {
        *static_cast<uint16_t*>(p) = (uint16_t)r.w[0];
    }
}
template <typename T, int V>
__device__ __forceinline__ void unpack(const Run<T, V>& r, float (&v)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if constexpr (sizeof(typename Elem<T>::raw) == 4)
            v[i] = __uint_as_float(r.w[i]);
        else
            v[i] = __uint_as_float(i & 1 ? r.w[i >> 1] & 0xFFFF0000u : r.w[i >> 1] << 16);
    }
}
template <typename T, int V>
__device__ __forceinline__ void repack(Run<T, V>& r, const float (&v)[V]) {
    if constexpr (sizeof(typename Elem<T>::raw) == 4) {
#pragma unroll
        for (int i = 0; i < V; ++i) r.w[i] = __float_as_uint(v[i]);
    } else if constexpr (V == 1) {
        r.w[0] = pack_bf16(v[0], 0.f);
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) r.w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
    }
}

// 256 pairs are eight blocks of 32 lanes at most.
constexpr int64_t kMaxHeadDim = 512, kMaxHeads = 65536;
constexpr int kWarps = 8;   // of a block
// Heads whose loads a lane issues together: with V = 8 more would cost blocks of registers; with V = 2
// four take 54 us instead of 48 (16384 tokens, 24 + 8 heads of 100, bf16).
template <int V>
__host__ __device__ constexpr int at_once() {
    return V == 8 ? 2 : 8;
}

// How the warps share the work: a warp takes one token, `lanes` items of its heads (V pairs
// each: 2 V elements in two runs) out of `blocks` times as many, and one of `parts` parts
// of its heads, `each` heads; `across` heads at a time.  What is not turned is copied `copy`
// elements an access, after the turned part or, with `split`, by a second warp.
struct RopePlan {
    int lanes, blocks, parts, each, across, copy, split;
};

// Every lane has the cosines and sines of its V pairs in registers and goes over the
// heads with them: they are made once for all heads.  V = 8 where rot_dim / 2 and all
// strides are multiples of 8 elements and the pointers of 8 elements' bytes; there the warp's
// lanes make the angles of its items together, and hand them over in shared memory.
template <typename T, int V, bool INTERLEAVED>
__global__ void __launch_bounds__(32 * kWarps) rope_kernel(const RopeArgs a, const RopePlan p) {
    using raw = typename Elem<T>::raw;
    __shared__ __align__(16) float2 angle[V == 8 ? kWarps : 1][V == 8 ? 256 : 1];
    constexpr int kAtOnce = at_once<V>();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t token = p.split ? (int64_t)blockIdx.x * (kWarps / 2) + (warp >> 1)
                                  : (int64_t)blockIdx.x * kWarps + warp;
    const bool turns = p.split ? !(warp & 1) : a.rot_dim > 0;
    if (token >= a.tokens) return;
    const int part = (int)blockIdx.y / p.blocks, block = (int)blockIdx.y - part * p.blocks;
    const uint32_t b = (uint32_t)token / (uint32_t)a.seq, s = (uint32_t)token - b * (uint32_t)a.seq;
    const raw* const x0 =
        static_cast<const raw*>(a.t[0].x) + b * a.t[0].x_batch_stride + s * a.t[0].x_seq_stride;
    const raw* const x1 =
        static_cast<const raw*>(a.t[1].x) + b * a.t[1].x_batch_stride + s * a.t[1].x_seq_stride;
    raw* const y0 =
        static_cast<raw*>(a.t[0].y) + b * a.t[0].y_batch_stride + s * a.t[0].y_seq_stride;
    raw* const y1 =
        static_cast<raw*>(a.t[1].y) + b * a.t[1].y_batch_stride + s * a.t[1].y_seq_stride;
    const int half = a.rot_dim >> 1, items = half / V;
    const int h0 = part * p.each, h1 = min(h0 + p.each, a.heads);
    auto in_of = [&](int h) {
        return h < a.heads0 ? x0 + h * a.t[0].x_head_stride
                            : x1 + (h - a.heads0) * a.t[1].x_head_stride;
    };
    auto out_of = [&](int h) {
        return h < a.heads0 ? y0 + h * a.t[0].y_head_stride
                            : y1 + (h - a.heads0) * a.t[1].y_head_stride;
    };

    if (turns) {
        const int sub = lane / p.lanes, own = lane - sub * p.lanes;
        const int item = block * 32 + own, f = item * V;
        const bool works = sub < p.across && item < items;
        const int e1 = INTERLEAVED ? 2 * f : f, e2 = INTERLEAVED ? 2 * f + V : f + half;
        Run<T, V> r1[kAtOnce], r2[kAtOnce];
        auto fetch = [&](int h) {
            if (!works || h >= h1) return;
            // behind the last head the last one again: a test for each would part the loads
            // (16384 tokens, 24 + 8 heads of 100, fp32: 131 us instead of 68; 64 tokens lose, bf16 3.3
            // instead of 2.9, and one test at the fifth head costs 80)
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                const raw* const x = in_of(min(h + k * p.across, h1 - 1));
                load_run(r1[k], x + e1);
                load_run(r2[k], x + e2);
            }
        };
        int h = h0 + sub;
        fetch(h);  // on its way while the angles are made
        const double pos = (double)(a.positions ? a.positions[token] : a.start + s);
        float2 turn[V];
        if constexpr (V == 8) {
            const int n = 8 * min(p.lanes, items - block * 32);
            for (int i = lane; i < n; i += 32)
                angle[warp][i] = cos_sin<T>(pos, a.inv_freq[block * 256 + i], a.magnitude, a.sign);
            __syncwarp();
            const float4* const q = reinterpret_cast<const float4*>(angle[warp] + 8 * own);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 t = q[i];
                turn[2 * i] = make_float2(t.x, t.y);
                turn[2 * i + 1] = make_float2(t.z, t.w);
            }
        } else {
            // also in lanes without work (the first pairs', unused): with the call in a branch
            // 16384 tokens of 50 of 128 take 155 us instead of 111
            const int from = works ? f : 0;
#pragma unroll
            for (int i = 0; i < V; ++i)
                turn[i] = cos_sin<T>(pos, a.inv_freq[from + i], a.magnitude, a.sign);
        }
        while (works && h < h1) {
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                const int hk = h + k * p.across;
                if (hk >= h1) continue;
                float u[V], v[V];
                unpack(r1[k], u);
                unpack(r2[k], v);
                if (INTERLEAVED && V > 1) {
                    // the runs are elements 2 f .. 2 f + 2 V - 1, pair i its 2 i and 2 i + 1
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        float* const w = i < V / 2 ? u : v;
                        const int e = 2 * (i % (V > 1 ? V / 2 : 1));
                        const float c = w[e], d = w[e + 1];
                        w[e] = c * turn[i].x - d * turn[i].y;
                        w[e + 1] = d * turn[i].x + c * turn[i].y;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float c = u[i], d = v[i];
                        u[i] = c * turn[i].x - d * turn[i].y;
                        v[i] = d * turn[i].x + c * turn[i].y;
                    }
                }
                repack(r1[k], u);
                repack(r2[k], v);
                raw* const y = out_of(hk);
                store_run(y + e1, r1[k]);
                store_run(y + e2, r2[k]);
            }
            h += kAtOnce * p.across;
            fetch(h);
        }
        if (p.split) return;
    }
    if (block > 0 || a.rot_dim == a.head_dim) return;
    // the rest of each head
    auto copy = [&](auto width) {
        constexpr int W = decltype(width)::value, kBatch = 4;
        const int rest = (a.head_dim - a.rot_dim) / W, n = (h1 - h0) * rest;
        for (int i0 = lane; i0 < n; i0 += 32 * kBatch) {
            Run<T, W> r[kBatch];
            raw* y[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int i = i0 + 32 * k;
                y[k] = nullptr;
                if (i < n) {
                    const int h = i / rest, e = a.rot_dim + (i - h * rest) * W;
                    const raw* const x = in_of(h0 + h);
                    y[k] = out_of(h0 + h);
                    if (x == y[k]) {
                        y[k] = nullptr;  // in place
                    } else {
                        load_run(r[k], x + e);
                        y[k] += e;
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
                if (y[k]) store_run(y[k], r[k]);
        }
    };
    if (p.copy == 8)
        copy(std::integral_constant<int, 8>{});
    else if (p.copy == 2)
        copy(std::integral_constant<int, 2>{});
    else
        copy(std::integral_constant<int, 1>{});
}

template <typename T, int V>
lm_status launch_rope(const RopeArgs& a, bool interleaved, int copy, cudaStream_t s) {
    const int sms = sm_count();
    if (sms <= 0) return LM_ERR_CUDA;
    const int items = (a.rot_dim >> 1) / V;
    RopePlan p;
    p.copy = copy;
    p.lanes = items < 32 ? (items > 0 ? items : 1) : 32;
    p.blocks = items > 32 ? (items + 31) / 32 : 1;
    p.across = 32 / p.lanes;
    // one part, or what gives every multiprocessor 16 warps
    const int64_t warps = a.tokens * p.blocks, want = (int64_t)sms * 16;
    const int64_t most = (a.heads + p.across - 1) / p.across;
    int64_t parts = warps < want ? (want + warps - 1) / warps : 1;
    if (parts > most) parts = most;
    p.each = (int)((a.heads + parts - 1) / parts + p.across - 1) / p.across * p.across;
    p.parts = (a.heads + p.each - 1) / p.each;
    // A second warp for the copy is worth it where few tokens leave the warps waiting (64 tokens,
    // 64 of 128, bf16: 2.5 us instead of 3.2; 1024 tokens 4.4 instead of 4.7; 2048 tokens 9.5 instead of
    // 8.1), and for chunks of fp32 (3999 tokens, 32 of 80: 14.7 instead of 16.2; bf16 8.0 instead of
    // 7.5).
    p.split = items > 0 && a.rot_dim < a.head_dim &&
              (a.tokens <= (int64_t)sms * 8 || (V == 8 && sizeof(typename Elem<T>::raw) == 4));
    const int tokens = p.split ? kWarps / 2 : kWarps;
    // parts * blocks is at most `want` where parts > 1, and 8 otherwise: within the grid's y
    const dim3 grid((unsigned)((a.tokens + tokens - 1) / tokens), (unsigned)(p.parts * p.blocks));
    timing_mark(s, 'r');
    if (interleaved)
        rope_kernel<T, V, true><<<grid, 32 * kWarps, 0, s>>>(a, p);
    else
        rope_kernel<T, V, false><<<grid, 32 * kWarps, 0, s>>>(a, p);
    return launch_status();
}

// Whether the output's strides give every (batch, seq, head) elements of its own.
bool separate(const lm_rope_tensor& t, int64_t batch, int64_t seq, int64_t head_dim) {
    int64_t n[3] = {batch, seq, t.heads};
    int64_t st[3] = {t.y_batch_stride, t.y_seq_stride, t.y_head_stride};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (st[j] < st[i]) {
                const int64_t a = st[i], b = n[i];
                st[i] = st[j], n[i] = n[j], st[j] = a, n[j] = b;
            }
    int64_t span = head_dim;  // elements that the dimensions so far reach over
    for (int i = 0; i < 3; ++i) {
        if (n[i] <= 1) continue;
        if (st[i] < span) return false;
        span += (n[i] - 1) * st[i];
    }
    return true;
}

}  // namespace
}  // namespace lm

extern "C" lm_status lm_rope(const lm_rope_tensor* tensors, int count, int64_t batch, int64_t seq,
                             int64_t head_dim, int64_t rot_dim, lm_dtype dtype,
                             const double* inv_freq, const int64_t* positions, int64_t start,
                             float magnitude, uint32_t flags, lm_stream_t stream) {
    using namespace lm;
    if (dtype != LM_DTYPE_BF16 && dtype != LM_DTYPE_F32) return LM_ERR_UNSUPPORTED_FORMAT;
    if (!tensors || count < 1 || count > 2 || batch < 0 || seq < 0 || head_dim <= 0 ||
        rot_dim < 0 || rot_dim > head_dim || rot_dim % 2 != 0 ||
        (flags & ~(LM_ROPE_INTERLEAVED | LM_ROPE_INVERSE)) || (rot_dim > 0 && !inv_freq) ||
        !(fabsf(magnitude) <= 3.0e38f))
        return LM_ERR_INVALID_ARG;
    const int64_t limit = int64_t(1) << 31;
    if (batch >= limit || seq >= limit || batch * seq >= limit || head_dim > kMaxHeadDim)
        return LM_ERR_UNSUPPORTED_SHAPE;
    RopeArgs a{};
    const unsigned size = dtype == LM_DTYPE_BF16 ? 2 : 4;
    const bool none = batch == 0 || seq == 0;
    // elements of an access: of the turned part they divide rot_dim / 2, of the copied one
    // rot_dim and head_dim, of both the strides
    int v = rot_dim % 16 == 0 ? 8 : rot_dim % 4 == 0 ? 2 : 1;
    int copy = rot_dim % 8 == 0 && head_dim % 8 == 0 ? 8 : head_dim % 2 == 0 ? 2 : 1;
    for (int i = 0; i < count; ++i) {
        const lm_rope_tensor& t = tensors[i];
        if (t.heads < 0) return LM_ERR_INVALID_ARG;
        if (t.heads > kMaxHeads) return LM_ERR_UNSUPPORTED_SHAPE;
        if (none || t.heads == 0) continue;
        if (!t.x || !t.y) return LM_ERR_INVALID_ARG;
        if (t.x_batch_stride < 0 || t.x_seq_stride < 0 || t.x_head_stride < 0 ||
            !separate(t, batch, seq, head_dim))
            return LM_ERR_INVALID_ARG;
        if (t.x == t.y && ((batch > 1 && t.x_batch_stride != t.y_batch_stride) ||
                           (seq > 1 && t.x_seq_stride != t.y_seq_stride) ||
                           (t.heads > 1 && t.x_head_stride != t.y_head_stride)))
            return LM_ERR_INVALID_ARG;
        if (!aligned_to(t.x, size) || !aligned_to(t.y, size)) return LM_ERR_ALIGNMENT;
        const int64_t strides = (batch > 1 ? t.x_batch_stride | t.y_batch_stride : 0) |
                                (seq > 1 ? t.x_seq_stride | t.y_seq_stride : 0) |
                                (t.heads > 1 ? t.x_head_stride | t.y_head_stride : 0);
        auto fits = [&](int n) {
            return strides % n == 0 && aligned_to(t.x, n * size) && aligned_to(t.y, n * size);
        };
        while (v > 1 && !fits(v)) v = v == 8 ? 2 : 1;
        while (copy > 1 && !fits(copy)) copy = copy == 8 ? 2 : 1;
        a.t[i] = t;
        a.heads += (int)t.heads;
        if (i == 0) a.heads0 = (int)t.heads;
    }
    // an output that is the other tensor's input or output
    if (a.t[0].y && (a.t[0].y == a.t[1].y || a.t[0].y == a.t[1].x || a.t[1].y == a.t[0].x))
        return LM_ERR_INVALID_ARG;
    if (!positions && start > INT64_MAX - seq) return LM_ERR_INVALID_ARG;
    if (!aligned_to(inv_freq, 8) || !aligned_to(positions, 8)) return LM_ERR_ALIGNMENT;
    if (none || a.heads == 0) return LM_OK;
    a.batch = batch, a.seq = seq, a.tokens = batch * seq;
    a.head_dim = (int)head_dim, a.rot_dim = (int)rot_dim;
    a.inv_freq = inv_freq, a.positions = positions, a.start = start;
    a.magnitude = magnitude, a.sign = flags & LM_ROPE_INVERSE ? -1.f : 1.f;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool il = flags & LM_ROPE_INTERLEAVED;
    if (dtype == LM_DTYPE_BF16)
        return v == 8   ? launch_rope<bf16_t, 8>(a, il, copy, s)
               : v == 2 ? launch_rope<bf16_t, 2>(a, il, copy, s)
                        : launch_rope<bf16_t, 1>(a, il, copy, s);
    return v == 8   ? launch_rope<f32_t, 8>(a, il, copy, s)
           : v == 2 ? launch_rope<f32_t, 2>(a, il, copy, s)
                    : launch_rope<f32_t, 1>(a, il, copy, s);
}

extern "C" lm_status lm_rope_inv_freq(double theta, int64_t rot_dim, lm_rope_scaling scaling,
                                      double factor, double context, double slow, double fast,
                                      double* inv_freq, float* magnitude) {
    if (!(theta > 0.0 && theta <= 1e300) || rot_dim < 0 || rot_dim % 2 != 0 ||
        (rot_dim > 0 && !inv_freq) || !magnitude)
        return LM_ERR_INVALID_ARG;
    if (scaling < LM_ROPE_UNSCALED || scaling > LM_ROPE_BY_PARTS) return LM_ERR_UNSUPPORTED_FORMAT;
    if (scaling != LM_ROPE_UNSCALED && !(factor >= 1.0 && factor <= 1e9)) return LM_ERR_INVALID_ARG;
    if (scaling == LM_ROPE_NTK && rot_dim <= 2) return LM_ERR_INVALID_ARG;
    if (scaling == LM_ROPE_BY_PARTS && !(context > 0.0 && slow >= 0.0 && fast > slow))
        return LM_ERR_INVALID_ARG;
    if (scaling == LM_ROPE_NTK) theta *= pow(factor, (double)rot_dim / (double)(rot_dim - 2));
    for (int64_t i = 0; i < rot_dim / 2; ++i) {
        double f = pow(theta, -(double)(2 * i) / (double)rot_dim);
        if (scaling == LM_ROPE_LINEAR) {
            f /= factor;
        } else if (scaling == LM_ROPE_BY_PARTS) {
            // the turns of this pair over the original context
            const double turns = context * f * lm::kInvTwoPi;
            const double g = fmin(fmax((turns - slow) / (fast - slow), 0.0), 1.0);
            f = f / factor * (1.0 - g) + f * g;
        }
        inv_freq[i] = f;
    }
    *magnitude = scaling == LM_ROPE_BY_PARTS ? (float)(0.1 * log(factor) + 1.0) : 1.0f;
    return LM_OK;
}
