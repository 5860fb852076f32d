// lm_rope.cu -- rotary positions of up to two tensors (Q and K) in one launch.
//
// Pair i of a head's first `rot_dim` elements is turned by the angle
// a = position * inv_freq[i]:
//
//   (x1, x2) -> m (x1 cos a - x2 sin a, x2 cos a + x1 sin a)
//
// (rotary position embedding: J. Su et al., "RoFormer", 2021); the backward pass
// is the same with the sine negated.  The angle is taken in turns in fp64,
// t = position * inv_freq / 2 pi, and only t - rint(t) goes to fp32, so the
// rotation is right at any position; no table is kept or read.  The other
// head_dim - rot_dim elements are copied (not touched in place).
#include "lm_chunk.cuh"
#include "lm_internal.h"
#include "lm_rows.h"

namespace lm {
namespace {

struct RopeArgs {
    lm_rope_tensor t[2];
    int64_t batch, seq, tokens;
    int heads0, heads, head_dim, rot_dim;
    const double* inv_freq;
    const int64_t* positions;
    int64_t start;
    float magnitude, sign;
};

constexpr double kInvTwoPi = 0.15915494309189533576888376337251;

// cos and sin of position * inv_freq, times the magnitude, the sine with `sign`.
__device__ __forceinline__ float2 cos_sin(double position, double inv_freq, float magnitude,
                                          float sign) {
    double t = position * (inv_freq * kInvTwoPi);
    t -= rint(t);
    float c, s;
    sincospif((float)(2.0 * t), &s, &c);
    return make_float2(c * magnitude, s * magnitude * sign);
}

// V elements that follow one another: V = 8 is a chunk, V = 1 a scalar.
template <typename T, int V>
struct Run {
    float v[V];
};
template <typename T, int V>
__device__ __forceinline__ void load_run(Run<T, V>& r, const void* p) {
    if constexpr (V == 8) {
        Chunk<T> c;
        ld_vec(c, p);
#pragma unroll
        for (int i = 0; i < 8; ++i) r.v[i] = get(c, i);
    } else if constexpr (sizeof(typename Elem<T>::raw) == 4) {
        r.v[0] = *static_cast<const float*>(p);
    } else {
        r.v[0] = __uint_as_float((uint32_t)*static_cast<const uint16_t*>(p) << 16);
    }
}
template <typename T, int V>
__device__ __forceinline__ void store_run(void* p, const Run<T, V>& r) {
    if constexpr (V == 8) {
        Chunk<T> c;
        put(c, r.v);
        st_vec(p, c);
    } else if constexpr (sizeof(typename Elem<T>::raw) == 4) {
        *static_cast<float*>(p) = r.v[0];
    } else {
        *static_cast<uint16_t*>(p) = (uint16_t)pack_bf16(r.v[0], 0.f);
    }
}

// 256 threads take an item each of a head of this size; 32 tokens' heads are counted in 32
// bits.
constexpr int64_t kMaxHeadDim = 512, kMaxHeads = 65536;
constexpr int kThreads = 256;
constexpr int kAngles = 2048;  // of a block, in shared memory: 16 KB
constexpr int kTokens = 32;    // of a block, at most
constexpr int kAtOnce = 4;     // heads whose loads a thread issues together

// A block takes `tokens` tokens: first their angles, each once for all heads, into shared
// memory; then every thread keeps one item of a head (V pairs: 2 V elements in two
// runs) and goes over the heads of the tokens, `at_once` at a time.  V = 8 where
// rot_dim / 2 and all strides are multiples of 8 elements and the pointers of 8 elements'
// bytes; V = 1 otherwise.
template <typename T, int V, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeArgs a, int tokens) {
    using raw = typename Elem<T>::raw;
    __shared__ __align__(16) float2 angle[kAngles];
    __shared__ const raw* from[2][kTokens];
    __shared__ raw* to[2][kTokens];
    const int half = a.rot_dim >> 1, heads = a.heads;
    const int64_t token0 = (int64_t)blockIdx.x * tokens;
    const int n = (int)(a.tokens - token0 < tokens ? a.tokens - token0 : tokens);
    for (int i = threadIdx.x; i < 2 * n; i += kThreads) {
        const int k = i >= n, t = i - k * n;
        const int64_t b = (token0 + t) / a.seq, s = token0 + t - b * a.seq;
        from[k][t] = static_cast<const raw*>(a.t[k].x) + b * a.t[k].x_batch_stride +
                     s * a.t[k].x_seq_stride;
        to[k][t] = static_cast<raw*>(a.t[k].y) + b * a.t[k].y_batch_stride +
                   s * a.t[k].y_seq_stride;
    }
    for (int i = threadIdx.x; i < n * half; i += kThreads) {
        const int t = i / half, f = i - t * half;
        const int64_t token = token0 + t;
        const int64_t pos = a.positions ? a.positions[token] : a.start + token % a.seq;
        angle[i] = cos_sin((double)pos, a.inv_freq[f], a.magnitude, a.sign);
    }
    __syncthreads();

    // the rotated part: `items` threads a head, `rows` heads at a time
    const int items = half / V;
    if (items > 0) {
        const int rows = kThreads / items, row = threadIdx.x / items;
        const int f = (threadIdx.x - row * items) * V;
        const int e1 = INTERLEAVED ? 2 * f : f, e2 = INTERLEAVED ? 2 * f + V : f + half;
        const int units = row < rows ? n * heads : 0;
        for (int u0 = row; u0 < units; u0 += rows * kAtOnce) {
            Run<T, V> x1[kAtOnce], x2[kAtOnce];
            raw* y[kAtOnce];
            const float2* cs[kAtOnce];
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                const int u = u0 + k * rows;
                y[k] = nullptr;
                if (u < units) {
                    const int t = u / heads, h = u - t * heads;
                    const int w = h >= a.heads0;
                    const int64_t hh = h - (w ? a.heads0 : 0);
                    const raw* x = from[w][t] + hh * (w ? a.t[1] : a.t[0]).x_head_stride;
                    y[k] = to[w][t] + hh * (w ? a.t[1] : a.t[0]).y_head_stride;
                    cs[k] = angle + t * half + f;
                    load_run(x1[k], x + e1);
                    load_run(x2[k], x + e2);
                }
            }
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                if (!y[k]) continue;
                float2 turn[V];
                if constexpr (V == 8) {
                    const float4* const p = reinterpret_cast<const float4*>(cs[k]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 q = p[i];
                        turn[2 * i] = make_float2(q.x, q.y);
                        turn[2 * i + 1] = make_float2(q.z, q.w);
                    }
                } else {
                    turn[0] = *cs[k];
                }
                if (INTERLEAVED && V > 1) {
                    // the runs are 2 f .. 2 f + 2 V - 1: pair i is elements 2 i and 2 i + 1 of them
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float2 c = turn[i];
                        float* const v = i < V / 2 ? x1[k].v : x2[k].v;
                        const int e = 2 * (i % (V / 2 > 0 ? V / 2 : 1));
                        const float p = v[e], q = v[e + 1];
                        v[e] = p * c.x - q * c.y;
                        v[e + 1] = q * c.x + p * c.y;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float2 c = turn[i];
                        const float p = x1[k].v[i], q = x2[k].v[i];
                        x1[k].v[i] = p * c.x - q * c.y;
                        x2[k].v[i] = q * c.x + p * c.y;
                    }
                }
                store_run(y[k] + e1, x1[k]);
                store_run(y[k] + e2, x2[k]);
            }
        }
    }
    // the rest of each head, copied
    const int rest = (a.head_dim - a.rot_dim) / V;
    const int copies = n * heads * rest;
    for (int i = threadIdx.x; i < copies; i += kThreads) {
        const int u = i / rest, e = a.rot_dim + (i - u * rest) * V;
        const int t = u / heads, h = u - t * heads;
        const int w = h >= a.heads0;
        const int64_t hh = h - (w ? a.heads0 : 0);
        const raw* x = from[w][t] + hh * (w ? a.t[1] : a.t[0]).x_head_stride;
        raw* y = to[w][t] + hh * (w ? a.t[1] : a.t[0]).y_head_stride;
        if (x == y) continue;
        if constexpr (V == 8) {
            Chunk<T> c;
            ld_vec(c, x + e);
            st_vec(y + e, c);
        } else {
            y[e] = x[e];
        }
    }
}

template <typename T, int V>
lm_status launch_rope(const RopeArgs& a, bool interleaved, cudaStream_t s) {
    const int sms = sm_count();
    if (sms <= 0) return LM_ERR_CUDA;
    const int half = a.rot_dim >> 1;
    // the heads that a block's threads take at once, kAtOnce times, in whole tokens; fewer
    // where that would leave multiprocessors idle
    const int items = half / V > 0 ? half / V : 1;
    int64_t tokens = ((int64_t)(kThreads / items) * kAtOnce + a.heads - 1) / a.heads;
    if (half > 0 && tokens > kAngles / half) tokens = kAngles / half;
    if (tokens > kTokens) tokens = kTokens;
    if (tokens > a.tokens / (2 * sms)) tokens = a.tokens / (2 * sms);
    if (tokens < 1) tokens = 1;
    const int64_t blocks = (a.tokens + tokens - 1) / tokens;
    timing_mark(s, 'r');
    if (interleaved)
        rope_kernel<T, V, true><<<(unsigned)blocks, kThreads, 0, s>>>(a, (int)tokens);
    else
        rope_kernel<T, V, false><<<(unsigned)blocks, kThreads, 0, s>>>(a, (int)tokens);
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
    // whole chunks, of both runs of an item and of what is copied
    bool vec = rot_dim % 16 == 0 && head_dim % 8 == 0;
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
        vec = vec && strides % 8 == 0 && aligned_to(t.x, 8 * size) && aligned_to(t.y, 8 * size);
        a.t[i] = t;
        a.heads += (int)t.heads;
        if (i == 0) a.heads0 = (int)t.heads;
    }
    if (!aligned_to(inv_freq, 8) || !aligned_to(positions, 8)) return LM_ERR_ALIGNMENT;
    if (none || a.heads == 0) return LM_OK;
    a.batch = batch, a.seq = seq, a.tokens = batch * seq;
    a.head_dim = (int)head_dim, a.rot_dim = (int)rot_dim;
    a.inv_freq = inv_freq, a.positions = positions, a.start = start;
    a.magnitude = magnitude, a.sign = flags & LM_ROPE_INVERSE ? -1.f : 1.f;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool il = flags & LM_ROPE_INTERLEAVED;
    if (dtype == LM_DTYPE_BF16)
        return vec ? launch_rope<bf16_t, 8>(a, il, s) : launch_rope<bf16_t, 1>(a, il, s);
    return vec ? launch_rope<f32_t, 8>(a, il, s) : launch_rope<f32_t, 1>(a, il, s);
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
