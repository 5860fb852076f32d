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
//
// HBM-bound: every element read and written once.
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

__device__ __forceinline__ float ld1(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }
__device__ __forceinline__ float ld1(const uint32_t* p) { return __uint_as_float(*p); }
__device__ __forceinline__ void st1(uint16_t* p, float v) { *p = (uint16_t)pack_bf16(v, 0.f); }
__device__ __forceinline__ void st1(uint32_t* p, float v) { *p = __float_as_uint(v); }

__device__ __forceinline__ void cos_sin(double position, double inv_freq, float magnitude,
                                        float sign, float& c, float& s) {
    double t = position * (inv_freq * kInvTwoPi);
    t -= rint(t);
    sincospif((float)(2.0 * t), &s, &c);
    c *= magnitude;
    s *= magnitude * sign;
}

// One thread a pair or a copied element of one head of one token.
template <typename T, bool INTERLEAVED>
__global__ void __launch_bounds__(256) rope_kernel(const RopeArgs a) {
    using raw = typename Elem<T>::raw;
    const int half = a.rot_dim >> 1, items = a.head_dim - half;
    const int64_t per_token = (int64_t)a.heads * items, n = a.tokens * per_token;
    for (int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x; k < n; k += (int64_t)gridDim.x * 256) {
        const int64_t token = k / per_token;
        const int64_t rest = k - token * per_token;
        int h = (int)(rest / items);
        const int i = (int)(rest - (int64_t)h * items);
        const lm_rope_tensor& t = h < a.heads0 ? a.t[0] : a.t[1];
        if (h >= a.heads0) h -= a.heads0;
        const int64_t b = token / a.seq, s = token - b * a.seq;
        const raw* x = static_cast<const raw*>(t.x) + b * t.x_batch_stride + s * t.x_seq_stride +
                       h * t.x_head_stride;
        raw* y = static_cast<raw*>(t.y) + b * t.y_batch_stride + s * t.y_seq_stride +
                 h * t.y_head_stride;
        if (i >= half) {  // not rotated
            const int e = i + half;
            if (x != y) y[e] = x[e];
            continue;
        }
        const double pos = (double)(a.positions ? a.positions[token] : a.start + s);
        float c, sn;
        cos_sin(pos, a.inv_freq[i], a.magnitude, a.sign, c, sn);
        const int e1 = INTERLEAVED ? 2 * i : i, e2 = INTERLEAVED ? 2 * i + 1 : i + half;
        const float x1 = ld1(x + e1), x2 = ld1(x + e2);
        st1(y + e1, x1 * c - x2 * sn);
        st1(y + e2, x2 * c + x1 * sn);
    }
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
    if (batch >= limit || seq >= limit || batch * seq >= limit || head_dim > 65536)
        return LM_ERR_UNSUPPORTED_SHAPE;
    RopeArgs a{};
    const unsigned size = dtype == LM_DTYPE_BF16 ? 2 : 4;
    const bool none = batch == 0 || seq == 0;
    for (int i = 0; i < count; ++i) {
        const lm_rope_tensor& t = tensors[i];
        if (t.heads < 0) return LM_ERR_INVALID_ARG;
        if (t.heads * head_dim >= (int64_t(1) << 30)) return LM_ERR_UNSUPPORTED_SHAPE;
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
    const int sms = sm_count();
    if (sms <= 0) return LM_ERR_CUDA;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int64_t n = a.tokens * a.heads * (head_dim - rot_dim / 2);
    const int64_t want = (n + 255) / 256, most = (int64_t)sms * 32;
    const unsigned grid = (unsigned)(want < most ? want : most);
    const bool il = flags & LM_ROPE_INTERLEAVED;
    timing_mark(s, 'r');
    if (dtype == LM_DTYPE_BF16) {
        if (il)
            rope_kernel<bf16_t, true><<<grid, 256, 0, s>>>(a);
        else
            rope_kernel<bf16_t, false><<<grid, 256, 0, s>>>(a);
    } else {
        if (il)
            rope_kernel<f32_t, true><<<grid, 256, 0, s>>>(a);
        else
            rope_kernel<f32_t, false><<<grid, 256, 0, s>>>(a);
    }
    return launch_status();
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
