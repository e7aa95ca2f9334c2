// sfm_rope.cu -- rotary positions of queries and outputs (sfm_rope) and the
// frequencies of the usual context stretchings (sfm_rope_frequencies, host).
//
// Every value is read and written once, so memory bounds it.  A block takes
// steps of 1024 units of one token (or one step of up to 16 tokens with few
// heads): each thread first issues the 16-byte loads of its four units, the
// block then computes the token's cosines and sines once for all heads into
// shared memory while those loads are in flight, and the units are rotated in
// fp32 and stored, one rounding per value.
//
// Measured on one GB300: 4093 tokens of 128 heads of 512 values with 64 of them
// rotated, half layout: 168 us, 6.4 TB/s; 18676 of 64 heads of 128 values: 112
// us; a decode batch of 32 tokens: 2.5 us, latency.  In place 4096 tokens of 128
// heads of 512 with 64 rotated: 27 us, 5.0 TB/s of the rotated part alone.
#include <math.h>

#include "sfm_internal.cuh"
#include "sfm_rope.cuh"

namespace sfm {
namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 4;                      // units of a thread
constexpr int kBlockUnits = kThreads * kUnits;
constexpr int kMaxTokens = 16;                 // tokens of a block
constexpr int kMaxPairs = 2048;                // cosines and sines of a block

struct RopeArgs {
    const void *x;
    void *y;
    const int32_t *positions;
    const double *inv_freq;
    int64_t xt, xh, yt, yh;                    // strides in elements
    int32_t tokens, heads, dim, rot, off;
    int32_t units, token_units, block_tokens;  // units per head, per token; tokens per block
    int32_t block_units, span_tokens;          // rows: units of a token per block, tokens one after the other
    FastDiv units_div, token_div;
    float amplitude;
    int32_t inverse, in_place;
};

// The common form: 16-byte accesses in the order of memory, out of place (or in
// place with interleaved pairs).  A half-layout vector also reads its partners
// (a neighbour loads them too, so they come from L1; by shuffle 8 % slower) and
// writes its own values only.  A block takes a run of a token's vectors, or of
// several tokens, as long as there are blocks enough for every SM: the
// frequencies are turned into steps of a turn once per block (64-bit floating
// point is slow here), the cosines worked out once per token.
template <typename T, bool HALF>
__global__ void __launch_bounds__(kThreads, 4) sfm_rope_rows_kernel(RopeArgs a)
{
    constexpr int kPer = HALF ? 8 : 4;                    // pairs of a vector, and one unused between vectors: then the
    __shared__ float2 cs[kMaxPairs + kMaxPairs / kPer];   // lanes' reads of their e-th pairs meet in no bank
    extern __shared__ unsigned long long step[];          // [rot / 2]
    const int tid = threadIdx.x, half = a.rot / 2;
    grid_follow();
    const int64_t end = min((int64_t)a.tokens, ((int64_t)blockIdx.x + 1) * a.span_tokens);
    bool fresh = true;                                    // the steps are still to come
    for (int64_t t0 = (int64_t)blockIdx.x * a.span_tokens; t0 < end; t0 += a.block_tokens) {
        const int ntok = (int)min((int64_t)a.block_tokens, end - t0);
        const int first = blockIdx.y * a.block_units;
        const int last = min(first + a.block_units, ntok * a.token_units);
        for (int base = first; base < last; base += kBlockUnits) {
            uint4 va[kUnits], vb[kUnits];
            int32_t tok[kUnits], head[kUnits], at[kUnits];
#pragma unroll
            for (int k = 0; k < kUnits; ++k) {
                const int u = base + k * kThreads + tid;
                if (u >= last) continue;
                tok[k] = (int)fdiv((uint32_t)u, a.token_div);
                const int r = u - tok[k] * a.token_units;
                head[k] = (int)fdiv((uint32_t)r, a.units_div);
                at[k] = (r - head[k] * a.units) * 8 + (a.in_place ? a.off : 0);
                const T *src = static_cast<const T *>(a.x) + (t0 + tok[k]) * a.xt + (int64_t)head[k] * a.xh + at[k];
                va[k] = *reinterpret_cast<const uint4 *>(src);
                const int in = at[k] - a.off;
                if (HALF && in >= 0 && in < a.rot) vb[k] = *reinterpret_cast<const uint4 *>(src + (in < half ? half : -half));
            }
            if (base == first) {                          // (the loads above are on their way)
                if (fresh) {
                    for (int i = tid; i < half; i += kThreads) step[i] = rope::turn_step(__ldg(a.inv_freq + i));
                    fresh = false;
                }
                __syncthreads();                          // the steps are there, the last tokens' cosines have been read
                for (int i = tid; i < ntok * half; i += kThreads) {
                    const int t = i / half, p = i - t * half;
                    cs[i + i / kPer] = rope::cos_sin(__ldg(a.positions + t0 + t), step[p], a.amplitude, a.inverse != 0);
                }
                __syncthreads();
            }
#pragma unroll
            for (int k = 0; k < kUnits; ++k) {
                if (base + k * kThreads + tid >= last) continue;
                const int in = at[k] - a.off;
                if (in >= 0 && in < a.rot) {
                    float p[8];
                    rope::unpack8<T>(va[k], p);
                    const float2 *c = cs + (tok[k] * half / kPer + (HALF ? (in < half ? in : in - half) : in) / 8) * (kPer + 1);
                    if (HALF) {
                        float q[8];
                        rope::unpack8<T>(vb[k], q);
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float2 t = c[e];
                            p[e] = fmaf(p[e], t.x, in < half ? -q[e] * t.y : q[e] * t.y);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 r = rope::rotate(p[2 * e], p[2 * e + 1], c[e]);
                            p[2 * e] = r.x;
                            p[2 * e + 1] = r.y;
                        }
                    }
                    va[k] = rope::pack8<T>(p);
                }
                T *dst = static_cast<T *>(a.y) + (t0 + tok[k]) * a.yt + (int64_t)head[k] * a.yh + at[k];
                *reinterpret_cast<uint4 *>(dst) = va[k];
            }
        }
    }
}

// The other forms: half layout in place, and rows without 16-byte accesses.
// VEC: values per access (8 or 1).  A unit is two accesses that hold the
// first and second members of VEC pairs, or one access outside the rotated
// part, which is copied.
template <typename T, int VEC, bool HALF>
__global__ void __launch_bounds__(kThreads) sfm_rope_kernel(RopeArgs a)
{
    using Access = typename std::conditional<VEC == 8, uint4, T>::type;
    __shared__ float2 cs[kMaxPairs];

    const int tid = threadIdx.x;
    grid_follow();
    const int64_t t0 = (int64_t)blockIdx.x * a.block_tokens;
    const int ntok = (int)min((int64_t)a.block_tokens, a.tokens - t0);
    const int first = blockIdx.y * kBlockUnits;
    const int last = min(first + kBlockUnits, ntok * a.token_units);
    const int pair_units = a.rot / 2 / VEC;

    Access va[kUnits], vb[kUnits];
    int64_t ya[kUnits];
    int32_t other[kUnits], pair[kUnits];       // distance to the second access (0: none); cs index (-1: copy)
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
        const int u = first + k * kThreads + tid;
        other[k] = 0;
        pair[k] = -2;
        if (u >= last) continue;
        const int tok = (int)fdiv((uint32_t)u, a.token_div);
        const int r = u - tok * a.token_units;
        const int head = (int)fdiv((uint32_t)r, a.units_div);
        const int i = r - head * a.units;
        const int64_t t = t0 + tok;
        int at;
        if (i < pair_units) {
            at = a.off + (HALF ? i * VEC : 2 * i);
            other[k] = HALF ? a.rot / 2 : 1;
            pair[k] = tok * (a.rot / 2) + i;
        } else {
            at = (i - pair_units) * VEC;
            if (at >= a.off) at += a.rot;
            pair[k] = -1;
        }
        const T *src = static_cast<const T *>(a.x) + t * a.xt + (int64_t)head * a.xh + at;
        va[k] = *reinterpret_cast<const Access *>(src);
        if (other[k]) vb[k] = *reinterpret_cast<const Access *>(src + other[k]);
        ya[k] = t * a.yt + (int64_t)head * a.yh + at;
    }

    const int np = ntok * (a.rot / 2);
    for (int i = tid; i < np; i += kThreads) {
        const int tok = i / (a.rot / 2), p = i - tok * (a.rot / 2);
        // the e-th pairs of all units side by side: neighbouring lanes read neighbouring words
        cs[i - p + (p % VEC) * (a.rot / 2 / VEC) + p / VEC] =
            rope::cos_sin(__ldg(a.positions + t0 + tok), rope::turn_step(__ldg(a.inv_freq + p)), a.amplitude, a.inverse != 0);
    }
    __syncthreads();

#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
        if (pair[k] == -2) continue;
        T *dst = static_cast<T *>(a.y) + ya[k];
        if (pair[k] >= 0) {
            if constexpr (VEC == 8) {
                float p[8], q[8];
                rope::unpack8<T>(va[k], p);
                rope::unpack8<T>(vb[k], q);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float2 r = rope::rotate(p[e], q[e], cs[pair[k] + e * (a.rot / 2 / VEC)]);
                    p[e] = r.x;
                    q[e] = r.y;
                }
                va[k] = rope::pack8<T>(p);
                vb[k] = rope::pack8<T>(q);
            } else {
                const float2 r = rope::rotate(rope::Pair<T>::one(va[k]), rope::Pair<T>::one(vb[k]), cs[pair[k]]);
                va[k] = rope::Pair<T>::round(r.x);
                vb[k] = rope::Pair<T>::round(r.y);
            }
        }
        *reinterpret_cast<Access *>(dst) = va[k];
        if (other[k]) *reinterpret_cast<Access *>(dst + other[k]) = vb[k];
    }
}

// whether two of the tokens x heads rows of `width` values share a value
// (what is written there would have no one answer)
bool rows_overlap(int64_t tokens, int64_t token_stride, int64_t heads, int64_t head_stride, int64_t width)
{
    int64_t span = width;
    const bool heads_inner = head_stride <= token_stride;
    for (int i = 0; i < 2; ++i) {
        const bool h = heads_inner == (i == 0);
        const int64_t n = h ? heads : tokens, stride = h ? head_stride : token_stride;
        if (n <= 1) continue;
        if (stride < span) return true;
        span += stride * (n - 1);
    }
    return false;
}

template <typename T, int VEC, bool HALF>
cudaError_t launch(const RopeArgs &a, dim3 grid, cudaStream_t st)
{
    return launch_dependent(sfm_rope_kernel<T, VEC, HALF>, grid, dim3(kThreads), 0, st, a);
}

template <typename T, bool HALF>
cudaError_t launch_rows(const RopeArgs &a, dim3 grid, cudaStream_t st)
{
    return launch_dependent(sfm_rope_rows_kernel<T, HALF>, grid, dim3(kThreads), (size_t)a.rot / 2 * 8, st, a);
}

template <typename T>
cudaError_t launch_type(const RopeArgs &a, int vec, bool half, bool rows, dim3 grid, cudaStream_t st)
{
    if (rows) return half ? launch_rows<T, true>(a, grid, st) : launch_rows<T, false>(a, grid, st);
    if (vec == 8) return launch<T, 8, true>(a, grid, st);
    return half ? launch<T, 1, true>(a, grid, st) : launch<T, 1, false>(a, grid, st);
}

}  // namespace
}  // namespace sfm

using namespace sfm;

extern "C" int sfm_rope_frequencies(const sfm_rope_spec *s, double *inv_freq, float *amplitude)
{
    if (!s || !inv_freq || !amplitude) return SFM_ERR_INVALID_ARG;
    if (s->rope_dim <= 0 || s->rope_dim % 2 || !(s->base > 1.0) || !isfinite(s->base) || s->reserved)
        return SFM_ERR_INVALID_ARG;
    if (s->scaling < SFM_ROPE_SCALING_NONE || s->scaling > SFM_ROPE_SCALING_YARN) return SFM_ERR_INVALID_ARG;
    if (s->scaling != SFM_ROPE_SCALING_NONE && (!(s->factor >= 1.0) || !isfinite(s->factor)))
        return SFM_ERR_INVALID_ARG;
    if (s->scaling == SFM_ROPE_SCALING_NTK && s->rope_dim <= 2) return SFM_ERR_INVALID_ARG;
    if (s->scaling == SFM_ROPE_SCALING_YARN &&
        (s->original_max_position <= 0 || !(s->beta_slow > 0.0) || !(s->beta_fast > s->beta_slow) ||
         !isfinite(s->beta_fast)))
        return SFM_ERR_INVALID_ARG;
    const int n = s->rope_dim;
    double base = s->base;
    if (s->scaling == SFM_ROPE_SCALING_NTK) base *= pow(s->factor, (double)n / (n - 2));
    // the pair index that turns `turns` times within the original context
    const double two_pi = 6.283185307179586;
    auto pair_of = [&](double turns) {
        return n * log(s->original_max_position / (turns * two_pi)) / (2.0 * log(base));
    };
    double lo = 0.0, hi = 0.0;
    if (s->scaling == SFM_ROPE_SCALING_YARN) {
        lo = fmax(floor(pair_of(s->beta_fast)), 0.0);
        hi = fmin(ceil(pair_of(s->beta_slow)), n - 1.0);
    }
    for (int i = 0; i < n / 2; ++i) {
        double f = pow(base, -2.0 * i / n);
        if (s->scaling == SFM_ROPE_SCALING_LINEAR) f /= s->factor;
        if (s->scaling == SFM_ROPE_SCALING_YARN) {
            const double ramp = fmin(fmax((i - lo) / fmax(hi - lo, 0.001), 0.0), 1.0);
            f = f / s->factor * ramp + f * (1.0 - ramp);
        }
        inv_freq[i] = f;
    }
    *amplitude = s->scaling == SFM_ROPE_SCALING_YARN ? (float)(0.1 * log(s->factor) + 1.0) : 1.0f;
    return SFM_OK;
}

extern "C" int sfm_rope(const sfm_rope_params *pp, const void *x, const int32_t *positions, const double *inv_freq,
                        void *y, sfm_stream_t stream)
{
    if (!pp) return SFM_ERR_INVALID_ARG;
    const sfm_rope_params &p = *pp;
    if (p.tokens < 0 || p.heads < 1 || p.head_dim < 1 || p.head_dim > 4096 || p.reserved) return SFM_ERR_INVALID_ARG;
    if (p.rope_dim < 2 || p.rope_dim % 2 || p.rope_offset < 0 || p.rope_offset > p.head_dim - p.rope_dim)
        return SFM_ERR_INVALID_ARG;
    if (p.rope_layout != SFM_ROPE_INTERLEAVED && p.rope_layout != SFM_ROPE_HALF) return SFM_ERR_INVALID_ARG;
    if (p.inverse != 0 && p.inverse != 1) return SFM_ERR_INVALID_ARG;
    if (p.dtype != SFM_DTYPE_BF16 && p.dtype != SFM_DTYPE_FP16) return SFM_ERR_INVALID_ARG;
    if (!isfinite(p.amplitude)) return SFM_ERR_INVALID_ARG;
    if (p.x_token_stride < 0 || p.x_head_stride < 0 || p.y_token_stride < 0 || p.y_head_stride < 0)
        return SFM_ERR_LAYOUT;
    if (p.tokens == 0) return SFM_OK;
    if (!x || !y || !positions || !inv_freq) return SFM_ERR_INVALID_ARG;
    if (((uintptr_t)x | (uintptr_t)y) & 1u || (uintptr_t)positions & 3u || (uintptr_t)inv_freq & 7u)
        return SFM_ERR_LAYOUT;
    const bool in_place = x == y;
    if (in_place && (p.x_token_stride != p.y_token_stride || p.x_head_stride != p.y_head_stride)) return SFM_ERR_LAYOUT;
    if (rows_overlap(p.tokens, p.y_token_stride, p.heads, p.y_head_stride, p.head_dim)) return SFM_ERR_LAYOUT;

    const bool half = p.rope_layout == SFM_ROPE_HALF;
    const int64_t strides = p.x_token_stride | p.x_head_stride | p.y_token_stride | p.y_head_stride;
    // whole 16-byte accesses where every row, and the rotated part in it, allows them
    const bool wide = (((uintptr_t)x | (uintptr_t)y) & 15u) == 0 && strides % 8 == 0 && p.head_dim % 8 == 0 &&
                      p.rope_offset % 8 == 0 && (half ? p.rope_dim / 2 : p.rope_dim) % 8 == 0;
    const int vec = wide ? 8 : 1;

    RopeArgs a = {};
    a.x = x;
    a.y = y;
    a.positions = positions;
    a.inv_freq = inv_freq;
    a.xt = p.x_token_stride;
    a.xh = p.x_head_stride;
    a.yt = p.y_token_stride;
    a.yh = p.y_head_stride;
    a.tokens = p.tokens;
    a.heads = p.heads;
    a.dim = p.head_dim;
    a.rot = p.rope_dim;
    a.off = p.rope_offset;
    a.inverse = p.inverse;
    a.in_place = in_place;
    a.amplitude = p.amplitude;
    const bool rows = vec == 8 && (!half || !in_place);
    a.units = (rows ? p.rope_dim / vec : p.rope_dim / 2 / vec) + (in_place ? 0 : (p.head_dim - p.rope_dim) / vec);
    const int64_t token_units = (int64_t)a.units * p.heads;
    int dev = 0, sms = 0;
    if (current_sms(&dev, &sms) != cudaSuccess) return SFM_ERR_CUDA;
    // rows: a block takes up to eight steps of 1024 units, of one token or of
    // several, while there are 16 blocks for every SM
    int64_t steps = 1;
    while (rows && steps < 8 && p.tokens * token_units / (2 * steps * kBlockUnits) >= 16 * (int64_t)sms) steps *= 2;
    a.block_units = (int32_t)(steps * kBlockUnits);
    const int64_t chunks = (token_units + a.block_units - 1) / a.block_units;
    if (chunks > 65535) return SFM_ERR_UNSUPPORTED;
    a.token_units = (int32_t)token_units;
    int64_t bt = kBlockUnits / token_units;
    bt = bt < kMaxPairs / (p.rope_dim / 2) ? bt : kMaxPairs / (p.rope_dim / 2);
    a.block_tokens = (int32_t)(bt < 1 ? 1 : bt > kMaxTokens ? kMaxTokens : bt);
    a.units_div = make_fastdiv((uint32_t)a.units);
    a.token_div = make_fastdiv((uint32_t)token_units);
    const int64_t groups = rows && chunks == 1 ? steps * kBlockUnits / (a.block_tokens * token_units) : 1;
    a.span_tokens = (int32_t)(a.block_tokens * (groups > 1 ? groups : 1));
    const int64_t span = rows ? a.span_tokens : a.block_tokens;
    const dim3 grid((unsigned)((p.tokens + span - 1) / span), (unsigned)chunks);
    const cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = p.dtype == SFM_DTYPE_BF16 ? launch_type<__nv_bfloat16>(a, vec, half, rows, grid, st)
                                                    : launch_type<__half>(a, vec, half, rows, grid, st);
    return e == cudaSuccess ? SFM_OK : SFM_ERR_CUDA;
}
