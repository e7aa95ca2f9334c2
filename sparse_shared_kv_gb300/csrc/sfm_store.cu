// sfm_store.cu -- the write side of the caches: RMS norm, rotary positions,
// quantisation and the store of each row at its slot (sfm_kv_store).
//
// Each value of x is read once and each cache byte written once, so memory
// bounds it.  A group of lanes holds one row in registers, eight values (one
// 16-byte load) per lane and step, so that 16 neighbouring lanes hold one
// 128-value tile: the sum of squares and each tile's largest magnitude are
// shuffles, and so are the partners of half-layout pairs where they sit in the
// same step.  The lanes of a group work out a token's cosines and sines
// together, hand them over through shared memory and keep their own for the
// token's other heads.  The next row's values are under way while a row is
// worked on.  Everything is held in fp32 until the one rounding to the
// cache's format.
//
// Measured on one GB300: 16381 rows of 512 values, normed, rotated and stored as
// bf16: 8.8 us (3.8 TB/s); 131072 index rows (2048 tokens of 64 heads) of 128
// values to E4M3: 17.0 us (3.0 TB/s) and 441488 such rows of 16 heads, normed, 56 us
// (3.0 TB/s), where instructions bound it more than memory; 16381 packed rows of
// 576: 12.4 us as E4M3, 13.7 as int8; 64 packed rows: 2.7 us, latency.  The
// quotients' remainders are 6 to 11 % of the quantised ones.  Eight lanes per row
// with sixteen values each need fewer shuffles but spill the half layout's cosines:
// better by a fifth on the 441488 rows, worse by a fifth on the 131072.
#include <math.h>

#include "sfm_internal.cuh"
#include "sfm_rope.cuh"

namespace sfm {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxDim = 576;
constexpr float kTiny = 0x1p-126f;

struct StoreArgs {
    const void *x;
    const float *weight;
    const int32_t *positions, *slots;
    const double *inv_freq;
    uint8_t *cache;
    float *scales;
    int32_t *status;
    int64_t xt, xh, row_stride, rows, total;   // total: rows of x
    int32_t heads, dim, norm_dim, rot, off, packed_rope;
    FastDiv heads_div;
    float eps, amplitude, inv_norm_dim;
    int32_t norm, half;
};

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d)
{
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)lo | ((uint32_t)hi << 16);
}

__device__ __forceinline__ uint32_t s8x4(float a, float b, float c, float d)
{
    const float f[4] = {a, b, c, d};
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) w |= ((uint32_t)__float2int_rn(fminf(fmaxf(f[i], -127.f), 127.f)) & 0xffu) << (8 * i);
    return w;
}

__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ float max_abs(float a, float b, float c)       // of magnitudes; NaN if one is
{
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

__device__ __forceinline__ float fast_inverse(float x)      // one unit in the last place
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// The quotients below are products with a reciprocal, corrected by what their
// exact remainder is worth (Markstein): q = a y, q += y (a - q b).  The remainder
// takes one multiply-add, and without it the product is off by up to two units in
// the last place, which rounds 0.1 % of the E4M3 codes of plain values the wrong
// way: quotients of 16-bit values meet the codes' halfway points exactly.

// most / M, M = 127 or 448: the quotient rounded to nearest for every magnitude
template <int M>
__device__ __forceinline__ float scale_of(float most)
{
    constexpr float m = (float)M, y = 1.f / m;
    const float q = most * y;
    return most < INFINITY ? fmaf(fmaf(-q, m, most), y, q) : most;      // (NaN and infinity stay)
}

// v / scale for the eight values of a lane, which get lost
__device__ __forceinline__ void quotients(float (&v)[8], float scale, float (&q)[8])
{
    if (scale < 0x1p-90f) {                      // remainders would fall below the least number
        scale *= 0x1p64f;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= 0x1p64f;
    }
    const float y = fast_inverse(scale);
    if (scale == INFINITY) scale = 0.f;          // finite values become 0 and have no remainder
#pragma unroll
    for (int e = 0; e < 8; e += 2)               // two in one instruction
        asm("{\n\t.reg .b64 x, y, s, q;\n\t"
            "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %4};\n\tmov.b64 s, {%5, %5};\n\t"
            "mul.rn.f32x2 q, x, y;\n\tfma.rn.f32x2 x, q, s, x;\n\tfma.rn.f32x2 q, x, y, q;\n\t"
            "mov.b64 {%0, %1}, q;\n\t}"
            : "=f"(q[e]), "=f"(q[e + 1]) : "f"(v[e]), "f"(v[e + 1]), "f"(y), "f"(-scale));
}

// LANES lanes per row, STEPS 16-byte accesses per lane; FORMAT: enum sfm_kv_format;
// ROPE: 0 none, 1 interleaved, 2 half with the rotated part inside one step, 3 half
template <typename T, int FORMAT, int LANES, int STEPS, int ROPE>
__global__ void __launch_bounds__(kThreads) sfm_store_kernel(StoreArgs a)
{
    constexpr int kGroups = kThreads / LANES;
    constexpr int kPairs = ROPE == 0 ? 1 : LANES * STEPS * 4 < kMaxDim / 2 ? LANES * STEPS * 4 : kMaxDim / 2;
    __shared__ unsigned long long step[kPairs];
    __shared__ __align__(16) float2 cs_all[kGroups][kPairs];
    extern __shared__ float turn_all[];          // ROPE 3: [kGroups][rot]

    const int tid = threadIdx.x, lane = tid % LANES, group = tid / LANES;
    grid_follow();
    float2 *cs = cs_all[group];
    float *turn = turn_all + group * a.rot;
    const int pairs = ROPE ? a.rot / 2 : 0;

    // a group takes a run of neighbouring rows, so that the heads of a token
    // share its cosines
    const int64_t groups = (int64_t)gridDim.x * kGroups;
    const int64_t per = (a.total + groups - 1) / groups;
    const int64_t r0 = ((int64_t)blockIdx.x * kGroups + group) * per;
    const int64_t r1 = min(r0 + per, a.total);

    // the next row: its values, and its token's position and slot
    uint4 w[STEPS];
    int32_t position = 0, slot;
    int token = a.heads == 1 ? (int)(r0 < r1 ? r0 : 0) : (int)fdiv((uint32_t)(r0 < r1 ? r0 : 0), a.heads_div);
    int head = (int)((r0 < r1 ? r0 : 0) - (int64_t)token * a.heads);
    const T *src = static_cast<const T *>(a.x) + (int64_t)token * a.xt + (int64_t)head * a.xh + lane * 8;
    const int64_t to_next = a.xt - (int64_t)(a.heads - 1) * a.xh;
    auto load_row = [&] {
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
            w[s] = (s * LANES + lane) * 8 < a.dim ? __ldg(reinterpret_cast<const uint4 *>(src + s * LANES * 8))
                                                  : make_uint4(0, 0, 0, 0);
    };
    auto load_token = [&] {
        slot = a.slots ? __ldg(a.slots + token) : token;
        if (ROPE) position = __ldg(a.positions + token);
    };
    load_row();
    load_token();
    if (ROPE) {
        for (int i = tid; i < pairs; i += kThreads) step[i] = rope::turn_step(__ldg(a.inv_freq + i));
        __syncthreads();
    }

    // cosines and sines of a lane's values: with one step per row (index rows, many heads per token) they stay in
    // registers while the token stays the same
    constexpr int kOwn = ROPE == 1 ? 4 : 8;
    constexpr bool kKeep = ROPE != 0 && STEPS == 1;
    float2 kept[kKeep ? kOwn : 1];
    auto own = [&](int at, float2 (&c)[kOwn]) {
        const int first = ROPE == 1 ? at / 2 : at >= pairs ? at - pairs : at;
#pragma unroll
        for (int e = 0; e < kOwn; e += 2) {
            const float4 two = *reinterpret_cast<const float4 *>(cs + first + e);
            // half layout: the sine's sign is that of the partner's part
            const bool minus = ROPE > 1 && at < pairs;
            c[e] = make_float2(two.x, minus ? -two.y : two.y);
            c[e + 1] = make_float2(two.z, minus ? -two.w : two.w);
        }
    };
    // one step per row: a lane's weights stay in registers too (441488 rows: by a tenth)
    float weight[8];
    if (STEPS == 1) {
#pragma unroll
        for (int e = 0; e < 8; ++e) weight[e] = a.weight && lane * 8 < a.norm_dim ? __ldg(a.weight + lane * 8 + e) : 1.f;
    }
    int last_token = -1;
    const int32_t left = (int32_t)(r1 - r0);     // zero or less: nothing to do for this group
    for (int32_t i = 0; i < (int32_t)per; ++i) { // every group runs the same count: warp collectives inside
        const bool live = i < left;
        float v[STEPS][8];
#pragma unroll
        for (int s = 0; s < STEPS; ++s) rope::unpack8<T>(w[s], v[s]);
        const int32_t this_token = token, this_position = position;
        const bool fresh = this_token != last_token;
        const int64_t row = (int64_t)slot * a.heads + head;
        const bool inside = slot >= 0 && ((int64_t)slot + 1) * a.heads <= a.rows;    // all of the token's rows
        if (live && slot >= 0 && !inside && lane == 0 && a.status) atomicOr(a.status, SFM_STATUS_BAD_BLOCK);
        last_token = this_token;
        if (i + 1 < left) {
            if (++head == a.heads) {
                head = 0;
                ++token;
                src += to_next;
                load_row();
                load_token();
            } else {
                src += a.xh;
                load_row();
            }
        }

        if (a.norm) {
            float sum = 0.f;
#pragma unroll
            for (int s = 0; s < STEPS; ++s)
                if ((s * LANES + lane) * 8 < a.norm_dim) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) sum = fmaf(v[s][e], v[s][e], sum);
                }
#pragma unroll
            for (int o = LANES / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            const float rs = rsqrtf(fmaf(sum, a.inv_norm_dim, a.eps));
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                const int at = (s * LANES + lane) * 8;
                if (at < a.norm_dim) {
                    if (STEPS == 1) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[s][e] = v[s][e] * rs * weight[e];
                    } else if (a.weight) {
                        const float4 w0 = __ldg(reinterpret_cast<const float4 *>(a.weight + at));
                        const float4 w1 = __ldg(reinterpret_cast<const float4 *>(a.weight + at + 4));
                        const float wt[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[s][e] = v[s][e] * rs * wt[e];
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[s][e] *= rs;
                    }
                }
            }
        }

        if (ROPE) {
            if (__any_sync(0xffffffffu, fresh)) {
                __syncwarp();
                for (int p = lane; p < pairs; p += LANES) cs[p] = rope::cos_sin(this_position, step[p], a.amplitude, false);
                __syncwarp();
                if constexpr (kKeep) {
                    const int at = lane * 8 - a.off;
                    if (at >= 0 && at < a.rot) own(at, kept);
                }
            }
            if (ROPE == 3) {
                __syncwarp();
#pragma unroll
                for (int s = 0; s < STEPS; ++s) {
                    const int at = (s * LANES + lane) * 8 - a.off;
                    if (at >= 0 && at < a.rot) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) turn[at + e] = v[s][e];
                    }
                }
                __syncwarp();
            }
            auto rotate_step = [&](float(&x)[8], int at) {
                const bool in = at >= 0 && at < a.rot;
                if (ROPE != 2 && !in) return;
                float2 c[kOwn];
                if constexpr (kKeep) {
#pragma unroll
                    for (int e = 0; e < kOwn; ++e) c[e] = kept[e];
                } else if (in) {
                    own(at, c);
                }
                if (ROPE == 1) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 q = rope::rotate(x[2 * e], x[2 * e + 1], c[e]);
                        x[2 * e] = q.x;
                        x[2 * e + 1] = q.y;
                    }
                } else {
                    const int away = at >= pairs ? -pairs : pairs;       // to the partner
                    const int from = (tid & 31) + (in ? away / 8 : 0);
                    float other[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) other[e] = ROPE == 2 ? __shfl_sync(0xffffffffu, x[e], from) : turn[at + away + e];
                    if (in) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) x[e] = fmaf(x[e], c[e % kOwn].x, other[e] * c[e % kOwn].y);
                    }
                }
            };
            const int at = lane * 8 - a.off;
            // half layout inside one step: the other steps rotate nothing in any lane
            const int only = ROPE == 2 ? a.off / (LANES * 8) : 0;
            if (ROPE != 2 || only == 0) rotate_step(v[0], at);
            if constexpr (STEPS > 1) {
                if (ROPE != 2 || only == 1) rotate_step(v[1], at + LANES * 8);
            }
            if constexpr (STEPS > 2) {
                if (ROPE != 2 || only == 2) rotate_step(v[2], at + 2 * LANES * 8);
            }
        }

        uint8_t *dst = a.cache + row * a.row_stride;
        const bool write = live && inside;
        if constexpr (FORMAT == SFM_KV_PLAIN) {
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                const int at = (s * LANES + lane) * 8;
                if (write && at < a.dim) *reinterpret_cast<uint4 *>(dst + at * 2) = rope::pack8<T>(v[s]);
            }
        } else {
            // largest magnitude per tile: 16 lanes of a step (packed) or the whole row (index rows)
            constexpr bool kRow = FORMAT == SFM_KV_FP8_ROWS;
            float most[STEPS];
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                most[s] = 0.f;
#pragma unroll
                for (int e = 0; e < 8; e += 2) most[s] = max_abs(most[s], v[s][e], v[s][e + 1]);
            }
            if (kRow) {
#pragma unroll
                for (int s = 1; s < STEPS; ++s) most[0] = max_nan(most[0], most[s]);
            }
#pragma unroll
            for (int s = 0; s < (kRow ? 1 : STEPS); ++s) {
#pragma unroll
                for (int o = (kRow ? LANES : 16) / 2; o > 0; o >>= 1)
                    most[s] = max_nan(most[s], __shfl_xor_sync(0xffffffffu, most[s], o));
            }
            constexpr int kMost = FORMAT == SFM_KV_INT8_PACKED ? 127 : 448;
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                const int at = (s * LANES + lane) * 8;
                if (!write || at >= a.dim) continue;
                if (!kRow && at >= 512) {            // the packed row's rope values
                    *reinterpret_cast<uint4 *>(dst + 512 + (at - 512) * 2) = rope::pack8<T>(v[s]);
                    continue;
                }
                const float scale = max_nan(scale_of<kMost>(most[kRow ? 0 : s]), kTiny);
                float f[8];
                quotients(v[s], scale, f);
                uint2 w;
                if (FORMAT == SFM_KV_INT8_PACKED) {
                    w.x = s8x4(f[0], f[1], f[2], f[3]);
                    w.y = s8x4(f[4], f[5], f[6], f[7]);
                } else {
                    w.x = e4m3x4(f[0], f[1], f[2], f[3]);
                    w.y = e4m3x4(f[4], f[5], f[6], f[7]);
                }
                *reinterpret_cast<uint2 *>(dst + at) = w;
                if (kRow) {
                    if (at == 0) a.scales[row] = scale;
                } else if (at % 128 == 0) {
                    reinterpret_cast<float *>(dst + 512 + 2 * a.packed_rope)[at / 128] = scale;
                }
            }
        }
    }
}

template <typename T, int FORMAT, int LANES, int STEPS>
cudaError_t launch(const StoreArgs &a, cudaStream_t st)
{
    constexpr int kGroups = kThreads / LANES;
    int dev = 0, sms = 0;
    const cudaError_t e = current_sms(&dev, &sms);
    if (e != cudaSuccess) return e;
    // four CTAs per SM, what its registers hold (131072 index rows, before the remainders: 16.7 us; with eight, two
    // waves, 17.9; with five of 48 registers 20.0)
    const int64_t want = (a.total + kGroups - 1) / kGroups, most = (int64_t)sms * 4;
    const unsigned grid = (unsigned)(want < most ? want : most);
    const int width = LANES * 8;
    const int form = !a.rot ? 0 : !a.half ? 1 : a.off / width == (a.off + a.rot - 1) / width ? 2 : 3;
    const size_t smem = form == 3 ? (size_t)kGroups * a.rot * sizeof(float) : 0;
    void (*kernel)(StoreArgs) = form == 0   ? sfm_store_kernel<T, FORMAT, LANES, STEPS, 0>
                                : form == 1 ? sfm_store_kernel<T, FORMAT, LANES, STEPS, 1>
                                : form == 2 ? sfm_store_kernel<T, FORMAT, LANES, STEPS, 2>
                                            : sfm_store_kernel<T, FORMAT, LANES, STEPS, 3>;
    return launch_dependent(kernel, dim3(grid), dim3(kThreads), smem, st, a);
}

template <typename T>
cudaError_t launch_type(const StoreArgs &a, int format, cudaStream_t st)
{
    switch (format) {
    case SFM_KV_PLAIN:
        return a.dim <= 128 ? launch<T, SFM_KV_PLAIN, 16, 1>(a, st) : launch<T, SFM_KV_PLAIN, 32, 2>(a, st);
    case SFM_KV_FP8_ROWS:
        return a.dim <= 128 ? launch<T, SFM_KV_FP8_ROWS, 16, 1>(a, st) : launch<T, SFM_KV_FP8_ROWS, 32, 2>(a, st);
    case SFM_KV_INT8_PACKED:
        return a.dim == 512 ? launch<T, SFM_KV_INT8_PACKED, 32, 2>(a, st) : launch<T, SFM_KV_INT8_PACKED, 32, 3>(a, st);
    default:
        return a.dim == 512 ? launch<T, SFM_KV_FP8_PACKED, 32, 2>(a, st) : launch<T, SFM_KV_FP8_PACKED, 32, 3>(a, st);
    }
}

}  // namespace
}  // namespace sfm

using namespace sfm;

extern "C" int sfm_kv_store(const sfm_store_params *pp, const void *x, const float *norm_weight,
                            const int32_t *positions, const double *inv_freq, const int32_t *slots, void *cache,
                            float *scales, int32_t *status, sfm_stream_t stream)
{
    if (!pp) return SFM_ERR_INVALID_ARG;
    const sfm_store_params &p = *pp;
    if (p.tokens < 0 || p.heads < 1 || p.reserved) return SFM_ERR_INVALID_ARG;
    if (p.dtype != SFM_DTYPE_BF16 && p.dtype != SFM_DTYPE_FP16) return SFM_ERR_INVALID_ARG;
    const bool packed = p.kv_format == SFM_KV_INT8_PACKED || p.kv_format == SFM_KV_FP8_PACKED;
    int64_t row_bytes;
    if (packed) {
        if (p.head_dim != 512 && p.head_dim != 576) return SFM_ERR_INVALID_ARG;
        row_bytes = 512 + 2 * (int64_t)(p.head_dim - 512) + 16;
    } else if (p.kv_format == SFM_KV_PLAIN || p.kv_format == SFM_KV_FP8_ROWS) {
        if (p.head_dim < 16 || p.head_dim > 512 || p.head_dim % 16) return SFM_ERR_INVALID_ARG;
        row_bytes = (int64_t)p.head_dim * (p.kv_format == SFM_KV_PLAIN ? 2 : 1);
    } else {
        return SFM_ERR_INVALID_ARG;
    }
    if (p.norm != 0 && p.norm != 1) return SFM_ERR_INVALID_ARG;
    if (p.norm && (!(p.norm_eps >= 0.f) || !isfinite(p.norm_eps))) return SFM_ERR_INVALID_ARG;
    if (p.rope_dim < 0 || p.rope_dim % 16 || p.rope_offset < 0 || p.rope_offset % 8 ||
        p.rope_offset > p.head_dim - p.rope_dim)
        return SFM_ERR_INVALID_ARG;
    if (p.rope_layout != SFM_ROPE_INTERLEAVED && p.rope_layout != SFM_ROPE_HALF) return SFM_ERR_INVALID_ARG;
    if (p.rope_dim && !isfinite(p.amplitude)) return SFM_ERR_INVALID_ARG;
    if (p.rows < 0 || p.rows > ((int64_t)1 << 31) - 2) return SFM_ERR_UNSUPPORTED;
    if ((int64_t)p.tokens * p.heads > ((int64_t)1 << 31) - 2) return SFM_ERR_UNSUPPORTED;
    if (p.row_stride < row_bytes || p.row_stride % 16) return SFM_ERR_LAYOUT;
    if (p.x_token_stride < 0 || p.x_head_stride < 0 || p.x_token_stride % 8 || p.x_head_stride % 8)
        return SFM_ERR_LAYOUT;
    if (norm_weight && !p.norm) return SFM_ERR_INVALID_ARG;
    if ((p.kv_format == SFM_KV_FP8_ROWS) != (scales != nullptr) && p.tokens > 0) return SFM_ERR_INVALID_ARG;
    if (p.tokens == 0) return SFM_OK;
    if (!x || !cache || (p.rope_dim && (!positions || !inv_freq))) return SFM_ERR_INVALID_ARG;
    if (((uintptr_t)x | (uintptr_t)cache | (uintptr_t)norm_weight) & 15u) return SFM_ERR_LAYOUT;
    if (((uintptr_t)positions | (uintptr_t)slots | (uintptr_t)scales) & 3u || (uintptr_t)inv_freq & 7u)
        return SFM_ERR_LAYOUT;

    StoreArgs a = {};
    a.x = x;
    a.weight = norm_weight;
    a.positions = positions;
    a.slots = slots;
    a.inv_freq = inv_freq;
    a.cache = static_cast<uint8_t *>(cache);
    a.scales = scales;
    a.status = status;
    a.xt = p.x_token_stride;
    a.xh = p.x_head_stride;
    a.row_stride = p.row_stride;
    a.rows = p.rows;
    a.total = (int64_t)p.tokens * p.heads;
    a.heads = p.heads;
    a.dim = p.head_dim;
    a.norm_dim = p.head_dim < 512 ? p.head_dim : 512;
    a.rot = p.rope_dim;
    a.off = p.rope_offset;
    a.packed_rope = packed ? p.head_dim - 512 : 0;
    a.heads_div = make_fastdiv((uint32_t)p.heads);
    a.eps = p.norm_eps;
    a.inv_norm_dim = 1.f / (float)a.norm_dim;
    a.amplitude = p.amplitude;
    a.norm = p.norm;
    a.half = p.rope_dim && p.rope_layout == SFM_ROPE_HALF;
    const cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = p.dtype == SFM_DTYPE_BF16 ? launch_type<__nv_bfloat16>(a, p.kv_format, st)
                                                    : launch_type<__half>(a, p.kv_format, st);
    return e == cudaSuccess ? SFM_OK : SFM_ERR_CUDA;
}
