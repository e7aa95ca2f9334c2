// sfm_merge.cu -- attention results over separate sets of keys, joined by
// their LSEs (sfm_merge).
//
//     M = max_n LSE_n,  w_n = e^(LSE_n - M),  O = sum_n w_n O_n / (sum_n w_n + e^(sink - M)),  LSE = M + log sum_n w_n
//
// Every value is read and written once, a few operations each: memory bounds it.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "sfm_internal.cuh"

namespace sfm {
namespace {

constexpr int kThreads = 256;

struct MergeArgs {
    const uint4 *outs[SFM_MERGE_MAX_PARTS];
    const float *lses[SFM_MERGE_MAX_PARTS];
    const float *sinks;
    uint4 *out;
    float *lse;
    int64_t rows;
    int32_t heads, chunks, parts;     // chunks: 16-byte pieces of a row
    FastDiv chunk_div;
};

template <typename T>
__device__ __forceinline__ void widen(uint4 v, float (&f)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (std::is_same<T, __nv_bfloat16>::value) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        } else {
            const float2 p = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            f[2 * i] = p.x;
            f[2 * i + 1] = p.y;
        }
    }
}

template <typename T>
__device__ __forceinline__ uint4 narrow(const float (&f)[8])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (std::is_same<T, __nv_bfloat16>::value) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&p);
        } else {
            const __half2 p = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&p);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// One thread per 16-byte piece of a row.
template <typename T>
__global__ void __launch_bounds__(kThreads) sfm_merge_kernel(const MergeArgs a)
{
    grid_follow();
    const int64_t at = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t row = at / a.chunks;
    if (row >= a.rows) return;
    float w[SFM_MERGE_MAX_PARTS], m = -INFINITY;
    for (int n = 0; n < a.parts; ++n) {
        w[n] = a.lses[n][row];
        m = w[n] > m || w[n] != w[n] ? w[n] : m;       // a NaN stays
    }
    float f[8] = {}, total = 0.f;
    if (m != -INFINITY) {
        for (int n = 0; n < a.parts; ++n) {
            if (w[n] == -INFINITY) continue;
            const float e = expf(w[n] - m);
            float x[8];
            widen<T>(a.outs[n][at], x);
            total += e;
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = fmaf(e, x[i], f[i]);
        }
        const float inv = 1.f / (a.sinks ? total + expf(a.sinks[row % a.heads] - m) : total);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= inv;
    }
    a.out[at] = narrow<T>(f);
    if (a.lse && at == row * a.chunks) a.lse[row] = m == -INFINITY ? m : m + logf(total);
}

}  // namespace
}  // namespace sfm

using namespace sfm;

extern "C" int sfm_merge(const sfm_merge_params *pp, const void *const *outs, const float *const *lses,
                         const float *sinks, void *out, float *lse, sfm_stream_t stream)
{
    if (!pp || !outs || !lses) return SFM_ERR_INVALID_ARG;
    const sfm_merge_params &p = *pp;
    if (p.tokens < 0 || p.heads < 1 || p.head_dim < 1 || p.parts < 1 || p.parts > SFM_MERGE_MAX_PARTS || p.reserved)
        return SFM_ERR_INVALID_ARG;
    if (p.dtype != SFM_DTYPE_BF16 && p.dtype != SFM_DTYPE_FP16) return SFM_ERR_INVALID_ARG;
    if (p.head_dim % 8) return SFM_ERR_LAYOUT;
    if (p.tokens == 0) return SFM_OK;
    if (!out || ((uintptr_t)sinks | (uintptr_t)lse) & 3u) return !out ? SFM_ERR_INVALID_ARG : SFM_ERR_LAYOUT;
    MergeArgs a = {};
    uintptr_t bits = (uintptr_t)out;
    for (int n = 0; n < p.parts; ++n) {
        if (!outs[n] || !lses[n]) return SFM_ERR_INVALID_ARG;
        bits |= (uintptr_t)outs[n] | ((uintptr_t)lses[n] & 3u);
        a.outs[n] = static_cast<const uint4 *>(outs[n]);
        a.lses[n] = lses[n];
    }
    if (bits & 15u) return SFM_ERR_LAYOUT;
    a.sinks = sinks;
    a.out = static_cast<uint4 *>(out);
    a.lse = lse;
    a.rows = (int64_t)p.tokens * p.heads;
    if (a.rows > INT32_MAX) return SFM_ERR_UNSUPPORTED;
    a.heads = p.heads;
    a.chunks = p.head_dim / 8;
    a.parts = p.parts;
    const int64_t blocks = (a.rows * a.chunks + kThreads - 1) / kThreads;
    if (blocks > INT32_MAX) return SFM_ERR_UNSUPPORTED;
    const cudaError_t e = p.dtype == SFM_DTYPE_BF16
                              ? launch_dependent(sfm_merge_kernel<__nv_bfloat16>, dim3((unsigned)blocks), dim3(kThreads), 0,
                                                 (cudaStream_t)stream, a)
                              : launch_dependent(sfm_merge_kernel<__half>, dim3((unsigned)blocks), dim3(kThreads), 0,
                                                 (cudaStream_t)stream, a);
    return e == cudaSuccess ? SFM_OK : SFM_ERR_CUDA;
}
