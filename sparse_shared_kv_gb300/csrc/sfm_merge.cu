// sfm_merge.cu -- attention results over separate sets of keys, joined by
// their LSEs (sfm_merge).
//
//     M = max_n LSE_n,  w_n = e^(LSE_n - M),  O = sum_n w_n O_n / (sum_n w_n + e^(sink - M)),  LSE = M + log sum_n w_n
//
// Every value is read and written once, a few operations each: memory bounds
// it.  A warp takes a row at a time; its lanes work out the same weights and
// take 16 bytes of the row each, all parts' loads before the first use.  4093 x 64
// rows of 512: fp16 119 us of two parts (6.8 TB/s), 150 of three (7.1), 193 of four,
// 342 of eight (7.1); bf16, whose kernels take more registers (three parts 110
// instead of 64, eight 189 instead of 118), 117 (6.9 TB/s), 189 (5.7), 201, 424
// (5.7).  A thread per 16 bytes that each found its row and weights took 242 of
// three fp16 parts.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "sfm_internal.cuh"

namespace sfm {
namespace {

constexpr int kWarps = 8;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct MergeArgs {
    const uint4 *outs[SFM_MERGE_MAX_PARTS];
    const float *lses[SFM_MERGE_MAX_PARTS];
    const float *sinks;
    uint4 *out;
    float *lse;
    int32_t rows, chunks, parts;      // chunks: 16-byte pieces of a row
    FastDiv heads_div;
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

// (small results are kept: they count where the other parts' values are 0)
__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// N: the number of parts, as far as the loads of a piece go out together
template <typename T, int N>
__global__ void __launch_bounds__(32 * kWarps) sfm_merge_kernel(const MergeArgs a)
{
    grid_follow();
    const int lane = threadIdx.x & 31;
    for (int64_t row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); row < a.rows; row += (int64_t)gridDim.x * kWarps) {
        const int64_t base = row * a.chunks;
        // the lane's first pieces are under way while the weights are worked out; a part without keys is not used
        uint4 v[N][2];
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (n < a.parts && lane + 32 * k < a.chunks) v[n][k] = a.outs[n][base + lane + 32 * k];
        float w[N], m = -INFINITY;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            w[n] = n < a.parts ? a.lses[n][row] : -INFINITY;
            m = w[n] > m || w[n] != w[n] ? w[n] : m;       // a NaN stays
        }
        float total = 0.f, inv = 0.f;
        if (m != -INFINITY) {
#pragma unroll
            for (int n = 0; n < N; ++n) {
                w[n] = w[n] == -INFINITY ? 0.f : exp2_fast((w[n] - m) * kLog2e);
                total += w[n];
            }
            // 1 / (total + e^(sink - m)), also where the sink lies so far above that the power leaves fp32's range
            float e = 1.f, under = total;
            if (a.sinks) {
                const int head = (int)((uint32_t)row - fdiv((uint32_t)row, a.heads_div) * a.heads_div.d);
                const float sink = __ldg(a.sinks + head);
                e = exp2_fast(0.5f * kLog2e * (m - fmaxf(m, sink)));
                under = fmaf(total, e * e, sink >= m ? 1.f : exp2_fast((sink - m) * kLog2e));
            }
            inv = e / under * e;
        }
        uint32_t used = 0;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            if (m != -INFINITY && w[n] != 0.f) used |= 1u << n;
            w[n] *= inv;
        }
        for (int c0 = 0; c0 < a.chunks; c0 += 64) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int c = c0 + 32 * k + lane;
                if (c >= a.chunks) continue;
                float f[8] = {};
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    if (!(used >> n & 1)) continue;
                    float x[8];
                    widen<T>(c0 == 0 ? v[n][k] : a.outs[n][base + c], x);
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[i] = fmaf(w[n], x[i], f[i]);
                }
                a.out[base + c] = narrow<T>(f);
            }
        }
        if (a.lse && lane == 0) a.lse[row] = m == -INFINITY ? m : m + __log2f(total) * kLn2;
    }
}

template <typename T>
cudaError_t launch(const MergeArgs &a, int sms, cudaStream_t st)
{
    // Sixteen CTAs per SM at most, so that a warp takes several rows of a long call.  How many an SM holds at once goes by the
    // registers: of three parts four in fp16 and two in bf16, of eight two and one.
    const int64_t blocks = ((int64_t)a.rows + kWarps - 1) / kWarps, most = (int64_t)sms * 16;
    const dim3 grid((unsigned)(blocks < most ? blocks : most)), block(32 * kWarps);
    switch (a.parts) {
    case 1: return launch_dependent(sfm_merge_kernel<T, 1>, grid, block, 0, st, a);
    case 2: return launch_dependent(sfm_merge_kernel<T, 2>, grid, block, 0, st, a);
    case 3: return launch_dependent(sfm_merge_kernel<T, 3>, grid, block, 0, st, a);
    case 4: return launch_dependent(sfm_merge_kernel<T, 4>, grid, block, 0, st, a);
    default: return launch_dependent(sfm_merge_kernel<T, SFM_MERGE_MAX_PARTS>, grid, block, 0, st, a);
    }
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
    if (!out) return SFM_ERR_INVALID_ARG;
    if ((int64_t)p.tokens * p.heads > INT32_MAX) return SFM_ERR_UNSUPPORTED;
    MergeArgs a = {};
    uintptr_t bits = (uintptr_t)out | (((uintptr_t)sinks | (uintptr_t)lse) & 3u);
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
    a.rows = p.tokens * p.heads;
    a.chunks = p.head_dim / 8;
    a.parts = p.parts;
    a.heads_div = make_fastdiv((uint32_t)p.heads);
    int device = 0, sms = 0;
    if (current_sms(&device, &sms) != cudaSuccess) return SFM_ERR_CUDA;
    const cudaError_t e = p.dtype == SFM_DTYPE_BF16 ? launch<__nv_bfloat16>(a, sms, (cudaStream_t)stream) : launch<__half>(a, sms, (cudaStream_t)stream);
    return e == cudaSuccess ? SFM_OK : SFM_ERR_CUDA;
}
