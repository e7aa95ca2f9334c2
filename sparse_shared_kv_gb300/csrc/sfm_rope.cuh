// sfm_rope.cuh -- angles of rotary positions, and the 16-bit value types.
//
// A pair's angle is position * f radians.  Only its fraction of a turn
// matters, so f / (2 pi) is held as a 64-bit binary fraction of a turn and
// multiplied by the position modulo 2^64.  The fraction is the product of f's 53
// bits with those of 1 / (2 pi) that they meet (the reduction of Payne and Hanek;
// 64-bit floating point is slow here, and a product with the rounded 1 / (2 pi)
// would be off by 2^-56 f of a turn per position): it is at most 1.001 * 2^-64 of
// a turn low for |f| < 2^53, and the angle of any 32-bit position, negative ones
// included, off by less than 2^-32 of a turn.  Its top 32 bits (cut off, another
// 2^-32 at most) then give it in half turns, rounded to fp32, which sincospif takes
// without a further reduction.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace sfm {
namespace rope {

__device__ __forceinline__ unsigned long long turn_step(double inv_freq)
{
    // 2^128 / (2 pi)
    constexpr unsigned __int128 kTurns = (unsigned __int128)0x28be60db9391054aull << 64 | 0x7f09d5f47d4d3770ull;
    const unsigned long long bits = (unsigned long long)__double_as_longlong(inv_freq);
    const int shift = 1075 - (int)(bits >> 52 & 0x7ff);
    const unsigned long long m = (bits & ((1ull << 52) - 1)) | 1ull << 52;
    if (shift < 0 || shift > 127) return 0;       // 2^53 and above; below 2^-75: no turn within 32 bits of position
    const unsigned long long step = (unsigned long long)((m * (kTurns >> shift)) >> 64);
    return inv_freq < 0.0 ? 0ull - step : step;
}

// (cos, sin) of position * inv_freq, times the amplitude
__device__ __forceinline__ float2 cos_sin(int32_t position, unsigned long long step, float amplitude, bool inverse)
{
    const unsigned long long turns = (unsigned long long)(long long)position * step;
    float s, c;
    sincospif((float)(int32_t)(turns >> 32) * 0x1p-31f, &s, &c);
    return make_float2(amplitude * c, inverse ? -amplitude * s : amplitude * s);
}

__device__ __forceinline__ float2 rotate(float a, float b, float2 cs)
{
    return make_float2(fmaf(a, cs.x, -b * cs.y), fmaf(b, cs.x, a * cs.y));
}

// the two 16-bit value types: pairs to and from fp32 (rounded to nearest even)
template <typename T> struct Pair;
template <> struct Pair<__nv_bfloat16> {
    static __device__ __forceinline__ float2 load(uint32_t w)
    {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
    static __device__ __forceinline__ uint32_t store(float a, float b)
    {
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
    static __device__ __forceinline__ float one(__nv_bfloat16 v) { return __bfloat162float(v); }
    static __device__ __forceinline__ __nv_bfloat16 round(float v) { return __float2bfloat16_rn(v); }
};
template <> struct Pair<__half> {
    static __device__ __forceinline__ float2 load(uint32_t w)
    {
        return __half22float2(*reinterpret_cast<const __half2 *>(&w));
    }
    static __device__ __forceinline__ uint32_t store(float a, float b)
    {
        const __half2 v = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
    static __device__ __forceinline__ float one(__half v) { return __half2float(v); }
    static __device__ __forceinline__ __half round(float v) { return __float2half_rn(v); }
};

template <typename T>
__device__ __forceinline__ void unpack8(const uint4 &w, float (&v)[8])
{
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 p = Pair<T>::load(u[i]);
        v[2 * i] = p.x;
        v[2 * i + 1] = p.y;
    }
}

template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&v)[8])
{
    return make_uint4(Pair<T>::store(v[0], v[1]), Pair<T>::store(v[2], v[3]), Pair<T>::store(v[4], v[5]),
                      Pair<T>::store(v[6], v[7]));
}

}  // namespace rope
}  // namespace sfm
