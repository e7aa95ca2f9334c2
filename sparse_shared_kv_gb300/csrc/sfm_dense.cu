// sfm_dense.cu -- attention of many queries over the same rows
// (sfm_dense_forward): prompts, single tokens over a cache, drafted trees.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "sfm_dense.cuh"

namespace sfm {
namespace {

constexpr int kD = 512;
constexpr int kWarps = 8;
constexpr float kLog2e = 1.4426950408889634f;

template <typename T>
__device__ __forceinline__ void widen(uint4 v, float *f)
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

// One warp per query row and head, one key at a time, with a running maximum
// and sum; lane l holds values [8 l, 8 l + 8) and [256 + 8 l, 256 + 8 l + 8).
template <typename T>
__global__ void __launch_bounds__(32 * kWarps) sfm_dense_rows_kernel(const DenseArgs a)
{
    grid_follow();
    const int lane = threadIdx.x & 31;
    const int64_t rows = (int64_t)a.total_q * a.heads, row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (row >= rows) return;
    const int t = (int)(row / a.heads), h = (int)(row % a.heads);
    int b = 0;
    if (a.cu_q) {
        while (b + 1 < a.batch && __ldg(a.cu_q + b + 1) <= t) ++b;
    } else {
        b = t / a.q_s;
    }
    const DenseSeq s = dense_seq(a, b);
    const int i = t - s.q0;
    uint4 *out = reinterpret_cast<uint4 *>(static_cast<T *>(a.out) + row * kD);
    if (i < 0 || i >= s.q_cap) {
        if (a.zero_rest) {
            out[lane] = out[lane + 32] = make_uint4(0, 0, 0, 0);
            if (a.lse && lane == 0) a.lse[row] = -INFINITY;
        }
        return;
    }
    float q[16], o[16] = {}, m = -INFINITY, l = 0.f;
    widen<T>(reinterpret_cast<const uint4 *>(static_cast<const T *>(a.q) + row * kD)[lane], q);
    widen<T>(reinterpret_cast<const uint4 *>(static_cast<const T *>(a.q) + row * kD)[lane + 32], q + 8);
    if (i < s.q_len) {
        const DenseRow r = dense_row(a, s, i);
        const int first = s.len - s.q_len;
        for (int j = 0; j < s.len; ++j) {
            bool seen = (j >= r.lo && j < r.hi) || j < s.prefix;
            int64_t pos = j;
            if (a.words && j >= first) {
                const int k = j - first;
                pos = __ldg(a.positions + s.q0 + k);
                seen = k < 64 * a.words && (__ldg(a.tree + (int64_t)t * a.words + (k >> 6)) >> (k & 63) & 1);
                if (a.mode == 4 && (pos < (int64_t)r.p - a.win_left || pos > (int64_t)r.p + a.win_right)) seen = false;
            }
            if (!seen) continue;
            int64_t at = s.kv0 + j;
            if (a.layout_kv == SFM_LAYOUT_PAGED) {
                const int id = __ldg(a.table + (int64_t)b * a.cols + j / a.block);
                at = (int64_t)id * a.block + j % a.block;
                if (id < 0 || ((int64_t)id + 1) * a.block > a.kv_rows) {
                    if (lane == 0) dense_status(a, SFM_STATUS_BAD_BLOCK);
                    continue;
                }
            }
            const uint4 *key = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(a.kv) + at * a.kv_row_stride);
            float k[16], x = 0.f;
            widen<T>(__ldg(key + lane), k);
            widen<T>(__ldg(key + lane + 32), k + 8);
#pragma unroll
            for (int d = 0; d < 16; ++d) x = fmaf(q[d], k[d], x);
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
            x *= a.scale;
            if (a.cap > 0.f) x = a.cap * tanhf(x / a.cap);
            if (a.slopes) x -= a.slopes[h] * fabsf((float)(r.p - pos));
            const float top = x > m || x != x ? x : m, old = top == -INFINITY ? 1.f : expf(m - top);
            const float e = top == -INFINITY ? 0.f : expf(x - top);
            l = l * old + e;
#pragma unroll
            for (int d = 0; d < 16; ++d) o[d] = fmaf(e, k[d], o[d] * old);
            m = top;
        }
    }
    const float inv = m == -INFINITY ? 0.f : 1.f / (a.sinks ? l + expf(a.sinks[h] - m) : l);
    uint16_t v[16];
#pragma unroll
    for (int d = 0; d < 16; ++d) {
        const T x = static_cast<T>(o[d] * inv);
        v[d] = *reinterpret_cast<const uint16_t *>(&x);
    }
    out[lane] = *reinterpret_cast<const uint4 *>(v);
    out[lane + 32] = *reinterpret_cast<const uint4 *>(v + 8);
    if (a.lse && lane == 0) a.lse[row] = m == -INFINITY ? m : m + logf(l);
}

int dense_check(const sfm_dense_params *pp)
{
    if (!pp) return SFM_ERR_INVALID_ARG;
    const sfm_dense_params &p = *pp;
    if (p.num_heads < 1 || p.num_heads > 128) return SFM_ERR_INVALID_ARG;
    if (p.head_dim != kD) return SFM_ERR_UNSUPPORTED;
    if (p.dtype != SFM_DTYPE_BF16 && p.dtype != SFM_DTYPE_FP16) return SFM_ERR_INVALID_ARG;
    if (p.layout_q != SFM_LAYOUT_BSND && p.layout_q != SFM_LAYOUT_TND) return SFM_ERR_LAYOUT;
    if (p.layout_kv != SFM_LAYOUT_BSND && p.layout_kv != SFM_LAYOUT_TND && p.layout_kv != SFM_LAYOUT_PAGED)
        return SFM_ERR_LAYOUT;
    if (p.layout_kv != SFM_LAYOUT_PAGED && p.layout_kv != p.layout_q) return SFM_ERR_LAYOUT;
    if (p.batch_size <= 0 || p.max_seqlen_kv <= 0) return SFM_ERR_INVALID_ARG;
    if (p.layout_q == SFM_LAYOUT_BSND ? p.max_seqlen_q < 0 : p.total_q < 0) return SFM_ERR_INVALID_ARG;
    if (p.mask_mode != 0 && p.mask_mode != 3 && p.mask_mode != 4) return SFM_ERR_INVALID_ARG;
    if (p.mask_mode == 4 && (p.win_left < -1 || p.win_right < -1)) return SFM_ERR_INVALID_ARG;
    if (p.layout_kv == SFM_LAYOUT_PAGED && (p.block_size < 16 || p.block_size > 1024 || p.block_size % 16)) return SFM_ERR_LAYOUT;
    if (p.tree_words < 0 || p.tree_words > 16 || p.split_keys < 0 || p.split_keys % 128) return SFM_ERR_INVALID_ARG;
    if (!std::isfinite(p.softmax_scale) || !(p.softcap >= 0.f) || !std::isfinite(p.softcap)) return SFM_ERR_INVALID_ARG;
    if (p.max_seqlen_kv > 1 << 30) return SFM_ERR_UNSUPPORTED;
    const int64_t tokens = p.layout_q == SFM_LAYOUT_TND ? p.total_q : (int64_t)p.batch_size * p.max_seqlen_q;
    if (tokens * p.num_heads > INT32_MAX - 256) return SFM_ERR_UNSUPPORTED;      // rows that a copy's coordinate names
    return SFM_OK;
}

}  // namespace
}  // namespace sfm

using namespace sfm;

extern "C" int sfm_dense_workspace_size(const sfm_dense_params *params, size_t *bytes)
{
    const int rc = dense_check(params);
    if (rc) return rc;
    if (!bytes) return SFM_ERR_INVALID_ARG;
    *bytes = 0;
    return SFM_OK;
}

extern "C" int sfm_dense_forward(const sfm_dense_params *pp, const sfm_dense_tensors *t, void *out, float *lse,
                                 void *workspace, size_t workspace_bytes, int32_t *status, sfm_stream_t stream)
{
    const int rc = dense_check(pp);
    if (rc) return rc;
    if (!t) return SFM_ERR_INVALID_ARG;
    const sfm_dense_params &p = *pp;
    const bool paged = p.layout_kv == SFM_LAYOUT_PAGED, tnd = p.layout_q == SFM_LAYOUT_TND;
    if (t->kv_row_stride < 2 * kD || t->kv_row_stride % 16 || t->kv_rows <= 0) return SFM_ERR_LAYOUT;
    if (t->kv_rows > ((int64_t)1 << 31) - 1024) return SFM_ERR_UNSUPPORTED;
    if (p.layout_kv == SFM_LAYOUT_BSND && t->kv_rows < (int64_t)p.batch_size * p.max_seqlen_kv) return SFM_ERR_LAYOUT;
    if ((tnd && !t->cu_seqlens_q) || (p.layout_kv == SFM_LAYOUT_TND && !t->cu_seqlens_kv)) return SFM_ERR_INVALID_ARG;
    if (paged ? !t->seqused_kv || !t->block_table || t->block_table_stride <= 0 : t->block_table != nullptr)
        return SFM_ERR_INVALID_ARG;
    if (p.tree_words ? !t->tree_mask || !t->positions || t->prefix_lens || t->key_begin || t->key_end
                     : t->tree_mask || t->positions)
        return SFM_ERR_INVALID_ARG;
    const int32_t tokens = tnd ? p.total_q : p.batch_size * p.max_seqlen_q;
    if (tokens == 0) return SFM_OK;
    if (!t->q || !t->kv || !out) return SFM_ERR_INVALID_ARG;
    if (((uintptr_t)t->q | (uintptr_t)t->kv | (uintptr_t)out) & 15u) return SFM_ERR_LAYOUT;
    if (((uintptr_t)lse | (uintptr_t)t->sinks | (uintptr_t)t->bias_slopes) & 3u || (uintptr_t)t->tree_mask & 7u) return SFM_ERR_LAYOUT;

    DenseArgs a = {};
    a.q = t->q;
    a.kv = t->kv;
    a.out = out;
    a.lse = lse;
    a.status = status;
    a.table = t->block_table;
    a.cu_q = tnd ? t->cu_seqlens_q : nullptr;
    a.cu_kv = p.layout_kv == SFM_LAYOUT_TND ? t->cu_seqlens_kv : nullptr;
    a.used_q = t->seqused_q;
    a.used_kv = t->seqused_kv;
    a.prefix = t->prefix_lens;
    a.begin = t->key_begin;
    a.end = t->key_end;
    a.positions = t->positions;
    a.sinks = t->sinks;
    a.slopes = t->bias_slopes;
    a.tree = reinterpret_cast<const uint64_t *>(t->tree_mask);
    a.kv_row_stride = t->kv_row_stride;
    a.kv_rows = t->kv_rows;
    a.heads = p.num_heads;
    a.batch = p.batch_size;
    a.q_s = p.max_seqlen_q;
    a.total_q = tokens;
    a.max_kv = p.max_seqlen_kv;
    a.mode = p.mask_mode;
    const int32_t far = 1 << 30;
    a.win_left = p.win_left < 0 || p.win_left > far ? far : p.win_left;
    a.win_right = p.win_right < 0 || p.win_right > far ? far : p.win_right;
    a.layout_kv = p.layout_kv;
    a.block = p.block_size;
    a.cols = t->block_table_stride;
    a.words = p.tree_words;
    a.zero_rest = p.zero_rest != 0;
    a.scale = p.softmax_scale;
    a.cap = p.softcap;
    a.block_div = make_fastdiv(paged ? (uint32_t)p.block_size : 1u);
    a.heads_div = make_fastdiv((uint32_t)p.num_heads);
    const int64_t rows = (int64_t)tokens * p.num_heads;
    const dim3 grid((unsigned)((rows + kWarps - 1) / kWarps));
    const cudaError_t e = p.dtype == SFM_DTYPE_BF16
                              ? launch_dependent(sfm_dense_rows_kernel<__nv_bfloat16>, grid, dim3(32 * kWarps), 0, (cudaStream_t)stream, a)
                              : launch_dependent(sfm_dense_rows_kernel<__half>, grid, dim3(32 * kWarps), 0, (cudaStream_t)stream, a);
    return e == cudaSuccess ? SFM_OK : SFM_ERR_CUDA;
}
