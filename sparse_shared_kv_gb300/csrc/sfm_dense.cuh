// sfm_dense.cuh -- what the kernels of sfm_dense_forward() agree on: their
// arguments, the lengths of a sequence and the keys that a query sees.
#pragma once

#include "sfm_internal.cuh"

namespace sfm {

struct DenseArgs {
    const void *q, *kv;
    void *out;
    float *lse;
    int32_t *status;
    const int32_t *table, *cu_q, *cu_kv, *used_q, *used_kv, *prefix, *begin, *end, *positions;
    const float *sinks, *slopes;
    const uint64_t *tree;
    int64_t kv_row_stride, kv_rows;
    int32_t heads, batch, q_s, total_q, max_kv, mode, win_left, win_right, layout_kv, block, cols, words, zero_rest;
    float scale, cap;
    FastDiv block_div, heads_div;
};

__device__ __forceinline__ void dense_status(const DenseArgs &a, int bits)
{
    if (a.status) atomicOr(a.status, bits);
}

// A sequence: its rows of q (the first q_len of q_cap count) and its keys.
struct DenseSeq {
    int32_t b, q0, q_cap, q_len, len, prefix;
    int64_t kv0;              // row of its first key (not paged)
};

// All loads go out before the first of them is looked at; lengths outside of what the buffers hold are cut.  (One copy in a
// kernel: the code that plans runs a few times, and to fetch it is most of what it costs.)
__device__ __noinline__ DenseSeq dense_seq(const DenseArgs &a, int b)
{
    const int32_t q0 = a.cu_q ? __ldg(a.cu_q + b) : b * a.q_s, q1 = a.cu_q ? __ldg(a.cu_q + b + 1) : q0 + a.q_s;
    const int32_t k0 = a.cu_kv ? __ldg(a.cu_kv + b) : 0, k1 = a.cu_kv ? __ldg(a.cu_kv + b + 1) : a.max_kv;
    const int32_t used_q = a.used_q ? __ldg(a.used_q + b) : 0, used_kv = a.used_kv ? __ldg(a.used_kv + b) : 0;
    const int32_t prefix = a.prefix ? __ldg(a.prefix + b) : 0;
    int bad = 0;
    auto cut = [&](int v, int lo, int hi) {
        const int c = min(max(v, lo), hi);
        bad |= c ^ v;
        return c;
    };
    DenseSeq s;
    s.b = b;
    s.q0 = cut(q0, 0, a.total_q);
    s.q_cap = cut(q1, s.q0, a.total_q) - s.q0;
    s.q_len = a.used_q ? cut(used_q, 0, s.q_cap) : s.q_cap;
    // paged and (b, S) caches: k0 = 0 and k1 = max_kv, which the host has cut to what a sequence's blocks hold
    const int rows = (int)min(a.kv_rows, (int64_t)INT32_MAX);
    const int first = cut(k0, 0, a.cu_kv ? rows : 0);
    int most = cut(k1, first, a.cu_kv ? rows : a.max_kv) - first;
    if (most > a.max_kv) {
        most = a.max_kv;
        bad = 1;
    }
    s.kv0 = a.layout_kv == SFM_LAYOUT_BSND ? (int64_t)b * a.max_kv : first;
    s.len = a.used_kv ? cut(used_kv, 0, most) : most;
    s.prefix = min(max(prefix, 0), s.len);
    if (__builtin_expect(bad, 0)) dense_status(a, SFM_STATUS_BAD_LENGTH);
    return s;
}

// bits [lo, hi) of a word whose bit 0 stands for key j0
__host__ __device__ __forceinline__ uint32_t bits_between(int lo, int hi, int j0)
{
    const int l = min(max(lo - j0, 0), 32), h = min(max(hi - j0, 0), 32);
    const uint32_t up = h >= 32 ? 0xffffffffu : (1u << h) - 1u, down = l >= 32 ? 0xffffffffu : (1u << l) - 1u;
    return h > l ? up & ~down : 0u;
}

// The drafted ones of keys [j0, j0 + 32), where the drafted keys begin at `first`.  Key j0 + c's own entry of positions and bit
// of tree_mask is j0 + c - first, of which the sequence has len - first: what these bits allow stays inside.  (Looked-up
// numbers cut to the sequence one by one made trees of 61 tokens 4 % slower: 1140 -> 1190 us.)
__host__ __device__ __forceinline__ uint32_t drafted_keys(int first, int len, int j0) { return bits_between(max(first, 0), len, j0); }

// What query i of a sequence sees: keys [0, prefix) and [lo, hi); with a tree
// [lo, hi) among the keys before `first`, and those of its bits from there on.
struct DenseRow {
    int32_t p, lo, hi;
};

__device__ __forceinline__ DenseRow dense_row(const DenseArgs &a, const DenseSeq &s, int i)
{
    DenseRow r;
    const int32_t first = s.len - s.q_len;
    r.p = a.words ? __ldg(a.positions + s.q0 + i) : first + i;
    int64_t lo = 0, hi = a.words ? max(first, 0) : s.len;
    if (a.mode == 3 && !a.words) hi = min(hi, (int64_t)r.p + 1);
    if (a.mode == 4) {
        lo = max(lo, (int64_t)r.p - a.win_left);
        hi = min(hi, (int64_t)r.p + a.win_right + 1);
    }
    if (a.begin) lo = max(lo, (int64_t)__ldg(a.begin + s.q0 + i));
    if (a.end) hi = min(hi, (int64_t)__ldg(a.end + s.q0 + i));
    if (lo >= hi) lo = hi = 0;
    r.lo = (int32_t)lo;
    r.hi = (int32_t)hi;
    return r;
}

}  // namespace sfm
