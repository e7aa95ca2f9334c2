// sfm_topk.cu -- the k best positions or blocks of every row of scores
// (sfm_topk_select).
//
// Every score becomes a 32-bit key whose unsigned order is the scores' order
// (no score: 0; always selected: all ones), so a block's value is the largest
// key, and the k-th largest key is found exactly by a radix selection.  The
// histogram of the top 11 bits (sign, exponent, two bits of the significand)
// is taken while the keys are made; the digit of the k-th key leaves a few
// percent of them, which are copied to a short list and searched to the last
// bit there.  Digits that leave too many for the list (equal scores) are
// followed by further passes over all keys.  One ordered sweep then writes the
// selected indices ascending, the first `take_equal` of those equal to the
// k-th key among them.
//
// Scores are read once: the keys of a row stay in the shared memory of the
// cluster of CTAs that works on it (one CTA for the many rows of a prompt, up
// to 16 for the long rows of a few requests), each CTA holding a contiguous
// slice; histograms and counts are added up through distributed shared memory,
// and the cluster's first CTA searches the list.
#include <cooperative_groups.h>

#include "sfm_internal.cuh"

namespace cg = cooperative_groups;

namespace sfm {
namespace {

constexpr int kBins = 2048;
constexpr int kCopies = 2;                     // histogram copies: fewer lanes of a warp meet in one word
constexpr int kList = kBins * kCopies;         // the list takes the histogram's place
constexpr int kMaxCluster = 16;
constexpr int kMaxSlice = 50176;               // keys of a CTA: 196 KB
constexpr uint32_t kForced = 0xffffffffu;

struct TopkArgs {
    const float *scores;
    const int32_t *lengths;
    int32_t *out;
    int32_t *status;
    int64_t stride;
    int32_t n, k, bs_log2, first, last, cluster;
    int32_t slice_cap;                         // keys the shared memory holds
    int32_t aligned;                           // rows start on 16-byte boundaries
};

struct Shared {
    uint32_t hist[kBins * kCopies];
    uint32_t total[kBins];                     // the cluster's histogram
    uint32_t above[kMaxCluster], equal[kMaxCluster];   // selected keys per CTA
    uint32_t warp_above[32], warp_equal[32];
    uint32_t list_n, list_base;
    uint32_t found[3];                         // digit, keys above it, keys in it
    uint32_t threshold, take_equal;
};

__device__ __forceinline__ uint32_t key_of(float x)
{
    const uint32_t b = __float_as_uint(x + 0.f);          // -0 becomes 0
    const uint32_t key = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
    return x > -INFINITY ? key : 0u;                      // NaN and -inf: no score
}

// the key of block j of a row: scores [j << l, min((j + 1) << l, len))
__device__ __forceinline__ uint32_t block_key(const float *row, int j, int l, int len)
{
    const int64_t a = (int64_t)j << l;
    const int64_t b = min((int64_t)len, a + (1 << l));
    uint32_t key = 0;
    for (int64_t i = a; i < b; ++i) key = max(key, key_of(__ldg(row + i)));
    return key;
}

// Find the bin that holds the need-th largest of the counted keys: its
// number, the keys above it and the keys in it, to *found.  All threads call
// it; BINS / NT bins each, from the top.  With fewer than `need` keys in all
// nothing is found (found[2] = 0).
template <int NT, int BINS>
__device__ __forceinline__ void find_bin(const uint32_t *bins, uint32_t need, uint32_t *warp_sums, uint32_t *found)
{
    constexpr int kEach = BINS > NT ? BINS / NT : 1;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool mine_any = tid * kEach < BINS;
    uint32_t mine = 0;
    if (mine_any) {
#pragma unroll
        for (int q = 0; q < kEach; ++q) mine += bins[BINS - 1 - tid * kEach - q];
    }
    uint32_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
    }
    if (lane == 31) warp_sums[warp] = upto;
    if (tid == 0) found[2] = 0;
    __syncthreads();
    uint32_t before = lane < warp ? warp_sums[lane] : 0;   // at most 32 warps
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
    upto += before;
    uint32_t above = upto - mine;
    if (above < need && need <= upto) {
#pragma unroll
        for (int q = 0; q < kEach; ++q) {
            const uint32_t b = bins[BINS - 1 - tid * kEach - q];
            if (above < need && above + b >= need) {
                found[0] = BINS - 1 - tid * kEach - q;
                found[1] = above;
                found[2] = b;
            }
            above += b;
        }
    }
    __syncthreads();
}

template <int NT, bool CACHED>
__global__ void __launch_bounds__(NT) sfm_topk_kernel(const TopkArgs a)
{
    constexpr int NW = NT / 32;
    __shared__ Shared sh;
    extern __shared__ __align__(16) uint32_t keys[];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t below = (1u << lane) - 1u;
    const int C = a.cluster;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = C > 1 ? (int)cluster.block_rank() : 0;
    const int64_t r = blockIdx.x / (unsigned)C;
    const float *row = a.scores + r * a.stride;
    int32_t *out = a.out + r * a.k;

    int len = a.n;
    if (a.lengths) {
        len = __ldg(a.lengths + r);
        if (len < 0 || len > a.n) {
            if (a.status && tid == 0 && rank == 0) atomicOr(a.status, SFM_STATUS_BAD_LENGTH);
            len = len < 0 ? 0 : a.n;
        }
    }
    const int l = a.bs_log2;
    const int have = (int)(((int64_t)len + (1 << l) - 1) >> l);
    const int per = (int)((((int64_t)have + C - 1) / C + 127) / 128 * 128);
    const int base = (int)min((int64_t)rank * per, (int64_t)have);
    const int cnt = min(per, have - base);
    const int last_from = have - a.last;
    const bool any_forced = a.first | a.last;

    for (int i = tid; i < kBins * kCopies; i += NT) sh.hist[i] = 0;
    if (C > 1) {
        for (int i = tid; i < kBins; i += NT) sh.total[i] = 0;
        if (tid == 0) sh.list_n = 0;
        cluster.barrier_arrive();             // zeros before anyone adds to them: waited for below
    }
    __syncthreads();

    auto forced = [&](int j) { return any_forced && (j < a.first || j >= last_from); };
    auto key_at = [&](int i) -> uint32_t {
        if (CACHED) return keys[i];
        return forced(base + i) ? kForced : block_key(row, base + i, l, len);
    };
    auto count = [&](uint32_t key) {
        if (key) atomicAdd(&sh.hist[(key >> 21) * kCopies + (lane & (kCopies - 1))], 1u);
    };

    // ---- keys, and the histogram of their top 11 bits ------------------------------
    if (CACHED && l == 0 && a.aligned) {
        const float4 *src = reinterpret_cast<const float4 *>(row + base);
        const int quads = cnt >> 2;
        auto quad = [&](int q, const float4 &v) {
            uint4 w = make_uint4(key_of(v.x), key_of(v.y), key_of(v.z), key_of(v.w));
            if (any_forced) {
                const int j = base + 4 * q;
                if (forced(j)) w.x = kForced;
                if (forced(j + 1)) w.y = kForced;
                if (forced(j + 2)) w.z = kForced;
                if (forced(j + 3)) w.w = kForced;
            }
            reinterpret_cast<uint4 *>(keys)[q] = w;
            count(w.x);
            count(w.y);
            count(w.z);
            count(w.w);
        };
        int q = tid;
        for (; q + 3 * NT < quads; q += 4 * NT) {
            float4 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = __ldg(src + q + i * NT);
#pragma unroll
            for (int i = 0; i < 4; ++i) quad(q + i * NT, v[i]);
        }
        for (; q < quads; q += NT) quad(q, __ldg(src + q));
        const int i = (quads << 2) + tid;
        if (i < cnt) {
            const uint32_t key = forced(base + i) ? kForced : key_of(__ldg(row + base + i));
            keys[i] = key;
            count(key);
        }
    } else if (CACHED && l == 0) {
        auto one = [&](int i, float v) {
            const uint32_t key = forced(base + i) ? kForced : key_of(v);
            keys[i] = key;
            count(key);
        };
        int i = tid;
        for (; i + 7 * NT < cnt; i += 8 * NT) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = __ldg(row + base + i + e * NT);
#pragma unroll
            for (int e = 0; e < 8; ++e) one(i + e * NT, v[e]);
        }
        for (; i < cnt; i += NT) one(i, __ldg(row + base + i));
    } else if (CACHED) {
        // g lanes per block, each up to four scores of it; four steps' loads in flight
        const int gl = l < 2 ? 0 : l - 2, g = 1 << gl, sub = lane & (g - 1);
        const int per_warp = 32 >> gl;
        for (int j0 = warp * per_warp; j0 < cnt; j0 += 4 * NW * per_warp) {
            uint32_t key[4];
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int j = j0 + s * NW * per_warp + (lane >> gl);
                const int64_t e = ((int64_t)(base + j) << l) + sub * 4;
                key[s] = 0;
                if (j >= cnt) continue;
                if (l >= 2 && a.aligned && e + 4 <= len) {
                    const float4 v = __ldg(reinterpret_cast<const float4 *>(row + e));
                    key[s] = max(max(key_of(v.x), key_of(v.y)), max(key_of(v.z), key_of(v.w)));
                } else {
                    const int64_t end = min((int64_t)len, ((int64_t)(base + j) << l) + min(1 << l, sub * 4 + 4));
                    for (int64_t i = e; i < end; ++i) key[s] = max(key[s], key_of(__ldg(row + i)));
                }
            }
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int j = j0 + s * NW * per_warp + (lane >> gl);
                for (int o = g >> 1; o > 0; o >>= 1) key[s] = max(key[s], __shfl_xor_sync(0xffffffffu, key[s], o));
                if (j < cnt && sub == 0) {
                    if (forced(base + j)) key[s] = kForced;
                    keys[j] = key[s];
                    count(key[s]);
                }
            }
        }
    } else {
        for (int i = tid; i < cnt; i += NT) count(key_at(i));
    }
    if (C > 1) cluster.barrier_wait();
    __syncthreads();

    // ---- the k-th largest key -------------------------------------------------
    // selected: key > threshold, and the first take_equal keys equal to it
    uint32_t prefix = 0, need = (uint32_t)a.k, threshold = 0, take_equal = 0;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        if (pass > 0) {                           // too many keys share the digits so far: count the next ones
            for (int i = tid; i < kBins * kCopies; i += NT) sh.hist[i] = 0;
            if (C > 1) {
                for (int i = tid; i < kBins; i += NT) sh.total[i] = 0;
                cluster.sync();
            } else {
                __syncthreads();
            }
            const int bits = pass == 1 ? 11 : 10;
            for (int i = tid; i < cnt; i += NT) {
                const uint32_t key = key_at(i);
                if (key != 0 && (key >> (shift + bits)) == prefix)
                    atomicAdd(&sh.hist[((key >> shift) & ((1u << bits) - 1)) * kCopies + (lane & (kCopies - 1))], 1u);
            }
            __syncthreads();
        }
        for (int b = tid; b < kBins; b += NT) {
            const uint2 h = reinterpret_cast<const uint2 *>(sh.hist)[b];
            const uint32_t s = h.x + h.y;
            if (C == 1) {
                sh.total[b] = s;
            } else if (s) {
                for (int q = 0; q < C; ++q) atomicAdd(cluster.map_shared_rank(&sh.total[b], q), s);
            }
        }
        if (C > 1) cluster.sync(); else __syncthreads();
        find_bin<NT, kBins>(sh.total, need, sh.warp_above, sh.found);
        const uint32_t in_bin = sh.found[2];
        if (in_bin == 0) break;                   // first pass: fewer scores than k, all are taken
        need -= sh.found[1];
        prefix = pass == 0 ? sh.found[0] : prefix << (pass == 1 ? 11 : 10) | sh.found[0];
        if (in_bin == need) {                     // the whole bin is taken
            threshold = (prefix << shift) - 1;
            break;
        }
        if (pass == 2) {
            threshold = prefix;
            take_equal = need;
            break;
        }
        if (in_bin > (uint32_t)kList) continue;

        // ---- the list of the keys in the bin, in the cluster's first CTA ----
        uint32_t *list = sh.hist;
        if (C == 1) {
            if (tid == 0) sh.list_n = 0;
            __syncthreads();                      // (also: the histogram has been read)
        }
        // a CTA of a cluster first learns where its keys go: one remote addition, not one per warp
        uint32_t *to = list, *n = &sh.list_n;
        if (C > 1) {
            if (tid == 0) {
                const uint2 h = reinterpret_cast<const uint2 *>(sh.hist)[prefix & (kBins - 1)];
                sh.list_base = atomicAdd(cluster.map_shared_rank(&sh.list_n, 0), h.x + h.y);
                sh.warp_equal[0] = 0;
            }
            cluster.sync();                       // every CTA has read its histogram: the first one's gives way to the list
            to = cluster.map_shared_rank(list, 0) + sh.list_base;
            n = &sh.warp_equal[0];
        }
        if (CACHED) {
            const int quads = (cnt + 3) >> 2;     // keys behind the slice are cleared to no key
            if (tid < 4 * quads - cnt) keys[cnt + tid] = 0;
            __syncthreads();
            for (int q = tid; q - lane < quads; q += NT) {
                uint4 w = make_uint4(0, 0, 0, 0);
                if (q < quads) w = reinterpret_cast<const uint4 *>(keys)[q];
                const uint32_t k4[4] = {w.x, w.y, w.z, w.w};
                uint32_t m[4], before = 0, all = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    m[e] = __ballot_sync(0xffffffffu, (k4[e] >> shift) == prefix);
                    before += __popc(m[e] & below);
                    all += __popc(m[e]);
                }
                if (all == 0) continue;
                uint32_t at = 0;
                if (lane == 0) at = atomicAdd(n, all);
                at = __shfl_sync(0xffffffffu, at, 0) + before;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (m[e] >> lane & 1u) to[at++] = k4[e];
            }
        } else {
            for (int i = tid; i < cnt; i += NT) {
                const uint32_t key = key_at(i);
                if ((key >> shift) == prefix) to[atomicAdd(n, 1u)] = key;
            }
        }
        if (C > 1) cluster.sync(); else __syncthreads();
        if (rank == 0) {
            uint32_t *bins = sh.total;
            uint32_t p = prefix, want = need, t = 0, te = 0;
            int at = shift;                       // bits still open
#pragma unroll 1
            while (true) {
                const int b = at < 7 ? at : 7;
                at -= b;
                for (int i = tid; i < 128; i += NT) bins[i] = 0;
                __syncthreads();
                for (uint32_t i = tid; i < in_bin; i += NT) {
                    const uint32_t key = list[i];
                    if ((key >> (at + b)) == p) atomicAdd(&bins[(key >> at) & ((1u << b) - 1)], 1u);
                }
                __syncthreads();
                find_bin<NT, 128>(bins, want, sh.warp_above, sh.found);
                want -= sh.found[1];
                p = p << b | sh.found[0];
                if (sh.found[2] == want) {
                    t = (p << at) - 1;
                    break;
                }
                if (at == 0) {
                    t = p;
                    te = want;
                    break;
                }
                __syncthreads();
            }
            if (tid < C) {
                *(C > 1 ? cluster.map_shared_rank(&sh.threshold, tid) : &sh.threshold) = t;
                *(C > 1 ? cluster.map_shared_rank(&sh.take_equal, tid) : &sh.take_equal) = te;
            }
        }
        if (C > 1) cluster.sync(); else __syncthreads();
        threshold = sh.threshold;
        take_equal = sh.take_equal;
        break;
    }

    // ---- the selected indices, ascending ------------------------------------------
    const int seg = ((cnt + NW - 1) / NW + 127) & ~127;
    const int s0 = min(warp * seg, cnt), s1 = min(s0 + seg, cnt);
    uint32_t n_above = 0, n_equal = 0;
    if (CACHED && !take_equal) {
        for (int i = s0 + 4 * lane; i < s1; i += 128) {
            const uint4 w = *reinterpret_cast<const uint4 *>(keys + i);
            n_above += (w.x > threshold) + (i + 1 < s1 && w.y > threshold) + (i + 2 < s1 && w.z > threshold) +
                       (i + 3 < s1 && w.w > threshold);
        }
    } else {
        for (int i = s0 + lane; i < s1; i += 32) {
            const uint32_t key = key_at(i);
            n_above += key > threshold;
            n_equal += take_equal && key == threshold;
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        n_above += __shfl_xor_sync(0xffffffffu, n_above, o);
        n_equal += __shfl_xor_sync(0xffffffffu, n_equal, o);
    }
    __syncthreads();                              // the last search has read its warp sums
    if (lane == 0) {
        sh.warp_above[warp] = n_above;
        sh.warp_equal[warp] = n_equal;
    }
    __syncthreads();
    uint32_t va = lane < NW ? sh.warp_above[lane] : 0, ve = lane < NW ? sh.warp_equal[lane] : 0;
    uint32_t before_above = lane < warp ? va : 0, before_equal = lane < warp ? ve : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        va += __shfl_xor_sync(0xffffffffu, va, o);
        ve += __shfl_xor_sync(0xffffffffu, ve, o);
        before_above += __shfl_xor_sync(0xffffffffu, before_above, o);
        before_equal += __shfl_xor_sync(0xffffffffu, before_equal, o);
    }
    uint32_t total_above = va, total_equal = ve;
    if (C > 1) {
        if (tid < C) {
            *cluster.map_shared_rank(&sh.above[rank], tid) = va;
            *cluster.map_shared_rank(&sh.equal[rank], tid) = ve;
        }
        cluster.sync();                           // the last remote access of this kernel lies before it
        total_above = total_equal = 0;
        for (int q = 0; q < C; ++q) {
            const uint32_t x = sh.above[q], y = sh.equal[q];
            total_above += x;
            total_equal += y;
            if (q < rank) {
                before_above += x;
                before_equal += y;
            }
        }
    }
    if (CACHED && !take_equal) {
        for (int i0 = s0; i0 < s1; i0 += 128) {
            const int i = i0 + 4 * lane;
            uint4 w = make_uint4(0, 0, 0, 0);
            if (i < s1) w = *reinterpret_cast<const uint4 *>(keys + i);
            const bool up[4] = {w.x > threshold, i + 1 < s1 && w.y > threshold, i + 2 < s1 && w.z > threshold,
                                i + 3 < s1 && w.w > threshold};
            uint32_t at = before_above, all = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t m = __ballot_sync(0xffffffffu, up[e]);
                at += __popc(m & below);
                all += __popc(m);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (up[e]) out[at++] = base + i + e;
            before_above += all;
        }
    } else {
        for (int i0 = s0; i0 < s1; i0 += 32) {
            const int i = i0 + lane;
            const uint32_t key = i < s1 ? key_at(i) : 0;
            const bool up = key > threshold, eq = take_equal && i < s1 && key == threshold;
            const uint32_t mu = __ballot_sync(0xffffffffu, up), me = __ballot_sync(0xffffffffu, eq);
            const uint32_t ea = before_equal + __popc(me & below);
            if (up || (eq && ea < take_equal)) {
                const uint32_t at = before_above + __popc(mu & below) + min(ea, take_equal);
                out[at] = base + i;
            }
            before_above += __popc(mu);
            before_equal += __popc(me);
        }
    }
    const int64_t filled = (int64_t)total_above + min(total_equal, take_equal);
    for (int64_t i = filled + rank * NT + tid; i < a.k; i += (int64_t)C * NT) out[i] = -1;
}

template <int NT, bool CACHED>
cudaError_t launch(const TopkArgs &a, int64_t rows, size_t smem, cudaStream_t st)
{
    auto kernel = sfm_topk_kernel<NT, CACHED>;
    cudaError_t e = cudaSuccess;
    if (smem > 16384) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess && a.cluster > 8) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * a.cluster));
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)a.cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace
}  // namespace sfm

using namespace sfm;

extern "C" int sfm_topk_select(const sfm_topk_params *pp, const float *scores, const int32_t *lengths, int32_t *indices,
                               int32_t *status, sfm_stream_t stream)
{
    if (!pp) return SFM_ERR_INVALID_ARG;
    const sfm_topk_params &p = *pp;
    if (p.rows < 0 || p.n < 1 || p.k < 1) return SFM_ERR_INVALID_ARG;
    if (p.block_size < 1 || p.block_size > 128 || (p.block_size & (p.block_size - 1))) return SFM_ERR_INVALID_ARG;
    if (p.first_blocks < 0 || p.last_blocks < 0 || (int64_t)p.first_blocks + p.last_blocks > p.k)
        return SFM_ERR_INVALID_ARG;
    if (p.score_stride < p.n) return SFM_ERR_LAYOUT;
    if (p.rows == 0) return SFM_OK;
    if (!scores || !indices) return SFM_ERR_INVALID_ARG;
    if (((uintptr_t)scores | (uintptr_t)lengths | (uintptr_t)indices) & 3u) return SFM_ERR_LAYOUT;

    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return SFM_ERR_CUDA;

    TopkArgs a = {};
    a.scores = scores;
    a.lengths = lengths;
    a.out = indices;
    a.status = status;
    a.stride = p.score_stride;
    a.n = p.n;
    a.k = p.k;
    while ((1 << a.bs_log2) < p.block_size) ++a.bs_log2;
    a.first = p.first_blocks;
    a.last = p.last_blocks;
    a.aligned = ((uintptr_t)scores & 15u) == 0 && p.score_stride % 4 == 0;
    const int64_t blocks = ((int64_t)p.n + p.block_size - 1) >> a.bs_log2;
    // CTAs of a row: as many as it takes to hold its keys, and to fill the
    // SMs while a CTA still has some thousand keys
    int c = 1;
    auto slice = [&](int q) { return ((blocks + q - 1) / q + 127) / 128 * 128; };
    while (c < kMaxCluster && (slice(c) > kMaxSlice || ((int64_t)p.rows * c < sms && slice(c) > 4096))) c *= 2;
    if ((int64_t)p.rows * c > INT32_MAX) return SFM_ERR_UNSUPPORTED;
    a.cluster = c;
    const bool cached = slice(c) <= kMaxSlice;
    a.slice_cap = cached ? (int32_t)slice(c) : 0;
    const size_t smem = (size_t)a.slice_cap * 4;
    const cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e;
    if (!cached) e = launch<1024, false>(a, p.rows, 0, st);
    else if (slice(c) > 16384) e = launch<1024, true>(a, p.rows, smem, st);
    else if (slice(c) > 2048) e = launch<512, true>(a, p.rows, smem, st);
    else e = launch<256, true>(a, p.rows, smem, st);
    return e == cudaSuccess ? SFM_OK : SFM_ERR_CUDA;
}
