// sfm_topk.cu -- the k best positions or blocks of every row of scores
// (sfm_topk_select).
//
// Every score becomes a 32-bit key whose unsigned order is the scores' order
// (no score: 0; always selected: all ones), so a block's value is the largest
// key and the k-th largest key is found exactly by a radix selection: the
// histogram of the top 8 bits tells the digit of the k-th key and how many
// keys lie above, the next 8 bits are counted among the keys that share the
// digits so far, and so on; it ends early when a digit's keys are all taken.
// One ordered sweep then writes the selected indices ascending, the first
// `need` of those equal to the k-th key among them.
//
// Scores are read once: the keys of a row stay in the shared memory of the
// cluster of CTAs that works on it (one CTA for the many rows of a prompt, up
// to 16 for the long rows of a few requests), each CTA holding a contiguous
// slice; histograms and counts are added up through distributed shared memory.
#include <cooperative_groups.h>

#include "sfm_internal.cuh"

namespace cg = cooperative_groups;

namespace sfm {
namespace {

constexpr int kBins = 256;
constexpr int kPasses = 4;
constexpr int kCopies = 8;                     // histogram copies: lanes of a warp rarely meet in one word
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
    uint32_t total[kPasses][kBins];            // the cluster's histogram of each pass
    uint32_t above[kMaxCluster], equal[kMaxCluster];   // selected keys per CTA
    uint32_t warp_above[32], warp_equal[32];
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

template <int NT, bool CACHED>
__global__ void __launch_bounds__(NT) sfm_topk_kernel(const TopkArgs a)
{
    constexpr int NW = NT / 32;
    __shared__ Shared sh;
    extern __shared__ uint32_t keys[];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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

    for (int i = tid; i < kPasses * kBins; i += NT) (&sh.total[0][0])[i] = 0;
    if (C > 1) cluster.sync(); else __syncthreads();      // the sums are zero before anyone adds to them

    auto forced = [&](int j) { return j < a.first || j >= last_from; };
    if (CACHED) {
        if (l == 0) {
            if (a.aligned) {
                const int quads = cnt >> 2;
                for (int q = tid; q < quads; q += NT) {
                    const float4 v = __ldg(reinterpret_cast<const float4 *>(row + base) + q);
                    const int j = base + 4 * q;
                    uint4 w = make_uint4(key_of(v.x), key_of(v.y), key_of(v.z), key_of(v.w));
                    if (forced(j)) w.x = kForced;
                    if (forced(j + 1)) w.y = kForced;
                    if (forced(j + 2)) w.z = kForced;
                    if (forced(j + 3)) w.w = kForced;
                    reinterpret_cast<uint4 *>(keys)[q] = w;
                }
                const int i = (quads << 2) + tid;
                if (i < cnt) keys[i] = forced(base + i) ? kForced : key_of(__ldg(row + base + i));
            } else {
#pragma unroll 4
                for (int i = tid; i < cnt; i += NT) keys[i] = forced(base + i) ? kForced : key_of(__ldg(row + base + i));
            }
        } else {
            // g lanes per block, each up to four scores of it per step
            const int gl = l < 2 ? 0 : l - 2, g = 1 << gl, sub = lane & (g - 1);
            const int per_warp = 32 >> gl;
            for (int j0 = warp * per_warp; j0 < cnt; j0 += NW * per_warp) {
                const int j = j0 + (lane >> gl);
                const int64_t e = ((int64_t)(base + j) << l) + sub * 4;
                uint32_t key = 0;
                if (j < cnt) {
                    if (l >= 2 && a.aligned && e + 4 <= len) {
                        const float4 v = __ldg(reinterpret_cast<const float4 *>(row + e));
                        key = max(max(key_of(v.x), key_of(v.y)), max(key_of(v.z), key_of(v.w)));
                    } else {
                        const int64_t end = min((int64_t)len, ((int64_t)(base + j) << l) + min(1 << l, sub * 4 + 4));
                        for (int64_t i = e; i < end; ++i) key = max(key, key_of(__ldg(row + i)));
                    }
                }
                for (int o = g >> 1; o > 0; o >>= 1) key = max(key, __shfl_xor_sync(0xffffffffu, key, o));
                if (j < cnt && sub == 0) keys[j] = forced(base + j) ? kForced : key;
            }
        }
        __syncthreads();
    }
    auto key_at = [&](int i) -> uint32_t {
        if (CACHED) return keys[i];
        return forced(base + i) ? kForced : block_key(row, base + i, l, len);
    };

    // ---- the k-th largest key -------------------------------------------------
    uint32_t prefix = 0, need = (uint32_t)a.k;
    uint32_t threshold = 0, take_equal = 0;       // selected: key > threshold, and the first take_equal equal ones
    for (int pass = 0; pass < kPasses; ++pass) {
        const int shift = 24 - 8 * pass;
        for (int i = tid; i < kBins * kCopies; i += NT) sh.hist[i] = 0;
        __syncthreads();
        for (int i = tid; i < cnt; i += NT) {
            const uint32_t key = key_at(i);
            const bool in = key != 0 && (pass == 0 || (key >> (shift + 8)) == prefix);
            if (in) atomicAdd(&sh.hist[((key >> shift) & 0xffu) * kCopies + (lane & (kCopies - 1))], 1u);
        }
        __syncthreads();
        for (int b = tid; b < kBins; b += NT) {
            uint32_t s = 0;
#pragma unroll
            for (int c = 0; c < kCopies; ++c) s += sh.hist[b * kCopies + c];
            if (C == 1) {
                sh.total[pass][b] = s;
            } else if (s) {
                for (int q = 0; q < C; ++q) atomicAdd(cluster.map_shared_rank(&sh.total[pass][b], q), s);
            }
        }
        if (C > 1) cluster.sync(); else __syncthreads();

        // every warp scans the 256 bins from the top: lane i holds bins 255 - 8 i .. 248 - 8 i
        uint32_t bin[8], mine = 0;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            bin[q] = sh.total[pass][255 - 8 * lane - q];
            mine += bin[q];
        }
        uint32_t upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
        }
        const uint32_t all = __shfl_sync(0xffffffffu, upto, 31);
        if (all <= need) {                        // only in the first pass: fewer scores than k
            threshold = 0;
            take_equal = 0;
            break;
        }
        const uint32_t before = upto - mine;
        const bool here = before < need && need <= upto;
        uint32_t digit = 0, above = before, in_bin = 0;
        if (here) {
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                if (in_bin == 0) {
                    if (above + bin[q] >= need) {
                        digit = 255 - 8 * lane - q;
                        in_bin = bin[q];
                    } else {
                        above += bin[q];
                    }
                }
            }
        }
        const int src = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
        digit = __shfl_sync(0xffffffffu, digit, src);
        above = __shfl_sync(0xffffffffu, above, src);
        in_bin = __shfl_sync(0xffffffffu, in_bin, src);
        need -= above;
        prefix = prefix << 8 | digit;
        if (pass == kPasses - 1) {
            threshold = prefix;
            take_equal = need;
        } else if (in_bin == need) {              // the whole bin is taken
            threshold = (prefix << shift) - 1;
            take_equal = 0;
            break;
        }
    }

    // ---- the selected indices, ascending ------------------------------------------
    const int seg = ((cnt + NW - 1) / NW + 31) & ~31;
    const int s0 = min(warp * seg, cnt), s1 = min(s0 + seg, cnt);
    uint32_t n_above = 0, n_equal = 0;
    for (int i = s0 + lane; i < s1; i += 32) {
        const uint32_t key = key_at(i);
        n_above += key > threshold;
        n_equal += take_equal && key == threshold;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        n_above += __shfl_xor_sync(0xffffffffu, n_above, o);
        n_equal += __shfl_xor_sync(0xffffffffu, n_equal, o);
    }
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
    const uint32_t below = (1u << lane) - 1u;
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
    const int64_t filled = (int64_t)total_above + min(total_equal, take_equal);
    for (int64_t i = filled + rank * NT + tid; i < a.k; i += (int64_t)C * NT) out[i] = -1;
}

template <int NT, bool CACHED>
cudaError_t launch(const TopkArgs &a, int64_t rows, size_t smem, cudaStream_t st)
{
    auto kernel = sfm_topk_kernel<NT, CACHED>;
    cudaError_t e = cudaSuccess;
    if (smem > 32768) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
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
    else if (slice(c) > 8192) e = launch<1024, true>(a, p.rows, smem, st);
    else e = launch<256, true>(a, p.rows, smem, st);
    return e == cudaSuccess ? SFM_OK : SFM_ERR_CUDA;
}
