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
// followed by further passes over all keys.  The sweep that fills the list also
// notes, one bit per key, which keys lie above the digit and which in it, so
// that the selected indices are then written, ascending, from the bits and the
// few keys in the digit alone; of those equal to the k-th key the first
// `take_equal` are taken.
//
// Scores are read once: the keys of a row stay in the shared memory of the
// cluster of CTAs that works on it (one CTA for the many rows of a prompt, up
// to 16 for the long rows of a few requests), each CTA holding a contiguous
// slice; histograms and counts are added up through distributed shared memory,
// and every CTA searches the list of all.  Where rows that no CTA can hold are
// many, each has one CTA that reads it twice and holds the marks alone.
//
// Measured on one GB300: 32 rows of 32768, k 512: 7.5 us; one row of 600001, k
// 2048: 15.8 us; 2048 causal rows of up to 8192, k 1024: 29.9 us (2.0 TB/s);
// 2048 causal rows of up to 16384 in blocks of 64, k 32: 32.2 us (3.9 TB/s);
// 529 causal rows of up to 63406, k 512: 79 us (1.7 TB/s).
// Loading and counting take half to two thirds of the prompt rows, some fifteen block
// barriers with little work between them the rest, and the many small passes'
// instructions (50 per 32 keys) more than memory bound the rows of 8192.  Rows
// kept as floats and counted in equal bins of a sample's range (34.5 us), a list
// of the scores above a sampled value (52) and loading later rows into L2 (35.5)
// were slower.
#include <cooperative_groups.h>

#include <type_traits>

#include "sfm_internal.cuh"

namespace cg = cooperative_groups;

namespace sfm {
namespace {

constexpr int kBins = 4096;                    // of a cluster's histogram
constexpr int kMaxCluster = 16;
constexpr int kMaxSlice = 40448;               // keys of a CTA: 158 KB and 10 KB of bits
constexpr int kMaxStream = 1 << 19;            // scores of a row that is read twice: 128 KB of bits
enum { kRecompute, kCached, kStreamed };       // where a CTA's keys are: nowhere, in shared memory, in the row itself
constexpr uint32_t kForced = 0xffffffffu;
constexpr uint32_t kLeast = 0x00800000u;       // the least key of a score: below it there is none

struct TopkArgs {
    const float *scores;
    const int32_t *lengths;
    int32_t *out;
    int32_t *status;
    int64_t stride;
    int32_t n, k, bs_log2, first, last, cluster;
    int32_t slice_cap;                         // keys the shared memory holds (a multiple of 512)
    int32_t aligned;                           // rows start on 16-byte boundaries
};

template <int BINS>
struct Shared {
    uint32_t hist[BINS];                       // then the list's place, in one CTA
    uint32_t search[256];                      // bins of the list's search
    uint32_t few[32];
    uint32_t warp_above[32], warp_equal[32];
    uint32_t list_n, few_n;
    uint32_t found[3];                         // digit, keys above it, keys in it
    uint32_t threshold, take_equal;
};

// Where key i of a slice is kept: groups of four, in an order that lets the lanes of a warp read four neighbouring
// groups each (16 keys) as well as one after the other without meeting in a bank.
__device__ __forceinline__ int quad_at(int q) { return q ^ ((q >> 2) & 7); }
__device__ __forceinline__ int key_slot(int i) { return quad_at(i >> 2) << 2 | (i & 3); }

// Behind the keys and their bits, in the CTAs of a cluster only.
struct ClusterShared {
    uint32_t total[kBins];                     // the cluster's histogram
    uint32_t list[kBins];
    uint32_t above[kMaxCluster], equal[kMaxCluster];   // selected keys per CTA
    uint32_t list_base[kMaxCluster];           // where this CTA's keys go in each CTA's list
    uint32_t list_n;
};

constexpr int kMaxDynamic = kMaxSlice * 4 + kMaxSlice / 4 + (int)sizeof(ClusterShared);
static_assert(kMaxDynamic + sizeof(Shared<kBins>) <= 232448, "shared memory budget");

// x's key.  NaN becomes -inf, whose key lies below kLeast, and -0 becomes 0.
__device__ __forceinline__ uint32_t key_of(float x)
{
    const uint32_t b = __float_as_uint(fmaxf(x + 0.f, -INFINITY));
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
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

// mark |= bit where key >= from (EQUAL) or key > from: a comparison and a
// predicated or, where the compiler makes three instructions of it (prompt rows:
// 31.3 us without, 30.0 with)
template <bool EQUAL>
__device__ __forceinline__ void mark_if(uint32_t &mark, uint32_t key, uint32_t from, uint32_t bit)
{
    if (EQUAL) asm("{\n\t.reg .pred p;\n\tsetp.ge.u32 p, %1, %2;\n\t@p or.b32 %0, %0, %3;\n\t}" : "+r"(mark) : "r"(key), "r"(from), "r"(bit));
    else asm("{\n\t.reg .pred p;\n\tsetp.gt.u32 p, %1, %2;\n\t@p or.b32 %0, %0, %3;\n\t}" : "+r"(mark) : "r"(key), "r"(from), "r"(bit));
}

// Find the bin that holds the need-th largest of the counted keys: its
// number, the keys above it and the keys in it, to *found.  All threads call
// it.  With fewer than `need` keys in all nothing is found (found[2] = 0).
// Warp w sums the w-th share of the bins from the top, four neighbouring bins
// per lane and step; the warp that holds the key looks closer.
template <int NT, int BINS>
__device__ __forceinline__ void find_bin(const uint32_t *bins, uint32_t need, uint32_t *warp_sums, uint32_t *found)
{
    constexpr int NW = NT / 32, kSteps = BINS / NW / 128;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int top = BINS / 4 - 1 - warp * (BINS / NW / 4) - lane;     // this lane's quad of the first step
    uint32_t sums[kSteps], mine = 0;
#pragma unroll
    for (int q = 0; q < kSteps; ++q) {
        const uint4 w = reinterpret_cast<const uint4 *>(bins)[top - 32 * q];
        sums[q] = w.x + w.y + w.z + w.w;
        mine += sums[q];
    }
    const uint32_t total = __reduce_add_sync(0xffffffffu, mine);
    if (lane == 0) warp_sums[warp] = total;
    if (tid == 0) found[2] = 0;
    __syncthreads();
    uint32_t above = __reduce_add_sync(0xffffffffu, lane < warp ? warp_sums[lane] : 0u);
    if (above < need && need <= above + total) {
#pragma unroll
        for (int q = 0; q < kSteps; ++q) {
            const uint32_t step = __reduce_add_sync(0xffffffffu, sums[q]);
            if (above < need && need <= above + step) {
                uint32_t upto = sums[q];
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t v = __shfl_up_sync(0xffffffffu, upto, o);
                    if (lane >= o) upto += v;
                }
                uint32_t a = above + upto - sums[q];
                if (a < need && need <= above + upto) {
                    const uint4 w = reinterpret_cast<const uint4 *>(bins)[top - 32 * q];
                    const uint32_t each[4] = {w.w, w.z, w.y, w.x};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (a < need && need <= a + each[e]) {
                            found[0] = 4 * (top - 32 * q) + 3 - e;
                            found[1] = a;
                            found[2] = each[e];
                        }
                        a += each[e];
                    }
                }
            }
            above += step;
        }
    }
    __syncthreads();
}

// One warp: the want-th largest of n <= 32 keys.
template <int BINS>
__device__ __forceinline__ void rank_few(Shared<BINS> &sh, const uint32_t *few, int n, uint32_t want)
{
    const int lane = threadIdx.x & 31;
    const uint32_t key = lane < n ? few[lane] : 0u;
    uint32_t above = 0, equal = 0;
#pragma unroll
    for (int o = 0; o < 32; ++o) {
        const uint32_t other = __shfl_sync(0xffffffffu, key, o);
        above += other > key;
        equal += other == key;
    }
    if (lane < n && above < want && want <= above + equal) {         // the lanes of one key alone
        sh.threshold = above + equal == want ? key - 1 : key;
        sh.take_equal = above + equal == want ? 0 : want - above;
    }
}

// The want-th largest of the n listed keys, all of which share the bits above
// `open`: selected are keys > sh.threshold and the first sh.take_equal equal to
// it.  All threads of the CTA call it.  Eight bits at a time; the last 32
// candidates are ranked in one warp.
template <int NT, int BINS>
__device__ __forceinline__ void search_list(Shared<BINS> &sh, const uint32_t *list, uint32_t n, int open, uint32_t prefix,
                                            uint32_t want)
{
    if (n <= 32) {
        if (threadIdx.x < 32) rank_few(sh, list, (int)n, want);
        __syncthreads();
        return;
    }
    const int tid = threadIdx.x, lane = tid & 31;
    while (true) {
        const int b = open < 8 ? open : 8;
        open -= b;
        if (tid < 64) reinterpret_cast<uint4 *>(sh.search)[tid] = make_uint4(0, 0, 0, 0);
        if (tid == 0) sh.few_n = 0;
        __syncthreads();
        for (uint32_t i = tid; i < n; i += NT) {
            const uint32_t key = list[i];
            if ((key >> (open + b)) == prefix) atomicAdd(&sh.search[(key >> open) & ((1u << b) - 1)], 1u);
        }
        __syncthreads();
        if (tid < 32) {                           // lane i: bins 255 - 8 i .. 248 - 8 i
            const uint4 hi = reinterpret_cast<const uint4 *>(sh.search)[63 - 2 * lane];
            const uint4 lo = reinterpret_cast<const uint4 *>(sh.search)[62 - 2 * lane];
            const uint32_t each[8] = {hi.w, hi.z, hi.y, hi.x, lo.w, lo.z, lo.y, lo.x};
            uint32_t mine = 0;
#pragma unroll
            for (int q = 0; q < 8; ++q) mine += each[q];
            uint32_t upto = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t v = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += v;
            }
            uint32_t above = upto - mine;
            if (above < want && want <= upto) {
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    if (above < want && want <= above + each[q]) {
                        sh.found[0] = 255 - 8 * lane - q;
                        sh.found[1] = above;
                        sh.found[2] = each[q];
                    }
                    above += each[q];
                }
            }
        }
        __syncthreads();
        const uint32_t in_bin = sh.found[2];
        want -= sh.found[1];
        prefix = prefix << b | sh.found[0];
        if (in_bin == want || open == 0) {
            if (tid == 0) {
                sh.threshold = in_bin == want ? (prefix << open) - 1 : prefix;
                sh.take_equal = in_bin == want ? 0 : want;
            }
            break;
        }
        if (in_bin <= 32) {
            for (uint32_t i = tid; i < n; i += NT) {
                const uint32_t key = list[i];
                if ((key >> open) == prefix) sh.few[atomicAdd(&sh.few_n, 1u)] = key;
            }
            __syncthreads();
            if (tid < 32) rank_few(sh, sh.few, (int)in_bin, want);
            break;
        }
        __syncthreads();                          // found has been read
    }
    __syncthreads();
}

// Keys of blocks of 4 << GL scores, eight 16-byte loads per lane: 256 >> GL
// whole blocks of a warp, which share GL lanes' bits.  Lanes swap half of what
// they hold while they hold more than one value, so eight values cost eight
// exchanges and not 8 GL.  store(block, value) gets each block once.
template <int GL, bool ALIGNED, typename Store>
__device__ __forceinline__ void pool_chunk(const float *src, int lane, Store store)
{
    constexpr int kSwaps = GL < 3 ? GL : 3;
    float v[8];
    {
        float4 w[8];
#pragma unroll
        for (int s = 0; s < 8; ++s) {
            const float *at = src + 4 * (32 * s + lane);
            w[s] = ALIGNED ? __ldg(reinterpret_cast<const float4 *>(at))
                           : make_float4(__ldg(at), __ldg(at + 1), __ldg(at + 2), __ldg(at + 3));
        }
#pragma unroll
        for (int s = 0; s < 8; ++s) v[s] = fmaxf(fmaxf(w[s].x, w[s].y), fmaxf(w[s].z, w[s].w));
    }
    int step = 0;
#pragma unroll
    for (int k = 0; k < kSwaps; ++k) {
        const int o = 1 << (GL - 1 - k), n = 8 >> (k + 1);
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float send = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
            v[i] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, send, o));
        }
        step += up ? n : 0;
    }
#pragma unroll
    for (int o = (1 << GL) >> (kSwaps + 1); o > 0; o >>= 1) v[0] = fmaxf(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
    constexpr int kRest = GL - kSwaps;            // lanes' bits that hold the same value
    if ((lane & ((1 << kRest) - 1)) == 0) {
#pragma unroll
        for (int i = 0; i < (8 >> kSwaps); ++i) store((step + i) * (32 >> GL) + (lane >> GL), v[i]);
    }
}

// POOLED: blocks of several scores.
// CTAs of at most 256 threads work on many short rows: fewer bins, and registers for five of 256 threads to share an
// SM (2048 rows of up to 8192: 32.4 us with four loads ahead, with eight, which spill, 33.9; four CTAs and eight 33.4).
template <int NT, int MODE, bool POOLED>
__global__ void __launch_bounds__(NT, NT > 512 ? 1 : NT > 256 ? 2 : 1280 / NT) sfm_topk_kernel(const TopkArgs a)
{
    constexpr int NW = NT / 32;
    constexpr bool CACHED = MODE == kCached, STREAMED = MODE == kStreamed, kBits = CACHED || STREAMED;
    constexpr int kTop = NT <= 256 ? 11 : 12, kMine = 1 << kTop;       // bits of the first digit, bins
    __shared__ Shared<kMine> sh;
    extern __shared__ __align__(16) uint32_t keys[];
    uint32_t *bits = keys + a.slice_cap;          // a word per 16 keys: above the digit, and (upper half) in it
    ClusterShared &cs = *reinterpret_cast<ClusterShared *>(bits + a.slice_cap / 16);

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t below = (1u << lane) - 1u;
    const int C = a.cluster;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = C > 1 ? (int)cluster.block_rank() : 0;
    const int64_t r = (gridDim.x - 1 - blockIdx.x) / (unsigned)C;    // a prompt's longest rows first
    const float *row = a.scores + r * a.stride;
    int32_t *out = a.out + r * a.k;

    auto clear = [&](uint32_t *words, int n) {
        for (int i = tid; i < n / 4; i += NT) reinterpret_cast<uint4 *>(words)[i] = make_uint4(0, 0, 0, 0);
    };
    clear(sh.hist, kMine);
    if (C > 1) {
        clear(cs.total, kBins);
        if (tid == 0) cs.list_n = 0;
        cluster.barrier_arrive();             // zeros before anyone adds to them: waited for below
    }
    grid_follow();

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
    __syncthreads();                              // the zeros are there

    auto forced = [&](int j) { return any_forced && (j < a.first || j >= last_from); };
    auto key_at = [&](int i) -> uint32_t {
        if (CACHED) return keys[key_slot(i)];
        return forced(base + i) ? kForced : block_key(row, base + i, l, len);
    };
    // Bins: the keys' top bits, or, once a row's CTA has seen the largest of its first keys, the four octaves below it
    // in steps of 1 << kNear, with all that lies outside in the first and last bin.  Then a bin holds a few keys, and
    // not some percent of the row, and the list is short.  Should the k-th key lie outside, the top bits are counted
    // after all.
    constexpr int kNear = 25 - kTop;
    uint32_t near = 0;                            // the key that the second bin starts at
    int bin_shift = 32 - kTop;
    auto look = [&](uint32_t most) {              // all threads call it
        most = __reduce_max_sync(0xffffffffu, most);
        if (lane == 0) sh.warp_above[warp] = most;
        __syncthreads();
        most = __reduce_max_sync(0xffffffffu, lane < NW ? sh.warp_above[lane] : 0u);
        if (most > kLeast + (kMine << kNear)) {
            near = ((most >> kNear) - (kMine - 3)) << kNear;
            bin_shift = kNear;
        }
    };
    auto count = [&](uint32_t key) {
        atomicAdd(&sh.hist[min((max(key, near) - near) >> bin_shift, (uint32_t)kMine - 1)], 1u);
    };

    // four scores of the row
    auto load4 = [&](int q) {
        const float *at = row + base + 4 * q;
        return a.aligned ? __ldg(reinterpret_cast<const float4 *>(at))
                         : make_float4(__ldg(at), __ldg(at + 1), __ldg(at + 2), __ldg(at + 3));
    };
    auto keys4 = [&](int q, const float4 &v) {
        uint4 w = make_uint4(key_of(v.x), key_of(v.y), key_of(v.z), key_of(v.w));
        if (any_forced) {
            const int j = base + 4 * q;
            if (forced(j)) w.x = kForced;
            if (forced(j + 1)) w.y = kForced;
            if (forced(j + 2)) w.z = kForced;
            if (forced(j + 3)) w.w = kForced;
        }
        return w;
    };

    // ---- keys, and their histogram ---------------------------------------------------
    if (STREAMED) {
        const int quads = cnt >> 2;
        constexpr int kAhead = 4;
        for (int q0 = 0; q0 < quads; q0 += kAhead * NT) {
            float4 v[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int q = q0 + i * NT + tid;
                v[i] = q < quads ? load4(q) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            if (q0 == 0) look(tid < quads ? key_of(fmaxf(fmaxf(v[0].x, v[0].y), fmaxf(v[0].z, v[0].w))) : 0u);
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                if (q0 + i * NT + tid < quads) {
                    const uint4 w = keys4(q0 + i * NT + tid, v[i]);
                    count(w.x);
                    count(w.y);
                    count(w.z);
                    count(w.w);
                }
            }
        }
        const int i = (quads << 2) + tid;
        if (i < cnt) count(key_at(i));
    } else if (CACHED && !POOLED && a.aligned) {
        const float4 *src = reinterpret_cast<const float4 *>(row + base);
        const int quads = cnt >> 2;
        auto quad = [&](int q, const float4 &v) {
            const uint4 w = keys4(q, v);
            reinterpret_cast<uint4 *>(keys)[quad_at(q)] = w;
            count(w.x);
            count(w.y);
            count(w.z);
            count(w.w);
        };
        constexpr int kAhead = 4;
        for (int q0 = 0; q0 < quads; q0 += kAhead * NT) {
            float4 v[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int q = q0 + i * NT + tid;
                v[i] = q < quads ? __ldg(src + q) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            if (C == 1 && q0 == 0) look(tid < quads ? key_of(fmaxf(fmaxf(v[0].x, v[0].y), fmaxf(v[0].z, v[0].w))) : 0u);
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                if (q0 + i * NT + tid < quads) quad(q0 + i * NT + tid, v[i]);
        }
        const int i = (quads << 2) + tid;
        if (i < cnt) {
            const uint32_t key = forced(base + i) ? kForced : key_of(__ldg(row + base + i));
            keys[key_slot(i)] = key;
            count(key);
        }
    } else if (CACHED && !POOLED) {
        for (int i0 = 0; i0 < cnt; i0 += 8 * NT) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int i = i0 + e * NT + tid;
                v[e] = i < cnt ? __ldg(row + base + i) : 0.f;
            }
            if (C == 1 && i0 == 0) look(tid < cnt ? key_of(v[0]) : 0u);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int i = i0 + e * NT + tid;
                if (i < cnt) {
                    const uint32_t key = forced(base + i) ? kForced : key_of(v[e]);
                    keys[key_slot(i)] = key;
                    count(key);
                }
            }
        }
    } else if (CACHED) {
        // a block's largest score is taken before it becomes a key: fmaxf passes over NaN
        auto store = [&](int j, float best) {
            const uint32_t key = forced(base + j) ? kForced : key_of(best);
            keys[key_slot(j)] = key;
            count(key);
        };
        const int gl = l - 2;
        int done = 0;                             // blocks of the chunks that lie inside the row
        if (l >= 2) {
            const int chunk = 256 >> gl;
            const int whole = (int)min((int64_t)cnt, (len >> l) - (int64_t)base) / chunk;
            const float *src = row + ((int64_t)base << l);
            for (int c = warp; c < whole; c += NW) {
                const float *from = src + (int64_t)c * 1024;
                auto put = [&](int b, float best) { store(c * chunk + b, best); };
                auto pool = [&](auto g) {
                    if (a.aligned) pool_chunk<g.value, true>(from, lane, put);
                    else pool_chunk<g.value, false>(from, lane, put);
                };
                switch (gl) {
                case 0: pool(std::integral_constant<int, 0>{}); break;
                case 1: pool(std::integral_constant<int, 1>{}); break;
                case 2: pool(std::integral_constant<int, 2>{}); break;
                case 3: pool(std::integral_constant<int, 3>{}); break;
                case 4: pool(std::integral_constant<int, 4>{}); break;
                default: pool(std::integral_constant<int, 5>{}); break;
                }
            }
            done = max(whole, 0) * chunk;
        }
        const int g = gl < 0 ? 1 : 1 << gl, shift = gl < 0 ? 0 : gl, sub = lane & (g - 1);
        for (int j0 = done + warp * (32 >> shift); j0 < cnt; j0 += NW * (32 >> shift)) {
            const int j = j0 + (lane >> shift);
            const int64_t b0 = (int64_t)(base + j) << l;
            const int64_t end = j < cnt ? min((int64_t)len, b0 + min(1 << l, sub * 4 + 4)) : 0;
            float best = -INFINITY;
            for (int64_t i = b0 + sub * 4; i < end; ++i) best = fmaxf(best, __ldg(row + i));
            for (int o = g >> 1; o > 0; o >>= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, o));
            if (j < cnt && sub == 0) store(j, best);
        }
    } else {
        for (int i = tid; i < cnt; i += NT) count(key_at(i));
    }
    if (C > 1) cluster.barrier_wait();
    __syncthreads();

    // ---- the k-th largest key -------------------------------------------------
    // selected: key > threshold, and the first take_equal keys equal to it
    uint32_t prefix = 0, need = (uint32_t)a.k, threshold = kLeast - 1, take_equal = 0;
    bool listed = false;
    // each warp's part of the slice, in order: 16 neighbouring keys per lane and step
    const int seg = ((cnt + NW - 1) / NW + 511) & ~511;
    const int s0 = min(warp * seg, cnt), s1 = min(s0 + seg, cnt);
    // (streamed: 16 keys that are four quads, 128 keys apart, so that a warp reads the row in order)
    auto read16 = [&](int i0, auto use) {
        if constexpr (STREAMED) {
            float4 v[4];
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int q = (i0 >> 2) + 32 * g + lane;
                v[g] = 4 * q + 3 < s1 ? load4(q) : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            }
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int q = (i0 >> 2) + 32 * g + lane;
                uint4 w = keys4(q, v[g]);
                if (4 * q < s1 && 4 * q + 3 >= s1) {       // the row's last quad
                    w.x = key_at(4 * q);
                    if (4 * q + 1 < s1) w.y = key_at(4 * q + 1);
                    if (4 * q + 2 < s1) w.z = key_at(4 * q + 2);
                }
                use(4 * g, w.x);
                use(4 * g + 1, w.y);
                use(4 * g + 2, w.z);
                use(4 * g + 3, w.w);
            }
        } else {
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const uint4 w = reinterpret_cast<const uint4 *>(keys)[quad_at((i0 >> 2) + 4 * lane + g)];
                use(4 * g, w.x);
                use(4 * g + 1, w.y);
                use(4 * g + 2, w.z);
                use(4 * g + 3, w.w);
            }
        }
    };
    auto valid16 = [&](int i0) -> uint32_t {      // keys of this lane that exist
        if (i0 + 512 <= s1) return 0xffffu;
        auto low = [](int n) -> uint32_t { return n >= 16 ? 0xffffu : n <= 0 ? 0u : (1u << n) - 1; };
        if constexpr (!STREAMED) return low(s1 - (i0 + 16 * lane));
        uint32_t m = 0;
#pragma unroll
        for (int g = 0; g < 4; ++g) m |= low(min(s1 - (i0 + 128 * g + 4 * lane), 4)) << (4 * g);
        return m;
    };
    auto place = [&](int i0, int e) { return STREAMED ? i0 + 128 * (e >> 2) + 4 * lane + (e & 3) : i0 + 16 * lane + e; };
    auto scan = [&](uint32_t v) {                 // sums over the lanes up to this one
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t x = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += x;
        }
        return v;
    };
    // pass -1: the bins near the largest key
#pragma unroll 1
    for (int pass = near ? -1 : 0; pass < 3; ++pass) {
        const int shift = pass < 0 ? kNear : pass == 0 ? 32 - kTop : pass == 1 ? 10 : 0;
        const int bits_n = pass == 0 ? kTop : pass == 1 ? 22 - kTop : 10;
        if (pass > 0 || (pass == 0 && near)) {    // too many keys share the digits so far: count the next ones
            clear(sh.hist, kMine);
            if (C > 1) {
                clear(cs.total, kBins);
                cluster.sync();
            } else {
                __syncthreads();
            }
            for (int i = tid; i < cnt; i += NT) {
                const uint32_t key = key_at(i);
                if (pass == 0 || (key >> (shift + bits_n)) == prefix)
                    atomicAdd(&sh.hist[(key >> shift) & ((1u << bits_n) - 1)], 1u);
            }
            __syncthreads();
        }
        if (C > 1) {
            for (int b = tid; b < kMine; b += NT) {
                const uint32_t s = sh.hist[b];
                if (s)
                    for (int q = 0; q < C; ++q) atomicAdd(cluster.map_shared_rank(&cs.total[b], q), s);
            }
            cluster.sync();
        }
        if (C > 1) find_bin<NT, kBins>(cs.total, need, sh.warp_above, sh.found);
        else find_bin<NT, kMine>(sh.hist, need, sh.warp_above, sh.found);
        const uint32_t in_bin = sh.found[2];
        if (pass < 0) {
            // outside of the fine bins, or too many equal keys for the list
            if (in_bin == 0 || in_bin > (uint32_t)kMine || sh.found[0] == 0 || sh.found[0] == kMine - 1) continue;
            prefix = (near >> kNear) + sh.found[0];
        } else {
            // first digit: fewer scores than k (or the k-th would be none), all are taken
            if (in_bin == 0 || (pass == 0 && sh.found[0] < kLeast >> shift)) break;
            prefix = prefix << bits_n | sh.found[0];
        }
        need -= sh.found[1];
        if (in_bin == need) {                     // the whole bin is taken
            threshold = (prefix << shift) - 1;
            break;
        }
        if (pass == 2) {
            threshold = prefix;
            take_equal = need;
            break;
        }
        if (in_bin > (uint32_t)kMine) continue;

        // ---- the list of the keys in the bin, in the histogram's place.  Every CTA of a cluster gets all CTAs' lists and
        // searches for itself: one that searches and tells the others costs one more barrier ----
        if (tid == 0) sh.list_n = 0;
        if (tid < C && C > 1)                     // where this CTA's keys go
            cs.list_base[tid] = atomicAdd(cluster.map_shared_rank(&cs.list_n, tid), sh.hist[prefix & ((1u << bits_n) - 1)]);
        __syncthreads();
        uint32_t *to = sh.hist;
        if (kBits) {
            listed = true;
            const uint32_t from = prefix << shift, last = from + ((1u << shift) - 1);
            for (int i0 = s0; i0 < s1; i0 += 512) {
                uint32_t above = 0, in = 0;
                read16(i0, [&](int e, uint32_t key) {
                    mark_if<true>(in, key, from, 1u << e);
                    mark_if<false>(above, key, last, 1u << e);
                });
                const uint32_t there = valid16(i0);
                in &= ~above & there;
                above &= there;
                bits[(i0 >> 4) + lane] = above | in << 16;
                if (!__any_sync(0xffffffffu, in)) continue;
                // one addition per warp reserves the places of its keys
                const uint32_t mine = __popc(in), upto = scan(mine);
                uint32_t at = 0;
                if (lane == 31 && upto) at = atomicAdd(&sh.list_n, upto);
                at = __shfl_sync(0xffffffffu, at, 31) + upto - mine;
                for (; in; in &= in - 1, ++at)
                    if (CACHED || at < (uint32_t)kMine) to[at] = key_at(place(i0, __ffs(in) - 1));
            }
        } else {
            for (int i = tid; i < cnt; i += NT) {
                const uint32_t key = key_at(i);
                if ((key >> shift) == prefix) {
                    const uint32_t at = atomicAdd(&sh.list_n, 1u);
                    if (at < (uint32_t)kMine) to[at] = key;
                }
            }
        }
        __syncthreads();
        if (C > 1) {
            const int n = (int)sh.list_n;
            for (int q = warp; q < C; q += NW) {
                uint32_t *there = cluster.map_shared_rank(cs.list, q) + cs.list_base[q];
                for (int i = lane; i < n; i += 32) there[i] = to[i];
            }
            cluster.sync();
        }
        search_list<NT, kMine>(sh, C > 1 ? cs.list : sh.hist, in_bin, shift, prefix, need);
        threshold = sh.threshold;
        take_equal = sh.take_equal;
        break;
    }

    // ---- the selected indices, ascending ------------------------------------------
    // bits: above the threshold, and (upper half) equal to it where ties matter
    uint32_t n_above = 0, n_equal = 0;
    if (kBits) {
        for (int i0 = s0; i0 < s1; i0 += 512) {
            uint32_t m = 0;
            if (listed) {                         // only the keys in the digit are still open
                const uint32_t was = bits[(i0 >> 4) + lane];
                m = was & 0xffffu;
                for (uint32_t in = was >> 16; in; in &= in - 1) {
                    const int e = __ffs(in) - 1;
                    const uint32_t key = key_at(place(i0, e));
                    m |= (uint32_t)(key > threshold) << e | (uint32_t)(take_equal && key == threshold) << (16 + e);
                }
            } else {
                read16(i0, [&](int e, uint32_t key) {
                    m |= (uint32_t)(key > threshold) << e | (uint32_t)(take_equal && key == threshold) << (16 + e);
                });
                m &= valid16(i0) * 0x10001u;
            }
            bits[(i0 >> 4) + lane] = m;
            n_above += __popc(m & 0xffffu);
            n_equal += __popc(m >> 16);
        }
    } else {
        for (int i = s0 + lane; i < s1; i += 32) {
            const uint32_t key = key_at(i);
            n_above += key > threshold;
            n_equal += take_equal && key == threshold;
        }
    }
    n_above = __reduce_add_sync(0xffffffffu, n_above);
    n_equal = __reduce_add_sync(0xffffffffu, n_equal);
    __syncthreads();                              // the last find_bin's warp sums have been read
    if (lane == 0) {
        sh.warp_above[warp] = n_above;
        sh.warp_equal[warp] = n_equal;
    }
    __syncthreads();
    const uint32_t va = lane < NW ? sh.warp_above[lane] : 0, ve = lane < NW ? sh.warp_equal[lane] : 0;
    uint32_t before_above = __reduce_add_sync(0xffffffffu, lane < warp ? va : 0u);
    uint32_t before_equal = __reduce_add_sync(0xffffffffu, lane < warp ? ve : 0u);
    uint32_t total_above = __reduce_add_sync(0xffffffffu, va), total_equal = __reduce_add_sync(0xffffffffu, ve);
    if (C > 1) {
        if (tid < C) {
            *cluster.map_shared_rank(&cs.above[rank], tid) = total_above;
            *cluster.map_shared_rank(&cs.equal[rank], tid) = total_equal;
        }
        cluster.sync();                           // the last remote access of this kernel lies before it
        total_above = total_equal = 0;
        for (int q = 0; q < C; ++q) {
            const uint32_t x = cs.above[q], y = cs.equal[q];
            total_above += x;
            total_equal += y;
            if (q < rank) {
                before_above += x;
                before_equal += y;
            }
        }
    }
    if (STREAMED) {
        auto four = [](uint32_t m) {              // the quads' numbers of marks, a byte each
            return (uint32_t)(__popc(m & 0xfu) | __popc(m & 0xf0u) << 8 | __popc(m & 0xf00u) << 16 | __popc(m & 0xf000u) << 24);
        };
        for (int i0 = s0; i0 < s1; i0 += 512) {
            const uint32_t m = bits[(i0 >> 4) + lane];
            const uint32_t up = four(m), up_to = scan(up), ups = __shfl_sync(0xffffffffu, up_to, 31);
            uint32_t eq = 0, eq_to = 0, eqs = 0;
            if (take_equal) {
                eq = four(m >> 16);
                eq_to = scan(eq);
                eqs = __shfl_sync(0xffffffffu, eq_to, 31);
            }
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                uint32_t at = before_above + ((up_to - up) >> (8 * g) & 0xffu), mine = m >> (4 * g) & 0xfu;
                before_above += ups >> (8 * g) & 0xffu;
                if (take_equal) {
                    uint32_t room = before_equal + ((eq_to - eq) >> (8 * g) & 0xffu);
                    at += min(room, take_equal);
                    before_equal += eqs >> (8 * g) & 0xffu;
                    for (uint32_t e = m >> (16 + 4 * g) & 0xfu; e && room < take_equal; e &= e - 1, ++room) mine |= e & -e;
                }
                for (; mine; mine &= mine - 1, ++at)
                    if (at < (uint32_t)a.k) out[at] = base + place(i0, 4 * g + __ffs(mine) - 1);
            }
        }
    } else if (CACHED) {
        for (int i0 = s0; i0 < s1; i0 += 512) {
            uint32_t m = bits[(i0 >> 4) + lane];
            uint32_t e = m >> 16;
            m &= 0xffffu;
            const uint32_t up = __popc(m), up_to = scan(up);
            uint32_t at = before_above + up_to - up;
            before_above += __shfl_sync(0xffffffffu, up_to, 31);
            if (take_equal) {
                const uint32_t eq = __popc(e), eq_to = scan(eq);
                uint32_t room = before_equal + eq_to - eq;       // equal keys before this lane's
                at += min(room, take_equal);
                before_equal += __shfl_sync(0xffffffffu, eq_to, 31);
                for (; e && room < take_equal; e &= e - 1, ++room) m |= e & -e;
            }
            for (; m; m &= m - 1) out[at++] = base + i0 + 16 * lane + __ffs(m) - 1;
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
                if (at < (uint32_t)a.k) out[at] = base + i;
            }
            before_above += __popc(mu);
            before_equal += __popc(me);
        }
    }
    const int64_t filled = (int64_t)total_above + min(total_equal, take_equal);
    for (int64_t i = filled + rank * NT + tid; i < a.k; i += (int64_t)C * NT) out[i] = -1;
}

template <int NT, int MODE, bool POOLED>
cudaError_t launch(const TopkArgs &a, int device, int64_t rows, size_t smem, cudaStream_t st)
{
    static std::atomic<bool> ready[kMaxDevices];
    auto kernel = sfm_topk_kernel<NT, MODE, POOLED>;
    return prepared_launch(
        ready, device,
        [&] {
            const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxDynamic);
            return e == cudaSuccess ? cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) : e;
        },
        [&] {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3((unsigned)(rows * a.cluster));
            cfg.blockDim = dim3(NT);
            cfg.dynamicSmemBytes = smem;
            cfg.stream = st;
            cudaLaunchAttribute attr[2];
            attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
            attr[0].val.programmaticStreamSerializationAllowed = 1;
            attr[1].id = cudaLaunchAttributeClusterDimension;
            attr[1].val.clusterDim.x = (unsigned)a.cluster;
            attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = a.cluster > 1 ? 2 : 1;
            return cudaLaunchKernelEx(&cfg, kernel, a);
        });
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
    if (current_sms(&dev, &sms) != cudaSuccess) return SFM_ERR_CUDA;

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
    // Rows that no CTA can hold, and enough of them for two thirds of the SMs: one CTA each, which reads its row twice
    // (the second time from L2) and keeps the marks alone, beats a cluster that holds it: 529 rows of up to 63406 79
    // us for 101, 256 of 131072 71 for 104, 152 of 60000 26 for 27, but 70 of 60000 24 for 12.  Rows of 32768, which
    // a CTA holds: 68 for 65.
    const bool pooled = a.bs_log2 > 0;
    const bool streamed = !pooled && (int64_t)p.rows * 3 > (int64_t)sms * 2 && p.n > kMaxSlice && p.n <= kMaxStream;
    // CTAs of a row: as many as it takes to hold its keys, and while a CTA still
    // has some thousand keys twice as many, up to six sevenths of the SMs (the
    // CTAs of a cluster share a GPC, so clusters of eight do not fill them all):
    // 32 rows of 32768 with 4 CTAs a row 9.3 us, with 8 10.3 us, with 2 10.4 us
    int c = 1;
    auto slice = [&](int q) { return ((blocks + q - 1) / q + 127) / 128 * 128; };
    while (!streamed && c < kMaxCluster && (slice(c) > kMaxSlice || ((int64_t)p.rows * c * 14 <= (int64_t)sms * 6 && slice(c) > 4096))) c *= 2;
    if ((int64_t)p.rows * c > INT32_MAX) return SFM_ERR_UNSUPPORTED;
    a.cluster = c;
    const bool cached = slice(c) <= kMaxSlice;
    a.slice_cap = cached && !streamed ? (int32_t)((slice(c) + 511) / 512 * 512) : 0;
    const size_t smem = streamed ? ((size_t)p.n + 511) / 512 * 128
                                 : (size_t)a.slice_cap * 4 + (size_t)a.slice_cap / 4 + (c > 1 ? sizeof(ClusterShared) : 0);
    const cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e;
    // Threads: a short slice has few keys per thread, and many small CTAs hide each other's barriers (2048 x
    // 16384 scores in blocks of 64, 256 keys a row: 35 us with 256 threads, 33 with 128; 2690 x 1055 in blocks of
    // 16: 20.4 and 13.6).  Slices of which an SM holds two at most take 512 (1024 x 16384: 39.1 us with 256, 31.6 with
    // 512; 1024 x 12000, three per SM: 26.7 and 28.8), those of which it holds one 1024 (1024 x 20000, two per SM: 52.2
    // with 1024, 40.3 with 512).
    if (streamed) e = launch<512, kStreamed, false>(a, dev, p.rows, smem, st);
    else if (!cached) e = launch<1024, kRecompute, false>(a, dev, p.rows, smem, st);
    else if (slice(c) > 22528)
        e = pooled ? launch<1024, kCached, true>(a, dev, p.rows, smem, st) : launch<1024, kCached, false>(a, dev, p.rows, smem, st);
    else if (c > 1 || slice(c) > 14336)
        e = pooled ? launch<512, kCached, true>(a, dev, p.rows, smem, st) : launch<512, kCached, false>(a, dev, p.rows, smem, st);
    else if (slice(c) > 2048)
        e = pooled ? launch<256, kCached, true>(a, dev, p.rows, smem, st) : launch<256, kCached, false>(a, dev, p.rows, smem, st);
    else e = pooled ? launch<128, kCached, true>(a, dev, p.rows, smem, st) : launch<128, kCached, false>(a, dev, p.rows, smem, st);
    return e == cudaSuccess ? SFM_OK : SFM_ERR_CUDA;
}
