// sfm_index.cu -- index scores (sfm_index_scores):
//     scores[t][j] = sum_h w[t][h] max(0, s[j] q[t][h] . k[j])
// over paged or contiguous index keys of 128 values (bf16, fp16 or E4M3).
//
// The products are a matrix product per sequence, keys x (queries x heads),
// followed by a clipped weighted sum over the heads.  A tile is 128 keys (the
// rows of the accumulator, one per TMEM lane) by the heads of up to 256 / HP
// queries (its columns, HP = the heads rounded up to 16, 32, 64 or 128): with
// keys on the lanes, the sum over the heads stays inside a thread, a key that
// must not count spoils nothing but its own lane, and scores of neighbouring
// keys are stored side by side.
//
// One persistent CTA per SM walks work units; a unit is a run of key tiles for
// one group of queries of one sequence, and the columns behind the group's last
// visible key, which only have to be set to -inf (16 tiles of them count as
// one).  With up to 1024 groups each CTA takes an equal share of all groups'
// work, counted from the lengths on the device when it starts: a decode batch
// whose sequences differ by a factor of two would keep the CTA with the most
// work busy for 1.6 times the mean otherwise.  More groups are dealt out in
// chunks.
//   warp 16       loads: the unit's queries (two buffers) and its key tiles
//                 (a ring of stages) by TMA into 128-byte-swizzled operands,
//                 one box per run of keys that lies inside a page;
//   warps 17, 19  tcgen05.mma, M = 128, N = queries x HP, K = 128 -> TMEM, in
//                 turns, so that one tile's waits and commits run beside the
//                 other's products (issuing blocks while the pipe is busy);
//   warp 18       brings the units' weights (two buffers), tells the sums which
//                 keys exist and brings their scales (cp.async), so that no sum
//                 waits for global memory;
//   warps 0-15    four warpgroups that drain the accumulator: a warpgroup
//                 takes 64 columns of a tile, a thread a key's 64 products,
//                 32 at a time: a clip each and a multiply-add per two of
//                 them, by weights that the warp reads as one from shared
//                 memory (two units' buffers).  Units of few queries are
//                 narrower than 256 columns: then TMEM holds more tiles and
//                 the warpgroups take different ones.
//
// Measured on one GB300: 32 sequences of up to 32768 E4M3 keys, one query each:
// 25 us, 4.3 TB/s, bound by reading the keys but for some 5 us of starting;
// 2048 queries of 64 heads over 8192 bf16 keys: 163 us, 1.47 PFLOP/s (75 % of
// what a library product reaches), bound by the clipped sums beside the matrix
// products (133 us without them), for some tenths of a second; back to back for
// longer the power cap lowers the clock from 2070 to 1920 MHz and it takes 174 us.
// Over as many E4M3 keys 149; 17 sequences of 974 queries and keys, in units of 4
// queries and 4 tiles: 131 us (a seventh more with the weights fetched by the
// sums); four short sequences: 5.7 us, latency.  Taken out because slower on the
// 2048 queries: weights in registers with 192 columns and twelve warps (174-180
// us), a register split (488), the next 32 columns loaded during the sums (190),
// 64 columns at once (176).
//
// Every wait is bounded as in the attention kernel (sfm_tc.cuh).
#include <cuda.h>
#include <math.h>

#include <type_traits>

#include "sfm_internal.cuh"
#include "sfm_tc.cuh"

namespace sfm {
namespace {

using namespace tc;

constexpr int kTile = 128;                     // keys per tile
constexpr int kDim = 128;                      // values per key
constexpr int kEpiWarps = 16;
constexpr int kThreads = (kEpiWarps + 4) * 32;   // 96 registers each
constexpr int kMaxStages = 8;
constexpr int kMaxAcc = 8;                     // accumulator tiles in TMEM
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kSmemLimit = 232448;
constexpr uint32_t kMiscBytes = 512 + 2048 + 1024;   // barriers, flags and masks, two units' weights, the HP 128 exchange
constexpr uint32_t kScaleBytes = kMaxAcc * kTile * 4;

struct IndexArgs {
    const float *weights, *k_scales;
    float *scores;
    int32_t *visible, *status;
    const int32_t *table, *cu_q, *cu_k, *used_q, *used_k, *residual;
    int64_t stride, k_rows;
    int32_t heads, batch, max_q, total_q, max_k, ratio, causal, layout_q, layout_kv, block, table_stride;
    int32_t groups_per_seq, groups, chunk, units;   // chunk: work of a unit (0: equal shares); units in all, then
    int32_t all_tiles;                         // tiles of max_k keys
    int32_t run, boxes_log2;                   // keys per TMA box, boxes per tile
    int32_t parts_log2;                        // 64-column parts of a tile: 1, 2 or 4
    int32_t stages;
    FastDiv block_div, ratio_div, groups_div, seq_div;
    uint32_t idesc;                            // instruction descriptor without N
    int32_t fp8;
};

constexpr int kShareGroups = 1024;             // groups up to which CTAs take equal shares
constexpr int kFillTiles = 16;                 // tiles of -inf that count as one tile of products

struct Unit {
    // the group
    int32_t b, t0, nq, rows;                   // sequence, first token, live queries, query rows to write
    int32_t len, seen, work;                   // keys, tiles with visible keys, work in all
    int64_t p0;                                // visible(i) = floor((p0 + i) / ratio) for query i of the group
    int64_t k_base;                            // first key row (contiguous layouts)
    // the unit
    int32_t first_tile, tiles;                 // its tiles
    int32_t fill0, fill1;                      // and its columns without a product
    bool begins;                               // it holds the group's first work
};

__device__ __forceinline__ int32_t clamp_to(int64_t v, int64_t lo, int64_t hi, bool *bad)
{
    if (v < lo || v > hi) {
        *bad = true;
        v = v < lo ? lo : hi;
    }
    return (int32_t)v;
}

__device__ __forceinline__ int32_t visible_of(const IndexArgs &a, const Unit &u, int i)
{
    if (i >= u.nq) return 0;
    if (!a.causal) return u.len;
    const int64_t p = u.p0 + i;                // tokens up to and including the query's own
    if (p <= 0) return 0;
    const int64_t v = p <= 0xffffffffll ? (int64_t)fdiv((uint32_t)p, a.ratio_div) : p / a.ratio;
    return (int32_t)(v < u.len ? v : u.len);
}

// Group g, without a unit of it.
__device__ __forceinline__ Unit group_of(const IndexArgs &a, int g, int queries, bool *bad)
{
    Unit u = {};
    u.b = (int)fdiv((uint32_t)g, a.seq_div);
    const int i0 = (g - u.b * a.groups_per_seq) * queries;
    int q_cap, t_base;
    if (a.layout_q == SFM_LAYOUT_BSND) {
        t_base = u.b * a.max_q;
        q_cap = a.max_q;
    } else {
        t_base = clamp_to(__ldg(a.cu_q + u.b), 0, a.total_q, bad);
        const int end = clamp_to(__ldg(a.cu_q + u.b + 1), t_base, a.total_q, bad);
        q_cap = clamp_to(end - t_base, 0, a.max_q, bad);
    }
    const int q_len = a.used_q ? clamp_to(__ldg(a.used_q + u.b), 0, q_cap, bad) : q_cap;
    u.t0 = t_base + i0;
    u.rows = min(max(q_cap - i0, 0), queries);
    u.nq = min(max(q_len - i0, 0), queries);

    int cap = a.max_k;
    u.k_base = 0;
    if (a.layout_kv == SFM_LAYOUT_BSND) {
        u.k_base = (int64_t)u.b * a.max_k;
    } else if (a.layout_kv == SFM_LAYOUT_TND) {
        const int64_t k0 = __ldg(a.cu_k + u.b), k1 = __ldg(a.cu_k + u.b + 1);
        u.k_base = k0 < 0 ? 0 : k0;
        if (k0 < 0) *bad = true;
        cap = clamp_to(k1 - u.k_base, 0, a.max_k, bad);
    }
    u.len = a.used_k ? clamp_to(__ldg(a.used_k + u.b), 0, cap, bad) : cap;
    const int64_t rest = a.residual ? (int64_t)__ldg(a.residual + u.b) : 0;
    u.p0 = (int64_t)u.len * a.ratio + rest - q_len + i0 + 1;
    const int most = u.nq > 0 ? visible_of(a, u, u.nq - 1) : 0;
    u.seen = (most + kTile - 1) / kTile;
    u.work = u.rows ? u.seen + (a.all_tiles - u.seen + kFillTiles - 1) / kFillTiles : 0;
    return u;
}

// Work [lo, hi) of the group: its tiles first, then the rest of its columns.
__device__ __forceinline__ void cut(const IndexArgs &a, Unit &u, int lo, int hi)
{
    u.begins = lo == 0;
    u.first_tile = lo;
    u.tiles = max(min(hi, u.seen) - lo, 0);
    u.fill0 = u.fill1 = 0;
    if (hi > u.seen) {
        const int64_t from = u.seen + (int64_t)(max(lo, u.seen) - u.seen) * kFillTiles;
        const int64_t to = u.seen + (int64_t)(hi - u.seen) * kFillTiles;
        u.fill0 = (int32_t)min(from * kTile, (int64_t)a.max_k);
        u.fill1 = (int32_t)min(to * kTile, (int64_t)a.max_k);
    }
}

// A CTA's share of all groups' work: [from, from + n) counted from the start of group g.
struct Share {
    int32_t g, from;
    int64_t n;
};

// One warp: every lane sums the work of a run of groups (at most 32), the warp
// finds the group that the CTA's share starts in.
__device__ __forceinline__ Share share_of(const IndexArgs &a, int queries, int lane, bool *bad)
{
    const int run = (a.groups + 31) / 32, g0 = lane * run, g1 = min(g0 + run, a.groups);
    int64_t mine = 0;
    for (int g = g0; g < g1; ++g) mine += group_of(a, g, queries, bad).work;
    int64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
    }
    const int64_t all = __shfl_sync(0xffffffffu, upto, 31), per = (all + gridDim.x - 1) / gridDim.x;
    const int64_t start = per * blockIdx.x;
    Share s = {0, 0, min(per, all - start)};
    if (s.n <= 0) return s;
    const uint32_t holds = __ballot_sync(0xffffffffu, upto - mine <= start && start < upto);
    const int src = __ffs(holds) - 1;
    int64_t rest = start - (upto - mine);
    int g = g0;
    if (lane == src && run > 1) {
        for (; g < g1; ++g) {
            const int w = group_of(a, g, queries, bad).work;
            if (rest < w) break;
            rest -= w;
        }
    }
    s.g = __shfl_sync(0xffffffffu, g, src);
    s.from = __shfl_sync(0xffffffffu, (int32_t)rest, src);
    return s;
}

// The units of a CTA.  For a whole warp (WARP) each lane works one of the next
// 32 groups out, and the warp takes them from there one after the other
// (working a group out is a long chain of dependent steps).
template <bool WARP>
struct Units {
    Unit ahead;
    int32_t k = 0, g, from;                    // groups taken so far; equal shares: the next group, and where to start in it
    int64_t left;                              // equal shares: work left

    __device__ __forceinline__ explicit Units(const Share &s) : g(s.g), from(s.from), left(s.n) {}

    __device__ __forceinline__ bool next(const IndexArgs &a, int queries, bool *bad, Unit &u)
    {
        const int lane = threadIdx.x & 31;
        while (true) {
            int lo, hi;
            if (a.chunk) {
                const int64_t unit = blockIdx.x + (int64_t)k * gridDim.x;
                if (unit >= a.units) return false;
                const int c = (int)fdiv((uint32_t)unit, a.groups_div);
                lo = c * a.chunk;
                hi = lo + a.chunk;
                const int64_t mine = unit + (WARP ? (int64_t)lane * gridDim.x : 0);
                if ((!WARP || (k & 31) == 0) && mine < a.units)
                    ahead = group_of(a, (int)(mine - (int64_t)fdiv((uint32_t)mine, a.groups_div) * a.groups), queries, bad);
            } else {
                if (left <= 0 || g >= a.groups) return false;
                lo = from;
                const int mine = g + (WARP ? lane : 0);
                if ((!WARP || (k & 31) == 0) && mine < a.groups) ahead = group_of(a, mine, queries, bad);
            }
            const int src = k & 31;
            auto take = [&](auto v) { return WARP ? __shfl_sync(0xffffffffu, v, src) : v; };
            u.b = take(ahead.b);
            u.t0 = take(ahead.t0);
            u.nq = take(ahead.nq);
            u.rows = take(ahead.rows);
            u.len = take(ahead.len);
            u.seen = take(ahead.seen);
            u.work = take(ahead.work);
            u.p0 = take(ahead.p0);
            u.k_base = take(ahead.k_base);
            ++k;
            if (!a.chunk) {
                hi = (int)min((int64_t)u.work, lo + left);
                left -= hi - lo;
                from = 0;
                ++g;
            }
            hi = min(hi, u.work);
            if (lo >= hi) continue;               // nothing of the group falls to this unit
            cut(a, u, lo, hi);
            return true;
        }
    }
};

// Cache rows of the boxes of a batch of tiles, one box per lane: tile lane >> boxes_log2 of the batch whose first key
// is j0, box lane & (boxes - 1) of it.  -1 where the box's first key does not exist or is not in the cache.
__device__ __forceinline__ int32_t rows_of(const IndexArgs &a, const Unit &u, int j0, int lane)
{
    const int64_t j = j0 + (int64_t)lane * a.run;
    if (j >= u.len) return -1;
    int64_t row = u.k_base + j;
    if (a.layout_kv == SFM_LAYOUT_PAGED) {
        const int page = (int)fdiv((uint32_t)j, a.block_div);
        const int32_t id = page < a.table_stride ? __ldg(a.table + (int64_t)u.b * a.table_stride + page) : -1;
        row = id < 0 ? -1 : (int64_t)id * a.block + (j - (int64_t)page * a.block);
    }
    return row < a.k_rows ? (int32_t)row : -1;
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
        ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
}

__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ void umma_f8(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n"
        ::"r"(d), "l"(ad), "l"(bd), "r"(idesc), "r"(accumulate) : "memory");
}

// Bounded wait of a whole warp, every lane polling: cheaper than one lane that
// tells the others when the phase is usually complete already.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int *abort)
{
    bool ok = mbar_try_wait(bar, parity);
    if (!__all_sync(0xffffffffu, ok)) {
        if (!ok) ok = mbar_wait(bar, parity, abort);
        ok = __all_sync(0xffffffffu, ok);
    }
    return ok;
}

__device__ __forceinline__ float clip(uint32_t x)          // max(0, x), NaN kept
{
    float r;
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(__uint_as_float(x)));
    return r;
}

// The columns of an E4M3 tile whose products are clipped as x + |x|, by half
// their weight: exact, on the multiply-add pipe and not beside the others on the
// narrower one of max().  E4M3 has no infinity, whose negative would
// become NaN.  (2048 queries of 64 heads over 8192 keys: 155.7 us without, with
// one column of four 151.2, two 151.9, three 153.7, all 155.9.)
__host__ __device__ constexpr bool doubled(int column) { return column % 4 == 3; }

__device__ __forceinline__ float clip_twice(uint32_t x)
{
    return __uint_as_float(x) + fabsf(__uint_as_float(x));
}

// two fp32 multiply-adds in one instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 z, x, y, z;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

// HP: columns per query; FULL: as many heads.  Without, a tile is drained only
// after its sums are known to need no second look (2048 queries of 48 heads over
// 8192 keys: 178 us, leaving columns out in every sum 206; of 64 heads 163).
// FP8: E4M3 queries and keys.
template <int HP, bool FULL, bool FP8>
__global__ void __launch_bounds__(kThreads, 1)
sfm_index_kernel(const IndexArgs a, const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map)
{
    constexpr int kQueries = 256 / HP;         // queries of a full tile
    constexpr int kSums = HP <= 64 ? 64 / HP : 1;   // queries whose heads a 64-column part holds
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int parts = 1 << a.parts_log2;
    const int queries = min(kQueries, parts * 64 / HP);
    const uint32_t elem = FP8 ? 1 : 2;
    const uint32_t q_rows = parts * 64;                       // rows of a Q buffer
    const uint32_t q_bytes = q_rows * kDim * elem, k_bytes = kTile * kDim * elem;

    const uint32_t base = smem_u32(smem_raw);
    uint8_t *gbase = smem_raw;
    const uint32_t q_smem = base, k_smem = base + 2 * q_bytes, misc = k_smem + a.stages * k_bytes;
    const uint32_t bars = misc;
    auto q_full = [&](int i) { return bars + 8u * i; };
    auto q_empty = [&](int i) { return bars + 16u + 8u * i; };
    // One barrier per stage and turn of the products' two warps: a barrier's phases are waited for by one thread, in
    // order (2 x stages of them; with one per stage and an odd number of stages, a thread could ask for a phase while
    // the one before, the other thread's, was not complete, and take the answer of the phase before that)
    auto k_full = [&](int i) { return bars + 32u + 8u * i; };
    auto k_empty = [&](int i) { return bars + 160u + 8u * i; };
    auto acc_full = [&](int i) { return bars + 224u + 8u * i; };   // the product, and the keys' mask and scales
    auto acc_empty = [&](int i) { return bars + 288u + 8u * i; };
    auto half_full = [&](int w) { return bars + 352u + 8u * w; };  // HP 128: a part's sums are in shared memory
    auto w_full = [&](int i) { return bars + 384u + 8u * i; };     // a unit's weights are there
    const uint32_t teardown = bars + 400u;                         // two
    uint8_t *gmisc = gbase + (misc - base);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(gmisc + 416);
    uint32_t *tmem_ptr = reinterpret_cast<uint32_t *>(gmisc + 420);
    volatile uint32_t *key_mask = reinterpret_cast<volatile uint32_t *>(gmisc + 424);     // [kMaxAcc] a bit per four keys
    Share *share = reinterpret_cast<Share *>(gmisc + 456);
    static_assert(sizeof(Share) <= 16, "room before the barriers behind it");
    auto w_empty = [&](int i) { return bars + 472u + 8u * i; };    // the sums have read a unit's weights
    float *weights = reinterpret_cast<float *>(gmisc + 512);                            // [2][256]: by column
    float *half_sum = weights + 512;                                                    // HP 128 only: [2 pairs][128]
    float *key_scales = reinterpret_cast<float *>(gmisc + kMiscBytes - (HP == 128 ? 0 : 1024));   // [kMaxAcc][kTile]

    const int accs = kMaxAcc >> a.parts_log2;                 // accumulator tiles of parts * 64 columns
    if (tid == 0) {
        *abort_flag = 0;
        for (int i = 0; i < 2; ++i) mbar_init(q_full(i), 1), mbar_init(q_empty(i), 2);
        for (int i = 0; i < 2 * a.stages; ++i) mbar_init(k_full(i), 1);
        for (int i = 0; i < a.stages; ++i) mbar_init(k_empty(i), 1);
        for (int i = 0; i < accs; ++i) mbar_init(acc_full(i), 34), mbar_init(acc_empty(i), 4 * parts);
        for (int i = 0; i < 4; ++i) mbar_init(half_full(i), 4);
        for (int i = 0; i < 2; ++i) mbar_init(w_full(i), 1), mbar_init(w_empty(i), kEpiWarps);
        mbar_init(teardown, 1), mbar_init(teardown + 8, 1);
        fence_barrier_init();
    }
    if (!FULL) {                                              // rows of padding heads: zeros that no load overwrites
        for (uint32_t i = tid * 16; i < 2 * q_bytes; i += kThreads * 16)
            *reinterpret_cast<uint4 *>(gbase + i) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
    }
    // (no early start of dependents: `visible` may be a length tensor of the next call, see where it is written)
    grid_dependency_wait();
    bool bad = false;
    if (warp == 17) {
        tmem_alloc(smem_u32(tmem_ptr), kTmemCols);
        tmem_relinquish();
    } else if (warp == 18 && a.chunk == 0) {
        const Share mine = share_of(a, queries, lane, &bad);
        if (lane == 0) *share = mine;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_ptr;
    const Share my_share = a.chunk ? Share{} : *share;

    if (warp == 16) {
        // ---------------- loads ----------------
        int stage = 0, kphase = 0, n = 0;                     // the next stage and its phase; units with tiles
        int kb = 0, fphase = 0, fills = 0;                    // the next fill's barrier and its phase; fills so far
        bool ok = true;
        Units<true> units(my_share);
        Unit u = {};
        while (ok && units.next(a, queries, &bad, u)) {
            if (u.tiles == 0) continue;
            const int qb = n & 1;
            ok = wait_warp(q_empty(qb), ((n >> 1) & 1) ^ 1, abort_flag);
            if (!ok) break;
            if (lane == 0) mbar_expect(q_full(qb), (uint32_t)(u.nq * a.heads) * kDim * elem);
            __syncwarp();
            for (int i = lane; i < u.nq; i += 32) {
                const uint32_t dst = q_smem + qb * q_bytes + i * HP * 128;
                const int row = (u.t0 + i) * a.heads;
                tma_load(dst, &q_map, 0, row, q_full(qb));
                if (!FP8) tma_load(dst + q_rows * 128, &q_map, 64, row, q_full(qb));
            }
            ++n;
            int32_t batch = -1;
            for (int t = 0; t < u.tiles; ++t) {
                const int in = (t << a.boxes_log2) & 31;      // the tile's first box in the batch
                if (in == 0) batch = rows_of(a, u, (u.first_tile + t) * kTile, lane);
                int32_t row = __shfl_sync(0xffffffffu, batch, in + (lane & ((1 << a.boxes_log2) - 1)));
                if (lane >> a.boxes_log2) row = -1;
                const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, row >= 0));
                ok = wait_warp(k_empty(stage), kphase ^ 1, abort_flag);
                if (!ok) break;
                if (lane == 0) mbar_expect(k_full(kb), boxes * a.run * kDim * elem);
                __syncwarp();
                if (row >= 0) {
                    const uint32_t dst = k_smem + stage * k_bytes + lane * a.run * 128;
                    tma_load(dst, &k_map, 0, row, k_full(kb));
                    if (!FP8) tma_load(dst + kTile * 128, &k_map, 64, row, k_full(kb));
                }
                ++fills;
                if (++stage == a.stages) stage = 0, kphase ^= 1;
                if (++kb == 2 * a.stages) kb = 0, fphase ^= 1;
            }
        }
        // The products' last arrivals on the stages and query buffers are asynchronous: they land before the CTA ends
        // (its shared memory may be another's a moment later).  Arrivals on acc_full are waited for by the sums.
        for (int i = 0; ok && i < a.stages; ++i) {
            ok = wait_warp(k_empty(stage), kphase ^ 1, abort_flag);
            if (ok && ++stage == a.stages) stage = 0, kphase ^= 1;
        }
        for (int i = 0; ok && i < 2; ++i) ok = wait_warp(q_empty((n + i) & 1), (((n + i) >> 1) & 1) ^ 1, abort_flag);
        if (!ok) {
            // given up: the copies in flight, at most the last `stages` fills and two query loads, must land before
            // the CTA ends
            const uint64_t t0 = globaltimer_ns();
            for (int i = 0; i < a.stages && i < fills; ++i) {
                if (--kb < 0) kb = 2 * a.stages - 1, fphase ^= 1;
                while (!mbar_try_wait(k_full(kb), fphase) && globaltimer_ns() - t0 < kTimeoutNs) {
                }
            }
            for (int q = 0; q < 2 && q < n; ++q) {
                const int last = (n - 1 - q) >> 1, qb = (n - 1 - q) & 1;
                while (!mbar_try_wait(q_full(qb), last & 1) && globaltimer_ns() - t0 < kTimeoutNs) {
                }
            }
        }
    } else if (warp == 17 || warp == 19) {
        // ---------------- products: one thread each, even and odd tiles of the CTA ----------------
        if (lane == 0) {
            const int odd = warp == 19;     // (and so are its accumulator tiles and k_full barriers: both rings are even)
            int64_t g = 0;
            int stage = 0, kb = 0, fphase = 0, acc = 0, aphase = 0, n = 0;
            bool ok = true;
            Units<false> units(my_share);
            Unit u = {};
            while (ok && units.next(a, queries, &bad, u)) {
                if (u.tiles == 0) continue;
                const int qb = n & 1;
                ok = mbar_wait(q_full(qb), (n >> 1) & 1, abort_flag);
                const uint32_t idesc = a.idesc | ((uint32_t)(u.nq * HP >> 3) << 17);
                const uint64_t bdesc = sdesc_sw128(q_smem + qb * q_bytes, 16, 1024);
                for (int t = 0; t < u.tiles && ok; ++t, ++g) {
                    if ((int)(g & 1) == odd) {
                        ok = mbar_wait(k_full(kb), fphase, abort_flag) && mbar_wait(acc_empty(acc), aphase ^ 1, abort_flag);
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t adesc = sdesc_sw128(k_smem + stage * k_bytes, 16, 1024);
                        const uint32_t d = tmem + acc * (parts * 64);
                        if (FP8) {
#pragma unroll
                            for (int k = 0; k < 4; ++k) umma_f8(d, adesc + 2 * k, bdesc + 2 * k, idesc, k > 0);
                        } else {
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                umma_f16(d, adesc + (k >> 2) * (kTile * 128 >> 4) + 2 * (k & 3),
                                         bdesc + (k >> 2) * (q_rows * 128 >> 4) + 2 * (k & 3), idesc, k > 0);
                        }
                        umma_commit(k_empty(stage));
                        umma_commit(acc_full(acc));
                    }
                    if (++stage == a.stages) stage = 0;
                    if (++kb == 2 * a.stages) kb = 0, fphase ^= 1;
                    if (++acc == accs) acc = 0, aphase ^= 1;
                }
                umma_commit(q_empty(qb));                     // this thread's products of the unit
                ++n;
            }
            if (!ok) {
                umma_commit(teardown + 8 * odd);
                const uint64_t t0 = globaltimer_ns();
                while (!mbar_try_wait(teardown + 8 * odd, 0) && globaltimer_ns() - t0 < kTimeoutNs) {
                }
            }
        }
        __syncwarp();
    } else if (warp == 18) {
        // ---------------- weights of the units, masks and scales of the keys ----------------
        int acc = 0, aphase = 0, units_n = 0;
        bool ok = true;
        Units<true> units(my_share);
        Unit u = {};
        while (ok && units.next(a, queries, &bad, u)) {
            if (u.tiles == 0) continue;
            const int most = visible_of(a, u, u.nq - 1);
            // zero for heads and queries that are not there
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int col = 32 * k + lane, i = col / HP, h = col % HP;
                v[k] = i < u.nq && h < a.heads ? __ldg(a.weights + (int64_t)(u.t0 + i) * a.heads + h) : 0.f;
                if (FP8 && doubled(lane)) v[k] *= 0.5f;
            }
            int32_t batch = rows_of(a, u, u.first_tile * kTile, lane);
            const int wb = units_n & 1;
            ok = wait_warp(w_empty(wb), ((units_n >> 1) & 1) ^ 1, abort_flag);
            if (!ok) break;
#pragma unroll
            for (int k = 0; k < 8; ++k) weights[wb * 256 + 32 * k + lane] = v[k];
            __syncwarp();
            if (lane == 0) mbar_arrive(w_full(wb));
            ++units_n;
            int j = u.first_tile * kTile + 4 * lane;          // four neighbouring keys per lane: they share a box
            for (int t = 0; t < u.tiles; ++t, j += kTile) {
                const int in = (t << a.boxes_log2) & 31;
                if (in == 0 && t > 0) batch = rows_of(a, u, (u.first_tile + t) * kTile, lane);
                int64_t row = __shfl_sync(0xffffffffu, batch, in + (4 * lane >> (7 - a.boxes_log2)));
                row = row >= 0 && j < u.len ? row + (4 * lane & (a.run - 1)) : -1;
                const int n = min(4, u.len - j);
                if (row > a.k_rows - n) row = -1;
                if (row < 0 && j < most && a.status) atomicOr(a.status, SFM_STATUS_BAD_BLOCK);
                ok = wait_warp(acc_empty(acc), aphase ^ 1, abort_flag);        // the slot's last tile has been summed
                if (!ok) break;
                if (a.k_scales && row >= 0) {
                    const float *src = a.k_scales + row;
                    const uint32_t dst = smem_u32(key_scales + acc * kTile + 4 * lane);
                    if (n == 4 && ((uintptr_t)src & 15u) == 0) {
                        cp_async16(dst, src, 16);
                    } else {
                        for (int i = 0; i < n; ++i) cp_async4(dst + 4 * i, src + i);
                    }
                }
                const uint32_t mask = __ballot_sync(0xffffffffu, row >= 0);
                cp_async_arrive_noinc(acc_full(acc));
                if (lane == 0) {
                    key_mask[acc] = mask;
                    mbar_arrive(acc_full(acc));
                }
                if (++acc == accs) acc = 0, aphase ^= 1;
            }
        }
        cp_async_wait_all();                                  // this warp's own copies
    } else {
        // ---------------- clipped sums ----------------
        const int wg = warp >> 2, part = wg & (parts - 1);
        const int turns = 4 >> a.parts_log2;                  // warpgroups that share a part take turns
        const int turn = wg >> a.parts_log2;
        const int i_part = HP <= 64 ? part * kSums : part >> 1;         // first query of this part
        const int key_lane = (warp & 3) * 32 + lane;
        int64_t done = 0;                                     // tiles of this CTA before the unit
        int halves = 0;                                       // HP 128: exchanges so far
        int n = 0;                                            // units with tiles
        bool ok = true;
        Units<true> units(my_share);
        Unit u = {};
        while (ok && units.next(a, queries, &bad, u)) {
            // It may be a length tensor of the planner behind this kernel, which reads lengths as soon as all CTAs have
            // ended: fenced beside the first unit's loads and products, and at the end for all others.  (Only there costs
            // few short sequences half a microsecond, after each unit 17 sequences of 974 queries and keys 7 %.)
            if (a.visible && u.begins && tid < u.rows) {
                a.visible[u.t0 + tid] = visible_of(a, u, tid);
                if (units.k == 1) __threadfence();
            }
            int vis[kSums];
            float *w = weights + (n & 1) * 256;
            if (u.tiles) {
#pragma unroll
                for (int q = 0; q < kSums; ++q) vis[q] = visible_of(a, u, i_part + q);
                ok = wait_warp(w_full(n & 1), (n >> 1) & 1, abort_flag);
                if (!ok) break;
                ++n;
            }
            w += part * 64;
            float *out = a.scores + (int64_t)(u.t0 + i_part) * a.stride;
            for (int t = 0; t < u.tiles; ++t) {
                const int64_t g = done + t;                   // the CTA's tile number
                if ((int)(g & (turns - 1)) != turn) continue;
                const int j = (u.first_tile + t) * kTile + key_lane;
                const int acc = (int)(g & (accs - 1)), phase = (int)((g >> (3 - a.parts_log2)) & 1);
                ok = wait_warp(acc_full(acc), phase, abort_flag);
                if (!ok) break;
                tc_fence_after();
                const bool there = key_mask[acc] >> (key_lane >> 2) & 1u;
                const float scale = a.k_scales ? *(volatile float *)(key_scales + acc * kTile + key_lane) : 1.f;
                float2 sum2[kSums];
                const uint32_t at = tmem + acc * (parts * 64) + part * 64 + ((uint32_t)((warp & 3) * 32) << 16);
                const bool live = i_part < u.nq;
                auto drained = [&] {                          // all of the part has left TMEM: the next product can start
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(acc_empty(acc));
                };
                auto add_up = [&](bool heads_only) {
#pragma unroll
                    for (int q = 0; q < kSums; ++q) sum2[q] = make_float2(0.f, 0.f);
#pragma unroll
                    for (int half = 0; half < 2; ++half) {    // 32 columns at a time
                        uint32_t r[32];
                        tmem_ld32(at + 32 * half, r);
                        tmem_wait_ld();
                        if (half == 1 && FULL) drained();
                        if (!FULL && heads_only) {
#pragma unroll
                            for (int e = 0; e < 32; ++e) {
                                const int h = HP <= 64 ? (32 * half + e) % HP : (part & 1) * 64 + 32 * half + e;
                                r[e] = h < a.heads ? r[e] : 0u;
                            }
                        }
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float4 v = *reinterpret_cast<const float4 *>(w + 32 * half + 4 * e);
                            float2 &s2 = sum2[(half * 8 + e) / (16 / kSums)];
                            auto cut_off = [&](int k) { return FP8 && doubled(k) ? clip_twice(r[4 * e + k]) : clip(r[4 * e + k]); };
                            s2 = fma2(make_float2(cut_off(0), cut_off(1)), make_float2(v.x, v.y), s2);
                            s2 = fma2(make_float2(cut_off(2), cut_off(3)), make_float2(v.z, v.w), s2);
                        }
                    }
                };
                if (live && FULL) {
                    add_up(false);
                } else if (live) {
                    // a column without a head is 0, or NaN for a key with an infinite value: then once more without it
                    bool again = false;
                    while (true) {
                        add_up(again);
                        bool nan = false;
#pragma unroll
                        for (int q = 0; q < kSums; ++q) nan |= isnan(sum2[q].x + sum2[q].y);
                        if (again || !__any_sync(0xffffffffu, nan)) {
                            drained();
                            break;
                        }
                        again = true;
                    }
                } else {
                    drained();
                }
                float sum[kSums];
#pragma unroll
                for (int q = 0; q < kSums; ++q) sum[q] = sum2[q].x + sum2[q].y;
                if constexpr (HP == 128) {                    // the odd part hands its half to the even one
                    float *mine = half_sum + (wg >> 1) * 128 + key_lane;
                    if (part & 1) {
                        ok = halves == 0 || wait_warp(half_full(wg ^ 1), (halves - 1) & 1, abort_flag);   // taken
                        if (!ok) break;
                        *mine = sum[0];
                    } else {
                        ok = wait_warp(half_full(wg ^ 1), halves & 1, abort_flag);
                        if (!ok) break;
                        sum[0] += *mine;
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(half_full(wg));
                    ++halves;
                    if (part & 1) continue;
                }
                if (live && j < a.max_k) {
                    float *dst = out + j;
#pragma unroll
                    for (int q = 0; q < kSums; ++q, dst += a.stride)
                        if (i_part + q < u.nq) *dst = j < vis[q] && there ? sum[q] * scale : -INFINITY;
                }
            }
            done += u.tiles;
            if (!ok) break;
            if (u.tiles) {
                __syncwarp();
                if (lane == 0) mbar_arrive(w_empty((n - 1) & 1));
            }
            // columns that no product reached, and under the products the rows without a query
            for (int i = warp; i < u.rows; i += kEpiWarps) {
                float *dst = a.scores + (int64_t)(u.t0 + i) * a.stride;
                for (int j = u.fill0 + lane; j < u.fill1; j += 32) dst[j] = -INFINITY;
                if (i >= u.nq) {
                    const int c0 = u.first_tile * kTile, c1 = min(c0 + u.tiles * kTile, a.max_k);
                    for (int j = c0 + lane; j < c1; j += 32) dst[j] = -INFINITY;
                }
            }
        }
        if (a.visible && warp == 0 && units.k > 1) __threadfence();
    }
    if (bad && a.status) atomicOr(a.status, SFM_STATUS_BAD_LENGTH);

    tc_fence_before();
    __syncthreads();
    if (tid == 0 && *abort_flag && a.status) atomicOr(a.status, SFM_STATUS_TIMEOUT);
    if (warp == 17) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

using EncodeFn = decltype(&cuTensorMapEncodeTiled);

// the driver's encoder of TMA descriptors (a pure host function), looked up once
EncodeFn encoder()
{
    static const EncodeFn fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeFn>(p);
    }();
    return fn;
}

int make_map(CUtensorMap *map, const void *ptr, int dtype, int64_t rows, int64_t row_bytes, int box_rows)
{
    const EncodeFn encode = encoder();
    if (!encode) return SFM_ERR_CUDA;
    const bool fp8 = dtype == SFM_DTYPE_E4M3;
    const CUtensorMapDataType type = fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                     : dtype == SFM_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                               : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const cuuint64_t dims[2] = {kDim, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)row_bytes};
    const cuuint32_t box[2] = {fp8 ? 128u : 64u, (cuuint32_t)box_rows}, steps[2] = {1, 1};
    const CUresult r = encode(map, type, 2, const_cast<void *>(ptr), dims, strides, box, steps,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? SFM_OK : SFM_ERR_CUDA;
}

template <int HP, bool FULL, bool FP8>
cudaError_t launch(const IndexArgs &a, const CUtensorMap &q, const CUtensorMap &k, int device, int grid, size_t smem,
                   cudaStream_t st)
{
    static std::atomic<bool> ready[kMaxDevices];
    return prepared_launch(
        ready, device,
        [&] {
            return cudaFuncSetAttribute(sfm_index_kernel<HP, FULL, FP8>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemLimit);
        },
        [&] {
            return launch_dependent(sfm_index_kernel<HP, FULL, FP8>, dim3((unsigned)grid), dim3(kThreads), smem, st, a, q, k);
        });
}

}  // namespace
}  // namespace sfm

using namespace sfm;

extern "C" int sfm_index_scores(const sfm_index_params *pp, const sfm_index_tensors *t, float *scores,
                                int64_t score_stride, int32_t *visible, int32_t *status, sfm_stream_t stream)
{
    if (!pp || !t) return SFM_ERR_INVALID_ARG;
    const sfm_index_params &p = *pp;
    if (p.num_heads < 1 || p.num_heads > 128) return SFM_ERR_INVALID_ARG;
    if (p.index_dim != kDim) return SFM_ERR_UNSUPPORTED;
    if (p.dtype != SFM_DTYPE_BF16 && p.dtype != SFM_DTYPE_FP16 && p.dtype != SFM_DTYPE_E4M3) return SFM_ERR_INVALID_ARG;
    if (p.layout_q != SFM_LAYOUT_BSND && p.layout_q != SFM_LAYOUT_TND) return SFM_ERR_LAYOUT;
    if (p.layout_kv != SFM_LAYOUT_BSND && p.layout_kv != SFM_LAYOUT_TND && p.layout_kv != SFM_LAYOUT_PAGED)
        return SFM_ERR_LAYOUT;
    if (p.layout_kv != SFM_LAYOUT_PAGED && p.layout_kv != p.layout_q) return SFM_ERR_LAYOUT;
    if (p.batch_size <= 0 || p.max_seqlen_q <= 0 || p.max_seqlen_kv <= 0 || p.cmp_ratio <= 0) return SFM_ERR_INVALID_ARG;
    if (p.mask_mode != 0 && p.mask_mode != 3) return SFM_ERR_INVALID_ARG;
    if (p.layout_q == SFM_LAYOUT_TND && p.total_q < 0) return SFM_ERR_INVALID_ARG;
    if (p.max_seqlen_kv > INT32_MAX - 2 * kTile) return SFM_ERR_UNSUPPORTED;    // columns are counted in whole tiles
    const int64_t tokens = p.layout_q == SFM_LAYOUT_TND ? p.total_q : (int64_t)p.batch_size * p.max_seqlen_q;
    if (tokens * p.num_heads > INT32_MAX) return SFM_ERR_UNSUPPORTED;      // rows that a copy's coordinate names
    const bool paged = p.layout_kv == SFM_LAYOUT_PAGED;
    if (paged && (p.block_size < 16 || p.block_size > 1024 || p.block_size % 16)) return SFM_ERR_LAYOUT;
    if (score_stride < p.max_seqlen_kv) return SFM_ERR_LAYOUT;
    const int elem = p.dtype == SFM_DTYPE_E4M3 ? 1 : 2;
    if (t->k_row_stride < kDim * elem || t->k_row_stride % 16 || t->k_rows <= 0) return SFM_ERR_LAYOUT;
    if (t->k_rows > ((int64_t)1 << 31) - 2) return SFM_ERR_UNSUPPORTED;
    if (p.layout_q == SFM_LAYOUT_TND && !t->cu_seqlens_q) return SFM_ERR_INVALID_ARG;
    if (p.layout_kv == SFM_LAYOUT_TND && !t->cu_seqlens_kv) return SFM_ERR_INVALID_ARG;
    if (paged ? !t->seqused_kv || !t->block_table || t->block_table_stride <= 0 : t->block_table != nullptr)
        return SFM_ERR_INVALID_ARG;
    if (p.mask_mode == 3 && p.cmp_ratio > 1 && !t->cmp_residual_kv) return SFM_ERR_INVALID_ARG;
    if (tokens == 0) return SFM_OK;
    if (!t->q || !t->k || !t->weights || !scores) return SFM_ERR_INVALID_ARG;
    if (((uintptr_t)t->q | (uintptr_t)t->k) & 15u) return SFM_ERR_LAYOUT;
    if (((uintptr_t)t->k_scales | (uintptr_t)t->weights | (uintptr_t)scores | (uintptr_t)visible) & 3u)
        return SFM_ERR_LAYOUT;

    int dev = 0, sms = 0;
    if (current_sms(&dev, &sms) != cudaSuccess) return SFM_ERR_CUDA;

    // a ragged batch may come with any upper bound: no sequence has more queries than all have
    const int32_t max_q = p.layout_q == SFM_LAYOUT_TND && p.total_q < p.max_seqlen_q ? p.total_q : p.max_seqlen_q;
    const int hp = p.num_heads <= 16 ? 16 : p.num_heads <= 32 ? 32 : p.num_heads <= 64 ? 64 : 128;
    IndexArgs a = {};
    a.weights = t->weights;
    a.k_scales = t->k_scales;
    a.scores = scores;
    a.visible = visible;
    a.status = status;
    a.table = t->block_table;
    a.table_stride = t->block_table_stride;
    a.cu_q = p.layout_q == SFM_LAYOUT_TND ? t->cu_seqlens_q : nullptr;
    a.cu_k = p.layout_kv == SFM_LAYOUT_TND ? t->cu_seqlens_kv : nullptr;
    a.used_q = t->seqused_q;
    a.used_k = t->seqused_kv;
    a.residual = t->cmp_residual_kv;
    a.stride = score_stride;
    a.k_rows = t->k_rows;
    a.heads = p.num_heads;
    a.batch = p.batch_size;
    a.max_q = max_q;
    a.total_q = p.total_q;
    a.max_k = p.max_seqlen_kv;
    a.ratio = p.cmp_ratio;
    a.causal = p.mask_mode == 3;
    a.layout_q = p.layout_q;
    a.layout_kv = p.layout_kv;
    a.block = p.block_size;
    a.block_div = make_fastdiv(paged ? (uint32_t)p.block_size : 1u);
    a.ratio_div = make_fastdiv((uint32_t)p.cmp_ratio);
    a.fp8 = p.dtype == SFM_DTYPE_E4M3;

    // 64-column parts of a tile: as many as one sequence's queries fill
    const int64_t cols = (int64_t)max_q * hp;
    a.parts_log2 = cols <= 64 ? 0 : cols <= 128 ? 1 : 2;
    const int queries = (64 << a.parts_log2) / hp;
    // accumulate in fp32; types of A and B; M = 128
    a.idesc = (1u << 4) | ((p.dtype == SFM_DTYPE_BF16 ? 1u : 0u) << 7) | ((p.dtype == SFM_DTYPE_BF16 ? 1u : 0u) << 10) |
              ((uint32_t)(kTile >> 4) << 24);
    // keys per box: the largest power of two that divides a page
    a.run = kTile;
    if (paged) {
        a.run = p.block_size & -p.block_size;
        if (a.run > kTile) a.run = kTile;
    }
    while ((a.run << a.boxes_log2) < kTile) ++a.boxes_log2;
    const uint32_t q_bytes = (64u << a.parts_log2) * kDim * elem, k_bytes = kTile * kDim * elem;
    const uint32_t scale_bytes = t->k_scales ? kScaleBytes : 0;
    const uint32_t misc_bytes = kMiscBytes - (hp == 128 ? 0 : 1024) + scale_bytes;
    const int fit = (int)((kSmemLimit - misc_bytes - 2 * q_bytes) / k_bytes);
    a.stages = fit < kMaxStages ? fit : kMaxStages;

    a.groups_per_seq = (int32_t)(((int64_t)max_q + queries - 1) / queries);
    const int64_t groups = (int64_t)a.groups_per_seq * p.batch_size;
    const int64_t tiles = ((int64_t)p.max_seqlen_kv + kTile - 1) / kTile;
    if (groups > INT32_MAX) return SFM_ERR_UNSUPPORTED;
    a.groups = (int32_t)groups;
    a.all_tiles = (int32_t)tiles;
    a.groups_div = make_fastdiv((uint32_t)groups);
    a.seq_div = make_fastdiv((uint32_t)a.groups_per_seq);
    int64_t units = groups * tiles;                // at most one CTA per tile
    if (groups > kShareGroups || units <= sms) {
        // one tile per CTA where that many CTAs are there (counting shares out would cost them a microsecond), else
        // units of 8 to 32 tiles, some six per CTA at least
        int64_t chunk = groups * tiles / (6 * (int64_t)sms);
        chunk = chunk < 8 ? 8 : chunk > 32 ? 32 : chunk;
        const int64_t chunks = (tiles + chunk - 1) / chunk;
        a.chunk = units <= sms ? 1 : (int32_t)((tiles + chunks - 1) / chunks);
        units = groups * ((tiles + a.chunk - 1) / a.chunk);
        if (units > INT32_MAX - sms) return SFM_ERR_UNSUPPORTED;
        a.units = (int32_t)units;
    }

    CUtensorMap q_map, k_map;
    int rc = make_map(&q_map, t->q, p.dtype, tokens * p.num_heads, (int64_t)kDim * elem, p.num_heads);
    if (!rc) rc = make_map(&k_map, t->k, p.dtype, t->k_rows, t->k_row_stride, a.run);
    if (rc) return rc;
    const size_t smem = 2 * q_bytes + (size_t)a.stages * k_bytes + misc_bytes;
    const int grid = (int)(units < sms ? units : sms);
    const cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e;
    const bool full = p.num_heads == hp;
    auto go = [&](auto width) {
        constexpr int kWidth = decltype(width)::value;
        auto run = a.fp8 ? full ? launch<kWidth, true, true> : launch<kWidth, false, true>
                         : full ? launch<kWidth, true, false> : launch<kWidth, false, false>;
        return run(a, q_map, k_map, dev, grid, smem, st);
    };
    switch (hp) {
    case 16: e = go(std::integral_constant<int, 16>{}); break;
    case 32: e = go(std::integral_constant<int, 32>{}); break;
    case 64: e = go(std::integral_constant<int, 64>{}); break;
    default: e = go(std::integral_constant<int, 128>{}); break;
    }
    return e == cudaSuccess ? SFM_OK : SFM_ERR_CUDA;
}
