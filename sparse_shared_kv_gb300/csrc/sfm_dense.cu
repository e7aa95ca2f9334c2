// sfm_dense.cu -- attention of many queries over the same rows
// (sfm_dense_forward): prompts, single tokens over a cache, drafted trees.
//
// A tile of the work is 128 rows of Q -- consecutive (token, head) rows of one
// sequence, whatever the number of heads -- against 128 keys at a time.  A pair
// of CTAs holds it, 64 rows each, and both products are pair products (M = 128):
//
//     S = Q K^T      N = 128 keys, K = 512    CTA c stages keys [64 c, 64 c + 64)
//     O += P V       N = 2 x 256, K = 128     CTA c stages 256 of the 512 columns of all 128 keys
//
// The rows are K and V at once, but a CTA's part of K and its part of V share a
// quarter of the tile only, and a pair product wants both CTAs' operands at the
// same offsets, so both are copied (TMA, 128 KB per tile and CTA; the second copy
// hits L2).  O fills half of the tensor memory (64 x 512 fp32 in 128 lanes x 256
// columns), four S tiles of 64 columns the other.
//
// Per CTA, 12 warps:
//   0      copies: Q of a unit, then K(0), K(1), K(2), V(0), K(3), V(1), ... in stages of 32 KB, one copy each (64 keys x 256
//          values as four blocks of 64 values; pages of fewer rows one each), four stages in a ring
//   1      products, in the pair's first CTA: S(0), S(1), S(2), O += P(0) V(0), S(3), O += P(1) V(1), ...
//   2      tensor memory; takes NaN and infinities out of V rows that some row must not see (below)
//   3      units: which rows and keys come next, three units ahead
//   4-11   softmax: four threads per row, 32 keys each; running maximum, moved (and O rescaled) only when it grows by more
//          than 8 in the log2 domain; P in dtype into shared memory; the results
//
// What bounds it: a tile is 2048 clocks of the tensor cores (16384 FLOP per clock and pair).  Of long ranges of keys it takes
// 2700 to 2800 (tensor cores 71 to 76 % busy, 1.60 to 1.68 PFLOP/s where the GPU is cool: 84 to 88 % of a 1914 TFLOP/s burst
// of matrix products); called again and again it runs into the GPU's power limit, as such products do (1721), and the
// clock falls to 1.6 to 1.75 GHz (1.46 to 1.49 PFLOP/s).  Every unit costs some 5000 clocks of the softmax's besides (its
// results are written, the next unit's rows looked up), which units of few tiles do not hide: 4096 causal tokens of 64
// heads 1.30, documents of some 1600 1.27 PFLOP/s, and prompts with a window of 128 (two or three tiles per unit) 1.5 to 2
// times what their rows of q and out take to move.  Single tokens over long keys (32 x 24 k keys of 64 heads 4.4 TB/s, with 10 us to
// plan and 9 us to join) wait for copies without filling the memory or the tensor cores (61 and 53 % busy): half of the ring
// holds V, which comes from L2, so that 64 KB per SM are on their way from memory, and a token's 64 rows are half of a pair's.
//
// A unit is a tile of Q and a piece of its range of keys.  Pieces of a range
// leave fp32 partial results in the workspace, which a second kernel joins.
//
// A weight of 0 for a key that a row does not see leaves NaN where the key's
// row holds NaN or an infinity.  Such a key has scores that are not finite for
// every row, so the softmax finds it among the keys it masks; the products
// then wait until the values that are not finite are zeros in the staged V.
//
// Every wait is bounded (2 s, of those that may take a unit 4 s without a tile); a
// timeout raises the CTA's abort flag, every role
// leaves its loop, copies and products in flight are waited for, tensor memory
// is freed and SFM_STATUS_TIMEOUT is set.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "sfm_dense.cuh"
#include "sfm_pair.cuh"

namespace sfm {
namespace {

using namespace tc;

constexpr int kD = 512;
constexpr int kThreads = 384;
constexpr int kRows = 128;                    // rows of Q of a pair
constexpr int kKeys = 128;                    // keys of a tile
constexpr int kStages = 4;
constexpr int kBlocks = 4;                    // blocks of 64 values x 64 rows (8 KB) of a stage
constexpr int kSteps = 8 / kBlocks;           // stages of K, and of V, of a tile
constexpr uint32_t kStageBytes = kBlocks * 8192;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescale = 8.0f;              // log2 units
// fp16 weights are 2^6 times what they stand for: 2^14 at most, and those far below the largest keep their bits down to 2^-20
// of it (from 1 on, to 2^-14)
template <bool kBf16>
constexpr float kLift = kBf16 ? 0.f : 6.f;

constexpr uint32_t Q_OFF = 0;                 // 8 blocks of 64 rows x 64 values
constexpr uint32_t P_OFF = 65536;             // 2 buffers x 2 blocks of 64 rows x 64 keys
constexpr uint32_t KV_OFF = P_OFF + 32768;
constexpr uint32_t MISC_OFF = KV_OFF + kStages * kStageBytes;
constexpr uint32_t kMiscBytes = 3 << 10, kSmemBytes = MISC_OFF + kMiscBytes;
static_assert(kSmemBytes <= 232448, "shared memory budget");

constexpr uint32_t TM_O = 0, TM_S = 256, kTmemCols = 512;

// barriers (8 bytes each) at MISC_OFF; "first": used in the pair's first CTA
enum Bar {
    B_KV_FULL = 0,       // [4] first: both CTAs' halves of a stage have landed
    B_KV_EMPTY = 4,      // [4] the products that read the stage are done
    B_Q_FULL = 8,        // first
    B_Q_EMPTY = 9,       // the unit's last S is done
    B_S_FULL = 10,       // [4] S of a tile
    B_P_FULL = 14,       // [2] first: P written, O rescaled, S read, by the 16 softmax warps of both CTAs
    B_O_DONE = 16,       // [2] O += P V of a tile
    B_O_FREE = 18,       // first: the 16 softmax warps have read the unit's O
    B_UNIT_FULL = 19,    // [kUnits]
    B_UNIT_EMPTY = 22,   // [kUnits]
    B_FIX = 25,          // rows to be made finite
    B_FIXED = 26,        // first: both CTAs have
    B_END = 27,          // after a timeout: all products are done
    B_CHECKED = 28,      // [kUnits] the unit's blocks have been looked at
    kBars = 31
};
constexpr int kUnits = 3;                     // units that are worked out ahead
constexpr int kAhead = 3;                     // tiles whose S is issued before the first of them gets its O += P V
constexpr uint32_t EXCH_REL = 256;            // [2][4][64] floats: the row's four maxima (or sums)
constexpr uint32_t UNIT_REL = EXCH_REL + 2048;   // [kUnits] Unit
constexpr uint32_t CAND_REL = UNIT_REL + kUnits * 128;    // first: [2][4] words of keys that may hold NaN or infinities
constexpr uint32_t FIX_REL = CAND_REL + 32;      // words, first stage, quit
constexpr uint32_t TMEM_REL = FIX_REL + 32;
constexpr uint32_t ABORT_REL = TMEM_REL + 4;
constexpr uint32_t BEAT_REL = ABORT_REL + 4;
static_assert(UNIT_REL % 128 == 0 && kBars * 8 <= EXCH_REL && BEAT_REL + 4 <= kMiscBytes, "misc area");

struct alignas(128) Unit {
    int64_t row0;            // first row of Q (and of the outputs)
    int64_t kv0;
    int32_t valid, b, rows, used;      // rows of the tile, and those of queries that count
    int32_t i0, h0;          // query and head of the first row
    int32_t q0, q_len, len, prefix;
    int32_t prefix_tiles, b0, tile0, tiles;    // tiles: [0, prefix_tiles) from key 0, then from key b0; this unit's part
    int32_t piece, splits, part, bad;  // of how many pieces of the tile's keys (first or not), where its partial result goes;
                                       // bad: a block of the range is outside the cache
};
static_assert(sizeof(Unit) <= 128, "unit area");

// A slot is a tile of Q of some sequence.  Either every slot's keys are cut into pieces of at most `chunk` tiles, at most
// `splits` of them, and units (slot, piece) go to the pairs in turns, or (balanced) the pairs get the same number of tiles:
// whole slots in turns first, as long as none gets more than its share, so that the pairs go through a sequence's keys side
// by side and find them in L2; then parts of the concatenation of the other slots' tiles, which begin and end in the middle
// of slots.  (With such parts alone every sequence is under way at once: 16 trees of 16 tokens over 200 MB of keys 509 us.)
struct Plan {
    int32_t slots, splits, chunk, box_rows, align, units, balanced, pairs;
    int32_t block_bytes, octet_bytes;     // of a stage's 64 keys: from one block of 64 values to the next, from eight keys to the next
    uint32_t idesc_s, idesc_o;
    float4 *part_o;          // partial results: [part][128][128]; balanced: part 2 n of the n-th part of the tiles continues a slot, 2 n + 1 begins one
    float2 *part_ml;         // [part][128]
    int4 *head;              // per slot, or (balanced) per part of the tiles for the slot that begins in it and goes on behind it: pieces, rows that
                             // count, first row, first part (balanced: of the tiles)
    FastDiv slots_div, per_seq_div;
    int32_t per_seq;         // BSND: tiles per sequence
};
constexpr int kMostBalanced = 1536;           // slots, and sequences: every CTA counts their tiles
constexpr int kLeastTiles = 4;                // of a pair's share
constexpr int kMostPairs = 512;

// First slot of a sequence of a TND batch whose first row is q0: at least one more per sequence than whole tiles lie before
// it, so that every sequence has as many slots as tiles.
__device__ __forceinline__ int slot_base(const DenseArgs &a, int b, int q0) { return (int)((int64_t)q0 * a.heads / kRows) + b; }

__device__ __forceinline__ int first_query(const DenseArgs &a, int b) { return min(max(__ldg(a.cu_q + b), 0), a.total_q); }

// The last sequence whose first slot is at most `slot`, by halves; query_of: a sequence's first row.
template <typename Fn>
__device__ __forceinline__ int sequence_by_halves(const DenseArgs &a, int slot, Fn query_of)
{
    int lo = 0, hi = a.batch - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (slot_base(a, mid, query_of(mid)) <= slot) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// The sequence of a slot, found by the whole warp 32 ways at a time, and the slot's number k in it (< 0: none).  Where offsets
// fall this search and the one by halves find different sequences, and the balanced plan was made with the latter: the units
// then go by it too, so that they are what the plan has counted.
__device__ __forceinline__ DenseSeq slot_sequence(const DenseArgs &a, const Plan &pl, int slot, int lane, int &k, bool falls)
{
    int b = 0;
    if (a.cu_q && falls) {
        b = sequence_by_halves(a, slot, [&](int i) { return first_query(a, i); });
    } else if (a.cu_q) {
        for (int n = a.batch; n > 1;) {
            const int step = (n + 31) / 32, i = b + lane * step;
            const bool below = lane * step < n && (lane == 0 || slot_base(a, i, first_query(a, i)) <= slot);
            const int w = 31 - __clz(__ballot_sync(0xffffffffu, below));
            b += w * step;
            n = min(step, n - w * step);
        }
    } else {
        b = (int)fdiv((uint32_t)slot, pl.per_seq_div);
    }
    const DenseSeq s = dense_seq(a, b);
    k = a.cu_q ? slot - slot_base(a, b, s.q0) : slot - b * pl.per_seq;
    return s;
}

__device__ __forceinline__ int warp_min(int v) { return __reduce_min_sync(0xffffffffu, v); }
__device__ __forceinline__ int warp_max(int v) { return __reduce_max_sync(0xffffffffu, v); }

// Cache row of key j (a multiple of the box's rows, so that its page holds the whole box), or a row behind the cache, which
// the copies fill with zeros.
__device__ __forceinline__ int32_t box_row(const DenseArgs &a, int b, int64_t kv0, int len, int j, bool *bad)
{
    if (j >= len) return (int32_t)a.kv_rows;
    if (a.layout_kv != SFM_LAYOUT_PAGED) return (int32_t)(kv0 + j);
    const int blk = (int)fdiv((uint32_t)j, a.block_div);
    const int32_t id = __ldg(a.table + (int64_t)b * a.cols + blk);
    if (id < 0 || ((int64_t)id + 1) * a.block > a.kv_rows) {
        *bad = true;
        return (int32_t)a.kv_rows;
    }
    return id * a.block + (j - blk * a.block);
}

// Keys [lo, hi) that queries [i0, i1] of a sequence see besides its prefix, by `lanes` threads of which this is the lane-th;
// each gets its share's.  Without ranges of their own the first query sees the first key and the last one the last.
__device__ __forceinline__ void span(const DenseArgs &a, const DenseSeq &s, int i0, int i1, int lane, int lanes, int &lo, int &hi)
{
    lo = INT32_MAX;
    hi = 0;
    if (a.begin || a.end || (a.words && a.mode == 4)) {
        for (int i = i0 + lane; i <= i1; i += lanes) {
            const DenseRow r = dense_row(a, s, i);
            if (r.hi > r.lo) {
                lo = min(lo, r.lo);
                hi = max(hi, r.hi);
            }
        }
    } else {
        lo = dense_row(a, s, i0).lo;       // 0 where that query sees nothing
        hi = dense_row(a, s, i1).hi;
    }
    if (a.words) {
        lo = min(lo, max(s.len - s.q_len, 0));
        hi = s.len;
    }
}

// Tiles of keys of a tile of Q whose queries see [0, prefix) and [lo, hi), and where those behind the prefix begin.
__device__ __forceinline__ int tiles_of(const Plan &pl, int prefix, int lo, int hi, int &b0)
{
    int tiles = (prefix + kKeys - 1) / kKeys;
    b0 = tiles * kKeys;
    if (hi > lo) {
        b0 = max(b0, lo & ~(pl.align - 1));
        if (hi > b0) tiles += (hi - b0 + kKeys - 1) / kKeys;
    }
    return tiles;
}

// The same from the batch's sequences in shared memory, by one thread.
__device__ __forceinline__ DenseSeq known_sequence(const DenseArgs &a, const Plan &pl, int slot, const DenseSeq *seqs, int &k)
{
    int b;
    if (a.cu_q) {
        b = sequence_by_halves(a, slot, [&](int i) { return seqs[i].q0; });
        k = slot - slot_base(a, b, seqs[b].q0);
    } else {
        b = (int)fdiv((uint32_t)slot, pl.per_seq_div);
        k = slot - b * pl.per_seq;
    }
    return seqs[b];
}

// What a slot counts among all (balanced), found by one thread: its tiles, one if it has rows without keys, none without
// rows; its first row and how many count.
__device__ __forceinline__ int slot_weight(const DenseArgs &a, const Plan &pl, int slot, const DenseSeq *seqs, int &row0, int &used)
{
    int k;
    const DenseSeq s = known_sequence(a, pl, slot, seqs, k);
    const int64_t row = (int64_t)k * kRows;
    row0 = used = 0;
    if (k < 0 || row >= (int64_t)s.q_cap * a.heads) return 0;
    row0 = (int)((int64_t)s.q0 * a.heads + row);
    used = (int)min(max((int64_t)s.q_len * a.heads - row, (int64_t)0), (int64_t)kRows);
    if (used == 0) return 1;
    int lo, hi, b0;
    span(a, s, (int)fdiv((uint32_t)row, a.heads_div), (int)fdiv((uint32_t)(row + used - 1), a.heads_div), 0, 1, lo, hi);
    return max(tiles_of(pl, s.prefix, lo, hi, b0), 1);
}

// A slot, worked out by the whole warp: everything but which of its tiles a unit takes.  -1: no rows; otherwise its tiles.
__device__ __forceinline__ int make_slot(const DenseArgs &a, const Plan &pl, int slot, int lane, Unit &w, const DenseSeq *seqs, bool falls)
{
    int k;
    const DenseSeq s = seqs ? known_sequence(a, pl, slot, seqs, k) : slot_sequence(a, pl, slot, lane, k, falls);
    const int64_t first_row = (int64_t)k * kRows, all = (int64_t)s.q_cap * a.heads;
    if (k < 0 || first_row >= all) return -1;
    w.row0 = (int64_t)s.q0 * a.heads + first_row;
    w.rows = (int32_t)min((int64_t)kRows, all - first_row);
    w.used = (int32_t)min(max((int64_t)s.q_len * a.heads - first_row, (int64_t)0), (int64_t)w.rows);
    w.i0 = (int32_t)fdiv((uint32_t)first_row, a.heads_div);
    w.h0 = (int32_t)(first_row - (int64_t)w.i0 * a.heads);
    int lo = INT32_MAX, hi = 0;
    if (w.used > 0) span(a, s, w.i0, (int)fdiv((uint32_t)(first_row + w.used - 1), a.heads_div), lane, 32, lo, hi);
    lo = warp_min(lo);
    hi = warp_max(hi);
    w.prefix = w.used > 0 ? s.prefix : 0;
    w.prefix_tiles = (w.prefix + kKeys - 1) / kKeys;
    w.valid = 1;
    w.b = s.b;
    w.kv0 = s.kv0;
    w.q0 = s.q0;
    w.q_len = s.q_len;
    w.len = s.len;
    return tiles_of(pl, w.prefix, lo, hi, w.b0);
}

// Blocks outside the cache among the unit's tiles, found by the whole warp.
__device__ __forceinline__ void check_blocks(const DenseArgs &a, Unit &w, int lane)
{
    w.bad = 0;
    if (a.layout_kv != SFM_LAYOUT_PAGED) return;
    // pages of the tiles in the prefix, then of those behind it
    bool bad = false;
    auto check = [&](int tile, int end, int key) {
        if (tile >= end) return;
        const int last = (min(key + (end - tile) * kKeys, w.len) - 1) / a.block;
#pragma unroll 4
        for (int i = key / a.block + lane; i <= last; i += 32) {
            const int32_t id = __ldg(a.table + (int64_t)w.b * a.cols + i);
            bad |= id < 0 || ((int64_t)id + 1) * a.block > a.kv_rows;
        }
    };
    const int end = w.tile0 + w.tiles, second = max(w.tile0, w.prefix_tiles);
    check(w.tile0, min(end, w.prefix_tiles), w.tile0 * kKeys);
    check(second, end, w.b0 + (second - w.prefix_tiles) * kKeys);
    w.bad = __any_sync(0xffffffffu, bad);
    if (w.bad && lane == 0) dense_status(a, SFM_STATUS_BAD_BLOCK);
}

// What every CTA works out for the balanced plan, in P's memory.
struct Balance {
    int32_t before[kMostBalanced + 1];    // a slot's weight, then the weights of all slots before it
    int32_t row0[kMostBalanced], used[kMostBalanced];     // its first row, and how many count
    int32_t begin[kMostPairs + 1];        // of the tiles behind the whole slots: where each pair's part begins
    int32_t rank[kMostPairs + 1];         // pairs before it whose part is not empty
    int32_t waves;                        // whole slots per pair
};

static_assert(sizeof(Balance) <= 32768 && kMostBalanced * sizeof(DenseSeq) <= kStages * kStageBytes, "counted in P's and the stages' memory");

// before, begin, rank and waves from the slots' weights, by one warp.
__device__ __forceinline__ void make_balance(const Plan &pl, Balance &b, int lane)
{
    const int n = pl.slots, G = pl.pairs, each = (n + 31) / 32, at = min(lane * each, n), end = min(at + each, n);
    int mine = 0;
    for (int i = at; i < end; ++i) mine += b.before[i];
    int sum = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += v;
    }
    const int total = __shfl_sync(0xffffffffu, sum, 31);
    sum -= mine;
    for (int i = at; i < end; ++i) {
        const int w = b.before[i];
        b.before[i] = sum;
        sum += w;
    }
    if (lane == 31) b.before[n] = total;
    __syncwarp();
    const int per = max((total + G - 1) / G, kLeastTiles);
    auto load = [&](int c, int waves) {
        int l = 0;
        for (int w = 0; w < waves; ++w) l += b.before[c + w * G + 1] - b.before[c + w * G];
        return l;
    };
    int waves = n / G;
    while (waves > 0) {
        bool over = false;
        for (int c = lane; c < G; c += 32) over |= load(c, waves) > per;
        if (!__any_sync(0xffffffffu, over)) break;
        --waves;
    }
    const int rest = total - b.before[min(waves * G, n)];
    int begin = 0, rank = 0;
    for (int c0 = 0; c0 < G; c0 += 32) {
        const int c = c0 + lane;
        int part = c < G ? per - load(c, waves) : 0, incl = part;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += v;
        }
        const int first = min(begin + incl - part, rest), last = min(begin + incl, rest);
        const uint32_t some = __ballot_sync(0xffffffffu, last > first);
        if (c < G) {
            b.begin[c] = first;
            b.rank[c] = rank + __popc(some & ((1u << lane) - 1u));
        }
        begin += __shfl_sync(0xffffffffu, incl, 31);
        rank += __popc(some);
    }
    if (lane == 0) {
        b.begin[G] = rest;
        b.rank[G] = rank;
        b.waves = waves;
    }
    __syncwarp();
}

// The last entry of n sorted ones that is at most x.
__device__ __forceinline__ int last_at_most(const int32_t *v, int n, int x)
{
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (v[mid] <= x) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// A pair's way through its whole slots and its part of the tiles behind them.
struct Share {
    int wave, waves, slot, off, at, end, rank;      // next slot and tile of it; that tile among all of the part's kind, the part's end
};

__device__ __forceinline__ Share make_share(const Plan &pl, const Balance &b, int c)
{
    Share s;
    const int first = min(b.waves * pl.pairs, pl.slots), base = b.before[first];
    s.wave = 0;
    s.waves = b.waves;
    s.at = b.begin[c];
    s.end = b.begin[c + 1];
    s.rank = b.rank[c];
    s.slot = last_at_most(b.before, pl.slots, base + s.at);      // (of slots without rows, which begin where the next does, the last)
    s.off = base + s.at - b.before[s.slot];
    return s;
}

// The next unit: of the pair's share, or (not balanced) piece and slot u.  False: there is nothing to do.
__device__ __forceinline__ bool make_unit(const DenseArgs &a, const Plan &pl, Share &s, int u, int c, int lane, Unit &w, const DenseSeq *seqs, bool falls)
{
    const bool wave = s.wave < s.waves;
    int slot, off = 0, split = 0;
    if (!pl.balanced) {
        split = (int)fdiv((uint32_t)u, pl.slots_div);
        slot = pl.slots - 1 - (u - split * pl.slots);
    } else if (wave) {
        slot = c + s.wave++ * pl.pairs;
    } else {
        slot = s.slot++;
        off = s.off;
        s.off = 0;
    }
    const int tiles = make_slot(a, pl, slot, lane, w, seqs, falls);
    if (pl.balanced) {
        if (tiles < 0) return false;
        const int weight = max(tiles, 1), take = wave ? weight : min(weight - off, s.end - s.at);
        if (take <= 0) return false;           // (no plan has such a part: the copies and products would take it for the end)
        if (!wave) s.at += take;
        w.tile0 = off;
        w.tiles = tiles ? take : 0;
        w.piece = off > 0;
        w.splits = take == weight ? 1 : 2;
        w.part = 2 * s.rank + (off == 0);
        return true;
    }
    w.splits = tiles > pl.chunk ? min((tiles + pl.chunk - 1) / pl.chunk, pl.splits) : 1;
    const int per = (max(tiles, 0) + w.splits - 1) / w.splits;
    if (per > 0) w.splits = (tiles + per - 1) / per;
    if (split == 0 && lane == 0 && pl.head) pl.head[slot] = tiles < 0 ? make_int4(0, 0, 0, 0) : make_int4(w.splits, w.used, (int32_t)w.row0, slot * pl.splits);
    if (tiles < 0 || split >= w.splits) return false;
    w.tile0 = min(split * per, tiles);
    w.tiles = min(per, tiles - w.tile0);
    w.piece = split;
    w.part = slot * pl.splits + split;
    return true;
}

// First key of the unit's i-th tile, from the last keys to the first: where scores fall with the distance a row's maximum
// is then found in its first tiles (from the first keys on, every tile of a steep head moved it and rescaled O: 900 to 1200
// clocks per tile).
__device__ __forceinline__ int tile_key(const Unit &w, int i)
{
    const int t = w.tile0 + w.tiles - 1 - i;
    return t < w.prefix_tiles ? t * kKeys : w.b0 + (t - w.prefix_tiles) * kKeys;
}

// The order of the products, and of the copies for them, over all units: S of a tile comes kAhead - 1 tiles before its
// O += P V, so that the softmax has two tiles in hand while the tensor cores work (with one the two waited for each other:
// half a softmax more per tile), across the ends of units too.  The first S of a unit comes behind the last but one O += P V
// of the unit before, when its Q has had the time to land.
struct Order {
    int k = 0, k_tiles = 0, v = 0, v_tiles = 0, later = 0;   // next tile and tiles of the units of S and of O; tiles of the unit after O's
    int units = 0, done = 0, ahead = 0;                      // units that S has entered and that O has left; tiles between the two
    bool over = false;
    __device__ bool at_new_unit() const { return k == k_tiles; }
    __device__ bool wants_scores() const
    {
        if (k < k_tiles) return ahead < kAhead;
        return !over && ahead < 2 && units - done <= 1;
    }
    __device__ void end() { over = true; }
    __device__ void enter(int tiles)
    {
        k = 0;
        k_tiles = tiles;
        if (units == done) v_tiles = tiles;
        else later = tiles;
        ++units;
    }
    __device__ void scores_done() { ++k, ++ahead; }
    __device__ void output_done()
    {
        --ahead;
        if (++v == v_tiles) {
            v = 0;
            v_tiles = later;
            ++done;
        }
    }
};

template <bool kBf16>
__device__ __forceinline__ uint32_t pack(float x, float y)
{
    if constexpr (kBf16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
    const __half2 v = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// The 128 softmax threads that share rows [0, 32) (0) or [32, 64) (1) meet; true if any of them says so.
__device__ __forceinline__ bool rows_meet_any(int who, bool yes)
{
    uint32_t any;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %2, 0;\n\tbar.red.or.pred p, %1, 128, q;\n\tselp.u32 %0, 1, 0, p;\n\t}\n"
                 : "=r"(any)
                 : "r"(1 + who), "r"(yes ? 1u : 0u)
                 : "memory");
    return any != 0;
}

template <uint32_t kBytes>
using Bytes = std::integral_constant<uint32_t, kBytes>;

// two fp32 operations at once
__device__ __forceinline__ uint64_t pair_bits(float2 v) { return static_cast<uint64_t>(__float_as_uint(v.y)) << 32 | __float_as_uint(v.x); }
__device__ __forceinline__ float2 pair_of(uint64_t b)
{
    return make_float2(__uint_as_float(static_cast<uint32_t>(b)), __uint_as_float(static_cast<uint32_t>(b >> 32)));
}
__device__ __forceinline__ float2 mul2(float2 x, float2 y)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pair_bits(x)), "l"(pair_bits(y)));
    return pair_of(r);
}
__device__ __forceinline__ float2 mul2(float2 x, float y) { return mul2(x, make_float2(y, y)); }
__device__ __forceinline__ float2 add2(float2 x, float2 y)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pair_bits(x)), "l"(pair_bits(y)));
    return pair_of(r);
}
__device__ __forceinline__ float2 add2(float2 x, float y) { return add2(x, make_float2(y, y)); }
__device__ __forceinline__ float2 fma2(float2 x, float2 y, float z)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(pair_bits(x)), "l"(pair_bits(y)), "l"(pair_bits(make_float2(z, z))));
    return pair_of(r);
}

// Hidden keys, blocks outside the cache and drafted keys are rare among a call's tiles: their code is kept away from the
// softmax's loop, which is long enough (with it in between, the jumps over it took 300 clocks per tile)
#define SFM_RARELY(x) __builtin_expect(!!(x), 0)

// cap tanh z of a row's 32 products with z = to_z * product.  For |z| <= 1, tanh z = z P(z^2) with the polynomial of degree 5
// that interpolates tanh(sqrt u) / sqrt u at the Chebyshev nodes of [0, 1] (off by 4.8e-7); tanh z = 1 - 2 / (e^2z + 1) for
// larger ones, and for five pairs of the sixteen anyway: the exponentials and quotients of these run beside the
// multiplications of the others (all by the second form, the scores of a tile took 1300 clocks; all by the first, 900).
// The second form is off by up to 2^-21 of the cap, however small the score is: 6e-5 at kWideCap, an eighth of an fp16 weight's
// half step.  Larger caps have a kernel of their own, which takes it for |z| > 1 alone (4096 causal tokens of 64 heads, bf16:
// 751 us with a cap of 30, 880 with one of 129, 1136 where many scores are larger than that).
constexpr float kWideCap = 128.f;
enum CapKind { kNoCap, kSmallCap, kLargeCap };

__device__ __forceinline__ float2 tanh_ratio(float2 u)
{
    float2 p = fma2(u, make_float2(-3.080409251e-03f, -3.080409251e-03f), 1.677677624e-02f);
    p = fma2(p, u, -5.163545866e-02f);
    p = fma2(p, u, 1.328251381e-01f);
    p = fma2(p, u, -3.332918032e-01f);
    return fma2(p, u, 9.999994421e-01f);
}

__device__ __forceinline__ float2 cap_wide(float2 z, float cap)
{
    const float2 t = mul2(z, 2.f * kLog2e);
    return make_float2(fmaf(__fdividef(-2.f, fast_exp2(t.x) + 1.f), cap, cap), fmaf(__fdividef(-2.f, fast_exp2(t.y) + 1.f), cap, cap));
}

// The latter form too where some row does not see all its keys: what it does not see does not choose the form, and so has no
// part in the last bits of others.  (To leave such keys out of the search for large ones made trees of 61 tokens 5 to 9 % slower.)
__device__ __forceinline__ void cap_scores(float2 (&y)[16], float to_z, float cap, bool all)
{
    float far = 0.f;
#pragma unroll
    for (int c = 0; c < 16; ++c) {
        y[c] = mul2(y[c], to_z);
        if (c < 11) far = fmaxf(far, fmaxf(fabsf(y[c].x), fabsf(y[c].y)));
    }
    if (!SFM_RARELY(!__all_sync(0xffffffffu, all && far <= 1.f))) {
#pragma unroll
        for (int c = 0; c < 16; ++c) {
            // (in the order in which the two kinds go out side by side)
            const int k = c % 3 == 2 ? 11 + c / 3 : c - c / 3;
            if (k >= 11) {
                y[k] = cap_wide(y[k], cap);
            } else {
                const float2 p = tanh_ratio(mul2(y[k], y[k]));
                y[k] = mul2(mul2(y[k], cap), p);
            }
        }
    } else {
#pragma unroll
        for (int c = 0; c < 16; ++c) y[c] = cap_wide(y[c], cap);
    }
}

// The same for caps above kWideCap: a score x = to_x * product is x P(z^2) for |z| <= 1, off in proportion to itself (and not
// to the cap, also where z is too small for fp32), whatever its neighbours are.
__device__ __forceinline__ void cap_scores_each(float2 (&y)[16], float to_z, float to_x, float cap)
{
    float far = 0.f;
#pragma unroll
    for (int c = 0; c < 16; ++c) far = fmaxf(far, fmaxf(fabsf(y[c].x), fabsf(y[c].y)));
    const bool some = __any_sync(0xffffffffu, far * fabsf(to_z) > 1.f);
#pragma unroll
    for (int c = 0; c < 16; ++c) {
        const float2 z = mul2(y[c], to_z);
        float2 x = mul2(mul2(y[c], to_x), tanh_ratio(mul2(z, z)));
        if (SFM_RARELY(some)) {
            const float2 t = cap_wide(z, cap);
            if (!(fabsf(z.x) <= 1.f)) x.x = t.x;
            if (!(fabsf(z.y) <= 1.f)) x.y = t.y;
        }
        y[c] = x;
    }
}

// 1 / (l + 2^(sink - m)), also where the sink lies so far above m that the power, or the quotient, leaves fp32's normal range
// (what is left of such a row is small, but values of the type).
__device__ __forceinline__ float beside_sink(float l, float m, float sink)
{
    const float top = fmaxf(m, sink), e = fast_exp2(0.5f * (m - top));
    return __fdividef(e, fmaf(l, e * e, sink >= m ? 1.f : fast_exp2(sink - m))) * e;
}

// 16 lanes x 64 columns of tensor memory: thread t gets of every eight columns 8 i the columns 8 i + 2 (t % 4) and the one
// behind it, of lane t / 4 in r[4 i], r[4 i + 1] and of lane t / 4 + 8 in r[4 i + 2], r[4 i + 3].
__device__ __forceinline__ void tmem_ld_quads(uint32_t taddr, uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}

// Thread q of four holds words 4 i + q (i = 0..7) of 32; afterwards words 8 q + i.
__device__ __forceinline__ void gather_quad(uint32_t (&w)[8], int lane)
{
    uint32_t a[8];
    // threads q and q ^ 2: the lower two take words of i < 4, the upper two the others; a[2 i], a[2 i + 1]: from the lower, the upper
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool up = lane & 2;
        const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? w[i] : w[i + 4], 2), own = up ? w[i + 4] : w[i];
        a[2 * i] = up ? got : own;
        a[2 * i + 1] = up ? own : got;
    }
    // threads q and q ^ 1: i of 0, 1 or of 2, 3
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const bool up = lane & 1;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? a[2 * i + k] : a[2 * i + 4 + k], 1), own = up ? a[2 * i + 4 + k] : a[2 * i + k];
            w[4 * i + 2 * k] = up ? got : own;
            w[4 * i + 2 * k + 1] = up ? own : got;
        }
    }
}

// 32 bytes, one sector of memory, at once where they are aligned to that
__device__ __forceinline__ void store32(void *to, const uint32_t *v, bool wide)
{
    if (!wide) {
        static_cast<uint4 *>(to)[0] = make_uint4(v[0], v[1], v[2], v[3]);
        static_cast<uint4 *>(to)[1] = make_uint4(v[4], v[5], v[6], v[7]);
        return;
    }
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
                 "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

template <bool kBf16, int kCap, bool kBias>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
sfm_dense_kernel(const __grid_constant__ DenseArgs a, const __grid_constant__ Plan pl, const __grid_constant__ CUtensorMap q_map,
                 const __grid_constant__ CUtensorMap kv_map)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    uint32_t sb = smem_u32(smem);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const uint32_t rank = cluster_rank();
    uint8_t *const misc = smem + MISC_OFF;
    volatile int *const abort_flag = reinterpret_cast<volatile int *>(misc + ABORT_REL);
    volatile int *const beat = reinterpret_cast<volatile int *>(misc + BEAT_REL);
    float *const exch = reinterpret_cast<float *>(misc + EXCH_REL);
    volatile uint32_t *const cand_words = reinterpret_cast<volatile uint32_t *>(misc + CAND_REL);
    volatile uint32_t *const fix_words = reinterpret_cast<volatile uint32_t *>(misc + FIX_REL);
    const int cluster = blockIdx.x >> 1, clusters = gridDim.x >> 1;

    if (warp == 0) {
        prefetch_map(&q_map);
        prefetch_map(&kv_map);
    }
    if (tid == 0) {
        auto init = [&](int i, int n) { mbar_init(sb + MISC_OFF + 8u * i, n); };
        for (int i = 0; i < kStages; ++i) {
            init(B_KV_FULL + i, 1);
            init(B_KV_EMPTY + i, 1);
        }
        init(B_Q_FULL, 1);
        init(B_Q_EMPTY, 1);
        for (int i = 0; i < 4; ++i) init(B_S_FULL + i, 1);
        for (int i = 0; i < 2; ++i) {
            init(B_P_FULL + i, 16);
            init(B_O_DONE + i, 1);
        }
        for (int i = 0; i < kUnits; ++i) {
            init(B_UNIT_FULL + i, 1);
            init(B_CHECKED + i, 1);
            init(B_UNIT_EMPTY + i, rank == 0 ? 10 : 9);
        }
        init(B_O_FREE, 16);
        init(B_FIX, 1);
        init(B_FIXED, 2);
        init(B_END, 1);
        for (int i = 0; i < 8; ++i) cand_words[i] = fix_words[i] = 0;
        *abort_flag = 0;
        *beat = 0;
        fence_barrier_init();
    }
    if (warp == 2) pair_alloc(sb + MISC_OFF + TMEM_REL, kTmemCols);
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t *>(misc + TMEM_REL), 0);
    sb = __shfl_sync(0xffffffffu, sb, 0);
    const uint32_t bar0 = sb + MISC_OFF;
    auto bar = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
    const uint32_t first0 = in_cta(bar0, 0);
    auto first_bar = [&](int i) { return first0 + 8u * static_cast<uint32_t>(i); };
    Unit *const units = reinterpret_cast<Unit *>(misc + UNIT_REL);
    grid_follow();
    DenseSeq *const seqs = reinterpret_cast<DenseSeq *>(smem + KV_OFF);
    Balance &balance = *reinterpret_cast<Balance *>(smem + P_OFF);
    bool falls = false;                       // balanced: offsets of q fall somewhere
    if (pl.balanced) {
        // the batch's sequences, then every slot's weight, then the pairs' parts (copies come and P goes here once there is a unit)
        for (int i = tid; i < a.batch; i += kThreads) seqs[i] = dense_seq(a, i);
        __syncthreads();
        for (int i = tid; i < pl.slots; i += kThreads) balance.before[i] = slot_weight(a, pl, i, seqs, balance.row0[i], balance.used[i]);
        for (int i = tid + 1; i < a.batch; i += kThreads) falls |= seqs[i].q0 < seqs[i - 1].q0;
        falls = __syncthreads_or(falls);
        if (warp == 3) make_balance(pl, balance, lane);
        fence_proxy_async_smem();
        __syncthreads();
        // what the joining of pieces has to know: at most one slot begins in a part and goes on behind it
        if (tid == 0 && rank == 0) {
            const int begin = balance.begin[cluster], end = balance.begin[cluster + 1], n = balance.rank[cluster];
            int4 head = make_int4(0, 0, 0, 0);
            if (end > begin) {
                const int base = balance.before[min(balance.waves * pl.pairs, pl.slots)];
                const int i = last_at_most(balance.before, pl.slots, base + end - 1), last = balance.before[i + 1] - base;
                if (balance.before[i] - base >= begin && last > end)
                    head = make_int4(balance.rank[last_at_most(balance.begin, pl.pairs, last - 1)] - n + 1, balance.used[i], balance.row0[i], n);
            }
            pl.head[end > begin ? n : balance.rank[pl.pairs] + cluster - n] = head;
        }
        __syncthreads();
    }

    // a wait that may take a whole unit, which has no longest time: it ends when no tile has gone by for some time
    auto wait_as_long_as_tiles_go_by = [&](uint32_t bar, uint32_t parity) {
        uint64_t t0 = globaltimer_ns();
        int seen = *beat;
        while (!__all_sync(0xffffffffu, pair_try_wait(bar, parity))) {
            bool ok = true;
            if (lane == 0) {
                if (*beat != seen) {
                    seen = *beat;
                    t0 = globaltimer_ns();
                } else if (globaltimer_ns() - t0 > 2 * kTimeoutNs) {
                    *abort_flag = 1;
                }
                ok = !*abort_flag;
            }
            if (!__shfl_sync(0xffffffffu, ok ? 1 : 0, 0)) return false;
        }
        return true;
    };

    if (warp == 3) {
        // ======================= units =======================
        int n = 0;
        Share share = {};
        if (pl.balanced) share = make_share(pl, balance, cluster);
        for (int u = cluster;; u += clusters) {
            Unit w;
            w.bad = 0;
            const bool end = pl.balanced ? share.wave >= share.waves && (share.at >= share.end || share.slot >= pl.slots) : u >= pl.units;
            if (end) w.valid = 0;
            else if (!make_unit(a, pl, share, u, cluster, lane, w, pl.balanced && n == 0 ? seqs : nullptr, falls)) continue;
            const int slot = n % kUnits;
            if (n >= kUnits && !wait_as_long_as_tiles_go_by(bar(B_UNIT_EMPTY + slot), n / kUnits - 1 & 1)) break;
            if (lane == 0) {
                units[slot] = w;
                mbar_arrive(bar(B_UNIT_FULL + slot));
            }
            // the copies and products may begin, the softmax waits for this too
            if (!end) check_blocks(a, w, lane);
            if (lane == 0) {
                units[slot].bad = w.bad;
                mbar_arrive(bar(B_CHECKED + slot));
            }
            __syncwarp();
            ++n;
            if (end) break;
        }
        if (!pl.balanced && a.cu_q && blockIdx.x == 0) {
            // offsets that fall, also where no slot leads to the sequence (the balanced plan has looked at all)
            bool bad = false;
            for (int i = lane; i < a.batch; i += 32) bad |= __ldg(a.cu_q + i + 1) < __ldg(a.cu_q + i);
            if (__any_sync(0xffffffffu, bad) && lane == 0) dense_status(a, SFM_STATUS_BAD_LENGTH);
        }
    } else if (warp == 0) {
        // ======================= copies =======================
        const int boxes = 64 / pl.box_rows;        // per block
        const bool paged = a.layout_kv == SFM_LAYOUT_PAGED;
        int n = 0, c = 0;                          // units, stages
        Order o;
        Unit wk = {};                                   // the unit of the next K
        bool ok = true;
        // lane l looks after the box of keys [l box_rows, (l + 1) box_rows) of a tile: its page's id is under way a tile
        // before it is needed
        auto page_of = [&](int i) {
            const int j = i < wk.tiles ? tile_key(wk, i) + lane * pl.box_rows : wk.len;
            const bool real = paged && lane < 2 * boxes && j < wk.len;
            return real ? __ldg(a.table + (int64_t)wk.b * a.cols + fdiv((uint32_t)j, a.block_div)) : 0;
        };
        auto row_of = [&](int i, int32_t id) {
            const int j = tile_key(wk, i) + lane * pl.box_rows;
            if (j >= wk.len) return (int32_t)a.kv_rows;
            if (!paged) return (int32_t)(wk.kv0 + j);
            if (id < 0 || ((int64_t)id + 1) * a.block > a.kv_rows) return (int32_t)a.kv_rows;
            return id * a.block + (j - (int)fdiv((uint32_t)j, a.block_div) * a.block);
        };
        auto stage = [&](int block, int half, int32_t row) {
            const int st = c & (kStages - 1), use = c / kStages;
            ++c;
            if (use > 0 && !pair_wait_warp(bar(B_KV_EMPTY + st), use - 1 & 1, abort_flag)) return false;
            const uint32_t dst = sb + KV_OFF + st * kStageBytes;
            if (!SFM_RARELY(boxes != 1)) {
                const int y = __shfl_sync(0xffffffffu, row, half);
                if (elect_one()) {
                    if (rank == 0) expect_tx(bar(B_KV_FULL + st), 2 * kStageBytes);
                    pair_load(dst, &kv_map, 0, y, block, first_bar(B_KV_FULL + st));
                }
            } else {
                // pages of 16 or 32 rows (or a multiple that has no 64): a copy each, eight rows of the four blocks after eight rows
                int y[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) y[k] = __shfl_sync(0xffffffffu, row, half * boxes + k & 31) >> 3;
                if (elect_one()) {
                    if (rank == 0) expect_tx(bar(B_KV_FULL + st), 2 * kStageBytes);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (k < boxes) pair_load_octets(dst + k * pl.box_rows * 512u, &kv_map, block, y[k], first_bar(B_KV_FULL + st));
                }
            }
            __syncwarp();
            return true;
        };
        // rows of the tiles whose K is copied and V is not yet: their V's copies find them in L2
        int32_t row0 = 0, row1 = 0, row2 = 0, page = 0;
        auto next_unit = [&]() -> int {            // tiles of the next unit with keys, 0 at the end, -1 on a timeout
            for (;;) {
                const int us = n % kUnits;
                if (!pair_wait_warp(bar(B_UNIT_FULL + us), n / kUnits & 1, abort_flag)) return -1;
                wk = units[us];
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_UNIT_EMPTY + us));
                ++n;
                if (!wk.valid) return 0;
                if (wk.tiles) return wk.tiles;
            }
        };
        while (ok) {
            while (ok && o.wants_scores()) {
                if (o.at_new_unit()) {
                    const int tiles = next_unit();
                    if (tiles <= 0) {
                        o.end();
                        ok = tiles == 0;
                        break;
                    }
                    o.enter(tiles);
                    if (o.units > 1 && !pair_wait_warp(bar(B_Q_EMPTY), o.units - 2 & 1, abort_flag)) {
                        ok = false;
                        break;
                    }
                    if (elect_one()) {
                        if (rank == 0) expect_tx(bar(B_Q_FULL), 2 * 65536);
                        pair_load(sb + Q_OFF, &q_map, 0, (int)wk.row0 + 64 * (int)rank, 0, first_bar(B_Q_FULL));
                    }
                    __syncwarp();
                    page = page_of(0);
                }
                const int32_t row = row_of(o.k, page);
                page = page_of(o.k + 1);
                if (o.ahead == 0) row0 = row;
                else if (o.ahead == 1) row1 = row;
                else row2 = row;
                for (int k = 0; k < kSteps && ok; ++k) ok = stage(kBlocks * k, (int)rank, row);
                o.scores_done();
            }
            if (!ok || o.ahead == 0) break;
            for (int k = 0; k < kSteps && ok; ++k) ok = stage(4 * (int)rank + (k >> 1) * kBlocks, k & 1, row0);
            row0 = row1;
            row1 = row2;
            o.output_done();
        }
        // The products' last arrivals at this CTA's barriers: none may be on its way when the CTA ends.  (S's are waited for by
        // the softmax, all of them.)
        const int tiles = c / (2 * kSteps);
        for (int i = max(c - kStages, 0); i < c && ok; ++i) ok = pair_wait_warp(bar(B_KV_EMPTY + (i & (kStages - 1))), i / kStages & 1, abort_flag);
        for (int i = max(tiles - 2, 0); i < tiles && ok; ++i) ok = pair_wait_warp(bar(B_O_DONE + (i & 1)), i >> 1 & 1, abort_flag);
        if (ok && o.units > 0) pair_wait_warp(bar(B_Q_EMPTY), o.units - 1 & 1, abort_flag);
    } else if (warp == 1) {
        // ======================= products =======================
        if (rank == 0) {
            int n = 0, c = 0, gk = 0, gv = 0, fixes = 0;      // units, stages, tiles of S and of O
            bool ok = true;
            Order o;
            const uint32_t id_s = pl.idesc_s, id_o = pl.idesc_o;
            const Desc q_desc = desc_sw128(sb + Q_OFF, 16, 1024), p_desc = desc_sw128(sb + P_OFF, 16, 1024);
            auto landed = [&](int k) { return pair_wait_warp(bar(B_KV_FULL + (k & (kStages - 1))), k / kStages & 1, abort_flag); };
            auto next_unit = [&]() -> int {
                for (;;) {
                    const int us = n % kUnits;
                    if (!pair_wait_warp(bar(B_UNIT_FULL + us), n / kUnits & 1, abort_flag)) return -1;
                    const int valid = __shfl_sync(0xffffffffu, units[us].valid, 0), tiles = __shfl_sync(0xffffffffu, units[us].tiles, 0);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(B_UNIT_EMPTY + us));
                    ++n;
                    if (!valid) return 0;
                    if (tiles) return tiles;
                }
            };
            // (twice, for the two ways in which keys lie in a stage: distances that the kernel has to add up made prompts a tenth slower)
            auto multiply = [&](auto block_bytes, auto octet_bytes) {
                constexpr uint32_t block = decltype(block_bytes)::value, octet = decltype(octet_bytes)::value;
                const Desc k_desc = desc_sw128(sb + KV_OFF, 16, octet), v_desc = desc_sw128(sb + KV_OFF, block, octet);
                while (ok) {
                    while (ok && o.wants_scores()) {
                        if (o.at_new_unit()) {
                            const int tiles = next_unit();
                            if (tiles <= 0) {
                                o.end();
                                ok = tiles == 0;
                                break;
                            }
                            o.enter(tiles);
                            ok = pair_wait_warp(bar(B_Q_FULL), o.units - 1 & 1, abort_flag);
                        }
                        const uint32_t d = tmem + TM_S + (gk & 3) * 64;
    #pragma unroll
                        for (int k = 0; k < kSteps; ++k) {
                            const uint32_t st = c & (kStages - 1);
                            ok = ok && landed(c);
                            ++c;
                            tc_fence_after();
                            if (ok && elect_one()) {
                                const Desc kd = {k_desc.lo + st * (kStageBytes >> 4), k_desc.hi};
    #pragma unroll
                                for (int j = 0; j < 4 * kBlocks; ++j) {
                                    const uint32_t sub = (j & 3) * 32u;
                                    pair_mma(d, desc_at(q_desc, k * kStageBytes + (j >> 2) * 8192u + sub), desc_at(kd, (j >> 2) * block + sub), id_s, (k | j) > 0);
                                }
                                pair_commit(bar(B_KV_EMPTY + st));
                                if (k == kSteps - 1) {
                                    pair_commit(bar(B_S_FULL + (gk & 3)));
                                    if (o.k + 1 == o.k_tiles) pair_commit(bar(B_Q_EMPTY));
                                }
                            }
                            __syncwarp();
                        }
                        ++gk;
                        o.scores_done();
                    }
                    if (!ok || o.ahead == 0) break;
                    const int buf = gv & 1;
                    ok = pair_wait_warp(bar(B_P_FULL + buf), gv >> 1 & 1, abort_flag);
                    if (o.v == 0 && o.done > 0) ok = ok && pair_wait_warp(bar(B_O_FREE), o.done - 1 & 1, abort_flag);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t found = lane < 4 ? cand_words[4 * buf + lane] : 0u;
                    if (__any_sync(0xffffffffu, found != 0)) {
                        // the staged V, made finite in both CTAs before it is used
                        for (int k = 0; k < kSteps && ok; ++k) ok = landed(c + k);
                        if (!ok) break;
                        for (uint32_t r = 0; r < 2; ++r) {
                            const uint32_t to = in_cta(bar0 + FIX_REL, r);
                            if (lane < 4) store_remote(to + 4 * lane, found);
                            if (lane == 4) store_remote(to + 16, (uint32_t)c & (kStages - 1));
                        }
                        if (lane < 4) cand_words[4 * buf + lane] = 0;
                        __syncwarp();
                        if (lane < 2) arrive_remote_release(in_cta(bar(B_FIX), lane));
                        __syncwarp();
                        ok = pair_wait_warp(bar(B_FIXED), fixes & 1, abort_flag);
                        ++fixes;
                        if (!ok) break;
                        fence_proxy_async_smem();
                    }
    #pragma unroll
                    for (int k = 0; k < kSteps; ++k) {
                        const uint32_t st = c & (kStages - 1);
                        ok = ok && landed(c);
                        ++c;
                        tc_fence_after();
                        if (ok && elect_one()) {
                            const Desc pd = {p_desc.lo + buf * (16384u >> 4), p_desc.hi}, vd = {v_desc.lo + st * (kStageBytes >> 4), v_desc.hi};
    #pragma unroll
                            for (int j = 0; j < 2 * kBlocks; ++j)        // columns of the stage, 16 keys of its 64
                                pair_mma(tmem + TM_O + ((k >> 1) * kBlocks / 2 + (j >> 2)) * 128, desc_at(pd, (k & 1) * 8192u + (j & 3) * 32u),
                                         desc_at(vd, (j >> 2) * 2 * block + (j & 3) * 2 * octet), id_o, o.v > 0 || (k & 1) || (j & 3) > 0);
                            pair_commit(bar(B_KV_EMPTY + st));
                            if (k == kSteps - 1) pair_commit(bar(B_O_DONE + buf));
                        }
                        __syncwarp();
                    }
                    ++gv;
                    o.output_done();
                }
            };
            if (SFM_RARELY(pl.octet_bytes != 1024)) multiply(Bytes<1024>(), Bytes<4096>());
            else multiply(Bytes<8192>(), Bytes<1024>());
            // no more rows to be made finite
            if (lane < 2) {
                store_remote(in_cta(bar0 + FIX_REL, lane) + 20, 1u);
                arrive_remote_release(in_cta(bar(B_FIX), lane));
            }
            __syncwarp();
            if (!ok) {
                // (the softmax has waited for all products otherwise) nothing is under way when tensor memory is freed
                if (elect_one()) pair_commit(bar(B_END));
                __syncwarp();
                const uint64_t t0 = globaltimer_ns();
                while (!pair_try_wait(bar(B_END), 0) && globaltimer_ns() - t0 < kTimeoutNs) {
                }
            }
        }
        __syncwarp();
    } else if (warp == 2) {
        // ======================= V rows made finite =======================
        for (int n = 0;;) {
            if (!wait_as_long_as_tiles_go_by(bar(B_FIX), n & 1)) break;
            ++n;
            if (fix_words[5]) break;
            const uint16_t inf = kBf16 ? 0x7f80 : 0x7c00;
            for (int q4 = 0; q4 < 4; ++q4) {
                uint32_t m = fix_words[q4];
                while (m) {
                    const int key = 32 * q4 + __ffs(m) - 1;
                    m &= m - 1;
                    // the key's 256 values in this CTA: four blocks, 128 bytes each, in the stages of its half of the keys
                    for (int q = 0; q < 4; ++q) {
                        const uint32_t st = fix_words[4] + q / kBlocks * 2 + (key >> 6) & (kStages - 1);
                        uint16_t *row = reinterpret_cast<uint16_t *>(smem + KV_OFF + st * kStageBytes + q % kBlocks * pl.block_bytes + (key >> 3 & 7) * pl.octet_bytes + (key & 7) * 128);
                        for (int k = lane; k < 64; k += 32)
                            if ((row[k] & inf) == inf) row[k] = 0;
                    }
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) arrive_remote_release(first_bar(B_FIXED));
        }
    } else {
        // ======================= softmax =======================
        const int part = (warp - 4) & 3, wg = (warp - 4) >> 2;
        const int r = (part & 1) * 32 + lane, half = part >> 1;     // row; keys and columns of O in halves
        const uint32_t lanes = static_cast<uint32_t>(part * 32) << 16;
        const int quarter = half * 2 + wg, c0 = half * 64 + wg * 32;      // this thread's keys of a tile: [c0, c0 + 32)
        const float sl2 = a.scale * kLog2e, cap2 = a.cap * kLog2e;
        const bool wide = (reinterpret_cast<uintptr_t>(a.out) & 31u) == 0;
        uint8_t *const p_row = smem + P_OFF + half * 8192;
        if (a.zero_rest && a.cu_q) {
            // rows of no sequence
            const int64_t lo = (int64_t)min(max(__ldg(a.cu_q), 0), a.total_q) * a.heads,
                          hi = (int64_t)min(max(__ldg(a.cu_q + a.batch), 0), a.total_q) * a.heads, all = (int64_t)a.total_q * a.heads;
            const int64_t rest = lo + max(all - max(hi, lo), (int64_t)0);
            for (int64_t i = (int64_t)blockIdx.x * 256 + (tid - 128); i < rest * 64; i += (int64_t)gridDim.x * 256) {
                const int64_t k = i >> 6, row = k < lo ? k : max(hi, lo) + (k - lo);
                if (a.zero_rest & 1) reinterpret_cast<uint4 *>(a.out)[row * 64 + (i & 63)] = make_uint4(0, 0, 0, 0);
                if (a.zero_rest & 2 && a.lse && (i & 63) == 0) a.lse[row] = -INFINITY;
            }
        }
        int n = 0, g = 0, ex = 0;
        bool ok = true;
        // a row's four values, through shared memory (a role that gave up ends the loops of all of them at the same place)
        auto row_values = [&](float v, float (&got)[4]) {
            float *e = exch + (ex & 1) * 256;
            ++ex;
            e[quarter * 64 + r] = v;
            ok = !rows_meet_any(part & 1, !ok);
#pragma unroll
            for (int k = 0; k < 4; ++k) got[k] = e[k * 64 + r];
        };
        // A unit's O is written after the first tile of the unit behind it, which the tensor cores wait for: what is needed then
        struct {
            bool any, out, parts;      // a unit is left; this row is written to the outputs, or to the workspace
            int last;                  // its last tile
            float inv;
            void *to;                  // this thread's 128 columns
        } left = {false, false, false, 0, 0.f, nullptr};
        auto write_left = [&]() {
            if (!left.any) return;
            left.any = false;
            if (ok) ok = pair_wait_warp(bar(B_O_DONE + (left.last & 1)), left.last >> 1 & 1, abort_flag);
            tc_fence_after();
            const uint32_t from = tmem + lanes + TM_O + wg * 128;
            if (__any_sync(0xffffffffu, left.parts)) {
#pragma unroll 1
                for (int c = 0; c < 128; c += 32) {
                    uint32_t o[32];
                    tmem_ld32(from + c, o);
                    tmem_wait_ld();
                    if (left.parts)
#pragma unroll
                        for (int k = 0; k < 32; k += 8) store32(static_cast<float *>(left.to) + c + k, o + k, true);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_remote(first_bar(B_O_FREE));
            } else {
                // Four threads per row, so that a store writes 128 bytes of each of eight rows.  A loop with a small body:
                // this code runs once per unit, and unrolled it took 3000 clocks to be fetched.
                const uint32_t rows_out = __ballot_sync(0xffffffffu, left.out), rows_none = __ballot_sync(0xffffffffu, left.inv == 0.f);
                // the warp's first row; rows lie 512 values apart
                uint16_t *const top = reinterpret_cast<uint16_t *>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(left.to), 0));
#pragma unroll 1
                for (int q = 0; q < 4; ++q) {
                    // 16 rows, 64 columns
                    const int h = q & 1, c = q >> 1;
                    uint32_t o[32];
                    tmem_ld_quads(from + c * 64 + (static_cast<uint32_t>(16 * h) << 16), o);
                    tmem_wait_ld();
                    if (q == 3) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) arrive_remote(first_bar(B_O_FREE));
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int rr = 16 * h + 8 * e + (lane >> 2);
                        const float inv = __shfl_sync(0xffffffffu, left.inv, rr);
                        uint32_t v[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            v[i] = pack<kBf16>(__uint_as_float(o[4 * i + 2 * e]) * inv, __uint_as_float(o[4 * i + 2 * e + 1]) * inv);
                        gather_quad(v, lane);
                        if (rows_none >> rr & 1)
#pragma unroll
                            for (int i = 0; i < 8; ++i) v[i] = 0u;
                        if (rows_out >> rr & 1) store32(top + rr * kD + 64 * c + 16 * (lane & 3), v, wide);
                    }
                }
            }
        };
        while (ok) {
            const int us = n % kUnits;
            if (rows_meet_any(part & 1, !pair_wait_warp(bar(B_CHECKED + us), n / kUnits & 1, abort_flag))) {
                ok = false;
                break;
            }
            const Unit w = units[us];
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_UNIT_EMPTY + us));
            ++n;
            if (!w.valid) break;
            const int R = 64 * (int)rank + r;
            const bool live = R < w.used;
            const int hr = w.h0 + R, di = (int)fdiv((uint32_t)hr, a.heads_div), i_q = w.i0 + di, head = hr - di * a.heads;
            DenseRow row = {0, 0, INT32_MAX};        // rows that do not count see all: nothing to mask
            const uint64_t *tree = nullptr;
            const int first = w.len - w.q_len;
            float slope = 0.f;
            if (live) {
                DenseSeq s;
                s.q0 = w.q0;
                s.q_len = w.q_len;
                s.len = w.len;
                row = dense_row(a, s, i_q);
                if (a.words) tree = a.tree + (int64_t)(w.q0 + i_q) * a.words;
                if constexpr (kBias) slope = __ldg(a.slopes + head) * kLog2e;
            }
            const float to_z = kCap && live ? a.scale / a.cap : 0.f;       // (rows that do not count do not choose the cap's form)
            const float to_x = live ? sl2 : 0.f;
            float m = -INFINITY;
            float2 sum = make_float2(0.f, 0.f);
            for (int i = 0; i < w.tiles; ++i) {
                const int gi = g + i, buf = gi & 1, j0 = tile_key(w, i) + c0;
                // what this row sees of its 32 keys
                uint32_t vis = bits_between(row.lo, row.hi, j0);
                if (live) {
                    vis |= bits_between(0, w.prefix, j0);
                    if (SFM_RARELY(tree && j0 + 32 > first && j0 < w.len)) {
                        // drafted keys: bits [j0 - first, j0 - first + 32) of the mask
                        const int o = j0 - first;
                        uint32_t bits;
                        if (o >= 0) {
                            const int word = o >> 6, sh = o & 63;
                            const uint64_t x0 = word < a.words ? __ldg(tree + word) : 0, x1 = word + 1 < a.words ? __ldg(tree + word + 1) : 0;
                            bits = (uint32_t)(sh ? x0 >> sh | x1 << (64 - sh) : x0);
                        } else {
                            bits = (uint32_t)(__ldg(tree) << -o);
                        }
                        bits &= drafted_keys(first, w.len, j0);
                        if (a.mode == 4) {
                            for (uint32_t rest = bits; rest; rest &= rest - 1) {
                                const int c = __ffs(rest) - 1;
                                const int64_t pos = __ldg(a.positions + w.q0 + o + c);
                                if (pos < (int64_t)row.p - a.win_left || pos > (int64_t)row.p + a.win_right) bits &= ~(1u << c);
                            }
                        }
                        vis |= bits;
                    }
                    if (SFM_RARELY(w.bad)) {
                        bool bad = false, worse = false;
                        box_row(a, w.b, 0, w.len, j0, &bad);
                        box_row(a, w.b, 0, w.len, j0 + 16, &worse);
                        if (bad) vis &= 0xffff0000u;
                        if (worse) vis &= 0x0000ffffu;
                    }
                }
                // P's buffer is free once the O += P V that read it is done
                if (ok && gi >= 2) ok = pair_wait_warp(bar(B_O_DONE + buf), (gi >> 1) - 1 & 1, abort_flag);
                ok = ok && pair_wait_warp(bar(B_S_FULL + (gi & 3)), gi >> 2 & 1, abort_flag);
                tc_fence_after();
                uint32_t raw[32];
                tmem_ld32(tmem + lanes + TM_S + (gi & 3) * 64 + wg * 32, raw);
                tmem_wait_ld();
                if (part == 0 && wg == 0 && lane == 0) *beat = gi;
                float2 y[16];
#pragma unroll
                for (int c = 0; c < 16; ++c) y[c] = make_float2(__uint_as_float(raw[2 * c]), __uint_as_float(raw[2 * c + 1]));
                if constexpr (kCap == kSmallCap) {
                    cap_scores(y, to_z, cap2, vis == 0xffffffffu);
                } else if constexpr (kCap == kLargeCap) {
                    cap_scores_each(y, to_z, to_x, cap2);
                } else {
#pragma unroll
                    for (int c = 0; c < 16; ++c) y[c] = mul2(y[c], sl2);
                }
                if constexpr (kBias) {
                    if (!SFM_RARELY(a.words && j0 + 31 >= first)) {
                        const float d0 = (float)(row.p - j0);
#pragma unroll
                        for (int c = 0; c < 16; ++c) {
                            y[c].x = fmaf(-slope, fabsf(d0 - (float)(2 * c)), y[c].x);
                            y[c].y = fmaf(-slope, fabsf(d0 - (float)(2 * c + 1)), y[c].y);
                        }
                    } else {
                        auto fall = [&](int c) {
                            // (a row that does not count masks nothing; of one that does, visible keys from `first` on are drafted_keys)
                            if (!live || !(vis >> c & 1)) return 0.f;
                            const int k = j0 + c - first;
                            return slope * fabsf((float)(row.p - (k < 0 ? j0 + c : __ldg(a.positions + w.q0 + k))));
                        };
#pragma unroll
                        for (int c = 0; c < 16; ++c) {
                            y[c].x -= fall(2 * c);
                            y[c].y -= fall(2 * c + 1);
                        }
                    }
                }
                if (SFM_RARELY(!__all_sync(0xffffffffu, vis == 0xffffffffu))) {
                    uint32_t odd = 0;
#pragma unroll
                    for (int c = 0; c < 32; ++c)
                        if (!(fabsf(__uint_as_float(raw[c])) < INFINITY)) odd |= 1u << c;
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        if (!(vis >> (2 * c) & 1)) y[c].x = -INFINITY;
                        if (!(vis >> (2 * c + 1) & 1)) y[c].y = -INFINITY;
                    }
                    odd = __reduce_or_sync(0xffffffffu, odd & ~vis);
                    if (odd && lane == 0) {
                        or_remote(first0 + CAND_REL + 16u * buf + 4u * quarter, odd);
                        fence_cluster();         // before this warp's arrival
                    }
                }
                float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < 16; ++c) tops[c & 3] = fmaxf(tops[c & 3], fmaxf(y[c].x, y[c].y));
                float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])), alpha = 1.f;
                // A row's four threads share their maxima only where one of them has left the range (or a role gave up)
                const bool beyond = top > m + kRescale || (m == -INFINITY && top != -INFINITY);
                if (SFM_RARELY(rows_meet_any(part & 1, beyond || !ok))) {
                    float got[4];
                    row_values(top, got);
                    if (!ok) break;
                    top = fmaxf(fmaxf(got[0], got[1]), fmaxf(got[2], got[3]));
                    if (top > m + kRescale || m == -INFINITY) {
                        if (m != -INFINITY) alpha = fast_exp2(m - top);
                        m = top;
                        sum.x *= alpha;
                        sum.y *= alpha;
                    }
                }
                const float back = m == -INFINITY ? 0.f : kLift<kBf16> - m;
                uint32_t pk[16];
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                    y[c] = add2(y[c], back);
                    y[c].x = fast_exp2(y[c].x);
                    y[c].y = fast_exp2(y[c].y);
                    pk[c] = pack<kBf16>(y[c].x, y[c].y);
                }
#pragma unroll
                for (int c = 0; c < 8; ++c) y[c] = add2(y[c], y[c + 8]);
#pragma unroll
                for (int c = 0; c < 4; ++c) y[c] = add2(y[c], y[c + 4]);
                sum = add2(sum, add2(add2(y[0], y[1]), add2(y[2], y[3])));
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    *reinterpret_cast<uint4 *>(p_row + buf * 16384 + sw128(r, wg * 4 + c)) =
                        make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
                if (SFM_RARELY(i > 0 && __any_sync(0xffffffffu, alpha != 1.f))) {
                    if (ok) ok = pair_wait_warp(bar(B_O_DONE + (buf ^ 1)), (gi - 1) >> 1 & 1, abort_flag);
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < 128; c += 32) {
                        tmem_ld32(tmem + lanes + TM_O + wg * 128 + c, raw);
                        tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < 32; ++k) raw[k] = __float_as_uint(__uint_as_float(raw[k]) * alpha);
                        tmem_st32(tmem + lanes + TM_O + wg * 128 + c, raw);
                    }
                    tmem_wait_st();
                }
                tc_fence_before();
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) arrive_remote(first_bar(B_P_FULL + buf));
                if (SFM_RARELY(i == 0)) write_left();
            }
            // the row's sum and LSE; its values come later (columns [256 half + 128 wg, + 128) of O)
            float got[4];
            row_values(sum.x + sum.y, got);
            if (!ok) break;
            const float l = (got[0] + got[1]) + (got[2] + got[3]);
            m -= kLift<kBf16>;
            const bool whole = w.splits == 1;
            const int64_t out_row = w.row0 + R;
            const bool empty = m == -INFINITY && l == 0.f;      // (a row of NaN has no maximum)
            float inv = 0.f;
            if (live && !empty) inv = a.sinks && whole ? beside_sink(l, m, __ldg(a.sinks + head) * kLog2e) : __fdividef(1.f, l);
            const int64_t part_row = (int64_t)w.part * kRows + R;
            const bool parts = live && !whole, out = !parts && R < w.rows && (live || w.piece == 0);
            if (quarter == 0) {
                if (parts) pl.part_ml[part_row] = make_float2(m, l);
                else if (out && a.lse) a.lse[out_row] = live && !empty ? (m + __log2f(l)) * kLn2 : -INFINITY;
            }
            const int col = 256 * half + 128 * wg;
            void *const to = parts ? static_cast<void *>(reinterpret_cast<float *>(pl.part_o) + part_row * kD + col)
                                   : static_cast<void *>(static_cast<uint16_t *>(a.out) + out_row * kD + col);
            // rows that do not count have no O: zeros now where others of the warp leave partial results, or no tile was
            if (out && (w.tiles == 0 || !whole)) {
                const uint32_t none[8] = {};
#pragma unroll
                for (int k = 0; k < 128; k += 16) store32(static_cast<uint16_t *>(to) + k, none, wide);
            }
            if (w.tiles > 0) {
                left.any = true;
                left.out = out && whole;
                left.parts = parts;
                left.last = g + w.tiles - 1;
                left.inv = inv;
                left.to = to;
                g += w.tiles;
            }
        }
        if (ok) write_left();
    }

    __syncwarp();
    if (*abort_flag) {
        // copies of a role that gave up may still be landing
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 2000000ull) __nanosleep(1000);
        if (tid == 0) dense_status(a, SFM_STATUS_TIMEOUT);
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    if (warp == 2) pair_dealloc(tmem, kTmemCols);
}

// Partial results of the pieces of a tile's keys, joined: a warp per row, four
// times four values per lane.
template <bool kBf16>
__global__ void __launch_bounds__(256) sfm_dense_join_kernel(const DenseArgs a, const Plan pl)
{
    grid_follow();
    const int r = (blockIdx.x & 15) * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int4 head = pl.head[blockIdx.x >> 4];
    if (head.x <= 1 || r >= head.y) return;
    // rows of the pieces' partial results
    auto row_of = [&](int s) { return (int64_t)(!pl.balanced ? head.w + s : s == 0 ? 2 * head.w + 1 : 2 * (head.w + s)) * kRows + r; };
    // the pieces' maxima and sums, 32 at a time
    float m = -INFINITY, l = 0.f;
    bool some = false;
    for (int s0 = 0; s0 < head.x; s0 += 32) {
        const float2 ml = s0 + lane < head.x ? pl.part_ml[row_of(s0 + lane)] : make_float2(-INFINITY, 0.f);
        float top = ml.x;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        m = fmaxf(m, top);
        some |= __any_sync(0xffffffffu, ml.x != -INFINITY || ml.y != 0.f);
    }
    const bool empty = !some;
    float4 o[4] = {};
#pragma unroll 2
    for (int s = 0; s < head.x; ++s) {
        const float2 ml = pl.part_ml[row_of(s)];
        const float4 *from = pl.part_o + row_of(s) * (kD / 4) + lane;
        float4 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = from[32 * k];
        if (ml.x == -INFINITY && ml.y == 0.f) continue;
        const float e = fast_exp2(ml.x - m);
        l = fmaf(e, ml.y, l);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            o[k].x = fmaf(e, v[k].x, o[k].x);
            o[k].y = fmaf(e, v[k].y, o[k].y);
            o[k].z = fmaf(e, v[k].z, o[k].z);
            o[k].w = fmaf(e, v[k].w, o[k].w);
        }
    }
    const int64_t row = (int64_t)head.z + r;
    float inv = 0.f;
    if (!empty) inv = a.sinks ? beside_sink(l, m, __ldg(a.sinks + row % a.heads) * kLog2e) : __fdividef(1.f, l);
    uint2 *out = reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + row * kD) + lane;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        out[32 * k] = inv != 0.f ? make_uint2(pack<kBf16>(o[k].x * inv, o[k].y * inv), pack<kBf16>(o[k].z * inv, o[k].w * inv)) : make_uint2(0u, 0u);
    if (a.lse && lane == 0) a.lse[row] = empty ? -INFINITY : (m + log2f(l)) * kLn2;
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
    if (p.batch_size <= 0 || p.max_seqlen_kv < (p.layout_kv == SFM_LAYOUT_PAGED)) return SFM_ERR_INVALID_ARG;
    if (p.layout_q == SFM_LAYOUT_BSND ? p.max_seqlen_q < 0 : p.total_q < 0) return SFM_ERR_INVALID_ARG;
    if (p.mask_mode != 0 && p.mask_mode != 3 && p.mask_mode != 4) return SFM_ERR_INVALID_ARG;
    if (p.mask_mode == 4 && (p.win_left < -1 || p.win_right < -1)) return SFM_ERR_INVALID_ARG;
    if (p.layout_kv == SFM_LAYOUT_PAGED && (p.block_size < 16 || p.block_size > 1024 || p.block_size % 16)) return SFM_ERR_LAYOUT;
    if (p.tree_words < 0 || p.tree_words > 16 || p.split_keys < 0 || p.split_keys % 128 || p.zero_rest & ~3) return SFM_ERR_INVALID_ARG;
    if (!std::isfinite(p.softmax_scale * kLog2e) || !(p.softcap == 0.f || (p.softcap >= 0x1p-100f && p.softcap <= 0x1p127f)) || (p.softcap > 0.f && !std::isfinite(p.softmax_scale / p.softcap)))
        return SFM_ERR_INVALID_ARG;
    if (p.max_seqlen_kv > 1 << 30) return SFM_ERR_UNSUPPORTED;
    const int64_t tokens = p.layout_q == SFM_LAYOUT_TND ? p.total_q : (int64_t)p.batch_size * p.max_seqlen_q;
    if (tokens * p.num_heads > INT32_MAX - 256) return SFM_ERR_UNSUPPORTED;      // rows that a copy's coordinate names
    return SFM_OK;
}

using EncodeFn = decltype(&cuTensorMapEncodeTiled);
using ReplaceFn = decltype(&cuTensorMapReplaceAddress);

// the driver's makers of TMA descriptors (pure host functions), looked up once
template <typename Fn>
Fn driver_function(const char *name)
{
    static const Fn fn = [name] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion(name, &p, 12000, cudaEnableDefault, &r) != cudaSuccess || r != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<Fn>(p);
    }();
    return fn;
}

// Rows of 512 values as eight blocks of 64: boxes of `blocks` blocks x `box_rows` rows land block after block, as the
// products read them.  Boxes of fewer than 64 rows, of which a stage takes several, land by eight rows instead: eight rows of
// each block, then the next eight, so that the distances stay the same across boxes (a copy per block and page took 64 of
// them for a tile of pages of 16: 16 trees of 16 tokens 607 us against 538, with pages of 48 657 against 577).
// The last map of a thread's (for queries, for keys) is kept with its sizes and gets another address
// where they are the same: encoding costs as much as the rest of a launch.
struct KeptMap {
    CUtensorMap map;
    int64_t rows = 0, row_bytes = 0;
    int dtype = 0, box_rows = 0, blocks = 0;
};

int make_map(CUtensorMap *map, KeptMap &kept, const void *ptr, int dtype, int64_t rows, int64_t row_bytes, int box_rows, int blocks)
{
    if (kept.rows != rows || kept.row_bytes != row_bytes || kept.dtype != dtype || kept.box_rows != box_rows || kept.blocks != blocks) {
        const EncodeFn encode = driver_function<EncodeFn>("cuTensorMapEncodeTiled");
        if (!encode) return SFM_ERR_CUDA;
        const bool octets = box_rows < 64;
        const cuuint64_t dims[4] = {64, (cuuint64_t)(octets ? 8 : rows), 8, (cuuint64_t)rows / 8}, strides[3] = {(cuuint64_t)row_bytes, 128, 8 * (cuuint64_t)row_bytes};
        const cuuint32_t box[4] = {64, (cuuint32_t)(octets ? 8 : box_rows), (cuuint32_t)blocks, (cuuint32_t)box_rows / 8}, steps[4] = {1, 1, 1, 1};
        kept.rows = 0;
        if (encode(&kept.map, dtype == SFM_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, octets ? 4 : 3,
                   const_cast<void *>(ptr), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return SFM_ERR_CUDA;
        kept.rows = rows;
        kept.row_bytes = row_bytes;
        kept.dtype = dtype;
        kept.box_rows = box_rows;
        kept.blocks = blocks;
        *map = kept.map;
        return SFM_OK;
    }
    const ReplaceFn replace = driver_function<ReplaceFn>("cuTensorMapReplaceAddress");
    if (!replace) return SFM_ERR_CUDA;
    *map = kept.map;
    return replace(map, const_cast<void *>(ptr)) == CUDA_SUCCESS ? SFM_OK : SFM_ERR_CUDA;
}

int64_t dense_tokens(const sfm_dense_params &p)
{
    return p.layout_q == SFM_LAYOUT_TND ? p.total_q : (int64_t)p.batch_size * p.max_seqlen_q;
}

// How the work is cut, from what the host knows, for a GPU that holds `clusters` pairs.
int dense_plan(const sfm_dense_params &p, int clusters, Plan *pl)
{
    const int64_t tokens = dense_tokens(p), rows = tokens * p.num_heads;
    pl->per_seq = (int32_t)(((int64_t)p.max_seqlen_q * p.num_heads + kRows - 1) / kRows);
    const int64_t slots = p.layout_q == SFM_LAYOUT_TND ? rows / kRows + p.batch_size : (int64_t)p.batch_size * pl->per_seq;
    const int64_t tiles = ((int64_t)p.max_seqlen_kv + kKeys - 1) / kKeys + 2;
    int64_t chunk = tiles;
    pl->balanced = 0;
    if (p.split_keys) {
        chunk = p.split_keys / kKeys;
    } else if (slots <= kMostBalanced && p.batch_size <= kMostBalanced && clusters <= kMostPairs && p.max_seqlen_kv > 8 * kKeys && slots * tiles < 1ll << 30) {
        pl->balanced = 1;
    }
    const int64_t splits = pl->balanced ? 2 : (tiles + chunk - 1) / chunk;
    if (slots * splits > INT32_MAX - 2 * (int64_t)clusters) return SFM_ERR_UNSUPPORTED;
    const int64_t most = pl->balanced ? (slots * tiles + kLeastTiles - 1) / kLeastTiles : slots * splits;
    pl->pairs = (int32_t)(most < clusters ? most : clusters);
    pl->slots = (int32_t)slots;
    pl->splits = (int32_t)splits;
    pl->chunk = (int32_t)chunk;
    pl->units = (int32_t)(slots * splits);
    return SFM_OK;
}

// workspace: partial rows, then their maxima and sums, then four integers per slot or part
size_t dense_parts(const Plan &pl) { return pl.splits <= 1 ? 0 : pl.balanced ? 2 * (size_t)pl.pairs : (size_t)pl.units; }
size_t dense_bytes(const Plan &pl)
{
    return pl.splits <= 1 ? 0 : dense_parts(pl) * kRows * (kD * 4 + 8) + (size_t)(pl.balanced ? pl.pairs : pl.slots) * 16;
}

using Kernel = void (*)(DenseArgs, Plan, CUtensorMap, CUtensorMap);

// Pairs of CTAs that the current device holds at once (the same for all of the kernel's forms, which have its whole
// shared memory).
int dense_clusters(int *device, int *clusters)
{
    static std::atomic<int> known[kMaxDevices];
    if (cudaGetDevice(device) != cudaSuccess) return SFM_ERR_CUDA;
    const bool keep = *device < kMaxDevices;
    *clusters = keep ? known[*device].load(std::memory_order_relaxed) : 0;
    if (*clusters > 0) return SFM_OK;
    const auto kernel = sfm_dense_kernel<true, kNoCap, false>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes) != cudaSuccess) return SFM_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(clusters, kernel, &cfg) != cudaSuccess || *clusters < 1) return SFM_ERR_CUDA;
    if (keep) known[*device].store(*clusters, std::memory_order_relaxed);
    return SFM_OK;
}

template <bool kBf16, int kCap, bool kBias>
cudaError_t launch(const DenseArgs &a, const Plan &pl, const CUtensorMap &q, const CUtensorMap &kv, int device, cudaStream_t st)
{
    static std::atomic<bool> ready[kMaxDevices];
    const Kernel kernel = sfm_dense_kernel<kBf16, kCap, kBias>;
    return prepared_launch(
        ready, device, [&] { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes); },
        [&] { return launch_dependent(kernel, dim3((unsigned)(2 * pl.pairs)), dim3(kThreads), (size_t)kSmemBytes, st, a, pl, q, kv); });
}

}  // namespace
}  // namespace sfm

using namespace sfm;

extern "C" int sfm_dense_workspace_size(const sfm_dense_params *params, size_t *bytes)
{
    int rc = dense_check(params);
    if (rc) return rc;
    if (!bytes) return SFM_ERR_INVALID_ARG;
    *bytes = 0;
    if (dense_tokens(*params) == 0) return SFM_OK;
    int device = 0, clusters = 0;
    rc = dense_clusters(&device, &clusters);
    if (rc) return rc;
    Plan pl = {};
    rc = dense_plan(*params, clusters, &pl);
    if (rc) return rc;
    *bytes = dense_bytes(pl);
    return SFM_OK;
}

extern "C" int sfm_dense_forward(const sfm_dense_params *pp, const sfm_dense_tensors *t, void *out, float *lse,
                                 void *workspace, size_t workspace_bytes, int32_t *status, sfm_stream_t stream)
{
    int rc = dense_check(pp);
    if (rc) return rc;
    if (!t) return SFM_ERR_INVALID_ARG;
    const sfm_dense_params &p = *pp;
    const bool paged = p.layout_kv == SFM_LAYOUT_PAGED, tnd = p.layout_q == SFM_LAYOUT_TND;
    if (t->kv_row_stride < 2 * kD || t->kv_row_stride % 16 || t->kv_rows < 0) return SFM_ERR_LAYOUT;
    if (t->kv_rows > ((int64_t)1 << 31) - 1024) return SFM_ERR_UNSUPPORTED;
    if (paged && t->kv_rows < p.block_size) return SFM_ERR_LAYOUT;
    if (p.layout_kv == SFM_LAYOUT_BSND && t->kv_rows < (int64_t)p.batch_size * p.max_seqlen_kv) return SFM_ERR_LAYOUT;
    if ((tnd && !t->cu_seqlens_q) || (p.layout_kv == SFM_LAYOUT_TND && !t->cu_seqlens_kv)) return SFM_ERR_INVALID_ARG;
    if (paged ? !t->seqused_kv || !t->block_table || t->block_table_stride <= 0 : t->block_table != nullptr)
        return SFM_ERR_INVALID_ARG;
    if (p.tree_words ? !t->tree_mask || !t->positions || t->prefix_lens || t->key_begin || t->key_end
                     : t->tree_mask || t->positions)
        return SFM_ERR_INVALID_ARG;
    const int32_t tokens = tnd ? p.total_q : p.batch_size * p.max_seqlen_q;
    if (tokens == 0) return SFM_OK;
    if (!t->q || (!t->kv && t->kv_rows) || !out) return SFM_ERR_INVALID_ARG;
    if (((uintptr_t)t->q | (uintptr_t)t->kv | (uintptr_t)out) & 15u) return SFM_ERR_LAYOUT;
    const void *const words[] = {lse, status, t->sinks, t->bias_slopes, t->block_table, t->cu_seqlens_q, t->cu_seqlens_kv, t->seqused_q, t->seqused_kv,
                                 t->prefix_lens, t->key_begin, t->key_end, t->positions};
    uintptr_t bits = 0;
    for (const void *x : words) bits |= (uintptr_t)x;
    if (bits & 3u || (uintptr_t)t->tree_mask & 7u) return SFM_ERR_LAYOUT;

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
    if (paged && (int64_t)t->block_table_stride * p.block_size < a.max_kv) a.max_kv = (int32_t)((int64_t)t->block_table_stride * p.block_size);
    a.mode = p.mask_mode;
    const int32_t far = 1 << 30;
    a.win_left = p.win_left < 0 || p.win_left > far ? far : p.win_left;
    a.win_right = p.win_right < 0 || p.win_right > far ? far : p.win_right;
    a.layout_kv = p.layout_kv;
    a.block = p.block_size;
    a.cols = t->block_table_stride;
    a.words = p.tree_words;
    a.zero_rest = p.zero_rest;
    a.scale = p.softmax_scale;
    a.cap = p.softcap;
    a.block_div = make_fastdiv(paged ? (uint32_t)p.block_size : 1u);
    a.heads_div = make_fastdiv((uint32_t)p.num_heads);

    int device = 0, clusters = 0;
    rc = dense_clusters(&device, &clusters);
    if (rc) return rc;
    Plan pl = {};
    rc = dense_plan(p, clusters, &pl);
    if (rc) return rc;
    if (workspace_bytes < dense_bytes(pl) || (dense_bytes(pl) && !workspace)) return SFM_ERR_WORKSPACE;
    if ((uintptr_t)workspace & 255u) return SFM_ERR_LAYOUT;
    // rows per box of keys: as many as a page holds whole boxes of, 64 at most
    pl.box_rows = 64;
    if (paged) {
        pl.box_rows = p.block_size & -p.block_size;
        if (pl.box_rows > 64) pl.box_rows = 64;
    }
    pl.align = paged ? pl.box_rows : 1;
    pl.block_bytes = pl.box_rows == 64 ? 8192 : 1024;
    pl.octet_bytes = pl.box_rows == 64 ? 1024 : 4096;
    pl.slots_div = make_fastdiv((uint32_t)pl.slots);
    pl.per_seq_div = make_fastdiv((uint32_t)(pl.per_seq > 0 ? pl.per_seq : 1));
    const bool bf16 = p.dtype == SFM_DTYPE_BF16;
    pl.idesc_s = idesc_f16(kRows, kKeys, bf16, false, false);
    pl.idesc_o = idesc_f16(kRows, 256, bf16, false, true);
    if (pl.splits > 1) {
        pl.part_o = static_cast<float4 *>(workspace);
        pl.part_ml = reinterpret_cast<float2 *>(pl.part_o + dense_parts(pl) * kRows * (kD / 4));
        pl.head = reinterpret_cast<int4 *>(pl.part_ml + dense_parts(pl) * kRows);
    }
    CUtensorMap q_map, kv_map;
    static thread_local KeptMap kept_q, kept_kv;
    rc = make_map(&q_map, kept_q, t->q, p.dtype, (int64_t)tokens * p.num_heads, 2 * kD, 64, 8);
    // (a map has a row at least; where kv has none no sequence has a key, and nothing is copied)
    if (!rc) rc = make_map(&kv_map, kept_kv, t->kv_rows ? t->kv : t->q, p.dtype, t->kv_rows ? t->kv_rows : 1, t->kv_row_stride, pl.box_rows, kBlocks);
    if (rc) return rc;
    const cudaStream_t st = (cudaStream_t)stream;
    const CapKind cap = a.cap > kWideCap ? kLargeCap : a.cap > 0.f ? kSmallCap : kNoCap;
    static constexpr decltype(&launch<true, kNoCap, true>) forms[2][3][2] = {
        {{launch<false, kNoCap, false>, launch<false, kNoCap, true>}, {launch<false, kSmallCap, false>, launch<false, kSmallCap, true>},
         {launch<false, kLargeCap, false>, launch<false, kLargeCap, true>}},
        {{launch<true, kNoCap, false>, launch<true, kNoCap, true>}, {launch<true, kSmallCap, false>, launch<true, kSmallCap, true>},
         {launch<true, kLargeCap, false>, launch<true, kLargeCap, true>}}};
    cudaError_t e = forms[bf16][cap][a.slopes != nullptr](a, pl, q_map, kv_map, device, st);
    if (e == cudaSuccess && pl.splits > 1)
        e = launch_dependent(bf16 ? sfm_dense_join_kernel<true> : sfm_dense_join_kernel<false>, dim3(16 * (unsigned)(pl.balanced ? pl.pairs : pl.slots)), dim3(256), 0, st, a, pl);
    return e == cudaSuccess ? SFM_OK : SFM_ERR_CUDA;
}
