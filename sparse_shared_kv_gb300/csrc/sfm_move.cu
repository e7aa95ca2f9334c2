// sfm_move.cu -- the rows of an accepted path moved to the front of the
// drafted ones (sfm_kv_move).
//
// path[i] >= i and it grows, so the row that step i writes lies before every
// row that a later step reads (path[k] >= k > i for k > i): a thread that owns
// one 16-byte column of a sequence's rows may take the steps in order, several
// reads ahead of their writes, and needs no other thread.
#include "sfm_internal.cuh"

namespace sfm {
namespace {

constexpr int kThreads = 64;
constexpr int kAhead = 8;             // rows read before the first of them is written

struct MoveArgs {
    const int32_t *path, *first, *table;
    uint8_t *cache;
    int32_t *status;
    int64_t row_stride, rows;
    int32_t max_path, pieces, block, seq_rows, cols;
    FastDiv block_div;
};

// Cache row of position j of sequence b, or -1.
__device__ __forceinline__ int64_t row_of(const MoveArgs &a, int b, int64_t j)
{
    int64_t row;
    if (j < 0 || j > INT32_MAX) return -1;
    if (a.block > 0) {
        const uint32_t blk = fdiv((uint32_t)j, a.block_div);
        if (blk >= (uint32_t)a.cols) return -1;
        const int32_t id = __ldg(a.table + (int64_t)b * a.cols + blk);
        if (id < 0) return -1;
        row = (int64_t)id * a.block + (j - (int64_t)blk * a.block);
    } else {
        if (j >= a.seq_rows) return -1;
        row = (int64_t)b * a.seq_rows + j;
    }
    return row < a.rows ? row : -1;
}

// grid (column groups, sequences)
__global__ void __launch_bounds__(kThreads) sfm_move_kernel(const MoveArgs a)
{
    grid_follow();
    const int b = blockIdx.y, piece = blockIdx.x * kThreads + threadIdx.x;
    const bool tell = a.status && piece == 0;
    if (piece >= a.pieces) return;
    const int32_t *path = a.path + (int64_t)b * a.max_path;
    const int64_t first = a.first[b];
    int32_t before = -1;
    bool more = true;
    for (int i0 = 0; i0 < a.max_path && more; i0 += kAhead) {
        // eight entries, then their pages, then their rows: three round trips for all of them
        int32_t from[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) from[k] = i0 + k < a.max_path ? __ldg(path + i0 + k) : -1;
        int64_t src[kAhead], dst[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            src[k] = row_of(a, b, from[k] >= 0 ? first + from[k] : -1);
            dst[k] = row_of(a, b, from[k] >= 0 ? first + i0 + k : -1);
        }
        uint4 v[kAhead];
        uint32_t moved = 0;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (!more) continue;
            if (from[k] <= before) {
                more = false;
                if (from[k] >= 0 && tell) atomicOr(a.status, SFM_STATUS_BAD_INDEX);
                continue;
            }
            before = from[k];
            if (src[k] < 0 || dst[k] < 0) {
                more = false;
                if (tell) atomicOr(a.status, SFM_STATUS_BAD_BLOCK);
                continue;
            }
            if (src[k] == dst[k]) continue;
            v[k] = *reinterpret_cast<const uint4 *>(a.cache + src[k] * a.row_stride + (int64_t)piece * 16);
            moved |= 1u << k;
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (moved >> k & 1) *reinterpret_cast<uint4 *>(a.cache + dst[k] * a.row_stride + (int64_t)piece * 16) = v[k];
    }
}

}  // namespace
}  // namespace sfm

using namespace sfm;

extern "C" int sfm_kv_move(const sfm_move_params *pp, const int32_t *path, const int32_t *first,
                           const int32_t *block_table, void *cache, int32_t *status, sfm_stream_t stream)
{
    if (!pp) return SFM_ERR_INVALID_ARG;
    const sfm_move_params &p = *pp;
    if (p.batch_size < 0 || p.max_path < 0 || p.row_bytes <= 0 || p.block_size < 0) return SFM_ERR_INVALID_ARG;
    if (p.row_bytes % 16 || p.row_stride < p.row_bytes || p.row_stride % 16 || p.rows <= 0) return SFM_ERR_LAYOUT;
    if (p.rows > ((int64_t)1 << 31) - 2) return SFM_ERR_UNSUPPORTED;
    if (p.block_size ? p.block_table_stride <= 0 : p.max_seqlen_kv <= 0) return SFM_ERR_INVALID_ARG;
    if ((p.block_size != 0) != (block_table != nullptr) && p.batch_size) return SFM_ERR_INVALID_ARG;
    if (p.batch_size == 0 || p.max_path == 0) return SFM_OK;
    if (!path || !first || !cache) return SFM_ERR_INVALID_ARG;
    if ((uintptr_t)cache & 15u || ((uintptr_t)path | (uintptr_t)first | (uintptr_t)block_table | (uintptr_t)status) & 3u)
        return SFM_ERR_LAYOUT;
    if (p.batch_size > 65535) return SFM_ERR_UNSUPPORTED;
    MoveArgs a = {};
    a.path = path;
    a.first = first;
    a.table = block_table;
    a.cache = static_cast<uint8_t *>(cache);
    a.status = status;
    a.row_stride = p.row_stride;
    a.rows = p.rows;
    a.max_path = p.max_path;
    a.pieces = p.row_bytes / 16;
    a.block = p.block_size;
    a.seq_rows = p.max_seqlen_kv;
    a.cols = p.block_table_stride;
    a.block_div = make_fastdiv(p.block_size ? (uint32_t)p.block_size : 1u);
    const dim3 grid((unsigned)((a.pieces + kThreads - 1) / kThreads), (unsigned)p.batch_size);
    return launch_dependent(sfm_move_kernel, grid, dim3(kThreads), 0, (cudaStream_t)stream, a) == cudaSuccess ? SFM_OK : SFM_ERR_CUDA;
}
