// sfm_move.cu -- the rows of an accepted path moved to the front of the
// drafted ones (sfm_kv_move).
//
// path[i] >= i and it grows, so the row that step i writes lies before every
// row that a later step reads (path[k] >= k > i for k > i), but it may be one
// that an earlier step reads.  A CTA takes a sequence's steps in batches: all of a
// batch's rows are read before the first of them is written.  A few round trips
// bound it: the path, the pages of its rows, the rows (32 sequences of up to 5
// rows of 1 KB 2.2 us, 512 of up to 24 rows of 256 bytes 2.9; one thread per
// 16-byte column that took eight steps at a time needed 7 for the latter).
#include "sfm_internal.cuh"

namespace sfm {
namespace {

constexpr int kThreads = 256;
constexpr int kEach = 4;              // rows per thread and batch

struct MoveArgs {
    const int32_t *path, *first, *table;
    uint8_t *cache;
    int32_t *status;
    int64_t row_stride, rows;
    int32_t max_path, pieces, block, seq_rows, cols, lanes_log2;
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

// grid (groups of 256 pieces, sequences).  A row is taken by 2^lanes_log2 threads, a 16-byte piece each.
__global__ void __launch_bounds__(kThreads) sfm_move_kernel(const MoveArgs a)
{
    __shared__ int64_t src[kThreads], dst[kThreads];
    __shared__ int good;
    grid_follow();
    const int b = blockIdx.y, tid = threadIdx.x, lane = tid & ((1 << a.lanes_log2) - 1), row = tid >> a.lanes_log2;
    const int rows = kThreads >> a.lanes_log2, piece = blockIdx.x * kThreads + lane;
    const int32_t *path = a.path + (int64_t)b * a.max_path;
    const int64_t first = a.first[b];
    for (int base = 0; base < a.max_path; base += kThreads) {
        // where the next 256 entries lead, and how many of them count
        const int i = base + tid, n = min(a.max_path - base, kThreads);
        if (tid == 0) good = n;
        __syncthreads();
        if (tid < n) {
            const int32_t from = __ldg(path + i), before = i > 0 ? __ldg(path + i - 1) : -1;
            const bool grows = from > before && from >= 0;
            src[tid] = grows ? row_of(a, b, first + from) : -1;
            dst[tid] = grows ? row_of(a, b, first + i) : -1;
            if (src[tid] < 0 || dst[tid] < 0) atomicMin(&good, tid);
        }
        __syncthreads();
        const int count = good;
        if (a.status && blockIdx.x == 0 && tid == count && count < n) {
            // the entry that ends the path, unless it is the negative one behind it
            const int32_t from = __ldg(path + i), before = i > 0 ? __ldg(path + i - 1) : -1;
            if (from >= 0) atomicOr(a.status, from > before ? SFM_STATUS_BAD_BLOCK : SFM_STATUS_BAD_INDEX);
        }
        for (int k0 = 0; k0 < count; k0 += rows * kEach) {
            uint4 v[kEach];
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                const int k = k0 + e * rows + row;
                if (k < count && piece < a.pieces) v[e] = *reinterpret_cast<const uint4 *>(a.cache + src[k] * a.row_stride + (int64_t)piece * 16);
            }
            __syncthreads();
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                const int k = k0 + e * rows + row;
                if (k < count && piece < a.pieces && src[k] != dst[k])
                    *reinterpret_cast<uint4 *>(a.cache + dst[k] * a.row_stride + (int64_t)piece * 16) = v[e];
            }
            __syncthreads();
        }
        if (count < n) return;
        __syncthreads();
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
    while (a.lanes_log2 < 8 && (1 << a.lanes_log2) < a.pieces) ++a.lanes_log2;
    const dim3 grid((unsigned)((a.pieces + kThreads - 1) / kThreads), (unsigned)p.batch_size);
    return launch_dependent(sfm_move_kernel, grid, dim3(kThreads), 0, (cudaStream_t)stream, a) == cudaSuccess ? SFM_OK : SFM_ERR_CUDA;
}
