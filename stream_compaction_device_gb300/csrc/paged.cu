// Block tables and slot maps of a paged key/value cache (sm_103a).
//
// A request whose cache holds c tokens keeps ceil(c / P) pages of P tokens,
// listed in its row of the block table.  All three operations are a count per
// row, the inclusive add-scan of the counts (geek-doc.cn "并行前缀和 scan ..."
// section 一: a scan turns counts into output positions), and a load-balanced
// expansion: output element g belongs to the first row whose scanned end is
// above g, found by a binary search of the ends.
//
//   extend  : count = pages that the new tokens of a row open;
//             table[row][have + j] = pages[free - 1 - g]
//   slots   : count = new tokens of a row;
//             slot[g] = table[row][pos / P] * P + pos % P
//   release : count = pages of a row that ended;
//             pages[free + g] = table[row][j]
//
// Split: the row counts are 4 to 9 bytes each while an output element moves 8
// to 20, so every block scans all the counts for itself (out of L2, into its
// shared memory) and takes an equal share of the output: one launch, no block
// waits for another, and one long row is spread over the whole GPU.
// Sums run in 64 bits and are stored saturated to INT32_MAX, so that lengths
// whose sum passes 32 bits cannot wrap into positions that look valid.
#include "core.cuh"
#include "launch.h"

namespace devscan {
namespace {

constexpr int kPagedThreads = 512;
constexpr int kPagedWarps = kPagedThreads / 32;

__device__ __forceinline__ long long blocks_of(long long tokens, int page) { return (tokens + page - 1) / page; }

// Pages that row `r` needs beyond those it has; false for a row that cannot
// be served whatever the pool holds (negative lengths, or wider than the
// table).
struct ExtendCount {
    const int32_t *cached, *fresh;
    int page, width;
    __device__ __forceinline__ bool count(int r, int &have, int &need) const
    {
        const long long c = cached[r], n = fresh[r];
        have = need = 0;
        if (c < 0 || n < 0) return false;
        const long long h = blocks_of(c, page), w = blocks_of(c + n, page);
        if (w > width) return false;
        have = static_cast<int>(h);
        need = static_cast<int>(w - h);
        return true;
    }
    __device__ __forceinline__ int operator()(int r) const
    {
        int have, need;
        count(r, have, need);
        return need;
    }
};

struct SlotCount {
    const int32_t *fresh;
    const uint8_t *granted;   // null: every row runs
    __device__ __forceinline__ int operator()(int r) const
    {
        if (granted != nullptr && granted[r] == 0) return 0;
        const int n = fresh[r];
        return n > 0 ? n : 0;
    }
};

struct ReleaseCount {
    const int32_t *cached;
    const uint8_t *done;
    int page, width;
    __device__ __forceinline__ int operator()(int r) const
    {
        if (done[r] == 0 || cached[r] <= 0) return 0;
        const long long b = blocks_of(cached[r], page);
        return static_cast<int>(b < width ? b : width);
    }
};

// ends[r] = min(count(0) + ... + count(r), INT32_MAX) for all rows, by one
// block; ends in shared or global memory.  Ends with a block barrier.
template <class Count>
__device__ void scan_rows(const Count &count, int rows, int32_t *ends)
{
    __shared__ long long s_warp[kPagedWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    long long base = 0;
    for (int r0 = 0; r0 < rows; r0 += kPagedThreads) {
        const int r = r0 + tid;
        long long v = r < rows ? count(r) : 0;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long u = __shfl_up_sync(kFullMask, v, d);
            if (lane >= d) v += u;
        }
        if (lane == 31) s_warp[warp] = v;
        __syncthreads();
        long long ahead = 0, all = 0;
#pragma unroll
        for (int w = 0; w < kPagedWarps; ++w) {
            if (w < warp) ahead += s_warp[w];
            all += s_warp[w];
        }
        const long long end = base + ahead + v;
        if (r < rows) ends[r] = static_cast<int32_t>(end < INT32_MAX ? end : INT32_MAX);
        base += all;
        __syncthreads();
    }
}

// First row whose end is above g; `rows` if none.
__device__ __forceinline__ int row_of(const int32_t *ends, int rows, int g)
{
    int lo = 0, hi = rows;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (ends[mid] > g) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

template <class Count>
__global__ void __launch_bounds__(kPagedThreads) row_ends_kernel(Count count, int rows, int32_t *ends)
{
    scan_rows(count, rows, ends);
}

// IN_SHARED: the block scans the counts into its own shared memory; else
// row_ends_kernel has left the ends in `g_ends`.
template <bool IN_SHARED, class Count>
__device__ __forceinline__ const int32_t *row_ends(const Count &count, int rows, const int32_t *g_ends)
{
    extern __shared__ int32_t s_ends[];
    if (!IN_SHARED) return g_ends;
    scan_rows(count, rows, s_ends);
    return s_ends;
}

__device__ __forceinline__ int clamp_free(const int32_t *free_count, int pool)
{
    const int f = *free_count;
    return f < 0 ? 0 : (f < pool ? f : pool);
}

template <bool IN_SHARED>
__global__ void __launch_bounds__(kPagedThreads)
extend_kernel(int32_t *__restrict__ table, size_t stride, int rows, ExtendCount count,
              const int32_t *__restrict__ pages, int pool, const int32_t *__restrict__ free_count,
              uint8_t *__restrict__ granted, int32_t *__restrict__ left, const int32_t *g_ends)
{
    const int32_t *ends = row_ends<IN_SHARED>(count, rows, g_ends);
    const int free = clamp_free(free_count, pool);
    // Rows are served in order while the pool lasts: those whose end is within it.
    const int served = row_of(ends, rows, free);
    const int total = served > 0 ? ends[served - 1] : 0;
    const int tid = blockIdx.x * kPagedThreads + threadIdx.x, threads = gridDim.x * kPagedThreads;
    for (int r = tid; r < rows; r += threads) {
        int have, need;
        const bool valid = count.count(r, have, need);
        granted[r] = valid && (need == 0 || ends[r] <= free);
    }
    if (tid == 0) *left = free - total;
    for (long long g = tid; g < total; g += threads) {
        const int r = row_of(ends, rows, static_cast<int>(g));
        int have, need;
        count.count(r, have, need);
        const int j = static_cast<int>(g) - (ends[r] - need);
        table[static_cast<size_t>(r) * stride + have + j] = pages[free - 1 - static_cast<int>(g)];
    }
}

template <bool IN_SHARED>
__global__ void __launch_bounds__(kPagedThreads)
slot_kernel(const int32_t *__restrict__ table, size_t stride, int rows, int width,
            const int32_t *__restrict__ cached, SlotCount count, int page, int tokens,
            int32_t *__restrict__ starts, long long *__restrict__ slots, int32_t *__restrict__ positions,
            int32_t *__restrict__ row_ids, const int32_t *g_ends)
{
    const int32_t *ends = row_ends<IN_SHARED>(count, rows, g_ends);
    const int tid = blockIdx.x * kPagedThreads + threadIdx.x, threads = gridDim.x * kPagedThreads;
    for (int r = tid; r < rows; r += threads) starts[r + 1] = ends[r];
    if (tid == 0) starts[0] = 0;
    for (long long g = tid; g < tokens; g += threads) {
        const int r = row_of(ends, rows, static_cast<int>(g));
        long long slot = -1;
        int pos = -1, id = -1;
        if (r < rows) {
            const int first = r > 0 ? ends[r - 1] : 0;
            const long long at = static_cast<long long>(cached[r]) + (g - first);
            id = r;
            const bool valid = at >= 0 && at <= INT32_MAX;
            pos = valid ? static_cast<int>(at) : -1;
            const long long b = at / page;
            if (valid && b < width) {
                const int entry = table[static_cast<size_t>(r) * stride + b];
                if (entry >= 0) slot = static_cast<long long>(entry) * page + at % page;
            }
        }
        slots[g] = slot;
        positions[g] = pos;
        row_ids[g] = id;
    }
}

template <bool IN_SHARED>
__global__ void __launch_bounds__(kPagedThreads)
release_kernel(const int32_t *__restrict__ table, size_t stride, int rows, ReleaseCount count,
               int32_t *__restrict__ pages, int pool, const int32_t *__restrict__ free_count,
               int32_t *__restrict__ left, const int32_t *g_ends)
{
    const int32_t *ends = row_ends<IN_SHARED>(count, rows, g_ends);
    const int free = clamp_free(free_count, pool);
    const int served = row_of(ends, rows, pool - free);   // rows whose pages fit the pool array
    const int total = served > 0 ? ends[served - 1] : 0;
    const int tid = blockIdx.x * kPagedThreads + threadIdx.x, threads = gridDim.x * kPagedThreads;
    if (tid == 0) *left = free + total;
    for (long long g = tid; g < total; g += threads) {
        const int r = row_of(ends, rows, static_cast<int>(g));
        const int first = r > 0 ? ends[r - 1] : 0;
        pages[free + static_cast<int>(g)] = table[static_cast<size_t>(r) * stride + (static_cast<int>(g) - first)];
    }
}

// Blocks for `most` output elements at the most.
unsigned paged_blocks(unsigned long long most, const Workspace &ws)
{
    const unsigned long long b = (most + kPagedThreads - 1) / kPagedThreads;
    const unsigned long long cap = static_cast<unsigned long long>(ws.num_sms) * 2;
    return static_cast<unsigned>(b < 1 ? 1 : (b < cap ? b : cap));
}

template <class Count>
cudaError_t prepare_ends(const Count &count, int rows, int32_t *scratch, size_t *shared_bytes, cudaStream_t s)
{
    *shared_bytes = 0;
    if (rows <= kPagedSharedRows) {
        *shared_bytes = static_cast<size_t>(rows) * sizeof(int32_t);
        return cudaSuccess;
    }
    row_ends_kernel<Count><<<1, kPagedThreads, 0, s>>>(count, rows, scratch);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_block_table_extend(int32_t *table, size_t stride, int rows, int width, const int32_t *cached,
                                      const int32_t *fresh, int page, const int32_t *pages, int pool,
                                      const int32_t *free_count, uint8_t *granted, int32_t *left, int32_t *scratch,
                                      const Workspace &ws, cudaStream_t s)
{
    const ExtendCount count{cached, fresh, page, width};
    size_t shared = 0;
    cudaError_t e = prepare_ends(count, rows, scratch, &shared, s);
    if (e != cudaSuccess) return e;
    unsigned long long most = static_cast<unsigned long long>(rows) * width;
    if (most > static_cast<unsigned long long>(pool)) most = pool;
    const unsigned blocks = paged_blocks(most, ws);
    if (rows <= kPagedSharedRows)
        extend_kernel<true><<<blocks, kPagedThreads, shared, s>>>(table, stride, rows, count, pages, pool, free_count,
                                                                  granted, left, nullptr);
    else
        extend_kernel<false><<<blocks, kPagedThreads, 0, s>>>(table, stride, rows, count, pages, pool, free_count,
                                                              granted, left, scratch);
    return cudaGetLastError();
}

cudaError_t launch_slot_map(const int32_t *table, size_t stride, int rows, int width, const int32_t *cached,
                            const int32_t *fresh, const uint8_t *granted, int page, int tokens, int32_t *starts,
                            int64_t *slots, int32_t *positions, int32_t *row_ids, int32_t *scratch,
                            const Workspace &ws, cudaStream_t s)
{
    const SlotCount count{fresh, granted};
    size_t shared = 0;
    cudaError_t e = prepare_ends(count, rows, scratch, &shared, s);
    if (e != cudaSuccess) return e;
    const unsigned blocks = paged_blocks(static_cast<unsigned long long>(tokens), ws);
    long long *out = reinterpret_cast<long long *>(slots);
    if (rows <= kPagedSharedRows)
        slot_kernel<true><<<blocks, kPagedThreads, shared, s>>>(table, stride, rows, width, cached, count, page,
                                                                tokens, starts, out, positions, row_ids, nullptr);
    else
        slot_kernel<false><<<blocks, kPagedThreads, 0, s>>>(table, stride, rows, width, cached, count, page, tokens,
                                                            starts, out, positions, row_ids, scratch);
    return cudaGetLastError();
}

cudaError_t launch_block_table_release(const int32_t *table, size_t stride, int rows, int width,
                                       const int32_t *cached, const uint8_t *done, int page, int32_t *pages, int pool,
                                       const int32_t *free_count, int32_t *left, int32_t *scratch,
                                       const Workspace &ws, cudaStream_t s)
{
    const ReleaseCount count{cached, done, page, width};
    size_t shared = 0;
    cudaError_t e = prepare_ends(count, rows, scratch, &shared, s);
    if (e != cudaSuccess) return e;
    unsigned long long most = static_cast<unsigned long long>(rows) * width;
    if (most > static_cast<unsigned long long>(pool)) most = pool;
    const unsigned blocks = paged_blocks(most, ws);
    if (rows <= kPagedSharedRows)
        release_kernel<true><<<blocks, kPagedThreads, shared, s>>>(table, stride, rows, count, pages, pool,
                                                                   free_count, left, nullptr);
    else
        release_kernel<false><<<blocks, kPagedThreads, 0, s>>>(table, stride, rows, count, pages, pool, free_count,
                                                               left, scratch);
    return cudaGetLastError();
}

}  // namespace devscan
