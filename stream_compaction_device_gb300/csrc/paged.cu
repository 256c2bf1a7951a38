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
// waits for another, and one long row is spread over the whole GPU.  A warp
// takes up to 128 or 256 neighbouring outputs and looks for the rows of the
// first and the last of them.
//
// What bounds it: a call of few rows its launch and one wait for memory (64
// rows 4.9 us, 256 rows 3.6 us by device time, of which an empty kernel takes
// more than half); more than 4,096 rows the one block that scans them (900 rows
// per us); 4,096 rows the scan in front (6.4 us with nothing to move)
// and then memory: with nothing in L2 they extend by 2.8 M pages in 16 us and
// release 2.1 M in 15 us (22 and 17 MB, 3.3 and 2.5 us at the copy rate), and
// 2.7 M slots of 1,000 rows take 12 us (44 MB, 6.5 us).
// Sums run in 64 bits and are stored saturated to INT32_MAX, so that lengths
// whose sum passes 32 bits cannot wrap into positions that look valid.  Rows
// and outputs are counted without sign: there may be nearly 2^31 of either,
// and a step past the last one must not wrap.
#include "core.cuh"
#include "launch.h"

namespace devscan {
namespace {

constexpr int kPagedThreads = 512;
constexpr int kPagedWarps = kPagedThreads / 32;
// Consecutive outputs that a warp takes at a time, at most.  Small chunks keep
// what the grid touches at one time close together in memory: 4,096 rows with
// nothing in L2 took (us, chunks of 128 : 256 : 512) 15.1 : 17.6 : 17.8 to
// release, 15.8 : 15.7 : 20.4 to extend, and 2.7 M slots 14.1 : 12.1 : 12.6.
constexpr int kMoveChunk = 128, kSlotChunk = 256;

// Division of any uint32 by the page size, by a multiplication with its
// reciprocal rounded up to 33 bits (Granlund and Montgomery, "Division by
// invariant integers using multiplication", 1994, figure 4.1).
struct Pages {
    uint32_t page, magic, shift;
    explicit Pages(uint32_t p) : page(p), magic(0), shift(0)
    {
        while ((1ull << shift) < p) ++shift;   // ceil(log2 p)
        magic = static_cast<uint32_t>(((1ull << 32) * ((1ull << shift) - p)) / p + 1);
    }
    __device__ __forceinline__ uint32_t div(uint32_t x) const
    {
        const uint32_t t = __umulhi(magic, x);
        return shift == 0 ? x : (t + ((x - t) >> 1)) >> (shift - 1);
    }
    __device__ __forceinline__ uint32_t blocks_of(uint32_t tokens) const
    {
        const uint32_t q = div(tokens);
        return q + (q * page != tokens ? 1u : 0u);
    }
};

// What a row brings: its number of outputs, and the place of its first one
// (in the row's table entries or tokens).
struct RowPart {
    int count, place;
};

constexpr int kRun = 8;   // neighbouring rows that a thread scans

// v[k] = p[r + k] for the rows before `rows`; 0 for the others.
__device__ __forceinline__ void load_run(const int32_t *p, unsigned r, unsigned rows, int (&v)[kRun])
{
    if (r + kRun <= rows && reinterpret_cast<uintptr_t>(p + r) % 16 == 0) {
        const int4 *q = reinterpret_cast<const int4 *>(p + r);
        const int4 a = __ldg(q), b = __ldg(q + 1);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
#pragma unroll
        for (int k = 0; k < kRun; ++k) v[k] = r + k < rows ? __ldg(p + r + k) : 0;
    }
}
// The same of flags; null: 1 for every row.
__device__ __forceinline__ void load_run(const uint8_t *p, unsigned r, unsigned rows, int (&v)[kRun])
{
    if (p != nullptr && r + kRun <= rows && reinterpret_cast<uintptr_t>(p + r) % 8 == 0) {
        const uint2 a = __ldg(reinterpret_cast<const uint2 *>(p + r));
#pragma unroll
        for (int k = 0; k < kRun; ++k) v[k] = ((k < 4 ? a.x : a.y) >> (k % 4 * 8)) & 255;
    } else {
#pragma unroll
        for (int k = 0; k < kRun; ++k) v[k] = r + k >= rows ? 0 : p == nullptr ? 1 : __ldg(p + r + k);
    }
}

// Pages that a row needs beyond those it has, and how many those are.  A row
// that cannot be served whatever the pool holds (negative lengths, or wider
// than the table) needs none; its place is -1.
struct ExtendCount {
    const int32_t *cached, *fresh;
    Pages pages;
    int width;
    __device__ __forceinline__ void load(unsigned r, unsigned rows, int (&a)[kRun], int (&b)[kRun]) const
    {
        load_run(cached, r, rows, a);
        load_run(fresh, r, rows, b);
    }
    __device__ __forceinline__ RowPart part(int c, int n) const
    {
        const uint32_t have = pages.blocks_of(c);
        const uint32_t want = pages.blocks_of(static_cast<uint32_t>(c) + static_cast<uint32_t>(n));
        if (c < 0 || n < 0 || want > static_cast<uint32_t>(width)) return {0, -1};
        return {static_cast<int>(want - have), static_cast<int>(have)};
    }
};

// Tokens of a row, from its length; without a flag it brings none.
struct SlotCount {
    const int32_t *cached, *fresh;
    const uint8_t *granted;   // null: every row runs
    __device__ __forceinline__ void load(unsigned r, unsigned rows, int (&a)[kRun], int (&b)[kRun]) const
    {
        int runs[kRun];
        load_run(cached, r, rows, a);
        load_run(fresh, r, rows, b);
        load_run(granted, r, rows, runs);
#pragma unroll
        for (int k = 0; k < kRun; ++k) b[k] = runs[k] != 0 && b[k] > 0 ? b[k] : 0;
    }
    __device__ __forceinline__ RowPart part(int c, int n) const { return {n, c}; }
};

struct ReleaseCount {
    const int32_t *cached;
    const uint8_t *done;
    Pages pages;
    int width;
    __device__ __forceinline__ void load(unsigned r, unsigned rows, int (&a)[kRun], int (&b)[kRun]) const
    {
        load_run(cached, r, rows, a);
        load_run(done, r, rows, b);
    }
    __device__ __forceinline__ RowPart part(int c, int ended) const
    {
        const uint32_t b = pages.blocks_of(c);
        if (ended == 0 || c <= 0) return {0, 0};
        return {static_cast<int>(b < static_cast<uint32_t>(width) ? b : static_cast<uint32_t>(width)), 0};
    }
};

// The scanned rows: ends[r] = min(count(0) + ... + count(r), INT32_MAX), and
// places[r] as the row gave it.  In shared memory, or in global scratch.
struct Ends {
    uint32_t *ends;
    int32_t *places;
};

// Scans the rows by one block, a run of neighbours per thread: one wait for
// memory and one for the other warps in 4,096 rows.  Ends with a block barrier.
template <class Count>
__device__ void scan_rows(const Count &count, unsigned rows, const Ends &out)
{
    __shared__ long long s_warp[2][kPagedWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    long long base = 0;
    int turn = 0;
    for (unsigned r0 = 0; r0 < rows; r0 += kPagedThreads * kRun, turn ^= 1) {
        const unsigned r = r0 + tid * kRun;
        int a[kRun], b[kRun];
        long long sum = 0;
        count.load(r, rows, a, b);
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
            const RowPart p = count.part(a[k], b[k]);
            a[k] = p.count, b[k] = p.place;
            sum += p.count;
        }
        long long incl = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long u = __shfl_up_sync(kFullMask, incl, d);
            if (lane >= d) incl += u;
        }
        if (lane == 31) s_warp[turn][warp] = incl;
        __syncthreads();
        long long parts = s_warp[turn][lane & (kPagedWarps - 1)];
#pragma unroll
        for (int d = 1; d < kPagedWarps; d <<= 1) {
            const long long u = __shfl_up_sync(kFullMask, parts, d);
            if ((lane & (kPagedWarps - 1)) >= d) parts += u;
        }
        const long long ahead = __shfl_sync(kFullMask, parts, (warp - 1) & 31);
        long long end = base + (warp > 0 ? ahead : 0) + incl - sum;
        base += __shfl_sync(kFullMask, parts, kPagedWarps - 1);
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
            end += a[k];
            if (r + k >= rows) continue;
            out.ends[r + k] = static_cast<uint32_t>(end < INT32_MAX ? end : INT32_MAX);
            out.places[r + k] = b[k];
        }
    }
    __syncthreads();
}

// First row in [lo, hi) whose end is above g; hi if none.
__device__ __forceinline__ unsigned row_of(const uint32_t *ends, unsigned lo, unsigned hi, unsigned g)
{
    while (lo < hi) {
        const unsigned mid = (lo + hi) >> 1;
        if (ends[mid] > g) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}
// The same over [lo, hi) by a whole warp: 32 probes a step.
__device__ __forceinline__ unsigned warp_row_of(const uint32_t *ends, unsigned lo, unsigned hi, unsigned g)
{
    const unsigned lane = threadIdx.x & 31;
    while (lo < hi) {
        const unsigned step = (hi - lo + 31) / 32, at = lo + lane * step;
        const unsigned above = __ballot_sync(kFullMask, at >= hi || ends[at] > g);
        const unsigned k = above == 0 ? 32 : __ffs(above) - 1;   // the first probe above; the one before it is not
        if (k < 32 && lo + k * step < hi) hi = lo + k * step;
        if (k > 0) lo = lo + (k - 1) * step + 1;
    }
    return lo;
}

template <class Count>
__global__ void __launch_bounds__(kPagedThreads) row_ends_kernel(Count count, unsigned rows, Ends out)
{
    scan_rows(count, rows, out);
}

// IN_SHARED: the block scans the counts into its own shared memory; else
// row_ends_kernel has left them in `scratch`.
template <bool IN_SHARED, class Count>
__device__ __forceinline__ Ends row_ends(const Count &count, unsigned rows, const Ends &scratch)
{
    extern __shared__ uint32_t s_rows[];
    if (!IN_SHARED) return scratch;
    const Ends e{s_rows, reinterpret_cast<int32_t *>(s_rows + rows)};
    scan_rows(count, rows, e);
    return e;
}

// store(c, g, load(c, g)) with c = of_row(row, the row's first output) for the
// outputs 0 .. total, dealt to the warps of the grid a chunk of neighbours at a
// time; row == rows past the last one.  A chunk of few rows goes row by row,
// with no search and one c for a run; one of many rows (a decode step brings
// one output a row, or none) searches for every output's.
template <int CHUNK, class OfRow, class Load, class Store>
__device__ __forceinline__ void each_output(const Ends &e, unsigned rows, unsigned total, OfRow of_row, Load load, Store store)
{
    constexpr unsigned kAtOnce = 4, kFewRows = 4;
    const unsigned lane = threadIdx.x & 31;
    const unsigned warps = gridDim.x * kPagedWarps;
    // Fewer to a chunk where that gives every warp one.
    const unsigned share = (total / warps + 32) / 32 * 32, chunk = share > CHUNK ? CHUNK : share;
    const auto start_of = [&](unsigned r) { return r > 0 ? e.ends[r - 1] : 0u; };
    for (unsigned g0 = (blockIdx.x * kPagedWarps + (threadIdx.x >> 5)) * chunk; g0 < total; g0 += warps * chunk) {
        const unsigned g1 = total - g0 < chunk ? total : g0 + chunk;
        const unsigned lo = warp_row_of(e.ends, 0, rows, g0);
        const unsigned hi = lo < rows && e.ends[lo] >= g1 ? lo : warp_row_of(e.ends, lo, rows, g1 - 1);
        if (hi - lo < kFewRows) {
            for (unsigned r = lo; r <= hi; ++r) {
                const unsigned start = start_of(r), end = r < rows && e.ends[r] < g1 ? e.ends[r] : g1;
                const auto c = of_row(r, start);
                for (unsigned g = (start > g0 ? start : g0) + lane; g < end; g += 32 * kAtOnce) {
                    decltype(load(c, 0)) v[kAtOnce];
#pragma unroll
                    for (unsigned u = 0; u < kAtOnce; ++u)
                        if (g + 32 * u < end) v[u] = load(c, g + 32 * u);
#pragma unroll
                    for (unsigned u = 0; u < kAtOnce; ++u)
                        if (g + 32 * u < end) store(c, g + 32 * u, v[u]);
                }
            }
        } else {
            for (unsigned g = g0 + lane; g < g1; g += 32) {
                const unsigned r = row_of(e.ends, lo, hi, g);
                const auto c = of_row(r, start_of(r));
                store(c, g, load(c, g));
            }
        }
    }
}

__device__ __forceinline__ int clamp_free(const int32_t *free_count, int pool)
{
    const int f = *free_count;
    return f < 0 ? 0 : (f < pool ? f : pool);
}

template <bool IN_SHARED>
__global__ void __launch_bounds__(kPagedThreads, 2)
extend_kernel(int32_t *__restrict__ table, size_t stride, unsigned rows, ExtendCount count,
              const int32_t *__restrict__ pages, int pool, const int32_t *__restrict__ free_count,
              uint8_t *__restrict__ granted, int32_t *__restrict__ left, Ends scratch)
{
    const unsigned free = clamp_free(free_count, pool);
    const Ends e = row_ends<IN_SHARED>(count, rows, scratch);
    // Rows are served in order while the pool lasts: those whose end is within it.
    const unsigned served = warp_row_of(e.ends, 0, rows, free);
    const unsigned total = served > 0 ? e.ends[served - 1] : 0;
    const unsigned tid = blockIdx.x * kPagedThreads + threadIdx.x, threads = gridDim.x * kPagedThreads;
    for (unsigned r = tid; r < rows; r += threads) {
        const unsigned end = e.ends[r];
        const bool needs = end == INT32_MAX ? count.part(count.cached[r], count.fresh[r]).count != 0
                                            : end != (r > 0 ? e.ends[r - 1] : 0u);
        granted[r] = e.places[r] >= 0 && (!needs || end <= free);
    }
    if (tid == 0) *left = free - total;
    each_output<kMoveChunk>(e, rows, total,
                            [&](unsigned r, unsigned start) {
                                return r * static_cast<long long>(stride) + e.places[r] - start;
                            },
                            [&](long long, unsigned g) { return __ldcs(pages + (free - 1 - g)); },
                            [&](long long row, unsigned g, int id) { table[row + g] = id; });
}

template <bool IN_SHARED>
__global__ void __launch_bounds__(kPagedThreads, 2)
slot_kernel(const int32_t *__restrict__ table, size_t stride, unsigned rows, int width, SlotCount count, Pages page,
            unsigned tokens, int32_t *__restrict__ starts, long long *__restrict__ slots, int32_t *__restrict__ positions,
            int32_t *__restrict__ row_ids, Ends scratch)
{
    const Ends e = row_ends<IN_SHARED>(count, rows, scratch);
    const unsigned tid = blockIdx.x * kPagedThreads + threadIdx.x, threads = gridDim.x * kPagedThreads;
    for (unsigned r = tid; r < rows; r += threads) starts[r + 1] = static_cast<int32_t>(e.ends[r]);
    if (tid == 0) starts[0] = 0;
    struct Row {
        const int32_t *entries;
        long long before;         // position of output g: before + g
        int id;                   // -1: past the last row
    };
    struct Place {
        int pos, entry, offset;   // -1: none
    };
    const auto row_at = [&](unsigned r, unsigned start) {
        return r < rows ? Row{table + static_cast<size_t>(r) * stride, static_cast<long long>(e.places[r]) - start,
                              static_cast<int>(r)}
                        : Row{nullptr, 0, -1};
    };
    const auto place_of = [&](const Row &row, unsigned g) {
        Place p{-1, -1, 0};
        const long long at = row.before + g;
        if (row.id < 0 || at < 0 || at > INT32_MAX) return p;
        p.pos = static_cast<int>(at);
        const uint32_t b = page.div(p.pos);
        p.offset = static_cast<int>(p.pos - b * page.page);
        if (b < static_cast<uint32_t>(width)) p.entry = __ldg(row.entries + b);
        return p;
    };
    each_output<kSlotChunk>(e, rows, tokens, row_at, place_of, [&](const Row &row, unsigned g, const Place &p) {
        __stcs(slots + g, p.entry < 0 ? -1ll : static_cast<long long>(p.entry) * page.page + p.offset);
        __stcs(positions + g, p.pos);
        __stcs(row_ids + g, row.id);
    });
}

template <bool IN_SHARED>
__global__ void __launch_bounds__(kPagedThreads, 2)
release_kernel(const int32_t *__restrict__ table, size_t stride, unsigned rows, ReleaseCount count,
               int32_t *__restrict__ pages, int pool, const int32_t *__restrict__ free_count,
               int32_t *__restrict__ left, Ends scratch)
{
    const unsigned free = clamp_free(free_count, pool);
    const Ends e = row_ends<IN_SHARED>(count, rows, scratch);
    const unsigned served = warp_row_of(e.ends, 0, rows, pool - free);   // rows whose pages fit the pool array
    const unsigned total = served > 0 ? e.ends[served - 1] : 0;
    if (blockIdx.x == 0 && threadIdx.x == 0) *left = free + total;
    each_output<kMoveChunk>(e, rows, total,
                            [&](unsigned r, unsigned start) { return r * static_cast<long long>(stride) - start; },
                            [&](long long row, unsigned g) { return __ldcs(table + row + g); },
                            [&](long long, unsigned g, int id) { pages[free + g] = id; });
}

// Blocks for `most` output elements at the most.
unsigned paged_blocks(unsigned long long most, const Workspace &ws)
{
    const unsigned long long b = (most + kPagedThreads - 1) / kPagedThreads;
    const unsigned long long cap = static_cast<unsigned long long>(ws.num_sms) * 2;
    return static_cast<unsigned>(b < 1 ? 1 : (b < cap ? b : cap));
}

// Where the rows are too many for a block's shared memory, the launch that
// scans them into `scratch`.
template <class Count>
cudaError_t prepare_ends(const Count &count, unsigned rows, const Ends &scratch, size_t *shared_bytes, cudaStream_t s)
{
    *shared_bytes = 0;
    if (rows <= kPagedSharedRows) {
        *shared_bytes = static_cast<size_t>(rows) * 2 * sizeof(int32_t);
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
    const ExtendCount count{cached, fresh, Pages(page), width};
    const Ends ends{reinterpret_cast<uint32_t *>(scratch), scratch + rows};
    size_t shared = 0;
    cudaError_t e = prepare_ends(count, rows, ends, &shared, s);
    if (e != cudaSuccess) return e;
    unsigned long long most = static_cast<unsigned long long>(rows) * width;
    if (most > static_cast<unsigned long long>(pool)) most = pool;
    const unsigned blocks = paged_blocks(most, ws);
    if (rows <= kPagedSharedRows)
        extend_kernel<true><<<blocks, kPagedThreads, shared, s>>>(table, stride, rows, count, pages, pool, free_count,
                                                                  granted, left, ends);
    else
        extend_kernel<false><<<blocks, kPagedThreads, 0, s>>>(table, stride, rows, count, pages, pool, free_count,
                                                              granted, left, ends);
    return cudaGetLastError();
}

cudaError_t launch_slot_map(const int32_t *table, size_t stride, int rows, int width, const int32_t *cached,
                            const int32_t *fresh, const uint8_t *granted, int page, int tokens, int32_t *starts,
                            int64_t *slots, int32_t *positions, int32_t *row_ids, int32_t *scratch,
                            const Workspace &ws, cudaStream_t s)
{
    const SlotCount count{cached, fresh, granted};
    const Ends ends{reinterpret_cast<uint32_t *>(scratch), scratch + rows};
    size_t shared = 0;
    cudaError_t e = prepare_ends(count, rows, ends, &shared, s);
    if (e != cudaSuccess) return e;
    const unsigned blocks = paged_blocks(static_cast<unsigned long long>(tokens), ws);
    long long *out = reinterpret_cast<long long *>(slots);
    if (rows <= kPagedSharedRows)
        slot_kernel<true><<<blocks, kPagedThreads, shared, s>>>(table, stride, rows, width, count, Pages(page), tokens,
                                                                starts, out, positions, row_ids, ends);
    else
        slot_kernel<false><<<blocks, kPagedThreads, 0, s>>>(table, stride, rows, width, count, Pages(page), tokens,
                                                            starts, out, positions, row_ids, ends);
    return cudaGetLastError();
}

cudaError_t launch_block_table_release(const int32_t *table, size_t stride, int rows, int width,
                                       const int32_t *cached, const uint8_t *done, int page, int32_t *pages, int pool,
                                       const int32_t *free_count, int32_t *left, int32_t *scratch,
                                       const Workspace &ws, cudaStream_t s)
{
    const ReleaseCount count{cached, done, Pages(page), width};
    const Ends ends{reinterpret_cast<uint32_t *>(scratch), scratch + rows};
    size_t shared = 0;
    cudaError_t e = prepare_ends(count, rows, ends, &shared, s);
    if (e != cudaSuccess) return e;
    unsigned long long most = static_cast<unsigned long long>(rows) * width;
    if (most > static_cast<unsigned long long>(pool)) most = pool;
    const unsigned blocks = paged_blocks(most, ws);
    if (rows <= kPagedSharedRows)
        release_kernel<true><<<blocks, kPagedThreads, shared, s>>>(table, stride, rows, count, pages, pool,
                                                                   free_count, left, ends);
    else
        release_kernel<false><<<blocks, kPagedThreads, 0, s>>>(table, stride, rows, count, pages, pool, free_count,
                                                               left, ends);
    return cudaGetLastError();
}

}  // namespace devscan
