// Tokens sorted by expert and back (sm_103a): every token goes to `choices`
// experts, and a pair (token, choice) to a place among its expert's rows.
//
// sort     : the stable counting sort of the pairs by expert -- lpnh.cn
//            "并行扫描" section 4.2's counts per digit, a prefix over them and a
//            scatter, with the expert as the only digit.  A segment of rows per
//            expert, each rounded up to a multiple of `align`.
// dispatch : xs[place(t, k)] = x[t]
// combine  : y[t] = sum over k of w(t, k) ys[place(t, k)]
// and the gradient of combine: dys[place] = w dy[t], dw = <dy[t], ys[place]>.
// The gradient of dispatch is combine without weights.
#include "cluster.cuh"
#include "convert.cuh"
#include "grid_sync.cuh"
#include "launch.h"

namespace devscan {
namespace {

// ---------------------------------------------------------------------------
// Sort.  One cluster of up to sixteen blocks: its blocks take equal runs of the
// pairs, and their warps equal runs of those, so that the order of warps is
// the order of pairs.  Every warp counts its pairs per expert in shared memory;
// a column of counts is scanned over the warps by one thread, over the blocks
// through distributed shared memory, and over the experts by the block.  Then
// each warp goes through its pairs again: lanes with the same expert find each
// other by a ballot per bit of the id, their ranks are counted from the mask,
// and the warp's counter moves on.  Ids come four per lane at once; where a
// warp has no more than those, they are read once.  `order` is put together in
// shared memory and written an expert's run at a time: written pair by pair, 32
// sectors per instruction, it was what bounded the call.  (Where a block's
// pairs do not fit there it is written so all the same.)  No scratch, no global
// atomics, one launch.
// Measured (device time): 128 pairs of 64 experts 2.9 us, of which the launch is
// two thirds; 4,096 pairs 8; 131,072 pairs of 256 experts 15.6, at 280 instructions
// per 32 pairs on sixteen SMs, which is what bounds it (24 with the match
// instruction on eight, 21 with ballots, 14 to 16 with order from shared memory
// on sixteen); a million pairs 58.  A sort over all SMs would need scratch or a
// second launch.
// ---------------------------------------------------------------------------
constexpr int kSortMostBlocks = 16;
constexpr int kSortWarps = 32, kSortFewWarps = 8;   // of a block; few, where there are few pairs and experts
constexpr int kSortAtOnce = 4;   // ids of a lane
constexpr size_t kSortPairsPerBlock = 4096;   // from where another block is worth it
constexpr size_t kSortDirect = 2048;          // pairs of a block that are written one by one
constexpr int kSortSmem = 224 << 10;

template <typename Id, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, 1) expert_sort_kernel(const __grid_constant__ ExpertSortCall p)
{
    constexpr int kThreads = 32 * WARPS;
    extern __shared__ unsigned s_counts[];            // [warp][expert], then by expert:
    unsigned *const s_total = s_counts + WARPS * p.experts;
    unsigned *const s_base = s_total + p.experts;     // first row of a segment
    unsigned *const s_filled = s_base + p.experts;    // behind the last row with a pair
    unsigned *const s_here = s_filled + p.experts;    // first row of this block's pairs
    unsigned *const s_local = s_here + p.experts;     // their first place in s_order
    unsigned short *const s_order = reinterpret_cast<unsigned short *>(s_local + p.experts);   // the block's pairs by expert
    __shared__ unsigned s_warp[WARPS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const unsigned rank = cluster_rank(), blocks = gridDim.x;
    const bool local = p.local;   // the block's pairs fit in s_order
    const Id *ids = static_cast<const Id *>(p.ids);
    const unsigned experts = static_cast<unsigned>(p.experts);
    const unsigned each = (p.pairs + blocks * kThreads - 1) / (blocks * kThreads) * 32;   // pairs of a warp
    const unsigned begin = (rank * WARPS + warp) * each;
    const unsigned end = begin < p.pairs ? (p.pairs - begin < each ? p.pairs : begin + each) : begin;
    unsigned *const mine = s_counts + warp * experts;
    unsigned e[kSortAtOnce];   // experts of pairs i0 + 32 j + lane; `experts` where there is none
    auto load = [&](unsigned i0) {
        Id id[kSortAtOnce];
#pragma unroll
        for (int j = 0; j < kSortAtOnce; ++j) {
            const unsigned i = i0 + 32 * j + lane;
            id[j] = i < end ? ids[i] : static_cast<Id>(-1);
        }
#pragma unroll
        for (int j = 0; j < kSortAtOnce; ++j)
            e[j] = id[j] >= 0 && id[j] < static_cast<Id>(experts) ? static_cast<unsigned>(id[j]) : experts;
    };

    allow_dependent_launch();   // dispatch, which waits for this launch's end
    for (unsigned k = lane; k < experts; k += 32) mine[k] = 0;
    __syncwarp();
    const bool once = each <= 32 * kSortAtOnce;
    unsigned used = 0;
    // One copy of the loop for counting and for placing: this is code that runs
    // a few times, and fetching it for the first time is what small calls pay.
#pragma unroll 1
    for (int placing = 0; placing < 2; ++placing) {
#pragma unroll 1
        for (unsigned i0 = begin; i0 < end; i0 += 32 * kSortAtOnce) {
            if (!placing || !once) load(i0);
            if (!placing) {
#pragma unroll
                for (int j = 0; j < kSortAtOnce; ++j)
                    if (e[j] < experts) atomicAdd(&mine[e[j]], 1u);
                continue;
            }
            unsigned all_same[kSortAtOnce];
#pragma unroll
            for (int j = 0; j < kSortAtOnce; ++j) all_same[j] = kFullMask;
#pragma unroll 1
            for (unsigned bit = 1; bit <= experts; bit *= 2)
#pragma unroll
                for (int j = 0; j < kSortAtOnce; ++j) {
                    const unsigned with = __ballot_sync(kFullMask, (e[j] & bit) != 0);
                    all_same[j] &= (e[j] & bit) != 0 ? with : ~with;
                }
#pragma unroll
            for (int j = 0; j < kSortAtOnce; ++j) {
                const unsigned i = i0 + 32 * j + lane, same = all_same[j];
                if (i0 + 32 * j >= end) break;
                const unsigned ahead = __popc(same & ((1u << lane) - 1u));
                const unsigned place = e[j] < experts ? mine[e[j]] + ahead : p.rows;
                __syncwarp();
                if (e[j] < experts && ahead == 0) mine[e[j]] += __popc(same);
                __syncwarp();
                if (i < end) p.places[i] = place < p.rows ? static_cast<int32_t>(place) : -1;
                if (local) {
                    if (e[j] < experts) s_order[place - s_here[e[j]] + s_local[e[j]]] = static_cast<unsigned short>(i - rank * WARPS * each);
                } else if (place < p.rows) {
                    p.order[place] = static_cast<int32_t>(i);
                }
            }
        }
        if (placing) break;
        __syncthreads();
        // a thread has an expert's counts; there are no more experts than threads
        const bool column = static_cast<unsigned>(tid) < experts;
        unsigned total = 0, before = 0;
#pragma unroll 8
        for (int w = 0; w < WARPS; ++w) total += column ? s_counts[w * experts + tid] : 0u;
        unsigned all = total;
        if (column) s_total[tid] = total;
        if (blocks > 1) {
            cluster_sync();   // the totals are there
            all = 0;
#pragma unroll 4
            for (unsigned q = 0; q < blocks; ++q) {
                const unsigned theirs = column ? ld_cluster(cluster_addr(&s_total[tid], q)) : 0u;
                before += q < rank ? theirs : 0u;
                all += theirs;
            }
        }
        // the segments' first rows, and the block's own: scans over the experts
        const unsigned room = (all + p.align - 1) / p.align * p.align;
        const unsigned base = block_excl_scan<kThreads>(room, s_warp, tid, used);
        unsigned place0 = 0;
        if (local) {
            unsigned in_block = 0;
            __syncthreads();
            place0 = block_excl_scan<kThreads>(total, s_warp, tid, in_block);
        }
        if (column) {
            s_base[tid] = base;
            s_filled[tid] = base + all;
            s_here[tid] = base + before;
            s_local[tid] = place0;
            unsigned upto = base + before;
#pragma unroll 1
            for (int w0 = 0; w0 < WARPS; w0 += 8) {
                unsigned count[8];
#pragma unroll
                for (int w = 0; w < 8; ++w) count[w] = s_counts[(w0 + w) * experts + tid];
#pragma unroll
                for (int w = 0; w < 8; ++w) {
                    s_counts[(w0 + w) * experts + tid] = upto;
                    upto += count[w];
                }
            }
            if (rank == 0) p.starts[tid] = static_cast<int32_t>(base), p.counts[tid] = static_cast<int32_t>(all);
        }
        if (rank == 0 && tid == 0) p.starts[experts] = static_cast<int32_t>(used);
        __syncthreads();
    }
    if (local) {
        __syncthreads();
        for (unsigned k = warp; k < experts; k += WARPS)
            for (unsigned i = lane; i < s_total[k]; i += 32) {
                const unsigned row = s_here[k] + i;
                if (row < p.rows) p.order[row] = static_cast<int32_t>(rank * WARPS * each + s_order[s_local[k] + i]);
            }
    }
    // rows without a pair: up to the end of their segment, and behind the last one
    for (unsigned e = rank * WARPS + warp; e < experts; e += blocks * WARPS) {
        unsigned to = e + 1 < experts ? s_base[e + 1] : used;
        to = to < p.rows ? to : p.rows;
        for (unsigned r = s_filled[e] + lane; r < to; r += 32) p.order[r] = kOrderPadding;
    }
    for (unsigned r = used + rank * kThreads + tid; r < p.rows; r += blocks * kThreads) p.order[r] = kOrderBehind;
    if (blocks > 1) cluster_sync();   // nobody leaves while its totals may be read
}

// ---------------------------------------------------------------------------
// Dispatch.  A warp takes a token's run of 32 * U vectors, reads it once and
// writes it to each of the token's places, so that x is read once and not once
// per choice; the warps behind those look through `order`, eight rows each, for
// rows of padding and clear them.  Every warp is a block: it ends, and makes room
// for the next, when its own writes are out (16,384 x 8 rows of 4 KB: 115 us
// with four warps to a block, 109 with one, 6.1 TB/s).  Rows that are not made
// of 16 bytes move in smaller pieces; an SM then needs more warps than blocks.
// ---------------------------------------------------------------------------
constexpr int kMoveWarps = 4;   // of a block that combines

// The rows among order[r0 .. r0 + kPadRows) that are padding, a bit each.
constexpr int kPadRows = 8;
__device__ __forceinline__ unsigned padding_rows(const int32_t *order, unsigned r0, unsigned rows, int lane)
{
    const unsigned r = r0 + lane;
    return __ballot_sync(kFullMask, lane < kPadRows && r < rows && order[r] == kOrderPadding);
}

template <typename V, int U, int WARPS>
__global__ void __launch_bounds__(32 * WARPS) expert_dispatch_kernel(const __grid_constant__ ExpertMoveCall p, unsigned vectors,
                                                                     unsigned runs)
{
    wait_primary_grid();   // a sort before this lets it start early
    const int lane = threadIdx.x & 31;
    const size_t item = static_cast<size_t>(blockIdx.x) * WARPS + (threadIdx.x >> 5);
    const size_t moves = static_cast<size_t>(p.tokens) * runs;
    if (item < moves) {
        const unsigned t = static_cast<unsigned>(item / runs), run = static_cast<unsigned>(item % runs);
        const V *from = reinterpret_cast<const V *>(static_cast<const char *>(p.from) + t * p.from_stride);
        const unsigned v0 = run * (32 * U) + lane;
        V v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (v0 + 32 * u < vectors) v[u] = __ldcs(from + v0 + 32 * u);
        const int32_t *places = p.places + static_cast<size_t>(t) * p.choices;
        for (int k0 = 0; k0 < p.choices; k0 += 32) {
            const int here = k0 + lane < p.choices ? places[k0 + lane] : -1;
            const int many = min(32, p.choices - k0);
            for (int k = 0; k < many; ++k) {
                const unsigned place = static_cast<unsigned>(__shfl_sync(kFullMask, here, k));
                if (place >= p.rows) continue;
                V *to = reinterpret_cast<V *>(static_cast<char *>(p.to) + place * p.to_stride);
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (v0 + 32 * u < vectors) __stcs(to + v0 + 32 * u, v[u]);
            }
        }
        return;
    }
    const size_t r0 = (item - moves) * kPadRows;
    if (p.order == nullptr || r0 >= p.rows) return;
    for (unsigned found = padding_rows(p.order, static_cast<unsigned>(r0), p.rows, lane); found != 0; found &= found - 1) {
        V *to = reinterpret_cast<V *>(static_cast<char *>(p.to) + (r0 + __ffs(found) - 1) * p.to_stride);
        for (unsigned i = lane; i < vectors; i += 32) to[i] = V{};
    }
}

template <typename V, int U, int WARPS = sizeof(V) == 16 ? 1 : 4>
cudaError_t dispatch(const ExpertMoveCall &call, cudaStream_t s)
{
    const unsigned vectors = static_cast<unsigned>(call.row_bytes / sizeof(V));
    const unsigned runs = (vectors + 32 * U - 1) / (32 * U);
    const size_t items = static_cast<size_t>(call.tokens) * runs + (call.order != nullptr ? (call.rows + kPadRows - 1u) / kPadRows : 0);
    if (items == 0) return cudaSuccess;
    const size_t blocks = (items + WARPS - 1) / WARPS;
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    return launch_dependent(expert_dispatch_kernel<V, U, WARPS>, static_cast<unsigned>(blocks), 32 * WARPS, s, call, vectors, runs);
}

// ---------------------------------------------------------------------------
// Combine.  A warp takes 32 * V columns of a token and adds the rows of its
// choices in their order, eight loads in flight, in fp32; one rounding.  (Where
// rows are not made of 16 bytes, U pieces of V values to a lane.)  Bound
// by the two loads behind each other, of places and of rows: 32 warps to an SM
// and small blocks (8,191 x 6 rows of 4 KB: 47 us with eight warps to a block
// and 24 to an SM, 40 so, 5.8 TB/s).
// ---------------------------------------------------------------------------
constexpr int kAtOnce = 8;   // choices whose rows are in flight together

template <typename T, int V, int U>
__global__ void __launch_bounds__(32 * kMoveWarps, 8) expert_combine_kernel(const __grid_constant__ ExpertCombineCall p,
                                                                         unsigned runs)
{
    using R = typename Raw<T, V>::type;
    const int lane = threadIdx.x & 31;
    const size_t item = static_cast<size_t>(blockIdx.x) * kMoveWarps + (threadIdx.x >> 5);
    if (item >= static_cast<size_t>(p.tokens) * runs) return;
    const unsigned t = static_cast<unsigned>(item / runs), run = static_cast<unsigned>(item % runs);
    constexpr int kRows = U > 1 ? kAtOnce / 2 : kAtOnce;   // whose pieces are in flight together
    unsigned c[U];
    bool live[U];   // a whole number of lanes is
#pragma unroll
    for (int u = 0; u < U; ++u) {
        c[u] = ((run * U + u) * 32 + lane) * V;
        live[u] = c[u] < p.width;
    }
    const T *y = static_cast<const T *>(p.y);
    const size_t pair0 = static_cast<size_t>(t) * p.choices;
    float sum[U][V] = {};
    for (int k0 = 0; k0 < p.choices; k0 += kRows) {
        const bool have = lane < kRows && k0 + lane < p.choices;
        const int place_here = have ? p.places[pair0 + k0 + lane] : -1;
        const float weight_here = have && p.weights != nullptr ? p.weights[pair0 + k0 + lane] : 1.0f;
        R r[kRows][U];
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
            const unsigned place = static_cast<unsigned>(__shfl_sync(kFullMask, place_here, j));
            const T *row = y + place * p.y_stride;
            if (place >= p.rows) continue;
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (live[u]) r[j][u] = *reinterpret_cast<const R *>(row + c[u]);
        }
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
            const unsigned place = static_cast<unsigned>(__shfl_sync(kFullMask, place_here, j));
            const float w = __shfl_sync(kFullMask, weight_here, j);
            if (place >= p.rows) continue;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (!live[u]) continue;
                float v[V];
                unpack<T, V>(r[j][u], v);
#pragma unroll
                for (int i = 0; i < V; ++i) sum[u][i] = fmaf(w, v[i], sum[u][i]);
            }
        }
    }
    T *out = static_cast<T *>(p.out) + t * p.out_stride;
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (live[u]) *reinterpret_cast<R *>(out + c[u]) = pack<T, V>(sum[u]);
}

// ---------------------------------------------------------------------------
// The gradient of combine.  A block of four warps takes a token: its row of
// gradients is read once per eight choices, each choice's row of y gives a
// piece of the weight's gradient, and the row's gradient is written.  The
// pieces are added lane, warp, block, in a fixed order.  Bound by memory latency:
// 8,191 x 6 rows of 4 KB 67 us right after combine, which leaves part of y in L2
// (77 with streaming loads, 85 with streaming stores too), 24 warps to an SM.
// ---------------------------------------------------------------------------
constexpr int kBackWarps = 4;

template <typename T, int V, int U>
__global__ void __launch_bounds__(32 * kBackWarps, U > 1 ? 4 : 6) expert_combine_backward_kernel(
    const __grid_constant__ ExpertCombineBackwardCall p)
{
    using R = typename Raw<T, V>::type;
    __shared__ float s_sum[kBackWarps][kAtOnce];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (blockIdx.x >= p.tokens) {   // rows of padding
        const size_t r0 = (static_cast<size_t>(blockIdx.x - p.tokens) * kBackWarps + warp) * kPadRows;
        if (r0 >= p.rows) return;
        for (unsigned found = padding_rows(p.order, static_cast<unsigned>(r0), p.rows, lane); found != 0;
             found &= found - 1) {
            T *to = static_cast<T *>(p.grad_y) + (r0 + __ffs(found) - 1) * p.grad_y_stride;
            for (unsigned c = lane * V; c < p.width; c += 32 * V) *reinterpret_cast<R *>(to + c) = R{};
        }
        return;
    }
    const unsigned t = blockIdx.x;
    const T *grad = static_cast<const T *>(p.grad) + t * p.grad_stride;
    const size_t pair0 = static_cast<size_t>(t) * p.choices;
    for (int k0 = 0; k0 < p.choices; k0 += kAtOnce) {
        const bool have = lane < kAtOnce && k0 + lane < p.choices;
        const int place_here = have ? p.places[pair0 + k0 + lane] : -1;
        const float weight_here = have && p.weights != nullptr ? p.weights[pair0 + k0 + lane] : 1.0f;
        unsigned place[kAtOnce];
        float weight[kAtOnce], sum[kAtOnce] = {};
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            place[j] = static_cast<unsigned>(__shfl_sync(kFullMask, place_here, j));
            weight[j] = __shfl_sync(kFullMask, weight_here, j);
        }
        constexpr unsigned kAcross = 32 * kBackWarps * V;   // columns that the block has at once
        for (unsigned c0 = threadIdx.x * V; c0 < p.width; c0 += U * kAcross) {
            R g[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (c0 + u * kAcross < p.width) g[u] = *reinterpret_cast<const R *>(grad + c0 + u * kAcross);
            constexpr int kRows = U > 1 ? kAtOnce / 2 : kAtOnce;   // whose pieces are in flight together
#pragma unroll
            for (int j0 = 0; j0 < kAtOnce; j0 += kRows) {
                R r[kRows][U];
                if (p.grad_weights != nullptr)
#pragma unroll
                    for (int j = 0; j < kRows; ++j)
                        if (place[j0 + j] < p.rows)
#pragma unroll
                            for (int u = 0; u < U; ++u)
                                if (c0 + u * kAcross < p.width)
                                    r[j][u] = *reinterpret_cast<const R *>(static_cast<const T *>(p.y) + place[j0 + j] * p.y_stride + c0 + u * kAcross);
#pragma unroll
                for (int j = 0; j < kRows; ++j) {
                    if (place[j0 + j] >= p.rows) continue;
                    T *to = static_cast<T *>(p.grad_y) + place[j0 + j] * p.grad_y_stride + c0;
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        if (c0 + u * kAcross >= p.width) continue;
                        float gv[V], v[V];
                        unpack<T, V>(g[u], gv);
                        if (p.grad_weights != nullptr) {
                            unpack<T, V>(r[j][u], v);
#pragma unroll
                            for (int i = 0; i < V; ++i) sum[j0 + j] = fmaf(gv[i], v[i], sum[j0 + j]);
                        }
#pragma unroll
                        for (int i = 0; i < V; ++i) v[i] = weight[j0 + j] * gv[i];
                        *reinterpret_cast<R *>(to + u * kAcross) = pack<T, V>(v);
                    }
                }
            }
        }
        if (p.grad_weights == nullptr) continue;
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j)
#pragma unroll
            for (int d = 16; d >= 1; d >>= 1) sum[j] += __shfl_xor_sync(kFullMask, sum[j], d);
        __syncthreads();   // the sums before have been read
        if (lane == 0)
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) s_sum[warp][j] = sum[j];
        __syncthreads();
        if (warp == 0 && have) {
            float all = 0.0f;
#pragma unroll
            for (int w = 0; w < kBackWarps; ++w) all += s_sum[w][lane];
            p.grad_weights[pair0 + k0 + lane] = static_cast<unsigned>(place_here) < p.rows ? all : 0.0f;
        }
    }
}

template <typename Id, int WARPS> cudaError_t sort(ExpertSortCall call, cudaStream_t s)
{
    static std::atomic<unsigned long long> done, wide;
    auto *kernel = expert_sort_kernel<Id, WARPS>;
    cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void *>(kernel), kSortSmem, done);
    if (e != cudaSuccess) return e;
    unsigned blocks = 1;
    while (blocks < kSortMostBlocks && static_cast<size_t>(call.pairs) > blocks * kSortPairsPerBlock) blocks *= 2;
    if (blocks > 8) {   // more than the portable size
        int dev = 0;
        if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
        if ((wide.load() >> (dev & 63) & 1) == 0) {
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e != cudaSuccess) return e;
            wide.fetch_or(1ull << (dev & 63));
        }
    }
    const size_t threads = 32 * WARPS, counts = (WARPS + 5) * static_cast<size_t>(call.experts) * sizeof(unsigned);
    const size_t each = (static_cast<size_t>(call.pairs) + blocks * threads - 1) / (blocks * threads) * threads;   // a block's
    call.local = each > kSortDirect && each <= 65536 && counts + 2 * each <= static_cast<size_t>(kSortSmem);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = counts + (call.local ? 2 * each : 0);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = blocks;   // one cluster spans the grid
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, call);
}

bool rows_of(size_t unit, const void *p, size_t stride, size_t width, size_t size)
{
    return reinterpret_cast<uintptr_t>(p) % unit == 0 && stride * size % unit == 0 && width * size % unit == 0;
}

template <typename T, int V, int U>
cudaError_t combine(const ExpertCombineCall &call, cudaStream_t s)
{
    const unsigned runs = (call.width + 32 * V * U - 1) / (32 * V * U);
    const size_t blocks = (static_cast<size_t>(call.tokens) * runs + kMoveWarps - 1) / kMoveWarps;
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    expert_combine_kernel<T, V, U><<<static_cast<unsigned>(blocks), 32 * kMoveWarps, 0, s>>>(call, runs);
    return cudaGetLastError();
}
template <typename T>
cudaError_t combine_any(const ExpertCombineCall &call, cudaStream_t s)
{
    const auto made_of = [&](size_t unit) {
        return rows_of(unit, call.y, call.y_stride, call.width, sizeof(T)) && rows_of(unit, call.out, call.out_stride, call.width, sizeof(T));
    };
    if (made_of(16)) return combine<T, 16 / sizeof(T), 1>(call, s);
    return made_of(2 * sizeof(T)) ? combine<T, 2, 4>(call, s) : combine<T, 1, 4>(call, s);
}

template <typename T, int V, int U>
cudaError_t combine_backward(const ExpertCombineBackwardCall &call, cudaStream_t s)
{
    const size_t blocks = static_cast<size_t>(call.tokens) +
                          (call.order != nullptr ? (call.rows + kPadRows * kBackWarps - 1u) / (kPadRows * kBackWarps) : 0);
    if (blocks == 0) return cudaSuccess;
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    expert_combine_backward_kernel<T, V, U><<<static_cast<unsigned>(blocks), 32 * kBackWarps, 0, s>>>(call);
    return cudaGetLastError();
}
template <typename T>
cudaError_t combine_backward_any(const ExpertCombineBackwardCall &call, cudaStream_t s)
{
    const size_t w = call.width, n = sizeof(T);
    const auto made_of = [&](size_t unit) {
        return rows_of(unit, call.grad, call.grad_stride, w, n) && rows_of(unit, call.grad_y, call.grad_y_stride, w, n) &&
               (call.grad_weights == nullptr || rows_of(unit, call.y, call.y_stride, w, n));
    };
    if (made_of(16)) return combine_backward<T, 16 / sizeof(T), 1>(call, s);
    return made_of(2 * n) ? combine_backward<T, 2, 4>(call, s) : combine_backward<T, 1, 4>(call, s);
}

}  // namespace

cudaError_t launch_expert_sort(ExpertSortCall call, bool wide_ids, cudaStream_t s)
{
    constexpr size_t few_pairs = 32 * kSortFewWarps * kSortAtOnce;
    const bool few = call.pairs <= few_pairs && call.experts <= 32 * kSortFewWarps;
    if (wide_ids) return few ? sort<int64_t, kSortFewWarps>(call, s) : sort<int64_t, kSortWarps>(call, s);
    return few ? sort<int32_t, kSortFewWarps>(call, s) : sort<int32_t, kSortWarps>(call, s);
}

cudaError_t launch_expert_dispatch(const ExpertMoveCall &call, cudaStream_t s)
{
    const size_t all = reinterpret_cast<uintptr_t>(call.from) | reinterpret_cast<uintptr_t>(call.to) | call.row_bytes |
                       call.from_stride | call.to_stride;
    // Large calls move most per warp (16,384 x 8 rows of 4 KB: 118 us at 4 vectors a lane, 115 at 8), small ones
    // have the most warps (16 x 8 rows: 2.8 and 2.3 us at 4 and 1).
    if (all % 16 == 0) {
        const size_t lanes = static_cast<size_t>(call.tokens) * (call.row_bytes / 16);
        if (lanes >= size_t(1) << 20) return dispatch<uint4, 8>(call, s);
        return lanes >= size_t(1) << 17 ? dispatch<uint4, 4>(call, s) : dispatch<uint4, 1>(call, s);
    }
    if (all % 8 == 0) return dispatch<uint2, 8>(call, s);
    if (all % 4 == 0) return dispatch<unsigned, 8>(call, s);
    if (all % 2 == 0) return dispatch<unsigned short, 8>(call, s);
    return dispatch<unsigned char, 8>(call, s);
}

cudaError_t launch_expert_combine(ValueType type, const ExpertCombineCall &call, cudaStream_t s)
{
    if (type == ValueType::F32) return combine_any<float>(call, s);
    return type == ValueType::F16 ? combine_any<__half>(call, s) : combine_any<__nv_bfloat16>(call, s);
}

cudaError_t launch_expert_combine_backward(ValueType type, const ExpertCombineBackwardCall &call, cudaStream_t s)
{
    if (type == ValueType::F32) return combine_backward_any<float>(call, s);
    return type == ValueType::F16 ? combine_backward_any<__half>(call, s) : combine_backward_any<__nv_bfloat16>(call, s);
}

}  // namespace devscan
