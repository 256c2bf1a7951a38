// Token draw from logits with temperature, top-k, top-p and min-p (sm_103a).
//
// Every row is one discrete draw by an exponential race: with weights
// w_i = exp((x_i - max) / T) and given Exp(1) noise q_i, the smallest q_i / w_i
// (the largest w_i / q_i) falls on token i with probability w_i / sum w, for
// whatever set of tokens takes part.  So truncation only has to find that set.
// All three truncations keep a prefix of one order, logit descending and
// index ascending among equals:
//   top-k : the first k;
//   top-p : of those, tokens whose mass ahead is below p times their total;
//   min-p : tokens with w_i >= m (the largest logit has w = 1).
//
// One thread-block cluster draws one row, a slice of it per block; with rows
// enough to fill the GPU the cluster is one block.  A row is read from memory
// once, for its maximum (and, for top-p alone, its sum).  Where the slices are
// small (64 KB, two blocks per SM) that pass keeps them in shared memory; else
// it leaves the maximum of every group of four 16-byte chunks there, an index
// by which later passes read again, out of L2, only the groups that hold a
// token above their bound: a few hundred tokens of a row of 100,000.  The noise
// is read only where a token is kept.  A row without truncation takes one pass
// over logits and noise side by side.
//
// Selection has two forms.
//   Short list.  Every full warp's j-th largest lane maximum is taken, and the
//     least of them is a bound with at least j tokens per warp above it: for
//     j = ceil(k / warps) the first k are all at or above the bound.  Those
//     tokens (a few hundred) are collected and sorted by one block as 64-bit
//     keys (ordered logit bits above the complement of the index), and top-k,
//     top-p (a scan of the sorted weights) and min-p are cuts of the sorted
//     list.  top-p without top-k takes the same list if its mass reaches p
//     times the row's.
//   Histograms.  Where the list would be too long (a wide top-k, a flat row,
//     a tie of many tokens), the cut is bracketed by a histogram of counts or
//     masses in shared memory, of equal bins of logits, then of ordered
//     bits, then of indices, each inside the bin where the last one crossed
//     the mark, until the tokens inside fit the list.  Masses there are
//     integers, summed in 64 bits, so no result depends on the order of the
//     atomics; each bin counts in a unit of its own, so that small weights keep
//     their digits as well.  Without kept slices such a row is left to
//     a second launch of wide clusters with them: read again by 2,048 threads
//     it takes 25 us, where one block of 256 took 350.
// Other sums are in fp32: a thread's in the order of its tokens, then over the
// threads and blocks in a fixed tree.  Weights below 2^-126 may count as 0.
//
// What bounds it (device time): rows that need no histogram, memory -- 256 x
// 131072 fp32 with temperature alone 46 us for 268 MB (5.9 TB/s, 86% of the
// copy rate), 512 x 131072 bf16 greedy 31 us for 134 MB, with top-k and top-p
// 35 us.  Few rows, the chain of cluster barriers (about 1,200 cycles each)
// and of steps in one block: 1 x 32768 bf16 with top-k and top-p 8.3 us, of
// which the pass over the row is 0.6, the bound 1.5, collecting 2.9, the sort
// 1.9, the cut and the race 1.4.  Flat rows, the two dense passes: 16 x 65536
// fp32 with top-p 20 to 24 us, by the rows, of which the histogram takes 2.5, its
// exchange 3.5, the race 4.0.  512 x 131072 bf16 of mixed settings take 72 to 77
// us: 35 for the rows that a list does for, 30 for the others beside the longest
// races.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <cfloat>
#include <cstring>

#include "core.cuh"
#include "launch.h"
#include "pipeline.cuh"

namespace devscan {
namespace {

using u64 = unsigned long long;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kGroup = 4;                  // chunks that a thread loads at once: an entry of the index
constexpr int kQueue = 64;                 // entries that a warp has waiting
// A row of at most kLoneChunks 16-byte chunks is one block's: 8,000 tokens took
// 7.3 us in one block and 8.3 in two (bf16, top-k and top-p), 8.6 and 10.0 in
// four (fp32, top-p).  Larger ones are dealt to up to kMaxCluster blocks while
// rows are few: 32,768 tokens of bf16 took 29, 24, 18 and 16 us in one, two, four
// and eight (top-p).
constexpr unsigned kLoneChunks = 2048;
constexpr unsigned kKeptChunks = 4096;     // of a kept slice, for two blocks per SM: 64 KB
constexpr unsigned kPolls = 1024;          // of the second launch for the first's rows, 64 ns apart
constexpr int kList = 1024;                // tokens the short list holds
constexpr int kBins = 1024;
constexpr float kCountSpan = 16.0f;        // first histogram of counts: logits below the largest, where nothing says how far
// First histogram of masses: kBinsPerBit bins to a factor of two in weight.  As
// many neighbouring bins share a unit, about 2^-kMassBits of the weight at which
// they begin: a weight, whose own error is 3 to 200 times 2^-24, is rounded to 23
// bits, which a float's addition does, and a word takes 500 masses without a
// carry.  (16 x 65536 f32 top-p: 23.6 us; 24 bits by a conversion 24.5; 31 bits,
// with a carry at every third, 25.3.)  The last bin holds all that lies further,
// in units of 2^-kDeepest.  Bins are added up in units of 2^-kMassUnit, in which
// 2^18 weights of 1 fit 64 bits.  With one unit of 2^-31 for all bins, a cut among
// weights of 2^-32 was off by a seventh of its tokens (131072 tokens 22
// temperatures below the largest).
constexpr int kUnitShift = 5, kBinsPerBit = 1 << kUnitShift, kMassBits = 23, kMassUnit = 45,
              kDeepest = kMassBits + (kBins - 1) / kBinsPerBit;
constexpr float kMassOfOne = 63.0f / 64.0f * (1 << kMassBits);
constexpr int kGuess = 256, kGuessEach = 16;   // tokens asked of the bound for top-p without top-k: in all, per warp at most

__device__ __forceinline__ float inf() { return __int_as_float(0x7f800000); }

// ---------------------------------------------------------------------------
// Cluster exchange: a word of this block's shared memory in another block.
// ---------------------------------------------------------------------------
__device__ __forceinline__ unsigned cluster_rank()
{
    unsigned r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ unsigned cluster_blocks()
{
    unsigned r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive()
{
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t remote(const void *p, unsigned rank)
{
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ void put(uint32_t *p, unsigned rank, uint32_t v)
{
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(remote(p, rank)), "r"(v) : "memory");
}
__device__ __forceinline__ void put(float *p, unsigned rank, float v)
{
    put(reinterpret_cast<uint32_t *>(p), rank, __float_as_uint(v));
}
__device__ __forceinline__ void put(u64 *p, unsigned rank, u64 v)
{
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(remote(p, rank)), "l"(v) : "memory");
}
__device__ __forceinline__ void put(uint4 *p, unsigned rank, const uint4 &v)
{
    asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(remote(p, rank)), "r"(v.x), "r"(v.y),
                 "r"(v.z), "r"(v.w)
                 : "memory");
}
__device__ __forceinline__ uint32_t shared_add(uint32_t *p, uint32_t v)
{
    uint32_t old;
    asm volatile("atom.shared::cta.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(smem_u32(p)), "r"(v) : "memory");
    return old;
}

// ---------------------------------------------------------------------------
// Values.
// ---------------------------------------------------------------------------
// Bits of x whose unsigned order is x's order (x not NaN; -0 counts as 0).
__device__ __forceinline__ uint32_t ordered(float x)
{
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t k)
{
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
constexpr uint32_t kOrderedMinusInf = 0x007fffffu;
constexpr uint32_t kOrderedMinusZero = 0x7fffffffu;   // of no value: unordered() compares equal to 0 there

// A token's place in the order: larger keys first.
__device__ __forceinline__ u64 key_of(uint32_t ord, unsigned i) { return (static_cast<u64>(ord) << 32) | ~i; }
__device__ __forceinline__ uint32_t ord_of(u64 key) { return static_cast<uint32_t>(key >> 32); }
__device__ __forceinline__ unsigned index_of(u64 key) { return ~static_cast<unsigned>(key); }

__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float reciprocal(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A 16-byte chunk of logits: kEach values, and the larger of two chunks value
// by value (a NaN loses to a number).
template <class T> struct Chunk;
template <> struct Chunk<float> {
    static constexpr int kEach = 4, kSpare = 0;   // kSpare: low bits of ordered() that no value uses
    static constexpr uint32_t kFill = 0xff800000u;
    static __device__ __forceinline__ float value(const uint32_t (&q)[4], int e) { return __uint_as_float(q[e]); }
    static __device__ __forceinline__ float most(const uint32_t (&q)[4], float m)
    {
#pragma unroll
        for (int e = 0; e < 4; ++e) m = fmaxf(m, __uint_as_float(q[e]));
        return m;
    }
};
template <> struct Chunk<__half> {
    static constexpr int kEach = 8, kSpare = 13;
    static constexpr uint32_t kFill = 0xfc00fc00u;
    static __device__ __forceinline__ float value(const uint32_t (&q)[4], int e)
    {
        const uint32_t b = (e & 1) ? q[e / 2] >> 16 : q[e / 2] & 0xffffu;
        return __half2float(__ushort_as_half(static_cast<unsigned short>(b)));
    }
    static __device__ __forceinline__ float most(const uint32_t (&q)[4], float m)
    {
        __half2 h[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) h[k] = *reinterpret_cast<const __half2 *>(&q[k]);
        const __half2 a = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
        return fmaxf(m, fmaxf(__low2float(a), __high2float(a)));
    }
};
template <> struct Chunk<__nv_bfloat16> {
    static constexpr int kEach = 8, kSpare = 16;
    static constexpr uint32_t kFill = 0xff80ff80u;
    static __device__ __forceinline__ float value(const uint32_t (&q)[4], int e)
    {
        return __uint_as_float((e & 1) ? q[e / 2] & 0xffff0000u : q[e / 2] << 16);
    }
    static __device__ __forceinline__ float most(const uint32_t (&q)[4], float m)
    {
        __nv_bfloat162 h[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) h[k] = *reinterpret_cast<const __nv_bfloat162 *>(&q[k]);
        const __nv_bfloat162 a = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
        return fmaxf(m, fmaxf(__low2float(a), __high2float(a)));
    }
};

struct Shared {
    u64 list[kList];                 // this block's collected tokens; a buffer of the sort
    uint32_t bins[kBins];            // of the list's sort
    uint4 edge[2];                   // the slice's chunks over the row's ends
    uint16_t queue[kWarps][kQueue];
    u64 warp64[kWarps];
    float warpf[kWarps];
    uint32_t warp_a[kWarps], warp_b[kWarps];
    // What the blocks tell each other, by rank.
    uint32_t top[kMaxCluster], bound[kMaxCluster];
    uint32_t found[2][kMaxCluster];
    float sum[2][kMaxCluster];
    float sum_all[kMaxCluster];
    u64 won[kMaxCluster];
    float rest[kMaxCluster];
    uint32_t tops[kMaxCluster];
    u64 cut;
    uint32_t next[2];
    // Results of one block's scans.
    u64 pick_key, pick_want;
    uint32_t pick_bin, pick_edge[2];
    uint32_t listed;                 // tokens collected by this block (counting stops above its region)
};
// Keys that block 0's inbox has room for: a wide cluster's blocks do not all
// bring the same number.
template <bool KEEP>
__host__ __device__ constexpr unsigned inbox_keys(unsigned blocks) { return blocks == 1 && !KEEP ? kList : 2 * kList; }
// Words of the histogram's parts that the blocks send each other.
template <bool KEEP> constexpr unsigned kPartWords = KEEP ? 2 * kBins : 0;
constexpr size_t kSharedBytes = (sizeof(Shared) + 127) / 128 * 128;

// 2^-48 over a token's noise; for noise that loses not above 0, or no number.
// The reciprocal flushes denormal numbers, and that of 0 would beat every other:
// so the noise is scaled first, and moved by 2^-126, which makes 0 and -0 lose as
// negative noise does and is below a number's last digit otherwise (the smallest
// denormal is 2^-101 here).  Noise from 2^78 on gives 0.  With weights of up to 1
// no score overflows, and a quotient of weight and noise of 2^-78 or more keeps
// its digits.  One multiply-add: 512 x 131072 bf16 of mixed settings take 76.3
// us, with a comparison and a select in its place 79.4.
__device__ __forceinline__ float pace(float q)
{
    return reciprocal(fmaf(q, 0x1p48f, -0x1p-126f));
}

// The race among the kept tokens that a thread has seen, and their weights'
// sum: `tops` of exactly 1, the others in `rest`, so that a small rest keeps
// its digits beside them.  Only a score above 0 can be drawn: what lies outside
// the row, is masked, or has noise that loses never is, whatever else there is.
struct Race {
    float score = 0.0f, rest = 0.0f;
    int at = 0x7fffffff;
    uint32_t tops = 0;
    __device__ __forceinline__ void offer(float w, float q, int i)
    {
        const float sc = w * pace(q);
        if (sc >= score && (sc > score || i < at)) score = sc, at = i;
        if (w == 1.0f) ++tops;
        else rest += w;
    }
    // Order of scores, the lowest index first among equals.
    __device__ __forceinline__ u64 key() const
    {
        return score > 0.0f ? (static_cast<u64>(__float_as_uint(score)) << 32) | ~static_cast<unsigned>(at) : 0ull;
    }
};

// One block's part in the draw of one row.  KEEP: the first pass leaves the
// slice in shared memory for the later ones; else it leaves the index.
//
// The code is kept small: most of it runs once per row, so that a call of few
// rows waits for instructions first (about 300 cycles for 128 bytes that no
// other block has fetched), and a loop of one copy beats an unrolled one.
template <class T, bool KEEP>
struct Draw {
    using C = Chunk<T>;
    static constexpr int kEach = C::kEach;
    static constexpr int kPair = 8 / kEach, kOwn = kPair * kEach;   // chunks, and values, that a dense pass takes at once

    Shared &s;
    u64 *inbox;                      // in block 0: the cluster's tokens, a region of `region` per block
    uint32_t *count, *carry;         // a histogram in the same memory: counts, or the masses' low words;
                                     // the masses' high words
    uint32_t *low_parts, *high_parts;   // every block's part of the bins that are this block's to sum
    uint32_t region;
    uint4 *kept;                     // with KEEP the slice
    float *index;                    // else the maxima of its groups of chunks
    const float *noise;              // of the row
    const T *row;
    const uint4 *source;             // the slice in memory
    unsigned tid, lane, warp, rank, blocks;
    unsigned vocab, chunks, mine;    // tokens and chunks of the row; chunks of the slice
    unsigned lo, hi;                 // the slice's whole chunks
    int first;                       // index of the slice's first value
    float top, t, scale;             // the largest logit, temperature, log2(e) / T
    float bins_per_unit;             // of the first histogram
    float per_weight;                // masses to a weight of 1, in the bin where a cut lies
    float reach;                     // logits below the largest where the first k are expected to end
    bool infinite = false;           // the largest is +inf: it counts as 0, all else as -inf
    int turn = 0;                    // which half of the double buffers is next

    __device__ __forceinline__ Draw(Shared &shared) : s(shared) {}

    // All threads of the cluster.
    __device__ __forceinline__ void meet() const
    {
        if (blocks == 1) {
            __syncthreads();
        } else {
            cluster_arrive();
            cluster_wait();
        }
    }

    // -----------------------------------------------------------------------
    // The row.
    // -----------------------------------------------------------------------
    static __device__ __forceinline__ void unpack(const uint4 &v, uint32_t (&q)[4])
    {
        q[0] = v.x, q[1] = v.y, q[2] = v.z, q[3] = v.w;
    }
    static __device__ __forceinline__ uint4 fill() { return make_uint4(C::kFill, C::kFill, C::kFill, C::kFill); }
    __device__ __forceinline__ int index_at(unsigned c) const { return first + static_cast<int>(c) * kEach; }

    // The block's slice of the row.  Rows may start anywhere: chunk 0 begins
    // at the 16-byte boundary at or before the row, and a chunk that reaches
    // over either end of the row is read value by value into shared memory,
    // filled with -inf.
    __device__ __forceinline__ void place(unsigned per)
    {
        const unsigned shift = static_cast<unsigned>(reinterpret_cast<uintptr_t>(row) % 16 / sizeof(T));
        const unsigned begin = rank * per;
        chunks = (vocab + shift + kEach - 1) / kEach;
        mine = begin < chunks ? min(per, chunks - begin) : 0;
        first = static_cast<int>(begin * kEach) - static_cast<int>(shift);
        source = reinterpret_cast<const uint4 *>(row - shift) + begin;
        const bool head = first < 0 && mine > 0, tail = mine > 0 && index_at(mine) > static_cast<int>(vocab);
        lo = head ? 1 : 0;
        hi = tail ? mine - 1 : mine;
        // The first loads' lines are on their way to L2 before the settings
        // have come, on which the first pass depends.
#pragma unroll
        for (int u = 0; u < kGroup; ++u)
            if (tid + u * kThreads >= lo && tid + u * kThreads < hi)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(source + tid + u * kThreads));
        if (head || tail) {
            // Thread 0 the head, 32 the tail; one chunk over both ends is a head.
            if ((tid == 0 && head) || (tid == 32 && tail && !(head && mine == 1))) {
                const unsigned c = tid == 0 ? 0 : mine - 1;
                T *v = reinterpret_cast<T *>(&s.edge[tid / 32]);
#pragma unroll 1
                for (int e = 0; e < kEach; ++e) {
                    const int i = index_at(c) + e;
                    v[e] = i >= 0 && i < static_cast<int>(vocab) ? row[i] : T(-inf());
                }
            }
            __syncthreads();
        }
    }
    __device__ __forceinline__ uint4 fetch(unsigned c) const
    {
        if (c >= lo && c < hi) return __ldg(source + c);
        if (c >= mine) return fill();
        return s.edge[c == 0 && lo == 1 ? 0 : 1];
    }

    // First pass: the thread's largest value, and with SUM the thread's sum of
    // weights relative to it.  A thread's chunks are tid + k * kThreads; entry
    // (k, tid) of the index is the largest of those from kGroup * k on.
    template <bool SUM>
    __device__ __forceinline__ float load(float *sum)
    {
        float most = -inf(), held = 0.0f;
        unsigned entry = tid;
#pragma unroll 1
        for (unsigned c0 = tid; c0 < mine; c0 += kGroup * kThreads, entry += kThreads) {
            uint4 v[kGroup];
            float group = -inf();
#pragma unroll
            for (int u = 0; u < kGroup; ++u) v[u] = fetch(c0 + u * kThreads);
#pragma unroll
            for (int u = 0; u < kGroup; ++u) {
                uint32_t q[4];
                unpack(v[u], q);
                group = C::most(q, group);
                if (KEEP && c0 + u * kThreads < mine) kept[c0 + u * kThreads] = v[u];
            }
            if (!KEEP) index[entry] = group;
            if (SUM && group > -inf()) {
                if (group > most) held *= fmaxf(exp2_approx((most - group) * scale), 0.0f);
                const float base = fmaxf(most, group);
#pragma unroll
                for (int u = 0; u < kGroup; ++u) {
                    uint32_t q[4];
                    unpack(v[u], q);
#pragma unroll
                    for (int e = 0; e < kEach; ++e)
                        held += fmaxf(exp2_approx((C::value(q, e) - base) * scale), 0.0f);
                }
            }
            most = fmaxf(most, group);
        }
        if (SUM) *sum = held;
        return most;
    }

    // A warp's queue: lanes put numbers in, and whenever 32 wait, or at the end
    // (`all`), each lane takes one and calls f(number).
    template <class F>
    __device__ __forceinline__ void queue_up(unsigned &waiting, bool in, unsigned number, bool all, F f)
    {
        uint16_t *queue = s.queue[warp];
        const unsigned some = __ballot_sync(kFullMask, in);
        if (in) queue[waiting + __popc(some & ((1u << lane) - 1))] = static_cast<uint16_t>(number);
        waiting += __popc(some);
        if (waiting < 32 && !(all && waiting > 0)) return;
        __syncwarp();
        const unsigned taken = min(waiting, 32u);
        const unsigned at = lane < taken ? queue[lane] : 0, moved = lane + 32 < waiting ? queue[lane + 32] : 0;
        __syncwarp();
        if (lane + 32 < waiting) queue[lane] = static_cast<uint16_t>(moved);
        waiting -= taken;
        if (lane < taken) f(at);
        __syncwarp();
    }

    // f(values, c) for every chunk c of the slice with a value of at least
    // `low`, where these are few: they are queued, a chunk of the kept slice or
    // an entry of the index at a time.
    template <class F>
    __device__ __forceinline__ void each_chunk(float low, F f)
    {
        constexpr unsigned kStep = KEEP ? kThreads : kGroup * kThreads;   // chunks to a round of entries
        unsigned waiting = 0;
        const unsigned rounds = (mine + kStep - 1) / kStep;
#pragma unroll 1
        for (unsigned k = 0; k <= rounds; ++k) {
            // An entry of the index is there if its first chunk is.
            const bool in = k < rounds && tid + k * kStep < mine &&
                            (KEEP ? reaches(tid + k * kStep, low) : index[k * kThreads + tid] >= low);
            queue_up(waiting, in, k * 32 + lane, k == rounds, [&](unsigned at) {
                const unsigned c = (at / 32) * kStep + warp * 32 + at % 32;
                if (KEEP) {
                    visit(kept[c], low, c, f);
                } else {
                    uint4 v[kGroup];
#pragma unroll
                    for (int u = 0; u < kGroup; ++u) v[u] = fetch(c + u * kThreads);
                    // Mostly one of the four reaches it: as many turns as the
                    // most that a lane has, not four.
                    uint32_t hits = 0;
#pragma unroll
                    for (int u = 0; u < kGroup; ++u) {
                        uint32_t q[4];
                        unpack(v[u], q);
                        hits |= infinite || C::most(q, -inf()) >= low ? 1u << u : 0u;
                    }
#pragma unroll 1
                    for (; hits != 0; hits &= hits - 1) {
                        const unsigned u = __ffs(hits) - 1;
                        uint4 x = v[0];
#pragma unroll
                        for (int o = 1; o < kGroup; ++o) x = u == o ? v[o] : x;
                        visit(x, low, c + u * kThreads, f);
                    }
                }
            });
        }
    }
    // Whether chunk c of the kept slice has a value of at least `low`.
    __device__ __forceinline__ bool reaches(unsigned c, float low) const
    {
        if (c >= mine) return false;
        uint32_t q[4];
        unpack(kept[c], q);
        if (infinite) only_infinite(q);
        return C::most(q, -inf()) >= low;
    }
    // Dense passes of a kept slice: every thread its own chunks, kPair at a
    // time (c and c + kThreads), in the order of their indices.  Whether one of
    // the pair at c has a value of at least `low`; its values.
    __device__ __forceinline__ bool own(unsigned c, float low, float (&x)[kOwn]) const
    {
        float most = -inf();
#pragma unroll
        for (int u = 0; u < kPair; ++u) {
            uint32_t q[4];
            unpack(c + u * kThreads < mine ? kept[c + u * kThreads] : fill(), q);
            if (infinite) only_infinite(q);
            most = C::most(q, most);
#pragma unroll
            for (int e = 0; e < kEach; ++e) x[u * kEach + e] = C::value(q, e);
        }
        return most >= low;
    }
    __device__ __forceinline__ int own_index(unsigned c, int e) const
    {
        return index_at(c + e / kEach * kThreads) + e % kEach;
    }
    __device__ __forceinline__ void own_noise(unsigned c, bool aligned, float (&n)[kOwn]) const
    {
#pragma unroll
        for (int u = 0; u < kPair; ++u) {
            float part[kEach];
            load_noise(c + u * kThreads, aligned, part);
#pragma unroll
            for (int e = 0; e < kEach; ++e) n[u * kEach + e] = part[e];
        }
    }
    template <class F>
    __device__ __forceinline__ void visit(const uint4 &v, float low, unsigned c, F &&f)
    {
        uint32_t q[4];
        unpack(v, q);
        if (infinite) only_infinite(q);
        if (!(C::most(q, -inf()) >= low)) return;
        float x[kEach];
#pragma unroll
        for (int e = 0; e < kEach; ++e) x[e] = C::value(q, e);
        f(x, c);
    }
    // 0 in place of every +inf, and -inf of everything else.
    static __device__ __forceinline__ void only_infinite(uint32_t (&q)[4])
    {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint32_t r = 0;
#pragma unroll
            for (int e = 0; e < kEach / 4; ++e)
                if (C::value(q, k * (kEach / 4) + e) != inf())
                    r |= kEach == 4 ? C::kFill : C::kFill & (0xffffu << (16 * e));
            q[k] = r;
        }
    }

    // Weight of any value (0 for -inf and NaN).  |error| <= (3 |d| + 3) 2^-24
    // relative, d = (v - top) / T.
    __device__ __forceinline__ float weight(float v) const { return fmaxf(exp2_approx((v - top) * scale), 0.0f); }
    // Weight of a number in the list, rounded as the definition's steps are.
    __device__ __forceinline__ float list_weight(float v) const
    {
        return v == top ? 1.0f : fmaxf(expf((v - top) / t), 0.0f);
    }
    // Masses to a weight of 1 in a bin of the first histogram: 63/64 of 2^(23 +
    // b / 32).  The bin's weights are at most 2^(1/64 - b / 32), so that a mass is
    // below 2^23, and in all bins but the last above half of that.
    static __device__ __forceinline__ float per_weight_in(int b)
    {
        return __int_as_float(__float_as_int(kMassOfOne) + (b >> kUnitShift << 23));
    }
    // w * per, rounded: the sum's last bit is worth 1.
    static __device__ __forceinline__ uint32_t mass_of(float w, float per)
    {
        return static_cast<uint32_t>(__float_as_int(fmaf(w, per, 8388608.0f)) - 0x4b000000);
    }
    // A bin's masses in units of 2^-kMassUnit, rounded down; and masses wanted in
    // that unit as masses of the bin, rounded up.  Both pass by 2^-kMassUnit of
    // the unit's first weight, where 2^18 masses still fit 64 bits.
    static __device__ __forceinline__ u64 common(u64 masses, unsigned b)
    {
        return masses << (kMassUnit - kMassBits) >> (b >> kUnitShift);
    }
    static __device__ __forceinline__ u64 in_bin(u64 wanted, unsigned b)
    {
        return ((wanted << (b >> kUnitShift)) + ((1u << (kMassUnit - kMassBits)) - 1)) >> (kMassUnit - kMassBits);
    }
    __device__ __forceinline__ uint32_t mass(float v) const { return mass_of(exp2_approx((v - top) * scale), per_weight); }

    // -----------------------------------------------------------------------
    // Races.
    // -----------------------------------------------------------------------
    // A race of all tokens needs no selection, so it takes one pass over the
    // logits and the noise side by side.  Weights are relative to the largest
    // logit that the thread has seen; what it holds is scaled down when a
    // larger one comes.  That adds up to 5 * 2^-24 relative each time (the
    // distances add up to the token's own), once per chunk in a row that rises
    // throughout: 262,144 such fp32 tokens in one block, 256 chunks per thread,
    // gave log-probabilities of -12 with errors of up to 2.6e-6, rows that fall
    // of up to 2.5e-6.
    __device__ __forceinline__ void rescale(Race &o, float &most, float to) const
    {
        const float f = fmaxf(exp2_approx((most - to) * scale), 0.0f);
        if (f != 1.0f) o.rest = (o.rest + static_cast<float>(o.tops)) * f, o.tops = 0;
        o.score *= f;
        most = to;
    }
    __device__ __forceinline__ float race_all(Race &o)
    {
        constexpr int kRaceLoads = kEach == 4 ? 4 : 2;   // chunks in flight, beside their noise
        const bool aligned = reinterpret_cast<uintptr_t>(noise + first) % 16 == 0;
        float most = -inf();
#pragma unroll 1
        for (unsigned c0 = tid; c0 < mine; c0 += kRaceLoads * kThreads) {
            uint4 x[kRaceLoads];
            float n[kRaceLoads][kEach];
#pragma unroll
            for (int u = 0; u < kRaceLoads; ++u) {
                const unsigned c = c0 + u * kThreads;
                x[u] = c >= lo && c < hi ? ld_stream(source + c) : fetch(c);
                load_noise(c, aligned, n[u]);
            }
#pragma unroll
            for (int u = 0; u < kRaceLoads; ++u) {
                uint32_t q[4];
                unpack(x[u], q);
                const float group = C::most(q, -inf());
                if (group == -inf()) continue;
                if (group > most) rescale(o, most, group);
                const int i = index_at(c0 + u * kThreads);
#pragma unroll
                for (int e = 0; e < kEach; ++e) {
                    // Indices rise within a thread, so the first of equals stays.
                    const float w = fmaxf(exp2_approx((C::value(q, e) - most) * scale), 0.0f);
                    const float sc = w * pace(n[u][e]);
                    o.at = sc > o.score ? i + e : o.at;
                    o.score = sc > o.score ? sc : o.score;
                    o.tops += w == 1.0f ? 1u : 0u;
                    o.rest += w == 1.0f ? 0.0f : w;
                }
            }
        }
        return most;
    }
    // A chunk's noise; 1 outside the row.
    __device__ __forceinline__ void load_noise(unsigned c, bool aligned, float (&n)[kEach]) const
    {
        const float *at = noise + index_at(c);
        if (aligned && c >= lo && c < hi) {
#pragma unroll
            for (int e = 0; e < kEach; e += 4) {
                const float4 q = __ldcs(reinterpret_cast<const float4 *>(at + e));
                n[e] = q.x, n[e + 1] = q.y, n[e + 2] = q.z, n[e + 3] = q.w;
            }
        } else {
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                const int i = index_at(c) + e;
                n[e] = c < mine && i >= 0 && i < static_cast<int>(vocab) ? __ldcs(at + e) : 1.0f;
            }
        }
    }

    // The race of a chunk's tokens for which keep(value, index) holds and
    // whose weight is at least m.  RISING: this thread's indices rise, so the
    // first of equal scores stays.
    template <bool RISING, int N, class Keep>
    __device__ __forceinline__ void race_chunk(const float (&x)[N], const float (&n)[N], unsigned c, float m, Keep keep,
                                               Race &o) const
    {
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const int i = own_index(c, e);
            float w = weight(x[e]);
            w = keep(x[e], i) & (w >= m) ? w : 0.0f;   // its score is not above 0
            const float sc = w * pace(n[e]);
            if (RISING) {
                o.at = sc > o.score ? i : o.at;
                o.score = sc > o.score ? sc : o.score;
            } else if (sc >= o.score && (sc > o.score || i < o.at)) {
                o.score = sc, o.at = i;
            }
            o.tops += w == 1.0f ? 1u : 0u;
            o.rest += w == 1.0f ? 0.0f : w;
        }
    }
    // Starts the noise of the chunks with a value of at least `low` towards L2.
    __device__ __forceinline__ void prefetch_noise(float low)
    {
#pragma unroll 1
        for (unsigned c = tid; c < mine; c += kThreads)
            if (reaches(c, low)) asm volatile("prefetch.global.L2 [%0];" ::"l"(noise + max(index_at(c), 0)));
    }

    __device__ __forceinline__ void write(u64 won, const Race &o, int32_t *token, float *logprob) const
    {
        if (won == 0) {   // no score above 0: the kept tokens' noise loses
            *token = -1;
            if (logprob != nullptr) *logprob = -inf();
            return;
        }
        const unsigned i = index_of(won);
        *token = static_cast<int32_t>(i);
        if (logprob == nullptr) return;
        const float v = static_cast<float>(row[i]);
        const float d = v == inf() || v == top ? 0.0f : (v - top) / t;
        *logprob = d - log1pf(o.rest + static_cast<float>(o.tops - 1));
    }

    // Joins the races of this block's threads, and with ALL those of the
    // cluster's blocks, and writes the row's answer.
    template <bool ALL>
    __device__ __forceinline__ void finish(Race &o, int32_t *token, float *logprob)
    {
        u64 won = o.key();
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) {
            const u64 u = __shfl_xor_sync(kFullMask, won, d);
            won = u > won ? u : won;
            o.rest += __shfl_xor_sync(kFullMask, o.rest, d);
        }
        o.tops = __reduce_add_sync(kFullMask, o.tops);
        __syncthreads();
        if (lane == 0) s.warp64[warp] = won, s.warpf[warp] = o.rest, s.warp_a[warp] = o.tops;
        __syncthreads();
        if (tid == 0) total(s.warp64, s.warpf, s.warp_a, kWarps, won, o);
        if (ALL && blocks > 1) {
            if (tid == 0) {
                put(&s.won[rank], 0, won);
                put(&s.rest[rank], 0, o.rest);
                put(&s.tops[rank], 0, o.tops);
            }
            meet();
            if (rank != 0) return;
            if (tid == 0) total(s.won, s.rest, s.tops, blocks, won, o);
        }
        if (tid == 0) write(won, o, token, logprob);
    }
    static __device__ __forceinline__ void total(const u64 *w, const float *r, const uint32_t *n, unsigned parts,
                                                 u64 &won, Race &o)
    {
        won = 0, o.rest = 0.0f, o.tops = 0;
#pragma unroll 1
        for (unsigned k = 0; k < parts; ++k) {
            won = w[k] > won ? w[k] : won;
            o.rest += r[k];
            o.tops += n[k];
        }
    }

    // -----------------------------------------------------------------------
    // Block-wide sums.
    // -----------------------------------------------------------------------
    // Exclusive prefix of v over the block's threads; *all its total.
    template <class V>
    __device__ __forceinline__ V block_scan(V v, V *s_warp, V *all)
    {
        V incl = v;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const V u = __shfl_up_sync(kFullMask, incl, d);
            if (lane >= d) incl += u;
        }
        __syncthreads();
        if (lane == 31) s_warp[warp] = incl;
        __syncthreads();
        V parts = s_warp[lane & (kWarps - 1)];
#pragma unroll
        for (int d = 1; d < kWarps; d <<= 1) {
            const V u = __shfl_up_sync(kFullMask, parts, d);
            if ((lane & (kWarps - 1)) >= d) parts += u;
        }
        *all = __shfl_sync(kFullMask, parts, kWarps - 1);
        const V ahead = __shfl_sync(kFullMask, parts, (warp - 1) & 31), before = __shfl_up_sync(kFullMask, incl, 1);
        return (warp == 0 ? V(0) : ahead) + (lane == 0 ? V(0) : before);
    }

    // -----------------------------------------------------------------------
    // The list.
    // -----------------------------------------------------------------------
    // Tokens for the list: begin_list(), then add_tokens() by any thread, then
    // merge_lists(), which returns their number over the cluster (the same in
    // every block).  Up to kList they are then in block 0, in any order; more
    // than kList is returned as well if a block has more than its region.
    // sum: a partial sum of each thread; *sum becomes the cluster's.
    __device__ __forceinline__ void begin_list()
    {
        if (tid == 0) s.listed = 0;
        __syncthreads();
    }
    // The chunk's tokens whose bits are set.
    __device__ __forceinline__ void add_tokens(const float (&x)[kEach], unsigned c, uint32_t which)
    {
        if (which == 0 || *const_cast<volatile uint32_t *>(&s.listed) > region) return;
        uint32_t k = shared_add(&s.listed, __popc(which));
        if (k + __popc(which) > region) return;
        u64 *list = rank == 0 ? inbox : s.list;
#pragma unroll
        for (int e = 0; e < kEach; ++e)
            if (which >> e & 1) list[k++] = key_of(ordered(x[e]), static_cast<unsigned>(index_at(c) + e));
    }
    __device__ __forceinline__ uint32_t merge_lists(float *sum)
    {
        const int now = turn;
        turn ^= 1;
        float part = 0.0f;
        if (sum != nullptr) block_scan(*sum, s.warpf, &part);
        else __syncthreads();
        const uint32_t n = s.listed;
        if (tid < blocks) {
            put(&s.found[now][rank], tid, n <= region ? n : kList + 1);
            if (sum != nullptr) put(&s.sum[now][rank], tid, part);
        }
        if (rank != 0 && n <= region)
            for (uint32_t k = tid; k < n; k += kThreads) put(&inbox[rank * region + k], 0, s.list[k]);
        meet();
        uint32_t all = 0, ahead = 0;
        float sums = 0.0f;
#pragma unroll 1
        for (unsigned b = 0; b < blocks; ++b) {
            if (b == warp) ahead = all;
            all += s.found[now][b];
            sums += s.sum[now][b];
        }
        if (sum != nullptr) *sum = sums;
        if (rank == 0 && blocks > 1 && all <= kList) {   // close the gaps, a warp per region
            static_assert(kWarps >= kMaxCluster, "a warp per block's region");
            if (warp < blocks)
                for (uint32_t k = lane; k < s.found[now][warp]; k += 32) s.list[ahead + k] = inbox[warp * region + k];
            __syncthreads();
        }
        return all;
    }

    // Puts the n <= kList merged tokens in descending order, by block 0, and
    // returns them; their ordered bits are in least .. most.  A counting sort in
    // bins of equal width from the largest down to the least (by value, then by index, so that ties fill their range
    // evenly too), then by key inside a bin, where there are one or two as a
    // rule: a fixed number of barriers, where a sort by comparisons took two to
    // three times as long.
    __device__ __forceinline__ const u64 *sort(uint32_t n, uint32_t most, uint32_t least)
    {
        u64 *from = blocks == 1 ? inbox : s.list, *to = blocks == 1 ? s.list : inbox;
        static_assert(kBins == 4 * kThreads, "a thread's bins are one 16-byte access");
        reinterpret_cast<uint4 *>(s.bins)[tid] = make_uint4(0, 0, 0, 0);
        if (least <= ordered(-FLT_MAX)) {   // no bound: the least token's
            least = most;
#pragma unroll 1
            for (uint32_t k = tid; k < n; k += kThreads) least = min(least, ord_of(from[k]));
            least = __reduce_min_sync(kFullMask, least);
            if (lane == 0) s.warp_b[warp] = least;
            __syncthreads();
            least = __reduce_min_sync(kFullMask, s.warp_b[lane & (kWarps - 1)]);
        }
        __syncthreads();
        // Steps of value below the largest, and the index as a fraction of one:
        // rounded, but never out of order.
        const float step = 1.0f / static_cast<float>(vocab);
        const float scaled = kBins / (static_cast<float>((most >> C::kSpare) - (least >> C::kSpare)) + 1.0f);
        const auto bin_of_key = [&](u64 key) {
            const float below = static_cast<float>((most >> C::kSpare) - (ord_of(key) >> C::kSpare));
            return min(static_cast<uint32_t>(fmaf(static_cast<float>(index_of(key)), step, below) * scaled), kBins - 1u);
        };
#pragma unroll 1
        for (uint32_t k = tid; k < n; k += kThreads) shared_add(&s.bins[bin_of_key(from[k])], 1);
        __syncthreads();
        uint4 b = reinterpret_cast<uint4 *>(s.bins)[tid];
        uint32_t all = 0;
        const uint32_t before = block_scan(b.x + b.y + b.z + b.w, s.warp_a, &all);
        reinterpret_cast<uint4 *>(s.bins)[tid] =
            make_uint4(before, before + b.x, before + b.x + b.y, before + b.x + b.y + b.z);
        __syncthreads();
        // A bin's start moves on to its end as its tokens take their places.
#pragma unroll 1
        for (uint32_t k = tid; k < n; k += kThreads) to[shared_add(&s.bins[bin_of_key(from[k])], 1)] = from[k];
        __syncthreads();
#pragma unroll 1
        for (uint32_t k = tid; k < n; k += kThreads) {
            const u64 key = to[k];
            const uint32_t at = bin_of_key(key), begin = at == 0 ? 0 : s.bins[at - 1], end = s.bins[at];
            uint32_t place = begin;
            for (uint32_t o = begin; o < end && end - begin > 1; ++o) place += to[o] > key ? 1u : 0u;
            from[place] = key;
        }
        __syncthreads();
        return from;
    }

    // -----------------------------------------------------------------------
    // Cuts by histograms.
    // -----------------------------------------------------------------------
    // The bin of the first histogram: falls as v grows.
    __device__ __forceinline__ int bin_of(float v) const
    {
        // The sum's last bit is worth 1: its low bits are the rounded bin.
        return __float_as_int(fminf(fmaf(top - v, bins_per_unit, 8388608.0f), 8388608.0f + (kBins - 1))) - 0x4b000000;
    }

    // One histogram level: adds what each value holds, then finds the bin
    // where the running total from bin 0 reaches want = wanted(total).  Returns
    // false if it does not; else `bin`, and `want` less what is in the bins
    // before it.  The last bin of counts, in which most of a peaked row may
    // fall, is summed in registers: its atomics would wait for one another.
    // (That of masses fills up only where a cut is wanted far down a tail.)
    // FIRST: masses in the bins' own units, totals in the common one; else both
    // in the unit of per_weight.
    template <bool MASS, bool FIRST, class Bin, class Want>
    __device__ __forceinline__ bool histogram(float low, Bin bin_in, Want wanted, u64 &want, uint32_t &bin)
    {
        reinterpret_cast<uint4 *>(count)[tid] = make_uint4(0, 0, 0, 0);
        reinterpret_cast<uint4 *>(carry)[tid] = make_uint4(0, 0, 0, 0);
        __syncthreads();
        uint32_t last = 0;
#pragma unroll 1
        for (unsigned c = tid; c < mine; c += kPair * kThreads) {
            float x[kOwn];
            if (!own(c, low, x)) continue;
            // Nothing branches before the chunk's atomics are all in flight: a
            // value that takes no part adds 0 to a word of its lane's own.
            uint32_t *at[kOwn], holds[kOwn], old[kOwn], carried = 0;
#pragma unroll
            for (int e = 0; e < kOwn; ++e) {
                const int b = bin_in(x[e], own_index(c, e));
                const bool in = b >= 0 & (MASS | b != kBins - 1);
                last += !MASS & b == kBins - 1 ? 1u : 0u;
                at[e] = count + (in ? b : kBins + static_cast<int>(lane));
                holds[e] = !in ? 0u : !MASS ? 1u : mass_of(exp2_approx((x[e] - top) * scale), FIRST ? per_weight_in(b) : per_weight);
            }
#pragma unroll
            for (int e = 0; e < kOwn; ++e) old[e] = shared_add(at[e], holds[e]);
            if (MASS) {
#pragma unroll
                for (int e = 0; e < kOwn; ++e) carried |= old[e] + holds[e] < old[e] ? 1u << e : 0u;
                if (carried != 0) {
#pragma unroll
                    for (int e = 0; e < kOwn; ++e)
                        if (carried >> e & 1) shared_add(at[e] + (kBins + 32), 1);
                }
            }
        }
        if (!MASS) {
            last = __reduce_add_sync(kFullMask, last);
            if (lane == 0 && last != 0) shared_add(&count[kBins - 1], last);
        }
        __syncthreads();
        // Every block sums an equal part of the bins.  The others send it
        // theirs before the barrier: stores that nobody waits for, where reading each other's counts took 8,000 cycles.
        const uint4 low4 = reinterpret_cast<uint4 *>(count)[tid], high4 = reinterpret_cast<uint4 *>(carry)[tid];
        const unsigned part = kBins / blocks, owner = 4 * tid / part, at = rank * part + 4 * tid % part;
        put(reinterpret_cast<uint4 *>(low_parts + at), owner, low4);
        put(reinterpret_cast<uint4 *>(high_parts + at), owner, high4);
        meet();
        // Its sums go to every block, into the memory of its own list, which is
        // not in use between merge_lists() and begin_list(); each block then
        // finds the bin for itself.
        u64 *sums = s.list;
#pragma unroll 1
        for (unsigned b = tid; b < part; b += kThreads) {
            u64 h = 0;
#pragma unroll 1
            for (unsigned r = 0; r < blocks; ++r)
                h += low_parts[r * part + b] | static_cast<u64>(high_parts[r * part + b]) << 32;
            if (MASS && FIRST) h = common(h, rank * part + b);
#pragma unroll 1
            for (unsigned r = 0; r < blocks; ++r) put(&sums[rank * part + b], r, h);
        }
        meet();
        const ulonglong2 h01 = reinterpret_cast<const ulonglong2 *>(sums)[2 * tid];
        const ulonglong2 h23 = reinterpret_cast<const ulonglong2 *>(sums)[2 * tid + 1];
        const u64 h[4] = {h01.x, h01.y, h23.x, h23.y};
        u64 all = 0, before = block_scan(h[0] + h[1] + h[2] + h[3], s.warp64, &all);
        want = wanted(all);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (before < want && want <= before + h[k]) s.pick_bin = 4 * tid + k, s.pick_want = want - before;
            before += h[k];
        }
        __syncthreads();
        if (all < want) return false;
        bin = s.pick_bin;
        want = s.pick_want;
        return true;
    }

    // The least ordered bits o with bin_of(o) <= b, by one warp: 32 probes cut
    // the range to a 32nd.
    __device__ __forceinline__ uint32_t edge(int b) const
    {
        uint32_t from = ordered(-FLT_MAX), to = ordered(top);
        // As a rule within a few roundings of where the bin ends.
        const uint32_t near = max(min(ordered(top - (static_cast<float>(b) + 0.5f) / bins_per_unit), to), from + 16) - 16;
        const unsigned probed = __ballot_sync(kFullMask, bin_of(unordered(min(near + lane, to))) <= b);
        if ((probed & 1) == 0 && probed != 0) return near + __ffs(probed) - 1;
#pragma unroll 1
        while (from < to) {
            const uint32_t step = (to - from) / 32 + 1;
            const uint32_t probe = from + min(lane * step, to - from);
            const unsigned in = __ballot_sync(kFullMask, bin_of(unordered(probe)) <= b);
            // The first probe inside is the new end; the one before it is outside.
            const uint32_t at = in == 0 ? 32 : __ffs(in) - 1;
            to = at < 32 ? __shfl_sync(kFullMask, probe, at) : to;
            from = at > 0 ? __shfl_sync(kFullMask, probe, at - 1) + 1 : to;
        }
        return to;
    }

    // A cut of the order: the key of the last token of the shortest prefix
    // that holds wanted(total), in tokens or mass.  Only tokens with keys >=
    // floor take part.
    struct Floor {
        float v;
        int i;
        __device__ __forceinline__ explicit Floor(u64 key)
            : v(key == 0 ? -FLT_MAX : unordered(ord_of(key))), i(key == 0 ? 0x7fffffff : static_cast<int>(index_of(key)))
        {
        }
        __device__ __forceinline__ bool takes(float x, int at) const { return x > v | (x == v & at <= i); }
    };

    // The range of ordered bits of the first histogram's bin where the cut
    // lies, and what is wanted inside it (masses in the bin's unit); false if all
    // that take part hold less than wanted.
    template <bool MASS, class Want>
    __device__ __forceinline__ bool bracket(const Floor &floor, Want wanted, u64 &want, uint32_t &lo_bits, uint32_t &hi_bits)
    {
        uint32_t bin = 0;
        bins_per_unit = fminf(MASS ? kBinsPerBit * scale : fmaxf((kBins - 1) / reach, 1e-30f), 1e30f);
        // A weight of less has no mass.
        const float least = MASS ? fmaxf(floor.v, top - (kDeepest + 1) / scale) : floor.v;
        if (!histogram<MASS, true>(least, [&](float v, int i) { return floor.takes(v, i) & v >= least ? bin_of(v) : -1; },
                                   wanted, want, bin))
            return false;
        if (MASS) {
            per_weight = per_weight_in(static_cast<int>(bin));
            want = in_bin(want, bin);
        }
        if (warp < 2) {   // bin -1 would begin above the largest
            const uint32_t o = bin < warp ? ordered(top) + 1 : edge(static_cast<int>(bin - warp));
            if (lane == 0) s.pick_edge[warp] = o;
        }
        __syncthreads();
        lo_bits = s.pick_edge[0], hi_bits = s.pick_edge[1] - 1;
        return true;
    }

    // Block 0 puts the n merged tokens in order, of which the first that hold
    // `want` are kept, calls kept(key) for each of those, and leaves the last
    // one's key in s.pick_key.
    template <bool MASS, class Kept>
    __device__ __forceinline__ void resolve(uint32_t n, uint32_t hi_bits, uint32_t lo_bits, u64 want, Kept keep)
    {
        const u64 *sorted = sort(n, hi_bits, lo_bits);
        u64 base = 0;
#pragma unroll 1
        for (uint32_t k0 = 0; k0 < n; k0 += kThreads) {
            u64 key = 0, holds = 0, all = 0;
            if (k0 + tid < n) {
                key = sorted[k0 + tid];
                holds = MASS ? mass(unordered(ord_of(key))) : 1;
            }
            const u64 ahead = base + block_scan(holds, s.warp64, &all);
            if (ahead < want && want <= ahead + holds) s.pick_key = key;
            if (ahead < want && key != 0) keep(key);
            base += all;
        }
        __syncthreads();
    }

    // The cut's key, from the range of ordered bits where it lies.
    template <bool MASS>
    __device__ __noinline__ u64 refine(Floor floor, uint32_t lo_bits, uint32_t hi_bits, u64 want)
    {
        uint32_t bin = 0, i_lo = 0, i_hi = vocab - 1;   // its index's range, once lo_bits == hi_bits
        const auto same = [&](u64) { return want; };
        for (;;) {
            // A range that ends at -0 ends below it: 0 compares equal, but its
            // bits are above the range, and its place in a histogram would be
            // far outside.
            if (hi_bits == kOrderedMinusZero) --hi_bits;
            const float v_lo = unordered(lo_bits), v_hi = unordered(hi_bits);
            const bool tie = lo_bits == hi_bits;
            const auto inside = [&](float v, int i) {
                return v >= v_lo & v <= v_hi & floor.takes(v, i) &
                       (!tie | (static_cast<unsigned>(i) >= i_lo & static_cast<unsigned>(i) <= i_hi));
            };
            begin_list();
            each_chunk(v_lo, [&](const float (&x)[kEach], unsigned c) {
                uint32_t which = 0;
#pragma unroll
                for (int e = 0; e < kEach; ++e) which |= inside(x[e], index_at(c) + e) ? 1u << e : 0u;
                add_tokens(x, c, which);
            });
            const uint32_t n = merge_lists(nullptr);
            if (n <= kList) {
                if (rank == 0) {
                    resolve<MASS>(n, hi_bits, lo_bits, want, [](u64) {});
                    if (tid < blocks) put(&s.cut, tid, s.pick_key);
                }
                meet();
                return s.cut;
            }
            // The next level's bins: of ordered bits, or of indices.
            const uint32_t width = tie ? i_hi - i_lo : hi_bits - lo_bits;
            unsigned shift = 0;
            while (width >> shift >= kBins) ++shift;
            histogram<MASS, false>(v_lo, [&](float v, int i) {
                if (!inside(v, i)) return -1;
                return static_cast<int>((tie ? static_cast<unsigned>(i) - i_lo : hi_bits - ordered(v)) >> shift);
            }, same, want, bin);
            if (tie) {
                i_lo += bin << shift;
                i_hi = min(i_hi, i_lo + ((1u << shift) - 1));
            } else {
                hi_bits -= bin << shift;
                lo_bits = max(lo_bits, hi_bits >= (1u << shift) - 1 ? hi_bits - ((1u << shift) - 1) : 0u);
            }
        }
    }

    // On a copy, so that this object's members can stay in registers.
    template <bool MASS>
    __device__ __forceinline__ u64 refined(const Floor &floor, uint32_t lo_bits, uint32_t hi_bits, u64 want)
    {
        Draw copy = *this;
        const u64 cut = copy.template refine<MASS>(floor, lo_bits, hi_bits, want);
        turn = copy.turn;
        return cut;
    }

    // The last cut and the race in one pass: tokens above the range where the
    // cut lies race at once, those in it are listed, and block 0 races the kept
    // ones.  Returns false, with `cut` alone, if they do not fit the list or
    // there is nothing to cut off.
    template <bool MASS, class Want>
    __device__ __forceinline__ bool cut_and_race(u64 floor_key, Want wanted, float m, u64 &cut, Race &o)
    {
        const Floor floor(floor_key);
        u64 want = 0;
        uint32_t lo_bits = 0, hi_bits = 0;
        cut = floor_key;
        if (!bracket<MASS>(floor, wanted, want, lo_bits, hi_bits)) return false;
        const float v_lo = unordered(lo_bits), v_hi = unordered(hi_bits), low = fmaxf(v_lo, floor.v);
        prefetch_noise(low);
        begin_list();
        const bool aligned = reinterpret_cast<uintptr_t>(noise + first) % 16 == 0;
        unsigned waiting = 0;
        const unsigned rounds = (mine + kPair * kThreads - 1) / (kPair * kThreads);
        const auto in_range = [&](float v, int i) { return v >= v_lo & v <= v_hi & floor.takes(v, i); };
        // A pair's noise is on its way while the pair before it races.
        float x[kOwn], n[kOwn];
        bool in = own(tid, low, x);
        if (in) own_noise(tid, aligned, n);
#pragma unroll 1
        for (unsigned k = 0; k <= rounds; ++k) {
            const unsigned c = k * kPair * kThreads + tid, then = c + kPair * kThreads;
            float x_then[kOwn], n_then[kOwn];
            const bool in_then = own(then, low, x_then);
            if (in_then) own_noise(then, aligned, n_then);
            bool some = false;
            if (in) {
                race_chunk<true>(x, n, c, m, [&](float v, int) { return v > v_hi; }, o);
#pragma unroll
                for (int e = 0; e < kOwn; ++e) some |= in_range(x[e], own_index(c, e));
            }
            queue_up(waiting, some, k * 32 + lane, k == rounds, [&](unsigned at) {
                const unsigned from = (at / 32) * kPair * kThreads + warp * 32 + at % 32;
#pragma unroll 1
                for (int u = 0; u < kPair; ++u) {
                    const unsigned f = from + u * kThreads;
                    if (f >= mine) continue;
                    visit(kept[f], low, f, [&](const float (&v)[kEach], unsigned) {
                        uint32_t which = 0;
#pragma unroll
                        for (int e = 0; e < kEach; ++e) which |= in_range(v[e], index_at(f) + e) ? 1u << e : 0u;
                        add_tokens(v, f, which);
                    });
                }
            });
            in = in_then;
#pragma unroll
            for (int e = 0; e < kOwn; ++e) x[e] = x_then[e], n[e] = n_then[e];
        }
        const uint32_t tokens = merge_lists(nullptr);
        if (tokens > kList) {
            o = Race();
            cut = refined<MASS>(floor, lo_bits, hi_bits, want);
            return false;
        }
        if (rank == 0)
            resolve<MASS>(tokens, hi_bits, lo_bits, want, [&](u64 key) {
                const float w = weight(unordered(ord_of(key)));
                const int i = static_cast<int>(index_of(key));
                if (w >= m) o.offer(w, noise[i], i);
            });
        return true;
    }
};

// Rows whose cut needs histograms, left by the first launch to the second.
// The second starts when every row of the first is either drawn, put down
// here, or in a race of all its tokens: these take longest, and go on beside it.
struct Deferred {
    uint32_t *rows;
    unsigned *count, *decided;       // rows put down; rows that are put down or will not be
    unsigned *next, *left;           // rows that the second launch has taken up; its blocks that are through

    // By one thread of the row's cluster, once.
    __device__ __forceinline__ void decide(bool put_down, unsigned row) const
    {
        if (rows == nullptr) return;
        if (put_down) rows[atomicAdd(count, 1u)] = row;
        __threadfence();   // the row before the word that counts it
        atomicAdd(decided, 1u);
    }
};

// What a row asks for.
struct Setting {
    float t, p, m;
    int k;                           // 0: all
    bool greedy, by_mass, plain, whole;
    __device__ __forceinline__ Setting(const SampleCall &call, unsigned r)
    {
        t = call.temperature != nullptr ? call.temperature[r] : 1.0f;
        k = call.top_k != nullptr ? call.top_k[r] : 0;
        if (k <= 0 || static_cast<unsigned>(k) >= call.vocab) k = 0;
        p = call.top_p != nullptr ? call.top_p[r] : 1.0f;
        m = call.min_p != nullptr ? call.min_p[r] : 0.0f;
        // One token stays, the first of the order: no draw.
        greedy = call.noise == nullptr || !(t > 0.0f) || k == 1 || call.vocab == 1 || !(p > 0.0f) || !(m <= 1.0f);
        by_mass = !(p >= 1.0f);
        plain = !greedy && k == 0 && !by_mass && !(m > 0.0f);   // a race of all tokens
        whole = !greedy && k == 0 && by_mass;                   // top-p over the whole row
    }
};

// What a launch does: every row, leaving out those that need histograms; every
// row; the rows that the first kind has left out, a cluster taking every so
// many of them.  Four blocks per SM for the first, whose rows are many and
// wait for memory; two for the others, whose passes want registers.
enum class Pass { Plain, Whole, Left };
template <Pass PASS> constexpr int kBlocksPerSm = PASS == Pass::Plain ? 4 : 2;
template <Pass PASS> constexpr bool kKeeps = PASS != Pass::Plain;

// One row by one cluster.
template <class T, Pass PASS>
__device__ __forceinline__ void draw_row(Draw<T, kKeeps<PASS>> &d, unsigned r, const SampleCall &call, unsigned per,
                                         const Deferred &later)
{
    constexpr bool HISTOGRAMS = kKeeps<PASS>;
    using D = Draw<T, HISTOGRAMS>;
    Shared &s = d.s;
    const unsigned vocab = d.vocab;
    d.row = static_cast<const T *>(call.logits) + static_cast<size_t>(r) * call.stride;
    d.noise = call.noise + static_cast<size_t>(r) * call.noise_stride;
    d.infinite = false;
    d.place(per);

    const Setting ask(call, r);
    const float t = ask.t, p = ask.p, m = ask.m;
    const int k = ask.k;
    const bool greedy = ask.greedy, by_mass = ask.by_mass, plain = ask.plain, whole = ask.whole;
    const bool cuts = !greedy && (k > 0 || by_mass), first_thread = d.rank == 0 && d.tid == 0;
    const bool listed = cuts && PASS != Pass::Left;   // rows are left because a list does not do
    if (!HISTOGRAMS && !listed && first_thread) later.decide(false, r);
    if (!HISTOGRAMS && plain) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    int32_t *token = call.tokens + r;
    float *logprob = call.logprobs != nullptr ? call.logprobs + r : nullptr;
    d.t = t;
    d.scale = fminf(fmaxf(1.4426950408889634f / t, FLT_TRUE_MIN), FLT_MAX);   // 0 times an infinite distance is none
    Race race;
    float most, sum = 0.0f;
    if (plain) most = d.race_all(race);
    else if (whole && listed) most = d.template load<true>(&sum);
    else most = d.template load<false>(nullptr);

    // The largest logit, and the bound for the short list: the least, over the
    // warps whose lanes all hold tokens, of the j-th largest lane maximum.
    const uint32_t lane_top = ordered(most);
    const uint32_t warp_top = __reduce_max_sync(kFullMask, lane_top);
    uint32_t bound = ~0u;
    bool bounded = false;
    if (listed) {
        const unsigned last = (d.chunks - 1) / per;   // the last block with any
        const unsigned full = min(d.mine / 32, static_cast<unsigned>(kWarps));
        const unsigned warps = last * min(per / 32, static_cast<unsigned>(kWarps)) +
                               min((d.chunks - last * per) / 32, static_cast<unsigned>(kWarps));
        const unsigned wanted = k > 0 ? static_cast<unsigned>(k) : min(static_cast<unsigned>(kGuess), kGuessEach * warps);
        const unsigned j = warps > 0 ? (wanted + warps - 1) / warps : 33;
        bounded = j <= 32;
        if (bounded && d.warp < full) {
            uint32_t left = lane_top;
#pragma unroll 1
            for (unsigned i = 0; i < j; ++i) {
                bound = __reduce_max_sync(kFullMask, left);
                const unsigned at = __ballot_sync(kFullMask, left == bound);
                if (d.lane == static_cast<unsigned>(__ffs(at) - 1)) left = 0;
            }
        }
    }
    // For a histogram of counts, the least lane maximum: as many tokens as
    // there are lanes are at or above it.
    if (HISTOGRAMS && cuts && !bounded) bound = __reduce_min_sync(kFullMask, d.tid < d.mine ? lane_top : ~0u);
    if (d.lane == 0) s.warp_a[d.warp] = warp_top, s.warp_b[d.warp] = bound;
    __syncthreads();
    uint32_t top = __reduce_max_sync(kFullMask, s.warp_a[d.lane & (kWarps - 1)]);
    bound = __reduce_min_sync(kFullMask, s.warp_b[d.lane & (kWarps - 1)]);
    if (d.blocks > 1) {
        if (d.tid < d.blocks) {
            put(&s.top[d.rank], d.tid, top);
            put(&s.bound[d.rank], d.tid, bound);
        }
        d.meet();
        const unsigned b = d.lane < d.blocks ? d.lane : 0;
        top = __reduce_max_sync(kFullMask, s.top[b]);
        bound = __reduce_min_sync(kFullMask, s.bound[b]);
    }
    if (top == kOrderedMinusInf) {
        if (first_thread) {
            *token = -1;
            if (logprob != nullptr) *logprob = -inf();
        }
        if (!HISTOGRAMS && listed && first_thread) later.decide(false, r);
        return;
    }
    d.top = unordered(top);
    if (d.top == inf()) {   // the draw is among the infinite ones, which weigh the same
        if (plain) d.template load<false>(nullptr), race = Race();
        d.infinite = true;
        d.top = 0.0f;
        bound = 0;          // all of them
    } else if (plain) {
        d.rescale(race, most, d.top);
        d.template finish<true>(race, token, logprob);
        return;
    }

    // A little further than the bound, and twice as far for more tokens than
    // lanes; what lies further still is in the histogram's last bin.
    d.reach = d.top - unordered(max(bound, kOrderedMinusInf));
    d.reach *= bounded || static_cast<unsigned>(k) <= d.blocks * kThreads ? 1.02f : 2.0f;
    if (!(d.reach > 0.0f && d.reach < FLT_MAX)) d.reach = kCountSpan;

    u64 cut = 0;
    if (greedy) {
        d.each_chunk(d.top, [&](const float (&x)[D::kEach], unsigned c) {
#pragma unroll
            for (int e = 0; e < D::kEach; ++e)
                if (x[e] == d.top) race.score = 1.0f, race.at = min(race.at, d.index_at(c) + e);
        });
        race.tops = first_thread ? 1 : 0;   // one token is kept
        d.template finish<true>(race, token, logprob);
        return;
    }
    if (cuts) {
        if (listed && !bounded && vocab > kList) {   // more tokens than the list holds
            if (!HISTOGRAMS && first_thread) later.decide(true, r);
        } else if (listed) {
            const float low = bounded ? fmaxf(unordered(max(bound, kOrderedMinusInf)), -FLT_MAX) : -FLT_MAX;
            float above = 0.0f, total = 0.0f;
            if (whole) {
                float part;
                d.block_scan(sum * fmaxf(exp2_approx((most - d.top) * d.scale), 0.0f), s.warpf, &part);
                if (d.tid < d.blocks) put(&s.sum_all[d.rank], d.tid, part);
            }
            const bool near = d.blocks > 1;   // few rows: the list's noise is fetched before it is known to be needed
            d.begin_list();
            d.each_chunk(low, [&](const float (&x)[D::kEach], unsigned c) {
                uint32_t which = 0;
#pragma unroll
                for (int e = 0; e < D::kEach; ++e) which |= x[e] >= low ? 1u << e : 0u;
                if (whole) {
#pragma unroll
                    for (int e = 0; e < D::kEach; ++e) above += x[e] >= low ? d.weight(x[e]) : 0.0f;
                }
                if (near && which != 0)
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(d.noise + d.index_at(c) + __ffs(which) - 1));
                d.add_tokens(x, c, which);
            });
            const uint32_t n = d.merge_lists(&above);
            bool enough = true;
            if (whole) {
#pragma unroll 1
                for (unsigned b = 0; b < d.blocks; ++b) total += s.sum_all[b];
                enough = !d.infinite && (low == -FLT_MAX || above > p * total * (1.0f + 1.0f / 4096));
            }
            const bool fits = n <= kList && enough;
            if (!HISTOGRAMS && first_thread) later.decide(!fits, r);
            if (fits) {
                if (d.rank != 0) return;
                const uint32_t limit = k > 0 ? min(static_cast<uint32_t>(k), n) : n;
                const u64 *sorted = d.sort(n, ordered(d.top), ordered(low));
                if (by_mass && !whole) {   // the first k's mass
                    float part = 0.0f;
#pragma unroll 1
                    for (uint32_t at = d.tid; at < limit; at += kThreads)
                        part += d.list_weight(unordered(ord_of(sorted[at])));
                    d.block_scan(part, s.warpf, &total);
                }
                const float bar = p * total;
                float listed = 0.0f;
#pragma unroll 1
                for (uint32_t at0 = 0; at0 < limit; at0 += kThreads) {
                    const uint32_t at = at0 + d.tid;
                    float w = 0.0f, all = 0.0f, ahead = 0.0f;
                    u64 key = 0;
                    if (at < limit) {
                        key = sorted[at];
                        w = d.list_weight(unordered(ord_of(key)));
                    }
                    if (by_mass) ahead = listed + d.block_scan(w, s.warpf, &all);
                    listed += all;
                    if (at < limit && (at == 0 || ((!by_mass || ahead < bar) && w >= m)))
                        race.offer(w, d.noise[index_of(key)], static_cast<int>(index_of(key)));
                }
                d.template finish<false>(race, token, logprob);
                return;
            }
        }
        if constexpr (!HISTOGRAMS) {
            return;
        } else {
            const auto tokens_wanted = [&](u64) { return static_cast<u64>(k); };
            const auto mass_wanted = [&](u64 mass) {
                const u64 want = static_cast<u64>(ceil(static_cast<double>(p) * static_cast<double>(mass)));
                return want > 1 ? want : 1ull;
            };
            bool done;
            if (!by_mass) {
                done = d.template cut_and_race<false>(0, tokens_wanted, m, cut, race);
            } else {
                if (k > 0) {
                    u64 want = 0;
                    uint32_t lo_bits = 0, hi_bits = 0;
                    const typename D::Floor all(0);
                    if (d.template bracket<false>(all, tokens_wanted, want, lo_bits, hi_bits))
                        cut = d.template refined<false>(all, lo_bits, hi_bits, want);
                }
                done = d.template cut_and_race<true>(cut, mass_wanted, m, cut, race);
            }
            if (done) {
                d.template finish<true>(race, token, logprob);
                return;
            }
        }
    }

    // Every kept token from the row.  A value that min-p leaves in, with room
    // for the rounding of its weight, bounds the chunks that are looked at.
    const typename D::Floor last_kept(cut);
    const float off = m > 0.0f ? t * logf(m) : -inf();
    const float least = fmaxf(last_kept.v, d.top + 1.001f * off - 1e-5f * t - fabsf(d.top) * 4e-7f);
    const bool aligned = reinterpret_cast<uintptr_t>(d.noise + d.first) % 16 == 0;
    d.each_chunk(fmaxf(least, -FLT_MAX), [&](const float (&x)[D::kEach], unsigned c) {
        float n[D::kEach];
        d.load_noise(c, aligned, n);
        d.template race_chunk<false>(x, n, c, m, [&](float v, int i) { return last_kept.takes(v, i); }, race);
    });
    d.template finish<true>(race, token, logprob);
}

template <class T, Pass PASS>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm<PASS>)
sample_kernel(const SampleCall call, unsigned per, const Deferred later)
{
    extern __shared__ __align__(16) unsigned char s_bytes[];
    Shared &s = *reinterpret_cast<Shared *>(s_bytes);
    constexpr bool kKeep = kKeeps<PASS>;
    Draw<T, kKeep> d(s);
    d.tid = threadIdx.x, d.lane = d.tid & 31, d.warp = d.tid >> 5;
    d.rank = cluster_rank(), d.blocks = cluster_blocks(), d.vocab = call.vocab;
    d.inbox = reinterpret_cast<u64 *>(s_bytes + kSharedBytes);
    d.count = reinterpret_cast<uint32_t *>(d.inbox);
    d.carry = d.count + kBins + 32;
    d.region = d.blocks == 1 ? kList : inbox_keys<kKeep>(d.blocks) / d.blocks;
    d.low_parts = reinterpret_cast<uint32_t *>(d.inbox + inbox_keys<kKeep>(d.blocks));
    d.high_parts = d.low_parts + kBins;
    d.kept = reinterpret_cast<uint4 *>(d.low_parts + kPartWords<kKeep>);
    d.index = reinterpret_cast<float *>(d.kept);
    if (d.blocks > 1) d.meet();   // the blocks' shared memory is there
    if constexpr (PASS != Pass::Left) {
        draw_row<T, PASS>(d, blockIdx.x / d.blocks, call, per, later);
    } else {
        // Every row of the first launch is decided when its blocks let this one
        // start, or about then; if that is not seen soon, at its end.
        unsigned decided = 0;
        for (unsigned polls = 0; polls < kPolls && decided != call.rows; ++polls) {
            asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(decided) : "l"(later.decided) : "memory");
            if (decided != call.rows) __nanosleep(64);
        }
        if (decided != call.rows) asm volatile("griddepcontrol.wait;" ::: "memory");
        __syncthreads();
        // A cluster's first row by its place, then whichever is next; asked for
        // while the row before it is drawn.
        const unsigned n = __ldcg(later.count), clusters = gridDim.x / d.blocks;
#pragma unroll 1
        for (unsigned w = blockIdx.x / d.blocks, turn = 0; w < n; w = s.next[turn], turn ^= 1) {
            unsigned next = 0;
            if (d.rank == 0 && d.tid == 0) next = clusters + atomicAdd(later.next, 1u);
            draw_row<T, PASS>(d, __ldcg(later.rows + w), call, per, later);
            if (d.rank == 0 && d.tid == 0) {
#pragma unroll 1
                for (unsigned b = 0; b < d.blocks; ++b) put(&s.next[turn], b, next);
            }
            d.meet();   // the shared memory is used again from here
        }
        // Not over before the first launch is.
        asm volatile("griddepcontrol.wait;" ::: "memory");
        if (d.tid == 0 && atomicAdd(later.left, 1u) == gridDim.x - 1) {   // every block is through
            *later.count = 0;
            *later.decided = 0;
            *later.next = 0;
            *later.left = 0;
        }
    }
}

template <class T, Pass PASS>
cudaError_t launch_clusters(const SampleCall &call, unsigned clusters, unsigned blocks, const Deferred &later,
                            cudaStream_t s)
{
    // Chunks of a row; one more where it starts inside its first.
    constexpr unsigned kEach = Chunk<T>::kEach;
    constexpr unsigned kEntryChunks = kGroup * kThreads;   // chunks to kThreads entries of the index
    constexpr size_t kMostChunks = (static_cast<size_t>(1) << 18) / kEach + 1;   // of the largest vocabulary
    constexpr bool kKeep = kKeeps<PASS>;
    constexpr size_t kMostEntries = (kMostChunks + kEntryChunks - 1) / kEntryChunks * kThreads;
    constexpr size_t kMostKept = (kMostChunks + kMaxCluster - 1) / kMaxCluster * 16;
    constexpr size_t kMostBytes = kSharedBytes + inbox_keys<kKeep>(kMaxCluster) * 8 + kPartWords<kKeep> * 4 +
                                  (kKeep ? kMostKept : kMostEntries * 4);
    static_assert(kMostBytes <= 227 * 1024, "the largest vocabulary fits");
    static_assert((kMostChunks + kEntryChunks - 1) / kEntryChunks * 32 <= 65536, "a warp's entries have 16-bit names");
    const unsigned chunks = (call.vocab + kEach - 1) / kEach;
    const unsigned per = (chunks + 1 + blocks - 1) / blocks;

    const auto kernel = sample_kernel<T, PASS>;
    static std::atomic<unsigned long long> attribute_set{0};   // one bit per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if ((attribute_set.load() & bit) == 0) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kMostBytes));
        if (e != cudaSuccess) return e;
        attribute_set.fetch_or(bit);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(clusters * blocks);
    cfg.blockDim = dim3(kThreads);
    const size_t entries = (per + kEntryChunks - 1) / kEntryChunks * kThreads;
    cfg.dynamicSmemBytes = kSharedBytes + inbox_keys<kKeep>(blocks) * 8 + kPartWords<kKeep> * 4 +
                           (kKeep ? static_cast<size_t>(per) * 16 : entries * 4);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = blocks;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    // The second launch may start before the first is over.
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = PASS == Pass::Left ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, call, per, later);
}

template <class T>
cudaError_t launch_typed(const SampleCall &call, const Workspace &ws, cudaStream_t s)
{
    const size_t rows = call.rows;
    const unsigned chunks = (call.vocab + Chunk<T>::kEach - 1) / Chunk<T>::kEach;
    const size_t sms = static_cast<size_t>(ws.num_sms), room = sms * kBlocksPerSm<Pass::Whole>;
    const unsigned wide = chunks > kLoneChunks ? kMaxCluster : 1;   // the most blocks that a row of this size is worth
    const unsigned n = static_cast<unsigned>(rows);
    DevState &state = *ws.state;
    const Deferred later{call.row_words, &state.sample_rows, &state.sample_decided, &state.sample_next,
                         &state.sample_left};
    // One launch of blocks that keep their slices, as many to a row as fit on
    // the GPU at once (clusters of eight leave gaps: fewer of them fit), where
    // the slices are small enough for two blocks per SM.  Against two launches
    // (us, one : two): 64 x 131072 bf16 top-k and top-p 12.4 : 16.9, of mixed
    // settings 35 : 46; 100 x 50001 f16 31 : 39; 300 x 8000 bf16 19 : 37; 512 x
    // 30000 bf16 top-p 53 : 116, top-k and top-p 18.8 : 16.8.
    unsigned blocks = 1;
    while (blocks < wide && rows * blocks * 2 <= (blocks * 2 == kMaxCluster ? room / 32 * 27 : room)) blocks *= 2;
    if (later.rows != nullptr && chunks <= blocks * kKeptChunks)
        return launch_clusters<T, Pass::Whole>(call, n, blocks, later, s);
    // Else a launch of blocks that do not, for the rows that need one or two
    // passes, and one of wide clusters for the others (512 x 131072 bf16 of
    // mixed settings: 82 us, in one launch of two or four blocks per row that
    // keep their slices 173 and 127).
    blocks = 1;
    while (blocks < wide && rows * blocks * 2 <= sms * kBlocksPerSm<Pass::Plain>) blocks *= 2;
    cudaError_t e = launch_clusters<T, Pass::Plain>(call, n, blocks, later, s);
    if (e != cudaSuccess || later.rows == nullptr) return e;
    const size_t most = room / wide;
    e = launch_clusters<T, Pass::Left>(call, static_cast<unsigned>(rows < most ? rows : most), wide, later, s);
    // The words that the second would have reset.
    if (e != cudaSuccess) (void)cudaMemsetAsync(&state.sample_rows, 0, 4 * sizeof(unsigned), s);
    return e;
}

}  // namespace
}  // namespace devscan
