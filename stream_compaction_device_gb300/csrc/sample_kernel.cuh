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
// once, for its maximum (and, for top-p alone, its sum).  That pass leaves the
// maximum of every group of four 16-byte chunks in shared memory, an index by
// which later passes read again, out of L2, only the groups that hold a token
// above their bound: a few hundred tokens of a row of 100,000.  The noise is
// read only where a token is kept.  A row without truncation takes one pass
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
//     masses in shared memory, 64 bins per unit of logit, then of ordered
//     bits, then of indices, each inside the bin where the last one crossed
//     the mark, until the tokens inside fit the list.  Masses there are
//     integers (w in units of 2^-31, summed in 64 bits), so no result depends
//     on the order of the atomics.
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
constexpr int kLoads = 8;                  // 16-byte loads in flight per thread
constexpr int kGroup = 4;                  // chunks to an entry of the index
constexpr int kQueue = 64;                 // index entries that a warp has waiting
constexpr unsigned kLeastChunks = 512;     // of a block's slice, where rows are few
constexpr int kList = 1024;                // tokens the short list holds
constexpr int kKeys = kList / kThreads;    // its keys per thread in the sort
constexpr int kBins = 1024;
constexpr float kBinsPerUnit = 64.0f;      // first histogram: bins per unit of logit
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
__device__ __forceinline__ uint4 get(const uint32_t *p, unsigned rank)   // four words, 16-byte aligned
{
    uint4 v;
    asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(remote(p, rank))
                 : "memory");
    return v;
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
    uint4 edge[2];                   // the slice's chunks over the row's ends
    uint16_t queue[kWarps][kQueue];
    uint32_t bins[kBins];            // of the list's sort
    u64 warp64[kWarps];
    float warpf[kWarps];
    uint32_t warp_max[kWarps], warp_bound[kWarps], warp_n[kWarps], warp_least[kWarps];
    // What the blocks tell each other, by rank.
    uint32_t top[kMaxCluster], bound[kMaxCluster];
    uint32_t found[2][kMaxCluster];
    float sum[2][kMaxCluster];
    float sum_all[kMaxCluster];
    u64 won[kMaxCluster];
    float rest[kMaxCluster];
    uint32_t tops[kMaxCluster];
    u64 cut;
    // Results of one block's scans.
    u64 pick_before;
    uint32_t pick_bin, pick_lo, pick_hi;
    uint32_t listed;                 // tokens collected by this block (counting stops above kList)
};
// Keys that block 0's inbox has room for: a wide cluster's blocks do not all
// bring the same number.
__host__ __device__ constexpr unsigned inbox_keys(unsigned blocks) { return blocks == 1 ? kList : 2 * kList; }
constexpr size_t kSharedBytes = (sizeof(Shared) + 127) / 128 * 128;

// KEEP: the first pass leaves the slice in shared memory for the later ones.
template <class T, bool KEEP>
struct Draw {
    using C = Chunk<T>;
    static constexpr int kEach = C::kEach;

    Shared &s;
    u64 *inbox;                      // in block 0: the cluster's tokens, a region of `region` per block
    uint32_t *count, *carry;         // a histogram in the same memory: counts, or the masses' low words;
                                     // the masses' high words
    uint32_t region;
    float *index;                    // maxima of this block's groups of chunks
    const float *noise;              // of the row
    const T *row;
    const uint4 *source;             // the slice
    uint4 *kept;                     // with KEEP its copy in shared memory
    unsigned tid, lane, warp, rank, blocks;
    unsigned vocab, chunks, mine;    // tokens and chunks of the row; chunks of the slice
    unsigned lo, hi;                 // the slice's whole chunks
    int first;                       // index of the slice's first value
    float top, t, scale;             // the largest logit, temperature, log2(e) / T
    bool infinite = false;           // the largest is +inf: it counts as 0, all else as -inf
    int turn = 0;                    // which half of the double buffers is next

    __device__ __forceinline__ Draw(Shared &shared) : s(shared) {}

    // The race among the kept tokens that this thread has seen.
    struct Best {
        float score = -1.0f;
        int at = 0x7fffffff;
        __device__ __forceinline__ void offer(float sc, int i)
        {
            if (sc >= score && (sc > score || i < at)) score = sc, at = i;
        }
        __device__ __forceinline__ u64 key() const
        {
            return score < 0.0f ? 0ull : (static_cast<u64>(__float_as_uint(score)) << 32) | ~static_cast<unsigned>(at);
        }
    };

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

    static __device__ __forceinline__ void unpack(const uint4 &v, uint32_t (&q)[4])
    {
        q[0] = v.x, q[1] = v.y, q[2] = v.z, q[3] = v.w;
    }

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
        const bool head = first < 0 && mine > 0;
        const bool tail = mine > 0 && first + static_cast<int>(mine) * kEach > static_cast<int>(vocab);
        lo = head ? 1 : 0;
        hi = tail ? mine - 1 : mine;
        // The first loads' lines are on their way to L2 before the settings
        // have come, on which the first pass depends.
#pragma unroll
        for (int u = 0; u < kLoads; ++u)
            if (tid + u * kThreads >= lo && tid + u * kThreads < hi)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(source + tid + u * kThreads));
        if (head || tail) {
            if (head && tid == 0) edge_chunk(0, &s.edge[0]);
            if (tail && !(head && mine == 1) && tid == 32) edge_chunk(mine - 1, &s.edge[1]);
            __syncthreads();
        }
    }
    __device__ void edge_chunk(unsigned c, uint4 *to)
    {
        T *v = reinterpret_cast<T *>(to);
        for (int e = 0; e < kEach; ++e) {
            const int i = first + static_cast<int>(c) * kEach + e;
            v[e] = i >= 0 && i < static_cast<int>(vocab) ? row[i] : T(-inf());
        }
    }
    static __device__ __forceinline__ uint4 fill() { return make_uint4(C::kFill, C::kFill, C::kFill, C::kFill); }
    __device__ __forceinline__ uint4 chunk(unsigned c) const
    {
        if (KEEP) return c < mine ? kept[c] : fill();
        return fetch(c);
    }
    __device__ __forceinline__ uint4 fetch(unsigned c) const
    {
        if (c >= lo && c < hi) return __ldg(source + c);
        if (c >= mine) return fill();
        return s.edge[c == 0 && lo == 1 ? 0 : 1];
    }

    // First pass: the thread's largest value, the index, and with SUM the
    // thread's sum of weights relative to it.  Entry (k, thread) of the index
    // is for the chunks thread + (kGroup * k + u) * kThreads.
    template <bool SUM>
    __device__ __forceinline__ float load(float *sum)
    {
        float most = -inf(), held = 0.0f;
        unsigned entry = tid;
        for (unsigned c0 = tid; c0 < mine; c0 += kLoads * kThreads) {
            uint4 v[kLoads];
#pragma unroll
            for (int u = 0; u < kLoads; ++u) v[u] = fetch(c0 + u * kThreads);
            if (KEEP) {
#pragma unroll
                for (int u = 0; u < kLoads; ++u)
                    if (c0 + u * kThreads < mine) kept[c0 + u * kThreads] = v[u];
            }
#pragma unroll
            for (int g = 0; g < kLoads; g += kGroup) {
                float group = -inf();
#pragma unroll
                for (int u = g; u < g + kGroup; ++u) {
                    uint32_t q[4];
                    unpack(v[u], q);
                    group = C::most(q, group);
                }
                if (g == 0 || c0 + g * kThreads < mine) index[entry] = group;
                entry += kThreads;
                if (SUM && group > -inf()) {
                    if (group > most) held *= fmaxf(exp2_approx((most - group) * scale), 0.0f);
                    const float base = fmaxf(most, group);
#pragma unroll
                    for (int u = g; u < g + kGroup; ++u) {
                        uint32_t q[4];
                        unpack(v[u], q);
#pragma unroll
                        for (int e = 0; e < kEach; ++e)
                            held += fmaxf(exp2_approx((C::value(q, e) - base) * scale), 0.0f);
                    }
                }
                most = fmaxf(most, group);
            }
        }
        if (SUM) *sum = held;
        return most;
    }

    // f(chunks, c) for every group with a value of at least `low`: its four
    // chunks, c + u * kThreads of the slice.  A warp queues the index entries
    // that reach `low` and reads 32 groups at a time, one per lane.
    template <class F>
    __device__ __forceinline__ void each_group(float low, F f)
    {
        uint16_t *queue = s.queue[warp];
        unsigned waiting = 0;
        const unsigned entries = (mine + kGroup * kThreads - 1) / (kGroup * kThreads);
        for (unsigned k = 0; k <= entries; ++k) {
            if (k < entries) {
                // A thread's group is there if its first chunk is.
                const bool in = tid + k * kGroup * kThreads < mine && index[k * kThreads + tid] >= low;
                const unsigned some = __ballot_sync(kFullMask, in);
                if (in) queue[waiting + __popc(some & ((1u << lane) - 1))] = static_cast<uint16_t>(k * 32 + lane);
                waiting += __popc(some);
                if (waiting < 32) continue;
            } else if (waiting == 0) {
                return;
            }
            __syncwarp();
            const unsigned taken = min(waiting, 32u);
            const unsigned at = lane < taken ? queue[lane] : 0;
            const unsigned moved = lane + 32 < waiting ? queue[lane + 32] : 0;
            __syncwarp();
            if (lane + 32 < waiting) queue[lane] = static_cast<uint16_t>(moved);
            waiting -= taken;
            if (lane < taken) {
                const unsigned c = (at / 32) * kGroup * kThreads + warp * 32 + at % 32;
                uint4 v[kGroup];
#pragma unroll
                for (int u = 0; u < kGroup; ++u) v[u] = chunk(c + u * kThreads);
                if (infinite) {
#pragma unroll
                    for (int u = 0; u < kGroup; ++u) v[u] = only_infinite(v[u]);
                }
                f(v, c);
            }
            __syncwarp();
        }
    }

    // f(values, i) for every chunk with a value of at least `low`: its kEach
    // values, of which the first is the row's i-th.
    template <class F>
    __device__ __forceinline__ void each_chunk(float low, F f)
    {
        each_group(low, [&](const uint4 (&v)[kGroup], unsigned c) {
#pragma unroll
            for (int u = 0; u < kGroup; ++u) {
                float x[kEach];
                if (values(v[u], x) >= low) f(x, first + static_cast<int>(c + u * kThreads) * kEach);
            }
        });
    }
    // f(value, index) for every value of those chunks.
    template <class F>
    __device__ __forceinline__ void each_above(float low, F f)
    {
        each_chunk(low, [&](const float (&x)[kEach], int i) {
#pragma unroll
            for (int e = 0; e < kEach; ++e) f(x[e], i + e);
        });
    }
    // A chunk's values; returns the largest.
    __device__ __forceinline__ float values(const uint4 &v, float (&x)[kEach]) const
    {
        uint32_t q[4];
        unpack(v, q);
#pragma unroll
        for (int e = 0; e < kEach; ++e) x[e] = C::value(q, e);
        return C::most(q, -inf());
    }

    // The race of the kept tokens of two chunks at a time, so that their noise
    // is in flight together.  keep(value, index).
    template <class Keep>
    __device__ __forceinline__ void race_group(const uint4 (&v)[kGroup], unsigned c, float m, Keep keep, Best &best,
                                               float &rest, uint32_t &tops) const
    {
        const bool aligned = reinterpret_cast<uintptr_t>(noise + first) % 16 == 0;
#pragma unroll
        for (int u0 = 0; u0 < kGroup; u0 += 2) {
            float w[2][kEach], n[2][kEach];
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const unsigned at = c + (u0 + p) * kThreads;
                const int i = first + static_cast<int>(at) * kEach;
                float x[kEach];
                values(v[u0 + p], x);
                bool some = false;
#pragma unroll
                for (int e = 0; e < kEach; ++e) {
                    const float weighs = weight(x[e]);
                    w[p][e] = keep(x[e], i + e) && weighs >= m ? weighs : -1.0f;
                    n[p][e] = 1.0f;
                    some |= w[p][e] >= 0.0f;
                }
                if (some && aligned && at >= lo && at < hi) {
#pragma unroll
                    for (int e = 0; e < kEach; e += 4) {
                        const float4 q = __ldcs(reinterpret_cast<const float4 *>(noise + i + e));
                        n[p][e] = q.x, n[p][e + 1] = q.y, n[p][e + 2] = q.z, n[p][e + 3] = q.w;
                    }
                } else if (some) {
#pragma unroll
                    for (int e = 0; e < kEach; ++e) n[p][e] = w[p][e] >= 0.0f ? __ldcs(noise + i + e) : 1.0f;
                }
            }
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const int i = first + static_cast<int>(c + (u0 + p) * kThreads) * kEach;
#pragma unroll
                for (int e = 0; e < kEach; ++e) {
                    if (w[p][e] < 0.0f) continue;
                    best.offer(fmaxf(__fdividef(w[p][e], n[p][e]), 0.0f), i + e);
                    if (w[p][e] == 1.0f) ++tops;
                    else rest += w[p][e];
                }
            }
        }
    }

    // The chunk with 0 in place of every +inf, and -inf of everything else.
    static __device__ __forceinline__ uint4 only_infinite(const uint4 &v)
    {
        uint32_t q[4];
        unpack(v, q);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint32_t r = 0;
#pragma unroll
            for (int e = 0; e < kEach / 4; ++e)
                if (C::value(q, k * (kEach / 4) + e) != inf()) r |= kEach == 4 ? C::kFill : C::kFill & (0xffffu << (16 * e));
            q[k] = r;
        }
        return make_uint4(q[0], q[1], q[2], q[3]);
    }

    // A race of all tokens needs no selection, so it takes one pass over the
    // logits and the noise side by side.  Weights are relative to the largest
    // logit that the thread has seen; what it holds is scaled down when a
    // larger one comes.
    struct Online {
        float most = -inf(), rest = 0.0f, score = -1.0f;
        uint32_t tops = 0;           // weights of exactly 1; `rest` sums the others
        int at = 0x7fffffff;
    };
    __device__ __forceinline__ void rescale(Online &o, float most) const
    {
        const float f = fmaxf(exp2_approx((o.most - most) * scale), 0.0f);
        o.rest = (o.rest + static_cast<float>(o.tops)) * f;
        o.tops = 0;
        if (o.score > 0.0f) o.score *= f;
        o.most = most;
    }
    template <int N>
    __device__ __forceinline__ void race(Online &o, const float (&v)[N], const float (&q)[N], int i) const
    {
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const float w = fmaxf(exp2_approx((v[e] - o.most) * scale), 0.0f);
            if (w == 1.0f) ++o.tops;
            else o.rest += w;
            const float score = __fdividef(w, q[e]);
            if (score > o.score) o.score = score, o.at = i + e;
        }
    }
    __device__ void race_edge(Online &o, int i0) const
    {
        for (int i = i0 < 0 ? 0 : i0; i < i0 + kEach && i < static_cast<int>(vocab); ++i) {
            const float v[1] = {static_cast<float>(row[i])}, n[1] = {noise[i]};
            if (!(v[0] > -inf())) continue;
            if (v[0] > o.most) rescale(o, v[0]);
            race(o, v, n, i);
        }
    }
    __device__ Online race_all()
    {
        constexpr int kRaceLoads = kEach == 4 ? 4 : 2;   // chunks in flight, beside their noise
        Online o;
        const float *beside = noise + first;
        if (lo == 1 && tid == 0) race_edge(o, first);
        const bool aligned = reinterpret_cast<uintptr_t>(beside) % 16 == 0;
        for (unsigned c0 = tid; c0 < hi; c0 += kRaceLoads * kThreads) {
            uint4 x[kRaceLoads];
            float4 n[kRaceLoads][kEach / 4];
#pragma unroll
            for (int u = 0; u < kRaceLoads; ++u) {
                const unsigned c = c0 + u * kThreads;
                const bool in = c >= lo && c < hi;
                x[u] = in ? ld_stream(source + c) : make_uint4(C::kFill, C::kFill, C::kFill, C::kFill);
#pragma unroll
                for (int k = 0; k < kEach / 4; ++k) {
                    const float *at = beside + static_cast<size_t>(c) * kEach + 4 * k;
                    if (!in) n[u][k] = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
                    else if (aligned) n[u][k] = __ldcs(reinterpret_cast<const float4 *>(at));
                    else n[u][k] = make_float4(__ldcs(at), __ldcs(at + 1), __ldcs(at + 2), __ldcs(at + 3));
                }
            }
#pragma unroll
            for (int u = 0; u < kRaceLoads; ++u) {
                uint32_t bits[4];
                unpack(x[u], bits);
                const float most = C::most(bits, -inf());
                if (most == -inf()) continue;
                if (most > o.most) rescale(o, most);
                float v[kEach], q[kEach];
#pragma unroll
                for (int e = 0; e < kEach; ++e) {
                    v[e] = C::value(bits, e);
                    const float4 &f = n[u][e / 4];
                    q[e] = e % 4 == 0 ? f.x : e % 4 == 1 ? f.y : e % 4 == 2 ? f.z : f.w;
                }
                race(o, v, q, first + static_cast<int>(c0 + u * kThreads) * kEach);
            }
        }
        if (hi < mine && mine > lo && tid == (mine - 1) % kThreads)
            race_edge(o, first + static_cast<int>(mine - 1) * kEach);
        return o;
    }

    // Weight of any value (0 for -inf and NaN): the race and the sums over
    // whole rows.  |error| <= (3 |d| + 3) 2^-24 relative, d = (v - top) / T.
    __device__ __forceinline__ float weight(float v) const { return fmaxf(exp2_approx((v - top) * scale), 0.0f); }
    // Weight of a number in the list, rounded as the definition's steps are.
    __device__ __forceinline__ float list_weight(float v) const
    {
        return v == top ? 1.0f : fmaxf(expf((v - top) / t), 0.0f);
    }
    __device__ __forceinline__ uint32_t mass(float v) const { return __float2uint_rn(weight(v) * 2147483648.0f); }

    __device__ __forceinline__ float block_sum(float v)
    {
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(kFullMask, v, d);
        __syncthreads();
        if (lane == 0) s.warpf[warp] = v;
        __syncthreads();
        v = lane < kWarps ? s.warpf[lane] : 0.0f;
#pragma unroll
        for (int d = kWarps / 2; d >= 1; d >>= 1) v += __shfl_xor_sync(kFullMask, v, d);
        return __shfl_sync(kFullMask, v, 0);
    }

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
        V ahead = 0, total = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < static_cast<int>(warp)) ahead += s_warp[w];
            total += s_warp[w];
        }
        *all = total;
        const V before = __shfl_up_sync(kFullMask, incl, 1);
        return ahead + (lane == 0 ? V(0) : before);
    }

    // Tokens for the list: begin_list(), then add_tokens() by any thread, then
    // merge_lists(), which returns their number over the cluster (the same in
    // every block).  Up to kList they are then in block 0, in any order; more
    // than kList is returned as well if a block has more than its region.
    // sum: a partial sum of each thread, summed into s.sum[which] of every
    // block by rank, with `which` as `turn` was before.
    __device__ __forceinline__ void begin_list()
    {
        if (tid == 0) s.listed = 0;
        __syncthreads();
    }
    // The group's tokens for which in(value, index) holds.  One atomic for a
    // thread's tokens of a group, then stores that wait for nothing.
    template <class In>
    __device__ __forceinline__ void add_tokens(const uint4 (&v)[kGroup], unsigned c, In in)
    {
        uint32_t which = 0;
#pragma unroll
        for (int u = 0; u < kGroup; ++u) {
            float x[kEach];
            values(v[u], x);
            const int i = first + static_cast<int>(c + u * kThreads) * kEach;
#pragma unroll
            for (int e = 0; e < kEach; ++e) which |= in(x[e], i + e) ? 1u << (u * kEach + e) : 0u;
        }
        if (which == 0 || *const_cast<volatile uint32_t *>(&s.listed) > region) return;
        uint32_t k = shared_add(&s.listed, __popc(which));
        if (k + __popc(which) > region) return;
        u64 *list = rank == 0 ? inbox : s.list;
#pragma unroll
        for (int u = 0; u < kGroup; ++u) {
            if ((which >> (u * kEach) & ((1u << kEach) - 1)) == 0) continue;
            float x[kEach];
            values(v[u], x);
            const int i = first + static_cast<int>(c + u * kThreads) * kEach;
#pragma unroll
            for (int e = 0; e < kEach; ++e)
                if (which >> (u * kEach + e) & 1) list[k++] = key_of(ordered(x[e]), static_cast<unsigned>(i + e));
        }
    }
    __device__ uint32_t merge_lists(float sum)
    {
        const int now = turn;
        turn ^= 1;
        const float total = block_sum(sum);
        const uint32_t n = s.listed;
        if (tid < blocks) {
            put(&s.found[now][rank], tid, n <= region ? n : kList + 1);
            put(&s.sum[now][rank], tid, total);
        }
        if (rank != 0 && n <= region)
            for (uint32_t k = tid; k < n; k += kThreads) put(&inbox[rank * region + k], 0, s.list[k]);
        meet();
        uint32_t all = 0;
        for (unsigned b = 0; b < blocks; ++b) all += s.found[now][b];
        if (rank == 0 && blocks > 1 && all <= kList) {   // close the gaps
            static_assert(kWarps >= kMaxCluster, "a warp per block's region");
            if (warp < blocks) {
                uint32_t at = 0;
                for (unsigned b = 0; b < warp; ++b) at += s.found[now][b];
                for (uint32_t k = lane; k < s.found[now][warp]; k += 32) s.list[at + k] = inbox[warp * region + k];
            }
            __syncthreads();
        }
        return all;
    }

    __device__ __forceinline__ float cluster_sum(int which) const
    {
        float v = 0.0f;
        for (unsigned b = 0; b < blocks; ++b) v += s.sum[which][b];
        return v;
    }

    // Puts the first `limit` of the n <= kList merged tokens in descending
    // order, by block 0.  Thread t gets the keys at t + h * kThreads; 0 past
    // the end.  A counting sort in bins of equal width from the largest down to
    // the least, then by key inside a bin, where there are one or two as a
    // rule: a fixed number of barriers, where a sort by comparisons took two to
    // three times as long (300 tokens: 6,300 to 10,900 cycles).
    __device__ void sort(uint32_t n, uint32_t limit, u64 (&a)[kKeys])
    {
        u64 *from = blocks == 1 ? inbox : s.list, *to = blocks == 1 ? s.list : inbox;
        constexpr int kPer = kBins / kThreads;
        u64 key[kKeys];
        uint32_t most = 0, least = ~0u;
#pragma unroll
        for (int h = 0; h < kKeys; ++h) {
            key[h] = tid + h * kThreads < n ? from[tid + h * kThreads] : 0;
            if (key[h] == 0) continue;
            most = max(most, ord_of(key[h]));
            least = min(least, ord_of(key[h]));
        }
        most = __reduce_max_sync(kFullMask, most);
        least = __reduce_min_sync(kFullMask, least);
        if (lane == 0) s.warp_max[warp] = most, s.warp_least[warp] = least;
        static_assert(kPer == 4, "a thread's bins are one 16-byte access");
        reinterpret_cast<uint4 *>(s.bins)[tid] = make_uint4(0, 0, 0, 0);
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            most = max(most, s.warp_max[w]);
            least = min(least, s.warp_least[w]);
        }
        // Places by value, then by index: ties fill their range evenly too.
        const u64 high = static_cast<u64>(most >> C::kSpare) * vocab + vocab - 1;
        const float scaled = kBins / static_cast<float>(high - static_cast<u64>(least >> C::kSpare) * vocab + 1);
        uint32_t bin[kKeys], order[kKeys];
#pragma unroll
        for (int h = 0; h < kKeys; ++h) {
            if (key[h] == 0) continue;
            const u64 at = static_cast<u64>(ord_of(key[h]) >> C::kSpare) * vocab + (vocab - 1 - index_of(key[h]));
            bin[h] = min(static_cast<uint32_t>(static_cast<float>(high - at) * scaled), kBins - 1u);
            order[h] = shared_add(&s.bins[bin[h]], 1);
        }
        __syncthreads();
        uint4 begin = reinterpret_cast<uint4 *>(s.bins)[tid];
        uint32_t all = 0;
        const uint32_t before = block_scan(begin.x + begin.y + begin.z + begin.w, s.warp_n, &all);
        const uint32_t n0 = begin.x, n1 = begin.y, n2 = begin.z;
        begin = make_uint4(before, before + n0, before + n0 + n1, before + n0 + n1 + n2);
        reinterpret_cast<uint4 *>(s.bins)[tid] = begin;
        __syncthreads();
#pragma unroll
        for (int h = 0; h < kKeys; ++h)
            if (key[h] != 0) to[s.bins[bin[h]] + order[h]] = key[h];
        __syncthreads();
#pragma unroll
        for (int h = 0; h < kKeys; ++h) {
            if (key[h] == 0) continue;
            const uint32_t first_of = s.bins[bin[h]], end = bin[h] + 1 < kBins ? s.bins[bin[h] + 1] : n;
            uint32_t place = first_of;
            if (end - first_of > 1)
                for (uint32_t k = first_of; k < end; ++k) place += to[k] > key[h] ? 1u : 0u;
            from[place] = key[h];
        }
        __syncthreads();
#pragma unroll
        for (int h = 0; h < kKeys; ++h) a[h] = tid + h * kThreads < min(n, limit) ? from[tid + h * kThreads] : 0;
    }

    __device__ __forceinline__ void write(u64 won, float rest, uint32_t tops, int32_t *token, float *logprob)
    {
        if (won == 0) {   // no score at all: noise that is not a number
            *token = -1;
            if (logprob != nullptr) *logprob = -inf();
            return;
        }
        const unsigned i = index_of(won);
        *token = static_cast<int32_t>(i);
        if (logprob == nullptr) return;
        const float v = static_cast<float>(row[i]);
        const float d = v == inf() || v == top ? 0.0f : (v - top) / t;
        *logprob = d - log1pf(rest + static_cast<float>(tops - 1));
    }

    // The block's race: thread 0 gets the winner and the sums.
    __device__ __forceinline__ void join(u64 &won, float &rest, uint32_t &tops)
    {
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) {
            const u64 u = __shfl_xor_sync(kFullMask, won, d);
            won = u > won ? u : won;
            rest += __shfl_xor_sync(kFullMask, rest, d);
        }
        tops = __reduce_add_sync(kFullMask, tops);
        __syncthreads();
        if (lane == 0) s.warp64[warp] = won, s.warpf[warp] = rest, s.warp_n[warp] = tops;
        __syncthreads();
        if (tid != 0) return;
#pragma unroll
        for (int w = 1; w < kWarps; ++w) {
            won = s.warp64[w] > won ? s.warp64[w] : won;
            rest += s.warpf[w];
            tops += s.warp_n[w];
        }
    }

    // Joins the blocks' races and writes the row's answer.
    __device__ __forceinline__ void finish(const Best &best, float rest, uint32_t tops, int32_t *token, float *logprob)
    {
        u64 won = best.key();
        join(won, rest, tops);
        if (blocks == 1) {
            if (tid == 0) write(won, rest, tops, token, logprob);
            return;
        }
        if (tid == 0) {
            put(&s.won[rank], 0, won);
            put(&s.rest[rank], 0, rest);
            put(&s.tops[rank], 0, tops);
        }
        meet();
        if (rank != 0 || tid != 0) return;
        won = 0, rest = 0.0f, tops = 0;
        for (unsigned b = 0; b < blocks; ++b) {
            won = s.won[b] > won ? s.won[b] : won;
            rest += s.rest[b];
            tops += s.tops[b];
        }
        write(won, rest, tops, token, logprob);
    }

    // The bin of the first histogram: falls as v grows.
    __device__ __forceinline__ int bin_of(float v) const
    {
        // The sum's last bit is worth 1: its low bits are the rounded bin.
        const float most = static_cast<float>(kBins - 1) / kBinsPerUnit;
        return __float_as_int(fmaf(fminf(top - v, most), kBinsPerUnit, 8388608.0f)) - 0x4b000000;
    }

    // One histogram level: adds what each value holds, then finds the bin
    // where the running total from bin 0 reaches want = wanted(total).  Returns
    // false if it does not; else `bin`, and `want` less what is in the bins
    // before it.
    template <bool MASS, class Bin, class Want>
    __device__ bool histogram(float low, Bin bin_in, Want wanted, u64 &want, uint32_t &bin)
    {
        for (unsigned b = tid; b < kBins; b += kThreads) count[b] = carry[b] = 0;
        __syncthreads();
        each_chunk(low, [&](const float (&x)[kEach], int i) {
            // All of a chunk's atomics are in flight before the first carry is
            // looked at.
            int b[kEach];
            uint32_t holds[kEach], old[kEach];
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                b[e] = bin_in(x[e], i + e);
                holds[e] = b[e] < 0 ? 0 : MASS ? mass(x[e]) : 1;
            }
#pragma unroll
            for (int e = 0; e < kEach; ++e) old[e] = holds[e] != 0 ? shared_add(&count[b[e]], holds[e]) : 0;
            if (MASS) {
#pragma unroll
                for (int e = 0; e < kEach; ++e)
                    if (old[e] + holds[e] < old[e]) shared_add(&carry[b[e]], 1);
            }
        });
        meet();
        // Thread t sums the four bins from 4 t on, of all blocks.
        constexpr int kPer = kBins / kThreads;
        static_assert(kPer == 4, "a thread's bins are one 16-byte read");
        u64 h[kPer] = {0, 0, 0, 0}, own = 0;
#pragma unroll 4
        for (unsigned r = 0; r < blocks; ++r) {
            const uint4 low4 = get(count + kPer * tid, r);
            h[0] += low4.x, h[1] += low4.y, h[2] += low4.z, h[3] += low4.w;
            if (MASS) {
                const uint4 high4 = get(carry + kPer * tid, r);
                h[0] += static_cast<u64>(high4.x) << 32, h[1] += static_cast<u64>(high4.y) << 32;
                h[2] += static_cast<u64>(high4.z) << 32, h[3] += static_cast<u64>(high4.w) << 32;
            }
        }
#pragma unroll
        for (int k = 0; k < kPer; ++k) own += h[k];
        u64 all = 0;
        u64 before = block_scan(own, s.warp64, &all);
        want = wanted(all);
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            if (before < want && want <= before + h[k]) {
                s.pick_bin = kPer * tid + k;
                s.pick_before = before;
            }
            before += h[k];
        }
        meet();   // the histogram's memory is used again from here
        if (all < want) return false;
        bin = s.pick_bin;
        want -= s.pick_before;
        return true;
    }

    // The least ordered bits o with bin_of(o) <= b, by one warp: 32 probes cut
    // the range to a 32nd.
    __device__ uint32_t edge(int b) const
    {
        uint32_t from = ordered(-FLT_MAX), to = ordered(top);
        while (from < to) {
            const uint32_t step = (to - from) / 32 + 1;
            const uint32_t probe = min(from + min(lane * step, to - from), to);
            const unsigned in = __ballot_sync(kFullMask, bin_of(unordered(probe)) <= b);
            const uint32_t at = in == 0 ? 31 : __ffs(in) - 1;   // the first probe inside, or the last outside
            const uint32_t found = __shfl_sync(kFullMask, probe, at);
            const uint32_t before = __shfl_sync(kFullMask, probe, at == 0 ? 0 : at - 1);
            if (in == 0) from = found + 1;
            else if (at == 0) return found;
            else from = before + 1, to = found;
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
        __device__ __forceinline__ bool takes(float x, int at) const { return x > v || (x == v && at <= i); }
    };

    // The range of ordered bits of the first histogram's bin where the cut
    // lies, and what is wanted inside it; false if all that take part hold less
    // than wanted.
    template <bool MASS, class Want>
    __device__ bool bracket(const Floor &floor, Want wanted, u64 &want, uint32_t &lo_bits, uint32_t &hi_bits)
    {
        uint32_t bin = 0;
        // Below top - 23 T a weight rounds to no mass.
        const float least = MASS ? fmaxf(floor.v, top - 23.0f * t) : floor.v;
        if (!histogram<MASS>(least, [&](float v, int i) { return floor.takes(v, i) ? bin_of(v) : -1; }, wanted, want,
                             bin))
            return false;
        if (warp == 0) {
            const uint32_t o = edge(static_cast<int>(bin));
            if (lane == 0) s.pick_lo = o;
        } else if (warp == 1) {
            const uint32_t o = bin == 0 ? ordered(top) : edge(static_cast<int>(bin) - 1) - 1;
            if (lane == 0) s.pick_hi = o;
        }
        __syncthreads();
        lo_bits = s.pick_lo, hi_bits = s.pick_hi;
        return true;
    }

    // Block 0 puts the n merged tokens in order, of which the first that hold
    // `want` are kept.  Thread t gets the keys at t + h * kThreads that are
    // kept, 0 for others; s.pick_before is the last one.
    template <bool MASS>
    __device__ void resolve(uint32_t n, u64 want, u64 (&key)[kKeys])
    {
        u64 base = 0;
        sort(n, n, key);
#pragma unroll
        for (int h = 0; h < kKeys; ++h) {
            u64 holds = 0, total = 0;
            if (tid + h * kThreads < n) holds = MASS ? mass(unordered(ord_of(key[h]))) : 1;
            const u64 ahead = base + block_scan(holds, s.warp64, &total);
            if (ahead < want && want <= ahead + holds) s.pick_before = key[h];
            if (ahead >= want) key[h] = 0;
            base += total;
        }
        __syncthreads();
    }

    // The cut's key, from the range of ordered bits where it lies.
    template <bool MASS>
    __device__ u64 refine(const Floor &floor, uint32_t lo_bits, uint32_t hi_bits, u64 want)
    {
        uint32_t bin = 0, i_lo = 0, i_hi = vocab - 1;   // its index's range, once lo_bits == hi_bits
        const auto same = [&](u64) { return want; };
        for (;;) {
            const float v_lo = unordered(lo_bits), v_hi = unordered(hi_bits);
            const bool tie = lo_bits == hi_bits;
            const auto inside = [&](float v, int i) {
                return v >= v_lo && v <= v_hi && floor.takes(v, i) &&
                       (!tie || (static_cast<unsigned>(i) >= i_lo && static_cast<unsigned>(i) <= i_hi));
            };
            begin_list();
            each_group(v_lo, [&](const uint4 (&v)[kGroup], unsigned c) { add_tokens(v, c, inside); });
            const uint32_t n = merge_lists(0.0f);
            if (n <= kList) {
                if (rank == 0) {
                    u64 key[kKeys];
                    resolve<MASS>(n, want, key);
                    if (tid < blocks) put(&s.cut, tid, s.pick_before);
                }
                meet();
                return s.cut;
            }
            unsigned shift = 0;
            if (!tie) {
                while ((hi_bits - lo_bits) >> shift >= kBins) ++shift;
                histogram<MASS>(v_lo, [&](float v, int i) {
                    return inside(v, i) ? static_cast<int>((hi_bits - ordered(v)) >> shift) : -1;
                }, same, want, bin);
                const uint32_t new_hi = hi_bits - (bin << shift), width = (1u << shift) - 1;
                lo_bits = new_hi - lo_bits > width ? new_hi - width : lo_bits;
                hi_bits = new_hi;
            } else {
                while ((i_hi - i_lo) >> shift >= kBins) ++shift;
                histogram<MASS>(v_lo, [&](float v, int i) {
                    return inside(v, i) ? static_cast<int>((static_cast<unsigned>(i) - i_lo) >> shift) : -1;
                }, same, want, bin);
                i_lo += bin << shift;
                i_hi = min(i_hi, i_lo + ((1u << shift) - 1));
            }
        }
    }

    // The last cut and the race in one pass: tokens in the bins before the
    // cut's race at once, those of its bin are listed, and block 0 races the
    // kept ones.  Returns false, with `cut` alone, if they do not fit the list
    // or there is nothing to cut off.
    template <bool MASS, class Want>
    __device__ bool cut_and_race(u64 floor_key, Want wanted, float m, u64 &cut, Best &best, float &rest, uint32_t &tops)
    {
        const Floor floor(floor_key);
        u64 want = 0;
        uint32_t lo_bits = 0, hi_bits = 0;
        cut = floor_key;
        if (!bracket<MASS>(floor, wanted, want, lo_bits, hi_bits)) return false;
        const float v_lo = unordered(lo_bits), v_hi = unordered(hi_bits);
        begin_list();
        each_group(fmaxf(v_lo, floor.v), [&](const uint4 (&v)[kGroup], unsigned c) {
            race_group(v, c, m, [&](float x, int) { return x > v_hi; }, best, rest, tops);
            add_tokens(v, c, [&](float x, int i) { return x >= v_lo && x <= v_hi && floor.takes(x, i); });
        });
        const uint32_t n = merge_lists(0.0f);
        if (n > kList) {
            best = Best();
            rest = 0.0f, tops = 0;
            cut = refine<MASS>(floor, lo_bits, hi_bits, want);
            return false;
        }
        if (rank == 0) {
            u64 key[kKeys];
            resolve<MASS>(n, want, key);
#pragma unroll
            for (int h = 0; h < kKeys; ++h) {
                if (key[h] == 0) continue;
                const float w = weight(unordered(ord_of(key[h])));
                if (!(w >= m)) continue;
                const int i = static_cast<int>(index_of(key[h]));
                best.offer(fmaxf(__fdividef(w, noise[i]), 0.0f), i);
                if (w == 1.0f) ++tops;
                else rest += w;
            }
        }
        return true;
    }
};

// Rows whose cut needs histograms, left by the first launch to the second.
struct Deferred {
    uint32_t *rows;
    unsigned *count, *left;          // rows put down; blocks of the second launch that are through
};

// One row by one cluster.  Without HISTOGRAMS a row that needs them is put
// down for later.
template <class T, bool HISTOGRAMS>
__device__ __forceinline__ void draw_row(Draw<T, HISTOGRAMS> &d, unsigned r, const SampleCall &call, unsigned per,
                                         const Deferred &later)
{
    using D = Draw<T, HISTOGRAMS>;
    Shared &s = d.s;
    const unsigned vocab = d.vocab;
    d.row = static_cast<const T *>(call.logits) + static_cast<size_t>(r) * call.stride;
    d.noise = call.noise + static_cast<size_t>(r) * call.noise_stride;
    d.infinite = false;
    d.place(per);

    const float t = call.temperature != nullptr ? call.temperature[r] : 1.0f;
    int k = call.top_k != nullptr ? call.top_k[r] : 0;
    if (k <= 0 || static_cast<unsigned>(k) >= vocab) k = 0;
    float p = call.top_p != nullptr ? call.top_p[r] : 1.0f;
    const float m = call.min_p != nullptr ? call.min_p[r] : 0.0f;
    // One token stays, the first of the order: no draw.
    const bool greedy = call.noise == nullptr || !(t > 0.0f) || k == 1 || vocab == 1 || !(p > 0.0f) || !(m <= 1.0f);
    const bool by_mass = !(p >= 1.0f);
    int32_t *token = call.tokens + r;
    float *logprob = call.logprobs != nullptr ? call.logprobs + r : nullptr;

    d.t = t;
    d.scale = fminf(1.4426950408889634f / t, FLT_MAX);
    const bool plain = !greedy && k == 0 && !by_mass && !(m > 0.0f);
    typename D::Online online;
    const bool whole = !greedy && k == 0 && by_mass;   // top-p over the whole row
    float most, sum = 0.0f;
    if (plain) {
        online = d.race_all();
        most = online.most;
    } else if (whole) {
        most = d.template load<true>(&sum);
    } else {
        most = d.template load<false>(nullptr);
    }

    // The largest logit, and the bound for the short list: the least, over the
    // warps whose lanes all hold tokens, of the j-th largest lane maximum.
    const uint32_t lane_top = ordered(most);
    const uint32_t warp_top = __reduce_max_sync(kFullMask, lane_top);
    const unsigned last = (d.chunks - 1) / per;   // the last block with any
    const unsigned full = min(d.mine / 32, static_cast<unsigned>(kWarps));
    const unsigned warps = last * min(per / 32, static_cast<unsigned>(kWarps)) +
                           min((d.chunks - last * per) / 32, static_cast<unsigned>(kWarps));
    const int wanted = k > 0 ? k : min(kGuess, kGuessEach * static_cast<int>(warps));
    const int j = warps > 0 ? (wanted + static_cast<int>(warps) - 1) / static_cast<int>(warps) : 33;
    const bool bounded = !greedy && (k > 0 || by_mass) && j <= 32;
    uint32_t bound = ~0u;
    if (bounded && d.warp < full) {
        uint32_t left = lane_top;
        for (int i = 0; i < j; ++i) {
            bound = __reduce_max_sync(kFullMask, left);
            const unsigned at = __ballot_sync(kFullMask, left == bound);
            if (d.lane == static_cast<unsigned>(__ffs(at) - 1)) left = 0;
        }
    }
    if (d.lane == 0) s.warp_max[d.warp] = warp_top, s.warp_bound[d.warp] = bound;
    __syncthreads();
    if (d.warp == 0) {
        const uint32_t a = __reduce_max_sync(kFullMask, s.warp_max[d.lane & (kWarps - 1)]);
        const uint32_t b = __reduce_min_sync(kFullMask, s.warp_bound[d.lane & (kWarps - 1)]);
        if (d.lane < d.blocks) {
            put(&s.top[d.rank], d.lane, a);
            put(&s.bound[d.rank], d.lane, b);
        }
    }
    d.meet();
    uint32_t top = 0;
    bound = ~0u;
    for (unsigned b = 0; b < d.blocks; ++b) {
        top = max(top, s.top[b]);
        bound = min(bound, s.bound[b]);
    }
    if (top == kOrderedMinusInf) {
        if (d.rank == 0 && d.tid == 0) {
            *token = -1;
            if (logprob != nullptr) *logprob = -inf();
        }
        return;
    }
    d.top = unordered(top);
    typename D::Best best;
    if (plain && d.top != inf()) {
        const float f = fmaxf(exp2_approx((online.most - d.top) * d.scale), 0.0f);
        if (online.at != 0x7fffffff) best.score = online.score * f, best.at = online.at;
        if (f != 1.0f) online.rest = (online.rest + static_cast<float>(online.tops)) * f, online.tops = 0;
        d.finish(best, online.rest, online.tops, token, logprob);
        return;
    }
    if (d.top == inf()) {   // the draw is among the infinite ones, which weigh the same
        if (plain) d.template load<false>(nullptr);
        d.infinite = true;
        d.top = 0.0f;
        bound = 0;          // all of them
    }
    if (greedy) {
        const float value = d.top;
        d.each_above(value, [&](float v, int i) {
            if (v == value) best.offer(1.0f, i);
        });
        d.finish(best, 0.0f, d.rank == 0 && d.tid == 0 ? 1 : 0, token, logprob);   // one token is kept
        return;
    }

    u64 cut = 0;
    if (k > 0 || by_mass) {
        const float low = bounded ? fmaxf(unordered(max(bound, kOrderedMinusInf)), -FLT_MAX) : -FLT_MAX;
        const float scaled = whole ? sum * fmaxf(exp2_approx((most - d.top) * d.scale), 0.0f) : 0.0f;
        float above = 0.0f;
        if (whole) {
            const float all = d.block_sum(scaled);
            if (d.tid < d.blocks) put(&s.sum_all[d.rank], d.tid, all);
        }
        const int now = d.turn;
        d.begin_list();
        d.each_group(low, [&](const uint4 (&v)[kGroup], unsigned c) {
            d.add_tokens(v, c, [&](float x, int) {
                if (whole && x >= low) above += d.weight(x);
                return x >= low;
            });
        });
        const uint32_t n = d.merge_lists(above);
        float total = 0.0f;
        bool enough = true;
        if (whole) {
            for (unsigned b = 0; b < d.blocks; ++b) total += s.sum_all[b];
            enough = !d.infinite && (low == -FLT_MAX || d.cluster_sum(now) > p * total * (1.0f + 1.0f / 4096));
        }
        if (n <= kList && enough) {
            if (d.rank != 0) return;
            const uint32_t limit = k > 0 ? min(static_cast<uint32_t>(k), n) : n;
            u64 key[kKeys], won = 0;
            d.sort(n, limit, key);
            float w[kKeys], ahead[kKeys], listed = 0.0f, rest = 0.0f;
            uint32_t tops = 0;
#pragma unroll
            for (int h = 0; h < kKeys; ++h)
                w[h] = d.tid + h * kThreads < limit ? d.list_weight(unordered(ord_of(key[h]))) : 0.0f;
            if (by_mass) {
#pragma unroll
                for (int h = 0; h < kKeys; ++h) {
                    if (h > 0 && limit <= static_cast<uint32_t>(h * kThreads)) break;
                    float all_h = 0.0f;
                    ahead[h] = listed + d.block_scan(w[h], s.warpf, &all_h);
                    listed += all_h;
                }
            }
            const float bar = p * (whole ? total : listed);
#pragma unroll
            for (int h = 0; h < kKeys; ++h) {
                const uint32_t place = d.tid + h * kThreads;
                const bool keep = place < limit && (place == 0 || ((!by_mass || ahead[h] < bar) && w[h] >= m));
                if (!keep) continue;
                const int i = static_cast<int>(index_of(key[h]));
                best.offer(fmaxf(w[h] / d.noise[i], 0.0f), i);
                if (unordered(ord_of(key[h])) == d.top) ++tops;
                else rest += w[h];
            }
            won = best.key();
            d.join(won, rest, tops);
            if (d.tid == 0) d.write(won, rest, tops, token, logprob);
            return;
        }
        if constexpr (!HISTOGRAMS) {
            if (d.rank == 0 && d.tid == 0) later.rows[atomicAdd(later.count, 1u)] = r;
            return;
        } else {
        const auto tokens_wanted = [&](u64) { return static_cast<u64>(k); };
        const auto mass_wanted = [&](u64 mass) {
            const u64 want = static_cast<u64>(ceil(static_cast<double>(p) * static_cast<double>(mass)));
            return want > 1 ? want : 1ull;
        };
        float rest = 0.0f;
        uint32_t tops = 0;
        bool done;
        if (!by_mass) {
            done = d.template cut_and_race<false>(0, tokens_wanted, m, cut, best, rest, tops);
        } else {
            if (k > 0) {
                u64 want = 0;
                uint32_t lo_bits = 0, hi_bits = 0;
                const typename D::Floor all(0);
                if (d.template bracket<false>(all, tokens_wanted, want, lo_bits, hi_bits))
                    cut = d.template refine<false>(all, lo_bits, hi_bits, want);
            }
            done = d.template cut_and_race<true>(cut, mass_wanted, m, cut, best, rest, tops);
        }
        if (done) {
            d.finish(best, rest, tops, token, logprob);
            return;
        }
        }
    }

    const typename D::Floor last_kept(cut);
    float rest = 0.0f;
    uint32_t tops = 0;
    // A value that min-p leaves in, with room for the rounding of its weight.
    const float off = m > 0.0f ? t * logf(m) : -inf();
    const float least = fmaxf(last_kept.v, d.top + 1.001f * off - 1e-5f * t - fabsf(d.top) * 4e-7f);
    d.each_group(fmaxf(least, -FLT_MAX), [&](const uint4 (&v)[kGroup], unsigned c) {
        d.race_group(v, c, m, [&](float x, int i) { return last_kept.takes(x, i); }, best, rest, tops);
    });
    d.finish(best, rest, tops, token, logprob);
}

// What a launch does: every row, leaving out those that need histograms; every
// row; the rows that the first kind has left out, a cluster taking every so
// many of them.  Four blocks per SM for the first, whose rows are many and
// wait for memory; two for the others, whose passes want registers.
enum class Pass { Plain, Whole, Left };
template <Pass PASS> constexpr int kBlocksPerSm = PASS == Pass::Plain ? 4 : 2;

template <class T, Pass PASS>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm<PASS>)
sample_kernel(const SampleCall call, unsigned per, const Deferred later)
{
    extern __shared__ __align__(16) unsigned char s_bytes[];
    Shared &s = *reinterpret_cast<Shared *>(s_bytes);
    constexpr bool kKeep = PASS != Pass::Plain;
    Draw<T, kKeep> d(s);
    d.tid = threadIdx.x, d.lane = d.tid & 31, d.warp = d.tid >> 5;
    d.rank = cluster_rank(), d.blocks = cluster_blocks(), d.vocab = call.vocab;
    d.inbox = reinterpret_cast<u64 *>(s_bytes + kSharedBytes);
    d.count = reinterpret_cast<uint32_t *>(d.inbox);
    d.carry = d.count + kBins;
    d.region = inbox_keys(d.blocks) / d.blocks;
    d.kept = reinterpret_cast<uint4 *>(d.inbox + inbox_keys(d.blocks));
    d.index = reinterpret_cast<float *>(d.kept + (kKeep ? per : 0));
    if (d.blocks > 1) d.meet();   // the blocks' shared memory is there
    if constexpr (PASS != Pass::Left) {
        draw_row<T, kKeep>(d, blockIdx.x / d.blocks, call, per, later);
    } else {
        const unsigned n = *later.count, clusters = gridDim.x / d.blocks;
        for (unsigned w = blockIdx.x / d.blocks; w < n; w += clusters) {
            draw_row<T, kKeep>(d, later.rows[w], call, per, later);
            d.meet();   // the shared memory is used again from here
        }
        if (d.tid == 0 && atomicAdd(later.left, 1u) == gridDim.x - 1) {   // every block has read the count
            *later.count = 0;
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
    constexpr bool kKeep = PASS != Pass::Plain;
    constexpr size_t kMostEntries = (kMostChunks + kEntryChunks - 1) / kEntryChunks * kThreads;
    constexpr size_t kMostKept = kKeep ? (kMostChunks + kMaxCluster - 1) / kMaxCluster * 16 : 0;
    constexpr size_t kMostBytes = kSharedBytes + inbox_keys(kMaxCluster) * 8 + kMostKept +
                                  (kKeep ? kMostEntries / kMaxCluster + kThreads : kMostEntries) * 4;
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
    cfg.dynamicSmemBytes = kSharedBytes + inbox_keys(blocks) * 8 + (kKeep ? static_cast<size_t>(per) * 16 : 0) +
                           static_cast<size_t>((per + kEntryChunks - 1) / kEntryChunks) * kThreads * 4;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = blocks;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, call, per, later);
}

template <class T>
cudaError_t launch_typed(const SampleCall &call, const Workspace &ws, cudaStream_t s)
{
    const Deferred later{call.row_words, &ws.state->sample_rows, &ws.state->sample_left};
    const size_t rows = call.rows;
    const unsigned chunks = (call.vocab + Chunk<T>::kEach - 1) / Chunk<T>::kEach;
    // One block per row, and more while all of them still fit on the GPU at
    // once and have enough of the row each.
    const size_t sms = static_cast<size_t>(ws.num_sms);
    unsigned blocks = 1, wide = 1;   // wide: the most that a row of this size is worth
    while (wide < kMaxCluster && wide * kLeastChunks < chunks) wide *= 2;
    while (blocks < wide && rows * blocks * 2 <= sms * kBlocksPerSm<Pass::Plain>) blocks *= 2;
    if (rows * blocks > 0x7fffffffull) return cudaErrorInvalidValue;
    const unsigned n = static_cast<unsigned>(rows);
    const size_t most = sms * kBlocksPerSm<Pass::Whole> / wide;   // wide clusters on the GPU at once
    if (later.rows != nullptr && rows <= most)
        return launch_clusters<T, Pass::Whole>(call, n, wide, later, s);
    const cudaError_t e = launch_clusters<T, Pass::Plain>(call, n, blocks, later, s);
    if (e != cudaSuccess || later.rows == nullptr) return e;
    // A row that needs histograms takes many times as long as the others:
    // these go to a second launch of wide clusters.
    return launch_clusters<T, Pass::Left>(call, static_cast<unsigned>(rows < most ? rows : most), wide, later, s);
}

}  // namespace
}  // namespace devscan
