// Gated linear recurrence over rows of tokens, and its gradient (sm_103a).
//
//   h_t = a_t h_{t-1} + b_t   for every channel of a row on its own,
//   decay   : a = gate,          b = x
//   log     : a = exp(gate),     b = x
//   sigmoid : a = 1 - r,         b = r x,   r = 1 / (1 + exp(gate))
//
// geek-doc.cn "并行前缀和 scan ..." section 一: any associative operator can be
// scanned, and so can the maps h -> A h + H, which compose to
// (A2, H2) o (A1, H1) = (A2 A1, A2 H1 + H2).  The levels are those of its
// sections 四 and 五: a thread's tokens in order, a block's warps through
// shared memory, the blocks of a cluster through distributed shared memory,
// and a running carry from one round of the cluster to its next.
//
// A row's first token replaces what came before instead of multiplying it by
// zero, so that an infinity or NaN of one row stays in that row.
//
// Layout.  Channels are contiguous, so lanes are channels (4 bytes of x each,
// 128 bytes per warp and token) and nothing is shuffled; a warp takes
// consecutive tokens, a block's eight warps lie behind each other.  Every
// value is read once: a warp's tokens of the next rounds come into its own ring
// of shared memory by asynchronous copies (no registers, no block barrier),
// the maps of a round's tokens are folded, handed on, and then the tokens are
// run again, from registers, from the right h.  Pairs of channels go through
// the two-wide fp32 instructions.  Tokens at odd multiples of 2 bytes cannot
// be copied that way; they are loaded into registers a round ahead.
//
// Split.  A cluster takes 32 lanes' channels of one span of whole rows.  Rows
// are handed out first, since rows need no exchange; a row is spread over up to
// sixteen blocks only where rows and channels alone do not fill the GPU.  No
// block waits for another but at the cluster barrier, and the order of sums
// follows from the call's sizes and starts.  Among packed rows, one longer than
// half of all tokens has a launch of its own beside the others'.
//
// What bounds it (device time, share of the measured copy rate): 8 x 4096 x 4096
// bf16 sigmoid 158 us forward (76%) and 266-270 us backward (90%): 52 and 91
// instructions per warp and token, with issue slots 62% busy; decay, at 38, is
// nearer to memory (135 us, 89%).  One row of 65,536 x 2048 bf16 log 171 us (70%): eight
// blocks to a cluster, and every round waits for the slowest of 64 warps
// (barrier stalls first, issue slots 48% busy).  Measured and dropped there: a
// round finished while the next is begun (223 us: the barrier's release waits
// for the writes in front of it, and fewer tokens fit in a round), 16 warps to a
// block (304), a relaxed barrier (169, and not sound), the maps of a cluster's
// blocks in dynamic shared memory (183).  Short packed rows leave spans uneven: 24
// rows, 8191 x 1000 fp32 decay, 27 us (54%).
#pragma once

#include <initializer_list>

#include "cluster.cuh"
#include "convert.cuh"
#include "grid_sync.cuh"
#include "launch.h"
#include "search.cuh"

namespace devscan {
namespace gated {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr unsigned kStepThreads = 128;   // of a decode step's block
constexpr int kPortableBlocks = 8, kMostBlocks = 16;   // of a cluster
constexpr int kMostPerSm = 3;   // blocks, where two stages of the ring fit
// Shared memory for a block's ring where an SM holds `blocks`: of its 228 KB,
// 1 KB and the exchange go off for each.
constexpr int ring_bytes(int blocks) { return (228 << 10) / blocks - (18 << 10); }
// Tokens of a warp and round where the values of a lane and token have `bytes`
// bytes: as many as two blocks per SM hold twice (long rows: fewer rounds), or
// fewer, where rows are short.
// `both`: the recurrence's a and b stay in registers; `values`: arrays beside
// the gates.  Without asynchronous copies it is registers that end it.
constexpr int tokens_per_round(int bytes, int copy, bool many, bool both, int values)
{
    if (copy == 0) return !many ? 8 : values > 1 ? 12 : both ? 16 : 24;
    const int most = ring_bytes(2) / (2 * kWarps * 32 * bytes) / 4 * 4;
    const int some = bytes <= 8 && !both ? 12 : 8;
    return !many ? some : both && most > 16 ? 16 : most;
}

// ---------------------------------------------------------------------------
// V neighbouring channels in fp32.  Two go through one instruction.
// ---------------------------------------------------------------------------
template <int V> struct alignas(4 * V) Lanes { float v[V]; };

__device__ __forceinline__ unsigned long long bits(const Lanes<2> &a) { return __builtin_bit_cast(unsigned long long, a); }
__device__ __forceinline__ Lanes<2> lanes(unsigned long long a) { return __builtin_bit_cast(Lanes<2>, a); }

__device__ __forceinline__ Lanes<1> fma(Lanes<1> a, Lanes<1> b, Lanes<1> c) { return {fmaf(a.v[0], b.v[0], c.v[0])}; }
__device__ __forceinline__ Lanes<1> operator*(Lanes<1> a, Lanes<1> b) { return {a.v[0] * b.v[0]}; }
__device__ __forceinline__ Lanes<1> operator+(Lanes<1> a, Lanes<1> b) { return {a.v[0] + b.v[0]}; }
__device__ __forceinline__ Lanes<2> fma(Lanes<2> a, Lanes<2> b, Lanes<2> c)
{
    unsigned long long d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(bits(a)), "l"(bits(b)), "l"(bits(c)));
    return lanes(d);
}
__device__ __forceinline__ Lanes<2> operator*(Lanes<2> a, Lanes<2> b)
{
    unsigned long long d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits(a)), "l"(bits(b)));
    return lanes(d);
}
__device__ __forceinline__ Lanes<2> operator+(Lanes<2> a, Lanes<2> b)
{
    unsigned long long d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits(a)), "l"(bits(b)));
    return lanes(d);
}
template <int V> __device__ __forceinline__ Lanes<V> all(float x)
{
    Lanes<V> a;
#pragma unroll
    for (int k = 0; k < V; ++k) a.v[k] = x;
    return a;
}
template <typename T, int V> __device__ __forceinline__ Lanes<V> lanes_of(typename Raw<T, V>::type raw)
{
    Lanes<V> a;
    unpack<T, V>(raw, a.v);
    return a;
}

// A product of decays.  TERMS: also 1 minus it, from its terms, 1 - p a = (1 - p)
// + (1 - a) p, each rounded relative to what is left of 1.  Decays that are given
// often repeat (those of 16 bits next to 1 are few, and a gate may be all
// tokens'), and then so do the roundings of a product, run after run, to one
// side: (1 - 2^-11)^24 multiplied up is off by 4 times 2^-24, which after 20,000
// tokens left the state 7e-6 off (1e-5 where fp16 decays are drawn).  Decays that
// are computed here have a rounding of their own, which the product's do not pass.
// PAIRS: of two tokens at once; decays of 16 bits have exact products of two
// (8 x 4096 x 4096 bf16: 134 us without terms, 135 with, 140 token by token).
// The terms are those of absolute values where that is free, in single lanes; two
// lanes' terms of decays in 32 bits, which next to -1 would be rounded to one side
// themselves, are left where a sign is negative, and the product is multiplied up.
template <int V, bool TERMS, bool PAIRS> struct Product {
    static constexpr bool kSigns = TERMS && !PAIRS && V > 1;
    Lanes<V> a = all<V>(1.0f), rest = all<V>(0.0f);
    unsigned signs[V] = {};
    // token i's decay, of all in turn
    template <int L> __device__ __forceinline__ void next(const Lanes<V> (&decays)[L], int i)
    {
        static_assert(L % 2 == 0, "whole pairs");
        if constexpr (!PAIRS)
            by(decays[i]);
        else if (i % 2 != 0)
            by(decays[i - 1] * decays[i]);
    }
    __device__ __forceinline__ void by(Lanes<V> b)
    {
        if constexpr (TERMS && V == 1) {
            rest.v[0] = fmaf(1.0f - fabsf(b.v[0]), fabsf(a.v[0]), rest.v[0]);
        } else if constexpr (TERMS) {
            rest = fma(fma(b, all<V>(-1.0f), all<V>(1.0f)), a, rest);
            if constexpr (kSigns)
#pragma unroll
                for (int k = 0; k < V; ++k) signs[k] |= __float_as_uint(b.v[k]);
        }
        a = a * b;
    }
    __device__ __forceinline__ Lanes<V> value() const
    {
        Lanes<V> v = a;
        if constexpr (TERMS)
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const bool small = fabsf(rest.v[k]) < 0.5f && (!kSigns || static_cast<int>(signs[k]) >= 0);
                const float p = 1.0f - rest.v[k];
                v.v[k] = small ? V == 1 ? copysignf(p, a.v[k]) : p : a.v[k];
            }
        return v;
    }
};

// ---------------------------------------------------------------------------
// Gates.  A decay next to 1 acts thousands of times, so its error must not
// lean to one side there: it is 1 plus or minus something small, rounded once.
// ---------------------------------------------------------------------------

// The hardware's 2^x and 1 / x (results below 2^-126 are 0).
__device__ __forceinline__ float hard_exp2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float kLog2E = 1.4426950408889634f;
__device__ __forceinline__ float hard_reciprocal(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// exp(g): near 0 as 1 + (its series to the fourth power, off by less than
// g^5 / 120 < 2^-26); elsewhere the hardware's, off by 2^-22 of values that act
// less than twenty times.
template <int V> __device__ __forceinline__ Lanes<V> exp_decay(Lanes<V> g)
{
    Lanes<V> s = fma(g, all<V>(1.0f / 24), all<V>(1.0f / 6));
    s = fma(g, s, all<V>(0.5f));
    s = fma(g, s, all<V>(1.0f));
    s = g * s;
    s = s + all<V>(1.0f);
    const Lanes<V> t = g * all<V>(kLog2E);
#pragma unroll
    for (int k = 0; k < V; ++k) s.v[k] = fabsf(g.v[k]) < 0.0625f ? s.v[k] : hard_exp2(t.v[k]);
    return s;
}

// With u = exp(-g): 1 / (1 + u) and r = u / (1 + u).  Where u is at most 1 that
// r is the smaller of the two and a is 1 - r, rounded once; elsewhere a is the
// quotient.  (u ends at 2^126: a at 2^-126.)
template <int V> __device__ __forceinline__ void sigmoid_decay(Lanes<V> g, Lanes<V> &a, Lanes<V> &r)
{
    Lanes<V> u = g * all<V>(-kLog2E);
#pragma unroll
    for (int k = 0; k < V; ++k) asm("min.NaN.f32 %0, %1, %2;" : "=f"(u.v[k]) : "f"(hard_exp2(u.v[k])), "f"(0x1p126f));
    a = u + all<V>(1.0f);
#pragma unroll
    for (int k = 0; k < V; ++k) a.v[k] = hard_reciprocal(a.v[k]);
    r = u * a;
    const Lanes<V> rest = fma(r, all<V>(-1.0f), all<V>(1.0f));
#pragma unroll
    for (int k = 0; k < V; ++k) a.v[k] = g.v[k] >= 0.0f ? rest.v[k] : a.v[k];
}

// a, and what x is multiplied by (sigmoid only), from a token's gate.
template <int KIND, int V> __device__ __forceinline__ void coefficients(Lanes<V> gate, Lanes<V> &a, Lanes<V> &r)
{
    a = gate;
    if constexpr (KIND == kGateLog) a = exp_decay(gate);
    if constexpr (KIND == kGateSigmoid) sigmoid_decay(gate, a, r);
}

// ---------------------------------------------------------------------------
// Rows and spans.
// ---------------------------------------------------------------------------

// Index of the last row that begins at or before token n; -1 if none does.
__device__ __forceinline__ int row_at(const GatedRows &rows, int n)
{
    return first_not(rows.rows + 1, [&](int r) { return __ldg(rows.starts + r) <= n; }) - 1;
}

// Index of the first of starts[0 .. count) that is at least `value`; count if
// none is.  A warp looks at 32 places at once: what a launch waits for first is
// two loads behind each other for a thousand rows, instead of ten.
__device__ __forceinline__ int first_start(const int32_t *starts, int count, int value, int lane)
{
    Probes p = {0, count};
    while (p.lo < p.hi) {
        const long long at = p.place(lane);
        p.narrow(__popc(__ballot_sync(kFullMask, at < p.hi && __ldg(starts + at) < value)));
    }
    return p.lo;
}

// A place between packed rows: the first row that begins at or behind `share`
// of the tokens, or, behind all rows (a padded batch, whose end is only cleared),
// the share itself.  And the long row, if it is one, in which the share lies.
struct Cut {
    unsigned at, row;   // where that row begins
    bool is_long;
};
__device__ __forceinline__ Cut cut_at(const GatedRows &rows, unsigned share)
{
    if (share == 0) return {0u, 0u, false};
    const unsigned all = rows.all(), real = min(static_cast<unsigned>(max(__ldg(rows.starts + rows.rows), 0)), all);
    const int r = first_start(rows.starts, rows.rows + 1, static_cast<int>(share), threadIdx.x & 31);
    if (r > rows.rows) return {share, share, false};
    Cut c;
    c.at = min(static_cast<unsigned>(__ldg(rows.starts + r)), all);              // >= share > 0
    c.row = r > 0 ? min(static_cast<unsigned>(max(__ldg(rows.starts + r - 1), 0)), c.at) : c.at;   // < share
    c.is_long = rows.long_from != 0 && c.at - c.row >= rows.long_from && c.at - c.row > real / 2;
    return c;
}

// The tokens of span j: whole rows, but for a row longer than half of all, which
// is the only span of a launch of its own; the middle token is one of its.
__device__ __forceinline__ void span_of(const GatedRows &rows, unsigned j, unsigned &begin, unsigned &end)
{
    if (rows.starts == nullptr) {
        begin = static_cast<unsigned>(static_cast<unsigned long long>(rows.rows) * j / rows.spans) * rows.tokens;
        end = static_cast<unsigned>(static_cast<unsigned long long>(rows.rows) * (j + 1) / rows.spans) * rows.tokens;
        return;
    }
    if (rows.long_row) {
        const Cut c = cut_at(rows, min(static_cast<unsigned>(max(__ldg(rows.starts + rows.rows), 0)), rows.all()) / 2 + 1);
        begin = c.row, end = c.is_long ? c.at : c.row;
        return;
    }
    const unsigned long long all = rows.all();
    const unsigned from = static_cast<unsigned>(all * j / rows.spans), to = static_cast<unsigned>(all * (j + 1) / rows.spans);
    const Cut last = cut_at(rows, to);
    begin = cut_at(rows, from).at, end = last.is_long ? last.row : last.at;
    if (end < begin) end = begin;   // the long row began before; or starts decrease
}

struct TokenPlace {
    int row;
    bool inside, first, last;
};
__device__ __forceinline__ TokenPlace place_of(const GatedRows &rows, unsigned n)
{
    TokenPlace p;
    if (rows.starts == nullptr) {
        const unsigned r = n / rows.tokens, t = n - r * rows.tokens;
        p.row = static_cast<int>(r);
        p.inside = true, p.first = t == 0, p.last = t + 1 == rows.tokens;
        return p;
    }
    // the last row that begins at or before n: of rows that begin alike, the one with tokens
    p.row = row_at(rows, static_cast<int>(n));
    p.inside = p.row >= 0 && p.row < rows.rows;
    // a row that begins in front of the tokens has its first one at 0
    p.first = p.inside && max(__ldg(rows.starts + p.row), 0) == static_cast<int>(n);
    p.last = p.inside && (__ldg(rows.starts + p.row + 1) == static_cast<int>(n + 1) || n + 1 == rows.all());
    return p;
}

// Whether row r has no tokens among those that there are.
__device__ __forceinline__ bool row_empty(const GatedRows &rows, int r)
{
    if (rows.starts == nullptr) return rows.tokens == 0;
    const int a = max(__ldg(rows.starts + r), 0), b = min(__ldg(rows.starts + r + 1), static_cast<int>(rows.all()));
    return a >= b;
}

// Where row r's state lies in a pool, if below its size; that state, or null.
__device__ __forceinline__ int slot_of(const GatedRows &rows, int r) { return rows.slots == nullptr ? r : __ldg(rows.slots + r); }
__device__ __forceinline__ float *state_of(const GatedRows &rows, float *states, int r)
{
    if (states == nullptr) return nullptr;
    const int slot = slot_of(rows, r);
    return static_cast<unsigned>(slot) < static_cast<unsigned>(rows.pool)
               ? states + static_cast<size_t>(slot) * rows.channels
               : nullptr;
}

// ---------------------------------------------------------------------------
// A warp's consecutive tokens n, n + 1, ... (DOWN: n, n - 1, ...).
// ---------------------------------------------------------------------------
struct Run {
    unsigned n, row, t;   // the first token, its row in the arrays and its place there
    int count;
    bool whole;           // all there, and in one row of the arrays
};
template <int L, bool DOWN> __device__ __forceinline__ Run run_of(const GatedRows &rows, unsigned n, int count)
{
    Run r;
    r.n = n, r.count = count;
    r.row = rows.per != rows.all() && count > 0 ? n / rows.per : 0u;
    r.t = n - r.row * rows.per;
    r.whole = count == L && (DOWN ? r.t + 1 >= L : r.t + L <= rows.per);
    return r;
}
__device__ __forceinline__ size_t element(const GatedArray &array, unsigned row, unsigned t)
{
    return row * array.row_stride + t * array.stride;
}

// fn(i, element) for each of the run's tokens.
template <int L, bool DOWN, typename Fn>
__device__ __forceinline__ void walk(const GatedRows &rows, const GatedArray &array, const Run &r, Fn &&fn)
{
    size_t at = element(array, r.row, r.t);
    if (r.whole) {
#pragma unroll
        for (int i = 0; i < L; ++i) {
            fn(i, at);
            at = DOWN ? at - array.stride : at + array.stride;
        }
        return;
    }
    const size_t turn = array.row_stride - (rows.per - 1) * array.stride;   // modulo 2^64
    unsigned t = r.t;
#pragma unroll
    for (int i = 0; i < L; ++i) {
        if (i < r.count) fn(i, at);
        const bool wrap = DOWN ? t == 0 : t + 1 == rows.per;
        if (DOWN) {
            at -= wrap ? turn : array.stride;
            t = wrap ? rows.per - 1 : t - 1;
        } else {
            at += wrap ? turn : array.stride;
            t = wrap ? 0 : t + 1;
        }
    }
}

// Asynchronous copy of up to W bytes (the rest become 0).
template <int W> __device__ __forceinline__ void copy_async(uint32_t to, const void *from, int bytes)
{
    if constexpr (W == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Copies the warp's channels (`bytes` of them, at `base`) of the run's tokens,
// BACK tokens before each, to `to`: 32 words of WORD bytes per token, W bytes
// at a time.
template <int L, bool DOWN, int BACK, int WORD, int W>
__device__ __forceinline__ void copy_tokens(const GatedRows &rows, const GatedArray &array, const Run &r, const char *base,
                                            size_t size, int bytes, uint32_t to, int lane)
{
    constexpr int kPieces = 32 * WORD / W;                        // of a token
    constexpr int kAtOnce = kPieces < 32 ? 32 / kPieces : 1;      // tokens per instruction
    constexpr int kParts = kPieces > 32 ? kPieces / 32 : 1;       // instructions per token
    const int i0 = kPieces < 32 ? lane / kPieces : 0, piece = kPieces < 32 ? lane % kPieces : lane;
    const int left = bytes - piece * W;
    to += i0 * (32 * WORD) + piece * W;
    if (r.whole && (BACK == 0 || r.t >= L)) {
        const size_t stride = array.stride * size;
        const char *from = base + element(array, r.row, r.t - BACK) * size + piece * W;
        from = DOWN ? from - i0 * stride : from + i0 * stride;
#pragma unroll
        for (int j = 0; j < L / kAtOnce; ++j) {
#pragma unroll
            for (int q = 0; q < kParts; ++q)
                if (left > q * 32 * W) copy_async<W>(to + (j * kAtOnce * 32 * WORD + q * 32 * W), from + q * 32 * W, min(left - q * 32 * W, W));
            from = DOWN ? from - kAtOnce * stride : from + kAtOnce * stride;
        }
        return;
    }
#pragma unroll 1
    for (int j = 0; j < L / kAtOnce; ++j) {
        const int i = j * kAtOnce + i0;
        if (i >= r.count) break;
        const unsigned n = DOWN ? r.n - i : r.n + i;
        const unsigned row = n / rows.per, t = n - row * rows.per;
        if (BACK > 0 && t < BACK) continue;   // nothing before it: not looked at
        const char *from = base + element(array, row, t - BACK) * size + piece * W;
#pragma unroll
        for (int q = 0; q < kParts; ++q)
            if (left > q * 32 * W) copy_async<W>(to + j * (kAtOnce * 32 * WORD) + q * 32 * W, from + q * 32 * W, min(left - q * 32 * W, W));
    }
}

// ---------------------------------------------------------------------------
// The exchange of one round: every warp hands in its map, and gets the value
// that comes into it.  The cluster's last warp hands on what goes out of it as
// the next round's carry.
// ---------------------------------------------------------------------------
template <int V, int BLOCKS> struct Exchange {   // BLOCKS: the most of a cluster
    Lanes<V> a[2][kWarps][32], h[2][kWarps][32];                       // this block's warps
    Lanes<V> all_a[2][BLOCKS][32], all_h[2][BLOCKS][32];     // the cluster's blocks
    Lanes<V> carry[2][32];
    unsigned cut[2][kWarps], all_cut[2][BLOCKS];                  // nonzero: the map forgets what comes in
};

template <int V> __device__ __forceinline__ Lanes<V> follow(bool cut, Lanes<V> a, Lanes<V> in, Lanes<V> h)
{
    const Lanes<V> next = fma(a, in, h);
#pragma unroll
    for (int k = 0; k < V; ++k) h.v[k] = cut ? h.v[k] : next.v[k];
    return h;
}
template <int V> __device__ __forceinline__ void st_lanes(uint32_t to, Lanes<V> a)
{
    if constexpr (V == 2)
        asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(to), "l"(bits(a)) : "memory");
    else
        st_cluster(to, a.v[0]);
}

// Two buffers in turn are enough: a block writes a round's buffer after the
// barrier of the round before, at which every reader of the round before that
// has arrived.
template <int V, int BLOCKS>
__device__ __forceinline__ Lanes<V> exchange(Exchange<V, BLOCKS> &x, int turn, int blocks, int rank, int warp, int lane,
                                             Lanes<V> a, Lanes<V> h, bool cut)
{
    x.a[turn][warp][lane] = a, x.h[turn][warp][lane] = h;
    if (lane == 0) x.cut[turn][warp] = cut;
    __syncthreads();
    const unsigned cuts = __ballot_sync(kFullMask, lane < kWarps && x.cut[turn][lane & (kWarps - 1)] != 0);
    if (blocks == 1) {
        Lanes<V> in = x.carry[turn][lane];
        if (cuts == 0) {
#pragma unroll
            for (int w = 0; w < kWarps - 1; ++w)
                if (w < warp) in = fma(x.a[turn][w][lane], in, x.h[turn][w][lane]);
        } else {
#pragma unroll 1
            for (int w = 0; w < warp; ++w) in = follow((cuts >> w) & 1u, x.a[turn][w][lane], in, x.h[turn][w][lane]);
        }
        return in;
    }
    // the map of the block's warps before this one, and of all of them
    Lanes<V> ba = all<V>(1.0f), bh = all<V>(0.0f), fa = ba, fh = bh;
    if (cuts == 0) {
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w == warp) ba = fa, bh = fh;
            const Lanes<V> wa = x.a[turn][w][lane];
            fh = fma(wa, fh, x.h[turn][w][lane]);
            fa = wa * fa;
        }
    } else {
#pragma unroll 1
        for (int w = 0; w < kWarps; ++w) {
            if (w == warp) ba = fa, bh = fh;
            const bool c = (cuts >> w) & 1u;
            const Lanes<V> wa = x.a[turn][w][lane];
            fh = follow(c, wa, fh, x.h[turn][w][lane]);
            fa = c ? wa : wa * fa;
        }
    }
#pragma unroll
    for (int q0 = 0; q0 < BLOCKS; q0 += kWarps) {   // warp q tells block q, and q + kWarps
        const int q = q0 + warp;
        if (q >= blocks) break;
        st_lanes<V>(cluster_addr(&x.all_a[turn][rank][lane], q), fa);
        st_lanes<V>(cluster_addr(&x.all_h[turn][rank][lane], q), fh);
        if (lane == 0) st_cluster(cluster_addr(&x.all_cut[turn][rank], q), cuts);
    }
    cluster_sync();
    Lanes<V> in = x.carry[turn][lane];
    const unsigned all_cuts = __ballot_sync(kFullMask, lane < blocks && x.all_cut[turn][lane & (BLOCKS - 1)] != 0);
    if (all_cuts == 0) {
#pragma unroll
        for (int q = 0; q < BLOCKS - 1; ++q)
            if (q < rank) in = fma(x.all_a[turn][q][lane], in, x.all_h[turn][q][lane]);
    } else {
#pragma unroll 1
        for (int q = 0; q < rank; ++q)
            in = follow((all_cuts >> q) & 1u, x.all_a[turn][q][lane], in, x.all_h[turn][q][lane]);
    }
    return follow((cuts & ((1u << warp) - 1u)) != 0, ba, in, bh);
}

// What goes out of the cluster's last warp.  Not after the last round: another
// block may have left by then.
template <int V, int BLOCKS>
__device__ __forceinline__ void hand_on(Exchange<V, BLOCKS> &x, int turn, int blocks, int rank, int warp, int lane, Lanes<V> h)
{
    if (rank != blocks - 1 || warp != kWarps - 1) return;
    if (blocks == 1) {
        x.carry[turn][lane] = h;
    } else {
        for (int q = 0; q < blocks; ++q) st_lanes<V>(cluster_addr(&x.carry[turn][lane], q), h);
    }
}

// What a block of the grid works on.
struct Work {
    int rank, blocks, channel;
    unsigned span, begin, end;
    bool behind;   // all rows
};
__device__ __forceinline__ Work work_of(const GatedRows &rows, int per_lane)
{
    Work w;
    w.rank = static_cast<int>(cluster_rank()), w.blocks = rows.blocks;
    const unsigned cluster = blockIdx.x / rows.blocks, groups = rows.groups;
    w.span = cluster / groups;
    w.channel = static_cast<int>((cluster % groups) * 32 + (threadIdx.x & 31)) * per_lane;
    span_of(rows, w.span, w.begin, w.end);
    w.behind = rows.starts != nullptr && !rows.long_row && static_cast<int>(w.begin) >= __ldg(rows.starts + rows.rows);
    return w;
}

// A span behind all rows becomes 0 and nothing of it is read.
template <typename R, typename X>
__device__ __forceinline__ void clear_span(const Work &w, const GatedArray &array, X *at)
{
    const unsigned warps = static_cast<unsigned>(w.blocks * kWarps);
    for (unsigned n = w.begin + static_cast<unsigned>(w.rank) * kWarps + (threadIdx.x >> 5); n < w.end; n += warps)
        *reinterpret_cast<R *>(at + element(array, 0, n)) = R{};
}

// The other rows' launch lets a long row's start beside it, which then must not
// end before it.
__device__ __forceinline__ void end_beside(const GatedRows &rows)
{
    if (rows.long_row && blockIdx.x == 0) wait_primary_grid();
}

// Rows that begin or end among a warp's tokens, a bit per token; lane i knows
// token i's row.
struct Edges {
    unsigned first, last, outside;
    int row;
    __device__ int row_of(int i) const { return __shfl_sync(kFullMask, row, i); }
};

// What a warp remembers of the row that it was in last, so that it looks for
// rows only where there may be edges.
struct InRow {
    unsigned begin = 1, end = 0;
};

template <int L, bool DOWN>
__device__ __forceinline__ Edges edges_of(const GatedRows &rows, const Run &r, int lane, InRow &in)
{
    Edges e = {0, 0, 0, 0};
    const unsigned low = DOWN ? r.n - (L - 1) : r.n;   // where count == L
    if (r.count == L && low > in.begin && low + L < in.end) return e;
    const bool mine = lane < r.count;
    TokenPlace p = {0, true, false, false};
    if (mine) p = place_of(rows, DOWN ? r.n - lane : r.n + lane);
    e.first = __ballot_sync(kFullMask, mine && p.first);
    e.last = __ballot_sync(kFullMask, mine && p.last);
    e.outside = __ballot_sync(kFullMask, mine && !p.inside);
    e.row = p.row;
    if (r.count > 0) {
        const bool some = __shfl_sync(kFullMask, p.inside, r.count - 1);   // the row that goes on
        const unsigned row = static_cast<unsigned>(__shfl_sync(kFullMask, p.row, r.count - 1));
        if (some && rows.starts == nullptr) {
            in.begin = row * rows.tokens, in.end = in.begin + rows.tokens;
        } else if (some) {
            in.begin = static_cast<unsigned>(max(__ldg(rows.starts + row), 0));
            in.end = min(static_cast<unsigned>(__ldg(rows.starts + row + 1)), rows.all());
        }
    }
    return e;
}

// Rows without tokens: what goes in comes out, 0 where nothing does.  All spans'
// warps share them, 32 rows at a time, of which a lane looks one up; those that
// have a state are then copied, four in flight.
template <int V>
__device__ __forceinline__ void empty_rows(const GatedRows &rows, const Work &w, bool live, const float *from, float *to)
{
    if (to == nullptr || rows.long_row || (rows.starts == nullptr && rows.tokens > 0)) return;
    const unsigned lane = threadIdx.x & 31, warp = static_cast<unsigned>(w.rank) * kWarps + (threadIdx.x >> 5);
    const long long turn = 32ll * rows.spans * w.blocks * kWarps;
    for (long long r0 = 32ll * (static_cast<long long>(warp) * rows.spans + w.span); r0 < rows.rows; r0 += turn) {
        const long long r = r0 + lane;
        int slot = -1;
        if (r < rows.rows && row_empty(rows, static_cast<int>(r))) slot = slot_of(rows, static_cast<int>(r));
        unsigned found = __ballot_sync(kFullMask, static_cast<unsigned>(slot) < static_cast<unsigned>(rows.pool));
        while (found != 0) {
            float v[4][V] = {};
            size_t at[4];
            int many = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (found == 0) break;
                at[i] = static_cast<size_t>(__shfl_sync(kFullMask, slot, __ffs(found) - 1)) * rows.channels + w.channel;
                found &= found - 1, many = i + 1;
                if (from != nullptr && live)
#pragma unroll
                    for (int k = 0; k < V; ++k) v[i][k] = from[at[i] + k];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < many && live)
#pragma unroll
                    for (int k = 0; k < V; ++k) to[at[i] + k] = v[i][k];
        }
    }
}

// ---------------------------------------------------------------------------
// A warp's ring: stages of a round's tokens, array after array, 32 lanes' words
// per token.  COPY: bytes of an asynchronous copy (16 or 4); 0: the round ahead
// waits in registers, and there is one stage.
// ---------------------------------------------------------------------------
template <typename X, typename G, int V, int L, int VALUES, int COPY> struct Ring {
    using RX = typename Raw<X, V>::type;
    using RG = typename Raw<G, V>::type;
    static constexpr int kTokens = L;
    static constexpr int kX = static_cast<int>(sizeof(RX)), kG = static_cast<int>(sizeof(RG));
    static constexpr int kPart = L * 32 * kX, kGates = VALUES * kPart, kStage = kGates + L * 32 * kG;   // bytes
    static constexpr int kPerSm = COPY > 0 && 2 * kWarps * kStage <= ring_bytes(kMostPerSm) ? kMostPerSm : 2;
    static constexpr int kFit = ring_bytes(kPerSm) / (kWarps * kStage), kStages = COPY == 0 ? 1 : kFit < 4 ? kFit : 4;
    static constexpr int kBytes = kWarps * kStages * kStage;
    static_assert(COPY == 0 || kStages >= 2, "a round is copied while another is read");
    static __device__ __forceinline__ Lanes<V> value(const char *stage, int array, int i, int lane)
    {
        return lanes_of<X, V>(reinterpret_cast<const RX *>(stage + array * kPart)[i * 32 + lane]);
    }
    static __device__ __forceinline__ Lanes<V> gate(const char *stage, int i, int lane)
    {
        return lanes_of<G, V>(reinterpret_cast<const RG *>(stage + kGates)[i * 32 + lane]);
    }
    // fp32 values in the place of a lane's own first value and gate
    static __device__ __forceinline__ void put(char *stage, int i, int lane, Lanes<V> b)
    {
        char *value = stage + (i * 32 + lane) * kX, *gate = stage + kGates + (i * 32 + lane) * kG;
        if constexpr (kG >= 4 * V) {
            *reinterpret_cast<Lanes<V> *>(gate) = b;
        } else {   // half of it in each
            __builtin_memcpy(value, &b, 2 * V);
            __builtin_memcpy(gate, reinterpret_cast<const char *>(&b) + 2 * V, 2 * V);
        }
    }
    static __device__ __forceinline__ Lanes<V> get(const char *stage, int i, int lane)
    {
        const char *value = stage + (i * 32 + lane) * kX, *gate = stage + kGates + (i * 32 + lane) * kG;
        Lanes<V> b;
        if constexpr (kG >= 4 * V) {
            b = *reinterpret_cast<const Lanes<V> *>(gate);
        } else {
            __builtin_memcpy(&b, value, 2 * V);
            __builtin_memcpy(reinterpret_cast<char *>(&b) + 2 * V, gate, 2 * V);
        }
        return b;
    }
};

template <typename X, typename G, int V, int VALUES> constexpr int kLaneBytes = V * (VALUES * static_cast<int>(sizeof(X)) + static_cast<int>(sizeof(G)));
template <typename X, typename G, int V, int VALUES, int COPY, bool MANY, bool BOTH>
using RingOf = Ring<X, G, V, tokens_per_round(kLaneBytes<X, G, V, VALUES>, COPY, MANY, BOTH, VALUES), VALUES, COPY>;
template <typename X, typename G, int V, int KIND, int COPY, bool MANY>
using ForwardRing = RingOf<X, G, V, 1, COPY, MANY, KIND == kGateSigmoid>;
template <typename X, typename G, int V, int KIND, int COPY, bool MANY>
using BackwardRing = RingOf<X, G, V, KIND == kGateSigmoid ? 3 : 2, COPY, MANY, false>;

// ---------------------------------------------------------------------------
// Forward.
// ---------------------------------------------------------------------------
template <typename X, typename G, int V, int KIND, int COPY, bool MANY, int BLOCKS>
__global__ void __launch_bounds__(kThreads, (ForwardRing<X, G, V, KIND, COPY, MANY>::kPerSm))
gated_scan_kernel(const __grid_constant__ GatedScanCall p)
{
    constexpr bool SIGMOID = KIND == kGateSigmoid;
    using R = ForwardRing<X, G, V, KIND, COPY, MANY>;
    constexpr int L = R::kTokens;
    using RX = typename R::RX;
    using RG = typename R::RG;
    extern __shared__ __align__(16) char s_ring[];
    __shared__ Exchange<V, BLOCKS> s_x;
    if (p.rows.long_from != 0 && !p.rows.long_row) allow_dependent_launch();
    const int lane = threadIdx.x & 31, warp = __shfl_sync(kFullMask, threadIdx.x >> 5, 0);
    const Work w = work_of(p.rows, V);
    const bool live = w.channel < p.rows.channels;   // a whole number of lanes is
    const int first_channel = w.channel - lane * V;
    const int wide = min(p.rows.channels - first_channel, 32 * V);   // channels of the warp
    const X *x = static_cast<const X *>(p.x.data);
    const G *gate = static_cast<const G *>(p.gate.data);
    X *out = static_cast<X *>(p.out.data) + w.channel;
    char *const ring = s_ring + warp * R::kStages * R::kStage;

    empty_rows<V>(p.rows, w, live, p.initial, p.final);
    if (w.behind) {   // the whole cluster
        if (live) clear_span<RX>(w, p.out, out);
        return;
    }
    if (p.rows.long_row && w.begin == w.end) return end_beside(p.rows);
    const unsigned round = static_cast<unsigned>(w.blocks * kWarps * L);
    const unsigned rounds = (w.end - w.begin + round - 1) / round;
    const unsigned start = w.begin + static_cast<unsigned>((w.rank * kWarps + warp) * L);
    auto run_at = [&](unsigned step) {
        const unsigned n = start + step * round;
        const bool some = step < rounds && n < w.end;
        return run_of<L, false>(p.rows, some ? n : w.begin, some ? static_cast<int>(min(w.end - n, static_cast<unsigned>(L))) : 0);
    };
    constexpr int kKept = COPY > 0 ? 1 : L;
    RX rx[kKept] = {};
    RG rg[kKept] = {};
    auto fetch = [&](unsigned step) {
        const Run r = run_at(step);
        if constexpr (COPY > 0) {
            if (r.count > 0) {
                const uint32_t to = smem_u32(ring + step % R::kStages * R::kStage);
                copy_tokens<L, false, 0, R::kX, COPY>(p.rows, p.x, r, reinterpret_cast<const char *>(x + first_channel),
                                                      sizeof(X), wide * static_cast<int>(sizeof(X)), to, lane);
                copy_tokens<L, false, 0, R::kG, COPY>(p.rows, p.gate, r, reinterpret_cast<const char *>(gate + first_channel),
                                                      sizeof(G), wide * static_cast<int>(sizeof(G)), to + R::kGates, lane);
            }
            copies_commit();
        } else if (live && r.count > 0) {
            walk<L, false>(p.rows, p.x, r, [&](int i, size_t at) { rx[i % kKept] = *reinterpret_cast<const RX *>(x + w.channel + at); });
            walk<L, false>(p.rows, p.gate, r, [&](int i, size_t at) { rg[i % kKept] = *reinterpret_cast<const RG *>(gate + w.channel + at); });
        }
    };
    for (unsigned step = 0; step == 0 || step + 1 < R::kStages; ++step) fetch(step);
    if (warp == 0) s_x.carry[0][lane] = all<V>(0.0f);
    if (w.blocks > 1) cluster_sync();   // every block is there before another writes to it
    InRow in_row;
    for (unsigned step = 0; step < rounds; ++step) {
        const Run r = run_at(step);
        char *const stage = ring + step % R::kStages * R::kStage;
        if constexpr (COPY > 0) {
            fetch(step + R::kStages - 1);   // into the stage that the round before has read
            copies_wait<R::kStages - 1>();
            __syncwarp();
        } else {
#pragma unroll
            for (int i = 0; i < L; ++i) {
                reinterpret_cast<RX *>(stage)[i * 32 + lane] = rx[i % kKept];
                reinterpret_cast<RG *>(stage + R::kGates)[i * 32 + lane] = rg[i % kKept];
            }
            fetch(step + 1);
        }
        const Edges e = edges_of<L, false>(p.rows, r, lane, in_row);
        const unsigned cut = e.first | e.outside;
        const bool plain = r.whole && (cut | e.last) == 0;
        // sigmoid keeps b; the others take x from the ring again
        Lanes<V> a[L], b[SIGMOID ? L : 1], h = all<V>(0.0f);
        Product<V, KIND == kGateDecay, KIND == kGateDecay && sizeof(G) == 2> product;
#pragma unroll
        for (int i = 0; i < L; ++i) {
            Lanes<V> rest;
            coefficients<KIND, V>(R::gate(stage, i, lane), a[i], rest);
            if constexpr (SIGMOID) b[i] = rest * R::value(stage, 0, i, lane);
        }
        auto given = [&](int i) {
            if constexpr (SIGMOID)
                return b[i];
            else
                return R::value(stage, 0, i, lane);
        };
        if (plain) {
#pragma unroll
            for (int i = 0; i < L; ++i) {
                h = fma(a[i], h, given(i));
                product.next(a, i);
            }
        } else {   // b stays in the ring, if not in registers: what it is made of may be overwritten before it is used again
#pragma unroll
            for (int i = 0; i < L; ++i) {
                Lanes<V> now = given(i);
                if (i >= r.count) a[i] = all<V>(1.0f);
                if (i >= r.count || ((e.outside >> i) & 1u)) now = all<V>(0.0f);
                if ((e.first >> i) & 1u) {
                    const float *from = state_of(p.rows, p.initial, e.row_of(i));
                    if (from != nullptr && live)
#pragma unroll
                        for (int k = 0; k < V; ++k) now.v[k] = fmaf(a[i].v[k], from[w.channel + k], now.v[k]);
                }
                if constexpr (SIGMOID)
                    b[i] = now;
                else
                    R::put(stage, i, lane, now);
                const bool c = (cut >> i) & 1u;
                h = follow(c, a[i], h, now);
                product.by(a[i]);   // not used behind a cut
            }
        }
        h = exchange(s_x, step & 1, w.blocks, w.rank, warp, lane, product.value(), h, cut != 0);
        if (plain) {
            X *to = out + element(p.out, r.row, r.t);
#pragma unroll
            for (int i = 0; i < L; ++i) {
                h = fma(a[i], h, given(i));
                if (live) *reinterpret_cast<RX *>(to) = pack<X, V>(h.v);
                to += p.out.stride;
            }
            if (step + 1 < rounds) hand_on(s_x, (step + 1) & 1, w.blocks, w.rank, warp, lane, h);
            __syncwarp();   // the stage has been read
            continue;
        }
#pragma unroll
        for (int i = 0; i < L; ++i) {
            Lanes<V> now;
            if constexpr (SIGMOID)
                now = b[i];
            else
                now = R::get(stage, i, lane);
            h = follow((cut >> i) & 1u, a[i], h, now);
            a[i] = h;
        }
        if (step + 1 < rounds) hand_on(s_x, (step + 1) & 1, w.blocks, w.rank, warp, lane, h);
        __syncwarp();   // the stage has been read
        if (live && r.count > 0)
            walk<L, false>(p.rows, p.out, r, [&](int i, size_t at) { *reinterpret_cast<RX *>(out + at) = pack<X, V>(a[i].v); });
        if (p.final != nullptr) {
#pragma unroll
            for (int i = 0; i < L; ++i) {
                if (((e.last >> i) & 1u) == 0) continue;
                float *to = state_of(p.rows, p.final, e.row_of(i));
                if (to != nullptr && live)
#pragma unroll
                    for (int k = 0; k < V; ++k) to[w.channel + k] = a[i].v[k];
            }
        }
    }
    end_beside(p.rows);
}

// ---------------------------------------------------------------------------
// Backward.  With w_t the gradient of h_t as it is used and handed on,
//   w_t = dh_t + f_{t+1},  f_t = a_t w_t  (f behind a row's last token: the
//   gradient of its final state),
// which is the same recurrence from the last token to the first, and
//   dx_t = w_t (sigmoid: r_t w_t),  da_t = w_t h_{t-1},  dinitial = f_first;
//   da / dgate = 1, a, or a r (h_{t-1} - x_t in place of h_{t-1}).
// h_{t-1} is what the forward call wrote, in its type.  It (and x) is taken
// from the ring after the exchange, so that registers hold a, dh and r only.
// ---------------------------------------------------------------------------
template <typename X, typename G, int V, int KIND, int COPY, bool MANY, int BLOCKS>
__global__ void __launch_bounds__(kThreads, (BackwardRing<X, G, V, KIND, COPY, MANY>::kPerSm))
gated_scan_backward_kernel(const __grid_constant__ GatedBackwardCall p)
{
    constexpr bool SIGMOID = KIND == kGateSigmoid;
    using R = BackwardRing<X, G, V, KIND, COPY, MANY>;   // grad, y, x
    constexpr int L = R::kTokens;
    using RX = typename R::RX;
    using RG = typename R::RG;
    extern __shared__ __align__(16) char s_ring[];
    __shared__ Exchange<V, BLOCKS> s_x;
    if (p.rows.long_from != 0 && !p.rows.long_row) allow_dependent_launch();
    const int lane = threadIdx.x & 31, warp = __shfl_sync(kFullMask, threadIdx.x >> 5, 0);
    const Work w = work_of(p.rows, V);
    const bool live = w.channel < p.rows.channels;
    const int first_channel = w.channel - lane * V;
    const int wide = min(p.rows.channels - first_channel, 32 * V);
    const X *grad = static_cast<const X *>(p.grad.data);
    const X *y = static_cast<const X *>(p.y.data);
    const X *x = static_cast<const X *>(p.x.data);
    const G *gate = static_cast<const G *>(p.gate.data);
    X *grad_x = static_cast<X *>(p.grad_x.data) + w.channel;
    G *grad_gate = static_cast<G *>(p.grad_gate.data) + w.channel;
    char *const ring = s_ring + warp * R::kStages * R::kStage;

    empty_rows<V>(p.rows, w, live, p.grad_final, p.grad_initial);
    if (w.behind) {   // the whole cluster
        if (live) clear_span<RX>(w, p.grad_x, grad_x), clear_span<RG>(w, p.grad_gate, grad_gate);
        return;
    }
    if (p.rows.long_row && w.begin == w.end) return end_beside(p.rows);
    const unsigned round = static_cast<unsigned>(w.blocks * kWarps * L);
    const unsigned tokens = w.end - w.begin, rounds = (tokens + round - 1) / round;
    const unsigned start = static_cast<unsigned>((w.rank * kWarps + warp) * L);   // tokens of the span behind this warp's
    auto run_at = [&](unsigned step) {
        const unsigned done = start + step * round;
        const bool some = step < rounds && done < tokens;
        return run_of<L, true>(p.rows, some ? w.end - 1 - done : w.begin,
                               some ? static_cast<int>(min(tokens - done, static_cast<unsigned>(L))) : 0);
    };
    constexpr int kKept = COPY > 0 ? 1 : L;
    RX rd[kKept] = {}, ry[kKept] = {}, rx[SIGMOID ? kKept : 1] = {};
    RG rg[kKept] = {};
    auto fetch = [&](unsigned step) {
        const Run r = run_at(step);
        if constexpr (COPY > 0) {
            if (r.count > 0) {
                constexpr int size = static_cast<int>(sizeof(X)), gate_size = static_cast<int>(sizeof(G));
                const uint32_t to = smem_u32(ring + step % R::kStages * R::kStage);
                copy_tokens<L, true, 0, R::kX, COPY>(p.rows, p.grad, r, reinterpret_cast<const char *>(grad + first_channel),
                                                     size, wide * size, to, lane);
                copy_tokens<L, true, 1, R::kX, COPY>(p.rows, p.y, r, reinterpret_cast<const char *>(y + first_channel),
                                                     size, wide * size, to + R::kPart, lane);
                if constexpr (SIGMOID)
                    copy_tokens<L, true, 0, R::kX, COPY>(p.rows, p.x, r, reinterpret_cast<const char *>(x + first_channel),
                                                         size, wide * size, to + 2 * R::kPart, lane);
                copy_tokens<L, true, 0, R::kG, COPY>(p.rows, p.gate, r, reinterpret_cast<const char *>(gate + first_channel),
                                                     gate_size, wide * gate_size, to + R::kGates, lane);
            }
            copies_commit();
        } else if (live && r.count > 0) {
            unsigned t = r.t;
            walk<L, true>(p.rows, p.grad, r, [&](int i, size_t at) { rd[i % kKept] = *reinterpret_cast<const RX *>(grad + w.channel + at); });
            walk<L, true>(p.rows, p.gate, r, [&](int i, size_t at) { rg[i % kKept] = *reinterpret_cast<const RG *>(gate + w.channel + at); });
            walk<L, true>(p.rows, p.y, r, [&](int i, size_t at) {
                if (t > 0) ry[i % kKept] = *reinterpret_cast<const RX *>(y + w.channel + (at - p.y.stride));
                t = t == 0 ? p.rows.per - 1 : t - 1;
            });
            if constexpr (SIGMOID)
                walk<L, true>(p.rows, p.x, r, [&](int i, size_t at) { rx[i % kKept] = *reinterpret_cast<const RX *>(x + w.channel + at); });
        }
    };
    for (unsigned step = 0; step == 0 || step + 1 < R::kStages; ++step) fetch(step);
    if (warp == 0) s_x.carry[0][lane] = all<V>(0.0f);
    if (w.blocks > 1) cluster_sync();   // every block is there before another writes to it
    InRow in_row;
    for (unsigned step = 0; step < rounds; ++step) {
        const Run r = run_at(step);
        char *const stage = ring + step % R::kStages * R::kStage;
        if constexpr (COPY > 0) {
            fetch(step + R::kStages - 1);   // into the stage that the round before has read
            copies_wait<R::kStages - 1>();
            __syncwarp();
        } else {
#pragma unroll
            for (int i = 0; i < L; ++i) {
                reinterpret_cast<RX *>(stage)[i * 32 + lane] = rd[i % kKept];
                reinterpret_cast<RX *>(stage + R::kPart)[i * 32 + lane] = ry[i % kKept];
                if constexpr (SIGMOID) reinterpret_cast<RX *>(stage + 2 * R::kPart)[i * 32 + lane] = rx[i % kKept];
                reinterpret_cast<RG *>(stage + R::kGates)[i * 32 + lane] = rg[i % kKept];
            }
            fetch(step + 1);
        }
        Lanes<V> a[L], rest[SIGMOID ? L : 1], d[L];
#pragma unroll
        for (int i = 0; i < L; ++i) {
            coefficients<KIND, V>(R::gate(stage, i, lane), a[i], rest[SIGMOID ? i : 0]);
            d[i] = R::value(stage, 0, i, lane);
        }
        const Edges e = edges_of<L, true>(p.rows, r, lane, in_row);
        const unsigned cut = e.last | e.outside;
        const bool plain = r.whole && (cut | e.first) == 0;
        Lanes<V> f = all<V>(0.0f);
        Product<V, KIND == kGateDecay, KIND == kGateDecay && sizeof(G) == 2> product;
        if (plain) {
#pragma unroll
            for (int i = 0; i < L; ++i) f = a[i] * (d[i] + f), product.next(a, i);
        } else {
#pragma unroll
            for (int i = 0; i < L; ++i) {
                const bool out = (e.outside >> i) & 1u;
                if (i >= r.count) a[i] = all<V>(1.0f);
                if (out) a[i] = all<V>(0.0f);
                if (i >= r.count || out) d[i] = all<V>(0.0f);
                if (((e.last >> i) & 1u) != 0 && p.grad_final != nullptr) {
                    const size_t at = static_cast<size_t>(e.row_of(i)) * p.rows.channels + w.channel;
                    if (live)
#pragma unroll
                        for (int k = 0; k < V; ++k) d[i].v[k] += p.grad_final[at + k];
                }
                const bool c = (cut >> i) & 1u;
                const Lanes<V> sum = d[i] + f;
#pragma unroll
                for (int k = 0; k < V; ++k) f.v[k] = c ? d[i].v[k] : sum.v[k];
                f = a[i] * f;
                product.by(a[i]);   // not used behind a cut
            }
        }
        f = exchange(s_x, step & 1, w.blocks, w.rank, warp, lane, product.value(), f, cut != 0);
        // the gradients of token i from w = v and h_{t-1}
        auto gradients = [&](int i, Lanes<V> v, Lanes<V> before, Lanes<V> &gx, Lanes<V> &gg) {
            gx = v;
            if constexpr (SIGMOID) {
                const Lanes<V> x_here = R::value(stage, 2, i, lane), share = rest[SIGMOID ? i : 0];
                gx = v * share;
                gg = (fma(x_here, all<V>(-1.0f), before) * (a[i] * share)) * v;
            } else {
                gg = (KIND == kGateLog ? before * a[i] : before) * v;
            }
        };
        if (plain) {
            X *to_x = grad_x + element(p.grad_x, r.row, r.t);
            G *to_gate = grad_gate + element(p.grad_gate, r.row, r.t);
#pragma unroll
            for (int i = 0; i < L; ++i) {
                Lanes<V> gx, gg;
                const Lanes<V> v = d[i] + f;
                f = a[i] * v;
                gradients(i, v, R::value(stage, 1, i, lane), gx, gg);
                if (live) {
                    *reinterpret_cast<RX *>(to_x) = pack<X, V>(gx.v);
                    *reinterpret_cast<RG *>(to_gate) = pack<G, V>(gg.v);
                }
                to_x -= p.grad_x.stride, to_gate -= p.grad_gate.stride;
            }
            if (step + 1 < rounds) hand_on(s_x, (step + 1) & 1, w.blocks, w.rank, warp, lane, f);
            __syncwarp();   // the stage has been read
            continue;
        }
        // no gradient for first gates without a state: not 0 times an infinity or NaN
        const unsigned no_gate = e.outside | (!SIGMOID && p.initial == nullptr ? e.first : 0u);
#pragma unroll
        for (int i = 0; i < L; ++i) {
            Lanes<V> v = d[i] + f, before = R::value(stage, 1, i, lane), gx, gg;
#pragma unroll
            for (int k = 0; k < V; ++k) v.v[k] = (cut >> i) & 1u ? d[i].v[k] : v.v[k];
            f = a[i] * v;
            if ((e.first >> i) & 1u) {
                const int row = e.row_of(i);
                const float *from = state_of(p.rows, p.initial, row);
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    before.v[k] = from != nullptr && live ? from[w.channel + k] : 0.0f;
                    if (p.grad_initial != nullptr && live)
                        p.grad_initial[static_cast<size_t>(row) * p.rows.channels + w.channel + k] = f.v[k];
                }
            }
            gradients(i, v, before, gx, gg);
            a[i] = (e.outside >> i) & 1u ? all<V>(0.0f) : gx, d[i] = (no_gate >> i) & 1u ? all<V>(0.0f) : gg;
        }
        if (step + 1 < rounds) hand_on(s_x, (step + 1) & 1, w.blocks, w.rank, warp, lane, f);
        if (live && r.count > 0) {
            walk<L, true>(p.rows, p.grad_x, r, [&](int i, size_t at) { *reinterpret_cast<RX *>(grad_x + at) = pack<X, V>(a[i].v); });
            walk<L, true>(p.rows, p.grad_gate, r, [&](int i, size_t at) { *reinterpret_cast<RG *>(grad_gate + at) = pack<G, V>(d[i].v); });
        }
        __syncwarp();   // the stage has been read
    }
    end_beside(p.rows);
}

// ---------------------------------------------------------------------------
// One token per row: a thread per N channels of a row, 16 bytes of x where that
// is aligned (512 x 4096 bf16 with fp32 states, 29 MB: 7.1 us from memory, 62% of the
// copy rate; where L2 holds them 4.3, and 7.7 with 4 bytes).
// ---------------------------------------------------------------------------
template <typename T, int N> constexpr int kPiece = N * sizeof(T) > 16 ? 16 / static_cast<int>(sizeof(T)) : N;   // values of an access
template <typename T, int N> __device__ __forceinline__ void load_values(const T *from, float (&v)[N])
{
    constexpr int P = kPiece<T, N>;
    typename Raw<T, P>::type raw[N / P];
#pragma unroll
    for (int i = 0; i < N / P; ++i) raw[i] = reinterpret_cast<const typename Raw<T, P>::type *>(from)[i];
#pragma unroll
    for (int i = 0; i < N / P; ++i) unpack<T, P>(raw[i], *reinterpret_cast<float(*)[P]>(v + i * P));
}
template <typename T, int N> __device__ __forceinline__ void store_values(T *to, const float (&v)[N])
{
    constexpr int P = kPiece<T, N>;
#pragma unroll
    for (int i = 0; i < N / P; ++i)
        reinterpret_cast<typename Raw<T, P>::type *>(to)[i] = pack<T, P>(*reinterpret_cast<const float(*)[P]>(v + i * P));
}

template <typename X, typename G, int N, int KIND>
__global__ void __launch_bounds__(kStepThreads) gated_step_kernel(const __grid_constant__ GatedScanCall p, unsigned lanes, unsigned blocks_per_row,
                                                                  unsigned rows_per_block)
{
    // a block has `rows_per_block` whole rows, or one of `blocks_per_row` parts of a row
    const unsigned part = blockIdx.x % blocks_per_row, in_block = threadIdx.x / lanes;
    const unsigned row = blockIdx.x / blocks_per_row * rows_per_block + (blocks_per_row == 1 ? in_block : 0u);
    const unsigned at = blocks_per_row == 1 ? threadIdx.x - in_block * lanes : part * kStepThreads + threadIdx.x;
    if (row >= static_cast<unsigned>(p.rows.rows) || at >= lanes || (blocks_per_row == 1 && in_block >= rows_per_block)) return;
    const int r = static_cast<int>(row);
    const size_t c = static_cast<size_t>(at) * N;
    float gate[N], b[N], h0[N];
    load_values<X, N>(static_cast<const X *>(p.x.data) + r * p.x.row_stride + c, b);
    load_values<G, N>(static_cast<const G *>(p.gate.data) + r * p.gate.row_stride + c, gate);
    const float *from = state_of(p.rows, p.initial, r);
    float *to = state_of(p.rows, p.final, r);
    if (from != nullptr) load_values<float, N>(from + c, h0);
#pragma unroll
    for (int k = 0; k < N; ++k) {
        Lanes<1> a, rest;
        coefficients<KIND, 1>(Lanes<1>{gate[k]}, a, rest);
        if constexpr (KIND == kGateSigmoid) b[k] *= rest.v[0];
        if (from != nullptr) b[k] = fmaf(a.v[0], h0[k], b[k]);
    }
    store_values<X, N>(static_cast<X *>(p.out.data) + r * p.out.row_stride + c, b);
    if (to != nullptr) store_values<float, N>(to + c, b);
}

// A few tokens per row (a draft's, checked at once): a thread goes through its
// channels' tokens, four of them in flight (512 rows x 4096 bf16 sigmoid with
// states, where L2 holds them: 2 tokens 7.0 us, 4 10.4, 16 59; clusters took 20.5,
// 29 and 84.  From memory 12.1, 19.0 and 58).
constexpr int kFewAtOnce = 4;
template <typename X, typename G, int N, int KIND>
__global__ void __launch_bounds__(kStepThreads) gated_few_kernel(const __grid_constant__ GatedScanCall p, unsigned lanes, unsigned blocks_per_row,
                                                                 unsigned rows_per_block)
{
    const unsigned part = blockIdx.x % blocks_per_row, in_block = threadIdx.x / lanes;
    const unsigned row = blockIdx.x / blocks_per_row * rows_per_block + (blocks_per_row == 1 ? in_block : 0u);
    const unsigned at = blocks_per_row == 1 ? threadIdx.x - in_block * lanes : part * kStepThreads + threadIdx.x;
    if (row >= static_cast<unsigned>(p.rows.rows) || at >= lanes || (blocks_per_row == 1 && in_block >= rows_per_block)) return;
    const int r = static_cast<int>(row);
    const size_t c = static_cast<size_t>(at) * N;
    const X *x = static_cast<const X *>(p.x.data) + r * p.x.row_stride + c;
    const G *gate = static_cast<const G *>(p.gate.data) + r * p.gate.row_stride + c;
    X *out = static_cast<X *>(p.out.data) + r * p.out.row_stride + c;
    const float *from = state_of(p.rows, p.initial, r);
    float *to = state_of(p.rows, p.final, r);
    float h[N] = {};
    if (from != nullptr) load_values<float, N>(from + c, h);
    bool state = from != nullptr;
    for (unsigned t0 = 0; t0 < p.rows.tokens; t0 += kFewAtOnce) {
        float b[kFewAtOnce][N], g[kFewAtOnce][N];
#pragma unroll
        for (int i = 0; i < kFewAtOnce; ++i)
            if (t0 + i < p.rows.tokens) {
                load_values<X, N>(x + (t0 + i) * p.x.stride, b[i]);
                load_values<G, N>(gate + (t0 + i) * p.gate.stride, g[i]);
            }
#pragma unroll
        for (int i = 0; i < kFewAtOnce; ++i) {
            if (t0 + i >= p.rows.tokens) break;
#pragma unroll
            for (int k = 0; k < N; ++k) {
                Lanes<1> a, rest;
                coefficients<KIND, 1>(Lanes<1>{g[i][k]}, a, rest);
                if constexpr (KIND == kGateSigmoid) b[i][k] *= rest.v[0];
                h[k] = state ? fmaf(a.v[0], h[k], b[i][k]) : b[i][k];
            }
            state = true;
            store_values<X, N>(out + (t0 + i) * p.out.stride, h);
        }
    }
    if (to != nullptr) store_values<float, N>(to + c, h);
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------

// The widest copies that a call's arrays allow: 16 or 4 bytes, or 0 where a
// lane's `per_lane` values are not aligned as one.
struct Width {
    int per_lane;
    size_t all = 0;
    bool whole = true;
    void add(const GatedArray &a, const GatedRows &rows, size_t size)
    {
        size_t bits = reinterpret_cast<uintptr_t>(a.data) | static_cast<size_t>(rows.channels) * size;
        if (rows.tokens > 1) bits |= a.stride * size;
        if (rows.starts == nullptr && rows.rows > 1) bits |= a.row_stride * size;
        whole = whole && bits % (per_lane * size) == 0;
        all |= bits;
    }
    int copy() const { return !whole ? 0 : all % 16 == 0 ? 16 : 4; }
};

// Tokens of a row as far as addresses go: where every array's rows lie behind
// each other, all tokens are one.
inline void lay_out(GatedRows &rows, std::initializer_list<const GatedArray *> arrays)
{
    bool flat = true;
    for (const GatedArray *a : arrays) flat = flat && (a->data == nullptr || a->row_stride == rows.tokens * a->stride);
    rows.per = flat || rows.starts != nullptr || rows.rows == 1 ? rows.all() : rows.tokens;
    if (rows.per == 0) rows.per = 1;
}

// Spans and blocks per cluster.  Rows are spread first; a span's rows are then
// spread over twice the blocks while there are places for all of them at once
// and every block has a round's tokens.  (An exchange between blocks costs about
// a fifth of a round: backward, 8 x 4096 x 4096, 266 us with one block for a
// span and 319 with two.)
inline void plan(GatedRows &rows, int per_lane, int tokens_per_warp, int places_per_sm, bool many, int sms)
{
    const size_t all = rows.all(), groups = (static_cast<size_t>(rows.channels) + 32 * per_lane - 1) / (32 * per_lane);
    const size_t places = static_cast<size_t>(sms) * places_per_sm, tile = static_cast<size_t>(kWarps) * tokens_per_warp;
    size_t spans = (4 * places + groups - 1) / groups;
    spans = spans < static_cast<size_t>(rows.rows) ? spans : static_cast<size_t>(rows.rows);
    const size_t most = all / (3 * tile);   // spans of three rounds at least: short rows fill a round together
    if (spans > most) spans = most;
    if (spans < 1) spans = 1;
    size_t blocks = 1;
    while (blocks < kPortableBlocks && 2 * groups * spans * blocks <= places && spans * blocks * tile < all) blocks *= 2;
    // More than the portable size where all of them leave half of the SMs without a
    // block (3 x 30,000 x 128 bf16: 57 us with eight blocks, 37 with sixteen).
    if (many && blocks == kPortableBlocks && kMostBlocks * groups * spans <= static_cast<size_t>(sms) && spans * blocks * tile < all)
        blocks = kMostBlocks;
    rows.groups = static_cast<unsigned>(groups), rows.spans = static_cast<unsigned>(spans);
    rows.blocks = static_cast<int>(blocks);
    rows.long_row = false, rows.long_from = 0;
    // Packed rows may hold one that is longer than all others together (a prompt
    // beside single tokens).  One span's blocks would go through it alone, so it
    // has a launch of its own, with up to eight blocks to a cluster: 200 rows of one
    // token and one of 8,000, 2048 bf16 log, 118 -> 48 us (backward 160 -> 58); 50 x 99 and
    // 60,000 770 -> 211.  Where there is none the launch looks and leaves: 0.6 us (24
    // rows, 8191 x 1000 fp32).  With it in front that was 1.9 (and 37 in the first
    // case), and rows of a quarter of all were slower.  Not for rows that one span's
    // blocks finish in eight rounds, nor where channels fill the GPU; nor for rows that
    // are shorter than a span's share (beside a long padded end), since they need
    // not reach a share's end, which is where spans leave them out.
    const size_t share = (all + spans - 1) / spans, rounds = 8 * tile * blocks, least = rounds > share ? rounds : share;
    if (rows.starts != nullptr && spans > 1 && all >= least && blocks < kPortableBlocks && 4 * blocks * groups <= places)
        rows.long_from = static_cast<unsigned>(least);
}

// A long row's own launch.
inline void plan_long(GatedRows &rows, int places_per_sm, int sms)
{
    const size_t places = static_cast<size_t>(sms) * places_per_sm;
    rows.long_row = true, rows.spans = 1;
    while (rows.blocks < kPortableBlocks && 2 * rows.blocks * rows.groups <= places) rows.blocks *= 2;
}

// Whether rows are long enough for many tokens per round (forward, log: 16 x
// 1024 x 4096 bf16 90 us with many and 76 with few; 2 x 8192 x 1024 32 and 37).
// Packed rows go by their average: the host does not know their lengths.
inline bool many_tokens(const GatedRows &rows) { return rows.all() / static_cast<unsigned>(rows.rows > 0 ? rows.rows : 1) >= 2048; }

template <typename Call>
cudaError_t launch_clusters(void (*kernel)(Call), const Call &call, int ring, std::atomic<unsigned long long> &done, cudaStream_t s)
{
    cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void *>(kernel), ring, done);
    if (e != cudaSuccess) return e;
    if (call.rows.blocks > kPortableBlocks &&
        (e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(call.rows.groups * call.rows.spans * static_cast<unsigned>(call.rows.blocks));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(ring);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(call.rows.blocks);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = call.rows.long_row ? 2 : 1;   // beside the others
    return cudaLaunchKernelEx(&cfg, kernel, call);
}

template <typename X, typename G, int V, int KIND, int COPY, bool MANY>
cudaError_t forward_of(GatedScanCall call, int sms, cudaStream_t s)
{
    static std::atomic<unsigned long long> done, more, longs;
    using R = ForwardRing<X, G, V, KIND, COPY, MANY>;
    lay_out(call.rows, {&call.x, &call.gate, &call.out});
    plan(call.rows, V, R::kTokens, R::kPerSm, MANY, sms);
    if constexpr (MANY)
        if (call.rows.blocks > kPortableBlocks)
            return launch_clusters(gated_scan_kernel<X, G, V, KIND, COPY, MANY, kMostBlocks>, call, R::kBytes, more, s);
    const cudaError_t e = launch_clusters(gated_scan_kernel<X, G, V, KIND, COPY, MANY, kPortableBlocks>, call, R::kBytes, done, s);
    if (e != cudaSuccess || call.rows.long_from == 0) return e;
    using Long = ForwardRing<X, G, V, KIND, COPY, true>;
    plan_long(call.rows, Long::kPerSm, sms);
    return launch_clusters(gated_scan_kernel<X, G, V, KIND, COPY, true, kPortableBlocks>, call, Long::kBytes, longs, s);
}
template <typename X, typename G, int V, int KIND, int COPY>
cudaError_t forward(const GatedScanCall &call, int sms, cudaStream_t s)
{
    if (many_tokens(call.rows)) return forward_of<X, G, V, KIND, COPY, true>(call, sms, s);
    return forward_of<X, G, V, KIND, COPY, false>(call, sms, s);
}
template <typename X, typename G, int N, int KIND>
cudaError_t step(const GatedScanCall &call, cudaStream_t s)
{
    const unsigned lanes = static_cast<unsigned>(call.rows.channels / N);
    const unsigned parts = (lanes + kStepThreads - 1) / kStepThreads, rows = lanes < kStepThreads ? kStepThreads / lanes : 1u;
    const size_t blocks = (static_cast<size_t>(call.rows.rows) + rows - 1) / rows * parts;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    if (call.rows.tokens == 1)
        gated_step_kernel<X, G, N, KIND><<<static_cast<unsigned>(blocks), kStepThreads, 0, s>>>(call, lanes, parts, rows);
    else
        gated_few_kernel<X, G, N, KIND><<<static_cast<unsigned>(blocks), kStepThreads, 0, s>>>(call, lanes, parts, rows);
    return cudaGetLastError();
}
// Whether a thread per channels goes through a row's tokens: where they are few,
// or rows make up for it (sigmoid, inputs in L2, clusters against this: 1 x 8 x 4096 bf16 4.7 and
// 4.3 us, 1 x 16 4.5 and 6.8, 8 x 32 6.9 and 11.2; 64 x 32 x 1024 12.0 and 11.5, 64 x 32
// x 4096 22.5 and 13.0, 64 x 64 35.7 and 47.5).
inline bool few_tokens(const GatedRows &rows, size_t lanes)
{
    return rows.starts == nullptr && rows.tokens >= 1 && (rows.tokens <= 8 || (rows.tokens <= 32 && rows.rows * lanes >= 8192));
}
template <typename X, typename G, int KIND>
cudaError_t forward_kind(const GatedScanCall &call, int sms, cudaStream_t s)
{
    constexpr int V = 4 / sizeof(X);
    Width width = {V};
    width.add(call.x, call.rows, sizeof(X));
    width.add(call.gate, call.rows, sizeof(G));
    width.add(call.out, call.rows, sizeof(X));
    const int copy = width.copy();
    constexpr int N = 16 / sizeof(X);
    const bool states = (reinterpret_cast<uintptr_t>(call.initial) | reinterpret_cast<uintptr_t>(call.final)) % 16 == 0;
    const bool vectors = copy == 16 && states && call.rows.channels % N == 0;
    if (few_tokens(call.rows, static_cast<size_t>(call.rows.channels) / (vectors ? N : 1)))
        return vectors ? step<X, G, N, KIND>(call, s) : step<X, G, 1, KIND>(call, s);
    if (copy == 16) return forward<X, G, V, KIND, 16>(call, sms, s);
    if (copy == 4) return forward<X, G, V, KIND, 4>(call, sms, s);
    if constexpr (V > 1) return forward<X, G, 1, KIND, 0>(call, sms, s);
    return cudaErrorInvalidValue;   // fp32 is aligned
}
template <typename X, typename G>
cudaError_t forward_any(const GatedScanCall &call, int sms, cudaStream_t s)
{
    if (call.kind == kGateDecay) return forward_kind<X, G, kGateDecay>(call, sms, s);
    if (call.kind == kGateLog) return forward_kind<X, G, kGateLog>(call, sms, s);
    return forward_kind<X, G, kGateSigmoid>(call, sms, s);
}

template <typename X, typename G, int V, int KIND, int COPY, bool MANY>
cudaError_t backward_of(GatedBackwardCall call, int sms, cudaStream_t s)
{
    static std::atomic<unsigned long long> done, more, longs;
    using R = BackwardRing<X, G, V, KIND, COPY, MANY>;
    lay_out(call.rows, {&call.grad, &call.gate, &call.y, &call.grad_x, &call.grad_gate, KIND == kGateSigmoid ? &call.x : &call.y});
    plan(call.rows, V, R::kTokens, R::kPerSm, MANY, sms);
    if constexpr (MANY)
        if (call.rows.blocks > kPortableBlocks)
            return launch_clusters(gated_scan_backward_kernel<X, G, V, KIND, COPY, MANY, kMostBlocks>, call, R::kBytes, more, s);
    const cudaError_t e = launch_clusters(gated_scan_backward_kernel<X, G, V, KIND, COPY, MANY, kPortableBlocks>, call, R::kBytes, done, s);
    if (e != cudaSuccess || call.rows.long_from == 0) return e;
    using Long = BackwardRing<X, G, V, KIND, COPY, true>;
    plan_long(call.rows, Long::kPerSm, sms);
    return launch_clusters(gated_scan_backward_kernel<X, G, V, KIND, COPY, true, kPortableBlocks>, call, Long::kBytes, longs, s);
}
template <typename X, typename G, int V, int KIND, int COPY>
cudaError_t backward(const GatedBackwardCall &call, int sms, cudaStream_t s)
{
    if (many_tokens(call.rows)) return backward_of<X, G, V, KIND, COPY, true>(call, sms, s);
    return backward_of<X, G, V, KIND, COPY, false>(call, sms, s);
}
template <typename X, typename G, int KIND>
cudaError_t backward_kind(const GatedBackwardCall &call, int sms, cudaStream_t s)
{
    constexpr int V = 4 / sizeof(X);
    Width width = {V};
    width.add(call.grad, call.rows, sizeof(X));
    width.add(call.y, call.rows, sizeof(X));
    if (KIND == kGateSigmoid) width.add(call.x, call.rows, sizeof(X));
    width.add(call.gate, call.rows, sizeof(G));
    width.add(call.grad_x, call.rows, sizeof(X));
    width.add(call.grad_gate, call.rows, sizeof(G));
    const int copy = width.copy();
    if (copy == 16) return backward<X, G, V, KIND, 16>(call, sms, s);
    if (copy == 4) return backward<X, G, V, KIND, 4>(call, sms, s);
    if constexpr (V > 1) return backward<X, G, 1, KIND, 0>(call, sms, s);
    return cudaErrorInvalidValue;
}
template <typename X, typename G>
cudaError_t backward_any(const GatedBackwardCall &call, int sms, cudaStream_t s)
{
    if (call.kind == kGateDecay) return backward_kind<X, G, kGateDecay>(call, sms, s);
    if (call.kind == kGateLog) return backward_kind<X, G, kGateLog>(call, sms, s);
    return backward_kind<X, G, kGateSigmoid>(call, sms, s);
}

}  // namespace gated
}  // namespace devscan
