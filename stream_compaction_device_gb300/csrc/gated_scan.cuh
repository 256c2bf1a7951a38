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
// 128 bytes per warp and token) and nothing is shuffled; a warp takes kTokens
// consecutive tokens, a block's eight warps lie behind each other.  Every
// value is read once and kept in registers while the carry comes: the maps of
// its tokens are folded, handed on, and then the tokens are run again from
// the right h.  The next round's loads are issued before the exchange.
//
// Split.  A cluster takes 32 lanes' channels of one span of whole rows.  Rows
// are handed out first, since rows need no exchange; a row is spread over up to
// eight blocks only where rows and channels alone do not fill the GPU.  No
// block waits for another but at the cluster barrier, and sums are made in an
// order that follows from the sizes alone.
#pragma once

#include "cluster.cuh"
#include "convert.cuh"
#include "launch.h"

namespace devscan {
namespace gated {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kMostBlocks = 8;   // of a cluster (the portable size)
constexpr int kForwardTokens = 16, kBackwardTokens = 8;   // per warp and round

// ---------------------------------------------------------------------------
// Gates.  A decay next to 1 acts thousands of times, so its error must not
// lean to one side there: it is 1 plus or minus something small, rounded once.
// ---------------------------------------------------------------------------

// exp(g): near 0 as 1 + (its series to the fifth power, off by less than
// g^6 / 720 < 2^-27); elsewhere the hardware's, off by 2^-22 of values that act
// less than ten times.
__device__ __forceinline__ float exp_decay(float g)
{
    const float s = g * fmaf(g, fmaf(g, fmaf(g, fmaf(g, 1.0f / 120, 1.0f / 24), 1.0f / 6), 0.5f), 1.0f);
    return fabsf(g) < 0.125f ? 1.0f + s : __expf(g);
}

// a = 1 / (1 + exp(-g)) and r = 1 - a, the smaller of the two from the quotient.
__device__ __forceinline__ void sigmoid_decay(float g, float &a, float &r)
{
    const float t = __expf(-fabsf(g));
    const float small = __fdividef(t, 1.0f + t), large = 1.0f - small;
    a = g >= 0.0f ? large : small;
    r = g >= 0.0f ? small : large;
}

// ---------------------------------------------------------------------------
// Rows and spans.
// ---------------------------------------------------------------------------

// Index of the first of starts[0 .. count) that is at least `value` (`above`:
// greater than it); count if none is.
template <bool above>
__device__ __forceinline__ int first_start(const int32_t *starts, int count, int value)
{
    int lo = 0, hi = count;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1, s = __ldg(starts + mid);
        if (above ? s <= value : s < value)
            lo = mid + 1;
        else
            hi = mid;
    }
    return lo;
}

// Where span j begins: at the first row that begins at or behind its share of
// the tokens.
__device__ __forceinline__ unsigned span_begin(const GatedRows &rows, unsigned j)
{
    const unsigned all = rows.all();
    if (j == 0) return 0u;
    if (j >= rows.spans) return all;
    if (rows.starts == nullptr)
        return static_cast<unsigned>(static_cast<unsigned long long>(rows.rows) * j / rows.spans) * rows.tokens;
    const int share = static_cast<int>(static_cast<unsigned long long>(all) * j / rows.spans);
    const int r = first_start<false>(rows.starts, rows.rows + 1, share);
    if (r > rows.rows) return all;
    const unsigned at = static_cast<unsigned>(__ldg(rows.starts + r));   // >= share >= 0
    return at < all ? at : all;
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
    p.row = first_start<true>(rows.starts, rows.rows + 1, static_cast<int>(n)) - 1;
    p.inside = p.row >= 0 && p.row < rows.rows;
    p.first = p.inside && __ldg(rows.starts + p.row) == static_cast<int>(n);
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

// Row r's state in a pool; null where it has none.
__device__ __forceinline__ float *state_of(const GatedRows &rows, float *states, int r)
{
    if (states == nullptr) return nullptr;
    const int slot = rows.slots == nullptr ? r : __ldg(rows.slots + r);
    return static_cast<unsigned>(slot) < static_cast<unsigned>(rows.pool)
               ? states + static_cast<size_t>(slot) * rows.channels
               : nullptr;
}

// The elements of consecutive tokens of a strided array: fn(i, element) for
// i = 0 .. count - 1, beginning with token n and going on (DOWN: back).
template <int COUNT, bool DOWN, typename Fn>
__device__ __forceinline__ void walk(const GatedRows &rows, const GatedArray &array, unsigned n, int count, Fn &&fn)
{
    const unsigned r = n / rows.tokens;
    unsigned t = n - r * rows.tokens;
    size_t at = r * array.row_stride + t * array.stride;
    if (count == COUNT && (DOWN ? t + 1 >= COUNT : t + COUNT <= rows.tokens)) {   // all in one row: no turns
#pragma unroll
        for (int i = 0; i < COUNT; ++i) {
            fn(i, at, DOWN ? t - i : t + i);
            at = DOWN ? at - array.stride : at + array.stride;
        }
        return;
    }
    const size_t turn = array.row_stride - (rows.tokens - 1) * array.stride;   // modulo 2^64
#pragma unroll
    for (int i = 0; i < COUNT; ++i) {
        if (i < count) fn(i, at, t);
        if (DOWN) {
            const bool wrap = t == 0;
            at -= wrap ? turn : array.stride;
            t = wrap ? rows.tokens - 1 : t - 1;
        } else {
            const bool wrap = t + 1 == rows.tokens;
            at += wrap ? turn : array.stride;
            t = wrap ? 0 : t + 1;
        }
    }
}

// ---------------------------------------------------------------------------
// The exchange of one round: every warp hands in its map, and gets the value
// that comes into it.
// ---------------------------------------------------------------------------
template <int V> struct Exchange {
    float a[2][kWarps][32 * V], h[2][kWarps][32 * V];             // this block's warps
    float all_a[2][kMostBlocks][32 * V], all_h[2][kMostBlocks][32 * V];   // the cluster's blocks
    unsigned cut[2][kWarps], all_cut[2][kMostBlocks];             // nonzero: the map forgets what comes in
};

// Two buffers in turn are enough: a block writes a round's buffer after the
// barrier of the round before, at which every reader of the round before that
// has arrived.
template <int V>
__device__ __forceinline__ void exchange(Exchange<V> &x, int turn, int blocks, int rank, int warp, int lane,
                                         const float (&a)[V], const float (&h)[V], bool cut, float (&carry)[V],
                                         float (&in)[V])
{
#pragma unroll
    for (int k = 0; k < V; ++k) x.a[turn][warp][lane * V + k] = a[k], x.h[turn][warp][lane * V + k] = h[k];
    if (lane == 0) x.cut[turn][warp] = cut;
    __syncthreads();
    if (blocks > 1) {
        if (warp == 0) {
            float fa[V], fh[V];
            unsigned any = 0;
#pragma unroll
            for (int k = 0; k < V; ++k) fa[k] = 1.0f, fh[k] = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const bool c = x.cut[turn][w] != 0;
                any |= c;
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const float wa = x.a[turn][w][lane * V + k], wh = x.h[turn][w][lane * V + k];
                    fh[k] = c ? wh : fmaf(wa, fh[k], wh);
                    fa[k] = c ? wa : wa * fa[k];
                }
            }
            for (int q = 0; q < blocks; ++q) {
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    st_cluster(cluster_addr(&x.all_a[turn][rank][lane * V + k], q), fa[k]);
                    st_cluster(cluster_addr(&x.all_h[turn][rank][lane * V + k], q), fh[k]);
                }
                if (lane == 0) st_cluster(cluster_addr(&x.all_cut[turn][rank], q), any);
            }
        }
        cluster_sync();
        float run[V];
#pragma unroll
        for (int k = 0; k < V; ++k) run[k] = carry[k];
        for (int q = 0; q < blocks; ++q) {
            const bool c = x.all_cut[turn][q] != 0;
#pragma unroll
            for (int k = 0; k < V; ++k) {
                if (q == rank) in[k] = run[k];
                const float qh = x.all_h[turn][q][lane * V + k];
                run[k] = c ? qh : fmaf(x.all_a[turn][q][lane * V + k], run[k], qh);
            }
        }
#pragma unroll
        for (int k = 0; k < V; ++k) carry[k] = run[k];
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k) in[k] = carry[k];
    }
    // the block's warps before this one; where the block is alone, all of them for the next round
    float run[V];
#pragma unroll
    for (int k = 0; k < V; ++k) run[k] = in[k];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w >= warp && blocks > 1) break;
        const bool c = x.cut[turn][w] != 0;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            if (w == warp) in[k] = run[k];
            const float wh = x.h[turn][w][lane * V + k];
            run[k] = c ? wh : fmaf(x.a[turn][w][lane * V + k], run[k], wh);
        }
    }
    if (blocks > 1) {
#pragma unroll
        for (int k = 0; k < V; ++k) in[k] = run[k];
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k) carry[k] = run[k];
    }
}

// What a block of the grid works on.
struct Work {
    int rank, blocks, channel;
    unsigned span, begin, end;
};
__device__ __forceinline__ Work work_of(const GatedRows &rows, int per_lane)
{
    Work w;
    w.rank = static_cast<int>(cluster_rank()), w.blocks = rows.blocks;
    const unsigned cluster = blockIdx.x / rows.blocks, groups = rows.groups;
    w.span = cluster / groups;
    w.channel = static_cast<int>((cluster % groups) * 32 + (threadIdx.x & 31)) * per_lane;
    w.begin = span_begin(rows, w.span), w.end = span_begin(rows, w.span + 1);
    if (w.end < w.begin) w.end = w.begin;   // only where starts decrease
    return w;
}

// Rows without tokens: what goes in comes out, 0 where nothing does.  fn(row)
// is called by a warp for each.
template <typename Fn>
__device__ __forceinline__ void empty_rows(const GatedRows &rows, const Work &w, Fn &&fn)
{
    if (w.span != 0) return;
    const int lane = threadIdx.x & 31, warp = w.rank * kWarps + (threadIdx.x >> 5), warps = w.blocks * kWarps;
    for (long long r0 = static_cast<long long>(warp) * 32; r0 < rows.rows; r0 += 32ll * warps) {
        unsigned found = __ballot_sync(kFullMask, r0 + lane < rows.rows && row_empty(rows, static_cast<int>(r0 + lane)));
        for (; found != 0; found &= found - 1) fn(static_cast<int>(r0) + __ffs(found) - 1);
    }
}

// ---------------------------------------------------------------------------
// Forward.
// ---------------------------------------------------------------------------
template <typename X, typename G, int V>
__global__ void __launch_bounds__(kThreads, 2) gated_scan_kernel(const __grid_constant__ GatedScanCall p)
{
    constexpr int L = kForwardTokens;
    using RX = typename Raw<X, V>::type;
    using RG = typename Raw<G, V>::type;
    __shared__ Exchange<V> s_x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Work w = work_of(p.rows, V);
    const bool live = w.channel < p.rows.channels;   // a whole number of lanes is
    const X *x = static_cast<const X *>(p.x.data) + w.channel;
    const G *gate = static_cast<const G *>(p.gate.data) + w.channel;
    X *out = static_cast<X *>(p.out.data) + w.channel;

    if (p.final != nullptr)
        empty_rows(p.rows, w, [&](int r) {
            float *to = state_of(p.rows, p.final, r);
            const float *from = state_of(p.rows, p.initial, r);
            if (to == nullptr || !live) return;
            for (int k = 0; k < V; ++k) to[w.channel + k] = from != nullptr ? from[w.channel + k] : 0.0f;
        });

    const unsigned round = static_cast<unsigned>(w.blocks * kWarps * L);
    const unsigned rounds = (w.end - w.begin + round - 1) / round;
    RX rx[L];
    RG rg[L];
    int count = 0;
    unsigned n = w.begin + static_cast<unsigned>((w.rank * kWarps + warp) * L);   // this warp's first token
    auto load = [&]() {
        count = n < w.end ? static_cast<int>(min(w.end - n, static_cast<unsigned>(L))) : 0;
        if (!live || count == 0) return;
        walk<L, false>(p.rows, p.x, n, count, [&](int i, size_t at, unsigned) {
            rx[i] = *reinterpret_cast<const RX *>(x + at);
        });
        walk<L, false>(p.rows, p.gate, n, count, [&](int i, size_t at, unsigned) {
            rg[i] = *reinterpret_cast<const RG *>(gate + at);
        });
    };
#pragma unroll
    for (int i = 0; i < L; ++i) rx[i] = RX{}, rg[i] = RG{};
    load();
    if (w.blocks > 1) cluster_sync();   // every block is there before another writes to it
    float carry[V] = {};
    for (unsigned step = 0; step < rounds; ++step) {
        float a[L][V], b[L][V];
#pragma unroll
        for (int i = 0; i < L; ++i) {
            float xv[V], gv[V];
            unpack<X, V>(rx[i], xv);
            unpack<G, V>(rg[i], gv);
#pragma unroll
            for (int k = 0; k < V; ++k) {
                a[i][k] = gv[k], b[i][k] = xv[k];
                if (p.kind == kGateLog) a[i][k] = exp_decay(gv[k]);
                if (p.kind == kGateSigmoid) {
                    float r;
                    sigmoid_decay(gv[k], a[i][k], r);
                    b[i][k] *= r;
                }
                if (i >= count) a[i][k] = 1.0f, b[i][k] = 0.0f;
            }
        }
        // Rows that begin or end among these tokens, a bit per token.
        TokenPlace place = {0, true, false, false};
        const bool mine = lane < count;
        if (mine) place = place_of(p.rows, n + lane);
        const unsigned first = __ballot_sync(kFullMask, mine && place.first);
        const unsigned last = __ballot_sync(kFullMask, mine && place.last);
        const unsigned outside = __ballot_sync(kFullMask, mine && !place.inside);
        const unsigned cut = first | outside;
        if (cut != 0) {
#pragma unroll
            for (int i = 0; i < L; ++i) {
                if ((first >> i) & 1u) {
                    const float *from = state_of(p.rows, p.initial, __shfl_sync(kFullMask, place.row, i));
                    if (from != nullptr && live)
#pragma unroll
                        for (int k = 0; k < V; ++k) b[i][k] = fmaf(a[i][k], from[w.channel + k], b[i][k]);
                }
                if ((outside >> i) & 1u)
#pragma unroll
                    for (int k = 0; k < V; ++k) b[i][k] = 0.0f;
            }
        }
        float fa[V], h[V];
#pragma unroll
        for (int k = 0; k < V; ++k) fa[k] = 1.0f, h[k] = 0.0f;
#pragma unroll
        for (int i = 0; i < L; ++i)
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const bool c = (cut >> i) & 1u;
                h[k] = c ? b[i][k] : fmaf(a[i][k], h[k], b[i][k]);
                fa[k] = c ? 0.0f : fa[k] * a[i][k];
            }
        const unsigned here = n;
        const int had = count;
        n += round;
        load();
        exchange<V>(s_x, step & 1, w.blocks, w.rank, warp, lane, fa, h, cut != 0, carry, h);
#pragma unroll
        for (int i = 0; i < L; ++i)
#pragma unroll
            for (int k = 0; k < V; ++k) {
                h[k] = (cut >> i) & 1u ? b[i][k] : fmaf(a[i][k], h[k], b[i][k]);
                b[i][k] = h[k];
            }
        if (live && had > 0)
            walk<L, false>(p.rows, p.out, here, had, [&](int i, size_t at, unsigned) {
                *reinterpret_cast<RX *>(out + at) = pack<X, V>(b[i]);
            });
        if (last != 0 && p.final != nullptr) {
#pragma unroll
            for (int i = 0; i < L; ++i) {
                if (((last >> i) & 1u) == 0) continue;
                float *to = state_of(p.rows, p.final, __shfl_sync(kFullMask, place.row, i));
                if (to != nullptr && live)
#pragma unroll
                    for (int k = 0; k < V; ++k) to[w.channel + k] = b[i][k];
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Backward.  With w_t the gradient of h_t as it is used and handed on,
//   w_t = dh_t + f_{t+1},  f_t = a_t w_t  (f behind a row's last token: the
//   gradient of its final state),
// which is the same recurrence from the last token to the first, and
//   dx_t = w_t (sigmoid: r_t w_t),  da_t = w_t h_{t-1},  dinitial = f_first;
//   da / dgate = 1, a, or a r (h_{t-1} - x_t in place of h_{t-1}).
// h_{t-1} is what the forward call wrote, in its type.
// ---------------------------------------------------------------------------
template <typename X, typename G, int V, bool SIGMOID>
__global__ void __launch_bounds__(kThreads, 2) gated_scan_backward_kernel(const __grid_constant__ GatedBackwardCall p)
{
    constexpr int L = kBackwardTokens;
    using RX = typename Raw<X, V>::type;
    using RG = typename Raw<G, V>::type;
    __shared__ Exchange<V> s_x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Work w = work_of(p.rows, V);
    const bool live = w.channel < p.rows.channels;
    const X *grad = static_cast<const X *>(p.grad.data) + w.channel;
    const X *y = static_cast<const X *>(p.y.data) + w.channel;
    const X *x = SIGMOID ? static_cast<const X *>(p.x.data) + w.channel : nullptr;
    const G *gate = static_cast<const G *>(p.gate.data) + w.channel;
    X *grad_x = static_cast<X *>(p.grad_x.data) + w.channel;
    G *grad_gate = static_cast<G *>(p.grad_gate.data) + w.channel;

    if (p.grad_initial != nullptr)
        empty_rows(p.rows, w, [&](int r) {
            if (!live) return;
            const size_t at = static_cast<size_t>(r) * p.rows.channels + w.channel;
            for (int k = 0; k < V; ++k) p.grad_initial[at + k] = p.grad_final != nullptr ? p.grad_final[at + k] : 0.0f;
        });

    const unsigned round = static_cast<unsigned>(w.blocks * kWarps * L);
    const unsigned tokens = w.end - w.begin, rounds = (tokens + round - 1) / round;
    RX rd[L], ry[L], rx[SIGMOID ? L : 1];
    RG rg[L];
    int count = 0;
    unsigned done = static_cast<unsigned>((w.rank * kWarps + warp) * L);   // tokens of the span behind this warp's
    auto load = [&]() {
        count = done < tokens ? static_cast<int>(min(tokens - done, static_cast<unsigned>(L))) : 0;
        if (!live || count == 0) return;
        const unsigned n = w.end - 1 - done;   // going back from here
        walk<L, true>(p.rows, p.grad, n, count, [&](int i, size_t at, unsigned) {
            rd[i] = *reinterpret_cast<const RX *>(grad + at);
        });
        walk<L, true>(p.rows, p.gate, n, count, [&](int i, size_t at, unsigned) {
            rg[i] = *reinterpret_cast<const RG *>(gate + at);
        });
        walk<L, true>(p.rows, p.y, n, count, [&](int i, size_t at, unsigned t) {
            if (t > 0) ry[i] = *reinterpret_cast<const RX *>(y + (at - p.y.stride));
        });
        if constexpr (SIGMOID)
            walk<L, true>(p.rows, p.x, n, count, [&](int i, size_t at, unsigned) {
                rx[i] = *reinterpret_cast<const RX *>(x + at);
            });
    };
#pragma unroll
    for (int i = 0; i < L; ++i) rd[i] = RX{}, ry[i] = RX{}, rx[SIGMOID ? i : 0] = RX{}, rg[i] = RG{};
    load();
    if (w.blocks > 1) cluster_sync();   // every block is there before another writes to it
    float carry[V] = {};
    for (unsigned step = 0; step < rounds; ++step) {
        const unsigned here = w.end - 1 - done;
        TokenPlace place = {0, true, false, false};
        const bool mine = lane < count;
        if (mine) place = place_of(p.rows, here - lane);
        const unsigned first = __ballot_sync(kFullMask, mine && place.first);
        const unsigned last = __ballot_sync(kFullMask, mine && place.last);
        const unsigned outside = __ballot_sync(kFullMask, mine && !place.inside);
        const unsigned cut = last | outside;
        // d: dh, then w; e: what w is multiplied by for the gate; m: for x
        float a[L][V], d[L][V], e[L][V], m[SIGMOID ? L : 1][V];
#pragma unroll
        for (int i = 0; i < L; ++i) {
            float gv[V], xv[V];
            unpack<X, V>(rd[i], d[i]);
            unpack<X, V>(ry[i], e[i]);
            unpack<X, V>(rx[SIGMOID ? i : 0], xv);
            unpack<G, V>(rg[i], gv);
            if ((first >> i) & 1u) {
                const float *from = state_of(p.rows, p.initial, __shfl_sync(kFullMask, place.row, i));
#pragma unroll
                for (int k = 0; k < V; ++k) e[i][k] = from != nullptr && live ? from[w.channel + k] : 0.0f;
            }
#pragma unroll
            for (int k = 0; k < V; ++k) {
                if constexpr (SIGMOID) {
                    float r;
                    sigmoid_decay(gv[k], a[i][k], r);
                    m[i][k] = r;
                    e[i][k] = (e[i][k] - xv[k]) * (a[i][k] * r);
                } else {
                    a[i][k] = p.kind == kGateLog ? exp_decay(gv[k]) : gv[k];
                    if (p.kind == kGateLog) e[i][k] *= a[i][k];
                }
                if (i >= count) a[i][k] = 1.0f, d[i][k] = 0.0f;
                if ((outside >> i) & 1u) {
                    a[i][k] = d[i][k] = e[i][k] = 0.0f;
                    if constexpr (SIGMOID) m[i][k] = 0.0f;
                }
            }
            if (((last >> i) & 1u) != 0 && p.grad_final != nullptr) {
                const int r = __shfl_sync(kFullMask, place.row, i);
                const size_t at = static_cast<size_t>(r) * p.rows.channels + w.channel;
#pragma unroll
                for (int k = 0; k < V; ++k) d[i][k] += live ? p.grad_final[at + k] : 0.0f;
            }
        }
        float fa[V], f[V];
#pragma unroll
        for (int k = 0; k < V; ++k) fa[k] = 1.0f, f[k] = 0.0f;
#pragma unroll
        for (int i = 0; i < L; ++i)
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const bool c = (cut >> i) & 1u;
                f[k] = a[i][k] * (c ? d[i][k] : d[i][k] + f[k]);
                fa[k] = c ? 0.0f : fa[k] * a[i][k];
            }
        const int had = count;
        done += round;
        load();
        exchange<V>(s_x, step & 1, w.blocks, w.rank, warp, lane, fa, f, cut != 0, carry, f);
#pragma unroll
        for (int i = 0; i < L; ++i)
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const float v = (cut >> i) & 1u ? d[i][k] : d[i][k] + f[k];
                f[k] = a[i][k] * v;
                e[i][k] *= v;
                d[i][k] = SIGMOID ? v * m[SIGMOID ? i : 0][k] : v;
                a[i][k] = f[k];
            }
        if (live && had > 0) {
            walk<L, true>(p.rows, p.grad_x, here, had, [&](int i, size_t at, unsigned) {
                *reinterpret_cast<RX *>(grad_x + at) = pack<X, V>(d[i]);
            });
            walk<L, true>(p.rows, p.grad_gate, here, had, [&](int i, size_t at, unsigned) {
                *reinterpret_cast<RG *>(grad_gate + at) = pack<G, V>(e[i]);
            });
        }
        if (first != 0 && p.grad_initial != nullptr) {
#pragma unroll
            for (int i = 0; i < L; ++i) {
                if (((first >> i) & 1u) == 0) continue;
                const int r = __shfl_sync(kFullMask, place.row, i);
                if (live)
#pragma unroll
                    for (int k = 0; k < V; ++k)
                        p.grad_initial[static_cast<size_t>(r) * p.rows.channels + w.channel + k] = a[i][k];
            }
        }
    }
}

// ---------------------------------------------------------------------------
// One token per row: a thread per V channels of a row.
// ---------------------------------------------------------------------------
template <typename X, typename G, int V>
__global__ void __launch_bounds__(256) gated_step_kernel(const __grid_constant__ GatedScanCall p, unsigned lanes)
{
    const size_t i = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x;
    const int r = static_cast<int>(i / lanes), c = static_cast<int>(i % lanes) * V;
    if (r >= p.rows.rows) return;
    X *out = static_cast<X *>(p.out.data) + r * p.out.row_stride + c;
    float a[V], b[V];
    unpack<X, V>(*reinterpret_cast<const typename Raw<X, V>::type *>(static_cast<const X *>(p.x.data) +
                                                                      r * p.x.row_stride + c), b);
    unpack<G, V>(*reinterpret_cast<const typename Raw<G, V>::type *>(static_cast<const G *>(p.gate.data) +
                                                                      r * p.gate.row_stride + c), a);
    const float *from = state_of(p.rows, p.initial, r);
    float *to = state_of(p.rows, p.final, r);
#pragma unroll
    for (int k = 0; k < V; ++k) {
        if (p.kind == kGateLog) a[k] = exp_decay(a[k]);
        if (p.kind == kGateSigmoid) {
            float rest;
            sigmoid_decay(a[k], a[k], rest);
            b[k] *= rest;
        }
        if (from != nullptr) b[k] = fmaf(a[k], from[c + k], b[k]);
    }
    *reinterpret_cast<typename Raw<X, V>::type *>(out) = pack<X, V>(b);
    if (to != nullptr)
#pragma unroll
        for (int k = 0; k < V; ++k) to[c + k] = b[k];
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
inline bool pairs(const GatedArray &a, size_t size)
{
    return reinterpret_cast<uintptr_t>(a.data) % (2 * size) == 0 && a.stride % 2 == 0 && a.row_stride % 2 == 0;
}

// Spans and blocks per cluster.  Rows are spread first; a span's rows are then
// spread over more blocks while the grid leaves places on the GPU empty and
// every block has a round's tokens.
inline void plan(GatedRows &rows, int per_lane, int tokens_per_warp, int sms)
{
    const size_t all = rows.all(), groups = (static_cast<size_t>(rows.channels) + 32 * per_lane - 1) / (32 * per_lane);
    const size_t places = static_cast<size_t>(sms) * 2, tile = static_cast<size_t>(kWarps) * tokens_per_warp;
    size_t spans = (4 * places + groups - 1) / groups;
    spans = spans < static_cast<size_t>(rows.rows) ? spans : static_cast<size_t>(rows.rows);
    const size_t most = (all + tile - 1) / tile;   // spans of a round at least
    if (spans > most) spans = most;
    if (spans < 1) spans = 1;
    size_t blocks = 1;
    while (blocks < kMostBlocks && groups * spans * blocks < places && spans * blocks * tile < all) blocks *= 2;
    rows.groups = static_cast<unsigned>(groups), rows.spans = static_cast<unsigned>(spans);
    rows.blocks = static_cast<int>(blocks);
}

template <typename... Params, typename... Args>
cudaError_t launch_clusters(void (*kernel)(Params...), const GatedRows &rows, cudaStream_t s, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(rows.groups * rows.spans * static_cast<unsigned>(rows.blocks));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(rows.blocks);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

template <typename X, typename G, int V>
cudaError_t forward(GatedScanCall call, int sms, cudaStream_t s)
{
    if (call.rows.starts == nullptr && call.rows.tokens == 1) {
        const unsigned lanes = static_cast<unsigned>(call.rows.channels / V);
        const size_t threads = static_cast<size_t>(call.rows.rows) * lanes;
        gated_step_kernel<X, G, V><<<static_cast<unsigned>((threads + 255) / 256), 256, 0, s>>>(call, lanes);
        return cudaGetLastError();
    }
    plan(call.rows, V, kForwardTokens, sms);
    return launch_clusters(gated_scan_kernel<X, G, V>, call.rows, s, call);
}

template <typename X, typename G>
cudaError_t forward_any(const GatedScanCall &call, int sms, cudaStream_t s)
{
    if constexpr (sizeof(X) == 2)
        if (call.rows.channels % 2 == 0 && pairs(call.x, 2) && pairs(call.gate, sizeof(G)) && pairs(call.out, 2))
            return forward<X, G, 2>(call, sms, s);
    return forward<X, G, 1>(call, sms, s);
}

template <typename X, typename G, int V>
cudaError_t backward(GatedBackwardCall call, int sms, cudaStream_t s)
{
    plan(call.rows, V, kBackwardTokens, sms);
    if (call.kind == kGateSigmoid)
        return launch_clusters(gated_scan_backward_kernel<X, G, V, true>, call.rows, s, call);
    return launch_clusters(gated_scan_backward_kernel<X, G, V, false>, call.rows, s, call);
}

template <typename X, typename G>
cudaError_t backward_any(const GatedBackwardCall &call, int sms, cudaStream_t s)
{
    if constexpr (sizeof(X) == 2)
        if (call.rows.channels % 2 == 0 && pairs(call.grad, 2) && (call.kind != kGateSigmoid || pairs(call.x, 2)) &&
            pairs(call.gate, sizeof(G)) && pairs(call.y, 2) && pairs(call.grad_x, 2) &&
            pairs(call.grad_gate, sizeof(G)))
            return backward<X, G, 2>(call, sms, s);
    return backward<X, G, 1>(call, sms, s);
}

}  // namespace gated
}  // namespace devscan
