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
// The order is the descending order of a 64-bit key, the logit's ordered bits
// above the complement of its index.  The last kept key is found by a radix
// select, most significant digit first, on counts (top-k) or on masses
// (top-p).  Masses are fixed-point integers (w in units of 2^-31, sums in 64
// bits), so they do not depend on the order of the adds.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "core.cuh"
#include "launch.h"

namespace devscan {
namespace {

constexpr int kSampleThreads = 512;
constexpr int kSampleWarps = kSampleThreads / 32;
constexpr int kIndexBits = 24;
constexpr int kKeyDigits = (32 + kIndexBits) / 8;

using u64 = unsigned long long;

__device__ __forceinline__ float as_float(float v) { return v; }
__device__ __forceinline__ float as_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float as_float(__nv_bfloat16 v) { return __bfloat162float(v); }

// Bits of x whose unsigned order is x's order; NaN counts as -inf, -0 as 0.
__device__ __forceinline__ uint32_t ordered(float x)
{
    if (x != x) x = -__int_as_float(0x7f800000);
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t k)
{
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
constexpr uint32_t kOrderedMinusInf = 0x007fffffu;

__device__ __forceinline__ u64 key_of(uint32_t ord, unsigned i)
{
    return (static_cast<u64>(ord) << kIndexBits) | ((1u << kIndexBits) - 1 - i);
}

template <class V, class F>
__device__ V block_fold(V v, V *s_fold, F f)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) v = f(v, __shfl_xor_sync(kFullMask, v, d));
    __syncthreads();
    if (lane == 0) s_fold[warp] = v;
    __syncthreads();
    v = s_fold[0];
    for (int w = 1; w < kSampleWarps; ++w) v = f(v, s_fold[w]);
    return v;
}

template <class T>
struct Row {
    const T *x;
    unsigned vocab;
    float top;      // the largest logit
    float t;        // temperature
    __device__ __forceinline__ uint32_t ord(unsigned i) const { return ordered(as_float(x[i])); }
    __device__ __forceinline__ float weight(uint32_t o) const
    {
        const float v = unordered(o);
        if (o == kOrderedMinusInf) return 0.0f;
        return v == top ? 1.0f : fmaxf(expf((v - top) / t), 0.0f);   // 0 for inf / inf
    }
    __device__ __forceinline__ uint32_t mass(uint32_t o) const { return __float2uint_rn(weight(o) * 2147483648.0f); }
};

// The largest key K such that what keys >= K hold (1 each, or their mass)
// reaches `want`; 0 if all of them do not.  Only keys >= `floor` take part.
template <bool MASS, class T>
__device__ u64 select(const Row<T> &row, u64 floor, u64 want, u64 *s_hist, u64 *s_pick)
{
    u64 prefix = 0;
    for (int digit = kKeyDigits - 1; digit >= 0; --digit) {
        const int shift = digit * 8;
        for (int b = threadIdx.x; b < 256; b += kSampleThreads) s_hist[b] = 0;
        __syncthreads();
        for (unsigned i = threadIdx.x; i < row.vocab; i += kSampleThreads) {
            const uint32_t o = row.ord(i);
            const u64 key = key_of(o, i);
            if (key < floor || (key >> shift >> 8) != prefix || o == kOrderedMinusInf) continue;
            atomicAdd(&s_hist[(key >> shift) & 255], MASS ? static_cast<u64>(row.mass(o)) : 1ull);
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            int b = 255;
            while (b >= 0 && s_hist[b] < want) want -= s_hist[b--];
            s_pick[0] = b < 0 ? ~0ull : static_cast<u64>(b);
            s_pick[1] = want;
        }
        __syncthreads();
        const u64 b = s_pick[0];
        want = s_pick[1];
        __syncthreads();
        if (b == ~0ull) return 0;
        prefix = (prefix << 8) | b;
    }
    return prefix;
}

template <class T>
__global__ void __launch_bounds__(kSampleThreads)
sample_kernel(const T *__restrict__ logits, size_t stride, unsigned vocab, const float *__restrict__ noise,
              size_t noise_stride, SampleAsk ask, int32_t *__restrict__ tokens, float *__restrict__ logprobs)
{
    __shared__ u64 s_fold[kSampleWarps];
    __shared__ u64 s_hist[256];
    __shared__ u64 s_pick[2];
    const unsigned r = blockIdx.x;
    const auto larger = [](u64 a, u64 b) { return a > b ? a : b; };
    const auto add = [](u64 a, u64 b) { return a + b; };
    Row<T> row{logits + r * stride, vocab, 0.0f, 1.0f};

    u64 best = 0;
    for (unsigned i = threadIdx.x; i < vocab; i += kSampleThreads) best = larger(best, key_of(row.ord(i), i));
    best = block_fold(best, s_fold, larger);
    const uint32_t top = static_cast<uint32_t>(best >> kIndexBits);
    const unsigned first = (1u << kIndexBits) - 1 - static_cast<unsigned>(best & ((1u << kIndexBits) - 1));
    const float t = ask.temperature != nullptr ? ask.temperature[r] : 1.0f;
    if (top == kOrderedMinusInf || noise == nullptr || !(t > 0.0f)) {
        if (threadIdx.x == 0) {
            const bool empty = top == kOrderedMinusInf;
            tokens[r] = empty ? -1 : static_cast<int32_t>(first);
            if (logprobs != nullptr) logprobs[r] = empty ? -__int_as_float(0x7f800000) : 0.0f;
        }
        return;
    }
    row.top = unordered(top);
    row.t = t;
    const int k = ask.top_k != nullptr ? ask.top_k[r] : 0;
    const float p = ask.top_p != nullptr ? ask.top_p[r] : 1.0f;
    const float m = ask.min_p != nullptr ? ask.min_p[r] : 0.0f;

    u64 last = 0;
    if (k > 0 && static_cast<unsigned>(k) < vocab) last = select<false>(row, 0, k, s_hist, s_pick);
    if (!(p >= 1.0f)) {
        u64 all = 0;
        for (unsigned i = threadIdx.x; i < vocab; i += kSampleThreads) {
            const uint32_t o = row.ord(i);
            if (key_of(o, i) >= last) all += row.mass(o);
        }
        all = block_fold(all, s_fold, add);
        const double part = p > 0.0f ? static_cast<double>(p) * static_cast<double>(all) : 0.0;
        const u64 want = static_cast<u64>(ceil(part));
        last = larger(last, select<true>(row, last, want > 1 ? want : 1, s_hist, s_pick));
    }
    u64 won = 0;
    float rest = 0.0f;   // the kept weights but the first's, which is 1
    const float *q = noise + r * noise_stride;
    for (unsigned i = threadIdx.x; i < vocab; i += kSampleThreads) {
        const uint32_t o = row.ord(i);
        const u64 key = key_of(o, i);
        if (key < last || o == kOrderedMinusInf) continue;
        const float w = row.weight(o);
        if (i != first && !(w >= m)) continue;
        if (i != first) rest += w;
        const float score = w / q[i];
        won = larger(won, (static_cast<u64>(score > 0.0f ? __float_as_uint(score) : 0u) << 32) | (0xffffffffu - i));
    }
    won = block_fold(won, s_fold, larger);
    float *s_rest = reinterpret_cast<float *>(s_hist);
    rest = block_fold(rest, s_rest, [](float a, float b) { return a + b; });
    if (threadIdx.x == 0) {
        const unsigned i = 0xffffffffu - static_cast<unsigned>(won);
        tokens[r] = static_cast<int32_t>(i);
        if (logprobs != nullptr) {
            const float v = unordered(row.ord(i));
            logprobs[r] = (v == row.top ? 0.0f : (v - row.top) / t) - log1pf(rest);
        }
    }
}

template <class T>
cudaError_t launch(const void *logits, size_t rows, size_t vocab, size_t stride, const float *noise,
                   size_t noise_stride, const SampleAsk &ask, int32_t *tokens, float *logprobs, cudaStream_t s)
{
    sample_kernel<T><<<static_cast<unsigned>(rows), kSampleThreads, 0, s>>>(
        static_cast<const T *>(logits), stride, static_cast<unsigned>(vocab), noise, noise_stride, ask, tokens,
        logprobs);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_sample(LogitType type, const void *logits, size_t rows, size_t vocab, size_t stride,
                          const float *noise, size_t noise_stride, const SampleAsk &ask, int32_t *tokens,
                          float *logprobs, cudaStream_t s)
{
    switch (type) {
    case LogitType::F32:
        return launch<float>(logits, rows, vocab, stride, noise, noise_stride, ask, tokens, logprobs, s);
    case LogitType::F16:
        return launch<__half>(logits, rows, vocab, stride, noise, noise_stride, ask, tokens, logprobs, s);
    case LogitType::BF16:
        return launch<__nv_bfloat16>(logits, rows, vocab, stride, noise, noise_stride, ask, tokens, logprobs, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace devscan
