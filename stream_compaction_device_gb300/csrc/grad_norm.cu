// The 2-norm over many tensors, and their clipping (sm_103a):
//   norm = sqrt(sum over tensors, elements of g^2),
//   out  = g min(1, max_norm / (norm + 1e-6)).
//
// The fold of geek-doc.cn "并行前缀和 scan ..." section 四 over arrays that lie
// anywhere: the tensors are cut into chunks of 16 KB, block b takes the chunks
// b, b + blocks, ... and leaves one partial sum; whoever needs the norm folds
// the partial sums, in their order, so that the same call gives the same bits.
// The tensors' table is a kernel parameter, so a launch holds up to
// kNormTensors of them and nothing is copied to the device first.  The second
// launch is a programmatic dependent: its blocks start as the first one's end
// and load their first chunk before they wait for the norm.
//
// Sums: a thread adds the squares of a chunk's share (32 values of 16 bits, 16 of 32) in
// fp32 and its shares in fp64.  Where a share's fp32 sum leaves the range in
// which no square that matters is lost or overflows, the share is added again
// with its values times a power of two (64 M values of 1e-25:
// 73 us; 284 with that second sum in fp64).  fp64 goes at two a clock and SM here, so one
// warp folds what a block has, and one thread takes the root (with all threads
// doing so, 1.3 M fp32 in 40 tensors took 19.5 us instead of 7.7).
//
// What bounds it: memory.  1.5 G values in 300 tensors (5.9 GB in and out, read
// once more for the norm) 1,422 us, 6.2 TB/s; the norm of 1 G bf16 321 us.
// Blocks of 512 threads cost small calls 6 us; two or eight loads in flight
// instead of four, large ones a third.
#include <algorithm>

#include "convert.cuh"
#include "core.cuh"
#include "grid_sync.cuh"
#include "launch.h"

namespace devscan {
namespace {

constexpr int kNormThreads = 256, kNormUnroll = 4;
constexpr int kNormPerSm = 4;   // blocks of an SM
constexpr unsigned kChunkBytes = kNormThreads * kNormUnroll * 16;

struct NormTable {
    const void *in[kNormTensors];
    void *out[kNormTensors];
    unsigned long long n[kNormTensors];
    unsigned end[kNormTensors];        // chunks up to and with this tensor's
    unsigned char type[kNormTensors];
    int count;
    unsigned chunks;
};

template <typename T> __device__ __forceinline__ void values_of(const uint4 &q, float (&v)[16 / sizeof(T)])
{
    unpack<T, 16 / sizeof(T)>(__builtin_bit_cast(typename Raw<T, 16 / sizeof(T)>::type, q), v);
}

// Where the chunk lies in its tensor: elements before the first 16-byte
// boundary go with chunk 0, and those behind the last whole vector with the
// last one.
struct Chunk {
    int tensor;
    unsigned long long first, vectors;   // its vectors
    unsigned head;                       // elements in front of the tensor's vectors
    unsigned long long tail;             // index of the first element behind them
    bool lead, trail;                    // the chunk takes the head, the tail
};

__host__ __device__ inline unsigned head_of(const void *p, unsigned long long n, unsigned size)
{
    const unsigned h = static_cast<unsigned>((16 - reinterpret_cast<uintptr_t>(p) % 16) % 16) / size;
    return n < h ? static_cast<unsigned>(n) : h;
}

template <unsigned size> __device__ __forceinline__ Chunk chunk_at(const NormTable &t, int tensor, unsigned index)
{
    Chunk c;
    c.tensor = tensor;
    const unsigned long long n = t.n[tensor];
    c.head = head_of(t.in[tensor], n, size);
    const unsigned long long all = (n - c.head) * size / 16;
    constexpr unsigned long long per = kChunkBytes / 16;
    c.first = index * per;
    c.vectors = all - c.first < per ? all - c.first : per;
    if (c.first >= all) c.vectors = 0;
    c.tail = c.head + all * (16 / size);
    c.lead = index == 0;
    c.trail = c.first + per >= all;
    return c;
}

__device__ __forceinline__ int tensor_of(const NormTable &t, unsigned chunk)
{
    int lo = 0, hi = t.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (t.end[mid] <= chunk)
            lo = mid + 1;
        else
            hi = mid;
    }
    return lo;
}

// Squares that count in fp32: sums in this range hold every square that is not
// below 2^-60 of them, and none overflows on the way.  Values whose sum is below
// it are less than 2^-40 and at least 2^-149: times 2^96 their squares lie between
// 2^-106 and 2^112.  Above it, times 2^-96, none passes 2^64, and what is lost is
// below 2^-70 of the sum.  (Infinity and NaN stay what they are.)
constexpr float kLeastSum = 0x1p-80f, kMostSum = 0x1p120f, kRaise = 0x1p96f, kLower = 0x1p-96f;

// A share added again, of values times `scale`.  That is rare, so it is a loop that
// reads them again (1.5 G values 1,422 us; from registers beside the first sum 1,478,
// as a function 1,441).
template <typename T> __device__ __forceinline__ float squares_again(const uint4 *vectors, unsigned count, int tid, float scale)
{
    constexpr int E = 16 / sizeof(T);
    float sum[2] = {0.0f, 0.0f};
#pragma unroll 1
    for (int u = 0; u < kNormUnroll; ++u) {
        const unsigned i = u * kNormThreads + tid;
        if (i >= count) continue;
        float v[E];
        values_of<T>(vectors[i], v);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float s = v[e] * scale;
            sum[e & 1] = fmaf(s, s, sum[e & 1]);
        }
    }
    return sum[0] + sum[1];
}

template <typename T> __device__ __forceinline__ double chunk_squares(const NormTable &t, int tensor, unsigned index, int tid)
{
    constexpr int E = 16 / sizeof(T);
    const Chunk c = chunk_at<sizeof(T)>(t, tensor, index);
    const T *base = static_cast<const T *>(t.in[tensor]);
    const uint4 *vectors = reinterpret_cast<const uint4 *>(base + c.head) + c.first;
    uint4 q[kNormUnroll];
#pragma unroll
    for (int u = 0; u < kNormUnroll; ++u) {
        const unsigned i = u * kNormThreads + tid;
        q[u] = i < c.vectors ? vectors[i] : make_uint4(0, 0, 0, 0);
    }
    float sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int u = 0; u < kNormUnroll; ++u) {
        float v[E];
        values_of<T>(q[u], v);
#pragma unroll
        for (int e = 0; e < E; ++e) sum[e & 1] = fmaf(v[e], v[e], sum[e & 1]);
    }
    const float all = sum[0] + sum[1];
    double total = all;
    if (!(all >= kLeastSum && all <= kMostSum)) {
        bool any = false;
#pragma unroll
        for (int u = 0; u < kNormUnroll; ++u) any |= (q[u].x | q[u].y | q[u].z | q[u].w) != 0;
        const bool raise = all < kLeastSum;
        const double back = raise ? kLower : kRaise;
        if (any) total = squares_again<T>(vectors, static_cast<unsigned>(c.vectors), tid, raise ? kRaise : kLower) * (back * back);
    }
    if (c.lead && static_cast<unsigned>(tid) < c.head) {
        const double v = to_float(base[tid]);
        total = fma(v, v, total);
    }
    if (c.trail && c.tail + tid < t.n[tensor]) {
        const double v = to_float(base[c.tail + tid]);
        total = fma(v, v, total);
    }
    return total;
}

// The sum of s_v[0 .. count), each lane's share in order and the lanes by a
// tree, to all lanes of the one warp that calls this.
__device__ __forceinline__ double warp_sum(const double *v, unsigned count, int lane)
{
    double sum = 0.0;
    for (unsigned i = lane; i < count; i += 32) sum += v[i];
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) sum += __shfl_xor_sync(kFullMask, sum, d);
    return sum;
}

__global__ void __launch_bounds__(kNormThreads, kNormPerSm) norm_partials_kernel(const __grid_constant__ NormTable t, double *partials)
{
    __shared__ double s_v[kNormThreads];
    const int tid = threadIdx.x;
    allow_dependent_launch();
    double total = 0.0;
    for (unsigned chunk = blockIdx.x; chunk < t.chunks; chunk += gridDim.x) {
        const int tensor = tensor_of(t, chunk);
        const unsigned index = chunk - (tensor > 0 ? t.end[tensor - 1] : 0u);
        switch (static_cast<ValueType>(t.type[tensor])) {
        case ValueType::F32: total += chunk_squares<float>(t, tensor, index, tid); break;
        case ValueType::F16: total += chunk_squares<__half>(t, tensor, index, tid); break;
        case ValueType::BF16: total += chunk_squares<__nv_bfloat16>(t, tensor, index, tid); break;
        }
    }
    s_v[tid] = total;
    __syncthreads();
    if (tid >= 32) return;
    total = warp_sum(s_v, kNormThreads, tid);
    if (tid == 0) partials[blockIdx.x] = total;
}

// The norm from the partial sums of all launches.
__global__ void __launch_bounds__(32) norm_kernel(const double *partials, unsigned count, float *norm)
{
    wait_primary_grid();
    const double v = sqrt(warp_sum(partials, count, threadIdx.x));
    if (threadIdx.x == 0) *norm = static_cast<float>(v);
}

// A chunk on its way through: loaded, then scaled and stored.
struct Loaded {
    Chunk c;
    uint4 q[kNormUnroll];
};
template <unsigned size> __device__ __forceinline__ void chunk_load(const NormTable &t, int tensor, unsigned index, int tid, Loaded &l)
{
    l.c = chunk_at<size>(t, tensor, index);
    const uint4 *vectors = reinterpret_cast<const uint4 *>(static_cast<const char *>(t.in[tensor]) + l.c.head * size) + l.c.first;
#pragma unroll
    for (int u = 0; u < kNormUnroll; ++u) {
        const unsigned i = u * kNormThreads + tid;
        if (i < l.c.vectors) l.q[u] = vectors[i];
    }
}
template <typename T> __device__ __forceinline__ void chunk_store(const NormTable &t, const Loaded &l, float scale, int tid)
{
    constexpr int E = 16 / sizeof(T);
    const Chunk &c = l.c;
    const T *base = static_cast<const T *>(t.in[c.tensor]);
    T *out = static_cast<T *>(t.out[c.tensor]);
    T *to = out + c.head + c.first * E;
    const bool aligned = reinterpret_cast<uintptr_t>(to) % 16 == 0;
#pragma unroll
    for (int u = 0; u < kNormUnroll; ++u) {
        const unsigned i = u * kNormThreads + tid;
        if (i >= c.vectors) continue;
        float v[E];
        values_of<T>(l.q[u], v);
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] *= scale;
        if (aligned) {
            __stcs(reinterpret_cast<uint4 *>(to) + i, __builtin_bit_cast(uint4, pack<T, E>(v)));
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) to[i * static_cast<size_t>(E) + e] = from_float<T>(v[e]);
        }
    }
    if (c.lead && static_cast<unsigned>(tid) < c.head) out[tid] = from_float<T>(to_float(base[tid]) * scale);
    if (c.trail && c.tail + tid < t.n[c.tensor]) out[c.tail + tid] = from_float<T>(to_float(base[c.tail + tid]) * scale);
}

// Blocks go through the chunks from the last to the first: what the sum read
// last still lies in L2.  `partials` and `norm` are touched behind the wait
// only; the tensors, which the launch before this one reads too, were written
// before that one began.
__global__ void __launch_bounds__(kNormThreads, kNormPerSm) norm_scale_kernel(const __grid_constant__ NormTable t, const double *partials,
                                                                              unsigned count, float max_norm, float *norm)
{
    __shared__ float s_scale;
    const int tid = threadIdx.x;
    float scale = 1.0f;
    bool told = false;
    for (unsigned i = blockIdx.x; i < t.chunks; i += gridDim.x) {
        const unsigned chunk = t.chunks - 1 - i;
        const int tensor = tensor_of(t, chunk);
        const unsigned index = chunk - (tensor > 0 ? t.end[tensor - 1] : 0u);
        const ValueType type = static_cast<ValueType>(t.type[tensor]);
        Loaded l;
        if (type == ValueType::F32)
            chunk_load<4>(t, tensor, index, tid, l);
        else
            chunk_load<2>(t, tensor, index, tid, l);
        if (!told) {
            wait_primary_grid();
            if (tid < 32) {
                const double v = sqrt(warp_sum(partials, count, tid));
                if (tid == 0) {
                    const float told_norm = static_cast<float>(v);
                    if (blockIdx.x == 0 && norm != nullptr) *norm = told_norm;
                    const double ratio = static_cast<double>(max_norm) / (v + kClipEps);
                    // a norm that is no number, or infinite as the caller reads it, clips nothing
                    s_scale = ratio < 1.0 && told_norm < __int_as_float(0x7f800000) ? static_cast<float>(ratio) : 1.0f;
                }
            }
            __syncthreads();
            scale = s_scale;
            told = true;
        }
        if (scale == 1.0f && t.in[tensor] == t.out[tensor]) continue;
        switch (type) {
        case ValueType::F32: chunk_store<float>(t, l, scale, tid); break;
        case ValueType::F16: chunk_store<__half>(t, l, scale, tid); break;
        case ValueType::BF16: chunk_store<__nv_bfloat16>(t, l, scale, tid); break;
        }
    }
}

unsigned size_of(ValueType type) { return type == ValueType::F32 ? 4u : 2u; }

// The launches for the tables behind the first wait for what is before them as
// any launch does.
cudaError_t launch_scale(const NormTable &t, unsigned blocks, const double *work, unsigned partials, float max_norm,
                         float *norm, cudaStream_t s)
{
    norm_scale_kernel<<<blocks, kNormThreads, 0, s>>>(t, work, partials, max_norm, norm);
    return cudaGetLastError();
}

// The table of tensors [first, first + kNormTensors) of a call.
bool fill(NormTable &t, const NormTensor *tensors, size_t first, size_t count)
{
    t.count = 0;
    unsigned long long chunks = 0;
    for (size_t i = first; i < count && t.count < kNormTensors; ++i) {
        const NormTensor &x = tensors[i];
        if (x.n == 0) continue;
        const unsigned long long vectors = (x.n - head_of(x.in, x.n, size_of(x.type))) * size_of(x.type) / 16;
        const unsigned long long own = (vectors + kChunkBytes / 16 - 1) / (kChunkBytes / 16);
        chunks += own > 0 ? own : 1;
        if (chunks > UINT32_MAX / 2) return false;
        t.in[t.count] = x.in, t.out[t.count] = x.out, t.n[t.count] = x.n;
        t.type[t.count] = static_cast<unsigned char>(x.type), t.end[t.count] = static_cast<unsigned>(chunks);
        ++t.count;
    }
    t.chunks = static_cast<unsigned>(chunks);
    return true;
}

}  // namespace

cudaError_t launch_grad_norm(const NormTensor *tensors, size_t count, bool clip, float max_norm, float *norm, double *work,
                             int sms, cudaStream_t s)
{
    const unsigned most = std::min(static_cast<unsigned>(sms) * kNormPerSm, kNormBlocks);
    static thread_local NormTable t;   // 15 KB, too much for a small stack
    unsigned partials = 0;
    for (size_t i = 0; i < count; i += kNormTensors) {
        if (!fill(t, tensors, i, count < i + kNormTensors ? count : i + kNormTensors)) return cudaErrorInvalidValue;
        if (t.chunks == 0) continue;
        const unsigned blocks = t.chunks < most ? t.chunks : most;
        norm_partials_kernel<<<blocks, kNormThreads, 0, s>>>(t, work + partials);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        partials += blocks;
    }
    bool told = false;
    if (clip)
        for (size_t i = 0; i < count; i += kNormTensors) {
            if (!fill(t, tensors, i, count < i + kNormTensors ? count : i + kNormTensors)) return cudaErrorInvalidValue;
            if (t.chunks == 0) continue;
            const unsigned blocks = t.chunks < most ? t.chunks : most;
            const cudaError_t e = told ? launch_scale(t, blocks, work, partials, max_norm, nullptr, s)
                                       : launch_dependent(norm_scale_kernel, blocks, kNormThreads, s, t, work, partials, max_norm, norm);
            if (e != cudaSuccess) return e;
            told = true;
        }
    if (told) return cudaSuccess;
    return launch_dependent(norm_kernel, 1, 32, s, work, partials, norm);
}

}  // namespace devscan
