// Neighbouring values of fp32, fp16 or bf16 as they lie in memory, and as
// floats (sm_103a).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace devscan {

// What V neighbouring values are loaded and stored as.
template <typename T, int V> struct Raw;
template <> struct Raw<float, 1> { using type = float; };
template <> struct Raw<float, 2> { using type = float2; };
template <> struct Raw<float, 4> { using type = float4; };
template <> struct Raw<__half, 1> { using type = unsigned short; };
template <> struct Raw<__half, 2> { using type = unsigned; };
template <> struct Raw<__half, 8> { using type = uint4; };
template <> struct Raw<__nv_bfloat16, 1> { using type = unsigned short; };
template <> struct Raw<__nv_bfloat16, 2> { using type = unsigned; };
template <> struct Raw<__nv_bfloat16, 8> { using type = uint4; };

__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(float v) { return v; }
template <typename T> __device__ __forceinline__ T from_float(float v);
template <> __device__ __forceinline__ float from_float<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

template <typename T, int V>
__device__ __forceinline__ void unpack(typename Raw<T, V>::type raw, float (&v)[V])
{
    T e[V];
    __builtin_memcpy(e, &raw, sizeof(e));
#pragma unroll
    for (int k = 0; k < V; ++k) v[k] = to_float(e[k]);
}
__device__ __forceinline__ void pair_from_floats(__half2 &p, float a, float b) { p = __floats2half2_rn(a, b); }
__device__ __forceinline__ void pair_from_floats(__nv_bfloat162 &p, float a, float b) { p = __floats2bfloat162_rn(a, b); }
template <typename T> struct PairOf;
template <> struct PairOf<__half> { using type = __half2; };
template <> struct PairOf<__nv_bfloat16> { using type = __nv_bfloat162; };

template <typename T, int V>
__device__ __forceinline__ typename Raw<T, V>::type pack(const float (&v)[V])
{
    typename Raw<T, V>::type raw;
    if constexpr (sizeof(T) == 2 && V % 2 == 0) {   // one conversion for two
        typename PairOf<T>::type e[V / 2];
#pragma unroll
        for (int k = 0; k < V / 2; ++k) pair_from_floats(e[k], v[2 * k], v[2 * k + 1]);
        __builtin_memcpy(&raw, e, sizeof(e));
    } else {
        T e[V];
#pragma unroll
        for (int k = 0; k < V; ++k) e[k] = from_float<T>(v[k]);
        __builtin_memcpy(&raw, e, sizeof(e));
    }
    return raw;
}

}  // namespace devscan
