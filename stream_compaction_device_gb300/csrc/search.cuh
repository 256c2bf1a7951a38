// Searches among up to INT32_MAX ordered places, in arithmetic that holds there
// (host and device: the host's tests run them over places that no memory holds).
#pragma once

namespace devscan {

// The first of places 0 .. count - 1 for which `before` does not hold; count if
// it holds for all.
template <typename Before> __host__ __device__ __forceinline__ int first_not(int count, Before &&before)
{
    int lo = 0, hi = count;
    while (lo < hi) {
        const int mid = lo + ((hi - lo) >> 1);
        if (before(mid))
            lo = mid + 1;
        else
            hi = mid;
    }
    return lo;
}

// The same with 32 places looked at at once, from [lo, hi): place(0 .. 31), of
// which those not below hi count; narrow() gets for how many of them `before`
// holds.
struct Probes {
    int lo, hi;
    __host__ __device__ __forceinline__ int step() const { return (hi - lo - 1) / 32 + 1; }
    __host__ __device__ __forceinline__ long long place(int i) const { return lo + static_cast<long long>(i) * step(); }
    __host__ __device__ __forceinline__ void narrow(int many)
    {
        const long long last = place(many - 1), next = place(many);   // the last for which it holds, and the first where it does not
        if (many == 0) {
            hi = lo;
            return;
        }
        lo = static_cast<int>(last + 1);
        hi = static_cast<int>(next < hi ? next : hi);
    }
};

}  // namespace devscan
