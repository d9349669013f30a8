// la_fastdiv.h - division by a number fixed for a launch.
#pragma once
#include <cuda_runtime.h>

namespace la {

// Division of 31-bit numbers by a fixed positive one: a high product and a shift.
struct FastDiv {
    unsigned d, mul, shift;
    FastDiv() = default;
    explicit FastDiv(unsigned n) : d(n), mul(0), shift(0) {
        if (n < 2) return;
        while ((1ull << shift) < n) ++shift;
        // n is between 2^(shift-1) and 2^shift: 2^(31 + shift) / n rounded up is below 2^32
        mul = static_cast<unsigned>(((1ull << (31 + shift)) + n - 1) / n);
    }
#ifdef __CUDACC__
    __device__ __forceinline__ unsigned div(unsigned x) const { return d < 2 ? x : __umulhi(x, mul) >> (shift - 1); }
    __device__ __forceinline__ unsigned divmod(unsigned x, unsigned& rem) const {
        const unsigned q = div(x);
        rem = x - q * d;
        return q;
    }
#endif
};

}  // namespace la
