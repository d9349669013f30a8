// la_rows.cuh - vectors of a row's elements, as they lie in memory and unpacked
// to fp32 (la_norm.cu, la_rotary.cu).
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

namespace la {

// V elements in accesses of A, kept packed until they are used, so that a load in
// flight holds half the registers.
template <typename T, int V, int A = V>
struct Raw {
    static constexpr int kBytes = A * static_cast<int>(sizeof(T));
    using word = std::conditional_t<
        kBytes == 16, uint4,
        std::conditional_t<kBytes == 8, uint2, std::conditional_t<kBytes == 4, uint32_t, unsigned short>>>;
    static_assert(kBytes == 16 || kBytes == 8 || kBytes == 4 || kBytes == 2, "one memory access");
    word r[V / A];

    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int k = 0; k < V / A; ++k) r[k] = *reinterpret_cast<const word*>(p + k * A);
    }
    __device__ __forceinline__ void store(T* p) const {
#pragma unroll
        for (int k = 0; k < V / A; ++k) *reinterpret_cast<word*>(p + k * A) = r[k];
    }
    __device__ __forceinline__ void unpack(float (&x)[V]) const {
#pragma unroll
        for (int k = 0; k < V / A; ++k) {
            if constexpr (sizeof(T) == 4) {
                const float* u = reinterpret_cast<const float*>(&r[k]);
#pragma unroll
                for (int i = 0; i < A; ++i) x[k * A + i] = u[i];
            } else if constexpr (A == 1) {
                x[k] = __uint_as_float(static_cast<uint32_t>(r[k]) << 16);
            } else {
                const uint32_t* u = reinterpret_cast<const uint32_t*>(&r[k]);
#pragma unroll
                for (int i = 0; i < A; i += 2) {
                    x[k * A + i] = __uint_as_float(u[i / 2] << 16);
                    x[k * A + i + 1] = __uint_as_float(u[i / 2] & 0xffff0000u);
                }
            }
        }
    }
    __device__ __forceinline__ void pack(const float (&x)[V]) {
#pragma unroll
        for (int k = 0; k < V / A; ++k) {
            if constexpr (sizeof(T) == 4) {
                float* u = reinterpret_cast<float*>(&r[k]);
#pragma unroll
                for (int i = 0; i < A; ++i) u[i] = x[k * A + i];
            } else if constexpr (A == 1) {
                r[k] = __bfloat16_as_ushort(__float2bfloat16_rn(x[k]));
            } else {
                __nv_bfloat162* u = reinterpret_cast<__nv_bfloat162*>(&r[k]);
#pragma unroll
                for (int i = 0; i < A; i += 2) u[i / 2] = __floats2bfloat162_rn(x[k * A + i], x[k * A + i + 1]);
            }
        }
    }
};

// Elementwise fp32 on V values, two to an instruction where V is even (sm_100a's
// packed fp32 arithmetic; the same roundings as one at a time).
__device__ __forceinline__ uint64_t pair2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpair2(uint64_t r, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r)); }

// x = y z
template <int V>
__device__ __forceinline__ void vmul(float (&x)[V], const float (&y)[V], const float (&z)[V]) {
    if constexpr (V % 2 == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            uint64_t r;
            asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pair2(y[i], y[i + 1])), "l"(pair2(z[i], z[i + 1])));
            unpair2(r, x[i], x[i + 1]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = y[i] * z[i];
    }
}
// x = y s
template <int V>
__device__ __forceinline__ void vscale(float (&x)[V], const float (&y)[V], float s) {
    if constexpr (V % 2 == 0) {
        const uint64_t ss = pair2(s, s);
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            uint64_t r;
            asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pair2(y[i], y[i + 1])), "l"(ss));
            unpair2(r, x[i], x[i + 1]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = y[i] * s;
    }
}
// x = y z + w
template <int V>
__device__ __forceinline__ void vfma(float (&x)[V], const float (&y)[V], const float (&z)[V], const float (&w)[V]) {
    if constexpr (V % 2 == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            uint64_t r;
            asm("fma.rn.f32x2 %0, %1, %2, %3;"
                : "=l"(r)
                : "l"(pair2(y[i], y[i + 1])), "l"(pair2(z[i], z[i + 1])), "l"(pair2(w[i], w[i + 1])));
            unpair2(r, x[i], x[i + 1]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = fmaf(y[i], z[i], w[i]);
    }
}
// x = y s + w
template <int V>
__device__ __forceinline__ void vfmas(float (&x)[V], const float (&y)[V], float s, const float (&w)[V]) {
    if constexpr (V % 2 == 0) {
        const uint64_t ss = pair2(s, s);
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            uint64_t r;
            asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(pair2(y[i], y[i + 1])), "l"(ss), "l"(pair2(w[i], w[i + 1])));
            unpair2(r, x[i], x[i + 1]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = fmaf(y[i], s, w[i]);
    }
}
// x = y + s
template <int V>
__device__ __forceinline__ void vshift(float (&x)[V], const float (&y)[V], float s) {
    if constexpr (V % 2 == 0) {
        const uint64_t ss = pair2(s, s);
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            uint64_t r;
            asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pair2(y[i], y[i + 1])), "l"(ss));
            unpair2(r, x[i], x[i + 1]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = y[i] + s;
    }
}

template <typename T, int V, int A = V>
__device__ __forceinline__ void store_row(T* p, const float (&x)[V]) {
    Raw<T, V, A> r;
    r.pack(x);
    r.store(p);
}

}  // namespace la
