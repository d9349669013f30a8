// la_rotary.cu - rotary positions: the pairs of a row's first R elements turned
// by angles pos * freq_i, on queries and keys in one launch.
//
//   (a, b) <- mscale (a cos - b sin, a sin + b cos)
//
// pairs (i, i + R/2) in the half layout, (2 i, 2 i + 1) in the interleaved one;
// elements behind R are copied.
//
// Bound by HBM: each row is read and written once.  The angle of a token is the
// same for all its heads, so a block takes a few tokens, computes their sines
// and cosines once into shared memory and turns every head of both tensors.
// Angles are taken modulo 2 pi in 64 bits: at position 10^6 an fp32 product
// would be off by 0.03 rad, here it is off by 2^-23.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "la_norm.h"

namespace la {
namespace rotary {
namespace {

constexpr int kThreads = 256;

template <int N>
struct alignas(N) Bytes {
    unsigned char b[N];
};

// V elements in accesses of A.
template <typename T, int V, int A>
__device__ __forceinline__ void load(const T* p, float (&x)[V]) {
#pragma unroll
    for (int k = 0; k < V; k += A) {
        const Bytes<A * sizeof(T)> r = *reinterpret_cast<const Bytes<A * sizeof(T)>*>(p + k);
        const T* h = reinterpret_cast<const T*>(&r);
#pragma unroll
        for (int i = 0; i < A; ++i) x[k + i] = static_cast<float>(h[i]);
    }
}
template <typename T, int V, int A>
__device__ __forceinline__ void store(T* p, const float (&x)[V]) {
#pragma unroll
    for (int k = 0; k < V; k += A) {
        Bytes<A * sizeof(T)> r;
        T* h = reinterpret_cast<T*>(&r);
#pragma unroll
        for (int i = 0; i < A; ++i) h[i] = static_cast<T>(x[k + i]);
        *reinterpret_cast<Bytes<A * sizeof(T)>*>(p + k) = r;
    }
}

// The roundings are spelt out, so that every vector width gives the same bits.
__device__ __forceinline__ void turn(float& a, float& b, float2 cs) {
    const float u = fmaf(a, cs.x, -__fmul_rn(b, cs.y));
    b = fmaf(a, cs.y, __fmul_rn(b, cs.x));
    a = u;
}

// One block: tokens t0 .. t0 + tokens - 1 of sequence b, heads h0 .. h0 + per - 1
// of the two tensors' heads counted through.
template <typename T, int V, int A, int kLayout>
__global__ void __launch_bounds__(kThreads) rotary_kernel(Args a, int tokens, int per, int tblocks, int hblocks, FastDiv by_items,
                                                          FastDiv by_tokens) {
    extern __shared__ float2 cs[];  // [tokens][R / 2]: cos, sin, times mscale
    const int hb = blockIdx.x % hblocks, tb = blockIdx.x / hblocks % tblocks, b = blockIdx.x / hblocks / tblocks;
    const int t0 = tb * tokens, nt = min(tokens, a.T - t0), pairs = a.R / 2;
    for (int i = threadIdx.x; i < nt * pairs; i += kThreads) {
        const int t = t0 + i / pairs;
        const long long pos = a.pos ? a.pos[b * a.pos_stride + t] : a.start + t;
        const double x = static_cast<double>(pos) * static_cast<double>(a.freq[i % pairs]);
        constexpr double k2Pi = 6.283185307179586477, k2PiLow = 2.449293598294706414e-16;  // 2 pi = their sum
        const double k = rint(x * 0.15915494309189533577);
        const float r = static_cast<float>(fma(-k, k2PiLow, fma(-k, k2Pi, x)));
        float s, c;
        sincosf(r, &s, &c);
        cs[i] = make_float2(a.mscale * c, a.direction * a.mscale * s);
    }
    __syncthreads();

    // Work items of a row: vectors of pairs, then vectors of the copied rest.
    const int turned = kLayout == LA_ROTARY_HALF ? pairs / V : a.R / V, items = turned + (a.D - a.R) / A;
    const int h0 = hb * per, nh = min(per, a.heads[0] + a.heads[1] - h0);
    for (int i = threadIdx.x; i < nh * tokens * items; i += kThreads) {
        unsigned item_u, t_u;
        const int hh = h0 + static_cast<int>(by_tokens.divmod(by_items.divmod(i, item_u), t_u));
        const int item = static_cast<int>(item_u), t = static_cast<int>(t_u);
        if (t >= nt) continue;  // the last block of a sequence has fewer tokens
        const int w = hh >= a.heads[0], h = w ? hh - a.heads[0] : hh;
        const View& xv = a.x[w];
        const View& ov = a.out[w];
        const T* x = static_cast<const T*>(xv.data) + b * xv.stride[0] + h * xv.stride[1] + (t0 + t) * xv.stride[2];
        T* o = static_cast<T*>(ov.data) + b * ov.stride[0] + h * ov.stride[1] + (t0 + t) * ov.stride[2];
        const float2* c = cs + t * pairs;
        if (item >= turned) {
            const int at = a.R + (item - turned) * A;
            float y[A];
            load<T, A, A>(x + at, y);
            store<T, A, A>(o + at, y);
        } else if constexpr (kLayout == LA_ROTARY_HALF) {
            const int at = item * V;
            float p[V], q[V];
            load<T, V, A>(x + at, p);
            load<T, V, A>(x + at + pairs, q);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                turn(p[j], q[j], c[at + j]);
            }
            store<T, V, A>(o + at, p);
            store<T, V, A>(o + at + pairs, q);
        } else {
            const int at = item * V;
            float p[V];
            load<T, V, A>(x + at, p);
#pragma unroll
            for (int j = 0; j < V; j += 2) {
                turn(p[j], p[j + 1], c[(at + j) / 2]);
            }
            store<T, V, A>(o + at, p);
        }
    }
}

template <typename T, int V, int A, int kLayout>
cudaError_t run(const Args& a) {
    // Tokens a block: as many as keep its angles within 16 KB and two blocks an
    // SM; few tokens: the heads are split instead.
    const int heads = a.heads[0] + a.heads[1], pairs = a.R / 2;
    int tokens = 2048 / pairs;
    if (tokens > 16) tokens = 16;
    if (tokens < 1) tokens = 1;
    while (tokens > 1 && static_cast<long long>(a.B) * ((a.T + tokens - 1) / tokens) < 296) tokens /= 2;
    const long long tblocks = (a.T + tokens - 1) / tokens;
    int hblocks = 1;
    while (hblocks < heads && a.B * tblocks * hblocks < 296) hblocks *= 2;
    const int per = (heads + hblocks - 1) / hblocks;
    hblocks = (heads + per - 1) / per;
    const long long grid = a.B * tblocks * hblocks;
    if (grid > 2147483647LL || tblocks > 2147483647LL) return cudaErrorNotSupported;
    const size_t smem = sizeof(float2) * tokens * pairs;
    const int items = (kLayout == LA_ROTARY_HALF ? pairs / V : a.R / V) + (a.D - a.R) / A;
    rotary_kernel<T, V, A, kLayout><<<static_cast<unsigned>(grid), kThreads, smem, a.stream>>>(a, tokens, per,
                                                                                           static_cast<int>(tblocks), hblocks,
                                                                                           FastDiv(items), FastDiv(tokens));
    return cudaGetLastError();
}

template <typename T>
cudaError_t typed(const Args& a) {
    const bool half = a.layout == LA_ROTARY_HALF;
    constexpr int kWide = 16 / sizeof(T);
    auto fits = [&](int v) {
        bool ok = a.D % v == 0 && (half ? a.R / 2 : a.R) % v == 0;
        for (int w = 0; w < 2; ++w) {
            if (!a.heads[w]) continue;
            for (const View* t : {&a.x[w], &a.out[w]}) {
                ok = ok && reinterpret_cast<uintptr_t>(t->data) % (v * sizeof(T)) == 0;
                const int n[3] = {a.B, a.heads[w], a.T};
                for (int i = 0; i < 3; ++i) ok = ok && (n[i] == 1 || t->stride[i] % v == 0);
            }
        }
        return ok;
    };
    if (half)
        return fits(kWide) ? run<T, kWide, kWide, LA_ROTARY_HALF>(a)
               : fits(2)   ? run<T, 2, 2, LA_ROTARY_HALF>(a)
                           : run<T, 1, 1, LA_ROTARY_HALF>(a);
    return fits(kWide) ? run<T, kWide, kWide, LA_ROTARY_INTERLEAVED>(a)
           : fits(2)   ? run<T, 2, 2, LA_ROTARY_INTERLEAVED>(a)
                       : run<T, 2, 1, LA_ROTARY_INTERLEAVED>(a);
}

}  // namespace

cudaError_t launch(const Args& a, la_dtype dtype) {
    return dtype == LA_BF16 ? typed<__nv_bfloat16>(a) : typed<float>(a);
}

}  // namespace rotary
}  // namespace la
