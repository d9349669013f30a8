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
// Angles are taken modulo 2 pi in 64 bits with what the product's rounding left: at
// position 10^6 an fp32 product would be off by 0.03 rad, at 2^45 a 64-bit one by
// 0.002; here the angle is off by 2^-23 up to 2^53.
// B8 H16+16 T4096 D128 bf16: 89 to 92 us, 0.90 to 0.94 of the measured copy rate (143 us with the
// sines read from shared memory for every head and one row in flight a thread).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "la_norm.h"
#include "la_rows.cuh"

namespace la {
namespace rotary {
namespace {

constexpr int kThreads = 256;

// The roundings are spelt out, so that every vector width gives the same bits.
__device__ __forceinline__ void turn(float& a, float& b, float2 cs) {
    const float u = fmaf(a, cs.x, -__fmul_rn(b, cs.y));
    b = fmaf(a, cs.y, __fmul_rn(b, cs.x));
    a = u;
}

// Rows (heads) a thread loads before it stores the first: the output may be the
// input, so the compiler cannot move a load over a store, and one row in flight a
// thread does not fill HBM's latency.
constexpr int kBatch = 4;

// One block: tokens t0 .. t0 + tokens - 1 of sequence b, heads h0 .. h0 + per - 1
// of the two tensors' heads counted through.  A thread keeps one token's item
// (V pairs or elements of a row) and its sines and cosines in registers, and
// walks the heads.
template <typename T, int V, int A, int kLayout>
__global__ void __launch_bounds__(kThreads, 2) rotary_kernel(Args a, int tokens, int per, int tblocks, int hblocks, int turned,
                                                          FastDiv by_items) {
    constexpr int PV = kLayout == LA_ROTARY_HALF ? V : V / 2;  // pairs of an item
    extern __shared__ float2 cs[];  // [tokens][PV][turned]: cos, sin, times mscale; a warp's reads are neighbours
    const int hb = blockIdx.x % hblocks, tb = blockIdx.x / hblocks % tblocks, b = blockIdx.x / hblocks / tblocks;
    const int t0 = tb * tokens, nt = min(tokens, a.T - t0), pairs = a.R / 2;
    for (int i = threadIdx.x; i < nt * pairs; i += kThreads) {
        const int t = i / pairs, pair = i % pairs;
        const long long pos = a.pos ? a.pos[b * a.pos_stride + t0 + t] : a.start + t0 + t;
        const double p = static_cast<double>(pos), f = static_cast<double>(a.freq[pair]), x = p * f;
        constexpr double k2Pi = 6.283185307179586477, k2PiLow = 2.449293598294706414e-16;  // 2 pi = their sum
        const double k = rint(x * 0.15915494309189533577);
        const float r = static_cast<float>(fma(-k, k2PiLow, fma(-k, k2Pi, x)) + fma(p, f, -x));
        float s, c;
        sincosf(r, &s, &c);
        cs[t * pairs + pair % PV * turned + pair / PV] = make_float2(a.mscale * c, a.direction * a.mscale * s);
    }
    __syncthreads();

    const int combos = nt * static_cast<int>(by_items.d), lanes = min(combos, kThreads);
    const int step = kThreads / lanes, first = threadIdx.x / lanes;
    if (first >= step) return;
    const int h0 = hb * per, h1 = min(h0 + per, a.heads[0] + a.heads[1]);
    constexpr bool kHalf = kLayout == LA_ROTARY_HALF;
    for (int i = threadIdx.x % lanes; i < combos; i += lanes) {
        unsigned item;
        const int t = static_cast<int>(by_items.divmod(i, item));
        const bool turns = static_cast<int>(item) < turned;
        float2 k[PV];
#pragma unroll
        for (int j = 0; j < PV; ++j) k[j] = turns ? cs[t * pairs + j * turned + item] : make_float2(1.f, 0.f);
        const int at = turns ? static_cast<int>(item) * V : a.R + (static_cast<int>(item) - turned) * V;
        // an odd rest: the last item copies one element (single accesses only)
        const bool whole = A == V || at + V <= a.D;
        auto row = [&](const View (&v)[2], int h) {
            const int w = h >= a.heads[0];
            return static_cast<T*>(v[w].data) + b * v[w].stride[0] + (h - (w ? a.heads[0] : 0)) * v[w].stride[1] +
                   (t0 + t) * v[w].stride[2] + at;
        };
        for (int h = h0 + first; h < h1; h += kBatch * step) {
            Raw<T, V, A> p[kBatch], q[kHalf ? kBatch : 1];
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
                if (h + u * step < h1) {
                    const T* r = row(a.x, h + u * step);
                    if (whole)
                        p[u].load(r);
                    else
                        *reinterpret_cast<T*>(&p[u].r[0]) = *r;
                    if (kHalf && turns) q[kHalf ? u : 0].load(r + pairs);
                }
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
                if (h + u * step < h1) {
                    T* r = row(a.out, h + u * step);
                    if (turns) {
                        float y[V];
                        p[u].unpack(y);
                        if constexpr (kHalf) {
                            float z[V];
                            q[u].unpack(z);
#pragma unroll
                            for (int j = 0; j < V; ++j) turn(y[j], z[j], k[j]);
                            store_row<T, V, A>(r + pairs, z);
                        } else {
#pragma unroll
                            for (int j = 0; j < V; j += 2) turn(y[j], y[j + 1], k[j / 2]);
                        }
                        store_row<T, V, A>(r, y);
                    } else if (whole) {
                        p[u].store(r);
                    } else {
                        *r = *reinterpret_cast<const T*>(&p[u].r[0]);
                    }
                }
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
    const int turned = kLayout == LA_ROTARY_HALF ? pairs / V : a.R / V;
    rotary_kernel<T, V, A, kLayout><<<static_cast<unsigned>(grid), kThreads, smem, a.stream>>>(
        a, tokens, per, static_cast<int>(tblocks), hblocks, turned, FastDiv(turned + (a.D - a.R + V - 1) / V));
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
