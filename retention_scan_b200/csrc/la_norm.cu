// la_norm.cu - the norm of a row with its weight, gate, scale and residual, and
// its gradients.
//
//   n = (x - mu) r        rms: mu = 0, r = (mean x^2 + eps)^-1/2
//                         layer: mu = mean x, r = (mean (x - mu)^2 + eps)^-1/2
//                         l2: mu = 0, r = (sum x^2 + eps)^-1/2
//   out = residual + scale * n * w * a(gate)          a = silu, sigmoid or 1
//
// Backward, with m = scale * dout and dn = m * w * a:
//   dx = r (dn - n <dn, n> / K - [layer] mean dn), K = D (l2: 1)
//   dgate = m * n * w * a'(gate)      dw = sum over rows of m * a * n
//
// Bound by HBM: every tensor crosses it once.  A team of G threads holds a row
// in registers, so that the statistics, taken in two passes (mean, then squared
// deviations), cost no second read.  Teams are 4 to 32 lanes of a warp for the
// head widths and a block of 256 for the model width.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "la_check.h"
#include "la_norm.h"

namespace la {
namespace norm {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxBlocks = 148 * 8;  // of the backward: each keeps one partial sum of dw

template <typename T, int V>
struct Vec;
template <>
struct Vec<__nv_bfloat16, 8> {
    using raw = uint4;
};
template <>
struct Vec<__nv_bfloat16, 2> {
    using raw = uint32_t;
};
template <>
struct Vec<__nv_bfloat16, 1> {
    using raw = unsigned short;
};
template <>
struct Vec<float, 4> {
    using raw = uint4;
};
template <>
struct Vec<float, 2> {
    using raw = uint2;
};
template <>
struct Vec<float, 1> {
    using raw = uint32_t;
};

template <int V>
__device__ __forceinline__ void load(const __nv_bfloat16* p, float (&x)[V]) {
    typename Vec<__nv_bfloat16, V>::raw r = *reinterpret_cast<const typename Vec<__nv_bfloat16, V>::raw*>(p);
    const __nv_bfloat16* h = reinterpret_cast<const __nv_bfloat16*>(&r);
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = __bfloat162float(h[i]);
}
template <int V>
__device__ __forceinline__ void load(const float* p, float (&x)[V]) {
    typename Vec<float, V>::raw r = *reinterpret_cast<const typename Vec<float, V>::raw*>(p);
    const float* h = reinterpret_cast<const float*>(&r);
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = h[i];
}
template <int V>
__device__ __forceinline__ void store(__nv_bfloat16* p, const float (&x)[V]) {
    typename Vec<__nv_bfloat16, V>::raw r;
    __nv_bfloat16* h = reinterpret_cast<__nv_bfloat16*>(&r);
#pragma unroll
    for (int i = 0; i < V; ++i) h[i] = __float2bfloat16_rn(x[i]);
    *reinterpret_cast<typename Vec<__nv_bfloat16, V>::raw*>(p) = r;
}
template <int V>
__device__ __forceinline__ void store(float* p, const float (&x)[V]) {
    typename Vec<float, V>::raw r;
    float* h = reinterpret_cast<float*>(&r);
#pragma unroll
    for (int i = 0; i < V; ++i) h[i] = x[i];
    *reinterpret_cast<typename Vec<float, V>::raw*>(p) = r;
}

// V weights; the address is 16-byte aligned wherever V > 1.
template <int V>
__device__ __forceinline__ void load_weight(const float* p, float (&x)[V]) {
    if constexpr (V % 4 == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const float4 r = *reinterpret_cast<const float4*>(p + i);
            x[i] = r.x;
            x[i + 1] = r.y;
            x[i + 2] = r.z;
            x[i + 3] = r.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = p[i];
    }
}

// Sum over the team's G threads; every one of them gets it.  `red` holds 8
// floats that no earlier call's readers still use.
template <int G>
__device__ __forceinline__ float team_sum(float x, float* red) {
#pragma unroll
    for (int o = 1; o < (G < 32 ? G : 32); o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if constexpr (G == kThreads) {
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
        __syncthreads();
        x = 0.f;
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) x += red[i];
    }
    return x;
}

__device__ __forceinline__ float sigmoid(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }

__device__ __forceinline__ long long at(const View& v, unsigned i0, unsigned i1, unsigned i2) {
    return i0 * v.stride[0] + i1 * v.stride[1] + i2 * v.stride[2];
}

// The row's statistics from its values; leaves x - mu in x.
template <int V, int G, int NV>
__device__ __forceinline__ float normalise(float (&x)[NV][V], int D, int lane, int kind, float eps, float* red) {
    if (kind == LA_NORM_LAYER) {
        float s = 0.f;
#pragma unroll
        for (int u = 0; u < NV; ++u)
#pragma unroll
            for (int i = 0; i < V; ++i) s += x[u][i];
        const float mu = team_sum<G>(s, red) / D;
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const bool in = (u * G + lane) * V < D;
#pragma unroll
            for (int i = 0; i < V; ++i) x[u][i] = in ? x[u][i] - mu : 0.f;
        }
    }
    float s = 0.f;
#pragma unroll
    for (int u = 0; u < NV; ++u)
#pragma unroll
        for (int i = 0; i < V; ++i) s = fmaf(x[u][i], x[u][i], s);
    s = team_sum<G>(s, red + 8);
    return rsqrtf((kind == LA_NORM_L2 ? s : s / D) + eps);
}

template <typename T, int V, int G, int NV>
__global__ void __launch_bounds__(kThreads) forward_kernel(Args a) {
    __shared__ float red[16];
    const int lane = threadIdx.x % G;
    const long long row = static_cast<long long>(blockIdx.x) * (kThreads / G) + threadIdx.x / G;
    const bool live = row < a.rows;
    // a warp's shuffles need all its lanes: a team behind the last row repeats it and stores nothing
    const long long rc = live ? row : a.rows - 1;
    unsigned i1, i2;
    const unsigned i0 = a.n1.divmod(a.n2.divmod(static_cast<unsigned>(rc), i2), i1);
    const T* xp = static_cast<const T*>(a.x.data) + at(a.x, i0, i1, i2);
    float x[NV][V], z[NV][V], rs[NV][V];
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        const int c = (u * G + lane) * V;
        if (c < a.D) {
            load<V>(xp + c, x[u]);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) x[u][i] = 0.f;
        }
    }
    if (a.gate.data) {
        const T* p = static_cast<const T*>(a.gate.data) + at(a.gate, i0, i1, i2);
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const int c = (u * G + lane) * V;
            if (c < a.D) load<V>(p + c, z[u]);
        }
    }
    if (a.residual.data) {
        const T* p = static_cast<const T*>(a.residual.data) + at(a.residual, i0, i1, i2);
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const int c = (u * G + lane) * V;
            if (c < a.D) load<V>(p + c, rs[u]);
        }
    }
    const float r = normalise<V, G, NV>(x, a.D, lane, a.kind, a.eps, red);
    T* op = static_cast<T*>(a.out.data) + at(a.out, i0, i1, i2);
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        const int c = (u * G + lane) * V;
        if (c < a.D) {
            float w[V];
            if (a.weight) load_weight<V>(a.weight + c, w);
            float o[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float y = a.scale * x[u][i] * r;
                if (a.weight) y *= w[i];
                if (a.gate.data) {
                    const float s = sigmoid(z[u][i]);
                    y *= a.activation == LA_GATE_SILU ? z[u][i] * s : s;
                }
                o[i] = a.residual.data ? rs[u][i] + y : y;
            }
            if (live) store<V>(op + c, o);
        }
    }
}

template <typename T, int V, int G, int NV>
__global__ void __launch_bounds__(kThreads) backward_kernel(Args a) {
    extern __shared__ float shared[];  // 32 floats, then a partial dw row per team
    float* red = shared;
    const int lane = threadIdx.x % G, team = threadIdx.x / G;
    constexpr int kTeams = kThreads / G;
    float dw[NV][V];
#pragma unroll
    for (int u = 0; u < NV; ++u)
#pragma unroll
        for (int i = 0; i < V; ++i) dw[u][i] = 0.f;
    // every team of a block makes the same number of rounds
    for (long long first = static_cast<long long>(blockIdx.x) * kTeams; first < a.rows;
         first += static_cast<long long>(gridDim.x) * kTeams) {
        const bool live = first + team < a.rows;
        const long long row = live ? first + team : a.rows - 1;
        unsigned i1, i2;
        const unsigned i0 = a.n1.divmod(a.n2.divmod(static_cast<unsigned>(row), i2), i1);
        const T* xp = static_cast<const T*>(a.x.data) + at(a.x, i0, i1, i2);
        const T* dp = static_cast<const T*>(a.dout.data) + at(a.dout, i0, i1, i2);
        const T* zp = a.gate.data ? static_cast<const T*>(a.gate.data) + at(a.gate, i0, i1, i2) : nullptr;
        float x[NV][V], m[NV][V], z[NV][V];
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const int c = (u * G + lane) * V;
            if (c < a.D) {
                load<V>(xp + c, x[u]);
                load<V>(dp + c, m[u]);
                if (zp) load<V>(zp + c, z[u]);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) x[u][i] = m[u][i] = 0.f;
            }
        }
        const float r = normalise<V, G, NV>(x, a.D, lane, a.kind, a.eps, red);
        T* gp = zp && live ? static_cast<T*>(a.dgate.data) + at(a.dgate, i0, i1, i2) : nullptr;
        float inner = 0.f, sum = 0.f;
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const int c = (u * G + lane) * V;
            if (c < a.D) {
                float w[V], dg[V];
                if (a.weight) load_weight<V>(a.weight + c, w);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float n = x[u][i] * r, wi = a.weight ? w[i] : 1.f;
                    float dn = a.scale * m[u][i];
                    if (zp) {
                        const float s = sigmoid(z[u][i]);
                        const bool silu = a.activation == LA_GATE_SILU;
                        const float da = silu ? s * fmaf(z[u][i], 1.f - s, 1.f) : s * (1.f - s);
                        dg[i] = dn * n * wi * da;
                        dn *= silu ? z[u][i] * s : s;
                    }
                    if (live) dw[u][i] = fmaf(dn, n, dw[u][i]);
                    dn *= wi;
                    x[u][i] = n;
                    m[u][i] = dn;
                    inner = fmaf(dn, n, inner);
                    sum += dn;
                }
                if (gp) store<V>(gp + c, dg);
            }
        }
        inner = team_sum<G>(inner, red + 16);
        if (a.kind != LA_NORM_L2) inner /= a.D;
        sum = a.kind == LA_NORM_LAYER ? team_sum<G>(sum, red + 24) / a.D : 0.f;
        if (live) {
            T* op = static_cast<T*>(a.dx.data) + at(a.dx, i0, i1, i2);
#pragma unroll
            for (int u = 0; u < NV; ++u) {
                const int c = (u * G + lane) * V;
                if (c < a.D) {
                    float o[V];
#pragma unroll
                    for (int i = 0; i < V; ++i) o[i] = r * (m[u][i] - fmaf(x[u][i], inner, sum));
                    store<V>(op + c, o);
                }
            }
        }
        if constexpr (G == kThreads) __syncthreads();  // red is written again in the next round
    }
    if (!a.partial) return;
    float* part = a.partial + static_cast<long long>(blockIdx.x) * a.D;
    if constexpr (kTeams == 1) {
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const int c = (u * G + lane) * V;
            if (c < a.D)
#pragma unroll
                for (int i = 0; i < V; ++i) part[c + i] = dw[u][i];
        }
    } else {
        float* mine = shared + 32 + team * a.D;
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const int c = (u * G + lane) * V;
            if (c < a.D)
#pragma unroll
                for (int i = 0; i < V; ++i) mine[c + i] = dw[u][i];
        }
        __syncthreads();
        for (int c = threadIdx.x; c < a.D; c += kThreads) {
            float s = 0.f;
            for (int t = 0; t < kTeams; ++t) s += shared[32 + t * a.D + c];
            part[c] = s;
        }
    }
}

// dw: the blocks' partial rows, in their order (8 threads a column).
__global__ void weight_kernel(const float* __restrict__ part, float* __restrict__ dw, int blocks, int D) {
    __shared__ float red[8][33];
    const int c = blockIdx.x * 32 + threadIdx.x;
    float s = 0.f;
    if (c < D)
        for (int b = threadIdx.y; b < blocks; b += 8) s += part[static_cast<long long>(b) * D + c];
    red[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && c < D) {
#pragma unroll
        for (int i = 1; i < 8; ++i) s += red[i][threadIdx.x];
        dw[c] = s;
    }
}

int team_blocks(long long rows, int teams) {
    const long long need = (rows + teams - 1) / teams;
    return static_cast<int>(need < kMaxBlocks ? need : kMaxBlocks);
}

template <typename T, int V, int G, int NV>
cudaError_t run(const Args& a, bool backward) {
    constexpr int kTeams = kThreads / G;
    if (!backward) {
        forward_kernel<T, V, G, NV><<<static_cast<unsigned>((a.rows + kTeams - 1) / kTeams), kThreads, 0, a.stream>>>(a);
        return cudaGetLastError();
    }
    const int blocks = team_blocks(a.rows, kTeams);
    const size_t smem = sizeof(float) * (32 + (kTeams > 1 && a.partial ? static_cast<size_t>(kTeams) * a.D : 0));
    backward_kernel<T, V, G, NV><<<blocks, kThreads, smem, a.stream>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess && a.partial) {
        weight_kernel<<<(a.D + 31) / 32, dim3(32, 8), 0, a.stream>>>(a.partial, a.dweight, blocks, a.D);
        e = cudaGetLastError();
    }
    return e;
}

// Threads a row: as few lanes as hold it in one vector each, up to a warp with
// four (D <= 32 * 4 * V); wider rows take the block, 2 to 64 values a thread.
template <typename T, int V>
cudaError_t teams(const Args& a, bool backward) {
    const int vecs = (a.D + V - 1) / V;
    if (vecs <= 4) return run<T, V, 4, 1>(a, backward);
    if (vecs <= 8) return run<T, V, 8, 1>(a, backward);
    if (vecs <= 16) return run<T, V, 16, 1>(a, backward);
    if (vecs <= 32) return run<T, V, 32, 1>(a, backward);
    if (vecs <= 64) return run<T, V, 32, 2>(a, backward);
    if (vecs <= 128) return run<T, V, 32, 4>(a, backward);
    if (vecs <= 256) return run<T, V, kThreads, 1>(a, backward);
    if (vecs <= 512) return run<T, V, kThreads, 2>(a, backward);
    if (vecs <= 1024) return run<T, V, kThreads, 4>(a, backward);
    if constexpr (V < 8) {
        if (vecs <= 2048) return run<T, V, kThreads, 8>(a, backward);
        if constexpr (V < 4) return vecs <= 4096 ? run<T, V, kThreads, 16>(a, backward) : run<T, V, kThreads, 32>(a, backward);
    }
    return cudaErrorNotSupported;
}

// Elements a load may take: the widest that every tensor's address, strides
// and the row width allow.
int vector_width(const Args& a, int es) {
    for (int v = 16 / es; v > 1; v = v > 2 ? 2 : 1) {
        bool ok = a.D % v == 0;
        for (const View* t : {&a.x, &a.gate, &a.residual, &a.out, &a.dout, &a.dx, &a.dgate}) {
            if (!t->data) continue;
            ok = ok && reinterpret_cast<uintptr_t>(t->data) % (v * es) == 0;
            for (int i = 0; i < 3; ++i) ok = ok && (a.n[i] == 1 || t->stride[i] % v == 0);
        }
        if (a.weight) ok = ok && reinterpret_cast<uintptr_t>(a.weight) % 16 == 0;
        if (ok) return v;
    }
    return 1;
}

template <typename T>
cudaError_t typed(const Args& a, bool backward) {
    constexpr int kWide = 16 / sizeof(T);
    const int v = vector_width(a, sizeof(T));
    if (v == kWide) return teams<T, kWide>(a, backward);
    if (v == 2) return teams<T, 2>(a, backward);
    return teams<T, 1>(a, backward);
}

}  // namespace

// The partial rows of dw for any alignment: no plan has more blocks.
size_t backward_workspace_bytes(long long rows, int D) {
    const long long b = rows < kMaxBlocks ? rows : kMaxBlocks;
    return check::round256(sizeof(float) * static_cast<size_t>(b) * D);
}

cudaError_t launch(const Args& args, la_dtype dtype, bool backward) {
    Args a = args;
    a.n1 = FastDiv(static_cast<unsigned>(a.n[1]));
    a.n2 = FastDiv(static_cast<unsigned>(a.n[2]));
    return dtype == LA_BF16 ? typed<__nv_bfloat16>(a, backward) : typed<float>(a, backward);
}

}  // namespace norm
}  // namespace la
