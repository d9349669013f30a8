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
#include "la_rows.cuh"
#include "la_sm100.cuh"

namespace la {
namespace norm {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxBlocks = 148 * 2;  // of the backward, resident at once: each keeps one partial sum of dw

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

// 1 / (1 + e^-z) = 1 / (1 + 2^t), t = -z log2 e, by the fast exponential and reciprocal;
// 2^t beyond the range is infinite and gives 0.  t rounded to fp32 is off by more the
// larger |z| is: 60 steps of 2^-24 of the result at z = -85.  That stays below a bf16
// step; fp32 tensors take what the rounding left along, 2^(hi + lo) = 2^hi (1 + lo ln 2)
// (B4 H16 T4096 D128 fp32: forward 67.6 us either way, gradients 128 and 131; by expf and a division 71.7 and 137).
template <typename T>
__device__ __forceinline__ float sigmoid(float z) {
    constexpr float kLog2E = 1.44269504088896341f, kLog2ELow = static_cast<float>(1.44269504088896341 - kLog2E);
    const float hi = -kLog2E * z;
    float e = ex2_approx(hi), r;
    if constexpr (sizeof(T) == 4) {
        const float lo = fmaf(-kLog2E, z, -hi) - kLog2ELow * z;
        if (fabsf(hi) < 127.f) e = fmaf(e, 0.693147180559945309f * lo, e);  // beyond, 2^t is 0 or infinite, and lo NaN for infinite z
        asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    } else {
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    }
    return r;
}

// The inner strides fit 32 bits (the entry points refuse others): one wide multiply each.
__device__ __forceinline__ long long at(const View& v, unsigned i0, unsigned i1, unsigned i2) {
    return i0 * v.stride[0] + static_cast<long long>(static_cast<unsigned long long>(i1) * static_cast<unsigned>(v.stride[1]) +
                                                     static_cast<unsigned long long>(i2) * static_cast<unsigned>(v.stride[2]));
}

template <int V>
__device__ __forceinline__ float lane_sum(const float (&acc)[V]) {
    float s = acc[0];
#pragma unroll
    for (int i = 1; i < V; ++i) s += acc[i];
    return s;
}

// The row's statistics from its values; leaves x - mu in x.  inv = 1 / D.
template <int V, int G, int NV>
__device__ __forceinline__ float normalise(float (&x)[NV][V], int D, float inv, int lane, int kind, float eps, float* red) {
    float acc[V];
    if (kind == LA_NORM_LAYER) {
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = 0.f;
#pragma unroll
        for (int u = 0; u < NV; ++u) vfmas(acc, x[u], 1.f, acc);
        const float mu = team_sum<G>(lane_sum(acc), red) * inv;
#pragma unroll
        for (int u = 0; u < NV; ++u)
            if ((u * G + lane) * V < D) vshift(x[u], x[u], -mu);  // what lies behind the row stays zero
    }
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
#pragma unroll
    for (int u = 0; u < NV; ++u) vfma(acc, x[u], x[u], acc);
    const float s = team_sum<G>(lane_sum(acc), red + 8);
    return rsqrtf((kind == LA_NORM_L2 ? s : s * inv) + eps);
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
    Raw<T, V> xr[NV], zr[NV], rr[NV];
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        const int c = (u * G + lane) * V;
        if (c < a.D) xr[u].load(xp + c);
    }
    if (a.gate.data) {
        const T* p = static_cast<const T*>(a.gate.data) + at(a.gate, i0, i1, i2);
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const int c = (u * G + lane) * V;
            if (c < a.D) zr[u].load(p + c);
        }
    }
    if (a.residual.data) {
        const T* p = static_cast<const T*>(a.residual.data) + at(a.residual, i0, i1, i2);
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const int c = (u * G + lane) * V;
            if (c < a.D) rr[u].load(p + c);
        }
    }
    float x[NV][V];
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        if ((u * G + lane) * V < a.D) {
            xr[u].unpack(x[u]);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) x[u][i] = 0.f;
        }
    }
    const float r = a.scale * normalise<V, G, NV>(x, a.D, a.inv, lane, a.kind, a.eps, red);
    T* op = static_cast<T*>(a.out.data) + at(a.out, i0, i1, i2);
    const bool silu = a.activation == LA_GATE_SILU;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        const int c = (u * G + lane) * V;
        if (c < a.D) {
            vscale(x[u], x[u], r);
            if (a.weight) {
                float w[V];
                load_weight<V>(a.weight + c, w);
                vmul(x[u], x[u], w);
            }
            if (a.gate.data) {
                float z[V], f[V];
                zr[u].unpack(z);
#pragma unroll
                for (int i = 0; i < V; ++i) f[i] = sigmoid<T>(z[i]);
                if (silu) vmul(f, f, z);
                vmul(x[u], x[u], f);
            }
            if (a.residual.data) {
                float rs[V];
                rr[u].unpack(rs);
                vfmas(x[u], x[u], 1.f, rs);
            }
            if (live) store_row<T, V>(op + c, x[u]);
        }
    }
}

// Rows on their way to a thread: where its accesses are 16 bytes, cp.async into
// slots of its own (no register holds a row in flight, and no barrier is needed);
// else none, the row is loaded when its turn comes.
template <typename T, int V, int NV>
struct Ahead {
    static constexpr bool on = V * sizeof(T) == 16;
    static constexpr int slots = !on ? 0 : NV <= 2 ? 3 : 2;
    static constexpr int bytes = slots * 3 * NV * kThreads * 16;
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

template <typename T, int V, int G, int NV>
__global__ void __launch_bounds__(kThreads, NV * V > 16 ? 1 : 2) backward_kernel(Args a) {
    using Ring = Ahead<T, V, NV>;
    // rows ahead (later a partial dw row per team), 32 floats, scale * weight
    extern __shared__ __align__(16) unsigned char ring[];
    float* shared = reinterpret_cast<float*>(ring + a.ahead);
    float* red = shared;
    float* ws = shared + 32;
    const int lane = threadIdx.x % G, team = threadIdx.x / G;
    constexpr int kTeams = kThreads / G;
    for (int c = threadIdx.x; c < a.D; c += kThreads) ws[c] = a.weight ? a.scale * a.weight[c] : a.scale;
    __syncthreads();
    float dw[NV][V];
#pragma unroll
    for (int u = 0; u < NV; ++u)
#pragma unroll
        for (int i = 0; i < V; ++i) dw[u][i] = 0.f;
    const bool silu = a.activation == LA_GATE_SILU;
    const bool gated = a.gate.data != nullptr;
    // A team takes a run of neighbouring rows: its addresses move by a stride and
    // are computed anew only where the innermost index wraps.  Every team makes
    // the same number of rounds.
    const unsigned teams = gridDim.x * kTeams, run = static_cast<unsigned>((a.rows + teams - 1) / teams);
    const long long row0 = static_cast<long long>(blockIdx.x * kTeams + team) * run;
    struct {
        unsigned i0, i1, i2;
        const T *x, *m, *z;
    } in;  // the next row to ask for
    struct {
        unsigned i0, i1, i2;
        T *x, *z;
    } to;  // the row worked on
    auto place_in = [&](long long row) {
        in.i0 = a.n1.divmod(a.n2.divmod(static_cast<unsigned>(row < a.rows ? row : a.rows - 1), in.i2), in.i1);
        in.x = static_cast<const T*>(a.x.data) + at(a.x, in.i0, in.i1, in.i2);
        in.m = static_cast<const T*>(a.dout.data) + at(a.dout, in.i0, in.i1, in.i2);
        in.z = static_cast<const T*>(a.gate.data) + (gated ? at(a.gate, in.i0, in.i1, in.i2) : 0);
    };
    auto place_to = [&](long long row) {
        to.i0 = a.n1.divmod(a.n2.divmod(static_cast<unsigned>(row < a.rows ? row : a.rows - 1), to.i2), to.i1);
        to.x = static_cast<T*>(a.dx.data) + at(a.dx, to.i0, to.i1, to.i2);
        to.z = static_cast<T*>(a.dgate.data) + (gated ? at(a.dgate, to.i0, to.i1, to.i2) : 0);
    };
    const uint32_t mine16 = static_cast<uint32_t>(__cvta_generic_to_shared(ring)) + 16 * threadIdx.x;
    auto slot = [&](unsigned k, int tensor, int u) {
        return ((k % (Ring::on ? Ring::slots : 1)) * 3 + tensor) * NV * kThreads * 16 + u * kThreads * 16;
    };
    auto advance_in = [&](unsigned k) {  // from row k to the next
        if (in.i2 + 1 < static_cast<unsigned>(a.n[2])) {
            ++in.i2;
            in.x += a.x.stride[2];
            in.m += a.dout.stride[2];
            in.z += a.gate.stride[2];
        } else {
            place_in(row0 + k + 1);
        }
    };
    auto ask = [&](unsigned k) {
        if (k < run && row0 + k < a.rows) {
#pragma unroll
            for (int u = 0; u < NV; ++u) {
                const int c = (u * G + lane) * V;
                if (c < a.D) {
                    copy16(mine16 + slot(k, 0, u), in.x + c);
                    copy16(mine16 + slot(k, 1, u), in.m + c);
                    if (gated) copy16(mine16 + slot(k, 2, u), in.z + c);
                }
            }
            advance_in(k);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    place_in(row0);
    place_to(row0);
    if constexpr (Ring::on) {
#pragma unroll
        for (int k = 0; k < Ring::slots; ++k) ask(k);
    }
    for (unsigned k = 0; k < run; ++k) {
        const bool live = row0 + k < a.rows;
        float x[NV][V], m[NV][V];
        Raw<T, V> z_raw[NV];
        if constexpr (Ring::on) asm volatile("cp.async.wait_group %0;" ::"n"(Ring::slots - 1) : "memory");
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const int c = (u * G + lane) * V;
            if (c < a.D && live) {
                Raw<T, V> xr, mr;
                if constexpr (Ring::on) {
                    const unsigned char* at16 = ring + 16 * threadIdx.x;
                    xr.load(reinterpret_cast<const T*>(at16 + slot(k, 0, u)));
                    mr.load(reinterpret_cast<const T*>(at16 + slot(k, 1, u)));
                    if (gated) z_raw[u].load(reinterpret_cast<const T*>(at16 + slot(k, 2, u)));
                } else {
                    xr.load(in.x + c);
                    mr.load(in.m + c);
                    if (gated) z_raw[u].load(in.z + c);
                }
                xr.unpack(x[u]);
                mr.unpack(m[u]);
            } else {  // behind the row, or a team behind the last row: zeros add nothing anywhere
                z_raw[u] = {};
#pragma unroll
                for (int i = 0; i < V; ++i) x[u][i] = m[u][i] = 0.f;
            }
        }
        if constexpr (Ring::on)
            ask(k + Ring::slots);
        else if (live)
            advance_in(k);
        T *dxp = to.x, *dgp = to.z;
        if (to.i2 + 1 < static_cast<unsigned>(a.n[2])) {
            ++to.i2;
            to.x += a.dx.stride[2];
            to.z += a.dgate.stride[2];
        } else {
            place_to(row0 + k + 1);
        }
        const float rn = normalise<V, G, NV>(x, a.D, a.inv, lane, a.kind, a.eps, red);
        const float r = live ? rn : 0.f;  // eps = 0: infinite for the zeros of no row
        float inner = 0.f, sum = 0.f;
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const int c = (u * G + lane) * V;
            if (c < a.D) {
                float w[V], dg[V];
                load_weight<V>(ws + c, w);
                // m is dout, then dn; dw takes its scale at the end
                if (gated) {
                    float z[V];
                    z_raw[u].unpack(z);
                    if (silu) {
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            const float s = sigmoid<T>(z[i]), act = z[i] * s, n = x[u][i] * r, t = m[u][i] * w[i];
                            dg[i] = t * n * fmaf(act, 1.f - s, s);  // silu' = s + z s (1 - s)
                            x[u][i] = n;
                            dw[u][i] = fmaf(m[u][i] * act, n, dw[u][i]);
                            m[u][i] = t * act;
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            const float s = sigmoid<T>(z[i]), n = x[u][i] * r, t = m[u][i] * w[i], d = t * s;
                            dg[i] = d * n * (1.f - s);  // sigmoid' = s (1 - s)
                            x[u][i] = n;
                            dw[u][i] = fmaf(m[u][i] * s, n, dw[u][i]);
                            m[u][i] = d;
                        }
                    }
                    if (live) store_row<T, V>(dgp + c, dg);
                } else {
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        x[u][i] *= r;
                        dw[u][i] = fmaf(m[u][i], x[u][i], dw[u][i]);
                        m[u][i] *= w[i];
                    }
                }
#pragma unroll
                for (int i = 0; i < V; ++i) inner = fmaf(m[u][i], x[u][i], inner);
                if (a.kind == LA_NORM_LAYER) {
#pragma unroll
                    for (int i = 0; i < V; ++i) sum += m[u][i];
                }
            }
        }
        inner = team_sum<G>(inner, red + 16);
        if (a.kind != LA_NORM_L2) inner *= a.inv;
        sum = a.kind == LA_NORM_LAYER ? team_sum<G>(sum, red + 24) * a.inv : 0.f;
        if (live) {
#pragma unroll
            for (int u = 0; u < NV; ++u) {
                const int c = (u * G + lane) * V;
                if (c < a.D) {
#pragma unroll
                    for (int i = 0; i < V; ++i) m[u][i] = r * (m[u][i] - fmaf(x[u][i], inner, sum));
                    store_row<T, V>(dxp + c, m[u]);
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
                for (int i = 0; i < V; ++i) part[c + i] = a.scale * dw[u][i];
        }
    } else {
        __syncthreads();  // the rows ahead have all been used
        float* rows = reinterpret_cast<float*>(ring);
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const int c = (u * G + lane) * V;
            if (c < a.D)
#pragma unroll
                for (int i = 0; i < V; ++i) rows[team * a.D + c + i] = dw[u][i];
        }
        __syncthreads();
        for (int c = threadIdx.x; c < a.D; c += kThreads) {
            float s = 0.f;
            for (int t = 0; t < kTeams; ++t) s += rows[t * a.D + c];
            part[c] = a.scale * s;
        }
    }
}

// dw: the blocks' partial rows, in a fixed order (32 threads a column).
__global__ void weight_kernel(const float* __restrict__ part, float* __restrict__ dw, int blocks, int D) {
    __shared__ float red[32][33];
    const int c = blockIdx.x * 32 + threadIdx.x;
    float s = 0.f;
    if (c < D)
        for (int b = threadIdx.y; b < blocks; b += 32) s += part[static_cast<long long>(b) * D + c];
    red[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    s = red[threadIdx.x][threadIdx.y];  // this warp's column
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const int out = blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x == 0 && out < D) dw[out] = s;
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
    // the rows ahead and, after them in the same place, the teams' partial rows; then 32 floats and the weight
    const size_t teams = kTeams > 1 && a.partial ? sizeof(float) * static_cast<size_t>(kTeams) * a.D : 0;
    const size_t rows_ahead = Ahead<T, V, NV>::bytes, ahead = teams <= rows_ahead ? rows_ahead : check::round256(teams);
    const size_t smem = ahead + sizeof(float) * (32 + static_cast<size_t>(a.D));
    Args b = a;
    b.ahead = static_cast<int>(ahead);
    cudaError_t s = cudaFuncSetAttribute(backward_kernel<T, V, G, NV>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem));
    if (s != cudaSuccess) return s;
    backward_kernel<T, V, G, NV><<<blocks, kThreads, smem, a.stream>>>(b);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess && a.partial) {
        weight_kernel<<<(a.D + 31) / 32, dim3(32, 32), 0, a.stream>>>(a.partial, a.dweight, blocks, a.D);
        e = cudaGetLastError();
    }
    return e;
}

// Threads a row: two vectors each, so that a row's index arithmetic and
// reductions are shared by 16 bf16 elements (forward, B8 H16 T4096 D128: one
// vector a lane took 38 instructions an element and 122 us, two, with two fp32
// values an instruction, 19 and 65 to 69 us), up to a warp with four; wider rows take
// the block, 1 to 32 vectors a thread.
template <typename T, int V>
cudaError_t teams(const Args& a, bool backward) {
    const int vecs = (a.D + V - 1) / V;
    if (vecs <= 4) return run<T, V, 4, 1>(a, backward);
    if (vecs <= 8) return run<T, V, 4, 2>(a, backward);
    if (vecs <= 16) return run<T, V, 8, 2>(a, backward);
    if (vecs <= 32) return run<T, V, 16, 2>(a, backward);
    if (vecs <= 64) return run<T, V, 32, 2>(a, backward);
    if (vecs <= 128) return run<T, V, 32, 4>(a, backward);
    if (vecs <= 256) return run<T, V, kThreads, 1>(a, backward);
    if (vecs <= 512) return run<T, V, kThreads, 2>(a, backward);
    if (vecs <= 1024) return run<T, V, kThreads, 4>(a, backward);
    if constexpr (V < 8) {
        if (vecs <= 2048) return run<T, V, kThreads, 8>(a, backward);
        if constexpr (V == 2) return run<T, V, kThreads, 16>(a, backward);  // 4096 vectors at most
        if constexpr (V == 1) return vecs <= 4096 ? run<T, V, kThreads, 16>(a, backward) : run<T, V, kThreads, 32>(a, backward);
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
    a.inv = 1.f / static_cast<float>(a.D);
    return dtype == LA_BF16 ? typed<__nv_bfloat16>(a, backward) : typed<float>(a, backward);
}

}  // namespace norm
}  // namespace la
