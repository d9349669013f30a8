// la_delta_decode.cu - one token of the gated delta rule, state updated in place.
//
//   e = v - g S^T k     y = scale (g S^T q + beta (k.q) e)     S <- g S + k (beta e)^T
//
// Bound by HBM: the whole fp32 state is read and written once (8 Dk Dv bytes
// per (b, h)) for 6 Dk Dv flops.  The update needs S^T k over all rows before
// it can change any of them, so a block holds its columns of S in registers
// between the read and the write (8 float4 a thread at Dk = 128): the
// state crosses HBM once each way, and y comes from the same sums (the last
// line above substitutes the updated state), not from a second pass.
// B256 H32 Dk = Dv = 128: 181 to 191 us, 0.88 to 0.92 of the measured copy rate (967 at
// Dv = 127, a column at a time).  Blocks of 32
// columns, ten and more an SM, so that one's loads run while another stores: with a
// whole head a block (two an SM) the same took 268 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "la_delta_internal.h"

namespace la {
namespace delta {
namespace {

constexpr int kThreads = 128;
constexpr int kRegs = 32;   // state values a thread holds
constexpr int kSlice = 32;  // value columns of a block: 128 rows of them fill its registers

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float* p, float x) { *p = x; }
__device__ __forceinline__ void from_f(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// One block per (b, h) and slice of value columns; a thread owns VEC
// neighbouring columns and every R-th row.
template <typename TIn, int VEC>
__global__ void __launch_bounds__(kThreads, 5) decode_kernel(DecodeArgs a, int slices) {
    constexpr int kRows = kRegs / VEC;
    __shared__ float ks[128], qs[128];
    __shared__ float sk[kThreads * VEC], sq[kThreads * VEC];
    __shared__ float us[kSlice];
    __shared__ float kq_s;
    const int tid = threadIdx.x;
    const long long bh = blockIdx.x / slices;
    const int c0 = blockIdx.x % slices * kSlice, Wc = min(kSlice, a.Dv - c0);
    const int b = static_cast<int>(bh / a.H), h = static_cast<int>(bh % a.H);
    const long long hk = static_cast<long long>(b) * a.Hk + h / (a.H / a.Hk);
    const int nc = Wc / VEC, R = kThreads / nc;
    const int c = tid % nc, r0 = tid / nc;
    const bool active = r0 < R;

    float S[kRows][VEC];
    float* base = a.state + bh * a.Dk * a.Dv + c0 + c * VEC;
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
        const int i = r0 + u * R;
        if (active && i < a.Dk) {
            if constexpr (VEC == 4) {
                const float4 x = __ldcs(reinterpret_cast<const float4*>(base + static_cast<long long>(i) * a.Dv));
                S[u][0] = x.x; S[u][1] = x.y; S[u][2] = x.z; S[u][3] = x.w;
            } else {
                S[u][0] = __ldcs(base + static_cast<long long>(i) * a.Dv);
            }
        }
    }
    if (tid < a.Dk) {
        ks[tid] = to_f(static_cast<const TIn*>(a.k)[hk * a.Dk + tid]);
        qs[tid] = to_f(static_cast<const TIn*>(a.q)[hk * a.Dk + tid]);
    }
    float lg = 0.f;
    if (a.decay_kind == LA_DECAY_PER_HEAD) lg = a.log_g[h];
    if (a.decay_kind == LA_DECAY_PER_STEP) lg = a.log_g[bh];
    const float g = expf(lg), beta = a.beta[bh];
    __syncthreads();

    float pk[VEC] = {}, pq[VEC] = {};
    if (active) {
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            const int i = r0 + u * R;
            if (i < a.Dk) {
#pragma unroll
                for (int x = 0; x < VEC; ++x) {
                    pk[x] = fmaf(ks[i], S[u][x], pk[x]);
                    pq[x] = fmaf(qs[i], S[u][x], pq[x]);
                }
            }
        }
#pragma unroll
        for (int x = 0; x < VEC; ++x) {
            sk[r0 * Wc + c * VEC + x] = pk[x];
            sq[r0 * Wc + c * VEC + x] = pq[x];
        }
    }
    if (tid < 32) {
        float kq = 0.f;
        for (int i = tid; i < a.Dk; i += 32) kq = fmaf(ks[i], qs[i], kq);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) kq += __shfl_xor_sync(0xffffffffu, kq, o);
        if (tid == 0) kq_s = kq;
    }
    __syncthreads();
    if (tid < Wc) {
        float sumk = 0.f, sumq = 0.f;
        for (int r = 0; r < R; ++r) {
            sumk += sk[r * Wc + tid];
            sumq += sq[r * Wc + tid];
        }
        const long long o = bh * a.Dv + c0 + tid;
        const float u = beta * fmaf(-g, sumk, to_f(static_cast<const TIn*>(a.v)[o]));
        us[tid] = u;
        from_f(static_cast<TIn*>(a.out) + o, a.scale * fmaf(kq_s, u, g * sumq));
    }
    __syncthreads();
    if (!active) return;
    float u4[VEC];
#pragma unroll
    for (int x = 0; x < VEC; ++x) u4[x] = us[c * VEC + x];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
        const int i = r0 + u * R;
        if (i < a.Dk) {
            const float ki = ks[i];
            if constexpr (VEC == 4) {
                float4 x;
                x.x = fmaf(ki, u4[0], g * S[u][0]);
                x.y = fmaf(ki, u4[1], g * S[u][1]);
                x.z = fmaf(ki, u4[2], g * S[u][2]);
                x.w = fmaf(ki, u4[3], g * S[u][3]);
                __stcs(reinterpret_cast<float4*>(base + static_cast<long long>(i) * a.Dv), x);
            } else {
                __stcs(base + static_cast<long long>(i) * a.Dv, fmaf(ki, u4[0], g * S[u][0]));
            }
        }
    }
}

template <typename TIn>
cudaError_t launch_typed(const DecodeArgs& a) {
    const long long BH = static_cast<long long>(a.B) * a.H;
    const int slices = (a.Dv + kSlice - 1) / kSlice;
    const unsigned grid = static_cast<unsigned>(BH * slices);
    if (a.Dv % 4 == 0)
        decode_kernel<TIn, 4><<<grid, kThreads, 0, a.stream>>>(a, slices);
    else
        decode_kernel<TIn, 1><<<grid, kThreads, 0, a.stream>>>(a, slices);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decode(const DecodeArgs& a) {
    return a.dtype == LA_BF16 ? launch_typed<__nv_bfloat16>(a) : launch_typed<float>(a);
}

}  // namespace delta
}  // namespace la
