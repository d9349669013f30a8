// la_delta_fwd.cuh - the gated delta rule's forward: the chunks' own matrices
// (prep), the scan over a sequence's chunks, and their launches.  The
// mathematics and the operand layouts are in la_delta.cuh.  Each
// la_delta_fwd_w*.cu holds the instances of one key width.
#pragma once
#include "la_delta.cuh"
#include "la_delta_internal.h"

namespace la {
namespace delta {
namespace {

// ---------------------------------------------------------------- fp32 inputs
// q or k as three bf16 planes, padded to DKP columns and whole chunks.
__global__ void split_kernel(const float* __restrict__ x, __nv_bfloat16* __restrict__ out, long long plane, int T, int Tp,
                             int Dk, int DKP, long long total) {
    const long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;  // one pair of columns
    if (i >= total) return;
    const int half = DKP / 2;
    const int c = static_cast<int>(i % half) * 2;
    const long long row = i / half;
    const int t = static_cast<int>(row % Tp);
    const float* src = x + (row / Tp * T + t) * Dk;
    const float a = t < T && c < Dk ? src[c] : 0.f, b = t < T && c + 1 < Dk ? src[c + 1] : 0.f;
    uint32_t p[3];
    split2<3>(a, b, p);
#pragma unroll
    for (int j = 0; j < 3; ++j) *reinterpret_cast<uint32_t*>(out + j * plane + row * DKP + c) = p[j];
}

// ---------------------------------------------------------------- prep
// One block per (b, h, chunk): the decays, P, and E = (I + A diag(beta))^-1 by
// forward substitution in fp32 (thread = column of E).  Independent of the
// state, so every chunk runs at once.
constexpr int kPrepThreads = 128;
constexpr int kNS = C + 4;  // row stride of the fp32 matrix: 16-byte rows

template <int DKP, int NI, int NM>
constexpr size_t prep_smem() {
    return 2 * sizeof(__nv_bfloat16) * NI * C * (DKP + kPad) + sizeof(float) * (C * kNS + C) + sizeof(double) * C;
}

template <int DKP, int NI, int NM, int NP>
__global__ void __launch_bounds__(kPrepThreads) prep_kernel(Planes q, Planes k, const float* __restrict__ beta,
                                                            const float* __restrict__ log_g, int decay_kind, float scale,
                                                            int H, int Hk, int T, int n, float* __restrict__ tok,
                                                            __nv_bfloat16* __restrict__ Eout,
                                                            __nv_bfloat16* __restrict__ Pout) {
    extern __shared__ __align__(16) unsigned char smem[];
    double* L = reinterpret_cast<double*>(smem);
    float* N = reinterpret_cast<float*>(L + C);
    float* bt = N + C * kNS;
    __nv_bfloat16* kt = reinterpret_cast<__nv_bfloat16*>(bt + C);
    __nv_bfloat16* qt = kt + NI * C * (DKP + kPad);
    constexpr int kRow = DKP + kPad;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long bh = blockIdx.x / n;
    const int chunk = blockIdx.x % n, t0 = chunk * C;
    const int b = static_cast<int>(bh / H), h = static_cast<int>(bh % H);
    const long long hk = static_cast<long long>(b) * Hk + h / (H / Hk);
    load_tile<DKP, NI>(kt, k, hk, t0, tid, kPrepThreads);
    load_tile<DKP, NI>(qt, q, hk, t0, tid, kPrepThreads);
    cp_commit();

    if (warp == 0) {  // inclusive prefix of log g in 64 bits: differences of L are taken later
        double a[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = t0 + 2 * lane + i;
            float g = 0.f;
            if (t < T) {
                if (decay_kind == LA_DECAY_PER_HEAD) g = log_g[h];
                if (decay_kind == LA_DECAY_PER_STEP) g = log_g[bh * T + t];
            }
            a[i] = g < kLogFloor ? kLogFloor : g;
            bt[2 * lane + i] = t < T ? beta[bh * T + t] : 0.f;
        }
        double s = a[0] + a[1];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double x = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += x;
        }
        L[2 * lane + 1] = s;
        L[2 * lane] = s - a[1];
    }
    cp_wait<0>();
    __syncthreads();

    if (tid < C) {
        float* tk = tok + (bh * n + chunk) * kTok;
        tk[tid] = expf(static_cast<float>(L[tid]));
        tk[C + tid] = expf(static_cast<float>(L[C - 1] - L[tid]));
        tk[2 * C + tid] = bt[tid];
    }

    // K K^T and Q K^T on and below the diagonal: warp w holds rows 16 w .. 16 w + 15
    float kk[8][4] = {}, qk[8][4] = {};
#pragma unroll
    for (int d = 0; d < DKP / 16; ++d) {
        uint32_t ak[NI][4], aq[NI][4];
#pragma unroll
        for (int p = 0; p < NI; ++p) {
            ldsm4(ak[p], smem_addr(kt + (p * C + 16 * warp) * kRow + 16 * d + off_rows(lane, kRow)));
            ldsm4(aq[p], smem_addr(qt + (p * C + 16 * warp) * kRow + 16 * d + off_rows(lane, kRow)));
        }
#pragma unroll
        for (int nn = 0; nn < 4; ++nn)
            if (nn <= warp) {
#pragma unroll
                for (int p = 0; p < NI; ++p) {
                    uint32_t bk[4];
                    ldsm4(bk, smem_addr(kt + (p * C + 16 * nn) * kRow + 16 * d + off_cols(lane, kRow)));
                    mma_planes<NI, NM>(kk[2 * nn], kk[2 * nn + 1], ak, p, bk);
                    mma_planes<NI, NM>(qk[2 * nn], qk[2 * nn + 1], aq, p, bk);
                }
            }
    }
    const long long cid = bh * n + chunk;
    __nv_bfloat16* P = Pout + cid * NP * C * C;
    const int g = lane >> 2, tq = (lane & 3) * 2;
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int t = 16 * warp + g + 8 * r, s = 8 * j + tq;
            float d0 = 0.f, d1 = 0.f;
            if (s <= t) d0 = expf(static_cast<float>(L[t] - L[s]));
            if (s + 1 <= t) d1 = expf(static_cast<float>(L[t] - L[s + 1]));
            if (8 * j < 16 * warp + 16) {
                uint32_t p[NP];
                split2<NP>(scale * d0 * qk[j][2 * r], scale * d1 * qk[j][2 * r + 1], p);
#pragma unroll
                for (int i = 0; i < NP; ++i) *reinterpret_cast<uint32_t*>(P + i * C * C + t * C + s) = p[i];
            }
            float2 x;
            x.x = s < t ? d0 * kk[j][2 * r] * bt[s] : 0.f;
            x.y = s + 1 < t ? d1 * kk[j][2 * r + 1] * bt[s + 1] : 0.f;
            *reinterpret_cast<float2*>(N + t * kNS + s) = x;
        }
    __syncthreads();

    if (tid < C) {
        float x[C];
#pragma unroll
        for (int t = 0; t < C; ++t) {
            float a0 = t == tid ? 1.f : 0.f, a1 = 0.f, a2 = 0.f, a3 = 0.f;
            x[t] = 0.f;
#pragma unroll
            for (int s = 0; s < (t + 3) / 4; ++s) {
                const float4 m = *reinterpret_cast<const float4*>(N + t * kNS + 4 * s);
                a0 = fmaf(-m.x, x[4 * s], a0);
                if (4 * s + 1 < t) a1 = fmaf(-m.y, x[4 * s + 1], a1);
                if (4 * s + 2 < t) a2 = fmaf(-m.z, x[4 * s + 2], a2);
                if (4 * s + 3 < t) a3 = fmaf(-m.w, x[4 * s + 3], a3);
            }
            x[t] = (a0 + a1) + (a2 + a3);
        }
        __nv_bfloat16* E = Eout + cid * NM * C * C;
#pragma unroll
        for (int t = 0; t < C; ++t) {
            uint32_t p[NM];
            split2<NM>(x[t], 0.f, p);
#pragma unroll
            for (int i = 0; i < NM; ++i) E[(i * C + t) * C + tid] = __ushort_as_bfloat16(static_cast<unsigned short>(p[i]));
        }
    }
}

// ---------------------------------------------------------------- scan
// One warp per 16 value columns of a (b, h); the block's warps share the
// chunk's K, Q, E and P tiles, loaded kStages - 1 chunks ahead.
// kOut: 1 = outputs y, 0 = the backward's recomputation: the incoming state
// and the errors E of every chunk, as bf16 planes.
template <int DKP, int NI, int NM, int NP, int NW, bool kOut, bool kF32>
struct ScanTiles {
    static constexpr int kRow = DKP + kPad, kV = 16 * NW + kPad;
    static constexpr int k = 0;
    static constexpr int q = k + 2 * NI * C * kRow;
    static constexpr int e = q + (kOut ? 2 * NI * C * kRow : 0);
    static constexpr int p = e + 2 * NM * C * kCS;
    static constexpr int v = p + (kOut ? 2 * NP * C * kCS : 0);
    static constexpr int tok = v + (kF32 ? 0 : 2 * C * kV);
    static constexpr int bytes = tok + 4 * kTok;
    static constexpr int stages = 3 * bytes <= 227 * 1024 ? 3 : 2 * bytes <= 227 * 1024 ? 2 : 1;
};

template <int DKP, int NI, int NM, int NP, int NW, bool kOut, typename TIn>
__global__ void __launch_bounds__(32 * NW) scan_kernel(ScanArgs a) {
    constexpr bool kF32 = sizeof(TIn) == 4;
    using Tl = ScanTiles<DKP, NI, NM, NP, NW, kOut, kF32>;
    constexpr int kRow = Tl::kRow, kS = Tl::stages;
    extern __shared__ __align__(16) unsigned char smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long bh = blockIdx.x / a.vblocks;
    const int vb = blockIdx.x % a.vblocks * 16 * NW, v0 = vb + 16 * warp;
    const bool active = v0 < a.Dv;
    const int b = static_cast<int>(bh / a.H), h = static_cast<int>(bh % a.H);
    const long long hk = static_cast<long long>(b) * a.Hk + h / (a.H / a.Hk);
    const TIn* vsrc = static_cast<const TIn*>(a.v) + bh * a.T * a.Dv;

    auto load = [&](int c) {
        if (c < a.n) {
            unsigned char* st = smem + static_cast<size_t>(c % kS) * Tl::bytes;
            const long long cid = bh * a.n + c;
            load_tile<DKP, NI>(reinterpret_cast<__nv_bfloat16*>(st + Tl::k), a.kp, hk, c * C, tid, 32 * NW);
            if (kOut) load_tile<DKP, NI>(reinterpret_cast<__nv_bfloat16*>(st + Tl::q), a.qp, hk, c * C, tid, 32 * NW);
            load_square(reinterpret_cast<__nv_bfloat16*>(st + Tl::e), a.E + cid * NM * C * C, NM * C, tid, 32 * NW);
            if (kOut) load_square(reinterpret_cast<__nv_bfloat16*>(st + Tl::p), a.P + cid * NP * C * C, NP * C, tid, 32 * NW);
            if constexpr (!kF32) {
                constexpr int kVec = 2 * NW;
                for (int i = tid; i < C * kVec; i += 32 * NW) {
                    const int r = i / kVec, col = (i % kVec) * 8, t = c * C + r;
                    const bool ok = t < a.T && vb + col < a.Dv;
                    cp16(reinterpret_cast<__nv_bfloat16*>(st + Tl::v) + r * Tl::kV + col,
                         ok ? vsrc + static_cast<long long>(t) * a.Dv + vb + col : vsrc, ok);
                }
            }
            for (int i = tid; i < kTok / 4; i += 32 * NW) cp16(st + Tl::tok + 16 * i, a.tok + cid * kTok + 4 * i, true);
        }
        cp_commit();
    };

    float S[DKP / 8][4];
    state_load<DKP>(S, a.init_state ? a.init_state + bh * a.Dk * a.Dv : nullptr, a.Dk, a.Dv, v0, lane);
#pragma unroll
    for (int c = 0; c < kS - 1; ++c) load(c);

    for (int c = 0; c < a.n; ++c) {
        if constexpr (kS > 1) {
            load(c + kS - 1);
            cp_wait<kS - 1>();
        } else {
            load(c);
            cp_wait<0>();
        }
        __syncthreads();
        if (active) {
            unsigned char* st = smem + static_cast<size_t>(c % kS) * Tl::bytes;
            const __nv_bfloat16* kt = reinterpret_cast<const __nv_bfloat16*>(st + Tl::k);
            const __nv_bfloat16* qt = reinterpret_cast<const __nv_bfloat16*>(st + Tl::q);
            const __nv_bfloat16* et = reinterpret_cast<const __nv_bfloat16*>(st + Tl::e);
            const __nv_bfloat16* pt = reinterpret_cast<const __nv_bfloat16*>(st + Tl::p);
            const float* gam = reinterpret_cast<const float*>(st + Tl::tok);
            const float* rest = gam + C;
            const float* beta = gam + 2 * C;
            const int tq = (lane & 3) * 2;
            const long long cid = bh * a.n + c;

            // X = (K S)^T, Y = (Q S)^T
            float X[8][4] = {}, Y[8][4] = {};
#pragma unroll
            for (int d = 0; d < DKP / 16; ++d) {
                uint32_t s[NM][4];
                split_frag<NM>(S[2 * d], S[2 * d + 1], s);
                if constexpr (!kOut)
                    frag_to_planes<NM>(s, a.Sst + cid * NM * a.DVP * DKP, static_cast<long long>(a.DVP) * DKP, DKP, v0, 16 * d,
                                       lane);
#pragma unroll
                for (int nn = 0; nn < 4; ++nn)
#pragma unroll
                    for (int p = 0; p < NI; ++p) {
                        uint32_t r[4];
                        ldsm4(r, smem_addr(kt + (p * C + 16 * nn) * kRow + 16 * d + off_cols(lane, kRow)));
                        mma_planes<NM, NM>(X[2 * nn], X[2 * nn + 1], s, p, r);
                        if constexpr (kOut) {
                            ldsm4(r, smem_addr(qt + (p * C + 16 * nn) * kRow + 16 * d + off_cols(lane, kRow)));
                            mma_planes<NM, NM>(Y[2 * nn], Y[2 * nn + 1], s, p, r);
                        }
                    }
            }
            // R = V - e^L (K S); E = (I + A diag(beta))^-1 R
            float R[8][4];
            if constexpr (kF32)
                values_from_global(R, vsrc, c * C, a.T, a.Dv, v0, lane);
            else
                values_from_tile(R, reinterpret_cast<const __nv_bfloat16*>(st + Tl::v), Tl::kV, 16 * warp, lane);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 gm = *reinterpret_cast<const float2*>(gam + 8 * j + tq);
                R[j][0] = fmaf(-gm.x, X[j][0], R[j][0]);
                R[j][1] = fmaf(-gm.y, X[j][1], R[j][1]);
                R[j][2] = fmaf(-gm.x, X[j][2], R[j][2]);
                R[j][3] = fmaf(-gm.y, X[j][3], R[j][3]);
                X[j][0] = X[j][1] = X[j][2] = X[j][3] = 0.f;
            }
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                uint32_t r[NM][4];
                split_frag<NM>(R[2 * m], R[2 * m + 1], r);
#pragma unroll
                for (int nn = m; nn < 4; ++nn)
#pragma unroll
                    for (int p = 0; p < NM; ++p) {
                        uint32_t e[4];
                        ldsm4(e, smem_addr(et + (p * C + 16 * nn) * kCS + 16 * m + off_cols(lane, kCS)));
                        mma_planes<NM, NM>(X[2 * nn], X[2 * nn + 1], r, p, e);
                    }
            }
            if constexpr (!kOut) {
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    uint32_t e[NM][4];
                    split_frag<NM>(X[2 * m], X[2 * m + 1], e);
                    frag_to_planes<NM>(e, a.Est + cid * NM * a.DVP * C, static_cast<long long>(a.DVP) * C, C, v0, 16 * m, lane);
                }
            }
            // U = diag(beta) E; Y = scale e^L (Q S) + P U
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 bt = *reinterpret_cast<const float2*>(beta + 8 * j + tq);
                X[j][0] *= bt.x;
                X[j][1] *= bt.y;
                X[j][2] *= bt.x;
                X[j][3] *= bt.y;
                if constexpr (kOut) {
                    const float2 gm = *reinterpret_cast<const float2*>(gam + 8 * j + tq);
                    Y[j][0] *= a.scale * gm.x;
                    Y[j][1] *= a.scale * gm.y;
                    Y[j][2] *= a.scale * gm.x;
                    Y[j][3] *= a.scale * gm.y;
                }
            }
            if constexpr (kOut) {
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    uint32_t u[NM][4];
                    split_frag<NM>(X[2 * m], X[2 * m + 1], u);
#pragma unroll
                    for (int nn = m; nn < 4; ++nn)
#pragma unroll
                        for (int p = 0; p < NP; ++p) {
                            uint32_t r[4];
                            ldsm4(r, smem_addr(pt + (p * C + 16 * nn) * kCS + 16 * m + off_cols(lane, kCS)));
                            mma_planes<NM, NM>(Y[2 * nn], Y[2 * nn + 1], u, p, r);
                        }
                }
                values_to_global(Y, static_cast<TIn*>(a.out) + bh * a.T * a.Dv, c * C, a.T, a.Dv, v0, lane);
            }
            // S <- e^(L_C) S + K^T diag(e^(L_C - L)) U.  The products are summed
            // apart and added in one rounded fma, so that a long sequence does
            // not gather the tensor core's truncations in S.
            uint32_t w[4][NM][4];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
#pragma unroll
                for (int j = 2 * m; j < 2 * m + 2; ++j) {
                    const float2 rs = *reinterpret_cast<const float2*>(rest + 8 * j + tq);
                    X[j][0] *= rs.x;
                    X[j][1] *= rs.y;
                    X[j][2] *= rs.x;
                    X[j][3] *= rs.y;
                }
                split_frag<NM>(X[2 * m], X[2 * m + 1], w[m]);
            }
            const float total = gam[C - 1];
#pragma unroll
            for (int d = 0; d < DKP / 16; ++d) {
                float acc[2][4] = {};
#pragma unroll
                for (int m = 0; m < 4; ++m)
#pragma unroll
                    for (int p = 0; p < NI; ++p) {
                        uint32_t r[4];
                        ldsm4t(r, smem_addr(kt + (p * C + 16 * m) * kRow + 16 * d + off_rows(lane, kRow)));
                        mma_planes<NM, NM>(acc[0], acc[1], w[m], p, r);
                    }
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) S[2 * d + j][i] = fmaf(total, S[2 * d + j][i], acc[j][i]);
            }
        }
        __syncthreads();  // the stage is free for the load two iterations on
    }
    if (active && a.final_state) state_store<DKP>(S, a.final_state + bh * a.Dk * a.Dv, a.Dk, a.Dv, v0, lane);
}

template <typename K>
cudaError_t allow_smem(K kernel, size_t bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
}

template <int DKP, int NI, int NM, int NP, typename TIn>
cudaError_t prep_run(const Plan& p, const Args& a) {
    auto kern = prep_kernel<DKP, NI, NM, NP>;
    constexpr size_t smem = prep_smem<DKP, NI, NM>();
    cudaError_t e = allow_smem(kern, smem);
    if (e != cudaSuccess) return e;
    kern<<<static_cast<unsigned>(p.BH * p.n), kPrepThreads, smem, a.stream>>>(p.q, p.k, a.beta, a.log_g, a.decay_kind, a.scale,
                                                                             a.H, a.Hk, a.T, p.n, p.tok, p.E, p.P);
    return cudaGetLastError();
}

template <int DKP, int NI, int NM, int NP, int NW, bool kOut, typename TIn>
cudaError_t scan_run(const Plan& p, const Args& a) {
    auto kern = scan_kernel<DKP, NI, NM, NP, NW, kOut, TIn>;
    using Tl = ScanTiles<DKP, NI, NM, NP, NW, kOut, sizeof(TIn) == 4>;
    static_assert(Tl::stages * Tl::bytes <= 227 * 1024, "the scan's tiles have to fit an SM");
    constexpr size_t smem = static_cast<size_t>(Tl::stages) * Tl::bytes;
    cudaError_t e = allow_smem(kern, smem);
    if (e != cudaSuccess) return e;
    ScanArgs s = scan_args(p, a);
    s.vblocks = (a.Dv + 16 * NW - 1) / (16 * NW);
    kern<<<static_cast<unsigned>(p.BH * s.vblocks), 32 * NW, smem, a.stream>>>(s);
    return cudaGetLastError();
}

template <int DKP, int NI, int NM, int NP, bool kOut, typename TIn>
cudaError_t scan_widths(const Plan& p, const Args& a) {
    switch (p.warps) {
        case 1: return scan_run<DKP, NI, NM, NP, 1, kOut, TIn>(p, a);
        case 2: return scan_run<DKP, NI, NM, NP, 2, kOut, TIn>(p, a);
        default: return scan_run<DKP, NI, NM, NP, 4, kOut, TIn>(p, a);
    }
}

template <int DKP>
cudaError_t split_inputs(const Plan& p, const Args& a) {
    const long long total = static_cast<long long>(a.B) * a.Hk * p.n * C * (DKP / 2);
    const unsigned grid = static_cast<unsigned>((total + 255) / 256);
    split_kernel<<<grid, 256, 0, a.stream>>>(static_cast<const float*>(a.q), p.qs, p.q.plane, a.T, p.n * C, a.Dk, DKP, total);
    split_kernel<<<grid, 256, 0, a.stream>>>(static_cast<const float*>(a.k), p.ks, p.k.plane, a.T, p.n * C, a.Dk, DKP, total);
    return cudaGetLastError();
}

template <int DKP>
cudaError_t forward_width(const Plan& p, const Args& a, bool outputs) {
    cudaError_t e;
    if (a.dtype == LA_F32) {
        if ((e = split_inputs<DKP>(p, a)) != cudaSuccess) return e;
        if ((e = prep_run<DKP, 3, 3, 3, float>(p, a)) != cudaSuccess) return e;
        return outputs ? scan_widths<DKP, 3, 3, 3, true, float>(p, a) : scan_widths<DKP, 3, 3, 3, false, float>(p, a);
    }
    if (outputs) {
        // y is rounded to bf16: one plane of P adds 2^-9 of the chunk's own part to that
        if ((e = prep_run<DKP, 1, 2, 1, __nv_bfloat16>(p, a)) != cudaSuccess) return e;
        return scan_widths<DKP, 1, 2, 1, true, __nv_bfloat16>(p, a);
    }
    if ((e = prep_run<DKP, 1, 2, 2, __nv_bfloat16>(p, a)) != cudaSuccess) return e;
    return scan_widths<DKP, 1, 2, 2, false, __nv_bfloat16>(p, a);
}

}  // namespace
}  // namespace delta
}  // namespace la
