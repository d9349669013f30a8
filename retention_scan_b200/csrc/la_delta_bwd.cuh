// la_delta_bwd.cuh - the gated delta rule's gradients.  After the forward's
// kernels have left every chunk's incoming state S, errors E, P and
// T = (I + A diag(beta))^-1 in the workspace:
//
//   reverse scan, dS the gradient of the state after the chunk (C tokens):
//     dU = P^T dY + diag(e^(L_C - L)) K dS         U = diag(beta) E
//     dR = T^T diag(beta) dU                       (= dV)
//     dS <- e^(L_C) dS + scale Q^T diag(e^L) dY - K^T diag(e^L) dR
//
//   every chunk by itself, with M = dY E^T, N = dR E^T (both C x C) and
//   Z = diag(e^(L_C - L)) E dS^T:
//     dP' = scale e^(L_t - L_s) beta_s M_ts  (s <= t)
//     dA' = -e^(L_t - L_s) beta_s N_ts       (s < t)
//     dQ  = scale diag(e^L) dY S^T + dP' K
//     dK  = [dA' K - diag(e^L) dR S^T] + [dP'^T Q + dA'^T K + diag(beta) Z] = dKrow + dKcol
//     dbeta_s = k_s.Z_s + sum_t P_ts M_ts - sum_t A_ts N_ts
//     dL_t = q_t.dQ_t + k_t.dKrow_t - k_t.dKcol_t, and <S_C, dS> for t = C,
//     where <S_C, dS> = e^(L_C) <S, dS> + sum_s beta_s k_s.Z_s
//     d log g_t = sum over the chunk's tokens from t on of dL
//
// dL's sums stay within a chunk: what later chunks contribute is all in
// <S_C, dS>, so that no difference of long sums enters the decay's gradient.
#pragma once
#include "la_delta.cuh"
#include "la_delta_internal.h"

namespace la {
namespace delta {
namespace {

// ---------------------------------------------------------------- reverse scan
// Warp = 16 value columns, dS^T in its accumulators, as in the forward scan; bound
// as that by the tensor rate with eight warps an SM, by its chain with fewer (2.5 us
// a chunk at B2 H16 T4096 D128, four warps a slice: 167 us by itself, cold).
struct RevArgs {
    const void* dy;
    const unsigned char* records;
    const float* d_final;
    float* d_init;
    void* dv;
    __nv_bfloat16 *dSst, *dRst;
    int* err;
    float scale;
    int planes_apart;
    int H, Hk, T, Dk, Dv, DVP, n, vblocks;
};

template <int DKP, int NI, int NM, int NW, typename TIn>
__global__ void __launch_bounds__(32 * NW) reverse_kernel(const __grid_constant__ CUtensorMap mk,
                                                                const __grid_constant__ CUtensorMap mq,
                                                                const __grid_constant__ CUtensorMap my, RevArgs a) {
    constexpr bool kF32 = sizeof(TIn) == 4;
    using Tl = ScanTiles<DKP, NI, 2 * NM, NW, true, !kF32>;
    constexpr int kS = Tl::stages;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t base = (smem_addr(smem_raw) + 1023) & ~1023u;
    unsigned char* smem = smem_raw + (base - smem_addr(smem_raw));
    Ring<kS>* ring = reinterpret_cast<Ring<kS>*>(smem + kS * Tl::bytes);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int bh = blockIdx.x / a.vblocks;
    const int vb = blockIdx.x % a.vblocks * 16 * NW, v0 = vb + 16 * warp;
    const int nv = min(NW, (a.Dv - vb + 15) / 16);
    const int b = bh / a.H, h = bh % a.H;

    Feed<Tl, NI, true, !kF32> feed;
    feed.mk = &mk;
    feed.mq = &mq;
    feed.mv = &my;
    feed.rec_bytes = record_bytes(2 * NM);
    feed.records = a.records + static_cast<long long>(bh) * a.n * feed.rec_bytes;
    feed.rec_used = 2 * NM * kSq;
    feed.hk = b * a.Hk + h / (a.H / a.Hk);
    feed.planes_apart = a.planes_apart;
    feed.bh = bh;
    feed.v0 = vb;
    feed.nv = nv;
    feed.warps = nv;
    start_ring<Tl>(feed, base, ring, a.n, a.n - 1, -1);
    if (warp >= nv) return;

    const TIn* ysrc = static_cast<const TIn*>(a.dy) + static_cast<long long>(bh) * a.T * a.Dv;
    const int tq = (lane & 3) * 2;
    const LaneOffsets oc = swz_cols(lane), orow = swz_rows(lane);
    float S[DKP / 8][4];
    state_load<DKP>(S, a.d_final ? a.d_final + static_cast<long long>(bh) * a.Dk * a.Dv : nullptr, a.Dk, a.Dv, v0, lane);

    for (int i = 0; i < a.n; ++i) {
        const int stage = i % kS, c = a.n - 1 - i;
        if (!wait_stage(ring, stage, i / kS, a.err)) return;
        const uint32_t st = base + stage * Tl::bytes;
        const uint32_t kt = st + Tl::k, qt = st + Tl::q, et = st + Tl::rec, pt = et + NM * kSq;
        const float* gam = reinterpret_cast<const float*>(smem + stage * Tl::bytes + Tl::tok);
        const float* rest = gam + C;
        const float* beta = gam + 2 * C;
        const long long cid = static_cast<long long>(bh) * a.n + c;

        // X = (K dS)^T, then dU = e^(L_C - L) X + (P^T dY)
        float X[8][4] = {};
#pragma unroll
        for (int d = 0; d < DKP / 16; ++d) {
            uint32_t s[NM][4];
            split_frag<NM>(S[2 * d], S[2 * d + 1], s);
            put_tiles<NM>(s, a.dSst + cid * NM * a.DVP * DKP, v0 / 16, DKP / 16, d, lane);
#pragma unroll
            for (int nn = 0; nn < 4; ++nn)
#pragma unroll
                for (int p = 0; p < NI; ++p) {
                    uint32_t r[4];
                    ldsm4(r, kt + p * Tl::kTile + 8192 * (d / 4) + 2048 * nn + oc.o[d % 4]);
                    mma_planes<NM, NM>(X[2 * nn], X[2 * nn + 1], s, p, r);
                }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float2 rs = *reinterpret_cast<const float2*>(rest + 8 * j + tq);
            X[j][0] *= rs.x;
            X[j][1] *= rs.y;
            X[j][2] *= rs.x;
            X[j][3] *= rs.y;
        }
        const float total = gam[C - 1];
        {
            float Y[8][4];
            if constexpr (kF32)
                values_from_global(Y, ysrc, c * C, a.T, a.Dv, v0, lane);
            else
                values_from_tile(Y, st + Tl::v + 2048 * warp, lane);
            uint32_t y[4][NM][4];
#pragma unroll
            for (int m = 0; m < 4; ++m) {  // tokens t of P's rows; columns s <= t
                uint32_t x[NI][4];
                split_frag<NI>(Y[2 * m], Y[2 * m + 1], x);
#pragma unroll
                for (int nn = 0; nn <= m; ++nn)
#pragma unroll
                    for (int p = 0; p < NM; ++p) {
                        uint32_t r[4];
                        ldsm4t(r, pt + p * kSq + 2048 * m + orow.o[nn]);
                        mma_planes<NI, NM>(X[2 * nn], X[2 * nn + 1], x, p, r);
                    }
#pragma unroll
                for (int j = 2 * m; j < 2 * m + 2; ++j) {
                    const float2 gm = *reinterpret_cast<const float2*>(gam + 8 * j + tq);
                    Y[j][0] *= a.scale * gm.x;
                    Y[j][1] *= a.scale * gm.y;
                    Y[j][2] *= a.scale * gm.x;
                    Y[j][3] *= a.scale * gm.y;
                }
                split_frag<NM>(Y[2 * m], Y[2 * m + 1], y[m]);
            }
            // dS <- e^(L_C) dS + scale (Q^T e^L dY); dR's part follows
#pragma unroll
            for (int d = 0; d < DKP / 16; ++d) {
                float acc[2][4] = {};
#pragma unroll
                for (int m = 0; m < 4; ++m)
#pragma unroll
                    for (int p = 0; p < NI; ++p) {
                        uint32_t r[4];
                        ldsm4t(r, qt + p * Tl::kTile + 8192 * (d / 4) + 2048 * m + orow.o[d % 4]);
                        mma_planes<NM, NM>(acc[0], acc[1], y[m], p, r);
                    }
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int x = 0; x < 4; ++x) S[2 * d + j][x] = fmaf(total, S[2 * d + j][x], acc[j][x]);
            }
        }
        // dR = T^T diag(beta) dU
        float R[8][4] = {};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float2 bt = *reinterpret_cast<const float2*>(beta + 8 * j + tq);
            X[j][0] *= bt.x;
            X[j][1] *= bt.y;
            X[j][2] *= bt.x;
            X[j][3] *= bt.y;
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            uint32_t x[NM][4];
            split_frag<NM>(X[2 * m], X[2 * m + 1], x);
#pragma unroll
            for (int nn = 0; nn <= m; ++nn)
#pragma unroll
                for (int p = 0; p < NM; ++p) {
                    uint32_t r[4];
                    ldsm4t(r, et + p * kSq + 2048 * m + orow.o[nn]);
                    mma_planes<NM, NM>(R[2 * nn], R[2 * nn + 1], x, p, r);
                }
        }
        values_to_global(R, static_cast<TIn*>(a.dv) + static_cast<long long>(bh) * a.T * a.Dv, c * C, a.T, a.Dv, v0, lane);
        uint32_t w[4][NM][4];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            split_frag<NM>(R[2 * m], R[2 * m + 1], w[m]);
            put_tiles<NM>(w[m], a.dRst + cid * NM * a.DVP * C, v0 / 16, C / 16, m, lane);
#pragma unroll
            for (int j = 2 * m; j < 2 * m + 2; ++j) {
                const float2 gm = *reinterpret_cast<const float2*>(gam + 8 * j + tq);
                R[j][0] *= -gm.x;
                R[j][1] *= -gm.y;
                R[j][2] *= -gm.x;
                R[j][3] *= -gm.y;
            }
            split_frag<NM>(R[2 * m], R[2 * m + 1], w[m]);
        }
#pragma unroll
        for (int d = 0; d < DKP / 16; ++d) {
            float acc[2][4] = {};
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int p = 0; p < NI; ++p) {
                    uint32_t r[4];
                    ldsm4t(r, kt + p * Tl::kTile + 8192 * (d / 4) + 2048 * m + orow.o[d % 4]);
                    mma_planes<NM, NM>(acc[0], acc[1], w[m], p, r);
                }
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int x = 0; x < 4; ++x) S[2 * d + j][x] += acc[j][x];
        }
        release_stage<Tl>(feed, base, ring, stage, c - kS);
    }
    if (a.d_init) state_store<DKP>(S, a.d_init + static_cast<long long>(bh) * a.Dk * a.Dv, a.Dk, a.Dv, v0, lane);
}

// The same with G warps a slice (la_delta.cuh).  dY is read by all; the parts of
// dS, and diag(beta) dU and diag(e^L) dR by token block, are exchanged.
template <int DKP, int NM, int G>
struct RevSpace {  // a slice's exchange, in 16-byte words
    static constexpr int kSteps = DKP / 16 / G, kBlocks = 4 / G;
    static constexpr int s = 0;                       // [DKP / 16][NM][32]
    static constexpr int u = s + DKP / 16 * NM * 32;  // [4][NM][32]
    static constexpr int w = u + 4 * NM * 32;
    static constexpr int words = w + 4 * NM * 32;
};

template <int DKP, int NI, int NM, int G, int NS, typename TIn>
__global__ void __launch_bounds__(32 * G * NS + 32) group_reverse_kernel(const __grid_constant__ CUtensorMap mk,
                                                                         const __grid_constant__ CUtensorMap mq,
                                                                         const __grid_constant__ CUtensorMap my, RevArgs a) {
    constexpr bool kF32 = sizeof(TIn) == 4;
    using Ex = RevSpace<DKP, NM, G>;
    using Tl = ScanTiles<DKP, NI, 2 * NM, NS, true, !kF32, 16 * Ex::words * NS>;
    constexpr int kS = Tl::stages, kSteps = Ex::kSteps, kBlocks = Ex::kBlocks, kCols = DKP / G;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t base = (smem_addr(smem_raw) + 1023) & ~1023u;
    unsigned char* smem = smem_raw + (base - smem_addr(smem_raw));
    FedRing<kS>* fed = reinterpret_cast<FedRing<kS>*>(smem + kS * Tl::bytes);
    Ring<kS>* ring = &fed->ring;
    const int tid = threadIdx.x, lane = tid & 31, slice = tid / (32 * G), w = (tid >> 5) % G;
    uint4* ex = reinterpret_cast<uint4*>(smem + Tl::extra) + slice * Ex::words;
    const int bh = blockIdx.x / a.vblocks;
    const int vb = blockIdx.x % a.vblocks * 16 * NS, v0 = vb + 16 * slice;
    const int nv = min(NS, (a.Dv - vb + 15) / 16);
    const int b = bh / a.H, h = bh % a.H;
    Feed<Tl, NI, true, !kF32> feed;
    feed.mk = &mk;
    feed.mq = &mq;
    feed.mv = &my;
    feed.rec_bytes = record_bytes(2 * NM);
    feed.records = a.records + static_cast<long long>(bh) * a.n * feed.rec_bytes;
    feed.rec_used = 2 * NM * kSq;
    feed.hk = b * a.Hk + h / (a.H / a.Hk);
    feed.planes_apart = a.planes_apart;
    feed.bh = bh;
    feed.v0 = vb;
    feed.nv = nv;
    feed.warps = G * nv;
    init_fed<Tl>(feed, fed);
    if (slice == NS) {
        if (tid == 32 * G * NS) feed_ring<Tl>(feed, base, fed, a.n, a.n - 1, -1, a.err);
        return;
    }
    if (slice >= nv) return;

    const TIn* ysrc = static_cast<const TIn*>(a.dy) + static_cast<long long>(bh) * a.T * a.Dv;
    const int tq = (lane & 3) * 2;
    const LaneOffsets oc = swz_cols(lane), orow = swz_rows(lane);
    float S[kCols / 8][4];
    state_load<kCols>(S, a.d_final ? a.d_final + static_cast<long long>(bh) * a.Dk * a.Dv : nullptr, a.Dk, a.Dv, v0, lane,
                      w * kCols);
    uint32_t so[kSteps][NM][4];  // this part's planes for the chunk that comes
#pragma unroll
    for (int d = 0; d < kSteps; ++d) {
        split_frag<NM>(S[2 * d], S[2 * d + 1], so[d]);
        put_planes<NM>(ex + Ex::s + (w * kSteps + d) * NM * 32, lane, so[d]);
    }

    for (int i = 0; i < a.n; ++i) {
        const int stage = i % kS, c = a.n - 1 - i;
        const long long cid = static_cast<long long>(bh) * a.n + c;
        if (!group_agree<G>(slice, wait_stage(ring, stage, i / kS, a.err))) return;
        const uint32_t st = base + stage * Tl::bytes;
        const uint32_t kt = st + Tl::k, qt = st + Tl::q, et = st + Tl::rec, pt = et + NM * kSq;
        const float* gam = reinterpret_cast<const float*>(smem + stage * Tl::bytes + Tl::tok);
        const float* rest = gam + C;
        const float* beta = gam + 2 * C;

#pragma unroll
        for (int d = 0; d < kSteps; ++d)
            put_tiles<NM>(so[d], a.dSst + cid * NM * a.DVP * DKP, v0 / 16, DKP / 16, w * kSteps + d, lane);
        // X = (K dS)^T for this warp's tokens, then dU = e^(L_C - L) X + (P^T dY)
        float X[kBlocks][2][4] = {};
#pragma unroll
        for (int o = 0; o < G; ++o) {
            const int x = (w + o) % G;
#pragma unroll
            for (int d = 0; d < kSteps; ++d) {
                uint32_t s[NM][4];
                if (o) {
                    get_planes<NM>(ex + Ex::s + (x * kSteps + d) * NM * 32, lane, s);
                } else {
#pragma unroll
                    for (int p = 0; p < NM; ++p)
#pragma unroll
                        for (int y = 0; y < 4; ++y) s[p][y] = so[d][p][y];
                }
#pragma unroll
                for (int j = 0; j < kBlocks; ++j)
#pragma unroll
                    for (int p = 0; p < NI; ++p) {
                        uint32_t r[4];
                        ldsm4(r, kt + p * Tl::kTile + 2048 * own_block<G>(w, j) + step_offset<DKP, G>(oc, x, d));
                        mma_planes<NM, NM>(X[j][0], X[j][1], s, p, r);
                    }
            }
        }
#pragma unroll
        for (int j = 0; j < kBlocks; ++j) block_scale(X[j], rest, own_block<G>(w, j), tq);
        // dY block by block: into dU of the tokens up to it, and with its factors into dS's update,
        // whose products are summed apart and added in one rounded fma, so that a long sequence does
        // not gather the tensor core's truncations in dS (summed into it: 2.6e-5 off at T4096 without
        // decay, fp32, all of it towards zero)
        float up[2 * kSteps][4] = {};
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            float Y[2][4];
            if constexpr (kF32)
                block_from_global(Y, ysrc, c * C + 16 * m, a.T, a.Dv, v0, lane);
            else
                block_from_tile(Y, st + Tl::v + 2048 * slice, m, lane);
            uint32_t x[NI][4], y[NM][4];
            split_frag<NI>(Y[0], Y[1], x);
#pragma unroll
            for (int j = 0; j < kBlocks; ++j) {
                const int blk = own_block<G>(w, j);
                if (blk <= m) {
#pragma unroll
                    for (int p = 0; p < NM; ++p) {
                        uint32_t r[4];
                        ldsm4t(r, pt + p * kSq + 2048 * m + (orow.o[0] ^ (blk << 5)));
                        mma_planes<NI, NM>(X[j][0], X[j][1], x, p, r);
                    }
                }
            }
            block_scale(Y, gam, m, tq, a.scale);
            split_frag<NM>(Y[0], Y[1], y);
#pragma unroll
            for (int d = 0; d < kSteps; ++d)
#pragma unroll
                for (int p = 0; p < NI; ++p) {
                    uint32_t r[4];
                    ldsm4t(r, qt + p * Tl::kTile + step_offset<DKP, G>(orow, w, d) + 2048 * m);
                    mma_planes<NM, NM>(up[2 * d], up[2 * d + 1], y, p, r);
                }
        }
        const float total = gam[C - 1];
#pragma unroll
        for (int d = 0; d < 2 * kSteps; ++d)
#pragma unroll
            for (int x = 0; x < 4; ++x) S[d][x] = fmaf(total, S[d][x], up[d][x]);
        uint32_t uo[kBlocks][NM][4];
#pragma unroll
        for (int j = 0; j < kBlocks; ++j) {
            const int blk = own_block<G>(w, j);
            block_scale(X[j], beta, blk, tq);
            split_frag<NM>(X[j][0], X[j][1], uo[j]);
            put_planes<NM>(ex + Ex::u + blk * NM * 32, lane, uo[j]);
        }
        group_sync<G>(slice);
        // dR = T^T diag(beta) dU for this warp's tokens
        float R[kBlocks][2][4] = {};
#pragma unroll
        for (int o = 0; o < G; ++o)
#pragma unroll
            for (int jm = 0; jm < kBlocks; ++jm) {
                const int m = own_block<G>((w + o) % G, jm);
                uint32_t u[NM][4];
                if (o) {
                    get_planes<NM>(ex + Ex::u + m * NM * 32, lane, u);
                } else {
#pragma unroll
                    for (int p = 0; p < NM; ++p)
#pragma unroll
                        for (int x = 0; x < 4; ++x) u[p][x] = uo[jm][p][x];
                }
#pragma unroll
                for (int j = 0; j < kBlocks; ++j) {
                    const int blk = own_block<G>(w, j);
                    if (blk <= m) {
#pragma unroll
                        for (int p = 0; p < NM; ++p) {
                            uint32_t r[4];
                            ldsm4t(r, et + p * kSq + 2048 * m + (orow.o[0] ^ (blk << 5)));
                            mma_planes<NM, NM>(R[j][0], R[j][1], u, p, r);
                        }
                    }
                }
            }
        uint32_t wo[kBlocks][NM][4], wp[4 - kBlocks][NM][4];
        TIn* out = static_cast<TIn*>(a.dv) + static_cast<long long>(bh) * a.T * a.Dv;
#pragma unroll
        for (int j = 0; j < kBlocks; ++j) {
            const int blk = own_block<G>(w, j);
            block_to_global(R[j], out, c * C + 16 * blk, a.T, a.Dv, v0, lane);
            split_frag<NM>(R[j][0], R[j][1], wo[j]);
            put_tiles<NM>(wo[j], a.dRst + cid * NM * a.DVP * C, v0 / 16, C / 16, blk, lane);
            block_scale(R[j], gam, blk, tq, -1.f);
            split_frag<NM>(R[j][0], R[j][1], wo[j]);
            put_planes<NM>(ex + Ex::w + blk * NM * 32, lane, wo[j]);
        }
        group_sync<G>(slice);
#pragma unroll
        for (int o = 1; o < G; ++o)
#pragma unroll
            for (int j = 0; j < kBlocks; ++j)
                get_planes<NM>(ex + Ex::w + own_block<G>((w + o) % G, j) * NM * 32, lane, wp[(o - 1) * kBlocks + j]);
#pragma unroll
        for (int d = 0; d < kSteps; ++d) {
            float acc[2][4] = {};
            const uint32_t at = kt + step_offset<DKP, G>(orow, w, d);
#pragma unroll
            for (int o = 0; o < G; ++o)
#pragma unroll
                for (int j = 0; j < kBlocks; ++j)
#pragma unroll
                    for (int p = 0; p < NI; ++p) {
                        uint32_t r[4];
                        ldsm4t(r, at + p * Tl::kTile + 2048 * own_block<G>((w + o) % G, j));
                        if (o)
                            mma_planes<NM, NM>(acc[0], acc[1], wp[(o ? o - 1 : 0) * kBlocks + j], p, r);
                        else
                            mma_planes<NM, NM>(acc[0], acc[1], wo[j], p, r);
                    }
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int x = 0; x < 4; ++x) S[2 * d + j][x] += acc[j][x];
            split_frag<NM>(S[2 * d], S[2 * d + 1], so[d]);
            put_planes<NM>(ex + Ex::s + (w * kSteps + d) * NM * 32, lane, so[d]);
        }
        release_fed(&fed->empty[stage]);
    }
    if (a.d_init)
        state_store<kCols>(S, a.d_init + static_cast<long long>(bh) * a.Dk * a.Dv, a.Dk, a.Dv, v0, lane, w * kCols);
}

// ---------------------------------------------------------------- gradients of a chunk
// One block per (b, h, chunk), 16 warps (8 at key width 32): warp (r, c) =
// (w % 4, w / 4) holds rows 16 r .. of every product and column group c.  The
// contraction over the value columns streams 16 of them at a time (S, dS, E, dR,
// dY) through a ring of bulk copies; then the C x C gradients go through shared
// memory as A operands of the products with K and Q.  At B2 H16 T4096 D128 (2048
// chunks) 255 to 261 us.  Of a block's 32 000 cycles 4 000 are its first loads, 16 000 the
// slices (the tensor pipe's 11 000 and as many of shared memory's reads), 3 000 the
// scores, 1 500 dP' and dA', 5 000 their products, 2 500 the outputs; nothing
// overlaps between blocks with one an SM (16 warps hold all registers).  8 warps took
// 287 us; blocks that run on into the next chunk, 278 (the loop's registers spill);
// eight stages instead of three, 255; a warp each for the stages' first copies, 265.
template <int DKP, int NI, int NM, bool kF32>
struct GradTiles {
    static constexpr int kGroups = DKP >= 64 ? 4 : 2;         // column groups
    static constexpr int kThreads = 128 * kGroups;
    static constexpr int kRow = DKP + kPad;
    static constexpr int s = 0;                               // one stage: the slice's blocks ...
    static constexpr int ds = s + 2 * NM * (DKP / 16) * kBlk;
    static constexpr int e = ds + 2 * NM * (DKP / 16) * kBlk;
    static constexpr int r = e + 2 * NM * (C / 16) * kBlk;
    static constexpr int y = r + 2 * NM * (C / 16) * kBlk;    // ... and dY's 64 x 16 tile (bf16)
    static constexpr int copied = y + (kF32 ? 0 : 2048);
    static constexpr int bytes = copied;
    static constexpr int stages = 3;
    static constexpr int dp = 0;                              // [NM][C][kCS], over the stages once they are done
    static constexpr int da = dp + 2 * NM * C * kCS;
    static constexpr int over = stages * bytes > 4 * NM * C * kCS ? stages * bytes : 4 * NM * C * kCS;
    static constexpr int ring = over;
    static constexpr int k = ring + 256;
    static constexpr int q = k + 2 * NI * C * kRow;
    static constexpr int tok = q + 2 * NI * C * kRow;         // kTail floats, sums
    static constexpr int sums = tok + 4 * kTail;                    // floats: [2][kGroups][C] row sums, [4][C] column sums, per warp
    static constexpr int smem = sums + 4 * (2 * kGroups * C + 4 * C + 64) + 128;
};

// Brings one slice into a stage.
template <typename Tl, int DKP, int NM, bool kF32>
struct GradFeed {
    const __nv_bfloat16 *S, *dS, *E, *dR;  // of this chunk
    const CUtensorMap* my;
    int t0, bh, warps;

    __device__ __forceinline__ void issue(uint32_t base, Ring<Tl::stages>* ring, int st, int sl) const {
        uint64_t* bar = &ring->full[st];
        const uint32_t at = base + st * Tl::bytes;
        constexpr int kState = NM * (DKP / 16) * kBlk, kTokens = NM * (C / 16) * kBlk;
        ring->issued[st] = ring->issued[st] + 1;
        mbar_arrive_expect_tx(bar, Tl::copied);
        bulk_load(at + Tl::s, S + static_cast<long long>(sl) * kState, 2 * kState, bar);
        bulk_load(at + Tl::ds, dS + static_cast<long long>(sl) * kState, 2 * kState, bar);
        bulk_load(at + Tl::e, E + static_cast<long long>(sl) * kTokens, 2 * kTokens, bar);
        bulk_load(at + Tl::r, dR + static_cast<long long>(sl) * kTokens, 2 * kTokens, bar);
        if (!kF32) tma_load(at + Tl::y, my, bar, 16 * sl, t0, bh);
    }
};

struct GradArgs {
    Planes qp, kp;
    const void* dy;
    const __nv_bfloat16 *S, *dS, *E, *dR;
    const unsigned char* records;
    float scale;
    void *dq, *dk;         // final, where key heads are not shared
    float *dqh, *dkh;      // else per value head
    float* dbeta;
    float* d_log_g;        // per step, or null
    double* dlog;          // per chunk (per-head decay), or null
    int* err;
    int from_zero;         // no initial state: the first token's decay multiplies nothing
    int H, Hk, T, Dk, Dv, DVP, n;
};

// A warp's rows 16 row .. of every product, its column group, and the 16 rows of
// <S, dS> that it sums (none from DKP / 16 on).  Of 16 warps, the ten on or below
// the diagonal also have a block of M and N: three of them on each of two
// schedulers (warp % 4), two on the others, which take more of <S, dS> (row =
// warp % 4 put four on one scheduler and one on another).
struct GradPlace {
    int row, col, inner;
};
template <int kGroups>
__device__ __forceinline__ GradPlace grad_place(int warp) {
    if constexpr (kGroups < 4) return {warp & 3, warp >> 2, warp};
    // row | col << 2 of warps 0 .. 15: above the diagonal are warps 0, 1, 2, 3, 6 and 7
    constexpr unsigned long long kPlaces = 0xFB73'A625'ED10'9C84ull;
    const int at = static_cast<int>(kPlaces >> (4 * warp)) & 15;
    return {at & 3, at >> 2, warp < 4 ? warp : warp < 12 && (warp & 2) ? 2 * (warp >> 2) + (warp & 1) + 2 : 16};
}

// Two neighbouring elements of a K or Q tile, its planes summed.
template <int NI, int kRow>
__device__ __forceinline__ float2 tile_pair(const __nv_bfloat16* tile, int t, int col) {
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int p = NI - 1; p >= 0; --p) {
        const uint32_t u = *reinterpret_cast<const uint32_t*>(tile + (p * C + t) * kRow + col);
        s.x += low_of(u);
        s.y += high_of(u);
    }
    return s;
}

template <int DKP, int NI, int NM, typename TIn>
__global__ void __launch_bounds__(DKP >= 64 ? 512 : 256) grad_kernel(const __grid_constant__ CUtensorMap my, GradArgs a) {
    constexpr bool kF32 = sizeof(TIn) == 4;
    using Tl = GradTiles<DKP, NI, NM, kF32>;
    constexpr int kRow = Tl::kRow, kGroups = Tl::kGroups, kCols = DKP / kGroups, kJ = kCols / 8, kS = Tl::stages;
    constexpr int kNB = C / 16 / kGroups;  // 16-column blocks of M and N a warp holds
    constexpr int kGradThreads = Tl::kThreads;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t base = (smem_addr(smem_raw) + 127) & ~127u;
    unsigned char* smem = smem_raw + (base - smem_addr(smem_raw));
    Ring<kS>* ring = reinterpret_cast<Ring<kS>*>(smem + Tl::ring);
    __nv_bfloat16* kt = reinterpret_cast<__nv_bfloat16*>(smem + Tl::k);
    __nv_bfloat16* qt = reinterpret_cast<__nv_bfloat16*>(smem + Tl::q);
    float* tok = reinterpret_cast<float*>(smem + Tl::tok);
    const float2* L = reinterpret_cast<const float2*>(tok + kTok);
    float* rowsum = reinterpret_cast<float*>(smem + Tl::sums);  // [dL, k.Z][kGroups][C]
    float* colsum = rowsum + 2 * kGroups * C;                             // [4 row groups][C]
    float* wsum = colsum + 4 * C;                               // per warp
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const GradPlace place = grad_place<kGroups>(warp);
    const int wr = place.row, wc = place.col;
    const int g = lane >> 2, tq = (lane & 3) * 2;
    const int bh = blockIdx.x / a.n;
    const int chunk = blockIdx.x % a.n, t0 = chunk * C;
    const int b = bh / a.H, h = bh % a.H;
    const long long hk = static_cast<long long>(b) * a.Hk + h / (a.H / a.Hk);
    const long long cid = static_cast<long long>(bh) * a.n + chunk;
    const TIn* ysrc = static_cast<const TIn*>(a.dy) + static_cast<long long>(bh) * a.T * a.Dv;
    const int slices = a.DVP / 16;

    GradFeed<Tl, DKP, NM, kF32> feed;
    feed.S = a.S + cid * NM * a.DVP * DKP;
    feed.dS = a.dS + cid * NM * a.DVP * DKP;
    feed.E = a.E + cid * NM * a.DVP * C;
    feed.dR = a.dR + cid * NM * a.DVP * C;
    feed.my = &my;
    feed.t0 = t0;
    feed.bh = bh;
    feed.warps = kGradThreads / 32;
    start_ring<Tl>(feed, base, ring, slices, 0, 1);
    load_tile<DKP, NI>(kt, a.kp, hk, t0, tid, kGradThreads);
    load_tile<DKP, NI>(qt, a.qp, hk, t0, tid, kGradThreads);
    for (int i = tid; i < kTail / 4; i += kGradThreads)
        cp16(tok + 4 * i, a.records + (cid + 1) * record_bytes(2 * NM) - 4 * kTail + 16 * i, true);
    cp_commit();

    float M[2 * kNB][4] = {}, N[2 * kNB][4] = {};
    float dQ[kJ][4] = {}, Kr[kJ][4] = {}, Z[kJ][4] = {};
    float in[2][4] = {};  // S dS^T over 16 columns of the key width: its diagonal is summed
    bool ok = true;
    for (int sl = 0; sl < slices; ++sl) {
        const int stage = sl % kS;
        ok = wait_stage(ring, stage, sl / kS, a.err);
        if (!ok) break;
        const uint32_t st = base + stage * Tl::bytes;
        const uint32_t lo = lane * 16;
        uint32_t ay[NI][4], ae[NM][4], ar[NM][4];
        if constexpr (kF32) {
            // rows t, columns v of dY straight from global memory
            float x[2][4];
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int t = t0 + 16 * wr + g + (i >> 1) * 8, v = 16 * sl + 8 * j + tq + (i & 1);
                    x[j][i] = t < a.T && v < a.Dv ? ysrc[static_cast<long long>(t) * a.Dv + v] : 0.f;
                }
            split_frag<NI>(x[0], x[1], ay);
        } else {
            ldsm4(ay[0], st + Tl::y + 512 * wr + (lane & 15) * 32 + (lane >> 4) * 16);
        }
#pragma unroll
        for (int p = 0; p < NM; ++p) {  // A operands: tokens are the blocks' columns
            uint32_t r[4];
            ldsm4t(r, st + Tl::e + (p * (C / 16) + wr) * 512 + lo);
            ae[p][0] = r[0];
            ae[p][1] = r[2];
            ae[p][2] = r[1];
            ae[p][3] = r[3];
            ldsm4t(r, st + Tl::r + (p * (C / 16) + wr) * 512 + lo);
            ar[p][0] = r[0];
            ar[p][1] = r[2];
            ar[p][2] = r[1];
            ar[p][3] = r[3];
        }
#pragma unroll
        for (int nn = 0; nn < kNB; ++nn)
            if (kNB * wc + nn <= wr) {
#pragma unroll
                for (int p = 0; p < NM; ++p) {
                    uint32_t r[4];
                    ldsm4t(r, st + Tl::e + (p * (C / 16) + kNB * wc + nn) * 512 + lo);
                    mma_planes<NI, NM>(M[2 * nn], M[2 * nn + 1], ay, p, r);
                    mma_planes<NM, NM>(N[2 * nn], N[2 * nn + 1], ar, p, r);
                }
            }
#pragma unroll
        for (int d = 0; d < kCols / 16; ++d)
#pragma unroll
            for (int p = 0; p < NM; ++p) {
                const uint32_t at = st + (p * (DKP / 16) + wc * (kCols / 16) + d) * 512 + lo;
                uint32_t r[4];
                ldsm4t(r, at + Tl::s);
                mma_planes<NI, NM>(dQ[2 * d], dQ[2 * d + 1], ay, p, r);
                mma_planes<NM, NM>(Kr[2 * d], Kr[2 * d + 1], ar, p, r);
                ldsm4t(r, at + Tl::ds);
                mma_planes<NM, NM>(Z[2 * d], Z[2 * d + 1], ae, p, r);
            }
        if (place.inner < DKP / 16) {
            uint32_t as[NM][4];
#pragma unroll
            for (int p = 0; p < NM; ++p) ldsm4(as[p], st + Tl::s + (p * (DKP / 16) + place.inner) * 512 + lo);
#pragma unroll
            for (int p = 0; p < NM; ++p) {
                uint32_t r[4], x[4];
                ldsm4(r, st + Tl::ds + (p * (DKP / 16) + place.inner) * 512 + lo);
                x[0] = r[0];
                x[1] = r[2];
                x[2] = r[1];
                x[3] = r[3];
                mma_planes<NM, NM>(in[0], in[1], as, p, x);
            }
        }
        release_stage<Tl>(feed, base, ring, stage, sl + kS < slices ? sl + kS : -1);
    }
    // all warps of a block give up together: no copy is in flight, the outputs are incomplete, the error word says so
    cp_wait<0>();
    if (!__syncthreads_and(ok)) return;
    // diagonal of the 16 x 16 accumulator: rows g, g + 8; columns 8 j + tq, + 1
    float inner = 0.f;
    if (g == tq) inner = in[0][0] + in[1][2];
    if (g == tq + 1) inner = in[0][1] + in[1][3];

    // The chunk's scores again (exact operands), in the layout of M and N.
    const float* gam = tok;
    const float* rest = tok + C;
    const float* beta = tok + 2 * C;
    float qk[2 * kNB][4] = {}, kk[2 * kNB][4] = {};
#pragma unroll
    for (int d = 0; d < DKP / 16; ++d) {
        uint32_t aq[NI][4], ak[NI][4];
#pragma unroll
        for (int p = 0; p < NI; ++p) {
            ldsm4(aq[p], smem_addr(qt + (p * C + 16 * wr) * kRow + 16 * d + off_rows(lane, kRow)));
            ldsm4(ak[p], smem_addr(kt + (p * C + 16 * wr) * kRow + 16 * d + off_rows(lane, kRow)));
        }
#pragma unroll
        for (int nn = 0; nn < kNB; ++nn)
            if (kNB * wc + nn <= wr) {
#pragma unroll
                for (int p = 0; p < NI; ++p) {
                    uint32_t r[4];
                    ldsm4(r, smem_addr(kt + (p * C + 16 * (kNB * wc + nn)) * kRow + 16 * d + off_cols(lane, kRow)));
                    mma_planes<NI, NM>(qk[2 * nn], qk[2 * nn + 1], aq, p, r);
                    mma_planes<NI, NM>(kk[2 * nn], kk[2 * nn + 1], ak, p, r);
                }
            }
    }
    // dP', dA' as planes in shared memory; dbeta's column sums.
    __nv_bfloat16* dpt = reinterpret_cast<__nv_bfloat16*>(smem + Tl::dp);
    __nv_bfloat16* dat = reinterpret_cast<__nv_bfloat16*>(smem + Tl::da);
#pragma unroll
    for (int j = 0; j < 2 * kNB; ++j) {
        const int s0 = 16 * kNB * wc + 8 * j + tq;
        float cs[2] = {0.f, 0.f};
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int t = 16 * wr + g + 8 * r;
            float p2[2], a2[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int s = s0 + x;
                const float d = s <= t ? decay_between(L[t], L[s]) : 0.f;
                const float m = a.scale * d * M[j][2 * r + x], w = s < t ? -d * N[j][2 * r + x] : 0.f;
                cs[x] += (s <= t ? m * qk[j][2 * r + x] : 0.f) + (s < t ? w * kk[j][2 * r + x] : 0.f);
                p2[x] = s <= t ? m * beta[s] : 0.f;
                a2[x] = w * beta[s];
            }
            uint32_t pl[NM];
            split2<NM>(p2[0], p2[1], pl);
#pragma unroll
            for (int p = 0; p < NM; ++p) *reinterpret_cast<uint32_t*>(dpt + (p * C + t) * kCS + s0) = pl[p];
            split2<NM>(a2[0], a2[1], pl);
#pragma unroll
            for (int p = 0; p < NM; ++p) *reinterpret_cast<uint32_t*>(dat + (p * C + t) * kCS + s0) = pl[p];
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) cs[x] += __shfl_xor_sync(0xffffffffu, cs[x], o);
            if (g == 0) colsum[wr * C + s0 + x] = cs[x];
        }
    }
    __syncthreads();

    // Row factors of the parts from the states, then the products with K and Q.
    float Kc[kJ][4];
    float zk[2] = {0.f, 0.f};  // k_t . Z_t over this warp's columns
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int t = 16 * wr + g + 8 * r;
        const float gm = gam[t], rs = rest[t], bt = beta[t];
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
            const float2 kv = tile_pair<NI, kRow>(kt, t, kCols * wc + 8 * j + tq);
            const float z0 = rs * Z[j][2 * r], z1 = rs * Z[j][2 * r + 1];
            dQ[j][2 * r] *= a.scale * gm;
            dQ[j][2 * r + 1] *= a.scale * gm;
            Kr[j][2 * r] *= -gm;
            Kr[j][2 * r + 1] *= -gm;
            zk[r] = fmaf(kv.x, z0, fmaf(kv.y, z1, zk[r]));
            Kc[j][2 * r] = bt * z0;
            Kc[j][2 * r + 1] = bt * z1;
        }
    }
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        uint32_t x[NM][4], y[NM][4], xt[NM][4], yt[NM][4];
        const bool below = m <= wr, above = m >= wr;  // blocks of dP'[rows, 16 m] and dP'[16 m, rows]^T
#pragma unroll
        for (int p = 0; p < NM; ++p) {
            if (below) {
                ldsm4(x[p], smem_addr(dpt + (p * C + 16 * wr) * kCS + 16 * m + off_rows(lane, kCS)));
                ldsm4(y[p], smem_addr(dat + (p * C + 16 * wr) * kCS + 16 * m + off_rows(lane, kCS)));
            }
            if (above) {
                ldsm4t(xt[p], smem_addr(dpt + (p * C + 16 * m) * kCS + 16 * wr + off_cols(lane, kCS)));
                ldsm4t(yt[p], smem_addr(dat + (p * C + 16 * m) * kCS + 16 * wr + off_cols(lane, kCS)));
            }
        }
#pragma unroll
        for (int d = 0; d < kCols / 16; ++d)
#pragma unroll
            for (int p = 0; p < NI; ++p) {
                uint32_t r[4];
                ldsm4t(r, smem_addr(kt + (p * C + 16 * m) * kRow + kCols * wc + 16 * d + off_rows(lane, kRow)));
                if (below) {
                    mma_planes<NM, NM>(dQ[2 * d], dQ[2 * d + 1], x, p, r);
                    mma_planes<NM, NM>(Kr[2 * d], Kr[2 * d + 1], y, p, r);
                }
                if (above) {
                    mma_planes<NM, NM>(Kc[2 * d], Kc[2 * d + 1], yt, p, r);
                    ldsm4t(r, smem_addr(qt + (p * C + 16 * m) * kRow + kCols * wc + 16 * d + off_rows(lane, kRow)));
                    mma_planes<NM, NM>(Kc[2 * d], Kc[2 * d + 1], xt, p, r);
                }
            }
    }

    // Outputs and the row sums of dL.
    const long long head = a.dqh ? bh : hk;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int t = 16 * wr + g + 8 * r;
        float dl = 0.f;
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
            const int col = kCols * wc + 8 * j + tq;
            const float2 kv = tile_pair<NI, kRow>(kt, t, col), qv = tile_pair<NI, kRow>(qt, t, col);
            dl = fmaf(qv.x, dQ[j][2 * r], dl);
            dl = fmaf(qv.y, dQ[j][2 * r + 1], dl);
            dl = fmaf(kv.x, Kr[j][2 * r] - Kc[j][2 * r], dl);
            dl = fmaf(kv.y, Kr[j][2 * r + 1] - Kc[j][2 * r + 1], dl);
            if (t0 + t < a.T) {
                const long long o = (head * a.T + t0 + t) * a.Dk + col;
                const float q0 = dQ[j][2 * r], q1 = dQ[j][2 * r + 1];
                const float k0 = Kr[j][2 * r] + Kc[j][2 * r], k1 = Kr[j][2 * r + 1] + Kc[j][2 * r + 1];
                if (a.dqh || sizeof(TIn) == 4) {
                    float* dq = a.dqh ? a.dqh : static_cast<float*>(a.dq);
                    float* dk = a.dkh ? a.dkh : static_cast<float*>(a.dk);
                    if (col < a.Dk) {
                        dq[o] = q0;
                        dk[o] = k0;
                    }
                    if (col + 1 < a.Dk) {
                        dq[o + 1] = q1;
                        dk[o + 1] = k1;
                    }
                } else if (col < a.Dk) {
                    *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.dq) + o) = pack(q0, q1);
                    *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.dk) + o) = pack(k0, k1);
                }
            }
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            dl += __shfl_xor_sync(0xffffffffu, dl, o);
            zk[r] += __shfl_xor_sync(0xffffffffu, zk[r], o);
        }
        if ((lane & 3) == 0) {
            rowsum[wc * C + t] = dl;
            rowsum[(kGroups + wc) * C + t] = zk[r];
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) inner += __shfl_xor_sync(0xffffffffu, inner, o);
    if (lane == 0) wsum[warp] = inner;
    __syncthreads();

    if (warp == 0) {
        float in = 0.f;
        for (int i = 0; i < kGradThreads / 32; ++i) in += wsum[i];
        double end = static_cast<double>(gam[C - 1]) * in, dl[2];
        float cz = 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = 2 * lane + i;
            float z = 0.f;
            dl[i] = 0.0;
#pragma unroll
            for (int x = 0; x < kGroups; ++x) {
                z += rowsum[(kGroups + x) * C + t];
                dl[i] += rowsum[x * C + t];
            }
            float db = z;
#pragma unroll
            for (int r = 0; r < 4; ++r) db += colsum[r * C + t];
            if (t0 + t < a.T) a.dbeta[bh * a.T + t0 + t] = db;
            cz = fmaf(beta[t], z, cz);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) cz += __shfl_xor_sync(0xffffffffu, cz, o);
        end += cz;
        double s = dl[0] + dl[1];  // suffix sums: this lane's two tokens and all after them
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double y = __shfl_down_sync(0xffffffffu, s, o);
            if (lane + o < 32) s += y;
        }
        const int t = t0 + 2 * lane;
        const double d0 = t == 0 && a.from_zero ? 0.0 : s + end, d1 = s - dl[0] + end;
        if (a.d_log_g) {
            if (t < a.T) a.d_log_g[bh * a.T + t] = static_cast<float>(d0);
            if (t + 1 < a.T) a.d_log_g[bh * a.T + t + 1] = static_cast<float>(d1);
        }
        if (a.dlog) {
            double c = (t < a.T ? d0 : 0.0) + (t + 1 < a.T ? d1 : 0.0);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
            if (lane == 0) a.dlog[cid] = c;
        }
    }
}

// Sum over the value heads of a key head, in their order: dq, then dk (blockIdx.y).
template <typename TOut>
__global__ void group_sum_kernel(const float* __restrict__ dqh, const float* __restrict__ dkh, TOut* __restrict__ dq,
                                 TOut* __restrict__ dk, int rep, long long inner, long long total) {
    const float* x = blockIdx.y ? dkh : dqh;
    TOut* out = blockIdx.y ? dk : dq;
    const long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i >= total) return;
    const long long key = i / inner, at = i % inner;
    float s = 0.f;
    for (int r = 0; r < rep; ++r) s += x[(key * rep + r) * inner + at];
    if constexpr (sizeof(TOut) == 2)
        out[i] = __float2bfloat16_rn(s);
    else
        out[i] = s;
}

template <int DKP, int NI, int NM, int NW, typename TIn>
cudaError_t reverse_run(const Plan& p, const Args& a, RevArgs r) {
    auto kern = reverse_kernel<DKP, NI, NM, NW, TIn>;
    using Tl = ScanTiles<DKP, NI, 2 * NM, NW, true, sizeof(TIn) == 2>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Tl::smem);
    if (e != cudaSuccess) return e;
    r.vblocks = (a.Dv + 16 * NW - 1) / (16 * NW);
    kern<<<static_cast<unsigned>(p.BH * r.vblocks), 32 * NW, Tl::smem, a.stream>>>(p.maps.k, p.maps.q, p.maps.dy, r);
    return cudaGetLastError();
}

template <int DKP, int NI, int NM, int G, int NS, typename TIn>
cudaError_t group_reverse_run(const Plan& p, const Args& a, RevArgs r) {
    auto kern = group_reverse_kernel<DKP, NI, NM, G, NS, TIn>;
    using Tl = ScanTiles<DKP, NI, 2 * NM, NS, true, sizeof(TIn) == 2, 16 * RevSpace<DKP, NM, G>::words * NS>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Tl::smem);
    if (e != cudaSuccess) return e;
    r.vblocks = (a.Dv + 16 * NS - 1) / (16 * NS);
    kern<<<static_cast<unsigned>(p.BH * r.vblocks), 32 * G * NS + 32, Tl::smem, a.stream>>>(p.maps.k, p.maps.q, p.maps.dy, r);
    return cudaGetLastError();
}

template <int DKP, int NI, int NM, typename TIn>
cudaError_t backward_typed(const Plan& p, const Args& a) {
    RevArgs r{};
    r.dy = a.dy;
    r.records = p.records;
    r.err = p.err;
    r.planes_apart = a.B * a.Hk;
    r.d_final = a.d_final_state;
    r.d_init = a.d_init_state;
    r.dv = a.dv;
    r.dSst = p.dS;
    r.dRst = p.dR;
    r.scale = a.scale;
    r.H = a.H;
    r.Hk = a.Hk;
    r.T = a.T;
    r.Dk = a.Dk;
    r.Dv = a.Dv;
    r.DVP = p.DVP;
    r.n = p.n;
    // four warps a slice, two where the key width has two 16-column steps (at B2 H16 T4096 D128,
    // two slices a block: four 163 us, two 169)
    constexpr int G = DKP >= 64 ? 4 : 2;
    cudaError_t e = p.group ? (p.warps == 1 ? group_reverse_run<DKP, NI, NM, G, 1, TIn>(p, a, r)
                                            : group_reverse_run<DKP, NI, NM, G, 2, TIn>(p, a, r))
                    : p.warps == 1 ? reverse_run<DKP, NI, NM, 1, TIn>(p, a, r)
                    : p.warps == 2 ? reverse_run<DKP, NI, NM, 2, TIn>(p, a, r)
                    : p.warps == 4 ? reverse_run<DKP, NI, NM, 4, TIn>(p, a, r)
                                   : reverse_run<DKP, NI, NM, 8, TIn>(p, a, r);
    if (e != cudaSuccess) return e;

    GradArgs g{};
    g.qp = p.q;
    g.kp = p.k;
    g.dy = a.dy;
    g.S = p.S;
    g.dS = p.dS;
    g.E = p.Er;
    g.dR = p.dR;
    g.records = p.records;
    g.scale = a.scale;
    g.dq = a.dq;
    g.dk = a.dk;
    g.dqh = p.dqh;
    g.dkh = p.dkh;
    g.dbeta = a.dbeta;
    g.d_log_g = a.decay_kind == LA_DECAY_PER_STEP ? a.d_log_g : nullptr;
    g.dlog = a.decay_kind == LA_DECAY_PER_HEAD && a.d_log_g ? p.dlog : nullptr;
    g.from_zero = !a.init_state;
    g.H = a.H;
    g.Hk = a.Hk;
    g.T = a.T;
    g.Dk = a.Dk;
    g.Dv = a.Dv;
    g.DVP = p.DVP;
    g.n = p.n;
    g.err = r.err;
    auto kern = grad_kernel<DKP, NI, NM, TIn>;
    using Tl = GradTiles<DKP, NI, NM, sizeof(TIn) == 4>;
    static_assert(Tl::smem <= 227 * 1024, "the gradient kernel's tiles have to fit an SM");
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Tl::smem)) != cudaSuccess) return e;
    kern<<<static_cast<unsigned>(p.BH * p.n), Tl::kThreads, Tl::smem, a.stream>>>(p.maps.dy, g);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if (p.dqh) {
        const long long inner = static_cast<long long>(a.T) * a.Dk, total = static_cast<long long>(a.B) * a.Hk * inner;
        const dim3 grid(static_cast<unsigned>((total + 255) / 256), 2);
        group_sum_kernel<<<grid, 256, 0, a.stream>>>(p.dqh, p.dkh, static_cast<TIn*>(a.dq), static_cast<TIn*>(a.dk), a.H / a.Hk, inner,
                                                     total);
        e = cudaGetLastError();
    }
    return e;
}

template <int DKP>
cudaError_t backward_width(const Plan& p, const Args& a) {
    if (a.dtype == LA_F32) return backward_typed<DKP, 3, 3, float>(p, a);
    if constexpr (DKP > kNarrowKeys)
        if (operand_planes(a, true) == 2) return backward_typed<DKP, 1, 2, __nv_bfloat16>(p, a);
    return backward_typed<DKP, 1, 3, __nv_bfloat16>(p, a);
}

}  // namespace
}  // namespace delta
}  // namespace la
