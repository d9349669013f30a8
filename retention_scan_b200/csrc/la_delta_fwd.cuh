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
// One block per (b, h, chunk): the decays, P, and E = (I + N)^-1, N = A diag(beta)
// strictly lower triangular, in blocks of 16:
//   E_jj by forward substitution in fp32 (a thread per column),
//   E_ij = -E_ii sum_{j <= k < i} N_ik E_kj  on tensor cores: warp j keeps block
//   column j transposed in its accumulators, as the scans keep the state, with as
//   many planes an operand as the record keeps of E.
// Independent of the state, so every chunk runs at once.  Bound by the latency of
// these steps with five blocks an SM.  A substitution of the whole 64 x 64 matrix
// by one thread a column was bound by fetching its 2700 unrolled instructions for
// two warps (766 us at B1 H32 T65536 D128); K and Q by cp.async spent 5000 of a
// block's 17 800 cycles on addresses (531 us); now 350 to 369 us.
constexpr int kPrepThreads = 128;
constexpr int kBS = 24;                // row stride of a 16 x 16 bf16 block: ldmatrix without bank conflicts
constexpr int kBlock = 16 * kBS;       // elements of such a block

// The blocks of N below the diagonal: (1,0), (2,0), (2,1), (3,0), ...
__host__ __device__ constexpr int low_block(int i, int k) { return i * (i - 1) / 2 + k; }

template <int DKP, int NI, int NM, int NP>
struct PrepTiles {
    static constexpr int kPanels = (DKP + 63) / 64, kTile = kPanels * 8192;
    static constexpr int kt = 0;                                  // K, Q tiles (64-column panels); then, over them,
    static constexpr int qt = kt + NI * kTile;
    static constexpr int rec = 0;                                 // the record, as it leaves,
    static constexpr int np = rec + (NM + NP) * kSq + 4 * kTail;  // [NM planes][6 blocks] of N below the diagonal,
    static constexpr int own = np + 2 * NM * 6 * kBlock;          // and per warp its diagonal block of N (fp32 [16][20]),
    static constexpr int kOwn = 2 * NM * kBlock;                  // then over it the planes of E_ii
    static_assert(kOwn >= 4 * 16 * 20, "a diagonal block has to fit its planes' place");
    static constexpr int end_a = qt + NI * kTile, end_b = own + 4 * kOwn;
    static constexpr int L = end_a > end_b ? end_a : end_b;       // float2: log2 of the decays' prefix, high and low part
    static constexpr int bt = L + 8 * C;                          // beta
    static constexpr int bar = bt + 4 * C;
    static constexpr int bytes = bar + 16 + 1024;                 // and the base's alignment
};

// NP: P's planes with a tile of their own, all NM of them or (NM = 2) one, the other folded.
template <int DKP, int NI, int NM, int NP>
__global__ void __launch_bounds__(kPrepThreads) prep_kernel(const __grid_constant__ CUtensorMap mk,
                                                            const __grid_constant__ CUtensorMap mq,
                                                            const float* __restrict__ beta, const float* __restrict__ log_g,
                                                            int decay_kind, float scale, int H, int Hk, int planes_apart,
                                                            int T, int n, unsigned char* __restrict__ records, int* err) {
    static_assert(NP == NM || (NP == 1 && NM == 2), "one plane fits above the diagonals");
    using Tl = PrepTiles<DKP, NI, NM, NP>;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t base = (smem_addr(smem_raw) + 1023) & ~1023u;
    unsigned char* smem = smem_raw + (base - smem_addr(smem_raw));
    float2* L = reinterpret_cast<float2*>(smem + Tl::L);
    float* bt = reinterpret_cast<float*>(smem + Tl::bt);
    unsigned char* rec = smem + Tl::rec;
    __nv_bfloat16* np = reinterpret_cast<__nv_bfloat16*>(smem + Tl::np);
    __nv_bfloat16* tp = reinterpret_cast<__nv_bfloat16*>(smem + Tl::own);  // [4 warps][NM planes]
    uint64_t* bar = reinterpret_cast<uint64_t*>(smem + Tl::bar);

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int bh = blockIdx.x / n, chunk = blockIdx.x % n, t0 = chunk * C;
    const int b = bh / H, h = bh % H;
    if (tid == 32) {
        const int hk = b * Hk + h / (H / Hk);
        mbar_init(bar, 1);
        fence_barrier_init();
        fence_async_smem();
        mbar_arrive_expect_tx(bar, 2 * NI * Tl::kTile);
        for (int p = 0; p < NI; ++p)
            for (int i = 0; i < Tl::kPanels; ++i) {
                tma_load(base + Tl::kt + p * Tl::kTile + 8192 * i, &mk, bar, 64 * i, t0, hk + p * planes_apart);
                tma_load(base + Tl::qt + p * Tl::kTile + 8192 * i, &mq, bar, 64 * i, t0, hk + p * planes_apart);
            }
    }
    float* diag = reinterpret_cast<float*>(smem + Tl::own + warp * Tl::kOwn);
    if (warp == 0) decay_prefix(L, lane, log_g, decay_kind, h, bh, t0, T);
    if (tid >= C) {
        const int t = t0 + tid - C;
        bt[tid - C] = t < T ? beta[static_cast<long long>(bh) * T + t] : 0.f;
    }
    __syncthreads();
    // every thread waits for the copies; a block whose copies do not land in time leaves its record as it was
    const bool landed = mbar_wait_bounded(bar, 0, kWaitLimitNs);
    if (!__syncthreads_and(landed)) {
        if (tid == 0 && err) atomicCAS(err, 0, kErrTmaWait);
        return;
    }

    // K K^T and Q K^T on and below the diagonal: warp w holds rows 16 w .. 16 w + 15
    const LaneOffsets oc = swz_cols(lane), orow = swz_rows(lane);
    float kk[8][4] = {}, qk[8][4] = {};
#pragma unroll
    for (int d = 0; d < DKP / 16; ++d) {
        uint32_t ak[NI][4], aq[NI][4];
#pragma unroll
        for (int p = 0; p < NI; ++p) {
            ldsm4(ak[p], base + Tl::kt + p * Tl::kTile + 8192 * (d / 4) + 2048 * warp + orow.o[d % 4]);
            ldsm4(aq[p], base + Tl::qt + p * Tl::kTile + 8192 * (d / 4) + 2048 * warp + orow.o[d % 4]);
        }
#pragma unroll
        for (int nn = 0; nn < 4; ++nn)
            if (nn <= warp) {
#pragma unroll
                for (int p = 0; p < NI; ++p) {
                    uint32_t bk[4];
                    ldsm4(bk, base + Tl::kt + p * Tl::kTile + 8192 * (d / 4) + 2048 * nn + oc.o[d % 4]);
                    mma_planes<NI, NM>(kk[2 * nn], kk[2 * nn + 1], ak, p, bk);
                    mma_planes<NI, NM>(qk[2 * nn], qk[2 * nn + 1], aq, p, bk);
                }
            }
    }
    __syncthreads();  // the tiles' space becomes N's

    if (tid < C) {
        float* tk = reinterpret_cast<float*>(rec + (NM + NP) * kSq);
        tk[tid] = decay_between(L[tid], make_float2(0.f, 0.f));
        tk[C + tid] = decay_between(L[C - 1], L[tid]);
        tk[2 * C + tid] = bt[tid];
        reinterpret_cast<float2*>(tk + kTok)[tid] = L[tid];
    }
    const int g = lane >> 2, tq = (lane & 3) * 2;
    const float2 lt[2] = {L[16 * warp + g], L[16 * warp + g + 8]};
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j / 2 <= warp) {
            const int s = 8 * j + tq;
            const float4 ls = *reinterpret_cast<const float4*>(L + s);
            const float2 bs = *reinterpret_cast<const float2*>(bt + s);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int t = 16 * warp + g + 8 * r;
                float d0 = decay_between(lt[r], make_float2(ls.x, ls.y)), d1 = decay_between(lt[r], make_float2(ls.z, ls.w));
                float p0 = scale * d0 * qk[j][2 * r], p1 = scale * d1 * qk[j][2 * r + 1];
                float x = d0 * kk[j][2 * r] * bs.x, y = d1 * kk[j][2 * r + 1] * bs.y;
                if (j / 2 == warp) {  // masked entries are zero whatever the scores are there
                    p0 = s <= t ? p0 : 0.f;
                    p1 = s + 1 <= t ? p1 : 0.f;
                    x = s < t ? x : 0.f;
                    y = s + 1 < t ? y : 0.f;
                    *reinterpret_cast<float2*>(diag + (t & 15) * 20 + (s & 15)) = make_float2(x, y);
                } else {
                    uint32_t m[NM];
                    split2<NM>(x, y, m);
#pragma unroll
                    for (int i = 0; i < NM; ++i)
                        *reinterpret_cast<uint32_t*>(np + (i * 6 + low_block(warp, j / 2)) * kBlock + (t & 15) * kBS + (s & 15)) = m[i];
                }
                uint32_t p[NM];
                split2<NM>(p0, p1, p);
#pragma unroll
                for (int i = 0; i < NP; ++i) *reinterpret_cast<uint32_t*>(rec + (NM + i) * kSq + swz64(t, s)) = p[i];
                if constexpr (NP < NM) {
                    const int col = 16 * fold_col(warp, j / 2) + (s & 15);
                    *reinterpret_cast<uint32_t*>(rec + fold_band(NM, warp, j / 2) + swz64(t & 15, col)) = p[NP];
                }
            }
        }
    __syncwarp();

    if (lane < 16) {  // the diagonal block of this warp's rows: lane = column
        float x[16];
#pragma unroll
        for (int t = 0; t < 16; ++t) {
            float a0 = t == lane ? 1.f : 0.f, a1 = 0.f;
#pragma unroll
            for (int s = 0; s < t; s += 2) {
                const float2 m = *reinterpret_cast<const float2*>(diag + t * 20 + s);
                a0 = fmaf(-m.x, x[s], a0);
                if (s + 1 < t) a1 = fmaf(-m.y, x[s + 1], a1);
            }
            x[t] = a0 + a1;
        }
        __syncwarp(0xffffu);  // the block's columns are all read
#pragma unroll
        for (int t = 0; t < 16; ++t) {
            uint32_t p[NM];
            split2<NM>(x[t], 0.f, p);
#pragma unroll
            for (int i = 0; i < NM; ++i) {
                const unsigned short u = static_cast<unsigned short>(p[i]);
                *reinterpret_cast<unsigned short*>(tp + (warp * NM + i) * kBlock + t * kBS + lane) = u;
                *reinterpret_cast<unsigned short*>(rec + i * kSq + swz64(16 * warp + t, 16 * warp + lane)) = u;
            }
        }
    }
    __syncthreads();

    // Block column `warp` of E below the diagonal, transposed: col[i] = E_ij^T as A operand planes.
    if (warp < 3) {
        uint32_t col[4][NM][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i == warp) {
#pragma unroll
                for (int p = 0; p < NM; ++p) ldsm4t(col[i][p], smem_addr(tp + (i * NM + p) * kBlock + off_cols(lane, kBS)));
            }
#pragma unroll
        for (int i = 1; i < 4; ++i)
            if (i > warp) {
                float acc[2][4] = {};
#pragma unroll
                for (int m = 0; m < i; ++m)
                    if (m >= warp) {
#pragma unroll
                        for (int p = 0; p < NM; ++p) {
                            uint32_t r[4];
                            ldsm4(r, smem_addr(np + (p * 6 + low_block(i, m)) * kBlock + off_cols(lane, kBS)));
                            mma_planes<NM, NM>(acc[0], acc[1], col[m], p, r);
                        }
                    }
                uint32_t a[NM][4];
                split_frag<NM>(acc[0], acc[1], a);
                float e[2][4] = {};
#pragma unroll
                for (int p = 0; p < NM; ++p) {
                    uint32_t r[4];
                    ldsm4(r, smem_addr(tp + (i * NM + p) * kBlock + off_cols(lane, kBS)));
                    mma_planes<NM, NM>(e[0], e[1], a, p, r);
                }
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int y = 0; y < 4; ++y) e[x][y] = -e[x][y];
                split_frag<NM>(e[0], e[1], col[i]);
#pragma unroll
                for (int p = 0; p < NM; ++p)
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        // registers: rows (columns of E) 8 (y & 1) .., tokens 8 (y >> 1) ..
                        const uint32_t u = mov_trans(col[i][p][y]);
                        *reinterpret_cast<uint32_t*>(rec + p * kSq + swz64(16 * i + 8 * (y >> 1) + g, 16 * warp + 8 * (y & 1) + tq)) = u;
                    }
            }
    }
    // Above the diagonal, where no plane is folded, the record keeps what shared memory held: no scan reads there.
    fence_async_smem();
    __syncthreads();
    constexpr long long kRec = record_bytes(NM + NP);
    if (tid == 0) bulk_store(records + static_cast<long long>(blockIdx.x) * kRec, smem_addr(rec), static_cast<uint32_t>(kRec));
}

// ---------------------------------------------------------------- scan
// One warp per 16 value columns of a (b, h); the block's warps share the
// chunk's K, Q and record, which TMA brings in up to three chunks ahead.  Warps
// meet only at the stages' barriers and run apart by up to a stage, so that
// one's loads and splits fill another's waits.
// kOut: 1 = outputs y, 0 = the backward's recomputation: the incoming state
// and the errors E of every chunk, as bf16 planes.
// Bound by the tensor core's rate for mma.sync: 504 instructions a warp and chunk
// at D128 (bf16), 8 cycles each on a scheduler, 8 060 cycles a chunk with eight warps
// an SM (9 300 measured; B8 H16 T4096: 402 us by itself, cold).
template <int DKP, int NI, int NM, int NP, int NW, bool kOut, typename TIn>
__global__ void __launch_bounds__(32 * NW) scan_kernel(const __grid_constant__ CUtensorMap mk,
                                                             const __grid_constant__ CUtensorMap mq,
                                                             const __grid_constant__ CUtensorMap mv, ScanArgs a) {
    constexpr bool kF32 = sizeof(TIn) == 4;
    using Tl = ScanTiles<DKP, NI, kOut ? NM + NP : NM, NW, kOut, !kF32>;
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

    Feed<Tl, NI, kOut, !kF32> feed;
    feed.mk = &mk;
    feed.mq = &mq;
    feed.mv = &mv;
    feed.rec_bytes = record_bytes(NM + NP);
    feed.records = a.records + static_cast<long long>(bh) * a.n * feed.rec_bytes;
    feed.rec_used = (kOut ? NM + NP : NM) * kSq;
    feed.hk = b * a.Hk + h / (a.H / a.Hk);
    feed.planes_apart = a.planes_apart;
    feed.bh = bh;
    feed.v0 = vb;
    feed.nv = nv;
    feed.warps = nv;
    start_ring<Tl>(feed, base, ring, a.n, 0, 1);
    if (warp >= nv) return;

    const TIn* vsrc = static_cast<const TIn*>(a.v) + static_cast<long long>(bh) * a.T * a.Dv;
    const int tq = (lane & 3) * 2;
    const LaneOffsets oc = swz_cols(lane), orow = swz_rows(lane);
    float S[DKP / 8][4];
    state_load<DKP>(S, a.init_state ? a.init_state + static_cast<long long>(bh) * a.Dk * a.Dv : nullptr, a.Dk, a.Dv, v0, lane);

    for (int c = 0; c < a.n; ++c) {
        const int stage = c % kS;
        if (!wait_stage(ring, stage, c / kS, a.err)) return;
        const uint32_t st = base + stage * Tl::bytes;
        const uint32_t kt = st + Tl::k, qt = st + Tl::q, et = st + Tl::rec, pt = et + NM * kSq;
        const float* gam = reinterpret_cast<const float*>(smem + stage * Tl::bytes + Tl::tok);
        const float* rest = gam + C;
        const float* beta = gam + 2 * C;
        const long long cid = static_cast<long long>(bh) * a.n + c;

        // X = (K S)^T, Y = (Q S)^T
        float X[8][4] = {}, Y[8][4] = {};
#pragma unroll
        for (int d = 0; d < DKP / 16; ++d) {
            uint32_t s[NM][4];
            split_frag<NM>(S[2 * d], S[2 * d + 1], s);
            if constexpr (!kOut)
                put_tiles<NM>(s, a.Sst + cid * NM * a.DVP * DKP, v0 / 16, DKP / 16, d, lane);
#pragma unroll
            for (int nn = 0; nn < 4; ++nn)
#pragma unroll
                for (int p = 0; p < NI; ++p) {
                    uint32_t r[4];
                    ldsm4(r, kt + p * Tl::kTile + 8192 * (d / 4) + 2048 * nn + oc.o[d % 4]);
                    mma_planes<NM, NM>(X[2 * nn], X[2 * nn + 1], s, p, r);
                    if constexpr (kOut) {
                        ldsm4(r, qt + p * Tl::kTile + 8192 * (d / 4) + 2048 * nn + oc.o[d % 4]);
                        mma_planes<NM, NM>(Y[2 * nn], Y[2 * nn + 1], s, p, r);
                    }
                }
        }
        // R = V - e^L (K S); E = (I + A diag(beta))^-1 R
        float R[8][4];
        if constexpr (kF32)
            values_from_global(R, vsrc, c * C, a.T, a.Dv, v0, lane);
        else
            values_from_tile(R, st + Tl::v + 2048 * warp, lane);
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
                    ldsm4(e, et + p * kSq + 2048 * nn + oc.o[m]);
                    mma_planes<NM, NM>(X[2 * nn], X[2 * nn + 1], r, p, e);
                }
        }
        if constexpr (!kOut) {
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                uint32_t e[NM][4];
                split_frag<NM>(X[2 * m], X[2 * m + 1], e);
                put_tiles<NM>(e, a.Est + cid * NM * a.DVP * C, v0 / 16, C / 16, m, lane);
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
                    for (int p = 0; p < NM; ++p) {
                        uint32_t r[4];
                        ldsm4(r, p < NP ? pt + p * kSq + 2048 * nn + oc.o[m] : et + fold_band(NM, nn, m) + oc.o[fold_col(nn, m)]);
                        mma_planes<NM, NM>(Y[2 * nn], Y[2 * nn + 1], u, p, r);
                    }
            }
            values_to_global(Y, static_cast<TIn*>(a.out) + static_cast<long long>(bh) * a.T * a.Dv, c * C, a.T, a.Dv, v0, lane);
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
                    ldsm4t(r, kt + p * Tl::kTile + 8192 * (d / 4) + 2048 * m + orow.o[d % 4]);
                    mma_planes<NM, NM>(acc[0], acc[1], w[m], p, r);
                }
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) S[2 * d + j][i] = fmaf(total, S[2 * d + j][i], acc[j][i]);
        }
        release_stage<Tl>(feed, base, ring, stage, c + kS < a.n ? c + kS : -1);
    }
    if (a.final_state)
        state_store<DKP>(S, a.final_state + static_cast<long long>(bh) * a.Dk * a.Dv, a.Dk, a.Dv, v0, lane);
}

// The same scan with G warps a slice (la_delta.cuh), for few (b, h): NS slices a
// block and a warp that feeds the stages.  Per chunk and slice three barriers:
// the state's parts, the right-hand sides R, and U are exchanged.  At B1 H32
// T65536 D128 (256 slices): one warp a slice 3.3 us a chunk, two 2.3 us.
template <int DKP, int NM, int G>
struct GroupSpace {  // a slice's exchange, in 16-byte words
    static constexpr int kSteps = DKP / 16 / G;       // k-steps of a warp's part of the key width
    static constexpr int kBlocks = 4 / G;             // token blocks of a warp
    static constexpr int s = 0;                       // [DKP / 16][NM][32]
    static constexpr int r = s + DKP / 16 * NM * 32;  // [4][NM][32], by token block
    static constexpr int u = r + 4 * NM * 32;
    static constexpr int w = u + 4 * NM * 32;
    static constexpr int words = w + 4 * NM * 32;
};

template <int DKP, int NI, int NM, int NP, int G, int NS, bool kOut, typename TIn>
__global__ void __launch_bounds__(32 * G * NS + 32) group_scan_kernel(const __grid_constant__ CUtensorMap mk,
                                                                      const __grid_constant__ CUtensorMap mq,
                                                                      const __grid_constant__ CUtensorMap mv, ScanArgs a) {
    constexpr bool kF32 = sizeof(TIn) == 4;
    using Ex = GroupSpace<DKP, NM, G>;
    using Tl = ScanTiles<DKP, NI, kOut ? NM + NP : NM, NS, kOut, !kF32, 16 * Ex::words * NS>;
    constexpr int kS = Tl::stages, kSteps = Ex::kSteps, kBlocks = Ex::kBlocks, kCols = DKP / G;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t base = (smem_addr(smem_raw) + 1023) & ~1023u;
    unsigned char* smem = smem_raw + (base - smem_addr(smem_raw));
    FedRing<kS>* fed = reinterpret_cast<FedRing<kS>*>(smem + kS * Tl::bytes);
    Ring<kS>* ring = &fed->ring;
    const int tid = threadIdx.x, lane = tid & 31, slice = tid / (32 * G);
    uint4* ex = reinterpret_cast<uint4*>(smem + Tl::extra) + slice * Ex::words;
    const int bh = blockIdx.x / a.vblocks;
    const int vb = blockIdx.x % a.vblocks * 16 * NS, v0 = vb + 16 * slice;
    const int nv = min(NS, (a.Dv - vb + 15) / 16);
    const int b = bh / a.H, h = bh % a.H;
    Feed<Tl, NI, kOut, !kF32> feed;
    feed.mk = &mk;
    feed.mq = &mq;
    feed.mv = &mv;
    feed.rec_bytes = record_bytes(NM + NP);
    feed.records = a.records + static_cast<long long>(bh) * a.n * feed.rec_bytes;
    feed.rec_used = (kOut ? NM + NP : NM) * kSq;
    feed.hk = b * a.Hk + h / (a.H / a.Hk);
    feed.planes_apart = a.planes_apart;
    feed.bh = bh;
    feed.v0 = vb;
    feed.nv = nv;
    feed.warps = G * nv;
    init_fed<Tl>(feed, fed);
    if (slice == NS) {
        if (tid == 32 * G * NS) feed_ring<Tl>(feed, base, fed, a.n, 0, 1, a.err);
        return;
    }
    if (slice >= nv) return;

    const TIn* vsrc = static_cast<const TIn*>(a.v) + static_cast<long long>(bh) * a.T * a.Dv;
    const int tq = (lane & 3) * 2;
    const LaneOffsets oc = swz_cols(lane), orow = swz_rows(lane);
    // two warps a slice: a body for each, whose block indices are constants (2258 us at the
    // size above against 2530, with P in one plane; 2343 with its second); four run one body (four would not fit the instruction cache)
    auto scan = [&](auto which) {
    const int w = which;
    float S[kCols / 8][4];
    state_load<kCols>(S, a.init_state ? a.init_state + static_cast<long long>(bh) * a.Dk * a.Dv : nullptr, a.Dk, a.Dv, v0, lane,
                      w * kCols);
    uint32_t so[kSteps][NM][4];  // this part's planes for the chunk that comes
#pragma unroll
    for (int d = 0; d < kSteps; ++d) {
        split_frag<NM>(S[2 * d], S[2 * d + 1], so[d]);
        put_planes<NM>(ex + Ex::s + (w * kSteps + d) * NM * 32, lane, so[d]);
    }

    for (int c = 0; c < a.n; ++c) {
        const int stage = c % kS;
        [[maybe_unused]] const long long cid = static_cast<long long>(bh) * a.n + c;
        if (!group_agree<G>(slice, wait_stage(ring, stage, c / kS, a.err))) return;
        const uint32_t st = base + stage * Tl::bytes;
        const uint32_t kt = st + Tl::k, et = st + Tl::rec;
        [[maybe_unused]] const uint32_t qt = st + Tl::q, pt = et + NM * kSq;
        const float* gam = reinterpret_cast<const float*>(smem + stage * Tl::bytes + Tl::tok);
        const float* rest = gam + C;
        const float* beta = gam + 2 * C;

        if constexpr (!kOut) {
#pragma unroll
            for (int d = 0; d < kSteps; ++d)
                put_tiles<NM>(so[d], a.Sst + cid * NM * a.DVP * DKP, v0 / 16, DKP / 16, w * kSteps + d, lane);
        }
        [[maybe_unused]] float early[kF32 ? kBlocks : 1][2][4];  // fp32 values come from global memory: their latency passes under the products
        if constexpr (kF32) {
#pragma unroll
            for (int j = 0; j < kBlocks; ++j)
                block_from_global(early[j], vsrc, c * C + 16 * own_block<G>(w, j), a.T, a.Dv, v0, lane);
        }
        // (K S)^T or (Q S)^T for this warp's tokens: its own part of S, then the others'
        auto through_state = [&](float (&acc)[kBlocks][2][4], uint32_t tile) {
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
                            for (int i = 0; i < 4; ++i) s[p][i] = so[d][p][i];
                    }
#pragma unroll
                    for (int j = 0; j < kBlocks; ++j)
#pragma unroll
                        for (int p = 0; p < NI; ++p) {
                            uint32_t r[4];
                            ldsm4(r, tile + p * Tl::kTile + 2048 * own_block<G>(w, j) + step_offset<DKP, G>(oc, x, d));
                            mma_planes<NM, NM>(acc[j][0], acc[j][1], s, p, r);
                        }
                }
            }
        };
        // acc += (lower triangular matrix) x (exchanged blocks at and before each of this warp's);
        // whole: its planes with a tile of their own
        auto through_blocks = [&](float (&acc)[kBlocks][2][4], uint32_t mat, int whole, const uint4* from,
                                  const uint32_t (&mine)[kBlocks][NM][4]) {
#pragma unroll
            for (int o = 0; o < G; ++o)
#pragma unroll
                for (int jm = 0; jm < kBlocks; ++jm) {
                    const int m = own_block<G>((w + o) % G, jm);
                    uint32_t r[NM][4];
                    if (o) {
                        get_planes<NM>(from + m * NM * 32, lane, r);
                    } else {
#pragma unroll
                        for (int p = 0; p < NM; ++p)
#pragma unroll
                            for (int i = 0; i < 4; ++i) r[p][i] = mine[jm][p][i];
                    }
#pragma unroll
                    for (int j = 0; j < kBlocks; ++j) {
                        const int blk = own_block<G>(w, j);
                        if (m <= blk) {
#pragma unroll
                            for (int p = 0; p < NM; ++p) {
                                uint32_t e[4];
                                ldsm4(e, p < whole ? mat + p * kSq + 2048 * blk + (oc.o[0] ^ (m << 5))
                                                   : et + fold_band(NM, blk, m) + (oc.o[0] ^ (fold_col(blk, m) << 5)));
                                mma_planes<NM, NM>(acc[j][0], acc[j][1], r, p, e);
                            }
                        }
                    }
                }
        };
        float X[kBlocks][2][4] = {};
        [[maybe_unused]] float Y[kBlocks][2][4] = {};
        through_state(X, kt);
        // R = V - e^L (K S), exchanged
        uint32_t ro[kBlocks][NM][4];
#pragma unroll
        for (int j = 0; j < kBlocks; ++j) {
            const int blk = own_block<G>(w, j);
            float R[2][4];
            if constexpr (kF32) {
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int i = 0; i < 4; ++i) R[x][i] = early[j][x][i];
            } else {
                block_from_tile(R, st + Tl::v + 2048 * slice, blk, lane);
            }
            block_scale(X[j], gam, blk, tq);
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    R[x][i] -= X[j][x][i];
                    X[j][x][i] = 0.f;
                }
            split_frag<NM>(R[0], R[1], ro[j]);
            put_planes<NM>(ex + Ex::r + blk * NM * 32, lane, ro[j]);
        }
        group_sync<G>(slice);
        // E for this warp's tokens: the blocks of (I + A diag(beta))^-1 R at and before each
        through_blocks(X, et, NM, ex + Ex::r, ro);
        // Q S is not on the way to the next state: its products fill the waits around E and U
        if constexpr (kOut) through_state(Y, qt);
        // U = diag(beta) E, and diag(e^(L_C - L)) U for the state, exchanged
        uint32_t uo[kBlocks][NM][4], wo[kBlocks][NM][4];
#pragma unroll
        for (int j = 0; j < kBlocks; ++j) {
            const int blk = own_block<G>(w, j);
            if constexpr (!kOut) {
                split_frag<NM>(X[j][0], X[j][1], uo[j]);
                put_tiles<NM>(uo[j], a.Est + cid * NM * a.DVP * C, v0 / 16, C / 16, blk, lane);
            }
            block_scale(X[j], beta, blk, tq);
            if constexpr (kOut) {
                split_frag<NM>(X[j][0], X[j][1], uo[j]);
                put_planes<NM>(ex + Ex::u + blk * NM * 32, lane, uo[j]);
            }
            block_scale(X[j], rest, blk, tq);
            split_frag<NM>(X[j][0], X[j][1], wo[j]);
            put_planes<NM>(ex + Ex::w + blk * NM * 32, lane, wo[j]);
        }
        group_sync<G>(slice);
        // This warp's part of S <- e^(L_C) S + K^T diag(e^(L_C - L)) U, and its planes for
        // the next chunk (the others read this chunk's before the last barrier)
        uint32_t wp[4 - kBlocks][NM][4];
#pragma unroll
        for (int o = 1; o < G; ++o)
#pragma unroll
            for (int j = 0; j < kBlocks; ++j)
                get_planes<NM>(ex + Ex::w + own_block<G>((w + o) % G, j) * NM * 32, lane, wp[(o - 1) * kBlocks + j]);
        const float total = gam[C - 1];
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
                for (int i = 0; i < 4; ++i) S[2 * d + j][i] = fmaf(total, S[2 * d + j][i], acc[j][i]);
            split_frag<NM>(S[2 * d], S[2 * d + 1], so[d]);
            put_planes<NM>(ex + Ex::s + (w * kSteps + d) * NM * 32, lane, so[d]);
        }
        if constexpr (kOut) {
#pragma unroll
            for (int j = 0; j < kBlocks; ++j) block_scale(Y[j], gam, own_block<G>(w, j), tq, a.scale);
            through_blocks(Y, pt, NP, ex + Ex::u, uo);
            TIn* out = static_cast<TIn*>(a.out) + static_cast<long long>(bh) * a.T * a.Dv;
#pragma unroll
            for (int j = 0; j < kBlocks; ++j) block_to_global(Y[j], out, c * C + 16 * own_block<G>(w, j), a.T, a.Dv, v0, lane);
        }
        release_fed(&fed->empty[stage]);
    }
    if (a.final_state)
        state_store<kCols>(S, a.final_state + static_cast<long long>(bh) * a.Dk * a.Dv, a.Dk, a.Dv, v0, lane, w * kCols);
    };
    const int w = (tid >> 5) % G;
    if constexpr (G == 2) {
        if (w)
            scan(std::integral_constant<int, 1>{});
        else
            scan(std::integral_constant<int, 0>{});
    } else {
        scan(w);
    }
}

template <typename K>
cudaError_t allow_smem(K kernel, size_t bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
}

template <int DKP, int NI, int NM, int NP>
cudaError_t prep_run(const Plan& p, const Args& a) {
    auto kern = prep_kernel<DKP, NI, NM, NP>;
    constexpr int smem = PrepTiles<DKP, NI, NM, NP>::bytes;
    cudaError_t e = allow_smem(kern, smem);
    if (e != cudaSuccess) return e;
    kern<<<static_cast<unsigned>(p.BH * p.n), kPrepThreads, smem, a.stream>>>(p.maps.k, p.maps.q, a.beta, a.log_g, a.decay_kind, a.scale,
                                                                             a.H, a.Hk, a.B * a.Hk, a.T, p.n, p.records,
                                                                             p.err);
    return cudaGetLastError();
}

template <int DKP, int NI, int NM, int NP, int NW, bool kOut, typename TIn>
cudaError_t scan_run(const Plan& p, const Args& a) {
    auto kern = scan_kernel<DKP, NI, NM, NP, NW, kOut, TIn>;
    using Tl = ScanTiles<DKP, NI, kOut ? NM + NP : NM, NW, kOut, sizeof(TIn) == 2>;
    cudaError_t e = allow_smem(kern, Tl::smem);
    if (e != cudaSuccess) return e;
    ScanArgs s = scan_args(p, a);
    s.vblocks = (a.Dv + 16 * NW - 1) / (16 * NW);
    kern<<<static_cast<unsigned>(p.BH * s.vblocks), 32 * NW, Tl::smem, a.stream>>>(p.maps.k, p.maps.q, p.maps.v, s);
    return cudaGetLastError();
}

template <int DKP, int NI, int NM, int NP, int G, int NS, bool kOut, typename TIn>
cudaError_t group_scan_run(const Plan& p, const Args& a) {
    auto kern = group_scan_kernel<DKP, NI, NM, NP, G, NS, kOut, TIn>;
    using Tl = ScanTiles<DKP, NI, kOut ? NM + NP : NM, NS, kOut, sizeof(TIn) == 2, 16 * GroupSpace<DKP, NM, G>::words * NS>;
    cudaError_t e = allow_smem(kern, Tl::smem);
    if (e != cudaSuccess) return e;
    ScanArgs s = scan_args(p, a);
    s.vblocks = (a.Dv + 16 * NS - 1) / (16 * NS);
    kern<<<static_cast<unsigned>(p.BH * s.vblocks), 32 * G * NS + 32, Tl::smem, a.stream>>>(p.maps.k, p.maps.q, p.maps.v, s);
    return cudaGetLastError();
}

template <int DKP, int NI, int NM, int NP, bool kOut, typename TIn>
cudaError_t scan_widths(const Plan& p, const Args& a) {
    constexpr int G = DKP >= 64 ? 4 : 2;  // each warp needs a 16-column step of the key width
    if (p.group)
        return p.warps == 1 ? group_scan_run<DKP, NI, NM, NP, G, 1, kOut, TIn>(p, a) : group_scan_run<DKP, NI, NM, NP, 2, 2, kOut, TIn>(p, a);
    switch (p.warps) {
        case 1: return scan_run<DKP, NI, NM, NP, 1, kOut, TIn>(p, a);
        case 2: return scan_run<DKP, NI, NM, NP, 2, kOut, TIn>(p, a);
        case 4: return scan_run<DKP, NI, NM, NP, 4, kOut, TIn>(p, a);
        default: return scan_run<DKP, NI, NM, NP, 8, kOut, TIn>(p, a);
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
        if ((e = prep_run<DKP, 3, 3, 3>(p, a)) != cudaSuccess) return e;
        return outputs ? scan_widths<DKP, 3, 3, 3, true, float>(p, a) : scan_widths<DKP, 3, 3, 3, false, float>(p, a);
    }
    if (outputs) {
        // P's second plane is folded.  Without it (P rounded to bf16) y was off by 2^-9 of each term of P U,
        // which keys and queries close to one another make several times y: 0.007 to 0.013 of it
        if ((e = prep_run<DKP, 1, 2, 1>(p, a)) != cudaSuccess) return e;
        return scan_widths<DKP, 1, 2, 1, true, __nv_bfloat16>(p, a);
    }
    if constexpr (DKP > kNarrowKeys) {
        if (operand_planes(a, true) == 2) {
            if ((e = prep_run<DKP, 1, 2, 2>(p, a)) != cudaSuccess) return e;
            return scan_widths<DKP, 1, 2, 2, false, __nv_bfloat16>(p, a);
        }
    }
    if ((e = prep_run<DKP, 1, 3, 3>(p, a)) != cudaSuccess) return e;
    return scan_widths<DKP, 1, 3, 3, false, __nv_bfloat16>(p, a);
}

}  // namespace
}  // namespace delta
}  // namespace la
