// la_delta.cuh - the gated delta rule's device code shared by its kernels.
//
//   S'  = g_t S_{t-1}                 e_t = v_t - S'^T k_t
//   S_t = S' + k_t (beta_t e_t)^T     y_t = scale * S_t^T q_t
//
// Chunked form (C = 64 tokens, L_t the chunk's inclusive prefix of log g,
// S the state before the chunk, A_ts = e^(L_t - L_s) k_t.k_s for s < t):
//
//   E = (I + A diag(beta))^-1 (V - diag(e^L) K S)        U = diag(beta) E
//   Y = scale diag(e^L) Q S + P U,  P_ts = scale e^(L_t - L_s) q_t.k_s, s <= t
//   S <- e^(L_C) S + (diag(e^(L_C - L)) K)^T U
//
// beta scales the columns of A, not its rows, so that E needs no division and
// a token with beta = 0 (padding) still has its error e_t for the gradient.
//
// The state's Dv columns never mix, so one warp owns 16 of them and carries
// S^T (16 x Dk, fp32) in the accumulator registers of mma.m16n8k16: the
// accumulator of one product has the register layout of the next product's A
// operand, and the whole chain S -> K S -> E -> U -> S runs without shared
// memory, shuffles or block barriers between the products.  Only K, Q, P and
// (I + A diag(beta))^-1 come through shared memory, as B operands, and are
// shared by the block's warps.
//
// Precision: the tensor core takes bf16.  An fp32 operand x is passed as
// x = x0 + x1 (+ x2), each x_i the bf16 rounding of what is left, and a product
// of operands with planes i and j is accumulated for i + j < NM: with NM = 2
// a product is within about 2^-16 of fp32's, with NM = 3 within 2^-23.  bf16
// inputs are exact in one plane and run with NM = 2, or 3 where a gradient needs it
// (operand_planes); fp32 inputs take three planes and NM = 3.  Plain bf16 or tf32 operands (2^-9, 2^-12) would leave
// the fp32 state and the fp32 gradients with three digits.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "la_internal.h"
#include "la_sm100.cuh"

namespace la {
namespace delta {

constexpr int C = 64;            // tokens per chunk
constexpr int kPad = 8;          // bf16 padding of a shared-memory row: ldmatrix without bank conflicts
constexpr int kCS = C + kPad;    // row stride of a C-wide tile
constexpr int kTok = 3 * C;      // floats per chunk of per-token factors: e^L, e^(L_C - L), beta
constexpr int kTail = 5 * C;     // and, behind them, the prefix L itself as pairs (decay_prefix)
constexpr int kSq = 2 * C * C;   // bytes of a C x C bf16 plane
constexpr uint64_t kWaitLimitNs = 1000000000ull;  // every barrier wait gives up after this long
constexpr float kLogFloor = -128.f;  // a decay below e^-128 is zero in fp32 next to anything it is added to

// What prep leaves for each chunk: [planes of (I + A diag(beta))^-1][planes of P]
// [kTail floats], the matrices as the 128-byte-row swizzled tiles the scans
// read, so that one bulk copy brings them into shared memory.
constexpr long long record_bytes(int planes) { return static_cast<long long>(planes) * kSq + sizeof(float) * kTail; }

// Both matrices are lower triangular, so their tiles' 16 x 16 blocks above the
// diagonal are free.  The forward of bf16 inputs keeps one tile of P and the second
// plane of P there (a third fewer bytes of P in the record and in a stage): its block
// (i, k), k < i, at (k, i) of P's own tile, its diagonal blocks above the diagonal of
// the first tile.  Byte offset of the block's 16-row band from the record's start,
// and its column block.
__host__ __device__ constexpr int fold_band(int nm, int i, int k) { return k < i ? nm * kSq + 2048 * k : i < 3 ? 0 : 2048; }
__host__ __device__ constexpr int fold_col(int i, int k) { return k < i ? i : i < 3 ? i + 1 : 2; }

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

// Byte offset of (row, col) of a 64-column bf16 tile whose 16-byte pieces are
// swizzled within each 128-byte row (TMA's 128-byte pattern).
__device__ __forceinline__ uint32_t swz64(int row, int col) {
    return row * 128 + ((((col >> 3) ^ row) & 7) << 4) + (col & 7) * 2;
}

// A lane's byte offsets of ldmatrix.x4 on the four 16-column blocks of a
// 16-row band of such a tile; band b, panel p: + 2048 b + 8192 p.  The lane
// orders are those of off_cols and off_rows below.
struct LaneOffsets {
    uint32_t o[4];
};
__device__ __forceinline__ LaneOffsets swz_cols(int lane) {
    const int row = (lane & 7) + ((lane >> 4) << 3), half = (lane >> 3) & 1;
    LaneOffsets r;
#pragma unroll
    for (int j = 0; j < 4; ++j) r.o[j] = row * 128 + (((2 * j + half) ^ (row & 7)) << 4);
    return r;
}
__device__ __forceinline__ LaneOffsets swz_rows(int lane) {
    const int row = lane & 15, half = lane >> 4;
    LaneOffsets r;
#pragma unroll
    for (int j = 0; j < 4; ++j) r.o[j] = row * 128 + (((2 * j + half) ^ (row & 7)) << 4);
    return r;
}

// One box of a 3-D tensor map.
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// Contiguous copy into shared memory (16-byte aligned, a multiple of 16 bytes), completing on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_addr(bar))
                 : "memory");
}
// Contiguous copy out of shared memory; returns once the source may be reused.
__device__ __forceinline__ void bulk_store(void* dst, uint32_t src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(reinterpret_cast<uint64_t>(dst)), "r"(src),
                 "r"(bytes)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint32_t mov_trans(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 16 bytes, or zeros where !valid (src stays a valid address either way).
__device__ __forceinline__ void cp16(void* dst, const void* src, bool valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(valid ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float low_of(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float high_of(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// The bf16 planes of the fp32 pair (x, y): p[i] rounds what planes 0..i-1 left.
template <int N>
__device__ __forceinline__ void split2(float x, float y, uint32_t (&p)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        p[i] = pack(x, y);
        x -= low_of(p[i]);
        y -= high_of(p[i]);
    }
}

// A operand (16 x 16) planes from two neighbouring accumulator tiles.
template <int N>
__device__ __forceinline__ void split_frag(const float (&x)[4], const float (&y)[4], uint32_t (&a)[N][4]) {
    uint32_t t[N];
    split2<N>(x[0], x[1], t);
#pragma unroll
    for (int i = 0; i < N; ++i) a[i][0] = t[i];
    split2<N>(x[2], x[3], t);
#pragma unroll
    for (int i = 0; i < N; ++i) a[i][1] = t[i];
    split2<N>(y[0], y[1], t);
#pragma unroll
    for (int i = 0; i < N; ++i) a[i][2] = t[i];
    split2<N>(y[2], y[3], t);
#pragma unroll
    for (int i = 0; i < N; ++i) a[i][3] = t[i];
}

// Lane addresses of ldmatrix.x4 on a 16 x 16 block of a bf16 tile with
// `stride` elements a row.  One lane order visits the four 8 x 8 matrices
// along the columns first, the other along the rows first:
//   B stored [n][k]: ldsm4 with off_cols;    B stored [k][n]: ldsm4t with off_rows
//   A stored [m][k]: ldsm4 with off_rows;    A stored [k][m]: ldsm4t with off_cols
// B registers 0, 1 are columns n..n+7, registers 2, 3 columns n+8..n+15.
__device__ __forceinline__ int off_cols(int lane, int stride) {
    return ((lane & 7) + ((lane >> 4) << 3)) * stride + ((lane >> 3) & 1) * 8;
}
__device__ __forceinline__ int off_rows(int lane, int stride) { return (lane & 15) * stride + (lane >> 4) * 8; }

// acc[j][:] += A B for the 16-column block of B whose registers are b: A
// planes NA, this B plane's index `pb`; keeps planes with pa + pb < NM.
template <int NA, int NM>
__device__ __forceinline__ void mma_planes(float (&d0)[4], float (&d1)[4], const uint32_t (&a)[NA][4], int pb,
                                           const uint32_t (&b)[4]) {
#pragma unroll
    for (int pa = 0; pa < NA; ++pa)
        if (pa + pb < NM) {
            mma(d0, a[pa], b[0], b[1]);
            mma(d1, a[pa], b[2], b[3]);
        }
}

// q or k as bf16 planes: plane p of head hk, token t starts at
// base + p * plane + hk * head + t * row; rows and cols hold data, the rest of
// a tile is zero.
struct Planes {
    const __nv_bfloat16* base;
    long long plane, head;
    int row, rows, cols;
};

// One C x DKP tile of every plane into shared memory (rows of DKP + kPad).
template <int DKP, int NI>
__device__ __forceinline__ void load_tile(__nv_bfloat16* dst, const Planes& src, long long hk, int t0, int tid, int nthreads) {
    constexpr int kVec = DKP / 8;
#pragma unroll
    for (int p = 0; p < NI; ++p) {
        const __nv_bfloat16* s = src.base + p * src.plane + hk * src.head;
        for (int i = tid; i < C * kVec; i += nthreads) {
            const int r = i / kVec, c = (i % kVec) * 8;
            const bool ok = t0 + r < src.rows && c < src.cols;
            cp16(dst + (p * C + r) * (DKP + kPad) + c, ok ? s + static_cast<long long>(t0 + r) * src.row + c : src.base, ok);
        }
    }
}

// Value-side operand ([B,H,T,Dv], bf16 or fp32) of one chunk, transposed into
// accumulator layout: x[j][0..1] = column v0 + g, tokens 8 j + 2 t', +1;
// x[j][2..3] = column v0 + g + 8 (g = lane / 4, t' = lane % 4).
// bf16: from the warp's shared tile of 16 columns (32-byte rows).
__device__ __forceinline__ void values_from_tile(float (&x)[8][4], uint32_t tile, int lane) {
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        uint32_t r[4];
        ldsm4t(r, tile + 512 * n + (lane & 15) * 32 + (lane >> 4) * 16);
        // r0: tokens 0-7, columns 0-7; r1: tokens 8-15, columns 0-7; r2, r3: columns 8-15
        x[2 * n][0] = low_of(r[0]);
        x[2 * n][1] = high_of(r[0]);
        x[2 * n + 1][0] = low_of(r[1]);
        x[2 * n + 1][1] = high_of(r[1]);
        x[2 * n][2] = low_of(r[2]);
        x[2 * n][3] = high_of(r[2]);
        x[2 * n + 1][2] = low_of(r[3]);
        x[2 * n + 1][3] = high_of(r[3]);
    }
}
// fp32: straight from global memory.
__device__ __forceinline__ void values_from_global(float (&x)[8][4], const float* base, int t0, int T, int Dv, int v0,
                                                   int lane) {
    const int g = lane >> 2, tq = (lane & 3) * 2;
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = t0 + 8 * j + tq + (i & 1), v = v0 + g + (i >> 1) * 8;
            x[j][i] = t < T && v < Dv ? base[static_cast<long long>(t) * Dv + v] : 0.f;
        }
}

// The same layout back to [T, Dv] rows.
__device__ __forceinline__ void values_to_global(const float (&x)[8][4], __nv_bfloat16* base, int t0, int T, int Dv, int v0,
                                                 int lane) {
    const int g = lane >> 2, tq = (lane & 3) * 2;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t lo = mov_trans(pack(x[j][0], x[j][1])), hi = mov_trans(pack(x[j][2], x[j][3]));
        const int t = t0 + 8 * j + g;
        if (t < T) {
            __nv_bfloat16* p = base + static_cast<long long>(t) * Dv + v0 + tq;
            *reinterpret_cast<uint32_t*>(p) = lo;
            *reinterpret_cast<uint32_t*>(p + 8) = hi;
        }
    }
}
__device__ __forceinline__ void values_to_global(const float (&x)[8][4], float* base, int t0, int T, int Dv, int v0,
                                                 int lane) {
    const int g = lane >> 2, tq = (lane & 3) * 2;
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = t0 + 8 * j + tq + (i & 1), v = v0 + g + (i >> 1) * 8;
            if (t < T && v < Dv) base[static_cast<long long>(t) * Dv + v] = x[j][i];
        }
}

// S^T in accumulator tiles (s[j]: columns 8 j .. 8 j + 7 of Dk) from and to a
// [Dk][Dv] fp32 state.
template <int DKP>
__device__ __forceinline__ void state_load(float (&s)[DKP / 8][4], const float* S, int Dk, int Dv, int v0, int lane, int d0 = 0) {
    const int g = lane >> 2, tq = (lane & 3) * 2;
#pragma unroll
    for (int j = 0; j < DKP / 8; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int d = d0 + 8 * j + tq + (i & 1), v = v0 + g + (i >> 1) * 8;
            s[j][i] = S && d < Dk && v < Dv ? S[d * Dv + v] : 0.f;
        }
}
template <int DKP>
__device__ __forceinline__ void state_store(const float (&s)[DKP / 8][4], float* S, int Dk, int Dv, int v0, int lane, int d0 = 0) {
    const int g = lane >> 2, tq = (lane & 3) * 2;
#pragma unroll
    for (int j = 0; j < DKP / 8; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int d = d0 + 8 * j + tq + (i & 1), v = v0 + g + (i >> 1) * 8;
            if (d < Dk && v < Dv) S[d * Dv + v] = s[j][i];
        }
}

// What the scans leave for the gradients (states, errors, ...): the operand
// planes of each 16 value columns x 16 columns block as four 8 x 8 tiles of 128
// contiguous bytes, [slice][plane][block][4][8][8].  A warp stores a register as
// one whole line, and ldmatrix on base + 16 lane finds a tile's rows side by
// side, without bank conflicts and in the order of the registers.
constexpr int kBlk = 256;  // elements of a block
template <int N>
__device__ __forceinline__ void put_tiles(const uint32_t (&a)[N][4], __nv_bfloat16* base, int slice, int blocks, int blk, int lane) {
#pragma unroll
    for (int p = 0; p < N; ++p) {
        __nv_bfloat16* r = base + (static_cast<long long>(slice * N + p) * blocks + blk) * kBlk + lane * 2;
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<uint32_t*>(r + 64 * i) = a[p][i];
    }
}

// ---------------------------------------------------------------- decays within a chunk
// One warp: the inclusive prefix L of log2 g over the chunk's tokens, summed in
// 64 bits and kept as the fp32 pair (L rounded, what that left), so that a
// difference of two of them is as good as one taken in 64 bits.
__device__ __forceinline__ void decay_prefix(float2* L, int lane, const float* __restrict__ log_g, int decay_kind, int h,
                                             long long bh, int t0, int T) {
    double a[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int t = t0 + 2 * lane + i;
        float g = 0.f;
        if (t < T) {
            if (decay_kind == LA_DECAY_PER_HEAD) g = log_g[h];
            if (decay_kind == LA_DECAY_PER_STEP) g = log_g[bh * T + t];
        }
        a[i] = static_cast<double>(g < kLogFloor ? kLogFloor : g) * 1.4426950408889634074;
    }
    double s = a[0] + a[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double x = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += x;
    }
    const double first = s - a[1];
    const float f = static_cast<float>(first), l = static_cast<float>(s);
    L[2 * lane] = make_float2(f, static_cast<float>(first - f));
    L[2 * lane + 1] = make_float2(l, static_cast<float>(s - l));
}
// 2^(L_t - L_s)
__device__ __forceinline__ float decay_between(float2 t, float2 s) { return ex2_approx((t.x - s.x) + (t.y - s.y)); }

// ---------------------------------------------------------------- the scans' pipeline
// Shared memory of one stage: the chunk's K (and Q) tiles as 64-column panels,
// the record's matrices and factors, the warps' value tiles.
template <int DKP, int NI, int kPlanes, int NW, bool kQ, bool kV, int kExtra = 0>
struct ScanTiles {
    static constexpr int kPanels = (DKP + 63) / 64;
    static constexpr int kTile = kPanels * 8192;  // one plane of K or Q
    static constexpr int k = 0;
    static constexpr int q = k + NI * kTile;
    static constexpr int rec = q + (kQ ? NI * kTile : 0);
    static constexpr int tok = rec + kPlanes * kSq;
    static constexpr int v = tok + 1024;
    static constexpr int bytes = (v + (kV ? 2048 * NW : 0) + 1023) / 1024 * 1024;
    static constexpr int kMost = (227 * 1024 - 1024 - 256 - kExtra) / bytes;
    static constexpr int stages = kMost > 3 ? 3 : kMost;
    static constexpr int extra = stages * bytes + 256;                 // behind the stages and their barriers
    static constexpr int smem = 1024 + extra + kExtra;                 // and the base's alignment
    static_assert(stages >= 1, "a chunk's tiles have to fit an SM");
};

// The stages' barriers and counts, behind the stages.
template <int kS>
struct Ring {
    uint64_t full[kS];  // completes when a stage's copies have landed
    int left[kS];       // warps that have not yet released the stage
    int issued[kS];     // chunks brought into the stage so far
    int abort;
};

// What brings a chunk into a stage.  No warp is a producer of its own (a ninth
// warp would halve the registers of eight): the warp that releases a stage last
// refills it, kS chunks on.
template <typename Tl, int NI, bool kQ, bool kV>
struct Feed {
    const CUtensorMap *mk, *mq, *mv;
    const unsigned char* records;  // of this (b, h)
    long long rec_bytes;
    int rec_used, hk, planes_apart, bh, v0, nv, warps;  // nv: value tiles, warps: those that read a stage

    __device__ __forceinline__ void issue(uint32_t base, Ring<Tl::stages>* ring, int s, int c) const {
        uint64_t* bar = &ring->full[s];
        const uint32_t st = base + s * Tl::bytes;
        ring->issued[s] = ring->issued[s] + 1;
        mbar_arrive_expect_tx(bar, (kQ ? 2 : 1) * NI * Tl::kTile + rec_used + 4 * kTok + (kV ? 2048 * nv : 0));
        for (int p = 0; p < NI; ++p)
            for (int i = 0; i < Tl::kPanels; ++i) {
                tma_load(st + Tl::k + p * Tl::kTile + 8192 * i, mk, bar, 64 * i, c * C, hk + p * planes_apart);
                if (kQ) tma_load(st + Tl::q + p * Tl::kTile + 8192 * i, mq, bar, 64 * i, c * C, hk + p * planes_apart);
            }
        const unsigned char* rec = records + c * rec_bytes;
        bulk_load(st + Tl::rec, rec, rec_used, bar);
        bulk_load(st + Tl::tok, rec + rec_bytes - 4 * kTail, 4 * kTok, bar);
        if (kV)
            for (int w = 0; w < nv; ++w) tma_load(st + Tl::v + 2048 * w, mv, bar, v0 + 16 * w, c * C, bh);
    }
};

// A warp's wait for a stage's `use`-th chunk; false once any warp of the block
// gave up, and then no copy of the block is still in flight (or none of them
// lands within the limit).
template <int kS>
__device__ __forceinline__ bool wait_stage(Ring<kS>* ring, int s, int use, int* err) {
    uint64_t* bar = &ring->full[s];
    bool got = mbar_try_wait(bar, use & 1);
    if (__all_sync(0xffffffffu, got)) return true;
    const uint64_t t0 = global_timer_ns();
    volatile int* abort = &ring->abort;
    while (true) {
        if (!got) got = mbar_try_wait_sleep(bar, use & 1, 20000);
        if (__all_sync(0xffffffffu, got)) return true;
        const bool late = *abort != 0 || global_timer_ns() - t0 > kWaitLimitNs;
        if (__any_sync(0xffffffffu, late)) {
            if ((threadIdx.x & 31) == 0) {
                *abort = 1;
                if (err) atomicCAS(err, 0, kErrTmaWait);
                for (int i = 0; i < kS; ++i) {
                    const int n = *static_cast<volatile int*>(&ring->issued[i]);
                    if (n > 0) mbar_wait_bounded(&ring->full[i], (n - 1) & 1, kWaitLimitNs);
                }
            }
            __syncwarp();
            return false;
        }
    }
}

// A warp has read all it needs of stage s; the last one brings chunk `next` in (or none: next < 0).
template <typename Tl, typename F>
__device__ __forceinline__ void release_stage(const F& feed, uint32_t base, Ring<Tl::stages>* ring, int s, int next) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) {
        __threadfence_block();  // this warp's reads come before the count
        if (atomicSub(&ring->left[s], 1) == 1) {
            __threadfence_block();  // and every other's before the copies
            ring->left[s] = feed.warps;
            if (next >= 0 && *static_cast<volatile int*>(&ring->abort) == 0) {
                fence_async_smem();
                feed.issue(base, ring, s, next);
            }
        }
    }
}

template <typename Tl, typename F>
__device__ __forceinline__ void start_ring(const F& feed, uint32_t base, Ring<Tl::stages>* ring, int n, int first, int step) {
    if (threadIdx.x == 0) {
        for (int s = 0; s < Tl::stages; ++s) {
            mbar_init(&ring->full[s], 1);
            ring->left[s] = feed.warps;
            ring->issued[s] = 0;
        }
        ring->abort = 0;
        fence_barrier_init();
        fence_async_smem();
        for (int s = 0; s < Tl::stages && s < n; ++s) feed.issue(base, ring, s, first + s * step);
    }
    __syncthreads();
}

// As release_stage and start_ring where a warp more than the slices need costs no
// registers that they lack: that warp's first lane refills the stages (feed_ring),
// and a release is one arrival (a release by count and refill: 200 cycles of a
// chunk's 5100 at the pair's rate).
template <int kS>
struct FedRing {
    Ring<kS> ring;      // left: unused
    uint64_t empty[kS];
};
template <typename Tl, typename F>
__device__ __forceinline__ void init_fed(const F& feed, FedRing<Tl::stages>* r) {
    if (threadIdx.x == 0) {
        for (int s = 0; s < Tl::stages; ++s) {
            mbar_init(&r->ring.full[s], 1);
            mbar_init(&r->empty[s], feed.warps);
            r->ring.issued[s] = 0;
        }
        r->ring.abort = 0;
        fence_barrier_init();
    }
    __syncthreads();
}
template <typename Tl, typename F>
__device__ __forceinline__ void feed_ring(const F& feed, uint32_t base, FedRing<Tl::stages>* r, int n, int first, int step, int* err) {
    constexpr int kS = Tl::stages;
    volatile int* abort = &r->ring.abort;
    int j = 0;
    for (; j < n; ++j) {
        const int s = j % kS;
        if (j >= kS && !mbar_wait_bounded(&r->empty[s], ((j / kS) - 1) & 1, kWaitLimitNs)) {
            *abort = 1;
            if (err) atomicCAS(err, 0, kErrTmaWait);
            break;
        }
        if (*abort) break;
        feed.issue(base, &r->ring, s, first + j * step);
    }
    // no copy may be in flight when the block ends
    for (int i = j > kS ? j - kS : 0; i < j; ++i) mbar_wait_bounded(&r->ring.full[i % kS], (i / kS) & 1, kWaitLimitNs);
}
__device__ __forceinline__ void release_fed(uint64_t* empty) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(empty);
}

// ---------------------------------------------------------------- several warps a slice
// Where a warp per slice leaves tensor cores idle, G = 2 or 4 share one.  Warp w has
// 1 / G of the key width of S^T in its accumulators and 4 / G of the chunk's
// 16-token blocks: {0, 3} or {1, 2} for two, which have the same share of the
// triangular products, block w for four.  What one needs of the others (split
// operands) passes through shared memory in register order, a 16-byte access a
// lane.
template <int G>
__device__ __forceinline__ int own_block(int w, int j) {
    return G == 4 ? w : w ? 1 + j : 3 * j;
}

// Planes [N][32 lanes] of an A operand.
template <int N>
__device__ __forceinline__ void put_planes(uint4* at, int lane, const uint32_t (&a)[N][4]) {
#pragma unroll
    for (int p = 0; p < N; ++p) at[p * 32 + lane] = make_uint4(a[p][0], a[p][1], a[p][2], a[p][3]);
}
template <int N>
__device__ __forceinline__ void get_planes(const uint4* at, int lane, uint32_t (&a)[N][4]) {
#pragma unroll
    for (int p = 0; p < N; ++p) {
        const uint4 x = at[p * 32 + lane];
        a[p][0] = x.x;
        a[p][1] = x.y;
        a[p][2] = x.z;
        a[p][3] = x.w;
    }
}

// The group's barrier (32 G threads).  It is reached by all its warps or, once a
// wait gave up, by none: group_agree() ends them together.
template <int G>
__device__ __forceinline__ void group_sync(int slice) {
    asm volatile("bar.sync %0, %1;" ::"r"(1 + slice), "n"(32 * G) : "memory");
}
template <int G>
__device__ __forceinline__ bool group_agree(int slice, bool ok) {
    uint32_t all;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %2, 0;\n\t"
        "bar.red.and.pred q, %1, %3, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}\n"
        : "=r"(all)
        : "r"(1 + slice), "r"(ok ? 1u : 0u), "n"(32 * G)
        : "memory");
    return all != 0;
}

// Byte offset, within a K or Q tile's row band, of 16-column step d of warp x's part
// of the key width (64-column panels, swizzled rows), from the lane's offsets of
// the first panel's four steps.
template <int DKP, int G>
__device__ __forceinline__ uint32_t step_offset(const LaneOffsets& l, int x, int d) {
    constexpr int kSteps = DKP / 16 / G;
    if constexpr (kSteps == 4) return l.o[d] + 8192 * x;
    if constexpr (kSteps == 2 && G == 4) return (l.o[d] ^ ((x & 1) << 6)) + 8192 * (x >> 1);
    return l.o[d] ^ (x * kSteps << 5);
}

// One 16-token block in accumulator layout, from the warp's tile or (fp32) from global memory ...
__device__ __forceinline__ void block_from_tile(float (&x)[2][4], uint32_t tile, int block, int lane) {
    uint32_t r[4];
    ldsm4t(r, tile + 512 * block + (lane & 15) * 32 + (lane >> 4) * 16);
    x[0][0] = low_of(r[0]);
    x[0][1] = high_of(r[0]);
    x[1][0] = low_of(r[1]);
    x[1][1] = high_of(r[1]);
    x[0][2] = low_of(r[2]);
    x[0][3] = high_of(r[2]);
    x[1][2] = low_of(r[3]);
    x[1][3] = high_of(r[3]);
}
__device__ __forceinline__ void block_from_global(float (&x)[2][4], const float* base, int t0, int T, int Dv, int v0, int lane) {
    const int g = lane >> 2, tq = (lane & 3) * 2;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = t0 + 8 * j + tq + (i & 1), v = v0 + g + (i >> 1) * 8;
            x[j][i] = t < T && v < Dv ? base[static_cast<long long>(t) * Dv + v] : 0.f;
        }
}
// ... and back.
__device__ __forceinline__ void block_to_global(const float (&x)[2][4], __nv_bfloat16* base, int t0, int T, int Dv, int v0,
                                                int lane) {
    const int g = lane >> 2, tq = (lane & 3) * 2;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const uint32_t lo = mov_trans(pack(x[j][0], x[j][1])), hi = mov_trans(pack(x[j][2], x[j][3]));
        const int t = t0 + 8 * j + g;
        if (t < T) {
            __nv_bfloat16* p = base + static_cast<long long>(t) * Dv + v0 + tq;
            *reinterpret_cast<uint32_t*>(p) = lo;
            *reinterpret_cast<uint32_t*>(p + 8) = hi;
        }
    }
}
__device__ __forceinline__ void block_to_global(const float (&x)[2][4], float* base, int t0, int T, int Dv, int v0, int lane) {
    const int g = lane >> 2, tq = (lane & 3) * 2;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = t0 + 8 * j + tq + (i & 1), v = v0 + g + (i >> 1) * 8;
            if (t < T && v < Dv) base[static_cast<long long>(t) * Dv + v] = x[j][i];
        }
}
// x[j] *= f of the block's tokens (f: the chunk's factors)
__device__ __forceinline__ void block_scale(float (&x)[2][4], const float* f, int block, int tq, float s = 1.f) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const float2 m = *reinterpret_cast<const float2*>(f + 16 * block + 8 * j + tq);
        x[j][0] *= s * m.x;
        x[j][1] *= s * m.y;
        x[j][2] *= s * m.x;
        x[j][3] *= s * m.y;
    }
}

}  // namespace delta
}  // namespace la
