// la_delta_internal.h - the gated delta rule's host-side plan: sizes, the
// workspace's regions, and the launchers that la_delta_api.cu calls.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "la.h"
#include "la_delta.cuh"

namespace la {
namespace delta {

struct Args {
    const void* q;             // [B,Hk,T,Dk]
    const void* k;
    const void* v;             // [B,H,T,Dv]
    const float* beta;         // [B,H,T]
    int decay_kind;
    const float* log_g;
    float scale;
    const float* init_state;   // [B,H,Dk,Dv] or null
    void* out;                 // forward: y; backward: unused
    float* final_state;        // or null
    int B, H, Hk, T, Dk, Dv;
    la_dtype dtype;
    cudaStream_t stream;
    // backward only
    const void* dy;
    const float* d_final_state;  // or null
    void* dq;
    void* dk;
    void* dv;
    float* dbeta;
    float* d_log_g;              // or null
    float* d_init_state;         // or null
};

// Tensor maps of the kernels' tiles: K and Q by 64 columns of 64 tokens (128-byte
// swizzle), the value-side operands v and dy (bf16 only) by 16 columns.
struct Maps {
    CUtensorMap k, q, v, dy;
};

// Where the workspace's regions start; everything a launch needs beyond Args.
struct Plan {
    Maps maps;    // set by make_maps, once a call
    int* err;     // the device error word
    long long BH;
    int n;        // chunks per sequence
    int DKP, DVP; // key width of the kernels, value width in whole 16-column slices
    int warps;    // 16-column slices per block of the scans
    bool group;   // several warps a slice
    Planes q, k;
    unsigned char* records;     // [BH][n][record_bytes(planes of both matrices)]
    __nv_bfloat16 *qs, *ks;     // fp32 inputs' planes
    // backward only
    __nv_bfloat16 *S, *dS;      // [BH][n] x planes of DVP x DKP (put_tiles): states before, gradients after each chunk
    __nv_bfloat16 *Er, *dR;     // [BH][n] x planes of DVP x C
    float *dqh, *dkh;           // [BH][T][Dk] per value head, where key heads are shared
    double* dlog;               // [BH][n]: a chunk's sum of d log g (per-head decay)
    size_t bytes;
};

struct ScanArgs {
    const void* v;
    const unsigned char* records;
    const float* init_state;
    void* out;
    float* final_state;
    __nv_bfloat16 *Sst, *Est;
    int* err;
    float scale;
    int planes_apart;  // key heads of a plane (fp32 inputs)
    int H, Hk, T, Dk, Dv, DVP, n, vblocks;
};

bool make_maps(Plan* p, const Args& a);

inline ScanArgs scan_args(const Plan& p, const Args& a) {
    ScanArgs s{};
    s.v = a.v;
    s.records = p.records;
    s.err = p.err;
    s.planes_apart = a.B * a.Hk;
    s.init_state = a.init_state;
    s.out = a.out;
    s.final_state = a.final_state;
    s.Sst = p.S;
    s.Est = p.Er;
    s.scale = a.scale;
    s.H = a.H;
    s.Hk = a.Hk;
    s.T = a.T;
    s.Dk = a.Dk;
    s.Dv = a.Dv;
    s.DVP = p.DVP;
    s.n = p.n;
    return s;
}

bool supports(int Dk, int Dv, la_dtype dtype);

// bf16 planes of an fp32 operand.  Two keep 16 bits, enough for states: 4e-6 of their
// norm.  fp32 inputs take three, and so do three kinds of bf16 backward, for their fp32
// outputs (dbeta, the decay's gradient).  Off 64 bits by (2-norm of the tensor; median
// and worst of 544 random cases, or worst) and us, with two planes and with three:
// - a decay per head, whose gradient sums over the whole sequence terms of both signs
//   that leave a small rest: 1.1e-4 and 9e-6 (one head), 2.3e-5 and 2e-6 (four);
//   575 and 818 us at B2 H16 T4096 D128.
// - fewer than 4096 tokens times heads, calls so small that the third plane costs
//   little: 3e-6 to 6e-6, worst 1.3e-5, and 5e-7 to 1.2e-6, worst 2e-6; 43 and 41 us at
//   64 of them, 48 and 60 at 1024, 83 and 108 at 4092 (D128).  At 4096 and more,
//   6e-6, worst 1.0e-5, and 1.3e-6; 60 and 76 us at B1 H8 T512, 568 and 810 at B2
//   H16 T4096.
// - keys of at most 32 dimensions: 8e-6 and 1.2e-6; 121 and 168 us at B2 H8 T2048
//   Dk32 Dv64.
constexpr int kNarrowKeys = 32;
constexpr long long kFewTokens = 4096;
inline int operand_planes(const Args& a, bool backward) {
    if (a.dtype == LA_F32) return 3;
    return backward && (a.decay_kind == LA_DECAY_PER_HEAD || a.Dk <= kNarrowKeys ||
                        static_cast<long long>(a.B) * a.H * a.T < kFewTokens) ? 3 : 2;
}
// Regions from `workspace` on (null: sizes only).
Plan make_plan(const Args& a, bool backward, void* workspace);

// prep and the scan over the chunks; outputs: y and the final state, else
// (backward) every chunk's incoming state and errors.
cudaError_t launch_forward(const Plan& p, const Args& a, bool outputs);
cudaError_t forward_w32(const Plan& p, const Args& a, bool outputs);
cudaError_t forward_w64(const Plan& p, const Args& a, bool outputs);
cudaError_t forward_w128(const Plan& p, const Args& a, bool outputs);
// After launch_forward(..., false): the reverse scan and the gradients.
cudaError_t launch_backward(const Plan& p, const Args& a);
cudaError_t backward_w32(const Plan& p, const Args& a);
cudaError_t backward_w64(const Plan& p, const Args& a);
cudaError_t backward_w128(const Plan& p, const Args& a);

struct DecodeArgs {
    const void* q;
    const void* k;
    const void* v;
    const float* beta;
    int decay_kind;
    const float* log_g;
    float scale;
    float* state;
    void* out;
    int B, H, Hk, Dk, Dv;
    la_dtype dtype;
    cudaStream_t stream;
};
cudaError_t launch_decode(const DecodeArgs& a);

}  // namespace delta
}  // namespace la
