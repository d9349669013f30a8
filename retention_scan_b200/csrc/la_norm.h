// la_norm.h - launch interface of la_norm.cu and la_rotary.cu.
#pragma once
#include <cuda_runtime.h>

#include "la.h"
#include "la_fastdiv.h"

namespace la {

// Rows of D dense elements at data + i0 stride[0] + i1 stride[1] + i2 stride[2].
struct View {
    void* data;
    long long stride[3];
};

namespace norm {

constexpr int kMaxWidth = 8192;

struct Args {
    View x, gate, residual, out;  // gate, residual: data null when absent
    View dout, dx, dgate;         // backward
    const float* weight;          // [D] or null
    float* dweight;               // backward, or null
    float* partial;               // its workspace, or null
    int ahead;                    // backward: bytes of shared memory before the reductions'
    int n[3];
    FastDiv n1, n2;               // division by n[1], n[2]
    long long rows;
    int D, kind, activation;
    float eps, scale, inv;        // inv: 1 / D
    cudaStream_t stream;
};
cudaError_t launch(const Args& a, la_dtype dtype, bool backward);
size_t backward_workspace_bytes(long long rows, int D);

}  // namespace norm

namespace rotary {

struct Args {
    View x[2], out[2];
    int heads[2];             // heads of each tensor (second 0: absent)
    const float* freq;        // [R / 2]
    const long long* pos;     // position of (b, t) at pos[b * pos_stride + t], or null: start + t
    long long pos_stride, start;
    int B, T, D, R, layout;
    float mscale, direction;  // direction: 1, or -1 for the inverse rotation
    cudaStream_t stream;
};
cudaError_t launch(const Args& a, la_dtype dtype);

}  // namespace rotary
}  // namespace la
