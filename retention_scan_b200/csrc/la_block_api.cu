// la_block_api.cu - the C ABI of the gated norm and the rotary positions:
// argument checks and dispatch.
#include <climits>
#include <cmath>

#include "la_check.h"
#include "la_norm.h"

namespace {

using namespace la::check;

bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// A view of n[0] x n[1] x n[2] rows; an output's rows have to be apart.
bool read_view(const la_view* v, const int (&n)[3], size_t es, bool output, la::View* to) {
    if (!v || !v->data || !aligned_to(v->data, es)) return false;
    to->data = v->data;
    for (int i = 0; i < 3; ++i) {
        if (v->stride[i] < 0 || (output && n[i] > 1 && v->stride[i] == 0)) return false;
        if (i > 0 && n[i] > 1 && v->stride[i] > UINT_MAX) return false;
        to->stride[i] = v->stride[i];
    }
    return true;
}

la_status check_norm(int n0, int n1, int n2, int D, int kind, int activation, float eps, float scale, la_dtype dtype,
                     la::norm::Args* a) {
    if (n0 < 0 || n1 < 0 || n2 < 0 || D < 1) return LA_ERR_INVALID_ARG;
    if (kind < LA_NORM_RMS || kind > LA_NORM_L2 || activation < LA_GATE_SILU || activation > LA_GATE_SIGMOID)
        return LA_ERR_INVALID_ARG;
    if (!std::isfinite(eps) || eps < 0.f || !std::isfinite(scale)) return LA_ERR_INVALID_ARG;
    if (dtype != LA_F32 && dtype != LA_BF16) return LA_ERR_INVALID_ARG;
    if (D > la::norm::kMaxWidth) return LA_ERR_UNSUPPORTED;
    a->n[0] = n0;
    a->n[1] = n1;
    a->n[2] = n2;
    // a zero among them makes the product zero whatever the others are
    a->rows = n0 == 0 || n1 == 0 || n2 == 0 ? 0 : static_cast<long long>(n0) * n1;
    if (a->rows > INT_MAX || a->rows * n2 > INT_MAX) return LA_ERR_UNSUPPORTED;
    a->rows *= n2;
    a->D = D;
    a->kind = kind;
    a->activation = activation;
    a->eps = eps;
    a->scale = scale;
    return LA_OK;
}

}  // namespace

extern "C" {

la_status la_gated_norm(const la_view* x, const la_view* gate, const float* weight, const la_view* residual,
                        const la_view* out, int n0, int n1, int n2, int D, int kind, int activation, float eps, float scale,
                        la_dtype dtype, la_stream_t stream) {
    la::norm::Args a{};
    const la_status st = check_norm(n0, n1, n2, D, kind, activation, eps, scale, dtype, &a);
    if (st != LA_OK) return st;
    if (a.rows == 0) return LA_OK;
    const size_t es = dtype == LA_BF16 ? 2 : 4;
    if (!read_view(x, a.n, es, false, &a.x) || !read_view(out, a.n, es, true, &a.out)) return LA_ERR_INVALID_ARG;
    if ((gate && !read_view(gate, a.n, es, false, &a.gate)) || (residual && !read_view(residual, a.n, es, false, &a.residual)))
        return LA_ERR_INVALID_ARG;
    if (weight && !aligned4(weight)) return LA_ERR_INVALID_ARG;
    if (launch_fault_injected()) return LA_ERR_CUDA;
    a.weight = weight;
    a.stream = reinterpret_cast<cudaStream_t>(stream);
    return la::norm::launch(a, dtype, false) == cudaSuccess ? LA_OK : LA_ERR_CUDA;
}

size_t la_gated_norm_backward_workspace_size(int n0, int n1, int n2, int D) {
    la::norm::Args a{};
    if (check_norm(n0, n1, n2, D, LA_NORM_RMS, LA_GATE_SILU, 0.f, 1.f, LA_BF16, &a) != LA_OK || a.rows == 0) return 0;
    return la::norm::backward_workspace_bytes(a.rows, D);
}

la_status la_gated_norm_backward(const la_view* dout, const la_view* x, const la_view* gate, const float* weight,
                                 const la_view* dx, const la_view* dgate, float* dweight, int n0, int n1, int n2, int D,
                                 int kind, int activation, float eps, float scale, la_dtype dtype, void* workspace,
                                 size_t workspace_bytes, la_stream_t stream) {
    la::norm::Args a{};
    const la_status st = check_norm(n0, n1, n2, D, kind, activation, eps, scale, dtype, &a);
    if (st != LA_OK) return st;
    if ((gate != nullptr) != (dgate != nullptr) || (dweight && !weight)) return LA_ERR_INVALID_ARG;
    if ((weight && !aligned4(weight)) || (dweight && !aligned4(dweight))) return LA_ERR_INVALID_ARG;
    const size_t es = dtype == LA_BF16 ? 2 : 4;
    if (a.rows > 0) {
        if (!read_view(x, a.n, es, false, &a.x) || !read_view(dout, a.n, es, false, &a.dout) ||
            !read_view(dx, a.n, es, true, &a.dx))
            return LA_ERR_INVALID_ARG;
        if (gate && (!read_view(gate, a.n, es, false, &a.gate) || !read_view(dgate, a.n, es, true, &a.dgate)))
            return LA_ERR_INVALID_ARG;
        if (dweight && (!workspace || !aligned16(workspace) ||
                        workspace_bytes < la_gated_norm_backward_workspace_size(n0, n1, n2, D)))
            return LA_ERR_INVALID_ARG;
    } else if (!dweight) {
        return LA_OK;
    }
    if (launch_fault_injected()) return LA_ERR_CUDA;
    a.stream = reinterpret_cast<cudaStream_t>(stream);
    if (a.rows == 0) return cudaMemsetAsync(dweight, 0, sizeof(float) * D, a.stream) == cudaSuccess ? LA_OK : LA_ERR_CUDA;
    a.weight = weight;
    a.dweight = dweight;
    a.partial = dweight ? static_cast<float*>(workspace) : nullptr;
    return la::norm::launch(a, dtype, true) == cudaSuccess ? LA_OK : LA_ERR_CUDA;
}

la_status la_rotary(const la_view* x, int H, const la_view* x2, int H2, const la_view* out, const la_view* out2,
                    const float* freq, const long long* positions, long long positions_stride, long long start, int B, int T,
                    int D, int R, int layout, float mscale, int backward, la_dtype dtype, la_stream_t stream) {
    if (B < 0 || H < 0 || H2 < 0 || T < 0 || D < 1 || R < 2 || R % 2 != 0 || R > D) return LA_ERR_INVALID_ARG;
    if (layout != LA_ROTARY_HALF && layout != LA_ROTARY_INTERLEAVED) return LA_ERR_INVALID_ARG;
    if (!std::isfinite(mscale) || (dtype != LA_F32 && dtype != LA_BF16)) return LA_ERR_INVALID_ARG;
    if (!x2 && H2 != 0) return LA_ERR_INVALID_ARG;
    if (positions && (!aligned_to(positions, 8) || positions_stride < 0)) return LA_ERR_INVALID_ARG;
    constexpr long long kFar = 1ll << 53;  // positions are exact in 64-bit floating point up to here
    if (!positions && (start < -kFar || start > kFar - T)) return LA_ERR_INVALID_ARG;
    if (D > la::norm::kMaxWidth) return LA_ERR_UNSUPPORTED;
    const long long heads = static_cast<long long>(H) + H2, tokens = static_cast<long long>(B) * T;
    // a block's items, heads * tokens * D, and the grid, B * T * heads at most, are counted in 32 bits
    if (heads * 16 * D > INT_MAX || tokens > INT_MAX || (tokens > 0 && heads > INT_MAX / tokens)) return LA_ERR_UNSUPPORTED;
    if (tokens == 0 || heads == 0) return LA_OK;
    if (!freq || !aligned4(freq)) return LA_ERR_INVALID_ARG;
    la::rotary::Args a{};
    const size_t es = dtype == LA_BF16 ? 2 : 4;
    const int n[3] = {B, H, T}, n2[3] = {B, H2, T};
    if (H && (!read_view(x, n, es, false, &a.x[0]) || !read_view(out, n, es, true, &a.out[0]))) return LA_ERR_INVALID_ARG;
    if (H2 && (!read_view(x2, n2, es, false, &a.x[1]) || !read_view(out2, n2, es, true, &a.out[1]))) return LA_ERR_INVALID_ARG;
    if (launch_fault_injected()) return LA_ERR_CUDA;
    a.heads[0] = H;
    a.heads[1] = H2;
    a.freq = freq;
    a.pos = positions;
    a.pos_stride = positions_stride;
    a.start = start;
    a.B = B;
    a.T = T;
    a.D = D;
    a.R = R;
    a.layout = layout;
    a.mscale = mscale;
    a.direction = backward ? -1.f : 1.f;
    a.stream = reinterpret_cast<cudaStream_t>(stream);
    return la::rotary::launch(a, dtype) == cudaSuccess ? LA_OK : LA_ERR_CUDA;
}

}  // extern "C"
