// la_delta_api.cu - the C ABI of the gated delta rule: argument checks, the
// workspace's plan and the launches' order.  Nothing here allocates device
// memory.
#include <cmath>

#include "la_check.h"
#include "la_delta_internal.h"

namespace la {
namespace delta {

bool supports(int Dk, int Dv, la_dtype dtype) {
    if (Dk > 128 || Dv > 128) return false;
    return dtype == LA_F32 || (Dk % 16 == 0 && Dv % 16 == 0);
}

// Blocks of the scans.  A block fills an SM's shared memory, so blocks beyond the
// SMs run in another round.  Few slices (16 value columns of a (b, h)) take one round
// with several warps each: four where a block has one slice (T777 D64 fp32, 16
// slices: 33 us against 43 with two), two where it has two (four's exchange fills
// shared memory's bandwidth: B1 H32 T65536 D128 2324 us against 2258).  Else a warp each: up to four have a
// tensor core of their own, eight share them and take about 1.7 times as long;
// the fewest rounds win, then the wider block.
static void plan_scan(Plan* p) {
    const int slices = p->DVP / 16;
    p->group = true;
    for (p->warps = 1; p->warps <= 2; ++p->warps)
        if (p->BH * ((slices + p->warps - 1) / p->warps) <= 148) return;
    p->group = false;
    double least = 0;
    for (int w = 1; w <= 8; w *= 2) {
        if (w > 1 && w / 2 >= slices) break;
        const long long blocks = p->BH * ((slices + w - 1) / w);
        const double t = static_cast<double>((blocks + 147) / 148) * (w == 8 ? 1.7 : 1.0);
        if (w == 1 || t <= least) {
            p->warps = w;
            least = t;
        }
    }
}

static bool make_map(CUtensorMap* map, const void* base, int width, long long rows, long long outer, long long row_elems,
                     int box_cols, bool swizzle) {
    EncodeTiledFn f = encode_tiled();
    if (!f) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(outer)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(row_elems) * 2, static_cast<cuuint64_t>(row_elems) * rows * 2};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(box_cols), C, 1}, elem[3] = {1, 1, 1};
    return f(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, elem,
             CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_maps(Plan* p, const Args& a) {
    p->err = device_error_word();
    const long long keys = static_cast<long long>(a.B) * a.Hk * (a.dtype == LA_F32 ? 3 : 1);
    Maps* m = &p->maps;
    if (!make_map(&m->k, p->k.base, p->k.cols, p->k.rows, keys, p->k.row, 64, true)) return false;
    if (!make_map(&m->q, p->q.base, p->q.cols, p->q.rows, keys, p->q.row, 64, true)) return false;
    m->v = m->dy = m->k;  // fp32 values are read without a map; any valid one stands in
    if (a.dtype == LA_F32) return true;
    if (!make_map(&m->v, a.v, a.Dv, a.T, p->BH, a.Dv, 16, false)) return false;
    return !a.dy || make_map(&m->dy, a.dy, a.Dv, a.T, p->BH, a.Dv, 16, false);
}

Plan make_plan(const Args& a, bool backward, void* workspace) {
    Plan p{};
    p.BH = static_cast<long long>(a.B) * a.H;
    p.n = static_cast<int>((static_cast<long long>(a.T) + C - 1) / C);
    p.DKP = a.Dk <= 32 ? 32 : a.Dk <= 64 ? 64 : 128;
    p.DVP = (a.Dv + 15) / 16 * 16;
    plan_scan(&p);
    const bool f32 = a.dtype == LA_F32;
    const size_t nm = operand_planes(a, backward), np = f32 || backward ? nm : 1, bf = sizeof(__nv_bfloat16);
    const size_t chunks = static_cast<size_t>(p.BH) * p.n, keys = static_cast<size_t>(a.B) * a.Hk;
    size_t at = 0;
    auto region = [&](size_t bytes) {
        void* r = workspace ? static_cast<char*>(workspace) + at : nullptr;
        at += check::round256(bytes);
        return r;
    };
    p.records = static_cast<unsigned char*>(region(chunks * record_bytes(static_cast<int>(nm + np))));
    if (f32) {
        const size_t plane = keys * p.n * C * p.DKP;
        p.qs = static_cast<__nv_bfloat16*>(region(bf * 3 * plane));
        p.ks = static_cast<__nv_bfloat16*>(region(bf * 3 * plane));
        p.q = {p.qs, static_cast<long long>(plane), static_cast<long long>(p.n) * C * p.DKP, p.DKP, p.n * C, p.DKP};
        p.k = p.q;
        p.k.base = p.ks;
    } else {
        p.q = {static_cast<const __nv_bfloat16*>(a.q), 0, static_cast<long long>(a.T) * a.Dk, a.Dk, a.T, a.Dk};
        p.k = p.q;
        p.k.base = static_cast<const __nv_bfloat16*>(a.k);
    }
    if (backward) {
        p.S = static_cast<__nv_bfloat16*>(region(bf * chunks * nm * p.DVP * p.DKP));
        p.dS = static_cast<__nv_bfloat16*>(region(bf * chunks * nm * p.DVP * p.DKP));
        p.Er = static_cast<__nv_bfloat16*>(region(bf * chunks * nm * p.DVP * C));
        p.dR = static_cast<__nv_bfloat16*>(region(bf * chunks * nm * p.DVP * C));
        if (a.H != a.Hk) {
            const size_t bytes = sizeof(float) * static_cast<size_t>(p.BH) * a.T * a.Dk;
            p.dqh = static_cast<float*>(region(bytes));
            p.dkh = static_cast<float*>(region(bytes));
        }
        p.dlog = static_cast<double*>(region(sizeof(double) * chunks));
    }
    p.bytes = at;
    return p;
}

cudaError_t launch_forward(const Plan& p, const Args& a, bool outputs) {
    return p.DKP == 32 ? forward_w32(p, a, outputs) : p.DKP == 64 ? forward_w64(p, a, outputs) : forward_w128(p, a, outputs);
}

// d log g of a head: its chunks' sums over every sequence, in a fixed order.
__global__ void head_decay_kernel(const double* __restrict__ part, float* __restrict__ out, int B, int H, int n) {
    const int h = blockIdx.x, lane = threadIdx.x;
    double s = 0.0;
    for (int b = 0; b < B; ++b)
        for (int c = lane; c < n; c += 32) s += part[(static_cast<long long>(b) * H + h) * n + c];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) out[h] = static_cast<float>(s);
}

cudaError_t launch_backward(const Plan& p, const Args& a) {
    cudaError_t e = p.DKP == 32 ? backward_w32(p, a) : p.DKP == 64 ? backward_w64(p, a) : backward_w128(p, a);
    if (e == cudaSuccess && a.d_log_g && a.decay_kind == LA_DECAY_PER_HEAD) {
        head_decay_kernel<<<a.H, 32, 0, a.stream>>>(p.dlog, a.d_log_g, a.B, a.H, p.n);
        e = cudaGetLastError();
    }
    return e;
}

}  // namespace delta
}  // namespace la

namespace {

using namespace la::check;
namespace delta = la::delta;

// As check_decay; with no token to decay (an empty log_g may have no address) only the kind counts.
la_status check_decay_for(const la_decay* decay, bool tokens, int* kind, const float** log_g) {
    if (tokens || !decay) return check_decay(decay, kind, log_g);
    return decay->kind < LA_DECAY_NONE || decay->kind > LA_DECAY_PER_STEP ? LA_ERR_INVALID_ARG : LA_OK;
}

// Sizes, types and what every call of the family shares.
la_status check_sizes(int B, int H, int Hk, int T, int Dk, int Dv, la_dtype dtype) {
    if (B < 0 || H < 0 || T < 0 || Dk < 1 || Dv < 1 || Hk < 0) return LA_ERR_INVALID_ARG;
    if (H > 0 && (Hk < 1 || H % Hk != 0)) return LA_ERR_INVALID_ARG;
    if (dtype != LA_F32 && dtype != LA_BF16) return LA_ERR_INVALID_ARG;
    if (!delta::supports(Dk, Dv, dtype)) return LA_ERR_UNSUPPORTED;
    const long long BH = static_cast<long long>(B) * H;
    if (T > (1 << 30) || !fits_int(BH * 8)) return LA_ERR_INVALID_ARG;
    // blocks are counted in 32 bits; fp32 inputs are split by one thread a column pair
    if (!fits_int(BH * ((T + 63LL) / 64) * 8) || (T > 0 && BH > LLONG_MAX / 1024 / T)) return LA_ERR_UNSUPPORTED;
    return LA_OK;
}

delta::Args size_args(int B, int H, int Hk, int T, int Dk, int Dv, la_dtype dtype) {
    delta::Args a{};
    a.B = B;
    a.H = H;
    a.Hk = Hk;
    a.T = T;
    a.Dk = Dk;
    a.Dv = Dv;
    a.dtype = dtype;
    return a;
}

size_t workspace_bytes(int B, int H, int Hk, int T, int Dk, int Dv, la_dtype dtype, int decay_kind, bool backward) {
    if (check_sizes(B, H, Hk, T, Dk, Dv, dtype) != LA_OK || B == 0 || H == 0 || T == 0) return 0;
    delta::Args a = size_args(B, H, Hk, T, Dk, Dv, dtype);
    a.decay_kind = decay_kind;
    return delta::make_plan(a, backward, nullptr).bytes;
}

cudaError_t copy_or_zero(float* dst, const float* src, size_t bytes, cudaStream_t s) {
    if (!dst) return cudaSuccess;
    return src ? cudaMemcpyAsync(dst, src, bytes, cudaMemcpyDeviceToDevice, s) : cudaMemsetAsync(dst, 0, bytes, s);
}

}  // namespace

extern "C" {

size_t la_delta_workspace_size(int B, int H, int Hk, int T, int Dk, int Dv, la_dtype dtype) {
    return workspace_bytes(B, H, Hk, T, Dk, Dv, dtype, LA_DECAY_NONE, false);
}

size_t la_delta_backward_workspace_size(int B, int H, int Hk, int T, int Dk, int Dv, la_dtype dtype, int decay_kind) {
    return workspace_bytes(B, H, Hk, T, Dk, Dv, dtype, decay_kind, true);
}

la_status la_delta_forward_ws(const void* q, const void* k, const void* v, const float* beta, const la_decay* decay,
                              float q_scale, const float* init_state, void* out, float* final_state, int B, int H, int Hk,
                              int T, int Dk, int Dv, la_dtype dtype, void* workspace, size_t workspace_bytes,
                              la_stream_t stream) {
    la_status st = check_sizes(B, H, Hk, T, Dk, Dv, dtype);
    if (st != LA_OK) return st;
    delta::Args a = size_args(B, H, Hk, T, Dk, Dv, dtype);
    const long long BH = static_cast<long long>(B) * H;
    if (check_decay_for(decay, BH > 0 && T > 0, &a.decay_kind, &a.log_g) != LA_OK || !std::isfinite(q_scale))
        return LA_ERR_INVALID_ARG;
    if ((init_state && !aligned16(init_state)) || (final_state && !aligned16(final_state))) return LA_ERR_INVALID_ARG;
    if (BH > 0 && T > 0) {
        for (const void* p : {q, k, v, static_cast<const void*>(out)})
            if (!p || !aligned16(p)) return LA_ERR_INVALID_ARG;
        if (!beta || !aligned4(beta)) return LA_ERR_INVALID_ARG;
        if (!workspace || !aligned16(workspace) ||
            workspace_bytes < la_delta_workspace_size(B, H, Hk, T, Dk, Dv, dtype))
            return LA_ERR_INVALID_ARG;
    }
    if (BH == 0) return LA_OK;
    if (launch_fault_injected()) return LA_ERR_CUDA;
    a.stream = reinterpret_cast<cudaStream_t>(stream);
    if (T == 0)
        return copy_or_zero(final_state, init_state, sizeof(float) * BH * Dk * Dv, a.stream) == cudaSuccess ? LA_OK
                                                                                                           : LA_ERR_CUDA;
    a.q = q;
    a.k = k;
    a.v = v;
    a.beta = beta;
    a.scale = q_scale;
    a.init_state = init_state;
    a.out = out;
    a.final_state = final_state;
    delta::Plan p = delta::make_plan(a, false, workspace);
    return delta::make_maps(&p, a) && delta::launch_forward(p, a, true) == cudaSuccess ? LA_OK : LA_ERR_CUDA;
}

la_status la_delta_backward_ws(const void* q, const void* k, const void* v, const float* beta, const la_decay* decay,
                               float q_scale, const float* init_state, const void* dy, const float* d_final_state, void* dq,
                               void* dk, void* dv, float* dbeta, float* d_log_g, float* d_init_state, int B, int H, int Hk,
                               int T, int Dk, int Dv, la_dtype dtype, void* workspace, size_t workspace_bytes,
                               la_stream_t stream) {
    la_status st = check_sizes(B, H, Hk, T, Dk, Dv, dtype);
    if (st != LA_OK) return st;
    delta::Args a = size_args(B, H, Hk, T, Dk, Dv, dtype);
    const long long BH = static_cast<long long>(B) * H;
    if (check_decay_for(decay, BH > 0 && T > 0, &a.decay_kind, &a.log_g) != LA_OK || !std::isfinite(q_scale))
        return LA_ERR_INVALID_ARG;
    const int kind = decay ? decay->kind : LA_DECAY_NONE;
    if (d_log_g && (kind == LA_DECAY_NONE || !aligned4(d_log_g))) return LA_ERR_INVALID_ARG;
    for (const void* p : {static_cast<const void*>(init_state), static_cast<const void*>(d_final_state),
                          static_cast<const void*>(d_init_state)})
        if (p && !aligned16(p)) return LA_ERR_INVALID_ARG;
    if (BH > 0 && T > 0) {
        for (const void* p : {q, k, v, dy, static_cast<const void*>(dq), static_cast<const void*>(dk), static_cast<const void*>(dv)})
            if (!p || !aligned16(p)) return LA_ERR_INVALID_ARG;
        if (!beta || !aligned4(beta) || !dbeta || !aligned4(dbeta)) return LA_ERR_INVALID_ARG;
        if (!workspace || !aligned16(workspace) ||
            workspace_bytes < la_delta_backward_workspace_size(B, H, Hk, T, Dk, Dv, dtype, kind))
            return LA_ERR_INVALID_ARG;
    }
    if (H == 0 && (!fits_int(static_cast<long long>(B) * Hk) || static_cast<long long>(B) * Hk > LLONG_MAX / 1024 / (T + 1LL)))
        return LA_ERR_UNSUPPORTED;
    const long long keys = H == 0 ? static_cast<long long>(B) * Hk * T : 0;
    if (keys > 0) {  // key heads that serve no value head: dq and dk are sums over nothing
        if (!dq || !aligned16(dq) || !dk || !aligned16(dk)) return LA_ERR_INVALID_ARG;
        if (launch_fault_injected()) return LA_ERR_CUDA;
        const size_t bytes = (dtype == LA_BF16 ? 2 : 4) * static_cast<size_t>(keys) * Dk;
        const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
        return cudaMemsetAsync(dq, 0, bytes, s) == cudaSuccess && cudaMemsetAsync(dk, 0, bytes, s) == cudaSuccess ? LA_OK
                                                                                                                : LA_ERR_CUDA;
    }
    if (H == 0 || (BH == 0 && !(d_log_g && kind == LA_DECAY_PER_HEAD))) return LA_OK;
    if (launch_fault_injected()) return LA_ERR_CUDA;
    a.stream = reinterpret_cast<cudaStream_t>(stream);
    if (T == 0 || BH == 0) {  // no token: the state's gradient passes through, a head's decay has none
        cudaError_t e = copy_or_zero(BH ? d_init_state : nullptr, d_final_state, sizeof(float) * BH * Dk * Dv, a.stream);
        if (e == cudaSuccess && kind == LA_DECAY_PER_HEAD) e = copy_or_zero(d_log_g, nullptr, sizeof(float) * H, a.stream);
        return e == cudaSuccess ? LA_OK : LA_ERR_CUDA;
    }
    a.q = q;
    a.k = k;
    a.v = v;
    a.beta = beta;
    a.scale = q_scale;
    a.init_state = init_state;
    a.dy = dy;
    a.d_final_state = d_final_state;
    a.dq = dq;
    a.dk = dk;
    a.dv = dv;
    a.dbeta = dbeta;
    a.d_log_g = d_log_g;
    a.d_init_state = d_init_state;
    delta::Plan p = delta::make_plan(a, true, workspace);
    if (!delta::make_maps(&p, a)) return LA_ERR_CUDA;
    cudaError_t e = delta::launch_forward(p, a, false);
    if (e == cudaSuccess) e = delta::launch_backward(p, a);
    return e == cudaSuccess ? LA_OK : LA_ERR_CUDA;
}

la_status la_delta_decode_step(const void* q, const void* k, const void* v, const float* beta, const la_decay* decay,
                               float q_scale, float* state, void* out, int B, int H, int Hk, int Dk, int Dv,
                               la_dtype dtype, la_stream_t stream) {
    if (B < 0 || H < 0 || Hk < 0 || Dk < 1 || Dv < 1) return LA_ERR_INVALID_ARG;
    if (H > 0 && (Hk < 1 || H % Hk != 0)) return LA_ERR_INVALID_ARG;
    if (dtype != LA_F32 && dtype != LA_BF16) return LA_ERR_INVALID_ARG;
    delta::DecodeArgs a{};
    const long long BH = static_cast<long long>(B) * H;
    if (check_decay_for(decay, BH > 0, &a.decay_kind, &a.log_g) != LA_OK || !std::isfinite(q_scale))
        return LA_ERR_INVALID_ARG;
    if (!fits_int(BH * 8)) return LA_ERR_INVALID_ARG;
    if (BH > 0) {
        for (const void* p : {q, k, v, static_cast<const void*>(out), static_cast<const void*>(state)})
            if (!p || !aligned16(p)) return LA_ERR_INVALID_ARG;
        if (!beta || !aligned4(beta)) return LA_ERR_INVALID_ARG;
    }
    if (Dk > 128 || Dv > 128) return LA_ERR_UNSUPPORTED;
    if (BH == 0) return LA_OK;
    if (launch_fault_injected()) return LA_ERR_CUDA;
    a.q = q;
    a.k = k;
    a.v = v;
    a.beta = beta;
    a.scale = q_scale;
    a.state = state;
    a.out = out;
    a.B = B;
    a.H = H;
    a.Hk = Hk;
    a.Dk = Dk;
    a.Dv = Dv;
    a.dtype = dtype;
    a.stream = reinterpret_cast<cudaStream_t>(stream);
    return delta::launch_decode(a) == cudaSuccess ? LA_OK : LA_ERR_CUDA;
}

}  // extern "C"
