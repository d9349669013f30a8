// la_delta_bwd_w128.cu - the gated delta rule's gradients at key width 128.
#include "la_delta_bwd.cuh"

namespace la {
namespace delta {
cudaError_t backward_w128(const Plan& p, const Args& a) { return backward_width<128>(p, a); }
}  // namespace delta
}  // namespace la
