// la_delta_bwd_w32.cu - the gated delta rule's gradients at key width 32.
#include "la_delta_bwd.cuh"

namespace la {
namespace delta {
cudaError_t backward_w32(const Plan& p, const Args& a) { return backward_width<32>(p, a); }
}  // namespace delta
}  // namespace la
