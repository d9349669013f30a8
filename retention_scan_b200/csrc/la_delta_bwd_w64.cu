// la_delta_bwd_w64.cu - the gated delta rule's gradients at key width 64.
#include "la_delta_bwd.cuh"

namespace la {
namespace delta {
cudaError_t backward_w64(const Plan& p, const Args& a) { return backward_width<64>(p, a); }
}  // namespace delta
}  // namespace la
