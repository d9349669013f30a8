// la_delta_fwd_w64.cu - the gated delta rule's forward at key width 64.
#include "la_delta_fwd.cuh"

namespace la {
namespace delta {
cudaError_t forward_w64(const Plan& p, const Args& a, bool outputs) { return forward_width<64>(p, a, outputs); }
}  // namespace delta
}  // namespace la
