// la_delta_fwd_w32.cu - the gated delta rule's forward at key width 32.
#include "la_delta_fwd.cuh"

namespace la {
namespace delta {
cudaError_t forward_w32(const Plan& p, const Args& a, bool outputs) { return forward_width<32>(p, a, outputs); }
}  // namespace delta
}  // namespace la
