// la_delta_fwd_w128.cu - the gated delta rule's forward at key width 128.
#include "la_delta_fwd.cuh"

namespace la {
namespace delta {
cudaError_t forward_w128(const Plan& p, const Args& a, bool outputs) { return forward_width<128>(p, a, outputs); }
}  // namespace delta
}  // namespace la
