// rule_f32_256.hip -- the chunked gated delta rule for f32 rows, d_k <= 256.
#include "rule_kernels.hpp"

namespace gdn {
template hipError_t rule_forward_launch<GDN_F32, 256>(const RuleArgs&, hipStream_t);
template hipError_t rule_backward_launch<GDN_F32, 256>(const RuleArgs&, hipStream_t);
}  // namespace gdn
