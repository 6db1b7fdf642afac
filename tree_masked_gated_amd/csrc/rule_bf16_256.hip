// rule_bf16_256.hip -- the chunked gated delta rule for bf16 rows, d_k <= 256.
#include "rule_kernels.hpp"

namespace gdn {
template hipError_t rule_forward_launch<GDN_BF16, 256>(const RuleArgs&, hipStream_t);
template hipError_t rule_backward_launch<GDN_BF16, 256>(const RuleArgs&, hipStream_t);
}  // namespace gdn
