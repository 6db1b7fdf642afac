// rule_bf16_128.hip -- the chunked gated delta rule for bf16 rows, d_k <= 128.
#include "rule_kernels.hpp"

namespace gdn {
template hipError_t rule_forward_launch<GDN_BF16, 128>(const RuleArgs&, hipStream_t);
template hipError_t rule_backward_launch<GDN_BF16, 128>(const RuleArgs&, hipStream_t);
}  // namespace gdn
