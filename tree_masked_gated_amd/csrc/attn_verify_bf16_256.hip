// attn_verify_bf16_256.hip -- tree attention over a paged cache: bf16, head sizes up to 256.
#include "attn_verify.hpp"

namespace gdn {

hipError_t attn_launch_bf16_256(const AttnArgs& a, hipStream_t stream) { return attn::launch_d<GDN_BF16, 256>(a, stream); }
size_t attn_bytes_bf16_256(int B, int N, int group, int Hk) { return attn::bytes_d<GDN_BF16, 256>(B, N, group, Hk); }

}  // namespace gdn
