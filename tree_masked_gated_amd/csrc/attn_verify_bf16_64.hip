// attn_verify_bf16_64.hip -- tree attention over a paged cache: bf16, head sizes up to 64.
#include "attn_verify.hpp"

namespace gdn {

hipError_t attn_launch_bf16_64(const AttnArgs& a, hipStream_t stream) { return attn::launch_d<GDN_BF16, 64>(a, stream); }
size_t attn_bytes_bf16_64(int B, int N, int group, int Hk) { return attn::bytes_d<GDN_BF16, 64>(B, N, group, Hk); }

}  // namespace gdn
