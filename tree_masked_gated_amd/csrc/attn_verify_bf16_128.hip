// attn_verify_bf16_128.hip -- tree attention over a paged cache: bf16, head sizes up to 128.
#include "attn_verify.hpp"

namespace gdn {

hipError_t attn_launch_bf16_128(const AttnArgs& a, hipStream_t stream) { return attn::launch_d<GDN_BF16, 128>(a, stream); }
size_t attn_bytes_bf16_128(int B, int N, int group, int Hk) { return attn::bytes_d<GDN_BF16, 128>(B, N, group, Hk); }

}  // namespace gdn
