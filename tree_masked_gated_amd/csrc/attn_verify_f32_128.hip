// attn_verify_f32_128.hip -- tree attention over a paged cache: f32, head sizes up to 128.
#include "attn_verify.hpp"

namespace gdn {

hipError_t attn_launch_f32_128(const AttnArgs& a, hipStream_t stream) { return attn::launch_d<GDN_F32, 128>(a, stream); }
size_t attn_bytes_f32_128(int B, int N, int group, int Hk) { return attn::bytes_d<GDN_F32, 128>(B, N, group, Hk); }

}  // namespace gdn
