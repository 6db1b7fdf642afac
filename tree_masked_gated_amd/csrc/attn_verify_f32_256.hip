// attn_verify_f32_256.hip -- tree attention over a paged cache: f32, head sizes up to 256.
#include "attn_verify.hpp"

namespace gdn {

hipError_t attn_launch_f32_256(const AttnArgs& a, hipStream_t stream) { return attn::launch_d<GDN_F32, 256>(a, stream); }
size_t attn_bytes_f32_256(int B, int N, int group, int Hk) { return attn::bytes_d<GDN_F32, 256>(B, N, group, Hk); }

}  // namespace gdn
