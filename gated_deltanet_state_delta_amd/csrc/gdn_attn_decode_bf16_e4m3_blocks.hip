// gdn_attn_decode_bf16_e4m3_blocks.hip -- attention over a paged cache, one instantiation set.
#include "gdn_attn_decode.hpp"

namespace gdn {
hipError_t launch_attn_bf16_e4m3_blocks(const AttnParams& p, int d, dim3 grid, hipStream_t stream) {
  return launch_attn_t<__bf16, e4m3, true>(p, d, grid, stream);
}
}  // namespace gdn
