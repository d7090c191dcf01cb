// gdn_attn_decode_f32.hip -- attention over a paged cache, one instantiation set.
#include "gdn_attn_decode.hpp"

namespace gdn {
hipError_t launch_attn_f32(const AttnParams& p, int d, dim3 grid, hipStream_t stream) {
  return launch_attn_t<float, float>(p, d, grid, stream);
}
}  // namespace gdn
