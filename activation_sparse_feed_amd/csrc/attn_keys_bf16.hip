// Instances of attn_keys for bfloat16.
#include "attn_kernels.cuh"

namespace sffn {

template <>
hipError_t launch_attn_keys<uint16_t>(const AttnArgs& a, int granule, bool compact, hipStream_t s) {
  SFFN_ATTN_BY_WIDTH(attn_keys_width, uint16_t, a, granule, compact, s);
}

}  // namespace sffn
