// Instances of attn_keys for float32.
#include "attn_kernels.cuh"

namespace sffn {

template <>
hipError_t launch_attn_keys<float>(const AttnArgs& a, int granule, bool compact, hipStream_t s) {
  SFFN_ATTN_BY_WIDTH(attn_keys_width, float, a, granule, compact, s);
}

}  // namespace sffn
