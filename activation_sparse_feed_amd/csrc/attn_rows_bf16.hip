// Instances of attn_rows for bfloat16.
#include "attn_kernels.cuh"

namespace sffn {

template <>
hipError_t launch_attn_rows<uint16_t>(const AttnArgs& a, int granule, hipStream_t s) {
  SFFN_ATTN_BY_WIDTH(attn_rows_width, uint16_t, a, granule, s);
}

}  // namespace sffn
