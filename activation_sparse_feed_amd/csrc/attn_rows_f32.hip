// Instances of attn_rows for float32.
#include "attn_kernels.cuh"

namespace sffn {

template <>
hipError_t launch_attn_rows<float>(const AttnArgs& a, int granule, hipStream_t s) {
  SFFN_ATTN_BY_WIDTH(attn_rows_width, float, a, granule, s);
}

}  // namespace sffn
