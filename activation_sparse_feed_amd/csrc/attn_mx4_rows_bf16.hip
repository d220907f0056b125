// Instances of attn_rows_mx4 for bfloat16.
#include "attn_mx4_kernels.cuh"

namespace sffn {

template <>
hipError_t launch_attn_rows_mx4<uint16_t>(const AttnMx4Args& m, bool near, hipStream_t s) {
  const AttnArgs& a = m.a;
  SFFN_ATTN_BY_WIDTH(attn_rows_mx4_width, uint16_t, m, near, s);
}

}  // namespace sffn
