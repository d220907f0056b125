// Instances of attn_rows_mx4 for float32.
#include "attn_mx4_kernels.cuh"

namespace sffn {

template <>
hipError_t launch_attn_rows_mx4<float>(const AttnMx4Args& m, bool near, hipStream_t s) {
  const AttnArgs& a = m.a;
  SFFN_ATTN_BY_WIDTH(attn_rows_mx4_width, float, m, near, s);
}

}  // namespace sffn
