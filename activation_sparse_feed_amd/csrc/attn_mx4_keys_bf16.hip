// Instances of attn_keys_mx4 for bfloat16.
#include "attn_mx4_kernels.cuh"

namespace sffn {

template <>
hipError_t launch_attn_keys_mx4<uint16_t>(const AttnMx4Args& m, int row_tiles, bool compact, hipStream_t s) {
  const int d = m.a.p.D;
  if (d <= 64) return attn_keys_mx4_width<uint16_t, 64>(m, row_tiles, compact, s);
  if (d <= 128) return attn_keys_mx4_width<uint16_t, 128>(m, row_tiles, compact, s);
  return attn_keys_mx4_width<uint16_t, 256>(m, row_tiles, compact, s);
}

}  // namespace sffn
