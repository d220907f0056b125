// Instances of attn_keys_mx4 for float32.
#include "attn_mx4_kernels.cuh"

namespace sffn {

template <>
hipError_t launch_attn_keys_mx4<float>(const AttnMx4Args& m, int tile_rows, int waves, bool near,
                                           bool compact, hipStream_t s) {
  const int d = m.a.p.D;
  if (d <= 64) return attn_keys_mx4_width<float, 64>(m, tile_rows, waves, near, compact, s);
  if (d <= 128) return attn_keys_mx4_width<float, 128>(m, tile_rows, waves, near, compact, s);
  return attn_keys_mx4_width<float, 256>(m, tile_rows, waves, near, compact, s);
}

}  // namespace sffn
