// Attention of new tokens over the 4-bit paged cache: which kernels a batch takes and
// how far its key ranges are split.
#include <hip/hip_runtime.h>

#include "attn_mx4_kernels.cuh"
#include "attn_plan.h"

namespace sffn {

template <> hipError_t launch_attn_rows_mx4<uint16_t>(const AttnMx4Args&, hipStream_t);
template <> hipError_t launch_attn_rows_mx4<float>(const AttnMx4Args&, hipStream_t);
template <> hipError_t launch_attn_keys_mx4<uint16_t>(const AttnMx4Args&, int, bool, hipStream_t);
template <> hipError_t launch_attn_keys_mx4<float>(const AttnMx4Args&, int, bool, hipStream_t);

namespace {

Plan keys_of(int dtype, const PagedAttn& p) {
  const int step = kMx4KeysWaves * 32;
  return plan_keys(p, dtype == 1 ? KeysTuning{step * 5, step * 2, step * 6, 4 * kCus}
                                 : KeysTuning{step * 2, step, step, 4 * kCus});
}
Plan rows_of(int dtype, const PagedAttn& p, const Plan& keys) {
  return plan_rows(p, keys.used, dtype == 1 ? 256 : 128);
}

template <typename T>
hipError_t launch(AttnMx4Args m, const Plan& keys, const Plan& rows, void* ws, hipStream_t s) {
  AttnArgs& a = m.a;
  const int dtype = sizeof(T) == 2 ? 1 : 0;
  hipError_t e = hipSuccess;
  if (rows.used) {
    place(&a, rows, (char*)ws + keys.bytes);
    e = launch_attn_rows_mx4<T>(m, s);
    if (e == hipSuccess) e = launch_join(dtype, kRowsTile, a, rows, s);
    if (e != hipSuccess) return e;
  }
  if (keys.used) {
    place(&a, keys, ws);
    // one tile of 16 rows where no sequence that the kernel takes has more
    const int row_tiles = (int64_t)a.p.max_q * a.g <= 16 ? 1 : 2;
    e = launch_attn_keys_mx4<T>(m, row_tiles, rows.used, s);
    if (e == hipSuccess) e = launch_join(dtype, kKeysTile, a, keys, s);
  }
  return e;
}

}  // namespace

bool plan_paged_attn_mx4(int dtype, const PagedAttn& p, size_t* bytes) {
  *bytes = 0;
  if (p.T == 0 || p.n_seqs == 0 || p.max_q == 0) return true;  // nothing is launched
  const Plan keys = keys_of(dtype, p), rows = rows_of(dtype, p, keys);
  if (!plan_fits(keys, rows, p, kMx4KeysWaves * kWave)) return false;
  *bytes = keys.bytes + rows.bytes;
  return true;
}

hipError_t launch_paged_attn_mx4(int dtype, const PagedAttn& p, const Mx4Rows& k, const Mx4Rows& v,
                                 void* ws, hipStream_t stream) {
  const Plan keys = keys_of(dtype, p), rows = rows_of(dtype, p, keys);
  const AttnMx4Args m = {attn_args(p), k, v};
  return dtype == 1 ? launch<uint16_t>(m, keys, rows, ws, stream)
                    : launch<float>(m, keys, rows, ws, stream);
}

}  // namespace sffn
