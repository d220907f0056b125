// Attention of new tokens over the 4-bit paged cache: which kernels a batch takes and
// how far its key ranges are split.
#include <hip/hip_runtime.h>

#include "attn_mx4_kernels.cuh"
#include "attn_plan.h"

namespace sffn {

template <> hipError_t launch_attn_rows_mx4<uint16_t>(const AttnMx4Args&, bool, hipStream_t);
template <> hipError_t launch_attn_rows_mx4<float>(const AttnMx4Args&, bool, hipStream_t);
template <> hipError_t launch_attn_keys_mx4<uint16_t>(const AttnMx4Args&, int, int, bool, bool, hipStream_t);
template <> hipError_t launch_attn_keys_mx4<float>(const AttnMx4Args&, int, int, bool, bool, hipStream_t);

namespace {

int tile_of(int dtype, const PagedAttn& p) {
  return keys_mx4_rows(dtype == 1 ? 2 : 4, p.D, p.max_q * (int64_t)(p.hq / p.hkv));
}
int waves_of(int dtype, const PagedAttn& p) {
  const int64_t g = p.hq / p.hkv, limit = keys_max(p), rows = p.max_q * g < limit ? p.max_q * g : limit;
  const int64_t tile = tile_of(dtype, p), tiles = (rows + tile - 1) / tile, groups = (int64_t)p.n_seqs * p.hkv;
  // A sequence of up to 32 rows has two tiles of 16 where it has one in attn_keys: a grid of
  // them with eight waves has 2^32 threads at half the sequences.  They get four from there on,
  // whose grid takes as many sequences as that of one tile with eight.
  if (tiles > 1 && groups * tiles * 8 * kWave >= 1ll << 32) return 4;
  return keys_mx4_waves(dtype == 1 ? 2 : 4, key_span(p, limit / g + 1));
}
Plan keys_of(int dtype, const PagedAttn& p) {
  const int step = waves_of(dtype, p) * 32, tile = tile_of(dtype, p);
  return plan_keys(p, dtype == 1 ? KeysTuning{step * 5, step * 2, step * 6, 4 * kCus, tile}
                                 : KeysTuning{step * 2, step, step, 4 * kCus, tile});
}
Plan rows_of(int dtype, const PagedAttn& p, const Plan& keys) {
  return plan_rows(p, keys.used, dtype == 1 ? 256 : 128);
}

template <typename T>
hipError_t launch(AttnMx4Args m, const Plan& keys, const Plan& rows, void* ws, hipStream_t s) {
  AttnArgs& a = m.a;
  const int dtype = sizeof(T) == 2 ? 1 : 0;
  // see RowPlace
  const Mx4Rows &k = m.k, &v = m.v;
  m.alike = k.page == v.page && k.token == v.token && k.s_page == v.s_page && k.s_token == v.s_token &&
            k.token < (1 << 24) && k.s_token < (1 << 24) && k.page < (1ll << 31) && k.s_page < (1ll << 31);
  const bool near = a.p.page_size % 16 == 0 && m.alike;
  hipError_t e = hipSuccess;
  if (rows.used) {
    place(&a, rows, (char*)ws + keys.bytes);
    e = launch_attn_rows_mx4<T>(m, near, s);
    if (e == hipSuccess) e = launch_join(dtype, kRowsTile, a, rows, s);
    if (e != hipSuccess) return e;
  }
  if (keys.used) {
    place(&a, keys, ws);
    m.tiles = FastDiv::make(a.tiles_per_seq);
    e = launch_attn_keys_mx4<T>(m, tile_of(dtype, a.p), waves_of(dtype, a.p), near, rows.used, s);
    if (e == hipSuccess) e = launch_join(dtype, kKeysTile, a, keys, s);
  }
  return e;
}

}  // namespace

bool plan_paged_attn_mx4(int dtype, const PagedAttn& p, size_t* bytes) {
  *bytes = 0;
  if (p.T == 0 || p.n_seqs == 0 || p.max_q == 0) return true;  // nothing is launched
  const Plan keys = keys_of(dtype, p), rows = rows_of(dtype, p, keys);
  if (!plan_fits(keys, rows, p, waves_of(dtype, p) * kWave)) return false;
  *bytes = keys.bytes + rows.bytes;
  return true;
}

hipError_t launch_paged_attn_mx4(int dtype, const PagedAttn& p, const Mx4Rows& k, const Mx4Rows& v,
                                 void* ws, hipStream_t stream) {
  const Plan keys = keys_of(dtype, p), rows = rows_of(dtype, p, keys);
  const AttnMx4Args m = {attn_args(p), k, v, FastDiv::make(p.hkv), {}, 0};
  return dtype == 1 ? launch<uint16_t>(m, keys, rows, ws, stream)
                    : launch<float>(m, keys, rows, ws, stream);
}

}  // namespace sffn
