// Attention of new tokens over a paged cache: which kernels a batch takes, how
// far its key ranges are split, the workspace of the splits.
#include <hip/hip_runtime.h>

#include "attn_plan.h"

namespace sffn {

template <> hipError_t launch_attn_rows<uint16_t>(const AttnArgs&, int, hipStream_t);
template <> hipError_t launch_attn_rows<float>(const AttnArgs&, int, hipStream_t);
template <> hipError_t launch_attn_keys<uint16_t>(const AttnArgs&, int, bool, hipStream_t);
template <> hipError_t launch_attn_keys<float>(const AttnArgs&, int, bool, hipStream_t);

namespace {

// A wave takes 1 to 2 us for 32 keys (3 us in float32, whose products are 16 times
// slower), the join and its launch 6 us: ranges of up to 5 (2) steps a wave
// are not split.  Longer ones into chunks of 2 (1) to 6 (1) steps: 6 even out
// ragged lengths better than 8 (32 tokens over up to 4096 keys 67.8 -> 63.8 us),
// fewer spread a few long ranges over the GPU.
Plan keys_of(int dtype, const PagedAttn& p) {
  const int step = attn_keys_waves(dtype == 1 ? 2 : 4, p.D) * 32;
  return plan_keys(p, dtype == 1 ? KeysTuning{step * 5, step * 2, step * 6, 4 * kCus, kKeysTile}
                                 : KeysTuning{step * 2, step, step, 4 * kCus, kKeysTile});
}
Plan rows_of(int dtype, const PagedAttn& p, const Plan& keys) {
  return plan_rows(p, keys.used, dtype == 1 ? 256 : 128);
}

template <typename T>
hipError_t launch(AttnArgs a, const Plan& keys, const Plan& rows, void* ws, hipStream_t s) {
  const int dtype = sizeof(T) == 2 ? 1 : 0;
  const PagedAttn& p = a.p;
  // see TileLoader: rows looked up together, lane offsets of less than 32 rows in
  // 32 bits.  Pages of 16: a 4096-token prompt 108 us, by 8 rows 112, row by row 121;
  // chunks beside single tokens 722, 737, 790.  Pages of 24: prompt 109 by 8 rows and 117
  // row by row (float32 chunks 84 and 81).
  const bool near = p.kc_token < (1 << 24) && p.vc_token < (1 << 24);
  const int granule = !near ? 0 : p.page_size % 16 == 0 ? 16 : p.page_size % 8 == 0 ? 8 : 0;
  hipError_t e = hipSuccess;
  if (rows.used) {
    place(&a, rows, (char*)ws + keys.bytes);
    e = launch_attn_rows<T>(a, granule, s);
    if (e != hipSuccess) return e;
    e = launch_join(dtype, kRowsTile, a, rows, s);
    if (e != hipSuccess) return e;
  }
  if (keys.used) {
    place(&a, keys, ws);
    // Beside attn_rows most of the tiles that the host counts are not there, so the items
    // are numbered on the device: chunks beside single tokens 713 us, with a workgroup for
    // each 721; 16 float32 sequences 88 and 98; but 5 float32 chunks 84 and 80.
    e = launch_attn_keys<T>(a, granule, rows.used, s);
    if (e != hipSuccess) return e;
    e = launch_join(dtype, kKeysTile, a, keys, s);
  }
  return e;
}

template <typename T>
void join(int tile_rows, bool early, const AttnArgs& a, dim3 grid, hipStream_t s) {
  if (tile_rows != kKeysTile) hipLaunchKernelGGL((attn_join<T, kRowsTile, false>), grid, dim3(256), 0, s, a);
  else if (early) hipLaunchKernelGGL((attn_join<T, kKeysTile, true>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((attn_join<T, kKeysTile, false>), grid, dim3(256), 0, s, a);
}

}  // namespace

hipError_t launch_attn_join(int dtype, int tile_rows, bool early, const AttnArgs& a, dim3 grid, hipStream_t s) {
  if (dtype == 1) join<uint16_t>(tile_rows, early, a, grid, s);
  else join<float>(tile_rows, early, a, grid, s);
  return hipGetLastError();
}

bool plan_paged_attn(int dtype, const PagedAttn& p, size_t* bytes) {
  *bytes = 0;
  if (p.T == 0 || p.n_seqs == 0 || p.max_q == 0) return true;  // nothing is launched
  const Plan keys = keys_of(dtype, p), rows = rows_of(dtype, p, keys);
  if (!plan_fits(keys, rows, p, attn_keys_waves(dtype == 1 ? 2 : 4, p.D) * kWave)) return false;
  *bytes = keys.bytes + rows.bytes;
  return true;
}

hipError_t launch_paged_attn(int dtype, const PagedAttn& p, void* ws, hipStream_t stream) {
  const Plan keys = keys_of(dtype, p), rows = rows_of(dtype, p, keys);
  const AttnArgs a = attn_args(p);
  return dtype == 1 ? launch<uint16_t>(a, keys, rows, ws, stream)
                    : launch<float>(a, keys, rows, ws, stream);
}

}  // namespace sffn
