// Attention of new tokens over a paged cache.
#include <hip/hip_runtime.h>

#include "attn.h"
#include "common.cuh"

namespace sffn {

namespace {

// One wave per (token, query head), 64 keys at a time: each lane the score of
// one key, then each lane up to four output elements over the 64 keys.
template <typename T>
__global__ __launch_bounds__(64) void attn_simple(PagedAttn p) {
  const int lane = lane_id();
  const int t = blockIdx.x, h = blockIdx.y;
  // the sequence that owns row t
  int s = -1, q0 = 0, q1 = 0;
  for (int i = 0; i < p.n_seqs; ++i) {
    const int a = max(0, p.q_start[i]), b = min(p.T, p.q_start[i + 1]);
    if (t >= a && t < b) {
      s = i, q0 = a, q1 = b;
      break;
    }
  }
  if (s < 0) return;
  const int nkv = max(0, min(min(p.kv_len[s], p.max_kv), p.max_pages * p.page_size));
  const int pos = nkv - (q1 - q0) + (t - q0);
  const int hi = p.causal ? min(nkv, pos + 1) : nkv;
  const int lo = p.window > 0 ? max(0, pos - p.window + 1) : 0;
  const int hk = h / (p.hq / p.hkv);
  const int32_t* bt = p.block_table + (size_t)s * p.max_pages;
  __shared__ float qs[256];
  for (int d = lane; d < p.D; d += kWave)
    qs[d] = Elt<T>::load1(p.q, (size_t)(t * p.q_token + h * p.q_head + d)) * p.scale;
  __syncthreads();
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int j0 = lo; j0 < hi; j0 += kWave) {
    const int j = j0 + lane;
    float sc = -INFINITY;
    if (j < hi) {
      const int page = min(max(bt[j / p.page_size], 0), p.n_pages - 1);
      const size_t at = (size_t)(page * p.kc_page + (j % p.page_size) * p.kc_token + hk * p.kc_head);
      sc = 0.f;
      for (int d = 0; d < p.D; d += Elt<T>::kPerChunk) {
        float k[Elt<T>::kPerChunk];
        Elt<T>::unpack(ldg16((const T*)p.k_cache + at + d), k);
#pragma unroll
        for (int i = 0; i < Elt<T>::kPerChunk; ++i) sc += k[i] * qs[d + i];
      }
    }
    float mx = sc;
#pragma unroll
    for (int x = 32; x >= 1; x >>= 1) mx = fmaxf(mx, __shfl_xor(mx, x, kWave));
    const float mn = fmaxf(m, mx);
    const float base = mn == -INFINITY ? 0.f : mn;
    const float f = __expf(m - base), w = __expf(sc - base);
    l = l * f + wave_sum(w);
    m = mn;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] *= f;
    const int n = min(kWave, hi - j0);
    for (int k = 0; k < n; ++k) {
      const int jj = j0 + k;
      const float wk = __shfl(w, k, kWave);
      const int page = min(max(bt[jj / p.page_size], 0), p.n_pages - 1);
      const size_t at = (size_t)(page * p.vc_page + (jj % p.page_size) * p.vc_token + hk * p.vc_head);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int d = lane + i * kWave;
        if (d < p.D) o[i] += wk * Elt<T>::load1(p.v_cache, at + d);
      }
    }
  }
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int d = lane + i * kWave;
    if (d < p.D) Elt<T>::store1(p.out, (size_t)(t * p.o_token + h * p.o_head + d), o[i] * inv);
  }
  if (p.lse != nullptr && lane == 0) p.lse[(size_t)t * p.hq + h] = l == 0.f ? -INFINITY : m + __logf(l);
}

}  // namespace

size_t paged_attn_workspace(int dtype, const PagedAttn& p) { return 0; }

hipError_t launch_paged_attn(int dtype, const PagedAttn& p, void* ws, hipStream_t stream) {
  const dim3 grid((unsigned)p.T, (unsigned)p.hq);
  if (dtype == 1) hipLaunchKernelGGL(attn_simple<uint16_t>, grid, dim3(64), 0, stream, p);
  else hipLaunchKernelGGL(attn_simple<float>, grid, dim3(64), 0, stream, p);
  return hipGetLastError();
}

}  // namespace sffn
