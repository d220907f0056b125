// Heads of q and k: per-head RMS norm and position rotation, forward and
// backward, and the forward that stores k and v in a paged cache.
//
// Every row (one head of one token) is a few hundred bytes, so these kernels
// are bound by HBM: each element is read and written once, in 16-byte chunks
// where the pairing of the rotation allows it.  At 16384 tokens of 32 + 8 heads of
// 128, bf16: forward 68 us for 344 MB (5.0 TB/s; a large copy runs at 4.8),
// backward 110 us for 512 MB (4.7 TB/s), append 82 us for 408 MB.  A decode step
// of 32 tokens takes 4.4 us, the latency of its dependent loads.  In float32, 4000
// tokens of the same heads: forward 38 us (4.4 TB/s), append 45 us (4.5 TB/s), backward
// 56 us (4.5 TB/s).  A row is held by G lanes
// (a power of two), each with two chunks of V elements: for pairs
// (i, i + rot/2) the chunks that are partners of each other, so that the
// rotation needs no data of other lanes; a wave holds 64 / G rows of one
// token, and the angles of the token's position stay in registers while it
// walks over the token's heads.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "attn.h"
#include "common.cuh"
#include "heads.cuh"

namespace sffn {

namespace {

template <typename T, int V>
__global__ __launch_bounds__(kHeadsBlock) void heads_fwd(HeadsFwd p) {
  const int t = uniform((int)(blockIdx.x * (kHeadsBlock / kWave) + threadIdx.x / kWave));
  if (t >= p.T) return;
  heads_fwd_part<T, V>(p, t, (int)blockIdx.y);
}

// A row's part of this lane as it lies in memory, x and the gradient.
template <typename T, int V> struct RawRow {
  typename Chunk<T, V>::raw_t x0, x1, g0, g1;
};

// Backward: one wave walks over tokens; the weight gradients of its unit stay in
// registers and are summed over the block's waves at the end, in a fixed order,
// into one row of partials per block.  The next rows are loaded before a row's
// arithmetic, so that loads are in flight all the time.
template <typename T, int V>
__global__ __launch_bounds__(kHeadsBlock) void heads_bwd(HeadsBwd p) {
  typedef Chunk<T, V> C;
  const int lane = lane_id(), w = threadIdx.x / kWave;
  const int G = p.lanes_per_row, u = lane & (G - 1), sub = lane / G, rpw = kWave / G;
  const bool adjacent = p.rot_adjacent != 0;
  const Unit un = unit_of<V>(u, p.D, p.rot, adjacent);
  const float inv_d = 1.f / (float)p.D;
  const bool has1 = un.live && un.o1 >= 0;
  float gw[2][2][V];
#pragma unroll
  for (int i = 0; i < V; ++i) gw[0][0][i] = gw[0][1][i] = gw[1][0][i] = gw[1][1][i] = 0.f;
  const int waves = (int)gridDim.x * (kHeadsBlock / kWave);
  RawWeight<T, V> weight[2];
  if (p.norm) {
    weight[0].load((const T*)p.q_weight, un);
    weight[1].load((const T*)p.k_weight, un);
  }

  auto load = [&](int which, int t, int h0) __attribute__((always_inline)) {
    RawRow<T, V> r = {};
    const int h = h0 + sub;
    if (!un.live || t >= p.T || h >= (which == 0 ? p.hq : p.hkv)) return r;
    const T* x = (const T*)(which == 0 ? p.q : p.k) +
                 (which == 0 ? t * p.q_token + h * p.q_head : t * p.k_token + h * p.k_head);
    const T* g = (const T*)(which == 0 ? p.gq_out : p.gk_out) +
                 (which == 0 ? t * p.gqo_token + h * p.gqo_head : t * p.gko_token + h * p.gko_head);
    if (p.norm) {
      r.x0 = *(const typename C::raw_t*)(x + un.o0);
      if (has1) r.x1 = *(const typename C::raw_t*)(x + un.o1);
    }
    r.g0 = *(const typename C::raw_t*)(g + un.o0);
    if (has1) r.g1 = *(const typename C::raw_t*)(g + un.o1);
    return r;
  };
  auto process = [&](auto which_c, const RawRow<T, V>& raw, int t, int h0, const float (&c)[V],
                     const float (&s)[V]) __attribute__((always_inline)) {
    constexpr int which = decltype(which_c)::value;
    const int h = h0 + sub, heads = which == 0 ? p.hq : p.hkv;
    Unit me = un;
    me.live = me.live && h < heads;
    float ga[V], gb[V];
    C::unpack(raw.g0, ga);
    C::unpack(raw.g1, gb);
    rotate<V>(un, adjacent, c, s, -1.f, ga, gb);
    if (p.norm) {
      float wa[V], wb[V], a[V], b[V];
      C::unpack(weight[which].a, wa);
      C::unpack(weight[which].b, wb);
      C::unpack(raw.x0, a);
      C::unpack(raw.x1, b);
      float ss = 0.f, dot = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        ss += a[i] * a[i] + b[i] * b[i];
        dot += ga[i] * wa[i] * a[i] + gb[i] * wb[i] * b[i];
      }
      ss = row_sum(ss, G);
      dot = row_sum(dot, G);
      const float rs = inverse_root(ss * inv_d + p.eps);
      const float m = dot * rs * inv_d;  // mean of (gn w) xhat
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float ha = a[i] * rs, hb = b[i] * rs;
        if (h < heads) {
          gw[which][0][i] += ga[i] * ha;
          gw[which][1][i] += gb[i] * hb;
        }
        ga[i] = rs * (ga[i] * wa[i] - ha * m);
        gb[i] = rs * (gb[i] * wb[i] - hb * m);
      }
    }
    T* gx = which == 0 ? (T*)p.gq + t * p.gq_token + h * p.gq_head : (T*)p.gk + t * p.gk_token + h * p.gk_head;
    store_unit<T, V>(gx, me, ga, gb);
  };

  int t = uniform((int)blockIdx.x * (kHeadsBlock / kWave) + w);
  float c[V], s[V];
  RawRow<T, V> row = load(p.hq > 0 ? 0 : 1, t, 0);
  if (t < p.T) load_angles<V>(un, adjacent, p.table, p.rot, p.max_pos, position_of(p.positions, p.rot, t), c, s);
  for (; t < p.T; t += waves) {
    const int tn = t + waves;
    const int pos_next = position_of(p.positions, p.rot, min(tn, p.T - 1));
    float cn[V], sn[V];
    for (int h0 = 0; h0 < p.hq; h0 += rpw) {
      const bool more = h0 + rpw < p.hq, k = p.hkv > 0;
      const RawRow<T, V> next = load(more || !k ? 0 : 1, more || k ? t : tn, more ? h0 + rpw : 0);
      process(std::integral_constant<int, 0>{}, row, t, h0, c, s);
      row = next;
    }
    load_angles<V>(un, adjacent, p.table, p.rot, p.max_pos, pos_next, cn, sn);
    for (int h0 = 0; h0 < p.hkv; h0 += rpw) {
      const bool more = h0 + rpw < p.hkv, q = p.hq > 0;
      const RawRow<T, V> next = load(more || !q ? 1 : 0, more ? t : tn, more ? h0 + rpw : 0);
      process(std::integral_constant<int, 1>{}, row, t, h0, c, s);
      row = next;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = cn[i], s[i] = sn[i];
  }
  if (p.partial == nullptr) return;
  // sum over the rows a wave holds side by side, then over the block's waves
  __shared__ float red[kHeadsBlock / kWave][2][256];
#pragma unroll
  for (int which = 0; which < 2; ++which)
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float v = gw[which][half][i];
        for (int o = G; o < kWave; o <<= 1) v += __shfl_xor(v, o, kWave);
        const int at = half == 0 ? un.o0 : un.o1;
        if (sub == 0 && un.live && at >= 0) red[w][which][at + i] = v;
      }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * p.D; i += kHeadsBlock) {
    const int which = i / p.D, d = i % p.D;
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < kHeadsBlock / kWave; ++k) v += red[k][which][d];
    p.partial[(size_t)blockIdx.x * 2 * p.D + i] = v;
  }
}

// Column sums of the partials, n rows of 2 D: 8 columns per workgroup, 32 threads
// a column, in a fixed order.
__global__ __launch_bounds__(256) void heads_gw_reduce(const float* __restrict__ part, int n, int D,
                                                       float* gq_weight, float* gk_weight) {
  __shared__ float red[32][9];
  const int c = threadIdx.x & 7, row = threadIdx.x >> 3, col = (int)blockIdx.x * 8 + c;  // 2 D % 8 == 0
  float v = 0.f;
#pragma unroll 8
  for (int i = row; i < n; i += 32) v += part[(size_t)i * 2 * D + col];
  red[row][c] = v;
  __syncthreads();
  if (row == 0) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += red[i][c];
    float* out = col < D ? gq_weight : gk_weight;
    if (out != nullptr) out[col % D] = t;
  }
}

// Blocks of the backward: two waves a SIMD, which is what the registers of the instance
// with the widest chunks allow (197), all resident at once.  512 / 768 / 1024 blocks, in us:
// 16384 bf16 tokens of 32 + 8 heads of 128 115 / 135 / 121, of 16 + 4 of 80 with
// adjacent pairs 73 / 93 / 82, 4000 float32 tokens of 32 + 8 of 128 57 / 61 / 62.  Instances
// of narrower chunks hold four waves a SIMD and lose by it: bf16, 80 wide, 40 rotated
// 65 / 53 / 49, float32, 80 wide, 40 rotated in adjacent pairs 83 / 74 / 73.  One pass a
// wave for few tokens took 1.4 us off 33 tokens (19.1), but added 6 us at 16384.
int bwd_blocks(int T) {
  const int need = (T + kHeadsBlock / kWave - 1) / (kHeadsBlock / kWave);
  return need < 512 ? need : 512;
}

template <template <typename, int> class F, typename P>
hipError_t by_type(int dtype, int V, P p, dim3 grid, hipStream_t stream) {
  if (dtype == 1) {
    if (V == 8) return F<uint16_t, 8>::go(p, grid, stream);
    if (V == 4) return F<uint16_t, 4>::go(p, grid, stream);
    return F<uint16_t, 2>::go(p, grid, stream);
  }
  if (V == 4) return F<float, 4>::go(p, grid, stream);
  return F<float, 2>::go(p, grid, stream);
}

template <typename T, int V> struct Fwd {
  static hipError_t go(const HeadsFwd& p, dim3 grid, hipStream_t stream) {
    hipLaunchKernelGGL((heads_fwd<T, V>), grid, dim3(kHeadsBlock), 0, stream, p);
    return hipGetLastError();
  }
};
template <typename T, int V> struct Bwd {
  static hipError_t go(const HeadsBwd& p, dim3 grid, hipStream_t stream) {
    hipLaunchKernelGGL((heads_bwd<T, V>), grid, dim3(kHeadsBlock), 0, stream, p);
    return hipGetLastError();
  }
};

}  // namespace

hipError_t launch_heads_fwd(int dtype, HeadsFwd p, hipStream_t stream) {
  const int V = chunk_elements(dtype, p.rot, p.rot_adjacent != 0);
  p.lanes_per_row = lanes_per_row(p.D, p.rot, p.rot_adjacent != 0, V);
  const int rpw = kWave / p.lanes_per_row;
  const int rows = p.hq + p.hkv + (p.slots != nullptr ? p.hkv : 0);
  const int passes = (rows + rpw - 1) / rpw;
  // few tokens: a wave for every pass over a token's heads, so that the rows
  // of a decode step are read side by side; many: one wave per token, which
  // keeps the angles.  A wave for every pass / one per token, in us: norm of 32 + 8 heads
  // of 128, bf16, 256 tokens 3.9 / 7.5, 1024 7.2 / 9.8, 2047 10.6 / 11.1, 4096 22.0 / 20.8,
  // 16384 80.5 / 69.0; append 32 tokens 3.6 / 7.9, 4096 26.8 / 25.5; float32, 16 + 4 heads of
  // 80, 512 tokens 3.9 / 5.7, 4096 13.1 / 11.5; but 32 + 8 of 128, 4000 37.2 / 37.9
  const int per_wave = p.T < 2048 ? 1 : passes;
  p.rows_per_wave = per_wave * rpw;
  const dim3 grid((unsigned)((p.T + 3) / 4), (unsigned)((passes + per_wave - 1) / per_wave));
  return by_type<Fwd>(dtype, V, p, grid, stream);
}

size_t heads_bwd_partial_bytes(int T, int D) { return (size_t)bwd_blocks(T) * 2 * D * 4; }

hipError_t launch_heads_bwd(int dtype, HeadsBwd p, bool weights, float* gq_weight,
                            float* gk_weight, hipStream_t stream) {
  if (!weights) p.partial = nullptr;
  const int V = chunk_elements(dtype, p.rot, p.rot_adjacent != 0);
  p.lanes_per_row = lanes_per_row(p.D, p.rot, p.rot_adjacent != 0, V);
  const int n = bwd_blocks(p.T);
  if (n > 0) {
    const hipError_t e = by_type<Bwd>(dtype, V, p, dim3((unsigned)n), stream);
    if (e != hipSuccess) return e;
  }
  if (!weights) return hipSuccess;
  hipLaunchKernelGGL(heads_gw_reduce, dim3((unsigned)(2 * p.D / 8)), dim3(256), 0, stream,
                     p.partial, n, p.D, gq_weight, gk_weight);
  return hipGetLastError();
}

}  // namespace sffn
