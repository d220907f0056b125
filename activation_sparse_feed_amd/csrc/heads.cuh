// Rows of heads: how a row's elements lie over lanes, the norm and rotation of the forward.
// Shared by the kernels that write values and by those that quantise k and v.
#pragma once

#include <hip/hip_runtime.h>

#include "attn.h"
#include "common.cuh"

namespace sffn {

// V elements of a row as one load or store (V * sizeof(T) = 4, 8 or 16 bytes).
template <typename T, int V> struct Chunk {
  static constexpr int kBytes = V * (int)sizeof(T);
  typedef uint32_t raw_t __attribute__((ext_vector_type(kBytes / 4)));
  __device__ static __forceinline__ void unpack(const raw_t& w, float (&o)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if constexpr (sizeof(T) == 4) o[i] = __uint_as_float(w[i]);
      else o[i] = (i & 1) ? bf16hi(w[i / 2]) : bf16lo(w[i / 2]);
    }
  }
  __device__ static __forceinline__ void load(const T* p, float (&o)[V]) { unpack(*(const raw_t*)p, o); }
  __device__ static __forceinline__ void store(T* p, const float (&v)[V]) {
    raw_t r;
#pragma unroll
    for (int i = 0; i < kBytes / 4; ++i) {
      if constexpr (sizeof(T) == 4) r[i] = __float_as_uint(v[i]);
      else r[i] = (uint32_t)f32_to_bf16(v[2 * i]) | ((uint32_t)f32_to_bf16(v[2 * i + 1]) << 16);
    }
    *(raw_t*)p = r;
  }
};

// Sum over the G lanes of a row (G a power of two, the same for all lanes),
// every lane getting it: quad_perm [1,0,3,2] and [2,3,0,1], then mirrors
// within 8 and 16 lanes (after the quads agree a mirror is an exchange).
__device__ __forceinline__ float row_sum(float v, int G) {
  if (G >= 2) v += dpp_f32<0xB1>(v);
  if (G >= 4) v += dpp_f32<0x4E>(v);
  if (G >= 8) v += dpp_f32<0x141>(v);
  if (G >= 16) v += dpp_f32<0x140>(v);
  if (G >= 32) v += __shfl_xor(v, 16, kWave);
  if (G >= 64) v += __shfl_xor(v, 32, kWave);
  return v;
}

// 1 / sqrt(v) to 1 ulp.  The instruction takes a subnormal for 0, which would make
// infinities of rows whose mean square is below 2^-126 (elements of 1e-19 with eps = 0): such
// values are scaled by an even power of two first.
__device__ __forceinline__ float inverse_root(float v) {
  const bool tiny = v < 0x1p-96f;
  const float r = __builtin_amdgcn_rsqf(tiny ? v * 0x1p60f : v);
  return tiny ? r * 0x1p30f : r;
}

// The two chunks of this lane's unit u, element offsets o0 and o1 (o1 < 0:
// none), and whether the unit exists and is rotated across its chunks.
struct Unit {
  int o0, o1;
  bool live, pair;
};

template <int V>
__device__ __forceinline__ Unit unit_of(int u, int D, int rot, bool adjacent) {
  Unit r;
  if (adjacent) {  // two neighbouring chunks, pairs inside each
    r.o0 = 2 * u * V;
    r.o1 = r.o0 + V < D ? r.o0 + V : -1;
    r.live = r.o0 < D;
    r.pair = false;
    return r;
  }
  const int np = (rot / 2) / V;  // units of partner chunks, then the rest of the row
  if (u < np) {
    r.o0 = u * V;
    r.o1 = rot / 2 + u * V;
    r.live = r.pair = true;
  } else {
    r.o0 = rot + 2 * (u - np) * V;
    r.o1 = r.o0 + V < D ? r.o0 + V : -1;
    r.live = r.o0 < D;
    r.pair = false;
  }
  return r;
}

// n floats of a row of the table, 4-byte aligned.
template <int N>
__device__ __forceinline__ void load_floats(const float* p, float* o) {
  typedef float vec_t __attribute__((ext_vector_type(N < 4 ? N : 4), aligned(4)));
  constexpr int kStep = N < 4 ? N : 4;
#pragma unroll
  for (int i = 0; i < N; i += kStep) {
    const vec_t v = *(const vec_t*)(p + i);
#pragma unroll
    for (int j = 0; j < kStep; ++j) o[i + j] = v[j];
  }
}

// cos and sin of a unit's pairs: for pair units V angles; for adjacent pairs
// V / 2 angles of each chunk (1, 0 beyond rot).  A position outside the table
// gives NaN.  `pos` is the token's.
template <int V>
__device__ __forceinline__ void load_angles(const Unit& u, bool adjacent, const float* table,
                                            int rot, int max_pos, int pos, float (&c)[V],
                                            float (&s)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) c[i] = 1.f, s[i] = 0.f;
  if (rot == 0) return;
  const bool ok = pos >= 0 && pos < max_pos;
  const float* row = table + (size_t)(ok ? pos : 0) * rot;
  const float bad = __builtin_nanf("");
  if (adjacent) {
#pragma unroll
    for (int i = 0; i < V; ++i) {  // i < V/2: the first chunk's pairs, else the second's
      const int e = (i < V / 2 ? u.o0 : u.o1) + 2 * (i % (V / 2));
      const bool in = e < rot && (i < V / 2 || u.o1 >= 0);
      const int at = in ? e / 2 : 0;
      const float ci = row[at], si = row[rot / 2 + at];
      c[i] = !in ? 1.f : ok ? ci : bad;
      s[i] = !in ? 0.f : ok ? si : bad;
    }
  } else if (u.pair) {
    load_floats<V>(row + u.o0, c);
    load_floats<V>(row + rot / 2 + u.o0, s);
    if (!ok) {
#pragma unroll
      for (int i = 0; i < V; ++i) c[i] = s[i] = bad;
    }
  }
}

// The position of token t, one for the wave: a scalar load.
__device__ __forceinline__ int position_of(const int32_t* positions, int rot, int t) {
  return rot == 0 ? 0 : *(const __attribute__((address_space(4))) int32_t*)(positions + t);
}

// Rotation of a unit in place; `sign` -1 applies the transposed rotation.
template <int V>
__device__ __forceinline__ void rotate(const Unit& u, bool adjacent, const float (&c)[V],
                                       const float (&s)[V], float sign, float (&a)[V],
                                       float (&b)[V]) {
  if (adjacent) {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      float p = a[2 * i], q = a[2 * i + 1];
      a[2 * i] = p * c[i] - sign * q * s[i];
      a[2 * i + 1] = q * c[i] + sign * p * s[i];
      p = b[2 * i], q = b[2 * i + 1];
      b[2 * i] = p * c[V / 2 + i] - sign * q * s[V / 2 + i];
      b[2 * i + 1] = q * c[V / 2 + i] + sign * p * s[V / 2 + i];
    }
  } else if (u.pair) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float p = a[i], q = b[i];
      a[i] = p * c[i] - sign * q * s[i];
      b[i] = q * c[i] + sign * p * s[i];
    }
  }
}

template <typename T, int V>
__device__ __forceinline__ void load_unit(const T* row, const Unit& u, float (&a)[V],
                                          float (&b)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) a[i] = b[i] = 0.f;
  if (u.live) Chunk<T, V>::load(row + u.o0, a);
  if (u.live && u.o1 >= 0) Chunk<T, V>::load(row + u.o1, b);
}

template <typename T, int V>
__device__ __forceinline__ void store_unit(T* row, const Unit& u, const float (&a)[V],
                                           const float (&b)[V]) {
  if (u.live) Chunk<T, V>::store(row + u.o0, a);
  if (u.live && u.o1 >= 0) Chunk<T, V>::store(row + u.o1, b);
}

// A unit's weights as they lie in memory (w null: ones).
template <typename T, int V> struct RawWeight {
  typename Chunk<T, V>::raw_t a, b;
  __device__ __forceinline__ void load(const T* w, const Unit& u) {
    constexpr uint32_t one = sizeof(T) == 4 ? 0x3f800000u : 0x3f803f80u;
#pragma unroll
    for (int i = 0; i < Chunk<T, V>::kBytes / 4; ++i) a[i] = b[i] = one;
    if (w != nullptr && u.live) {
      a = *(const typename Chunk<T, V>::raw_t*)(w + u.o0);
      if (u.o1 >= 0) b = *(const typename Chunk<T, V>::raw_t*)(w + u.o1);
    }
  }
};

constexpr int kHeadsBlock = 256;

// Part `part` of a token's heads, by one wave: the rows of q, then of k, then (to
// a cache) of v, 64 / G at a time.
// Q: of q alone.
template <typename T, int V, bool Q = false>
__device__ __forceinline__ void heads_fwd_part(const HeadsFwd& p, int t, int part) {
  const int lane = lane_id();
  const int G = p.lanes_per_row, u = lane & (G - 1), sub = lane / G, rpw = kWave / G;
  const bool adjacent = p.rot_adjacent != 0;
  const Unit un = unit_of<V>(u, p.D, p.rot, adjacent);
  int64_t kc = (int64_t)t * p.ko_token, vc = 0;
  bool stored = true;
  if (!Q && p.slots != nullptr) {
    const int slot = p.slots[t];
    stored = slot >= 0 && (int64_t)slot < (int64_t)p.n_pages * p.page_size;
    const int page = stored ? slot / p.page_size : 0, off = stored ? slot % p.page_size : 0;
    kc = page * p.kc_page + off * p.ko_token;
    vc = page * p.vc_page + off * p.vc_token;
  }
  float c[V], s[V];
  load_angles<V>(un, adjacent, p.table, p.rot, p.max_pos, position_of(p.positions, p.rot, t), c, s);
  RawWeight<T, V> wq, wk;
  if (p.norm) {
    wq.load((const T*)p.q_weight, un);
    if (!Q) wk.load((const T*)p.k_weight, un);
  }
  const int n_v = p.slots != nullptr ? p.hkv : 0;
  const int rows = Q ? p.hq : p.hq + p.hkv + n_v;
  const float inv_d = 1.f / (float)p.D;
  for (int r0 = part * p.rows_per_wave; r0 < min(rows, (part + 1) * p.rows_per_wave);
       r0 += rpw) {
    const int r = r0 + sub;
    const bool in = r < rows;
    const bool is_q = Q || r < p.hq, is_k = !is_q && r < p.hq + p.hkv;
    const int h = is_q ? r : is_k ? r - p.hq : r - p.hq - p.hkv;
    const T* src = is_q ? (const T*)p.q + t * p.q_token + h * p.q_head
                 : is_k ? (const T*)p.k + t * p.k_token + h * p.k_head
                        : (const T*)p.v + t * p.v_token + h * p.v_head;
    T* dst = is_q ? (T*)p.q_out + t * p.qo_token + h * p.qo_head
           : is_k ? (T*)p.k_out + kc + h * p.ko_head
                  : (T*)p.v_out + vc + h * p.vc_head;
    Unit me = un;
    me.live = me.live && in && (is_q || stored);
    float a[V], b[V];
    load_unit<T, V>(src, me, a, b);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) ss += a[i] * a[i] + b[i] * b[i];
    ss = row_sum(ss, G);
    if (is_q || is_k) {
      if (p.norm) {
        const float rs = inverse_root(ss * inv_d + p.eps);
        float wa[V], wb[V];
        Chunk<T, V>::unpack(is_q ? wq.a : wk.a, wa);
        Chunk<T, V>::unpack(is_q ? wq.b : wk.b, wb);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          a[i] = a[i] * rs * wa[i];
          b[i] = b[i] * rs * wb[i];
        }
      }
      rotate<V>(un, adjacent, c, s, 1.f, a, b);
    }
    store_unit<T, V>(dst, me, a, b);
  }
}

// Elements per chunk: the widest load of at most 16 bytes whose chunks hold
// whole partners (pairs (i, i + rot/2) need V to divide rot/2; head_dim and
// rot_dim are multiples of 8 and 4).
inline int chunk_elements(int dtype, int rot, bool adjacent) {
  const int widest = dtype == 1 ? 8 : 4;
  if (adjacent || rot == 0) return widest;
  int v = widest;
  while ((rot / 2) % v != 0) v /= 2;
  return v;
}

inline int lanes_per_row(int D, int rot, bool adjacent, int V) {
  int units;
  if (adjacent) units = (D / V + 1) / 2;
  else units = rot / 2 / V + ((D - rot) / V + 1) / 2;
  int g = 1;
  while (g < units) g *= 2;
  return g;  // at most 64: head_dim <= 256 and V >= 2
}

}  // namespace sffn
