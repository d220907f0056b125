// Writing keys and values into the 4-bit paged cache, and reading them back.
//
// heads_mx4: a wave takes a token's heads of q (as in heads_fwd) or of k and v.  At 16384
// tokens of 32 + 8 heads of 128, bf16: 71 to 77 us for 362 MB (4.7 to 5.1 TB/s; a large copy
// runs at 4.9).  q waits for memory, k and v are arithmetic (about 31 of 55 us of it), so
// both run side by side: one after the other took 89 us.  Those are normed heads: keys that
// lie right on borders between codes take 64 bits (see KeyRotation), up to 205 us where all are
// zero, 114 for bf16 heads rotated by half without a norm (91 with one).  32 tokens 4.9 us,
// dependent loads (position, angles) and code that is fetched once.  mx4_read: 18 us for 85 MB (4.7
// TB/s), 3.6 us for 77 rows.
#include <hip/hip_runtime.h>

#include "attn.h"
#include "common.cuh"
#include "heads.cuh"
#include "mx4.cuh"

namespace sffn {

namespace {

// A lane holds eight neighbouring elements of a row of k or v, four lanes a block.
constexpr int kPiece = 8;

// As they lie in memory.
template <typename T> struct Piece {
  static constexpr int kChunks = kPiece / Elt<T>::kPerChunk;
  u32x4_t c[kChunks];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kChunks; ++i) c[i] = ldg16(p + i * Elt<T>::kPerChunk);
  }
  __device__ __forceinline__ void fill(uint32_t w) {
#pragma unroll
    for (int i = 0; i < kChunks; ++i) c[i] = u32x4_t{w, w, w, w};
  }
  __device__ __forceinline__ void unpack(float (&o)[kPiece]) const {
#pragma unroll
    for (int i = 0; i < kChunks; ++i) Elt<T>::unpack(c[i], o + i * Elt<T>::kPerChunk);
  }
};

// A value at a uniform address that no kernel writes while this one runs: a scalar load.
__device__ __forceinline__ int load_once(const int32_t* p) {
  return *(const __attribute__((address_space(4))) int32_t*)p;
}

// Sum over the G lanes of a row (G at least 4), every lane getting the same.
__device__ __forceinline__ double row_sum64(double v, int G) {
  for (int o = 1; o < G; o <<= 1) v += __shfl_xor(v, o, kWave);
  return v;
}

// Norm and rotation of k for a lane's elements: r (x a + y b), where y is the partner in a
// rotated pair and a, b hold the angles and weights of x and y.  The partner is the
// neighbour (adjacent pairs) or is read once more, V elements at a time (V divides rot / 2).
//
// What is quantised is the 64-bit result rounded to float32: the codes of a token then do not
// hang on which kernel, order of sums or chunk of a prompt wrote it, and a value next to the
// border between two codes falls on its own side.  In float32 the result is off by less than
// 24 * 2^-24 of r (|x a| + |y b|): the sum of squares by 14 units of 2^-24 (8 products of a lane,
// up to 5 steps over the lanes), the mean and eps by 3, their inverse root r by half of that and
// 2, the rest by 4; and where numbers are subnormal by 2^-149 r and, since |r x| <= 16, by
// 2^-146 besides.  So a wave takes 64 bits only where that leaves a scale, a code or a sign
// open, or where the mean square is near the ends of float32.  (All of k in 64 bits took
// 131 us for 16384 tokens of 32 + 8 heads of 128, most of it conversions: now 77.)  That is
// under 1% of the waves with a norm; but the bound is one for a lane's elements, exact ones
// too: a zero has an open sign, and what is copied (from rot on without a norm) is, in bf16, often
// right on a border, so that most waves of such heads take 64 bits.
template <typename T, int V> struct KeyRotation {
  float a[kPiece], b[kPiece];
  int other[kPiece / V];  // partners of V elements, from the row's start

  __device__ __forceinline__ void init(const HeadsFwd& p, int at, bool live) {
#pragma unroll
    for (int i = 0; i < kPiece / V; ++i) {
      const int e = at + i * V, half = p.rot / 2;
      other[i] = !live ? 0 : p.rot_adjacent || e >= p.rot ? e : e < half ? e + half : e - half;
    }
  }
  // cos and +-sin of the elements' angles.
  __device__ __forceinline__ void load_angles(const HeadsFwd& p, int at, bool live, int pos) {
    const bool known = p.rot == 0 || (pos >= 0 && pos < p.max_pos);
    const int half = p.rot / 2;
    const float* angles = p.table + (size_t)(known ? pos : 0) * p.rot;
#pragma unroll
    for (int i = 0; i < kPiece / V; ++i) {
      const int e = at + i * V;
      if (p.rot > 0 && !p.rot_adjacent) {
        const int angle = !live || e >= p.rot ? 0 : e < half ? e : e - half;
        const uint32_t sign = e < half ? 0x80000000u : 0u;
        load_floats<V>(angles + angle, a + i * V);
        load_floats<V>(angles + half + angle, b + i * V);
#pragma unroll
        for (int j = 0; j < V; ++j) b[i * V + j] = __uint_as_float(__float_as_uint(b[i * V + j]) ^ sign);
      }
    }
    if (p.rot > 0 && p.rot_adjacent) {
#pragma unroll
      for (int i = 0; i < kPiece; i += 4) {  // rot is a multiple of 4
        const int angle = live && at + i < p.rot ? (at + i) / 2 : 0;
        float c[2], s[2];
        load_floats<2>(angles + angle, c);
        load_floats<2>(angles + half + angle, s);
#pragma unroll
        for (int j = 0; j < 4; ++j) a[i + j] = c[j / 2], b[i + j] = j & 1 ? s[j / 2] : -s[j / 2];
      }
    }
    if (p.rot != p.D || !known) {
#pragma unroll
      for (int i = 0; i < kPiece; ++i) {
        const bool in = at + i < p.rot;
        a[i] = !in ? 1.f : known ? a[i] : __builtin_nanf("");
        b[i] = !in ? 0.f : known ? b[i] : __builtin_nanf("");
      }
    }
  }
  __device__ __forceinline__ void load_weights(const HeadsFwd& p, int at, bool live, Piece<T>& w, Piece<T>& pw) const {
    const T* kw = (const T*)p.k_weight;
    w.fill(sizeof(T) == 4 ? 0x3f800000u : 0x3f803f80u);
    pw = w;
    if (p.norm && kw != nullptr && live) {
      w.load(kw + at);
      load_partners(kw, pw);
    }
  }
  // Angles become angles times weights.
  __device__ __forceinline__ void weigh(const HeadsFwd& p, const Piece<T>& w, const Piece<T>& pw) {
    float x[kPiece], y[kPiece];
    w.unpack(x);
    pw.unpack(y);
#pragma unroll
    for (int i = 0; i < kPiece; ++i) {
      a[i] *= x[i];
      b[i] *= p.rot_adjacent ? x[i ^ 1] : y[i];
    }
  }
  __device__ __forceinline__ void load_partners(const T* row, Piece<T>& y) const {
    typedef typename Chunk<T, V>::raw_t raw_t;
#pragma unroll
    for (int i = 0; i < kPiece / V; ++i) {
      const raw_t r = *(const raw_t*)(row + other[i]);
#pragma unroll
      for (int j = 0; j < (int)sizeof(raw_t) / 4; ++j) {
        const int word = i * ((int)sizeof(raw_t) / 4) + j;
        y.c[word / 4][word % 4] = r[j];
      }
    }
  }
  // o: the result in float32; how far its elements may be off (infinite: nothing is known).
  __device__ __forceinline__ float apply(const HeadsFwd& p, int G, const Piece<T>& raw, const Piece<T>& partner,
                                         float (&o)[kPiece]) const {
    float x[kPiece], y[kPiece];
    raw.unpack(x);
    partner.unpack(y);
    float r = 1.f;
    bool sure = true;
    if (p.norm) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < kPiece; ++i) ss += x[i] * x[i];
      const float v = row_sum(ss, G) * (1.f / (float)p.D) + p.eps;
      sure = v >= 0x1p-96f && v <= 0x1p112f;
      r = inverse_root(v);
    }
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < kPiece; ++i) {
      const float n = x[i] * a[i], m = (p.rot_adjacent ? x[i ^ 1] : y[i]) * b[i];
      o[i] = (n + m) * r;
      most = fmaxf(most, __builtin_fabsf(n) + __builtin_fabsf(m));
    }
    return sure ? fmaxf(most * r * (24.f * 0x1p-24f), r * 0x1p-148f + 0x1p-145f) : INFINITY;
  }
  // The same in 64 bits, element by element from memory: what is rare keeps no registers
  // (unrolled it took 115 instead of 74, and 16384 tokens 86 us instead of 77).
  __device__ __forceinline__ void apply64(const HeadsFwd& p, int G, const T* row, int at, bool live, int pos,
                                          float (&o)[kPiece]) const {
    double r = 1.0;
    if (p.norm) {
      double ss = 0.0;
      if (live) {
#pragma unroll 4
        for (int i = 0; i < kPiece; ++i) {
          const double x = Elt<T>::load1(row, at + i);
          ss += x * x;
        }
      }
      r = 1.0 / __builtin_sqrt(row_sum64(ss, G) / p.D + (double)p.eps);
    }
    if (!live) return;
    const T* kw = (const T*)p.k_weight;
    const bool weighted = p.norm && kw != nullptr;
    const bool known = pos >= 0 && pos < p.max_pos;
    const float* angles = p.table + (size_t)(known ? pos : 0) * p.rot;
    const int half = p.rot / 2;
#pragma unroll 2
    for (int i = 0; i < kPiece; ++i) {
      const int e = at + i;
      double n = (double)Elt<T>::load1(row, e) * r;
      if (weighted) n *= (double)Elt<T>::load1(kw, e);
      if (e < p.rot) {
        const bool first = p.rot_adjacent ? (e & 1) == 0 : e < half;
        const int q = p.rot_adjacent ? e ^ 1 : first ? e + half : e - half;
        const int angle = p.rot_adjacent ? e / 2 : first ? e : q;
        double m = (double)Elt<T>::load1(row, q) * r;
        if (weighted) m *= (double)Elt<T>::load1(kw, q);
        n = n * (double)angles[angle] + (first ? -m : m) * (double)angles[half + angle];
        if (!known) n = __builtin_nan("");
      }
#pragma unroll
      for (int j = 0; j < kPiece; ++j) o[j] = i == j ? (float)n : o[j];
    }
  }
};

// The largest magnitude's bits of a block: over the four lanes that share it.
__device__ __forceinline__ uint32_t block_top(const float (&e)[kPiece]) {
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < kPiece; ++j) top = max(top, __float_as_uint(e[j]) & 0x7fffffffu);
  top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0xB1, 0xf, 0xf, false));
  return max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0x4E, 0xf, 0xf, false));
}

// A row's part of a lane into the cache; codes and scales: of its block's row.
__device__ __forceinline__ void store_block(uint8_t* codes, uint8_t* scales, const float (&e)[kPiece], int u,
                                            bool live) {
  const uint32_t b = mx_scale_byte(block_top(e));
  if (!live) return;
  *(uint32_t*)(codes + u * 4) = b == 255 ? 0u : mx_encode8(e, mx_scale(b));
  if ((u & 3) == 0) scales[u / 4] = (uint8_t)b;
}

// Rows of k and v of token t into the cache, from key head h0 on, kGroups times 64 / G heads,
// G lanes a row.  All loads of a wave are under way before its arithmetic.
template <typename T, int V, int kGroups>
__device__ __forceinline__ void store_rows(const HeadsFwd& p, const Mx4Rows& kc, const Mx4Rows& vc, int t, int h0,
                                           int G) {
  const int lane = lane_id(), u = lane & (G - 1), at = u * kPiece, rows = kWave / G, sub = lane / G;
  const int slot = load_once(p.slots + t);
  const int pos = position_of(p.positions, p.rot, t);
  const T* const k = (const T*)p.k + t * p.k_token + h0 * p.k_head + sub * p.k_head;
  const T* const v = (const T*)p.v + t * p.v_token + h0 * p.v_head + sub * p.v_head;
  const bool turns = p.norm || p.rot > 0;
  KeyRotation<T, V> rot;
  Piece<T> xk[kGroups], yk[kGroups], xv[kGroups];
  bool live[kGroups];
#pragma unroll
  for (int i = 0; i < kGroups; ++i) {
    live[i] = h0 + i * rows + sub < p.hkv && at < p.D;
    xk[i].fill(0u);
    xv[i].fill(0u);
    if (live[i]) {
      xk[i].load(k + i * rows * p.k_head + at);
      xv[i].load(v + i * rows * p.v_head + at);
    }
  }
  if (turns) {
    rot.init(p, at, at < p.D);
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      yk[i] = xk[i];
      if (live[i] && p.rot > 0 && !p.rot_adjacent) rot.load_partners(k + i * rows * p.k_head, yk[i]);
    }
    Piece<T> w, pw;
    rot.load_weights(p, at, at < p.D, w, pw);
    rot.load_angles(p, at, at < p.D, pos);
    rot.weigh(p, w, pw);
  }
  const bool stored = slot >= 0 && (int64_t)slot < (int64_t)p.n_pages * p.page_size;
  const int page = stored ? slot / p.page_size : 0, off = stored ? slot % p.page_size : 0;
  uint8_t* const k_codes = kc.codes + page * kc.page + off * kc.token + h0 * kc.head + sub * kc.head;
  uint8_t* const v_codes = vc.codes + page * vc.page + off * vc.token + h0 * vc.head + sub * vc.head;
  uint8_t* const k_scales = kc.scales + page * kc.s_page + off * kc.s_token + h0 * kc.s_head + sub * kc.s_head;
  uint8_t* const v_scales = vc.scales + page * vc.s_page + off * vc.s_token + h0 * vc.s_head + sub * vc.s_head;
#pragma unroll
  for (int i = 0; i < kGroups; ++i) {
    if (h0 + i * rows >= p.hkv) break;
    float e[kPiece];
    xv[i].unpack(e);
    store_block(v_codes + i * rows * vc.head, v_scales + i * rows * vc.s_head, e, u, live[i] && stored);
    xk[i].unpack(e);
    if (turns) {
      // the least and the most that the results can be give the same codes under one scale,
      // or this is done in 64 bits; what is not finite makes the bounds so, too
      float far = rot.apply(p, G, xk[i], yk[i], e), lo[kPiece], hi[kPiece];
      if (at >= p.D) {  // nothing of a row: 0 times an infinite r is not 0
        far = 0.f;
#pragma unroll
        for (int j = 0; j < kPiece; ++j) e[j] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < kPiece; ++j) lo[j] = e[j] - far, hi[j] = e[j] + far;
      far = fmaxf(far, dpp_f32<0xB1>(far));
      far = fmaxf(far, dpp_f32<0x4E>(far));
      const float top = __uint_as_float(block_top(e));
      const uint32_t b = mx_scale_byte(__float_as_uint(top + far));
      const float scale = mx_scale(b);
      const bool open = b == 255 || b != mx_scale_byte(__float_as_uint(fmaxf(top - far, 0.f))) ||
                        mx_encode8(lo, scale) != mx_encode8(hi, scale);
      if (__any(open && live[i])) rot.apply64(p, G, k + i * rows * p.k_head, at, live[i], pos, e);
    }
    store_block(k_codes + i * rows * kc.head, k_scales + i * rows * kc.s_head, e, u, live[i] && stored);
  }
}

// A token a wave: parts of q, then of k and v.  The parts of a token run side by side: those
// of q wait for memory, those of k and v are mostly arithmetic.
template <typename T, int V, int kGroups>
__global__ __launch_bounds__(kHeadsBlock) void heads_mx4(HeadsFwd p, Mx4Rows k, Mx4Rows v, int q_parts, int G) {
  const int group = (int)(blockIdx.z * gridDim.y + blockIdx.y);
  const int t = uniform(group * (kHeadsBlock / kWave) + (int)threadIdx.x / kWave);
  if (t >= p.T) return;
  const int part = (int)blockIdx.x, kv = part - q_parts;
  if (kv < 0) heads_fwd_part<T, V, true>(p, t, part);
  else store_rows<T, V, kGroups>(p, k, v, t, kv * kGroups * (kWave / G), G);
}

// Rows back as values: G lanes a row, eight elements of K and of V each.
template <typename T>
__global__ __launch_bounds__(256) void mx4_read(Mx4Read p, int G) {
  const int lane = lane_id(), u = lane & (G - 1), at = u * kPiece;
  const int64_t wave = (int64_t)blockIdx.x * (256 / kWave) + threadIdx.x / kWave;
  const int64_t r = wave * (kWave / G) + lane / G;  // row: token, head
  if (r >= (int64_t)p.T * p.hkv || at >= p.D) return;
  const int t = (int)(r / p.hkv), h = (int)(r - (int64_t)t * p.hkv);
  const int slot = p.slots[t];
  if (slot < 0 || (int64_t)slot >= (int64_t)p.n_pages * p.page_size) return;
  const int page = slot / p.page_size, off = slot % p.page_size;
  uint32_t w[2];
  uint32_t b[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (p.out[i] == nullptr) continue;
    const Mx4Rows& c = p.cache[i];
    w[i] = *(const uint32_t*)(c.codes + page * c.page + off * c.token + h * c.head + u * 4);
    b[i] = c.scales[page * c.s_page + off * c.s_token + h * c.s_head + u / 4];
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (p.out[i] == nullptr) continue;
    u32x4_t x[Mx<T>::kChunks];
    Mx<T>::decode8(w[i], mx_scale(b[i]), x);
    T* o = (T*)p.out[i] + t * p.o_token[i] + h * p.o_head[i] + at;
#pragma unroll
    for (int j = 0; j < Mx<T>::kChunks; ++j) *(u32x4_t*)(o + j * Elt<T>::kPerChunk) = x[j];
  }
}

template <typename T, int V>
hipError_t append(const HeadsFwd& p, const Mx4Rows& k, const Mx4Rows& v, int q_parts, int G, int groups,
                  dim3 grid, hipStream_t stream) {
  if (groups == 1)
    hipLaunchKernelGGL((heads_mx4<T, V, 1>), grid, dim3(kHeadsBlock), 0, stream, p, k, v, q_parts, G);
  else
    hipLaunchKernelGGL((heads_mx4<T, V, 2>), grid, dim3(kHeadsBlock), 0, stream, p, k, v, q_parts, G);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_heads_mx4(int dtype, HeadsFwd p, Mx4Rows k, Mx4Rows v, hipStream_t stream) {
  const int V = chunk_elements(dtype, p.rot, p.rot_adjacent != 0);
  p.lanes_per_row = lanes_per_row(p.D, p.rot, p.rot_adjacent != 0, V);
  const int rpw = kWave / p.lanes_per_row, q_passes = (p.hq + rpw - 1) / rpw;
  // q as in the append without quantisation: few tokens, a wave for every pass
  const int q_each = p.T < 2048 ? 1 : q_passes;
  p.rows_per_wave = q_each * rpw;
  const int q_parts = p.hq == 0 ? 0 : (q_passes + q_each - 1) / q_each;
  int G = 4;  // lanes of a row of k or v: whole blocks
  while (G * kPiece < p.D) G *= 2;
  // k and v: few tokens, a wave for every 64 / G heads, too
  const int n = p.T < 2048 ? 1 : 2, heads = n * kWave / G, fours = (p.T + 3) / 4, most = 1 << 15;
  const dim3 grid((unsigned)(q_parts + (p.hkv + heads - 1) / heads), (unsigned)(fours < most ? fours : most),
                  (unsigned)((fours + most - 1) / most));
  if (dtype == 1) {
    if (V == 8) return append<uint16_t, 8>(p, k, v, q_parts, G, n, grid, stream);
    if (V == 4) return append<uint16_t, 4>(p, k, v, q_parts, G, n, grid, stream);
    return append<uint16_t, 2>(p, k, v, q_parts, G, n, grid, stream);
  }
  if (V == 4) return append<float, 4>(p, k, v, q_parts, G, n, grid, stream);
  return append<float, 2>(p, k, v, q_parts, G, n, grid, stream);
}

hipError_t launch_mx4_read(int dtype, const Mx4Read& p, hipStream_t stream) {
  int G = 1;
  while (G * kPiece < p.D) G *= 2;
  const int64_t rows = (int64_t)p.T * p.hkv, per = (256 / kWave) * (kWave / G);
  const dim3 grid((unsigned)((rows + per - 1) / per));
  if (dtype == 1) hipLaunchKernelGGL((mx4_read<uint16_t>), grid, dim3(256), 0, stream, p, G);
  else hipLaunchKernelGGL((mx4_read<float>), grid, dim3(256), 0, stream, p, G);
  return hipGetLastError();
}

}  // namespace sffn
