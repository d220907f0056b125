// Writing keys and values into the 4-bit paged cache, and reading them back.
#include <hip/hip_runtime.h>

#include "attn.h"
#include "common.cuh"
#include "heads.cuh"
#include "mx4.cuh"

namespace sffn {

namespace {

// A lane holds eight neighbouring elements of a row of k or v, four lanes a block.
constexpr int kPiece = 8;

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&o)[kPiece]) {
  constexpr int kN = Elt<T>::kPerChunk;
#pragma unroll
  for (int i = 0; i < kPiece; i += kN) Elt<T>::unpack(ldg16(p + i), o + i);
}

// Two neighbouring elements (an even one first).
template <typename T>
__device__ __forceinline__ void load2(const T* p, float* o) {
  if constexpr (sizeof(T) == 2) {
    const uint32_t w = *(const uint32_t*)p;
    o[0] = bf16lo(w), o[1] = bf16hi(w);
  } else {
    o[0] = p[0], o[1] = p[1];
  }
}

// Sum over the G lanes of a row, every lane getting it (the same order in each).
__device__ __forceinline__ double row_sum64(double v, int G) {
  for (int o = 1; o < G; o <<= 1) v += __shfl_xor(v, o, kWave);
  return v;
}

// A lane's elements x of a row of k, normalised and rotated in 64 bits: the partner of
// an element in a rotated pair is in the same lane (adjacent pairs) or read once more, with
// its weight.  64 bits cost nothing here (k is a tenth of the elements, and the kernel waits
// for memory), and what is rounded to 4 bits is then the correctly rounded float32 value:
// the codes of a token do not hang on which kernel, order of sums or chunk of a prompt
// wrote it, and a value next to the border between two codes falls on its own side.
template <typename T>
__device__ __forceinline__ void norm_rotate64(const HeadsFwd& p, const T* row, int at, bool live, int G,
                                              const float* angles, bool known, float (&x)[kPiece]) {
  double n[kPiece], r = 1.0;
  if (p.norm) {
    double ss = 0.0;
#pragma unroll
    for (int i = 0; i < kPiece; ++i) ss += (double)x[i] * x[i];
    ss = row_sum64(ss, G);
    r = 1.0 / __builtin_sqrt(ss / p.D + (double)p.eps);
  }
  const T* w = (const T*)p.k_weight;
  const bool weighted = p.norm && w != nullptr;
  if (!live) return;
  float wt[kPiece];
  if (weighted) load8(w + at, wt);
#pragma unroll
  for (int i = 0; i < kPiece; ++i) {
    n[i] = p.norm ? x[i] * r : (double)x[i];
    if (weighted) n[i] *= wt[i];
  }
  const int half = p.rot / 2;
  if (p.rot_adjacent) {
#pragma unroll
    for (int i = 0; i < kPiece; i += 2) {
      if (at + i >= p.rot) continue;
      const double c = angles[(at + i) / 2], s = angles[half + (at + i) / 2];
      const double a = n[i], b = n[i + 1];
      n[i] = a * c - b * s;
      n[i + 1] = b * c + a * s;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPiece; i += 2) {  // half is even: a pair of neighbours has neighbours as partners
      const int e = at + i;
      if (e >= p.rot) continue;
      const bool first = e < half;
      const int other = first ? e + half : e - half, angle = first ? e : other;
      float y[2], yw[2] = {1.f, 1.f};
      load2(row + other, y);
      if (weighted) load2(w + other, yw);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const double c = angles[angle + j], s = angles[half + angle + j];
        double m = p.norm ? y[j] * r : (double)y[j];
        if (weighted) m *= yw[j];
        n[i + j] = first ? n[i + j] * c - m * s : n[i + j] * c + m * s;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kPiece; ++i) x[i] = !known && at + i < p.rot ? __builtin_nanf("") : (float)n[i];
}

// Rows of k and v of token t from number r0 on, one pass of a wave, into the cache.
template <typename T>
__device__ __forceinline__ void store_rows(const HeadsFwd& p, const Mx4Rows& kc, const Mx4Rows& vc, int t,
                                           int part, int passes) {
  const int lane = lane_id();
  const int slot = p.slots[t];
  if (slot < 0 || (int64_t)slot >= (int64_t)p.n_pages * p.page_size) return;
  const int page = slot / p.page_size, off = slot % p.page_size;
  int G = 4;
  while (G * kPiece < p.D) G *= 2;
  const int u = lane & (G - 1), sub = lane / G, rpw = kWave / G, at = u * kPiece;
  const int pos = position_of(p.positions, p.rot, t);
  const bool known = p.rot == 0 || (pos >= 0 && pos < p.max_pos);
  const float* angles = p.table + (size_t)(known ? pos : 0) * p.rot;
  const int first = part * passes * rpw, last = min(first + passes * rpw, 2 * p.hkv);
  for (int r0 = first; r0 < last; r0 += rpw) {
    const int r = r0 + sub;
    const bool is_k = r < p.hkv, live = r < last && at < p.D;
    const int h = is_k ? r : r - p.hkv;
    const T* row = is_k ? (const T*)p.k + t * p.k_token + h * p.k_head
                        : (const T*)p.v + t * p.v_token + h * p.v_head;
    float x[kPiece];
#pragma unroll
    for (int i = 0; i < kPiece; ++i) x[i] = 0.f;
    if (live) load8(row + at, x);
    // lanes of a v row pass through with the k rows of the wave, for the sums
    if (r0 < p.hkv && (p.norm || p.rot > 0)) {
      float y[kPiece];
#pragma unroll
      for (int i = 0; i < kPiece; ++i) y[i] = x[i];
      norm_rotate64<T>(p, row, at, live && is_k, G, angles, known, y);
#pragma unroll
      for (int i = 0; i < kPiece; ++i) x[i] = is_k ? y[i] : x[i];
    }
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kPiece; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
    top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0xB1, 0xf, 0xf, false));
    top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0x4E, 0xf, 0xf, false));
    const uint32_t b = mx_scale_byte(top);
    if (!live) continue;
    const Mx4Rows& c = is_k ? kc : vc;
    *(uint32_t*)(c.codes + page * c.page + off * c.token + h * c.head + u * 4) =
        b == 255 ? 0u : mx_encode8(x, mx_scale(b));
    if ((u & 3) == 0)
      c.scales[page * c.s_page + off * c.s_token + h * c.s_head + u / 4] = (uint8_t)b;
  }
}

// One wave per (token, part of its heads): parts of q, then of k and v.
template <typename T, int V>
__global__ __launch_bounds__(kHeadsBlock) void heads_mx4(HeadsFwd p, Mx4Rows k, Mx4Rows v, int q_parts,
                                                         int passes) {
  const int t = uniform((int)(blockIdx.x * (kHeadsBlock / kWave) + threadIdx.x / kWave));
  if (t >= p.T) return;
  if ((int)blockIdx.y < q_parts) {
    HeadsFwd q = p;
    q.hkv = 0;
    q.slots = nullptr;
    heads_fwd_part<T, V>(q, t, (int)blockIdx.y);
  } else {
    store_rows<T>(p, k, v, t, (int)blockIdx.y - q_parts, passes);
  }
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
hipError_t append(const HeadsFwd& p, const Mx4Rows& k, const Mx4Rows& v, int q_parts, int passes,
                  dim3 grid, hipStream_t stream) {
  hipLaunchKernelGGL((heads_mx4<T, V>), grid, dim3(kHeadsBlock), 0, stream, p, k, v, q_parts, passes);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_heads_mx4(int dtype, HeadsFwd p, Mx4Rows k, Mx4Rows v, hipStream_t stream) {
  const int V = chunk_elements(dtype, p.rot, p.rot_adjacent != 0);
  p.lanes_per_row = lanes_per_row(p.D, p.rot, p.rot_adjacent != 0, V);
  const int rpw = kWave / p.lanes_per_row, q_passes = (p.hq + rpw - 1) / rpw;
  int G = 4;
  while (G * kPiece < p.D) G *= 2;
  const int kv_passes = (2 * p.hkv * G + kWave - 1) / kWave;
  // few tokens: a wave for every pass, as in the append without quantisation
  const bool few = p.T < 2048;
  const int q_each = few ? 1 : q_passes, kv_each = few ? 1 : kv_passes;
  p.rows_per_wave = q_each * rpw;
  const int q_parts = p.hq == 0 ? 0 : (q_passes + q_each - 1) / q_each;
  const dim3 grid((unsigned)((p.T + 3) / 4), (unsigned)(q_parts + (kv_passes + kv_each - 1) / kv_each));
  if (dtype == 1) {
    if (V == 8) return append<uint16_t, 8>(p, k, v, q_parts, kv_each, grid, stream);
    if (V == 4) return append<uint16_t, 4>(p, k, v, q_parts, kv_each, grid, stream);
    return append<uint16_t, 2>(p, k, v, q_parts, kv_each, grid, stream);
  }
  if (V == 4) return append<float, 4>(p, k, v, q_parts, kv_each, grid, stream);
  return append<float, 2>(p, k, v, q_parts, kv_each, grid, stream);
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
