// Attention over a paged cache on matrix instructions: the tile shared by the
// kernels of paged_attn.cuh.
//
// A wave holds 32 query rows and walks over keys in blocks of 32, transposed:
//   S^T [key, row] = K Q^T      O^T [d, row] += V^T P^T
// with 32x32 matrix instructions.  Lane l holds column (row) l % 32 of S^T and
// O^T, so the softmax statistics of a row, its running maximum, sum and the
// factor of its output, are plain values of a lane: the maximum over keys
// is 16 values in a lane and one exchange with lane l ^ 32.  A lane's S^T values
// are the keys 8 (i / 4) + 4 (l / 32) + i % 4, i < 16, which is also the order in
// which the second product takes its B operand when V^T is read in that
// order, so P stays in its registers.
//
// K and V tiles are copied to LDS with 16-byte asynchronous loads.  Row r keeps
// its 16-byte chunk c at chunk c ^ swizzle(r), so that the reads of a column of
// chunks (K) and the transposing reads of V spread over the banks.
#pragma once

#include <hip/hip_runtime.h>

#include "attn.h"
#include "common.cuh"

namespace sffn {

typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) uint8_t lds_u8_t;

// n / d for 0 <= n < 2^31: (mulhi(n, mul) + (n & one)) >> shift.
struct FastDiv {
  uint32_t mul, one, shift;
  int d;
  static FastDiv make(int d) {
    FastDiv f;
    f.d = d;
    int l = 0;
    while ((1ll << l) < d) ++l;  // 2^l >= d
    // with p = 31 + l, ceil(2^p / d) < 2^32 divides exactly below 2^31; d = 1
    // would need 2^32: the product is n itself
    f.mul = l == 0 ? 0u : (uint32_t)(((1ull << (31 + l)) + (uint64_t)d - 1) / (uint64_t)d);
    f.one = l == 0 ? ~0u : 0u;
    f.shift = l == 0 ? 0 : (uint32_t)(l - 1);
    return f;
  }
  __device__ __forceinline__ int div(int n) const {
    return (int)((__umulhi((uint32_t)n, mul) + ((uint32_t)n & one)) >> shift);
  }
};

// The arguments of the attention kernels.
struct AttnArgs {
  PagedAttn p;
  FastDiv page, group;   // page_size; query heads per key head
  int g;                 // query heads per key head
  float c;               // |scale| log2(e): scores are kept as q . k, exponents in base 2
  int negate;            // scale < 0: q is negated
  int chunk;             // keys per split, a multiple of the key tile
  int min_rows;          // attn_rows takes sequences with more rows than this
  int max_rows;          // attn_keys takes sequences with at most so many
  int tiles_per_seq;     // attn_keys
  int n_tiles;           // (bound of) row tiles of one key head
  float* part_o;         // [split][slot][D] outputs before the division, for split rows
  float* part_ml;        // [split][slot][2] maximum (base 2) and sum
  size_t part_rows;      // slots of one split
};

// ------------------------------------------------------------------ arithmetic
template <typename T> struct Frag;
template <> struct Frag<uint16_t> {
  typedef bf16x8_t type;
  __device__ static __forceinline__ f32x16_t mma(u32x4_t a, u32x4_t b, f32x16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                   __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
  }
  __device__ static __forceinline__ u32x4_t negate(u32x4_t a) { return a ^ 0x80008000u; }
};
template <> struct Frag<float> {
  __device__ static __forceinline__ f32x16_t mma(u32x4_t a, u32x4_t b, f32x16_t c) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a[e]), __uint_as_float(b[e]), c, 0, 0, 0);
    return c;
  }
  __device__ static __forceinline__ u32x4_t negate(u32x4_t a) { return a ^ 0x80000000u; }
};

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  b2 v;
  v.x = (__bf16)a;
  v.y = (__bf16)b;
  return __builtin_bit_cast(uint32_t, v);
}

// Maximum / sum with the other half of the wave (lane ^ 32).
__device__ __forceinline__ float other_half(float v) { return __shfl_xor(v, 32, kWave); }

// ------------------------------------------------------------------ the tile
// T: uint16_t (bf16) or float; DP: head_dim rounded up to the instances below;
// KT: keys of an LDS tile (a multiple of 32).
template <typename T, int DP, int KT>
struct AttnTile {
  static constexpr int kEpc = 16 / (int)sizeof(T);         // elements of a 16-byte chunk
  static constexpr int kRowElems = DP <= 64 ? 64 : DP <= 128 ? 128 : 256;
  static constexpr int kPitch = kRowElems * (int)sizeof(T);  // bytes of a row in LDS
  static constexpr int kCpr = kPitch / 16;                 // chunks of a row
  static constexpr int kRpi = kWave / kCpr;                // rows of one wave-wide load
  static constexpr int kLoads = KT / kRpi;                 // wave-wide loads of a K or V tile
  static constexpr int kKeyBlocks = KT / 32;
  static constexpr int kQ = DP / (2 * kEpc);               // Q and K fragments of a row
  static constexpr int kDt = DP / 32;                      // 32-wide blocks of the output
  static constexpr int kTileBytes = KT * kPitch;           // of K, and again of V
  static_assert(kRpi >= 1 && KT % 32 == 0 && DP % 32 == 0, "");

  // Chunk permutation of row r.  K is read by 32 rows at one chunk: any 16
  // neighbouring rows get 16 different chunks (8 when a row has 8).  V is read
  // as 64 bytes of 8 neighbouring rows.
  __device__ static __forceinline__ int swz_k(int r) { return r & (kCpr < 16 ? kCpr - 1 : 15); }
  __device__ static __forceinline__ int swz_v(int r) {
    if constexpr (sizeof(T) == 4) return 0;  // read row by row: no conflicts
    else return kCpr >= 16 ? ((r & 3) << 2) : ((r & 2) << 1);
  }

  u32x4_t q[kQ];
  f32x16_t o[kDt];
  float m, l;

  __device__ __forceinline__ void init() {
#pragma unroll
    for (int d = 0; d < kDt; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[d][i] = 0.f;
    m = -INFINITY;
    l = 0.f;
  }

  // This lane's part of query row `row` (B operand: chunks 2 i + lane / 32).
  __device__ __forceinline__ void load_q(const T* row, int D, bool negate) {
    const int h = lane_id() >> 5;
#pragma unroll
    for (int i = 0; i < kQ; ++i) {
      const int e = (2 * i + h) * kEpc;
      u32x4_t v = {0u, 0u, 0u, 0u};
      if (e < D) v = ldg16(row + e);
      q[i] = negate ? Frag<T>::negate(v) : v;
    }
  }

  // S^T of key block kb of the K tile at `k`.
  __device__ __forceinline__ f32x16_t scores(const uint8_t* k, int kb) const {
    const int lane = lane_id(), r = lane & 31, h = lane >> 5;
    const uint8_t* row = k + (kb * 32 + r) * kPitch;
    f32x16_t s;
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = 0.f;
#pragma unroll
    for (int i = 0; i < kQ; ++i) {
      const u32x4_t a = *(const u32x4_t*)(row + (((2 * i + h) ^ swz_k(r)) << 4));
      s = Frag<T>::mma(a, q[i], s);
    }
    return s;
  }

  // Index within a key block of a lane's S^T value i.
  __device__ static __forceinline__ int key_of(int i, int half) { return 8 * (i >> 2) + 4 * half + (i & 3); }

  // Softmax step over the tile's scores: s becomes the weights.  The maximum
  // is only moved (and l and o scaled) when it grows by more than 2^8 in some
  // row: weights up to 2^8 keep their relative precision in any type, and most
  // tiles then leave o alone.
  __device__ __forceinline__ void softmax(f32x16_t (&s)[kKeyBlocks], float c) {
    float mx = s[0][0];
#pragma unroll
    for (int b = 0; b < kKeyBlocks; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[b][i]);
    mx = fmaxf(mx, other_half(mx));
    const float mn = fmaxf(m, mx);
    if (__any((mn - m) * c > 8.f)) {
      const float f = mn == -INFINITY ? 1.f : __builtin_amdgcn_exp2f((m - mn) * c);
      l *= f;
#pragma unroll
      for (int d = 0; d < kDt; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] *= f;
      m = mn;
    }
    const float mc = m == -INFINITY ? 0.f : m * c;
    float sum = 0.f;
#pragma unroll
    for (int b = 0; b < kKeyBlocks; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(s[b][i], c, -mc));
        s[b][i] = w;
        sum += w;
      }
    l += sum;
  }

  // V^T fragment (A operand): rows (d) dt * 32 + lane % 32, the 16 keys of step
  // ks in the order of the weights.  Two transposing reads: 16 lanes read 4 keys
  // x 16 elements and each gets one element of the 4 keys.
  __device__ static __forceinline__ u32x4_t v_frag(const uint8_t* v, int ks, int dt) {
    const int lane = lane_id(), i = lane & 15, g = lane >> 4;
    const int r = ks * 16 + 4 * (g >> 1) + (i >> 2);
    const int c = dt * 4 + 2 * (g & 1) + ((i & 3) >> 1);
    const uint8_t* a0 = v + r * kPitch + ((c ^ swz_v(r)) << 4) + (i & 1) * 8;
    const uint8_t* a1 = v + (r + 8) * kPitch + ((c ^ swz_v(r + 8)) << 4) + (i & 1) * 8;
    const s16x4_t x0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4_t*)a0);
    const s16x4_t x1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4_t*)a1);
    typedef short s16x8 __attribute__((ext_vector_type(8)));
    return __builtin_bit_cast(u32x4_t, __builtin_shufflevector(x0, x1, 0, 1, 2, 3, 4, 5, 6, 7));
  }

  // o += V^T P^T.
  __device__ __forceinline__ void accumulate(const uint8_t* v, const f32x16_t (&s)[kKeyBlocks]) {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int ks = 0; ks < KT / 16; ++ks) {
        u32x4_t pf;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          pf[j] = pack_bf16(s[ks / 2][8 * (ks & 1) + 2 * j], s[ks / 2][8 * (ks & 1) + 2 * j + 1]);
#pragma unroll
        for (int d = 0; d < kDt; ++d) o[d] = Frag<T>::mma(v_frag(v, ks, d), pf, o[d]);
      }
    } else {
      const int r0 = 4 * (lane_id() >> 5), col = lane_id() & 31;
#pragma unroll
      for (int b = 0; b < kKeyBlocks; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i)
#pragma unroll
          for (int d = 0; d < kDt; ++d) {
            const float x = *(const float*)(v + (b * 32 + 8 * (i >> 2) + (i & 3) + r0) * kPitch +
                                            (d * 32 + col) * 4);
            o[d] = __builtin_amdgcn_mfma_f32_32x32x2f32(x, s[b][i], o[d], 0, 0, 0);
          }
    }
  }

  // A key that a row does not see has weight 0, but 0 times an infinite or NaN
  // value is NaN.  So in tiles with hidden keys such values are looked for, and
  // if there are any, added directly to the outputs of the rows that see them
  // (add_infinite) and replaced by 0 in LDS (clear_infinite).
  // The 16-byte chunks of the tile are shared by n threads, this being thread i.
  __device__ static __forceinline__ bool infinite_bits(u32x4_t x) {
    bool bad = false;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      bad |= (x[j] & 0x7f800000u) == 0x7f800000u || (sizeof(T) == 2 && (x[j] & 0x7f80u) == 0x7f80u);
    return bad;
  }
  __device__ static __forceinline__ bool find_infinite(const uint8_t* v, int i, int n) {
    bool bad = false;
    for (int at = i * 16; at < kTileBytes; at += n * 16) bad |= infinite_bits(*(const u32x4_t*)(v + at));
    return bad;
  }
  __device__ static __forceinline__ void clear_infinite(uint8_t* v, int i, int n) {
    for (int at = i * 16; at < kTileBytes; at += n * 16) {
      u32x4_t x = *(const u32x4_t*)(v + at);
      if (!infinite_bits(x)) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(T) == 2) {
          if ((x[j] & 0x7f80u) == 0x7f80u) x[j] &= 0xffff0000u;
          if ((x[j] & 0x7f800000u) == 0x7f800000u) x[j] &= 0x0000ffffu;
        } else if ((x[j] & 0x7f800000u) == 0x7f800000u) {
          x[j] = 0u;
        }
      }
      *(u32x4_t*)(v + at) = x;
    }
  }
  __device__ __forceinline__ void add_infinite(const uint8_t* v, int j0, int lo, int hi) {
    const int h = lane_id() >> 5;
#pragma unroll 1
    for (int r = 0; r < KT; ++r) {
      const bool seen = j0 + r >= lo && j0 + r < hi;
#pragma unroll
      for (int d = 0; d < kDt; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int e = d * 32 + 8 * (i >> 2) + 4 * h + (i & 3);
          const T* x = (const T*)(v + r * kPitch + (((e / kEpc) ^ swz_v(r)) << 4)) + e % kEpc;
          const float f = Elt<T>::load1(x, 0);
          if (seen && (__float_as_uint(f) & 0x7f800000u) == 0x7f800000u) o[d][i] += f;
        }
    }
  }

  // Scores of keys that the row does not see (it sees lo .. hi - 1) become -inf.
  __device__ static __forceinline__ void hide(f32x16_t (&s)[kKeyBlocks], int j0, int lo, int hi) {
    const int h = lane_id() >> 5;
#pragma unroll
    for (int b = 0; b < kKeyBlocks; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int j = j0 + b * 32 + key_of(i, h);
        s[b][i] = j >= lo && j < hi ? s[b][i] : -INFINITY;
      }
  }

  // One tile that starts at key j0: scores, softmax, product with V.  whole: every
  // row of the wave sees every key.
  __device__ __forceinline__ void step(const uint8_t* k, const uint8_t* v, int j0, int lo, int hi,
                                       bool whole, float c) {
    f32x16_t s[kKeyBlocks];
#pragma unroll
    for (int b = 0; b < kKeyBlocks; ++b) s[b] = scores(k, b);
    if (!whole) hide(s, j0, lo, hi);
    softmax(s, c);
    accumulate(v, s);
  }
};

// ------------------------------------------------------------------ the loads
__device__ __forceinline__ void copy16(const void* src, uint8_t* dst) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                   (__attribute__((address_space(3))) void*)dst, 16, 0, 0);
}

// A value that no kernel writes while this one runs, at a uniform address: a scalar
// load, which does not wait behind the tile loads.
__device__ __forceinline__ int load_uniform(const int32_t* p) {
  return *(const __attribute__((address_space(4))) int32_t*)p;
}

// Copies key rows to LDS, N wave-wide loads per tile.  FAST: the rows of a granule
// of G lie in one page (page_size a multiple of 16) and fill their LDS rows
// (head_dim == kRowElems), so a page is looked up once a granule with scalar
// instructions and a lane only adds a constant offset; otherwise every lane
// looks up its own rows.  Pages are looked up one tile ahead.
template <typename T, int DP, int KT, bool FAST, int N>
struct TileLoader {
  typedef AttnTile<T, DP, KT> Tile;
  const int32_t* bt;
  const uint8_t *k, *v;         // of the key head
  uint64_t k_page, v_page;      // bytes
  int64_t k_token, v_token;
  FastDiv per_page;
  int last_page, first, last;   // keys that exist for this tile: the others repeat one of them
  int i0, n_chunks;             // this wave's first wave-wide load of a tile; chunks of a row
  static constexpr int kG = !FAST ? Tile::kRpi : N * Tile::kRpi < 16 ? N * Tile::kRpi : 16;
  static constexpr int kPerG = kG / Tile::kRpi;  // wave-wide loads of a granule
  int page[N / kPerG], off[N / kPerG];           // of the next tile

  __device__ __forceinline__ void init(const AttnArgs& a, int seq, int hk, int lo, int hi, int load0) {
    const PagedAttn& p = a.p;
    bt = p.block_table + (size_t)seq * p.max_pages;
    k = (const uint8_t*)((const T*)p.k_cache + hk * p.kc_head);
    v = (const uint8_t*)((const T*)p.v_cache + hk * p.vc_head);
    k_page = (uint64_t)p.kc_page * sizeof(T);
    v_page = (uint64_t)p.vc_page * sizeof(T);
    k_token = p.kc_token * (int64_t)sizeof(T);
    v_token = p.vc_token * (int64_t)sizeof(T);
    per_page = a.page;
    last_page = p.n_pages - 1;
    first = lo, last = hi - 1;
    i0 = load0;
    n_chunks = p.D / Tile::kEpc;
  }

  __device__ __forceinline__ void look_up(int j0) {
#pragma unroll
    for (int n = 0; n < N / kPerG; ++n) {
      int j = j0 + i0 * Tile::kRpi + n * kG;
      if constexpr (FAST) j = min(max(j, first & -kG), last & -kG);
      else j = min(max(j + lane_id() / Tile::kCpr, first), last);
      const int pg = per_page.div(j);
      off[n] = j - pg * per_page.d;
      if constexpr (FAST) page[n] = load_uniform(bt + pg);
      else page[n] = bt[pg];
    }
  }

  // Starts the loads of the tile that was looked up.
  __device__ __forceinline__ void start(uint8_t* k_tile, uint8_t* v_tile) const {
    const int rin = lane_id() / Tile::kCpr, chunk = lane_id() % Tile::kCpr;
#pragma unroll
    for (int g = 0; g < N / kPerG; ++g) {
      const uint32_t pg = (uint32_t)min(max(page[g], 0), last_page);
      const uint8_t* kr = k + (pg * k_page + off[g] * k_token);
      const uint8_t* vr = v + (pg * v_page + off[g] * v_token);
#pragma unroll
      for (int m = 0; m < kPerG; ++m) {
        const int i = i0 + g * kPerG + m, r = i * Tile::kRpi + rin;
        const int ck = chunk ^ Tile::swz_k(r), cv = chunk ^ Tile::swz_v(r);
        uint8_t* kd = k_tile + i * 1024;
        uint8_t* vd = v_tile + i * 1024;
        if constexpr (FAST) {
          copy16(kr + m * Tile::kRpi * k_token + ((uint32_t)rin * (uint32_t)k_token + ck * 16), kd);
          copy16(vr + m * Tile::kRpi * v_token + ((uint32_t)rin * (uint32_t)v_token + cv * 16), vd);
        } else {
          if (ck < n_chunks) copy16(kr + ck * 16, kd);
          if (cv < n_chunks) copy16(vr + cv * 16, vd);
        }
      }
    }
  }
};

}  // namespace sffn
