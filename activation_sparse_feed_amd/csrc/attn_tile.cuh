// Attention over a paged cache on matrix instructions: the tile shared by the
// kernels of attn_kernels.cuh.
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
// With 64 rows a wave the fragments read from LDS would serve twice the products,
// but output, queries and two blocks of scores leave registers for one wave a SIMD
// only: 2.92 ms instead of 2.14 to 2.16 for a 16384-token prompt (32 heads on 8,
// width 128).
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
  FastDiv chunk;         // keys per split, a multiple of the key tile
  int min_rows;          // attn_rows takes sequences with more rows than this
  int max_rows;          // attn_keys takes sequences with at most so many
  int tiles_per_seq;     // attn_keys
  int slot_rows;         // attn_keys: slots of a sequence and key head, for all rows it can have
  int splits;            // (bound of) splits of a key range
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

// The value of lane ^ 32 is in one of the two results of the swap, the lane's own in
// the other.
__device__ __forceinline__ float max_halves(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float sum_halves(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// ------------------------------------------------------------------ the tile
// T: uint16_t (bf16) or float; DP: head_dim rounded up to the instances below;
// KT: keys of an LDS tile, 32 or 64: K and V tiles are walked over in blocks of 32.
template <typename T, int DP, int KT>
struct AttnTile {
  static constexpr int kEpc = 16 / (int)sizeof(T);         // elements of a 16-byte chunk
  static constexpr int kRowElems = DP <= 64 ? 64 : DP <= 128 ? 128 : 256;
  static constexpr int kPitch = kRowElems * (int)sizeof(T);  // bytes of a row in LDS
  static constexpr int kCpr = kPitch / 16;                 // chunks of a row
  static constexpr int kRpi = kWave / kCpr;                // rows of one wave-wide load
  static constexpr int kLoads = KT / kRpi;                 // wave-wide loads of a K or V tile
  static constexpr int kQ = DP / (2 * kEpc);               // Q and K fragments of a row
  static constexpr int kDt = DP / 32;                      // 32-wide blocks of the output
  static constexpr int kTileBytes = KT * kPitch;           // of K, and again of V
  static constexpr int kBlockBytes = 32 * kPitch;
  static_assert(kRpi >= 1 && KT % 32 == 0 && DP % 32 == 0, "");

  // Chunk permutation of row r.  K is read by 32 rows at one chunk: any 16
  // neighbouring rows get 16 different chunks (8 when a row has 8).  V is read
  // as 64 bytes of 8 neighbouring rows.  Bank conflicts are under 3% of
  // the LDS cycles at width 128 (none in attn_rows), a third at 64; r / 2 & 7 in
  // swz_k takes those away, but no time (a 4096-token prompt 87 us instead of 84).
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

  // This lane's part of query row `row` (B operand: chunks 2 i + lane / 32).  A negative
  // scale is applied by negate(), once the loads are done.
  __device__ __forceinline__ void load_q(const T* row, int D) {
    const int h = lane_id() >> 5;
#pragma unroll
    for (int i = 0; i < kQ; ++i) {
      const int e = (2 * i + h) * kEpc;
      q[i] = u32x4_t{0u, 0u, 0u, 0u};
      if (e < D) q[i] = ldg16(row + e);
    }
  }
  __device__ __forceinline__ void negate() {
#pragma unroll
    for (int i = 0; i < kQ; ++i) q[i] = Frag<T>::negate(q[i]);
  }

  // S^T of the 32 keys at `k`.
  __device__ __forceinline__ f32x16_t scores(const uint8_t* k) const {
    const int lane = lane_id(), r = lane & 31, h = lane >> 5;
    const int at = r * kPitch + ((h ^ swz_k(r)) << 4);
    u32x4_t a[kQ];
#pragma unroll
    for (int i = 0; i < kQ; ++i) a[i] = *(const u32x4_t*)(k + (at ^ (i << 5)));
    f32x16_t s;
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = 0.f;
#pragma unroll
    for (int i = 0; i < kQ; ++i) s = Frag<T>::mma(a[i], q[i], s);
    return s;
  }

  // Index within a block of a lane's S^T value i.
  __device__ static __forceinline__ int key_of(int i, int half) { return 8 * (i >> 2) + 4 * half + (i & 3); }

  // Scores of keys that the row does not see (it sees lo .. hi - 1) become -inf; j:
  // the block's first key.
  __device__ static __forceinline__ void hide(f32x16_t& s, int j, int lo, int hi) {
    const int h = lane_id() >> 5;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int k = j + key_of(i, h);
      s[i] = k >= lo && k < hi ? s[i] : -INFINITY;
    }
  }

  // Moves the running maximum to that of the scores (and scales l and o) where
  // some row's grows by more than a factor of 2^8: weights up to 2^8 keep their
  // relative precision in any type, and most blocks then leave o alone.  A row
  // without a maximum yet has l = 0, and in o nothing but infinite values that
  // add_infinite put there: they stay (the factor exp2(-inf) = 0 would make NaN of them).
  __device__ __forceinline__ void raise(const f32x16_t& s, float c) {
    float mx = s[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) mx = fmaxf(mx, s[i]);
    const float mn = fmaxf(m, max_halves(mx));
    if (__any((mn - m) * c > 8.f)) {
      const float f = m == -INFINITY ? 1.f : __builtin_amdgcn_exp2f((m - mn) * c);
      l *= f;
#pragma unroll
      for (int d = 0; d < kDt; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] *= f;
      m = mn;
    }
  }

  // s becomes the weights, their sum is added to l.
  __device__ __forceinline__ void weights(f32x16_t& s, float c) {
    const float mc = m == -INFINITY ? 0.f : m * c;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      s[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], c, -mc));
      sum += s[i];
    }
    l += sum;
  }

  // V^T fragment (A operand) of the 32 keys at v: rows (d) dt * 32 + lane % 32, the
  // 16 keys of half ks in the order of the weights.  Two transposing reads: 16
  // lanes read 4 keys x 16 elements and each gets one element of the 4 keys.
  __device__ static __forceinline__ u32x4_t v_frag(const uint8_t* v, int ks, int dt) {
    const int lane = lane_id(), i = lane & 15, g = lane >> 4;
    const int r = 4 * (g >> 1) + (i >> 2);  // swz_v(r + 8) is swz_v(r)
    const int c = (2 * (g & 1) + ((i & 3) >> 1)) ^ swz_v(r);
    const uint8_t* a = v + ks * 16 * kPitch + ((r * kPitch + (c << 4) + (i & 1) * 8) ^ (dt << 6));
    typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;
    const s16x4_t x0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)a);
    const s16x4_t x1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(a + 8 * kPitch));
    return __builtin_bit_cast(u32x4_t, __builtin_shufflevector(x0, x1, 0, 1, 2, 3, 4, 5, 6, 7));
  }

  // o += V^T P^T over the 32 keys at v.  In bf16 the weights are rounded to bf16 here,
  // since the matrix instruction takes both operands in one type; their sum l is that of the
  // unrounded ones, and o is float32.  Relative error against 64 bits 2.0e-3 to 2.3e-3,
  // where rounding the output alone gives 1.5e-3 to 1.7e-3 (standard normal inputs).
  __device__ __forceinline__ void accumulate(const uint8_t* v, const f32x16_t& s) {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        u32x4_t pf;
#pragma unroll
        for (int j = 0; j < 4; ++j) pf[j] = pack_bf16(s[8 * ks + 2 * j], s[8 * ks + 2 * j + 1]);
#pragma unroll
        for (int d = 0; d < kDt; ++d) o[d] = Frag<T>::mma(v_frag(v, ks, d), pf, o[d]);
      }
    } else {
      const uint8_t* at = v + 4 * (lane_id() >> 5) * kPitch + (lane_id() & 31) * 4;
#pragma unroll
      for (int i = 0; i < 16; ++i)
#pragma unroll
        for (int d = 0; d < kDt; ++d) {
          const float x = *(const float*)(at + (8 * (i >> 2) + (i & 3)) * kPitch + d * 128);
          o[d] = __builtin_amdgcn_mfma_f32_32x32x2f32(x, s[i], o[d], 0, 0, 0);
        }
    }
  }

  // One block of 32 keys whose scores are in s, and the scores of the next one: its
  // matrix instructions do not depend on this block's exponentials, so a wave has
  // both to issue side by side.
  __device__ __forceinline__ void step(f32x16_t& s, const uint8_t* k_next, const uint8_t* v, float c) {
    raise(s, c);
    const f32x16_t next = scores(k_next);
    weights(s, c);
    accumulate(v, s);
    s = next;
  }

  // A key that a row does not see has weight 0, but 0 times an infinite or NaN
  // value is NaN.  So in tiles with hidden keys such values are looked for, and
  // if there are any, added directly to the outputs of the rows that see them
  // (add_infinite) and replaced by 0 in LDS (clear_infinite).  The search runs over
  // whole LDS rows, so what lies in them beyond head_dim has to be finite.  Rows that no query
  // sees (behind a sequence's end, before a window), which may hold anything, are only
  // replaced: add_infinite takes 70 us, and stale ones made 103 us of 34 (bf16, 128 rows of 32 heads on 8
  // over 4096 keys).
  // The 16-byte chunks of the tile are shared by N threads, this being thread i.
  __device__ static __forceinline__ bool infinite_bits(u32x4_t x) {
    bool bad = false;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      bad |= (x[j] & 0x7f800000u) == 0x7f800000u || (sizeof(T) == 2 && (x[j] & 0x7f80u) == 0x7f80u);
    return bad;
  }
  template <int N>
  __device__ static __forceinline__ bool find_infinite(const uint8_t* v, int i) {
    bool bad = false;
#pragma unroll
    for (int at = 0; at < kTileBytes; at += N * 16) bad |= infinite_bits(*(const u32x4_t*)(v + at + i * 16));
    return bad;
  }
  // Only in the tile's rows lo .. hi - 1.  UNROLL: attn_rows all steps (in bf16, 2048 tokens of 16 heads
  // on 4 of width 96 51.8 us, as a loop 53.2), the others 1 (attn_rows_mx4 of width 256 108.8, 112.3
  // unrolled; attn_keys in float32, 32 tokens of width 64 70.6, 71.4).
  template <int N, int UNROLL>
  __device__ static __forceinline__ bool find_infinite_in(const uint8_t* v, int i, int lo, int hi) {
    bool bad = false;
#pragma unroll UNROLL
    for (int at0 = 0; at0 < kTileBytes; at0 += N * 16) {
      const int at = at0 + i * 16;
      bad |= at / kPitch >= lo && at / kPitch < hi && infinite_bits(*(const u32x4_t*)(v + at));
    }
    return bad;
  }
  template <int N>
  __device__ static __forceinline__ void clear_infinite(uint8_t* v, int i) {
    for (int at = i * 16; at < kTileBytes; at += N * 16) {
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
  // j0: the tile's first key.
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

// Copies the key rows of one cache (K or V) to LDS, N wave-wide loads per tile and
// wave.  Pages are looked up one tile ahead.
//   G > 0  page_size is a multiple of G: G neighbouring rows lie in one page, which
//          is looked up with scalar instructions; a lane adds a constant offset.
//   G = 0  any page size: lane r looks up row r of the wave's part of a tile, and the
//          loads get their rows' offsets from it.
template <typename T, int DP, int KT, int G, int N, bool K>
struct TileLoader {
  typedef AttnTile<T, DP, KT> Tile;
  static constexpr int kRows = N * Tile::kRpi;               // of the wave, in a tile
  static constexpr int kG = G < kRows ? G : kRows;           // rows of one lookup
  static constexpr int kLookups = G == 0 ? 1 : kRows / (G == 0 ? 1 : kG);
  static_assert(kRows <= kWave && (G == 0 || kG >= Tile::kRpi), "");
  const int32_t* bt;
  const uint8_t* base;          // of the key head
  uint64_t page_bytes;
  int64_t token_bytes;
  FastDiv per_page;
  int last_page, first, last;   // keys that exist for this tile: the others repeat one of them
  int i0, n_chunks;             // this wave's first wave-wide load of a tile; chunks of a row
  int page[kLookups], off[kLookups];  // of the next tile

  __device__ __forceinline__ void init(const AttnArgs& a, int seq, int hk, int lo, int hi, int load0) {
    const PagedAttn& p = a.p;
    bt = p.block_table + (size_t)seq * p.max_pages;
    base = K ? (const uint8_t*)((const T*)p.k_cache + hk * p.kc_head)
             : (const uint8_t*)((const T*)p.v_cache + hk * p.vc_head);
    page_bytes = (uint64_t)(K ? p.kc_page : p.vc_page) * sizeof(T);
    token_bytes = (K ? p.kc_token : p.vc_token) * (int64_t)sizeof(T);
    per_page = a.page;
    last_page = p.n_pages - 1;
    first = lo, last = hi - 1;
    i0 = load0;
    n_chunks = p.D / Tile::kEpc;
  }

  // The tile of the keys j0 .. j0 + KT - 1 (j0 a multiple of 32).
  __device__ __forceinline__ void look_up(int j0) {
#pragma unroll
    for (int n = 0; n < kLookups; ++n) {
      int j = j0 + i0 * Tile::kRpi;
      if constexpr (G > 0) j = min(max(j + n * kG, first & -kG), last & -kG);
      else j = min(max(j + min(lane_id(), kRows - 1), first), last);
      const int pg = per_page.div(j);
      off[n] = j - pg * per_page.d;
      if constexpr (G > 0) page[n] = load_uniform(bt + pg);
      else page[n] = bt[pg];
    }
  }

  // Starts the loads of the tile that was looked up.  Rows that fill their LDS rows
  // need no mask.
  __device__ __forceinline__ void start(uint8_t* tile) const {
    if (n_chunks == Tile::kCpr) start_all<false>(tile);
    else start_all<true>(tile);
  }
  template <bool MASK>
  __device__ __forceinline__ void start_all(uint8_t* tile) const {
    const int rin = lane_id() / Tile::kCpr, chunk = lane_id() % Tile::kCpr;
    const uint64_t lane_row = (uint32_t)min(max(page[0], 0), last_page) * page_bytes + off[0] * token_bytes;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int r = (i0 + n) * Tile::kRpi + rin;  // row of the tile
      const int c = chunk ^ (K ? Tile::swz_k(r) : Tile::swz_v(r));
      uint8_t* to = tile + (i0 + n) * 1024;
      const uint8_t* row;
      uint32_t lane_bytes = c * 16;
      if constexpr (G > 0) {
        const int at = n * Tile::kRpi, g = at / kG;
        row = base + ((uint32_t)min(max(page[g], 0), last_page) * page_bytes +
                      (off[g] + at % kG) * token_bytes);
        lane_bytes += (uint32_t)rin * (uint32_t)token_bytes;
      } else {
        const int from = n * Tile::kRpi + rin;
        const uint32_t lo = __shfl((uint32_t)lane_row, from, kWave);
        const uint32_t hi = __shfl((uint32_t)(lane_row >> 32), from, kWave);
        row = base + (((uint64_t)hi << 32) | lo);
      }
      if (!MASK || c < n_chunks) copy16(row + lane_bytes, to);
    }
  }
};

}  // namespace sffn
