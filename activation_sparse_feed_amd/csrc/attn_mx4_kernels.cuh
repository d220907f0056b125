// Kernels of attention over the 4-bit paged cache.  Rows, tiles, splits and their joining
// are those of attn_kernels.cuh; what differs is how keys and values come to the matrix
// instructions: codes and scales are loaded into registers, a tile ahead, and turned into
// bfloat16 there, two elements an instruction at the full rate, with nothing rounded.
//
//   attn_rows_mx4  many rows (chunks of prompts): the tiles of attn_rows, K and V tiles
//                  written to LDS by the threads that decode them, a 16-byte run of codes of a
//                  row a thread (width 128).  Bound by the matrix cores at the clock that
//                  the card's power allows, like attn_rows: 2.06 to 2.16 ms for a 16384-token
//                  prompt (32 heads on 8, width 128, bf16: 2.20 TFLOP, 1.02 to 1.07 PFLOP/s) where
//                  attn_rows takes 2.15 to 2.28; the decoding hides beside the matrix instructions.
//                  Eight waves (256 rows, half the decoding a row) gave 2.22 beside 2.26, but
//                  719 us instead of 694 for chunks beside single tokens: not kept.  Both widths
//                  of loads in one instance, chosen at run time, made its loads wait where the two
//                  join: 744 us instead of 674.  float32: 122 us for 2048 tokens (16 heads on
//                  4, width 128), 295 on the float32 matrix instructions.  Width 256 spills (24
//                  to 48 bytes a lane in bf16, 560 to 648 in float32) and runs at 590 TFLOP/s in
//                  bf16.
//   attn_keys_mx4  few rows (single tokens, drafts): tiles of 16 rows on 16x16
//                  instructions.  A wave holds S^T [key, row] = K Q^T; lane l has the key
//                  (as operand) or row (as result) l % 16.  The head's elements are split
//                  over the four groups of 16 lanes, DP / 4 neighbouring ones each: the
//                  contraction may take them in any order as long as q is in the same,
//                  and a lane then needs one run of codes of its key (16 bytes at width
//                  128, one MX block with one scale).  So K goes from memory to the
//                  matrix instruction in registers.  V has to be transposed: it is decoded
//                  the same way, written to the wave's LDS as rows of values and read
//                  with transposing loads.  Bound by HBM for long sequences (three of 31191 to
//                  131000 keys, 261 MB: 44 us where the Infinity Cache helps, 52 without, 5.0
//                  TB/s), by its start, six steps a wave and its end for a batch (32 tokens
//                  over 196 to 4096 keys, 70 MB: 19 us), by its chain of loads for one token (257
//                  keys 5.9 us).  Scalar page lookups and constant lane offsets took 75 to 69
//                  us and 733 to 684 for chunks beside tokens; the rest of the way was the code
//                  registers (see the loop).
#pragma once

#include "attn_kernels.cuh"
#include "mx4.cuh"

namespace sffn {

struct AttnMx4Args {
  AttnArgs a;
  Mx4Rows k, v;
  FastDiv heads, tiles;  // key heads; attn_keys_mx4: tiles_per_seq
  int alike;             // see RowPlace
};

// Words of codes of a row's elements at, at + 8, ...; row: its first word (4-byte aligned).
// From head_dim on there is nothing to load: 0.  (32 tokens of 32 + 8 heads of 80: 30 us; with the
// row's last word in place of nothing 37, with whole runs from before the row's end, which
// are not aligned, 57.)
template <int W, bool WHOLE>
__device__ __forceinline__ void load_codes(const uint8_t* row, int at, int D, uint32_t (&w)[W]) {
  if constexpr (WHOLE) {
    constexpr int kN = W < 4 ? W : 4;
    typedef uint32_t vec_t __attribute__((ext_vector_type(kN), aligned(4)));
#pragma unroll
    for (int i = 0; i < W; i += kN) {
      const vec_t v = *(const vec_t*)(row + at / 2 + 4 * i);
#pragma unroll
      for (int j = 0; j < kN; ++j) w[i + j] = v[j];
    }
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = at + 8 * i < D ? *(const uint32_t*)(row + at / 2 + 4 * i) : 0u;
  }
}

// The scale bytes of a row's blocks from number b on, with the last one's beyond it.
template <int B, bool WHOLE>
__device__ __forceinline__ void load_scales(const uint8_t* row, int b, int n_blocks, uint32_t (&s)[B]) {
#pragma unroll
  for (int i = 0; i < B; ++i) s[i] = row[WHOLE ? b + i : min(b + i, n_blocks - 1)];
}

// float32 queries: a value and its rest in bfloat16, three of them exactly the 24 bits that
// float32 has (cut off, not rounded, so that nothing overflows).  What a 4-bit cache holds
// is bfloat16, so a product with float32 is three with bfloat16 and their sum, all in
// float32: five times as fast as on the float32 matrix instructions, and as exact.
__device__ __forceinline__ float cut(float x) { return __uint_as_float(__float_as_uint(x) & 0xffff0000u); }
// The upper halves of two: the second in the upper half of the result.
__device__ __forceinline__ uint32_t pack_cut(float a, float b) {
  return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}
// Parts 0 .. 2 of pairs of values, largest first.  An infinite or NaN one has no rest.
template <int N>
__device__ __forceinline__ void split_parts(const float (&x)[2 * N], uint32_t (&o)[3][N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float r[2][2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float v = x[2 * i + j];  // a NaN is a quiet one: it stays one when it is cut
      const bool fine = (__float_as_uint(v) & 0x7f800000u) != 0x7f800000u;
      r[0][j] = fine ? v - cut(v) : 0.f;
      r[1][j] = r[0][j] - cut(r[0][j]);
    }
    o[0][i] = pack_cut(x[2 * i], x[2 * i + 1]);
    o[1][i] = pack_cut(r[0][0], r[0][1]);
    o[2][i] = pack_cut(r[1][0], r[1][1]);
  }
}

// ------------------------------------------------------------------ many rows
// Where a row of codes and its scales lie.
//   G = 16  page_size is a multiple of 16 and the caches are alike: a wave's 16
//           neighbouring rows lie in one page, which is looked up with scalar instructions,
//           and a lane adds an offset that never changes.
//   G = 0   any page size and strides: a lane looks up its own row.
// Caches are alike where K and V have the same strides, of less than 2^24 bytes for a token
// and 2^31 for a page.
template <int G>
struct RowPlace {
  int page, off;

  // j: the row (G = 0), or the first of the wave's (G = 16).
  __device__ __forceinline__ void look_up(const int32_t* bt, const FastDiv& per_page, int j, int first, int last) {
    if constexpr (G > 0) j = min(max(j, first & -G), last & -G);
    else j = min(max(j, first), last);
    const int pg = per_page.div(j);
    off = j - pg * per_page.d;
    if constexpr (G > 0) page = load_uniform(bt + pg);
    else page = bt[pg];
  }
  // Bytes from the start of the cache to that row, near: strides of alike caches.
  __device__ __forceinline__ uint64_t near(int last_page, int64_t page_bytes, int64_t token_bytes) const {
    const uint32_t pg = (uint32_t)min(max(page, 0), last_page);
    return (uint64_t)pg * (uint32_t)page_bytes + (uint64_t)(uint32_t)off * (uint32_t)token_bytes;
  }
  __device__ __forceinline__ uint64_t far(int last_page, int64_t page_bytes, int64_t token_bytes) const {
    return min(max(page, 0), last_page) * page_bytes + off * token_bytes;
  }
  __device__ __forceinline__ uint64_t bytes(int last_page, int64_t page_bytes, int64_t token_bytes) const {
    return G > 0 ? near(last_page, page_bytes, token_bytes) : far(last_page, page_bytes, token_bytes);
  }
};

// Tiles of KT rows of one cache: every thread has kPer elements of one row of a tile.  Pages
// are looked up two tiles ahead, codes loaded one ahead, and turned into values in LDS
// in the layout of AttnTile (from head_dim to the end of an LDS row: 0).
template <int DP, int KT, int NT, int G, bool WHOLE, bool K>
struct Mx4Loader {
  typedef uint16_t T;  // of the values in LDS
  typedef AttnTile<T, DP, KT> Tile;
  static constexpr int kPer = KT * Tile::kRowElems / NT;
  static constexpr int kParts = Tile::kRowElems / kPer;  // threads of a row
  static constexpr int kW = kPer / 8;
  static constexpr int kB = kPer < kMxBlock ? 1 : kPer / kMxBlock;
  static_assert(kPer % 8 == 0 && kPer * kParts == Tile::kRowElems && kWave / kParts == 16, "");
  const int32_t* bt;
  const uint8_t *codes, *scales;  // of the key head
  int64_t page_bytes, token_bytes, s_page, s_token;
  uint32_t lane_codes, lane_scales;  // G > 0: this lane's row, from the wave's first
  FastDiv per_page;
  int last_page, first, last, row, part, D;
  RowPlace<G> at;
  uint32_t w[kW], s[kB];

  __device__ __forceinline__ void init(const AttnArgs& a, const Mx4Rows& c, int seq, int hk, int lo, int hi) {
    row = (int)threadIdx.x / kParts, part = (int)threadIdx.x % kParts;
    bt = a.p.block_table + (size_t)seq * a.p.max_pages;
    codes = c.codes + hk * c.head;
    scales = c.scales + hk * c.s_head;
    page_bytes = c.page, token_bytes = c.token, s_page = c.s_page, s_token = c.s_token;
    const int r = G > 0 ? lane_id() / kParts : 0;
    lane_codes = (uint32_t)r * (uint32_t)c.token + (WHOLE ? part * (kPer / 2) : 0);
    lane_scales = (uint32_t)r * (uint32_t)c.s_token + (WHOLE ? part * kPer / kMxBlock : 0);
    per_page = a.page;
    last_page = a.p.n_pages - 1;
    first = lo, last = hi - 1;
    D = a.p.D;
  }
  __device__ __forceinline__ void look_up(int j0) {
    at.look_up(bt, per_page, j0 + (G > 0 ? uniform(row) : row), first, last);
  }
  __device__ __forceinline__ void start() {
    const uint8_t* c = codes + at.bytes(last_page, page_bytes, token_bytes) + lane_codes;
    const uint8_t* b = scales + at.bytes(last_page, s_page, s_token) + lane_scales;
    load_codes<kW, WHOLE>(c, WHOLE ? 0 : part * kPer, D, w);
    load_scales<kB, WHOLE>(b, WHOLE ? 0 : part * kPer / kMxBlock, mx_blocks(D), s);
  }
  // Eight neighbouring threads, two rows' parts, write 16 bytes each at a time: their words
  // go in an order of their own, so that the eight lie in different banks (in the same
  // order 270 of 675 M LDS cycles were conflicts, now none: 2.15 -> 2.09 ms for a 16384-token
  // prompt, but 664 -> 673 us for chunks beside single tokens).
  __device__ __forceinline__ void finish(uint8_t* tile) {
    const int odd = row & 1;
    const int first = kW == 2 ? (K ? 0 : odd) : kW == 4 ? (part & 2) | (K ? 0 : odd) : K ? part * 2 : part;
#pragma unroll
    for (int bit = 1; bit < kW; bit *= 2)
#pragma unroll
      for (int i = 0; i < kW; ++i)
        if ((i & bit) == 0) {
          const uint32_t x = w[i], y = w[i | bit];
          w[i] = first & bit ? y : x;
          w[i | bit] = first & bit ? x : y;
        }
    const int swz = K ? Tile::swz_k(row) : Tile::swz_v(row);
    const int at = row * Tile::kPitch + (((part * kW + first) ^ swz) << 4);  // of word `first`
#pragma unroll
    for (int i = 0; i < kW; ++i) {
      u32x4_t x[1];
      // a thread's words have one scale, or (width 256) two, of four each
      const uint32_t b = kB == 1 ? s[0] : (i ^ first) & 4 ? s[kB - 1] : s[0];
      Mx<T>::decode8(w[i], mx_scale(b), x);
      *(u32x4_t*)(tile + (at ^ (i << 4))) = x[0];
    }
  }
};

// The tile of the rows kernel: that of a bfloat16 cache, with float32 queries and weights in
// three parts.
template <typename T, int DP, int KT> struct RowsTile : AttnTile<uint16_t, DP, KT> {};
template <int DP, int KT> struct RowsTile<float, DP, KT> : AttnTile<uint16_t, DP, KT> {
  typedef AttnTile<uint16_t, DP, KT> Base;
  typedef Frag<uint16_t> F;
  u32x4_t qs[3][Base::kQ];

  __device__ __forceinline__ void load_q(const float* row, int D) {
    const int h = lane_id() >> 5;
#pragma unroll
    for (int i = 0; i < Base::kQ; ++i) {
      const int e = (2 * i + h) * 8;
      float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (e < D) {
        Elt<float>::unpack(ldg16(row + e), x);
        Elt<float>::unpack(ldg16(row + e + 4), x + 4);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = __builtin_canonicalizef(x[j]);
      }
      uint32_t p[3][4];
      split_parts<4>(x, p);
#pragma unroll
      for (int k = 0; k < 3; ++k) qs[k][i] = u32x4_t{p[k][0], p[k][1], p[k][2], p[k][3]};
    }
  }
  __device__ __forceinline__ void negate() {
#pragma unroll
    for (int k = 0; k < 3; ++k)
#pragma unroll
      for (int i = 0; i < Base::kQ; ++i) qs[k][i] = F::negate(qs[k][i]);
  }
  __device__ __forceinline__ f32x16_t scores(const uint8_t* k) const {
    const int lane = lane_id(), r = lane & 31, h = lane >> 5;
    const int at = r * Base::kPitch + ((h ^ Base::swz_k(r)) << 4);
    f32x16_t s;
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = 0.f;
#pragma unroll
    for (int i = 0; i < Base::kQ; ++i) {
      const u32x4_t a = *(const u32x4_t*)(k + (at ^ (i << 5)));
#pragma unroll
      for (int p = 2; p >= 0; --p) s = F::mma(a, qs[p][i], s);
    }
    return s;
  }
  __device__ __forceinline__ void accumulate(const uint8_t* v, const f32x16_t& s) {
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      float x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = s[8 * ks + j];
      uint32_t p[3][4];
      split_parts<4>(x, p);
#pragma unroll
      for (int d = 0; d < Base::kDt; ++d) {
        const u32x4_t f = Base::v_frag(v, ks, d);
#pragma unroll
        for (int k = 2; k >= 0; --k)
          this->o[d] = F::mma(f, u32x4_t{p[k][0], p[k][1], p[k][2], p[k][3]}, this->o[d]);
      }
    }
  }
  __device__ __forceinline__ void step(f32x16_t& s, const uint8_t* k_next, const uint8_t* v, float c) {
    this->raise(s, c);
    const f32x16_t next = scores(k_next);
    this->weights(s, c);
    accumulate(v, s);
    s = next;
  }
};

template <typename T, int DP, int KT, int NW, int G, bool WHOLE>
__global__ __launch_bounds__(NW * 64, DP <= (sizeof(T) == 2 ? 128 : 64) ? 2 : 1) void attn_rows_mx4(
    AttnMx4Args m) {
  typedef RowsTile<T, DP, KT> Tile;
  constexpr int TM = NW * 32;
  __shared__ __align__(1024) uint8_t k0[Tile::kTileBytes], k1[Tile::kTileBytes], v0[Tile::kTileBytes],
      v1[Tile::kTileBytes];
  const AttnArgs& a = m.a;
  const PagedAttn& p = a.p;
  // the order of the workgroups is that of attn_rows
  const int all = (int)(gridDim.x * gridDim.y);
  int id = (int)(blockIdx.y * gridDim.x + blockIdx.x);
  if (DP <= 128 && all <= 2 * kCus && id >= kCus) id = all - 1 - (id - kCus);
  const int split = id / (int)gridDim.x, th = id - split * (int)gridDim.x;
  const int hk = th % p.hkv, t = th / p.hkv;
  RowsPlace pl;
  if (!pl.template init<TM>(a, t, hk, split)) return;
  const int b = pl.b, e = pl.e, x = pl.x, y = pl.y;
  Tile tile;
  tile.init();
  Mx4Loader<DP, KT, NW * 64, G, WHOLE, true> load_k;
  Mx4Loader<DP, KT, NW * 64, G, WHOLE, false> load_v;
  load_k.init(a, m.k, pl.w.seq, hk, b, e);
  load_v.init(a, m.v, pl.w.seq, hk, b, e);
  // as in attn_rows the K tile beside a V tile is 32 keys ahead of it
  f32x16_t s;
  int j0 = b & ~(KT - 1);
  if (e > b) {
    load_k.look_up(j0 + 32 - KT);
    load_v.look_up(j0);
    load_k.start();
    load_v.start();
    tile.load_q((const T*)p.q + pl.q_offset(p), p.D);
    load_k.look_up(j0 + 32);
    load_k.finish(k1);
    load_k.start();
    load_v.look_up(j0 + KT);
    load_v.finish(v0);
    load_v.start();
    load_k.look_up(j0 + KT + 32);
    load_v.look_up(j0 + 2 * KT);
    load_k.finish(k0);
    load_k.start();
    load_k.look_up(j0 + 2 * KT + 32);
    if (a.negate) tile.negate();
    __syncthreads();
    s = tile.scores(k1 + KT * Tile::kPitch - Tile::kBlockBytes);
    __syncthreads();  // k1 has been read
  }
  auto iteration = [&](uint8_t* k, uint8_t* v, uint8_t* k_next, uint8_t* v_next) __attribute__((always_inline)) {
    // the next tiles: their codes have been on their way for a whole iteration
    if (j0 + KT < e) {
      load_k.finish(k_next);
      load_v.finish(v_next);
      if (j0 + 2 * KT < e) {
        load_k.start();
        load_v.start();
        load_k.look_up(j0 + 3 * KT + 32);
        load_v.look_up(j0 + 3 * KT);
      }
    }
    if (!(j0 >= x && j0 + KT <= y) &&  // some row of the workgroup does not see some key
        __syncthreads_or(Tile::template find_infinite<NW * 64>(v, threadIdx.x))) {
      if (__syncthreads_or(Tile::template find_infinite_in<NW * 64, 1>(v, threadIdx.x, b - j0, e - j0))) {
        tile.add_infinite(v, j0, pl.row_lo, pl.row_hi);
        __syncthreads();
      }
      Tile::template clear_infinite<NW * 64>(v, threadIdx.x);
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < KT / 32; ++i) {
      const int j = j0 + i * 32;
      if (pl.sees_none(j)) {
        s = tile.scores(k + i * Tile::kBlockBytes);
      } else {
        if (!pl.sees_all(j)) Tile::hide(s, j, pl.row_lo, pl.row_hi);
        tile.step(s, k + i * Tile::kBlockBytes, v + i * Tile::kBlockBytes, a.c);
      }
    }
    j0 += KT;
    __syncthreads();  // k and v have been read, the next ones are in LDS
  };
  while (j0 < e) {
    iteration(k0, v0, k1, v1);
    if (j0 >= e) break;
    iteration(k1, v1, k0, v0);
  }
  write_rows<T, TM>(a, pl, tile, t, hk, split);
}

// ------------------------------------------------------------------ few rows

__device__ __forceinline__ f32x4_t mma16(u32x4_t a, u32x4_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                 __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

// Over the four lanes with one l % 16.
__device__ __forceinline__ float max_quads(float v) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return max_halves(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}
__device__ __forceinline__ float sum_quads(float v) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return sum_halves(__uint_as_float(r[0]) + __uint_as_float(r[1]));
}

// RT tiles of 16 rows over blocks of 32 keys.  DP: 64, 128 or 256.
template <typename T, int DP, int RT>
struct KeysTile {
  static constexpr int kLane = DP / 4;                       // elements of a lane
  static constexpr int kW = kLane / 8;                       // its words of codes
  static constexpr int kB = kLane < kMxBlock ? 1 : kLane / kMxBlock;  // its scales
  static constexpr int kParts = sizeof(T) == 2 ? 1 : 3;      // of queries and weights
  static constexpr int kDt = DP / 16;                        // 16-wide blocks of the output
  static constexpr int kPitch = DP * 2;                      // of a row of V in LDS
  static constexpr int kVBytes = 32 * kPitch;
  static constexpr int kOutBytes = RT * 16 * DP * 4;
  static constexpr int kLdsBytes = kVBytes > kOutBytes ? kVBytes : kOutBytes;

  // Chunk c of row r lies at c ^ swz(r).  Rows are written by 16 lanes, a row each, at one
  // chunk: eight neighbouring rows get different chunks.  They are read as 32 bytes of four
  // neighbouring rows.
  __device__ static __forceinline__ int swz(int r) { return ((r & 3) << 1) | ((r >> 2) & 1); }

  u32x4_t q[RT][kParts][kW];
  f32x4_t o[RT][kDt];
  float m[RT], l[RT];

  __device__ __forceinline__ void init() {
#pragma unroll
    for (int t = 0; t < RT; ++t) {
#pragma unroll
      for (int d = 0; d < kDt; ++d) o[t][d] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      m[t] = -INFINITY;
      l[t] = 0.f;
    }
  }
  // Loads without conditions, so that they are in flight together; finish_q once they are
  // all under way.
  static constexpr int kRaw = kW * (int)sizeof(T) / 2;  // 16-byte loads of a row
  template <bool WHOLE>
  __device__ static __forceinline__ void load_q(const T* row, int D, u32x4_t (&raw)[kRaw]) {
    constexpr int kEpc = 16 / (int)sizeof(T);
    const int e0 = (lane_id() >> 4) * kLane;
#pragma unroll
    for (int i = 0; i < kRaw; ++i) raw[i] = ldg16(row + (WHOLE ? e0 + i * kEpc : min(e0 + i * kEpc, D - kEpc)));
  }
  template <bool WHOLE>
  __device__ __forceinline__ void finish_q(int t, int D, bool negate, const u32x4_t (&raw)[kRaw]) {
    const int e0 = (lane_id() >> 4) * kLane;
    const uint32_t sign = negate ? 0x80008000u : 0u;
#pragma unroll
    for (int i = 0; i < kW; ++i) {
      if constexpr (sizeof(T) == 2) {
        q[t][0][i] = raw[i];
      } else {
        float x[8];
        Elt<float>::unpack(raw[2 * i], x);
        Elt<float>::unpack(raw[2 * i + 1], x + 4);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = __builtin_canonicalizef(x[j]);
        uint32_t p[3][4];
        split_parts<4>(x, p);
#pragma unroll
        for (int k = 0; k < 3; ++k) q[t][k][i] = u32x4_t{p[k][0], p[k][1], p[k][2], p[k][3]};
      }
#pragma unroll
      for (int k = 0; k < kParts; ++k) {
        if (!WHOLE && e0 + 8 * i >= D) q[t][k][i] = u32x4_t{0u, 0u, 0u, 0u};
        q[t][k][i] ^= sign;
      }
    }
  }

  // Codes and scales of one row of K or V, this lane's part.
  struct Codes {
    uint32_t w[kW], s[kB];
  };
  // Word i's scale.  A NaN block of V counts as (about) 0 here: 0 times NaN would be NaN for
  // the rows that do not see it.  The rows that do get their NaN at the end.
  static __device__ __forceinline__ float scale_k(const Codes& c, int i) {
    return mx_scale(c.s[i / 4 < kB ? i / 4 : 0]);
  }
  static __device__ __forceinline__ float scale_v(const Codes& c, int i) {
    const uint32_t s = c.s[i / 4 < kB ? i / 4 : 0];
    return __uint_as_float((s >= kMxBad ? 0u : s) << 23);
  }

  // Scores of 16 keys: s[t] has the keys 4 (lane / 16) + i of row lane % 16.
  __device__ __forceinline__ void scores(const Codes& k, f32x4_t (&s)[RT]) const {
#pragma unroll
    for (int t = 0; t < RT; ++t) s[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < kW; ++i) {
      u32x4_t x[1];
      Mx<uint16_t>::decode8(k.w[i], scale_k(k, i), x);
#pragma unroll
      for (int p = kParts - 1; p >= 0; --p)
#pragma unroll
        for (int t = 0; t < RT; ++t) s[t] = mma16(x[0], q[t][p][i], s[t]);
    }
  }

  // V rows b * 16 + lane % 16 to LDS.
  __device__ static __forceinline__ void write_v(uint8_t* lds, int b, const Codes& v) {
    const int lane = lane_id(), r = b * 16 + (lane & 15), c0 = (lane >> 4) * kW;
#pragma unroll
    for (int i = 0; i < kW; ++i) {
      u32x4_t x[1];
      Mx<uint16_t>::decode8(v.w[i], scale_v(v, i), x);
      *(u32x4_t*)(lds + r * kPitch + (((c0 + i) ^ swz(r)) << 4)) = x[0];
    }
  }

  // o += V^T P^T over the 32 keys in LDS.  A lane's weights are those of the keys 4 (lane / 16)
  // + i and 16 more: the order in which the B operand takes them when V^T is read alike.  In
  // bf16 they are rounded to bf16 here, as in AttnTile::accumulate (their sum l is not), since the
  // matrix instruction takes both operands in one type and two parts would be twice the products:
  // relative error against 64 bits 2.0e-3 to 2.35e-3 where rounding the output alone gives
  // 1.5e-3 to 1.7e-3 (standard normal inputs).  In float32 three parts keep all 24 bits.
  __device__ __forceinline__ void accumulate(const uint8_t* lds, const f32x4_t (&s)[2][RT]) {
    const int lane = lane_id(), i = lane & 15, g = lane >> 4;
    u32x4_t pf[RT][kParts];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      if constexpr (sizeof(T) == 2) {
        pf[t][0] = u32x4_t{pack_bf16(s[0][t][0], s[0][t][1]), pack_bf16(s[0][t][2], s[0][t][3]),
                           pack_bf16(s[1][t][0], s[1][t][1]), pack_bf16(s[1][t][2], s[1][t][3])};
      } else {
        const float x[8] = {s[0][t][0], s[0][t][1], s[0][t][2], s[0][t][3],
                            s[1][t][0], s[1][t][1], s[1][t][2], s[1][t][3]};
        uint32_t p[3][4];
        split_parts<4>(x, p);
#pragma unroll
        for (int k = 0; k < 3; ++k) pf[t][k] = u32x4_t{p[k][0], p[k][1], p[k][2], p[k][3]};
      }
    }
    const int r = 4 * g + (i >> 2);  // swz(r + 16) is swz(r)
    const int at = r * kPitch + ((((i & 3) >> 1) ^ swz(r)) << 4) + (i & 1) * 8;
    typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;
#pragma unroll
    for (int d = 0; d < kDt; ++d) {
      const uint8_t* v = lds + (at ^ (d << 5));
      const s16x4_t x0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)v);
      const s16x4_t x1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(v + 16 * kPitch));
      const u32x4_t f = __builtin_bit_cast(u32x4_t, __builtin_shufflevector(x0, x1, 0, 1, 2, 3, 4, 5, 6, 7));
#pragma unroll
      for (int p = kParts - 1; p >= 0; --p)
#pragma unroll
        for (int t = 0; t < RT; ++t) o[t][d] = mma16(f, pf[t][p], o[t][d]);
    }
  }

  // As in AttnTile, of the 32 keys whose scores are in s.
  __device__ __forceinline__ void raise(int t, const f32x4_t& a, const f32x4_t& b, float c) {
    float mx = a[0];
#pragma unroll
    for (int i = 1; i < 4; ++i) mx = fmaxf(mx, a[i]);
#pragma unroll
    for (int i = 0; i < 4; ++i) mx = fmaxf(mx, b[i]);
    const float mn = fmaxf(m[t], max_quads(mx));
    if (__any((mn - m[t]) * c > 8.f)) {
      const float f = m[t] == -INFINITY ? 1.f : __builtin_amdgcn_exp2f((m[t] - mn) * c);
      l[t] *= f;
#pragma unroll
      for (int d = 0; d < kDt; ++d) o[t][d] *= f;
      m[t] = mn;
    }
  }
  __device__ __forceinline__ void weights(int t, f32x4_t& s, float c) {
    const float mc = m[t] == -INFINITY ? 0.f : m[t] * c;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], c, -mc));
      l[t] += s[i];
    }
  }
};

// The rows of K and V of a wave's blocks of 32 keys: lane l has key l % 16 of both halves.
// Pages are looked up one block before codes are loaded.
template <typename T, int DP, int RT, int G, bool WHOLE>
struct KeysLoader {
  typedef KeysTile<T, DP, RT> Tile;
  const int32_t* bt;
  Mx4Rows k, v;                  // of the key head
  uint32_t lane_codes, lane_scales;  // G > 0: this lane's row, from the one that was looked up
  FastDiv per_page;
  int last_page, first, last, D, e0;
  bool alike;
  RowPlace<G> at[2];

  __device__ __forceinline__ void init(const AttnMx4Args& m, int seq, int hk, int lo, int hi) {
    e0 = (lane_id() >> 4) * Tile::kLane;
    bt = m.a.p.block_table + (size_t)seq * m.a.p.max_pages;
    k = m.k, v = m.v;
    k.codes += hk * k.head, k.scales += hk * k.s_head;
    v.codes += hk * v.head, v.scales += hk * v.s_head;
    const uint32_t r = G > 0 ? lane_id() & 15 : 0;
    lane_codes = r * (uint32_t)k.token, lane_scales = r * (uint32_t)k.s_token;
    alike = m.alike != 0;
    per_page = m.a.page;
    last_page = m.a.p.n_pages - 1;
    first = lo, last = hi - 1;
    D = m.a.p.D;
  }
  __device__ __forceinline__ void look_up(int j0) {
#pragma unroll
    for (int b = 0; b < 2; ++b)
      at[b].look_up(bt, per_page, j0 + 16 * b + (G > 0 ? 0 : lane_id() & 15), first, last);
  }
  __device__ __forceinline__ void one(const uint8_t* codes, const uint8_t* scales, typename Tile::Codes& x) const {
    load_codes<Tile::kW, WHOLE>(codes, e0, D, x.w);
    load_scales<Tile::kB, WHOLE>(scales, e0 / kMxBlock, mx_blocks(D), x.s);
  }
  __device__ __forceinline__ void start(typename Tile::Codes (&kc)[2], typename Tile::Codes (&vc)[2]) const {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      if (G > 0 || alike) {  // one place in both caches, products of 32-bit strides
        const uint64_t c = at[b].near(last_page, k.page, k.token) + lane_codes;
        const uint64_t s = at[b].near(last_page, k.s_page, k.s_token) + lane_scales;
        one(k.codes + c, k.scales + s, kc[b]);
        one(v.codes + c, v.scales + s, vc[b]);
      } else {
        one(k.codes + at[b].far(last_page, k.page, k.token), k.scales + at[b].far(last_page, k.s_page, k.s_token), kc[b]);
        one(v.codes + at[b].far(last_page, v.page, v.token), v.scales + at[b].far(last_page, v.s_page, v.s_token), vc[b]);
      }
    }
  }
};

// Rows of an attn_keys_mx4 tile: two tiles of 16 share what is decoded where the registers
// hold their outputs.
constexpr int keys_mx4_rows(int elt_bytes, int head_dim, int64_t rows) {
  return rows > 16 && elt_bytes == 2 && head_dim <= 128 ? 32 : 16;
}
// Waves of a workgroup: eight where the longest key range that its tiles can see is short
// enough for eight to walk over it in five steps, so that it is not split, four otherwise.
// 24 drafts in a window of 1000 (8 heads a key head, width 64): 9.8 us, in splits of four
// waves and a join 18.7; but split ranges of 32 tokens over up to 4096 keys: 22.8 us with four
// waves, 26.0 with eight; float32 chunks (of 16 rows) 78.0 and 80.8.
constexpr int kKeysWhole = 8 * 32 * 5;
constexpr int keys_mx4_waves(int elt_bytes, int64_t span) { return elt_bytes == 2 && span <= kKeysWhole ? 8 : 4; }
// Waves of a SIMD that the registers are meant for.
constexpr int keys_mx4_occupancy(int elt_bytes, int dp, int row_tiles, bool compact) {
  if (elt_bytes == 4) return dp > 128 ? 1 : 2;
  if (dp > 128) return compact ? 1 : 2;
  return row_tiles == 2 ? 2 : compact ? 3 : 4;
}

// The wave's keys once more, where one of them had a NaN block of V: rows that see its key
// get NaN in the block's elements.  Out of the way of the loop: on the rows that the wave has
// left in LDS, by lane.
template <typename T, int DP, int RT, int G, typename Loader>
__device__ __forceinline__ void mark_nan(const AttnMx4Args& m, Loader& load, const Work& w, int hk, int r0, int rows,
                                      int j0, int end, int step, uint8_t* lds) {
  const AttnArgs& a = m.a;
  const int lane = lane_id(), n_blocks = mx_blocks(a.p.D);
  for (; j0 < end; j0 += step) {
    load.look_up(j0);
    for (int h = 0; h < 2; ++h) {
      const uint8_t* row = load.v.scales + load.at[h].bytes(load.last_page, load.v.s_page, load.v.s_token) +
                           (G > 0 ? (int64_t)(lane & 15) * load.v.s_token : 0);
      for (int n = 0; n < n_blocks; ++n) {
        uint64_t bad = __ballot(lane < 16 && row[n] >= kMxBad);
        while (bad != 0) {
          const int j = j0 + 16 * h + (int)__builtin_ctzll(bad);
          bad &= bad - 1;
          for (int r = 0; r < rows; ++r) {
            int lo, hi;
            key_range(a.p, w, a.group.div(r0 + r), &lo, &hi);
            const int e = n * kMxBlock + lane;
            if (j >= lo && j < hi && lane < kMxBlock && e < a.p.D)
              *(float*)(lds + r * (DP * 4) + (((e / 4) ^ (r & 7)) << 4) + (e & 3) * 4) = __builtin_nanf("");
          }
        }
      }
    }
  }
}

template <typename T, int DP, int RT, int NW, int G, bool WHOLE, bool COMPACT>
__global__ __launch_bounds__(NW * 64, keys_mx4_occupancy(sizeof(T), DP, RT, COMPACT)) void attn_keys_mx4(AttnMx4Args args) {
  typedef KeysTile<T, DP, RT> Tile;
  constexpr int TM = 16 * RT;
  __shared__ __align__(1024) uint8_t lds[NW][Tile::kLdsBytes];
  __shared__ float ml[NW][TM][2];
  const AttnArgs& a = args.a;
  const PagedAttn& p = a.p;
  const int wave = uniform((int)threadIdx.x / kWave), lane = lane_id(), quad = lane >> 4;
  uint8_t* const mine = lds[wave];
  // items as in attn_keys
  KeysItems<TM> items;
  if constexpr (COMPACT) items.init(a);
  for (int item = blockIdx.x;; item += gridDim.x) {
    KeysWork kw;
    const int hk = item - args.heads.div(item) * p.hkv;
    if constexpr (COMPACT) {
      if (!items.get(a, args.heads.div(item), &kw)) break;
    } else {
      kw.split = blockIdx.y;
      const int t = args.heads.div(item), s = args.tiles.div(t);
      read_sequence(p, s, &kw.w);
      kw.w.tile = t - s * a.tiles_per_seq;
      const int all = kw.w.nq * a.g;
      if (kw.w.tile * TM >= all || all > a.max_rows) break;
      sequence_range(a, &kw);
      if (kw.split >= kw.n_split) break;
    }
    const Work w = kw.w;
    const int r0 = w.tile * TM, rows = min(TM, w.nq * a.g - r0);
    int lo, hi, b, e, x, y;
    key_range(p, w, a.group.div(r0), &lo, &y);
    key_range(p, w, a.group.div(r0 + rows - 1), &x, &hi);
    split_range(a, kw.split, kw.lo, kw.hi, &b, &e);
    b = max(b, lo);
    e = min(e, hi);
    int row_lo[RT], row_hi[RT];
    Tile tile;
    tile.init();
    KeysLoader<T, DP, RT, G, WHOLE> load;
    load.init(args, w.seq, hk, b, e);
    int j0 = (b & ~31) + wave * 32;
    const int end = b < e ? e : j0, step = NW * 32;
    typename Tile::Codes kc[2], vc[2];
    uint32_t worst = 0;  // scale byte of V
    if (j0 < end) {
      load.look_up(j0);
      load.start(kc, vc);
      load.look_up(j0 + step);
    }
    u32x4_t raw[RT][Tile::kRaw];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const int r = r0 + min(16 * t + (lane & 15), rows - 1);
      const int token = a.group.div(r), head = hk * a.g + r - token * a.g;
      key_range(p, w, token, &row_lo[t], &row_hi[t]);
      Tile::template load_q<WHOLE>((const T*)p.q + (int64_t)(w.q0 + token) * p.q_token + head * p.q_head, p.D,
                                   raw[t]);
    }
#pragma unroll
    for (int t = 0; t < RT; ++t) tile.template finish_q<WHOLE>(t, p.D, a.negate, raw[t]);
    // Blocks of 32 keys.  Once a block's codes have become operands those of the next are
    // loaded in their place: with four waves a SIMD that is enough under way (with a second
    // set of registers and three waves: decode of 32 tokens 25.0 us instead of 23.1, of three
    // long sequences 69.2 instead of 59.4).
    for (; j0 < end; j0 += step) {
      const bool whole = j0 >= x && j0 + 32 <= y;
      f32x4_t s[2][RT];
#pragma unroll
      for (int h = 0; h < 2; ++h) tile.scores(kc[h], s[h]);
      if (!whole) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int j = j0 + 16 * h + 4 * quad + i;
              s[h][t][i] = j >= row_lo[t] && j < row_hi[t] ? s[h][t][i] : -INFINITY;
            }
          // keys that no row sees are loaded with their neighbours: what lies there, the end of
          // a page or what was before a window, is no NaN block to look for (one
          // such byte: 41 us instead of 26 for a token over 131072 keys, 280 and 139 over 2^20)
          const int j = j0 + 16 * h + (lane & 15);
#pragma unroll
          for (int n = 0; n < Tile::kB; ++n) vc[h].s[n] = j >= b && j < e ? vc[h].s[n] : 0u;
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int n = 0; n < Tile::kB; ++n) worst = max(worst, vc[h].s[n]);
#pragma unroll
      for (int h = 0; h < 2; ++h) Tile::write_v(mine, h, vc[h]);
      if (j0 + step < end) {
        load.start(kc, vc);
        load.look_up(j0 + 2 * step);
      }
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        tile.raise(t, s[0][t], s[1][t], a.c);
        tile.weights(t, s[0][t], a.c);
        tile.weights(t, s[1][t], a.c);
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      tile.accumulate(mine, s);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    // Join the waves: each leaves its rows in its LDS, row r's 16-byte chunk c at c ^ (r % 8).
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const int row = 16 * t + (lane & 15);
      const float l = sum_quads(tile.l[t]);
#pragma unroll
      for (int d = 0; d < Tile::kDt; ++d)
        *(f32x4_t*)(mine + row * (DP * 4) + (((4 * d + quad) ^ (row & 7)) << 4)) = tile.o[t][d];
      if (quad == 0) {
        ml[wave][row][0] = tile.m[t] * a.c;
        ml[wave][row][1] = l;
      }
    }
    if (__any(worst >= kMxBad)) {
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      mark_nan<T, DP, RT, G>(args, load, w, hk, r0, rows, (b & ~31) + wave * 32, end, step, mine);
    }
    __syncthreads();
    const int quads = p.D / 4;
    for (int i = threadIdx.x; i < rows * quads; i += NW * 64) {
      const int rr = i / quads, c = i - rr * quads, d = c * 4;
      float m = -INFINITY, l = 0.f;
#pragma unroll
      for (int k = 0; k < NW; ++k) m = fmaxf(m, ml[k][rr][0]);
      f32x4_t v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < NW; ++k) {
        const float mk = ml[k][rr][0];
        const float f = mk == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(mk - m);
        l += f * ml[k][rr][1];
        v += f * *(const f32x4_t*)(lds[k] + rr * (DP * 4) + ((c ^ (rr & 7)) << 4));
      }
      const int tk = a.group.div(r0 + rr), hd = hk * a.g + r0 + rr - tk * a.g;
      if (kw.n_split == 1) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        store4<T>((T*)p.out + (int64_t)(w.q0 + tk) * p.o_token + hd * p.o_head + d, v[0] * inv,
                  v[1] * inv, v[2] * inv, v[3] * inv);
        if (d == 0 && p.lse != nullptr) p.lse[(int64_t)(w.q0 + tk) * p.hq + hd] = finish_lse(m, l);
      } else {
        const size_t slot = kw.split * a.part_rows + ((size_t)w.seq * p.hkv + hk) * a.slot_rows + r0 + rr;
        *(f32x4_t*)(a.part_o + slot * p.D + d) = v;
        if (d == 0) {
          a.part_ml[2 * slot] = m;
          a.part_ml[2 * slot + 1] = l;
        }
      }
    }
    if constexpr (!COMPACT) break;
    __syncthreads();  // the waves' results are read before the next item's rows arrive
  }
}

// Launches of one element type, in files of their own.  near: rows can be looked up by 16.
template <typename T> hipError_t launch_attn_rows_mx4(const AttnMx4Args& m, bool near, hipStream_t s);
template <typename T>
hipError_t launch_attn_keys_mx4(const AttnMx4Args& m, int tile_rows, int waves, bool near, bool compact,
                                hipStream_t s);

template <typename T, int DP, bool WHOLE>
hipError_t attn_rows_mx4_go(const AttnMx4Args& m, bool near, hipStream_t s) {
  constexpr int kKeys = RowsShape<uint16_t, DP>::kKeys, kWaves = RowsShape<uint16_t, DP>::kWaves;
  const AttnArgs& a = m.a;
  const dim3 grid((unsigned)(a.n_tiles * a.p.hkv), (unsigned)a.splits), block(kWaves * 64);
  if (near) hipLaunchKernelGGL((attn_rows_mx4<T, DP, kKeys, kWaves, 16, WHOLE>), grid, block, 0, s, m);
  else hipLaunchKernelGGL((attn_rows_mx4<T, DP, kKeys, kWaves, 0, WHOLE>), grid, block, 0, s, m);
  return hipGetLastError();
}

template <typename T, int DP>
hipError_t attn_rows_mx4_width(const AttnMx4Args& m, bool near, hipStream_t s) {
  if constexpr (DP == AttnTile<uint16_t, DP, 64>::kRowElems)
    if (m.a.p.D == DP) return attn_rows_mx4_go<T, DP, true>(m, near, s);
  return attn_rows_mx4_go<T, DP, false>(m, near, s);
}

template <typename T, int DP, int RT, int G, bool WHOLE, int kWaves>
hipError_t attn_keys_mx4_go(const AttnMx4Args& m, bool compact, hipStream_t s) {
  const AttnArgs& a = m.a;
  const int64_t items = (int64_t)a.n_tiles * a.p.hkv * a.splits, most = 2 * kCus;
  const dim3 all((unsigned)(a.n_tiles * a.p.hkv), (unsigned)a.splits);
  const dim3 some((unsigned)(items < most ? items : most)), block(kWaves * 64);
  if (compact) hipLaunchKernelGGL((attn_keys_mx4<T, DP, RT, kWaves, G, WHOLE, true>), some, block, 0, s, m);
  else hipLaunchKernelGGL((attn_keys_mx4<T, DP, RT, kWaves, G, WHOLE, false>), all, block, 0, s, m);
  return hipGetLastError();
}

template <typename T, int DP, int RT, int kWaves>
hipError_t attn_keys_mx4_rows(const AttnMx4Args& m, bool near, bool compact, hipStream_t s) {
  if (!near)
    return m.a.p.D == DP ? attn_keys_mx4_go<T, DP, RT, 0, true, kWaves>(m, compact, s)
                         : attn_keys_mx4_go<T, DP, RT, 0, false, kWaves>(m, compact, s);
  return m.a.p.D == DP ? attn_keys_mx4_go<T, DP, RT, 16, true, kWaves>(m, compact, s)
                       : attn_keys_mx4_go<T, DP, RT, 16, false, kWaves>(m, compact, s);
}

// tile_rows: of keys_mx4_rows; waves: of keys_mx4_waves.
template <typename T, int DP>
hipError_t attn_keys_mx4_width(const AttnMx4Args& m, int tile_rows, int waves, bool near, bool compact,
                               hipStream_t s) {
  if constexpr (keys_mx4_rows(sizeof(T), DP, 32) == 32) {
    if (tile_rows == 32)
      return waves == 8 ? attn_keys_mx4_rows<T, DP, 2, 8>(m, near, compact, s)
                        : attn_keys_mx4_rows<T, DP, 2, 4>(m, near, compact, s);
  }
  if constexpr (sizeof(T) == 2) {
    if (waves == 8) return attn_keys_mx4_rows<T, DP, 1, 8>(m, near, compact, s);
  }
  return attn_keys_mx4_rows<T, DP, 1, 4>(m, near, compact, s);
}

}  // namespace sffn
