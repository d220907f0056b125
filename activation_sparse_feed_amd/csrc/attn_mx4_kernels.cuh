// Kernels of attention over the 4-bit paged cache.  Rows, tiles, splits and their joining
// are those of attn_kernels.cuh; what differs is how keys and values come to the matrix
// instructions: codes and scales are loaded into registers, a tile ahead, and turned into
// bfloat16 (or float32) there, with nothing rounded.
//
//   attn_rows_mx4  many rows (chunks of prompts): the tiles of attn_rows, K and V tiles
//                  written to LDS by the threads that decode them.
//   attn_keys_mx4  few rows (single tokens, drafts): tiles of 16 rows on 16x16
//                  instructions.  A wave holds S^T [key, row] = K Q^T; lane l has the key
//                  (as operand) or row (as result) l % 16.  The head's elements are split
//                  over the four groups of 16 lanes, DP / 4 neighbouring ones each: the
//                  contraction may take them in any order as long as q is in the same,
//                  and a lane then needs one run of codes of its key (16 bytes at width
//                  128, one MX block with one scale).  So K goes from memory to the
//                  matrix instruction in registers.  V has to be transposed: it is decoded
//                  the same way, written to the wave's LDS as rows of values and read
//                  with transposing loads.
#pragma once

#include "attn_kernels.cuh"
#include "mx4.cuh"

namespace sffn {

struct AttnMx4Args {
  AttnArgs a;
  Mx4Rows k, v;
};

// Words of codes at p (4-byte aligned); `at`: the element that the first belongs to.
// Elements from D on read as 0.
template <int W, bool WHOLE>
__device__ __forceinline__ void load_codes(const uint8_t* p, int at, int D, uint32_t (&w)[W]) {
  if constexpr (WHOLE) {
    constexpr int kN = W < 4 ? W : 4;
    typedef uint32_t vec_t __attribute__((ext_vector_type(kN), aligned(4)));
#pragma unroll
    for (int i = 0; i < W; i += kN) {
      if constexpr (kN == 1) {
        w[i] = *(const uint32_t*)(p + 4 * i);
      } else {
        const vec_t v = *(const vec_t*)(p + 4 * i);
#pragma unroll
        for (int j = 0; j < kN; ++j) w[i + j] = v[j];
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = at + 8 * i < D ? *(const uint32_t*)(p + 4 * i) : 0u;
  }
}

// The scale bytes of the blocks from number b on; 127 (a scale of 1) beyond the head.
template <int B, bool WHOLE>
__device__ __forceinline__ void load_scales(const uint8_t* p, int b, int n_blocks, uint32_t (&s)[B]) {
#pragma unroll
  for (int i = 0; i < B; ++i) s[i] = WHOLE || b + i < n_blocks ? p[b + i] : 127u;
}

// ------------------------------------------------------------------ many rows
// Tiles of KT rows of one cache: every thread has PER elements of one row of a tile.  Pages
// are looked up two tiles ahead, codes loaded one ahead, and turned into values in LDS
// in the layout of AttnTile (elements from head_dim to the end of an LDS row: 0).
template <typename T, int DP, int KT, int NT, bool K>
struct Mx4Loader {
  typedef AttnTile<T, DP, KT> Tile;
  static constexpr int kPer = KT * Tile::kRowElems / NT;
  static constexpr int kParts = Tile::kRowElems / kPer;  // threads of a row
  static constexpr int kW = kPer / 8;
  static constexpr int kB = kPer < kMxBlock ? 1 : kPer / kMxBlock;
  static_assert(kPer % 8 == 0 && kPer * kParts == Tile::kRowElems, "");
  const int32_t* bt;
  const uint8_t *codes, *scales;  // of the key head, at this thread's elements
  int64_t page_bytes, token_bytes, s_page, s_token;
  FastDiv per_page;
  int last_page, first, last, row, part, D;
  int page, off;
  uint32_t w[kW], s[kB];

  __device__ __forceinline__ void init(const AttnArgs& a, const Mx4Rows& c, int seq, int hk, int lo, int hi) {
    row = (int)threadIdx.x / kParts, part = (int)threadIdx.x % kParts;
    bt = a.p.block_table + (size_t)seq * a.p.max_pages;
    codes = c.codes + hk * c.head + part * (kPer / 2);
    scales = c.scales + hk * c.s_head;
    page_bytes = c.page, token_bytes = c.token, s_page = c.s_page, s_token = c.s_token;
    per_page = a.page;
    last_page = a.p.n_pages - 1;
    first = lo, last = hi - 1;
    D = a.p.D;
  }
  __device__ __forceinline__ void look_up(int j0) {
    const int j = min(max(j0 + row, first), last);
    const int pg = per_page.div(j);
    off = j - pg * per_page.d;
    page = bt[pg];
  }
  __device__ __forceinline__ void start() {
    const int64_t pg = min(max(page, 0), last_page);
    const uint8_t* c = codes + pg * page_bytes + off * token_bytes;
    const uint8_t* b = scales + pg * s_page + off * s_token;
    if (D == Tile::kRowElems) {
      load_codes<kW, true>(c, 0, D, w);
      load_scales<kB, true>(b, part * kPer / kMxBlock, 0, s);
    } else {
      load_codes<kW, false>(c, part * kPer, D, w);
      load_scales<kB, false>(b, part * kPer / kMxBlock, mx_blocks(D), s);
    }
  }
  __device__ __forceinline__ void finish(uint8_t* tile) const {
    const int swz = K ? Tile::swz_k(row) : Tile::swz_v(row);
#pragma unroll
    for (int i = 0; i < kW; ++i) {
      u32x4_t x[Mx<T>::kChunks];
      Mx<T>::decode8(w[i], mx_scale(s[i / 4 < kB ? i / 4 : 0]), x);
#pragma unroll
      for (int j = 0; j < Mx<T>::kChunks; ++j) {
        const int c = (part * kW + i) * Mx<T>::kChunks + j;
        *(u32x4_t*)(tile + row * Tile::kPitch + ((c ^ swz) << 4)) = x[j];
      }
    }
  }
};

template <typename T, int DP, int KT, int NW>
__global__ __launch_bounds__(NW * 64, DP <= 128 && sizeof(T) == 2 && NW == 4 ? 2 : 1) void attn_rows_mx4(
    AttnMx4Args m) {
  typedef AttnTile<T, DP, KT> Tile;
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
  Mx4Loader<T, DP, KT, NW * 64, true> load_k;
  Mx4Loader<T, DP, KT, NW * 64, false> load_v;
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
      tile.add_infinite(v, j0, pl.row_lo, pl.row_hi);
      __syncthreads();
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

template <typename T> struct Frag16;
template <> struct Frag16<uint16_t> {
  __device__ static __forceinline__ f32x4_t mma(u32x4_t a, u32x4_t b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                   __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
  }
};
template <> struct Frag16<float> {
  __device__ static __forceinline__ f32x4_t mma(u32x4_t a, u32x4_t b, f32x4_t c) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[e]), __uint_as_float(b[e]), c, 0, 0, 0);
    return c;
  }
};

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
  static constexpr int kC = Mx<T>::kChunks;                  // chunks of a word's values
  static constexpr int kEpc = 16 / (int)sizeof(T);
  static constexpr int kDt = DP / 16;                        // 16-wide blocks of the output
  static constexpr int kPitch = DP * (int)sizeof(T);         // of a row of V in LDS
  static constexpr int kVBytes = 32 * kPitch;
  static constexpr int kOutBytes = RT * 16 * DP * 4;
  static constexpr int kLdsBytes = kVBytes > kOutBytes ? kVBytes : kOutBytes;

  // Chunk c of row r lies at c ^ swz(r).  Rows are written by 16 lanes, a row each, at one
  // chunk: eight neighbouring rows get different chunks.  bfloat16 is read as 32 bytes of
  // four neighbouring rows, float32 as 64 bytes of every fourth row.
  __device__ static __forceinline__ int swz(int r) {
    if constexpr (sizeof(T) == 2) return ((r & 3) << 1) | ((r >> 2) & 1);
    else return (((r >> 2) & 3) << 2) | (r & 3);
  }

  u32x4_t q[RT][kW * kC];
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
  __device__ __forceinline__ void load_q(int t, const T* row, int D, bool negate) {
    const int e0 = (lane_id() >> 4) * kLane;
#pragma unroll
    for (int i = 0; i < kW * kC; ++i) {
      const int e = e0 + i * kEpc;
      q[t][i] = u32x4_t{0u, 0u, 0u, 0u};
      if (e < D) q[t][i] = ldg16(row + e);
    }
    if (negate)
#pragma unroll
      for (int i = 0; i < kW * kC; ++i) q[t][i] = Frag<T>::negate(q[t][i]);
  }

  // Codes and scales of one row of K or V, this lane's part.
  struct Codes {
    uint32_t w[kW], s[kB];
  };
  static __device__ __forceinline__ float scale_of(const Codes& c, int i) {
    return mx_scale(c.s[i / 4 < kB ? i / 4 : 0]);
  }

  // Scores of 16 keys: s[t] has the keys 4 (lane / 16) + i of row lane % 16.
  __device__ __forceinline__ void scores(const Codes& k, f32x4_t (&s)[RT]) const {
#pragma unroll
    for (int t = 0; t < RT; ++t) s[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < kW; ++i) {
      u32x4_t x[kC];
      Mx<T>::decode8(k.w[i], scale_of(k, i), x);
#pragma unroll
      for (int j = 0; j < kC; ++j)
#pragma unroll
        for (int t = 0; t < RT; ++t) s[t] = Frag16<T>::mma(x[j], q[t][i * kC + j], s[t]);
    }
  }

  // V rows b * 16 + lane % 16 to LDS.
  __device__ static __forceinline__ void write_v(uint8_t* lds, int b, const Codes& v) {
    const int lane = lane_id(), r = b * 16 + (lane & 15), c0 = (lane >> 4) * (kW * kC);
#pragma unroll
    for (int i = 0; i < kW; ++i) {
      u32x4_t x[kC];
      Mx<T>::decode8(v.w[i], scale_of(v, i), x);
#pragma unroll
      for (int j = 0; j < kC; ++j)
        *(u32x4_t*)(lds + r * kPitch + (((c0 + i * kC + j) ^ swz(r)) << 4)) = x[j];
    }
  }

  // o += V^T P^T over the 32 keys in LDS.  A lane's weights are those of the keys 4 (lane / 16)
  // + i and 16 more: the order in which the B operand takes them when V^T is read alike.
  __device__ __forceinline__ void accumulate(const uint8_t* lds, const f32x4_t (&s)[2][RT]) {
    const int lane = lane_id(), i = lane & 15, g = lane >> 4;
    if constexpr (sizeof(T) == 2) {
      u32x4_t pf[RT];
#pragma unroll
      for (int t = 0; t < RT; ++t)
        pf[t] = u32x4_t{pack_bf16(s[0][t][0], s[0][t][1]), pack_bf16(s[0][t][2], s[0][t][3]),
                        pack_bf16(s[1][t][0], s[1][t][1]), pack_bf16(s[1][t][2], s[1][t][3])};
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
        for (int t = 0; t < RT; ++t) o[t][d] = Frag16<T>::mma(f, pf[t], o[t][d]);
      }
    } else {
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int r = 16 * b + 4 * g + k;
          const int at = r * kPitch + (((i >> 2) ^ swz(r)) << 4) + (i & 3) * 4;
#pragma unroll
          for (int d = 0; d < kDt; ++d) {
            const float v = *(const float*)(lds + (at ^ (d << 6)));
#pragma unroll
            for (int t = 0; t < RT; ++t)
              o[t][d] = __builtin_amdgcn_mfma_f32_16x16x4f32(v, s[b][t][k], o[t][d], 0, 0, 0);
          }
        }
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

  // A NaN block of V in a tile with hidden keys: rows that see its key get NaN in its
  // elements, and it becomes 0 for the others (0 times NaN is NaN).  j: this lane's
  // key, jb: the block's first.
  __device__ __forceinline__ void take_nan(Codes& v, int jb, const int (&lo)[RT], const int (&hi)[RT]) {
#pragma unroll
    for (int n = 0; n < kB; ++n) {
      uint64_t bad = __ballot(v.s[n] >= kMxBad);
      if (bad == 0) continue;
      while (bad != 0) {
        const int at = (int)__builtin_ctzll(bad);
        bad &= bad - 1;
        const int j = jb + (at & 15), e0 = (at >> 4) * kLane + n * kMxBlock;
        const int e1 = e0 + (kLane < kMxBlock ? kLane : kMxBlock);
#pragma unroll
        for (int t = 0; t < RT; ++t)
          if (j >= lo[t] && j < hi[t]) {
#pragma unroll
            for (int d = 0; d < kDt; ++d)
              if (d * 16 >= e0 && d * 16 < e1)
                o[t][d] = f32x4_t{1.f, 1.f, 1.f, 1.f} * __builtin_nanf("");
          }
      }
      if (v.s[n] >= kMxBad) {
        v.s[n] = 0;
#pragma unroll
        for (int i = 0; i < kW; ++i)
          if ((i / 4 < kB ? i / 4 : 0) == n) v.w[i] = 0;
      }
    }
  }
};

// The rows of K and V of a wave's blocks of 32 keys: lane l has key l % 16 of both halves.
// Pages are looked up one block before codes are loaded.
template <typename T, int DP, int RT, bool WHOLE>
struct KeysLoader {
  typedef KeysTile<T, DP, RT> Tile;
  const int32_t* bt;
  Mx4Rows k, v;                  // of the key head, at this lane's elements
  FastDiv per_page;
  int last_page, first, last, D, at;
  int page[2], off[2];

  __device__ __forceinline__ void init(const AttnMx4Args& m, int seq, int hk, int lo, int hi) {
    at = (lane_id() >> 4) * Tile::kLane;
    bt = m.a.p.block_table + (size_t)seq * m.a.p.max_pages;
    k = m.k, v = m.v;
    k.codes += hk * k.head + at / 2, k.scales += hk * k.s_head;
    v.codes += hk * v.head + at / 2, v.scales += hk * v.s_head;
    per_page = m.a.page;
    last_page = m.a.p.n_pages - 1;
    first = lo, last = hi - 1;
    D = m.a.p.D;
  }
  __device__ __forceinline__ void look_up(int j0) {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int j = min(max(j0 + 16 * b + (lane_id() & 15), first), last);
      const int pg = per_page.div(j);
      off[b] = j - pg * per_page.d;
      page[b] = bt[pg];
    }
  }
  __device__ __forceinline__ void one(const Mx4Rows& c, int64_t pg, int b, typename Tile::Codes& x) const {
    load_codes<Tile::kW, WHOLE>(c.codes + pg * c.page + off[b] * c.token, at, D, x.w);
    load_scales<Tile::kB, WHOLE>(c.scales + pg * c.s_page + off[b] * c.s_token, at / kMxBlock,
                                 mx_blocks(D), x.s);
  }
  __device__ __forceinline__ void start(typename Tile::Codes (&kc)[2], typename Tile::Codes (&vc)[2]) const {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int64_t pg = min(max(page[b], 0), last_page);
      one(k, pg, b, kc[b]);
      one(v, pg, b, vc[b]);
    }
  }
};

template <typename T, int DP, int RT, int NW, bool WHOLE, bool COMPACT>
__global__ __launch_bounds__(NW * 64, DP <= 128 ? 2 : 1) void attn_keys_mx4(AttnMx4Args args) {
  typedef KeysTile<T, DP, RT> Tile;
  constexpr int TM = 16 * RT;
  __shared__ __align__(1024) uint8_t lds[NW][Tile::kLdsBytes];
  __shared__ float ml[NW][TM][2];
  const AttnArgs& a = args.a;
  const PagedAttn& p = a.p;
  const int wave = uniform((int)threadIdx.x / kWave), lane = lane_id(), quad = lane >> 4;
  uint8_t* const mine = lds[wave];
  // items as in attn_keys
  KeysItems items;
  if constexpr (COMPACT) items.init(a);
  for (int item = blockIdx.x;; item += gridDim.x) {
    KeysWork kw;
    const int hk = item % p.hkv;
    if constexpr (COMPACT) {
      if (!items.get(a, item / p.hkv, &kw)) break;
    } else {
      kw.split = blockIdx.y;
      const int t = item / p.hkv, s = t / a.tiles_per_seq;
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
    KeysLoader<T, DP, RT, WHOLE> load;
    load.init(args, w.seq, hk, b, e);
    int j0 = (b & ~31) + wave * 32;
    const int end = b < e ? e : j0, step = NW * 32;
    typename Tile::Codes ka[2], va[2], kb[2], vb[2];
    if (j0 < end) {
      load.look_up(j0);
      load.start(ka, va);
      load.look_up(j0 + step);
      if (j0 + step < end) load.start(kb, vb);
      load.look_up(j0 + 2 * step);
    }
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const int r = r0 + min(16 * t + (lane & 15), rows - 1);
      const int token = a.group.div(r), head = hk * a.g + r - token * a.g;
      key_range(p, w, token, &row_lo[t], &row_hi[t]);
      if (j0 < end)
        tile.load_q(t, (const T*)p.q + (int64_t)(w.q0 + token) * p.q_token + head * p.q_head, p.D, a.negate);
    }
    // One block of 32 keys, whose codes have been on their way for two of the wave's
    // blocks; those of the block after the next take their place.
    auto block = [&](typename Tile::Codes (&kc)[2], typename Tile::Codes (&vc)[2]) __attribute__((always_inline)) {
      const bool whole = j0 >= x && j0 + 32 <= y;
      f32x4_t s[2][RT];
#pragma unroll
      for (int h = 0; h < 2; ++h) tile.scores(kc[h], s[h]);
      if (!whole) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          tile.take_nan(vc[h], j0 + 16 * h, row_lo, row_hi);
#pragma unroll
          for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int j = j0 + 16 * h + 4 * quad + i;
              s[h][t][i] = j >= row_lo[t] && j < row_hi[t] ? s[h][t][i] : -INFINITY;
            }
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) Tile::write_v(mine, h, vc[h]);
      if (j0 + 2 * step < end) {
        load.start(kc, vc);
        load.look_up(j0 + 3 * step);
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
      j0 += step;
    };
    while (j0 < end) {
      block(ka, va);
      if (j0 >= end) break;
      block(kb, vb);
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

constexpr int kMx4KeysWaves = 4;

// Launches of one element type, in files of their own.
template <typename T> hipError_t launch_attn_rows_mx4(const AttnMx4Args& m, hipStream_t s);
template <typename T> hipError_t launch_attn_keys_mx4(const AttnMx4Args& m, int row_tiles, bool compact, hipStream_t s);

template <typename T, int DP>
hipError_t attn_rows_mx4_width(const AttnMx4Args& m, hipStream_t s) {
  constexpr int kKeys = RowsShape<T, DP>::kKeys, kWaves = RowsShape<T, DP>::kWaves;
  const AttnArgs& a = m.a;
  const dim3 grid((unsigned)(a.n_tiles * a.p.hkv), (unsigned)a.splits), block(kWaves * 64);
  hipLaunchKernelGGL((attn_rows_mx4<T, DP, kKeys, kWaves>), grid, block, 0, s, m);
  return hipGetLastError();
}

template <typename T, int DP, int RT, bool WHOLE>
hipError_t attn_keys_mx4_go(const AttnMx4Args& m, bool compact, hipStream_t s) {
  const AttnArgs& a = m.a;
  const int64_t items = (int64_t)a.n_tiles * a.p.hkv * a.splits, most = 2 * kCus;
  const dim3 all((unsigned)(a.n_tiles * a.p.hkv), (unsigned)a.splits);
  const dim3 some((unsigned)(items < most ? items : most)), block(kMx4KeysWaves * 64);
  if (compact) hipLaunchKernelGGL((attn_keys_mx4<T, DP, RT, kMx4KeysWaves, WHOLE, true>), some, block, 0, s, m);
  else hipLaunchKernelGGL((attn_keys_mx4<T, DP, RT, kMx4KeysWaves, WHOLE, false>), all, block, 0, s, m);
  return hipGetLastError();
}

template <typename T, int DP>
hipError_t attn_keys_mx4_width(const AttnMx4Args& m, int row_tiles, bool compact, hipStream_t s) {
  if (m.a.p.D == DP)
    return row_tiles == 1 ? attn_keys_mx4_go<T, DP, 1, true>(m, compact, s)
                          : attn_keys_mx4_go<T, DP, 2, true>(m, compact, s);
  return row_tiles == 1 ? attn_keys_mx4_go<T, DP, 1, false>(m, compact, s)
                        : attn_keys_mx4_go<T, DP, 2, false>(m, compact, s);
}

}  // namespace sffn
