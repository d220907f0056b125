// Kernels of attention over a paged cache.
//
// The rows of a sequence under one key head are its new tokens times the query
// heads that share the key head: row r is token r / g, head r % g, so that the
// heads of a group share every key and value that is loaded.
//
//   attn_rows  many rows (chunks of prompts): four waves of 32 rows each, K and V
//              tiles shared in LDS, double buffered.  Bound by the matrix cores at the
//              clock that the card's power allows: 2.15 to 2.28 ms for a 16384-token
//              prompt (32 heads on 8, width 128, bf16: 2.20 TFLOP, so 1.0 PFLOP/s;
//              a large library product runs at 1.14), matrix cores busy half of the
//              cycles at 1.75 to 2.0 GHz.  In copies of this kernel for timing (2.31
//              ms that day) leaving out the exponentials gave 2.24, the whole
//              softmax 2.07, the fragment reads 2.0, the tile loads 1.97,
//              everything but the products 1.40.  Eight waves (256 rows a tile,
//              half the tile loads) gave 2.10 to 2.13 beside 2.15, orderings of the
//              step by hand 2.21 to 2.34 beside 2.16, wave priorities 2.15 to 2.20
//              beside 2.15.
//   attn_keys  few rows (single tokens, drafts): the waves of a workgroup hold the
//              same 32 rows and take the key tiles in turn, each with its own
//              LDS and no barriers; their results are joined at the end.  Bound by
//              HBM for many or long sequences (three of 31191 to 131000 keys, 983 MB:
//              179 us, 5.5 TB/s), by its chain of dependent loads and steps for
//              few (one of 257 keys: 8.6 us).
//   attn_join  joins the splits of a long key range: for each row the maximum of the
//              splits' maxima, then their sums and outputs scaled to it.  5.0 us
//              for 64 splits of three tokens, 4.8 for 32 tokens: latency.
//
// attn_rows of width 256 takes a wave's 512 registers: 505 in bf16 (560 TFLOP/s at a 4096-token
// prompt, 32 heads on 8), and 68 to 80 bytes a lane of scratch memory in float32.
#pragma once

#include "attn_tile.cuh"

namespace sffn {

constexpr int kCus = 256;

template <int N>
__device__ __forceinline__ void wait_loads() {  // vmcnt <= N
  __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}

// A sequence and the part of its rows that a workgroup takes.
struct Work {
  int seq, q0, nq, nkv, tile;  // tile < 0: none
};

// Its rows and keys from q_start[s], q_start[s + 1] and kv_len[s], within the bounds
// that the host knows: whatever these hold, no row, key or split beyond them is used.
__device__ __forceinline__ void bound_sequence(const PagedAttn& p, int q0, int q1, int len, Work* w) {
  w->q0 = min(max(q0, 0), p.T);
  w->nq = min(min(max(q1, w->q0), p.T) - w->q0, p.max_q);
  w->nkv = min(max(len, 0), p.max_kv);
}

__device__ __forceinline__ void read_sequence(const PagedAttn& p, int s, Work* w) {
  w->seq = uniform(s);
  bound_sequence(p, load_uniform(p.q_start + w->seq), load_uniform(p.q_start + w->seq + 1),
                 load_uniform(p.kv_len + w->seq), w);
}

// Row tile number `t` of the sequences with more than min_rows rows.  Among 64
// neighbouring sequences the longest come first, and of a sequence the last rows,
// which see most keys: tiles start in order of their work, so that the last ones
// to end are short.  `t` runs over the tiles of 64 sequences in that order.
template <int TM>
__device__ __forceinline__ Work find_tile(const AttnArgs& a, int t) {
  const PagedAttn& p = a.p;
  Work w;
  w.tile = -1;
  w.seq = w.q0 = w.nq = w.nkv = 0;
  for (int s0 = 0; s0 < p.n_seqs; s0 += kWave) {
    const int s = s0 + lane_id();
    int n = 0, len = -1;
    if (s < p.n_seqs) {
      Work x;
      bound_sequence(p, p.q_start[s], p.q_start[s + 1], p.kv_len[s], &x);
      const int rows = x.nq * a.g;
      n = rows > a.min_rows ? (rows + TM - 1) / TM : 0;
      len = x.nkv;
    }
    // tiles of the sequences before this one, and of all
    int before = 0, all = 0;
    for (int k = 0; k < min(p.n_seqs - s0, kWave); ++k) {
      const int nk = __builtin_amdgcn_readlane(n, k), lk = __builtin_amdgcn_readlane(len, k);
      all += nk;
      before += lk > len || (lk == len && k < lane_id()) ? nk : 0;
    }
    const uint64_t hit = __ballot(t >= before && t < before + n);
    if (hit != 0) {
      const int k = (int)__builtin_ctzll(hit);
      read_sequence(p, s0 + k, &w);
      w.tile = __builtin_amdgcn_readlane(n, k) - 1 - (t - __builtin_amdgcn_readlane(before, k));
      break;
    }
    t -= all;
  }
  return w;
}

// The keys [lo, hi) that token i (0 .. nq - 1) sees; lo == hi: none.
__device__ __forceinline__ void key_range(const PagedAttn& p, const Work& w, int i, int* lo, int* hi) {
  const int pos = w.nkv - w.nq + i;
  *hi = p.causal ? max(pos + 1, 0) : w.nkv;
  *lo = p.window > 0 ? max(pos - p.window + 1, 0) : 0;
  *lo = min(*lo, *hi);
}

// Keys of one split: chunk number `split` of those that the range [lo, hi) of all
// rows touches.  Returns the number of splits of the range (at least 1).
__device__ __forceinline__ int split_range(const AttnArgs& a, int split, int lo, int hi, int* b, int* e) {
  if (hi <= lo) {
    *b = *e = lo;
    return 1;
  }
  const int c0 = a.chunk.div(lo), n = a.chunk.div(hi - 1) - c0 + 1;
  *b = max(lo, (c0 + split) * a.chunk.d);
  *e = (int)min((int64_t)hi, (int64_t)(c0 + split + 1) * a.chunk.d);
  return n;
}

// Inclusive prefix sum over the wave: shifts by 1, 2, 4, 8 within rows of 16 lanes,
// then the last lane of a row to the next row(s).
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_add(int v) {
  return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xf, false);
}
__device__ __forceinline__ int prefix_sum(int v) {
  v = dpp_add<0x111, 0xf>(v);
  v = dpp_add<0x112, 0xf>(v);
  v = dpp_add<0x114, 0xf>(v);
  v = dpp_add<0x118, 0xf>(v);
  v = dpp_add<0x142, 0xa>(v);  // row_bcast:15 into rows 1 and 3
  return dpp_add<0x143, 0xc>(v);  // row_bcast:31 into rows 2 and 3
}

// Row tiles of 32 of the sequences that attn_keys takes (1 .. max_rows rows), and the
// splits of their key ranges: one range for all tiles of a sequence.
struct KeysWork {
  Work w;
  int split, n_split, lo, hi;  // of the sequence; split: number within n_split
};

__device__ __forceinline__ void sequence_range(const AttnArgs& a, KeysWork* k) {
  int x, y;
  key_range(a.p, k->w, 0, &k->lo, &y);
  key_range(a.p, k->w, max(k->w.nq - 1, 0), &x, &k->hi);
  k->n_split = split_range(a, 0, k->lo, k->hi, &x, &y);
}

// The items (sequence, tile, split) of attn_keys, numbered through; 64 sequences are
// held by the lanes of a wave at a time, and the numbers asked for only grow.  TM: rows
// of a tile.
template <int TM>
struct KeysItems {
  int s0, base, total;          // first sequence of the 64, items before and in them
  int before, n;                // lane's items before its sequence, and of it
  KeysWork k;                   // lane's sequence

  __device__ __forceinline__ void group(const AttnArgs& a, int first) {
    const PagedAttn& p = a.p;
    s0 = first;
    const int s = s0 + lane_id();
    n = 0;
    k.w.seq = s;
    k.w.q0 = k.w.nq = k.w.nkv = 0;
    if (s < p.n_seqs) bound_sequence(p, p.q_start[s], p.q_start[s + 1], p.kv_len[s], &k.w);
    const int rows = k.w.nq * a.g;
    sequence_range(a, &k);
    if (rows > 0 && rows <= a.max_rows) n = (rows + TM - 1) / TM * k.n_split;
    before = prefix_sum(n);
    total = __builtin_amdgcn_readlane(before, kWave - 1);
    before -= n;
  }
  __device__ __forceinline__ void init(const AttnArgs& a) {
    base = 0;
    group(a, 0);
  }
  // Item v, or false past the last one.
  __device__ __forceinline__ bool get(const AttnArgs& a, int v, KeysWork* out) {
    while (v - base >= total) {
      base += total;
      if (s0 + kWave >= a.p.n_seqs) {
        total = 0;
        s0 = a.p.n_seqs;
        return false;
      }
      group(a, s0 + kWave);
    }
    const int u = v - base;
    const int lane = (int)__builtin_ctzll(__ballot(u >= before && u < before + n));
    out->w.seq = s0 + lane;
    out->w.q0 = __builtin_amdgcn_readlane(k.w.q0, lane);
    out->w.nq = __builtin_amdgcn_readlane(k.w.nq, lane);
    out->w.nkv = __builtin_amdgcn_readlane(k.w.nkv, lane);
    out->lo = __builtin_amdgcn_readlane(k.lo, lane);
    out->hi = __builtin_amdgcn_readlane(k.hi, lane);
    out->n_split = __builtin_amdgcn_readlane(k.n_split, lane);
    out->split = u - __builtin_amdgcn_readlane(before, lane);
    out->w.tile = 0;
    while (out->split >= out->n_split) {  // few tiles
      out->split -= out->n_split;
      ++out->w.tile;
    }
    return true;
  }
};

// Writes one row's outputs (lane: d = 8 * quad + 4 * half + 0..3 of each 32): the
// result, or its part of a split.
template <typename T>
__device__ __forceinline__ void store4(T* p, float a, float b, float c, float d) {
  if constexpr (sizeof(T) == 2) {
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    u32x2 v;
    v.x = pack_bf16(a, b);
    v.y = pack_bf16(c, d);
    *(u32x2*)p = v;
  } else {
    f32x4_t v = {a, b, c, d};
    *(f32x4_t*)p = v;
  }
}

__device__ __forceinline__ float finish_lse(float m, float l) {
  return l == 0.f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * 0.69314718055994530942f;
}

// The place of a workgroup of attn_rows: its tile of TM rows of a sequence, its keys, and
// this lane's row.
struct RowsPlace {
  Work w;
  int wave, r0, r1;            // first and last row of the tile
  int b, e, n_split;           // keys of this split, splits of the tile
  int x, y;                    // keys that all rows of the tile see
  int r, token, head;          // this lane's row
  int row_lo, row_hi;          // the keys that it sees
  int w_lo0, w_hi0, w_lo1, w_hi1;  // those of the wave's first and last row
  bool wave_live;

  // False: nothing to do.
  template <int TM>
  __device__ __forceinline__ bool init(const AttnArgs& a, int t, int hk, int split) {
    const PagedAttn& p = a.p;
    w = find_tile<TM>(a, t);
    if (w.tile < 0) return false;
    wave = uniform((int)threadIdx.x / kWave);
    const int lane = lane_id(), rows = w.nq * a.g;
    r0 = w.tile * TM, r1 = min(r0 + TM, rows) - 1;
    int lo, hi;
    key_range(p, w, a.group.div(r0), &lo, &y);
    key_range(p, w, a.group.div(r1), &x, &hi);
    n_split = split_range(a, split, lo, hi, &b, &e);
    if (split >= n_split) return false;
    const int wr0 = min(r0 + wave * 32, rows - 1), wr1 = min(wr0 + 31, r1);
    r = min(r0 + wave * 32 + (lane & 31), r1);
    token = a.group.div(r), head = hk * a.g + r - token * a.g;
    key_range(p, w, token, &row_lo, &row_hi);
    key_range(p, w, a.group.div(wr0), &w_lo0, &w_hi0);
    key_range(p, w, a.group.div(wr1), &w_lo1, &w_hi1);
    wave_live = r0 + wave * 32 <= r1;
    return true;
  }
  __device__ __forceinline__ int64_t q_offset(const PagedAttn& p) const {
    return (int64_t)(w.q0 + token) * p.q_token + head * p.q_head;
  }
  // Of the 32 keys from j on, the wave's rows see none; all.
  __device__ __forceinline__ bool sees_none(int j) const { return !wave_live || j >= w_hi1 || j + 32 <= w_lo0; }
  __device__ __forceinline__ bool sees_all(int j) const { return j >= w_lo1 && j + 32 <= w_hi0; }
};

// The wave's rows of such a tile, result or part of a split.
template <typename T, int TM, typename Tile>
__device__ __forceinline__ void write_rows(const AttnArgs& a, const RowsPlace& pl, Tile& tile, int t, int hk,
                                           int split) {
  const PagedAttn& p = a.p;
  const int lane = lane_id(), half = lane >> 5;
  tile.l = sum_halves(tile.l);
  const float m = tile.m * a.c;
  if (pl.r0 + pl.wave * 32 + (lane & 31) > pl.r1) return;
  if (pl.n_split == 1) {
    const float inv = tile.l == 0.f ? 0.f : 1.f / tile.l;
    T* out = (T*)p.out + (int64_t)(pl.w.q0 + pl.token) * p.o_token + pl.head * p.o_head;
#pragma unroll
    for (int d = 0; d < Tile::kDt; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = d * 32 + 8 * i + 4 * half;
        if (at < p.D)
          store4<T>(out + at, tile.o[d][4 * i] * inv, tile.o[d][4 * i + 1] * inv,
                    tile.o[d][4 * i + 2] * inv, tile.o[d][4 * i + 3] * inv);
      }
    if (p.lse != nullptr && half == 0)
      p.lse[(int64_t)(pl.w.q0 + pl.token) * p.hq + pl.head] = finish_lse(m, tile.l);
  } else {
    const size_t slot = split * a.part_rows + ((size_t)t * p.hkv + hk) * TM + (pl.r - pl.r0);
    float* out = a.part_o + slot * p.D;
#pragma unroll
    for (int d = 0; d < Tile::kDt; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = d * 32 + 8 * i + 4 * half;
        if (at < p.D)
          store4<float>(out + at, tile.o[d][4 * i], tile.o[d][4 * i + 1], tile.o[d][4 * i + 2],
                        tile.o[d][4 * i + 3]);
      }
    if (half == 0) {
      a.part_ml[2 * slot] = m;
      a.part_ml[2 * slot + 1] = tile.l;
    }
  }
}

template <typename T, int DP, int KT, int NW, int G>
__global__ __launch_bounds__(NW * 64, DP <= 128 && sizeof(T) == 2 ? 2 : 1) void attn_rows(AttnArgs a) {
  typedef AttnTile<T, DP, KT> Tile;
  constexpr int TM = NW * 32;
  // separate arrays, and a loop unrolled over them: the compiler then knows that
  // reads of one do not wait for the loads into another
  __shared__ __align__(1024) uint8_t k0[Tile::kTileBytes], k1[Tile::kTileBytes], v0[Tile::kTileBytes],
      v1[Tile::kTileBytes];
  const PagedAttn& p = a.p;
  // key heads run fastest over the workgroups, which go round the XCDs: with
  // eight of them (or a multiple) an XCD's L2 holds the keys of one head.  Where all
  // workgroups run at once, two a CU, the second 256 come in reverse order, which puts
  // the splits with most work beside those with least (a 4096-token prompt, 8
  // heads on 1: 85 -> 73 us).
  const int all = (int)(gridDim.x * gridDim.y);
  int id = (int)(blockIdx.y * gridDim.x + blockIdx.x);
  if (DP <= 128 && all <= 2 * kCus && id >= kCus) id = all - 1 - (id - kCus);
  const int split = id / (int)gridDim.x, th = id - split * (int)gridDim.x;
  const int hk = th % p.hkv, t = th / p.hkv;
  RowsPlace pl;
  if (!pl.template init<TM>(a, t, hk, split)) return;
  const int wave = pl.wave, b = pl.b, e = pl.e, x = pl.x, y = pl.y, row_lo = pl.row_lo, row_hi = pl.row_hi;
  Tile tile;
  tile.init();
  // chunks that no load writes, but that are read: up to DP by the products, up to the
  // end of the LDS row by the search for infinite values
  if (p.D != Tile::kRowElems) {
    for (int i = threadIdx.x * 16; i < Tile::kTileBytes; i += NW * 64 * 16)
      *(u32x4_t*)(k0 + i) = *(u32x4_t*)(k1 + i) = *(u32x4_t*)(v0 + i) = *(u32x4_t*)(v1 + i) =
          u32x4_t{0u, 0u, 0u, 0u};
    __syncthreads();
  }
  constexpr int kPer = Tile::kLoads / NW;
  static_assert(kPer >= 1, "");
  TileLoader<T, DP, KT, G, kPer, true> load_k;
  TileLoader<T, DP, KT, G, kPer, false> load_v;
  load_k.init(a, pl.w.seq, hk, b, e, wave * kPer);
  load_v.init(a, pl.w.seq, hk, b, e, wave * kPer);
  const T* q = (const T*)p.q + pl.q_offset(p);
  // The K tile that is in LDS beside a V tile is 32 keys ahead of it: step()
  // needs the next block's K with a block's V.
  f32x16_t s;
  int j0 = b & ~(KT - 1);
  if (e > b) {
    load_k.look_up(j0 + 32 - KT);
    load_v.look_up(j0);
    load_k.start(k1);
    load_k.look_up(j0 + 32);
    load_v.start(v0);
    load_v.look_up(j0 + KT);
    load_k.start(k0);
    load_k.look_up(j0 + KT + 32);
    tile.load_q(q, p.D);
    wait_loads<0>();
    __syncthreads();
    if (a.negate) tile.negate();
    s = tile.scores(k1 + KT * Tile::kPitch - Tile::kBlockBytes);
  }
  auto iteration = [&](uint8_t* k, uint8_t* v, uint8_t* k_next, uint8_t* v_next) __attribute__((always_inline)) {
    wait_loads<0>();
    __syncthreads();  // k and v are in LDS, and nobody reads the others any more
    if (j0 + KT < e) {
      load_v.start(v_next);
      load_v.look_up(j0 + 2 * KT);
      load_k.start(k_next);
      load_k.look_up(j0 + 2 * KT + 32);
    }
    if (!(j0 >= x && j0 + KT <= y) &&  // some row of the workgroup does not see some key
        __builtin_expect(__syncthreads_or(Tile::template find_infinite<NW * 64>(v, threadIdx.x)), 0)) {
      if (__builtin_expect(
              __syncthreads_or(Tile::template find_infinite_in<NW * 64, 64>(v, threadIdx.x, b - j0, e - j0)), 0)) {
        tile.add_infinite(v, j0, row_lo, row_hi);
        __syncthreads();
      }
      Tile::template clear_infinite<NW * 64>(v, threadIdx.x);
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < KT / 32; ++i) {
      const int j = j0 + i * 32;
      // the wave's rows see none of the block's keys, or not all of them
      if (pl.sees_none(j)) {
        s = tile.scores(k + i * Tile::kBlockBytes);
      } else {
        if (!pl.sees_all(j)) Tile::hide(s, j, row_lo, row_hi);
        tile.step(s, k + i * Tile::kBlockBytes, v + i * Tile::kBlockBytes, a.c);
      }
    }
    j0 += KT;
  };
  while (j0 < e) {
    iteration(k0, v0, k1, v1);
    if (j0 >= e) break;
    iteration(k1, v1, k0, v0);
  }
  write_rows<T, TM>(a, pl, tile, t, hk, split);
}

template <typename T, int DP, int NW, int G, bool COMPACT>
__global__ __launch_bounds__(NW * 64, DP <= 128 ? 2 : 1) void attn_keys(AttnArgs a) {
  constexpr int KT = 32;
  typedef AttnTile<T, DP, KT> Tile;
  __shared__ __align__(1024) uint8_t k_lds[NW][Tile::kTileBytes], v_lds[NW][Tile::kTileBytes];
  __shared__ float ml[NW][32][2];
  const PagedAttn& p = a.p;
  const int wave = uniform((int)threadIdx.x / kWave), lane = lane_id(), half = lane >> 5;
  uint8_t *const k = k_lds[wave], *const v = v_lds[wave];
  auto clear = [&]() __attribute__((always_inline)) {  // as in attn_rows
    if (p.D == Tile::kRowElems) return;
    for (int i = lane * 16; i < Tile::kTileBytes; i += kWave * 16)
      *(u32x4_t*)(k + i) = *(u32x4_t*)(v + i) = u32x4_t{0u, 0u, 0u, 0u};
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): written
  };
  clear();
  // Items (sequence, tile, split) are numbered from bounds of the lengths: the item of
  // a workgroup is at hand, but may not exist.  A workgroup without work still waits
  // for its place in LDS, so where most are expected to be of that kind (COMPACT:
  // chunks of prompts beside single tokens) only the items that exist are numbered,
  // for 1.5 us to look over the sequences, and a limited grid goes over them.
  KeysItems<32> items;
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
      if (kw.w.tile * 32 >= all || all > a.max_rows) break;
      sequence_range(a, &kw);
      if (kw.split >= kw.n_split) break;
    }
    const Work w = kw.w;
    const int r0 = w.tile * 32, rows = min(32, w.nq * a.g - r0);
    // the tile's keys in this split
    int lo, hi, b, e, x, y;
    key_range(p, w, a.group.div(r0), &lo, &y);
    key_range(p, w, a.group.div(r0 + rows - 1), &x, &hi);
    split_range(a, kw.split, kw.lo, kw.hi, &b, &e);
    b = max(b, lo);
    e = min(e, hi);
    const int r = r0 + min(lane & 31, rows - 1);
    const int token = a.group.div(r), head = hk * a.g + r - token * a.g;
    int row_lo, row_hi;
    key_range(p, w, token, &row_lo, &row_hi);
    Tile tile;
    tile.init();
    TileLoader<T, DP, KT, G, Tile::kLoads, true> load_k;
    TileLoader<T, DP, KT, G, Tile::kLoads, false> load_v;
    // All but the newest tile's loads are done.  Every tile is kLoads of them (a
    // wave-wide load has lanes within head_dim); with page lookups among the loads
    // their order is the compiler's, so all are waited for.
    auto wait_one = [&]() __attribute__((always_inline)) {
      if constexpr (G > 0) wait_loads<Tile::kLoads>();
      else wait_loads<0>();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    };
    load_k.init(a, w.seq, hk, b, e, 0);
    load_v.init(a, w.seq, hk, b, e, 0);
    int j0 = (b & ~(KT - 1)) + wave * KT;
    const int end = b < e ? e : j0;  // nothing to do: no iteration
    if (j0 < end) {
      load_k.look_up(j0);
      load_v.look_up(j0);
      tile.load_q((const T*)p.q + (int64_t)(w.q0 + token) * p.q_token + head * p.q_head, p.D);
      load_k.start(k);
      load_v.start(v);
      load_k.look_up(j0 + NW * KT);
      load_v.look_up(j0 + NW * KT);
      wait_one();
      if (a.negate) tile.negate();
    }
    // One tile each of K and V: the next K is loaded as soon as the scores have read
    // this one, the next V after the product, so that one of them is always in flight.
    for (; j0 < end; j0 += NW * KT) {
      const bool more = j0 + NW * KT < end, whole = j0 >= x && j0 + KT <= y;
      wait_one();  // K is here
      f32x16_t s = tile.scores(k);
      __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): it has been read
      __builtin_amdgcn_sched_barrier(0);
      if (more) {
        load_k.start(k);
        load_k.look_up(j0 + 2 * NW * KT);
      }
      if (!whole) Tile::hide(s, j0, row_lo, row_hi);
      tile.raise(s, a.c);
      tile.weights(s, a.c);
      if (more) wait_one();  // V is here
      else wait_loads<0>();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
      if (__builtin_expect(!whole && __any(Tile::template find_infinite<kWave>(v, lane)), 0)) {
        if (__builtin_expect(__any(Tile::template find_infinite_in<kWave, 1>(v, lane, b - j0, e - j0)), 0))
          tile.add_infinite(v, j0, row_lo, row_hi);
        Tile::template clear_infinite<kWave>(v, lane);
      }
      tile.accumulate(v, s);
      __builtin_amdgcn_s_waitcnt(0xC07F);
      __builtin_amdgcn_sched_barrier(0);
      if (more) {
        load_v.start(v);
        load_v.look_up(j0 + 2 * NW * KT);
      }
    }
    tile.l = sum_halves(tile.l);
    // Join the waves: each leaves its rows in its LDS, 32 x 32 floats for each block of
    // 32 outputs, row r's 16-byte chunk c at c ^ (r % 8).
    constexpr int kPerArray = Tile::kTileBytes / 4096;
    static_assert(kPerArray * 2 >= Tile::kDt, "");
    auto part = [&](int wv, int d) { return (d < kPerArray ? v_lds[wv] + d * 4096 : k_lds[wv] + (d - kPerArray) * 4096); };
    {
      const int row = lane & 31;
#pragma unroll
      for (int d = 0; d < Tile::kDt; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          store4<float>((float*)(part(wave, d) + row * 128 + (((2 * i + half) ^ (row & 7)) << 4)),
                        tile.o[d][4 * i], tile.o[d][4 * i + 1], tile.o[d][4 * i + 2], tile.o[d][4 * i + 3]);
      if (half == 0) {
        ml[wave][row][0] = tile.m * a.c;
        ml[wave][row][1] = tile.l;
      }
    }
    __syncthreads();
    const int quads = p.D / 4;
    for (int i = threadIdx.x; i < rows * quads; i += NW * 64) {
      const int rr = i / quads, d = (i - rr * quads) * 4;
      float m = -INFINITY, l = 0.f;
#pragma unroll
      for (int k = 0; k < NW; ++k) m = fmaxf(m, ml[k][rr][0]);
      f32x4_t v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < NW; ++k) {
        const float mk = ml[k][rr][0];
        const float f = mk == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(mk - m);
        l += f * ml[k][rr][1];
        v += f * *(const f32x4_t*)(part(k, d / 32) + rr * 128 + (((d % 32 / 4) ^ (rr & 7)) << 4));
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
    wait_loads<0>();   // the outputs are written (they count among the loads)
    __syncthreads();  // the waves' results are read before the next item's tiles arrive
    clear();
  }
}

// Joins the splits of the rows of one tile (TM rows; 32: of attn_keys).  A wave's lanes
// hold the maxima and sums of up to 64 splits, then D / 4 lanes a split's outputs,
// several splits side by side.  attn_keys' rows are few and may have many splits:
// the four waves of a workgroup share a row; otherwise each has its own.
// EARLY (of attn_keys): the first row's parts are loaded before their number is known, those
// that were not written, too, and are dropped.
template <typename T, int TM, bool EARLY>
__global__ __launch_bounds__(256) void attn_join(AttnArgs a) {
  static_assert(TM == 32 || !EARLY, "");
  constexpr int kShare = TM == 32 ? 4 : 1;  // waves of a row
  constexpr int kAhead = 8;                 // loads of a lane in flight
  __shared__ f32x4_t sums[kShare][kWave];
  const PagedAttn& p = a.p;
  const int hk = (int)blockIdx.x % p.hkv, t = (int)blockIdx.x / p.hkv;
  const int lane = lane_id(), wave = (int)threadIdx.x / kWave;
  int width = 1;  // lanes of one split's outputs
  while (width * 4 < p.D) width *= 2;
  const int side = kWave / width, sub = lane / width, d = (lane & (width - 1)) * 4;
  const int s_first = kShare == 4 ? wave * side : 0, s_step = side * kShare;
  // rows from the tile's first: where their parts lie does not depend on the lengths
  const int seq = TM == 32 ? t / a.tiles_per_seq : 0, tile_row = TM == 32 ? (t - seq * a.tiles_per_seq) * 32 : 0;
  const size_t slots = TM == 32 ? ((size_t)seq * p.hkv + hk) * a.slot_rows + tile_row
                                : ((size_t)t * p.hkv + hk) * TM;
  const int i_first = kShare == 4 ? (int)blockIdx.y : (int)blockIdx.y * 4 + wave;
  const float* const outputs = a.part_o + (d < p.D ? d : 0);
  float m_ahead = -INFINITY, l_ahead = 0.f;
  f32x4_t o_ahead[EARLY ? kAhead : 1];
  const bool there = EARLY && tile_row + i_first < a.slot_rows;
  if constexpr (EARLY) {
    if (there) {
      const size_t slot = slots + i_first;
      const size_t at = (size_t)min(lane, a.splits - 1) * a.part_rows + slot;
      m_ahead = a.part_ml[2 * at];
      l_ahead = a.part_ml[2 * at + 1];
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (s_first + k * s_step < a.splits)
          o_ahead[k] = *(const f32x4_t*)(outputs + ((size_t)min(s_first + k * s_step + sub, a.splits - 1) *
                                                    a.part_rows + slot) * p.D);
    }
  }
  Work w;
  int n;
  if constexpr (TM == 32) {
    KeysWork k;
    read_sequence(p, seq, &k.w);
    const int all = k.w.nq * a.g;
    k.w.tile = t - seq * a.tiles_per_seq;
    if (k.w.tile * 32 >= all || all > a.max_rows) return;
    sequence_range(a, &k);
    n = k.n_split;
    w = k.w;
  } else {
    w = find_tile<TM>(a, t);
    if (w.tile < 0) return;
  }
  const int rows = w.nq * a.g, r0 = w.tile * TM, r1 = min(r0 + TM, rows) - 1;
  if constexpr (TM != 32) {
    int lo, hi, b, e, x, y;
    key_range(p, w, a.group.div(r0), &lo, &y);
    key_range(p, w, a.group.div(r1), &x, &hi);
    n = split_range(a, 0, lo, hi, &b, &e);
  }
  if (n == 1) return;  // written by the kernel before
  for (int i = i_first; r0 + i <= r1; i += (int)gridDim.y * (4 / kShare)) {
    const int r = r0 + i;
    const bool ahead = EARLY && there && i == i_first;
    const size_t slot = slots + i;
    float ms = -INFINITY, ls = 0.f;
    if (lane < n) {
      const size_t at = lane * a.part_rows + slot;
      ms = ahead ? m_ahead : a.part_ml[2 * at];
      ls = ahead ? l_ahead : a.part_ml[2 * at + 1];
    }
    float m = ms;
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, kWave));
    const float f = ms == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(ms - m);
    const float l = wave_sum(f * ls);
    f32x4_t v = {0.f, 0.f, 0.f, 0.f};
    // a split past the last one is dropped.  A factor of 0 drops nothing: NaN times it stays
    // NaN, as in a sum over all keys
    auto add = [&](int s0, const f32x4_t& x) __attribute__((always_inline)) {
      const int s = s0 + sub;
      const float fs = __shfl(f, min(s, n - 1), kWave);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += s < n ? fs * x[i] : 0.f;
    };
    int s0 = s_first;
    if constexpr (EARLY) {
      if (ahead) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
          if (s_first + k * s_step < n) add(s_first + k * s_step, o_ahead[k]);
        s0 += kAhead * s_step;
      }
    }
    // loads without conditions, so that they are in flight together
#pragma unroll 8
    for (; s0 < n; s0 += s_step)
      add(s0, *(const f32x4_t*)(outputs + ((size_t)min(s0 + sub, n - 1) * a.part_rows + slot) * p.D));
    for (int k = width; k < kWave; k <<= 1)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += __shfl_xor(v[i], k, kWave);
    if constexpr (kShare == 4) {
      sums[wave][lane] = v;
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kShare; ++k) v = k == 0 ? sums[0][lane] : v + sums[k][lane];
    }
    const int token = a.group.div(r), head = hk * a.g + r - token * a.g;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    if (kShare == 1 || wave == 0) {
      if (sub == 0 && d < p.D)
        store4<T>((T*)p.out + (int64_t)(w.q0 + token) * p.o_token + head * p.o_head + d, v[0] * inv,
                  v[1] * inv, v[2] * inv, v[3] * inv);
      if (lane == 0 && p.lse != nullptr)
        p.lse[(int64_t)(w.q0 + token) * p.hq + head] = finish_lse(m, l);
    }
    if constexpr (kShare == 4) __syncthreads();
  }
}

// Waves of an attn_keys workgroup: tiles of K and V (32 rows of 64, 128 or 256 elements)
// for all of them in 64 KB, so that two workgroups share a CU.
constexpr int attn_keys_waves(int elt_bytes, int head_dim) {
  return (64 << 10) / (2 * 32 * (head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256) * elt_bytes);
}

// Launches of one element type, in files of their own.
template <typename T> hipError_t launch_attn_rows(const AttnArgs& a, int granule, hipStream_t s);
template <typename T> hipError_t launch_attn_keys(const AttnArgs& a, int granule, bool compact, hipStream_t s);

// Key tile and waves of attn_rows.
template <typename T, int DP> struct RowsShape {
  static constexpr int kWaves = 4;
  static constexpr int kKeys = sizeof(T) == 2 ? 64 : 32;
};
#define SFFN_ATTN_BY_WIDTH(F, T, ...)                  \
  do {                                                 \
    const int d_ = a.p.D;                              \
    if (d_ <= 64) return F<T, 64>(__VA_ARGS__);        \
    if (d_ <= 96) return F<T, 96>(__VA_ARGS__);        \
    if (d_ <= 128) return F<T, 128>(__VA_ARGS__);      \
    if (d_ <= 192) return F<T, 192>(__VA_ARGS__);      \
    return F<T, 256>(__VA_ARGS__);                     \
  } while (0)

template <typename T, int DP>
hipError_t attn_rows_width(const AttnArgs& a, int granule, hipStream_t s) {
  constexpr int kKeys = RowsShape<T, DP>::kKeys, kWaves = RowsShape<T, DP>::kWaves;
  const dim3 grid((unsigned)(a.n_tiles * a.p.hkv), (unsigned)a.splits), block(kWaves * 64);
  if (granule == 16) hipLaunchKernelGGL((attn_rows<T, DP, kKeys, kWaves, 16>), grid, block, 0, s, a);
  else if (granule == 8) hipLaunchKernelGGL((attn_rows<T, DP, kKeys, kWaves, 8>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((attn_rows<T, DP, kKeys, kWaves, 0>), grid, block, 0, s, a);
  return hipGetLastError();
}

template <typename T, int DP>
hipError_t attn_keys_width(const AttnArgs& a, int granule, bool compact, hipStream_t s) {
  constexpr int kWaves = attn_keys_waves(sizeof(T), DP);
  const int64_t items = (int64_t)a.n_tiles * a.p.hkv * a.splits, most = 2 * kCus;
  const dim3 all((unsigned)(a.n_tiles * a.p.hkv), (unsigned)a.splits);
  const dim3 some((unsigned)(items < most ? items : most)), block(kWaves * 64);
#define SFFN_KEYS(G)                                                                            \
  if (compact) hipLaunchKernelGGL((attn_keys<T, DP, kWaves, G, true>), some, block, 0, s, a);   \
  else hipLaunchKernelGGL((attn_keys<T, DP, kWaves, G, false>), all, block, 0, s, a)
  if (granule == 16) { SFFN_KEYS(16); }
  else if (granule == 8) { SFFN_KEYS(8); }
  else { SFFN_KEYS(0); }
#undef SFFN_KEYS
  return hipGetLastError();
}

}  // namespace sffn
