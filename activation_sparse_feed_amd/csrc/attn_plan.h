// Which kernels a batch of attention over a paged cache takes, how far its key ranges are
// split and the workspace of the splits: the same for both forms of the cache but for a
// few measured numbers.
#pragma once

#include "attn_kernels.cuh"

namespace sffn {

constexpr int kRowsTile = 128;  // rows of an attn_rows workgroup
constexpr int kKeysTile = 32;   // rows of an attn_keys workgroup
constexpr int kMaxSplits = 64;  // lanes of the join
// Partial results of one launch: max_kv is often the model's limit and not the batch's
// longest sequence, and 1024 single tokens (8 key heads of 4 rows, width 128) would have
// 1.1 GB of them in 64 splits.  They get 15 splits here, with which a sequence
// of 131072 keys among short ones still has 120 workgroups.
constexpr int64_t kMaxPartBytes = 256ll << 20;

inline size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

// What one launch takes: row tiles, splits, workspace.
struct Plan {
  bool used;
  int tiles, tiles_per_seq, min_rows, max_rows, slot_rows, chunk, splits;
  size_t part_rows, bytes;
};

// Rows of a sequence up to which attn_keys takes it: two tiles where that covers the
// whole batch, so that attn_rows does not run (drafts of up to 5 tokens in a window,
// 8 heads a key head: 13 us, with one tile and attn_rows beside it 31; 16 sequences of
// up to 16 tokens, 4 heads: 38 and 49); otherwise one, since two tiles read the keys
// twice and attn_rows runs in any case (64 sequences of up to 17 tokens: 61 us, with
// two tiles 92; 16 of up to 40: 65 and 72; 8 of up to 30, 48 heads: 37 and 52; but 8 of
// up to 20 over up to 20000 keys: 142 and 132).
inline int keys_max(const PagedAttn& p) {
  return p.max_q * (int64_t)(p.hq / p.hkv) <= 2 * kKeysTile ? 2 * kKeysTile : kKeysTile;
}

// Keys that the rows of one tile of at most `tokens` tokens can see.
inline int64_t key_span(const PagedAttn& p, int64_t tokens) {
  if (p.window == 0) return p.max_kv;
  const int64_t w = (int64_t)p.window + (p.causal ? tokens - 1 : p.max_q - 1);
  return w < p.max_kv ? w : p.max_kv;
}

// Splits of a key range of at most `span` keys for `groups` workgroups: enough to
// put `want` workgroups on the GPU, chunks of least .. most keys, and at most kMaxPartBytes
// of partial results.
inline void split(Plan* pl, const PagedAttn& p, int64_t span, int64_t groups, int64_t want, int least, int most) {
  int64_t n = groups > 0 ? (want + groups - 1) / groups : 1;
  // a range that does not start at a multiple of the chunk touches one more
  const int64_t slot = (int64_t)(pl->part_rows * (p.D * 4 + 8)), fit = slot > 0 ? kMaxPartBytes / slot : kMaxSplits;
  int64_t most_splits = fit < kMaxSplits ? fit : kMaxSplits;
  if (p.window > 0) --most_splits;
  if (most_splits < 1) most_splits = 1;
  int64_t chunk = (span + n - 1) / n;
  if (chunk > most) chunk = most;
  if (chunk < least) chunk = least;
  if (chunk < (span + most_splits - 1) / most_splits) chunk = (span + most_splits - 1) / most_splits;
  chunk = (chunk + 63) / 64 * 64;
  pl->chunk = (int)chunk;
  pl->splits = (int)((span + chunk - 1) / chunk);
  if (pl->splits > 1 && p.window > 0) ++pl->splits;
  if (pl->splits < 1) pl->splits = 1;
  // one chunk must hold the whole range wherever it starts
  if (pl->splits == 1) pl->chunk = 1 << 30;
  pl->bytes = pl->splits > 1 ? align256((size_t)pl->splits * pl->part_rows * p.D * 4) +
                                   align256((size_t)pl->splits * pl->part_rows * 8)
                             : 0;
}

// Key ranges of up to `whole` keys are not split, longer ones into chunks of least .. most.
struct KeysTuning {
  int whole, least, most, want;  // want: workgroups
  int tile;                      // rows of one
};

inline Plan plan_keys(const PagedAttn& p, const KeysTuning& n) {
  Plan pl = {};
  const int64_t g = p.hq / p.hkv, rows = p.max_q * g;
  const int limit = keys_max(p);
  // where every sequence has max_q tokens and so more rows than fit, attn_rows takes
  // them all
  const bool equal = p.T == (int64_t)p.n_seqs * p.max_q;
  pl.used = g <= limit && (rows <= limit || !equal);
  if (!pl.used) return pl;
  pl.max_rows = limit;
  pl.tiles_per_seq = (int)(((rows < limit ? rows : limit) + n.tile - 1) / n.tile);
  pl.tiles = p.n_seqs * pl.tiles_per_seq;
  pl.slot_rows = (int)(rows < limit ? rows : limit);
  pl.part_rows = (size_t)p.n_seqs * p.hkv * pl.slot_rows;
  const int64_t span = key_span(p, limit / g + 1);
  if (span <= n.whole) split(&pl, p, span, 1, 1, n.whole, n.whole);
  else split(&pl, p, span, (int64_t)pl.tiles * p.hkv, n.want, n.least, n.most);
  return pl;
}

// least: keys of a split.
inline Plan plan_rows(const PagedAttn& p, bool with_keys, int least) {
  Plan pl = {};
  const int64_t g = p.hq / p.hkv;
  pl.min_rows = with_keys ? keys_max(p) : 0;
  pl.used = p.max_q * g > pl.min_rows;
  if (!pl.used) return pl;
  const int64_t rows = p.T * g;
  // every taken sequence has at most one tile that is not full
  int64_t part = rows / (pl.min_rows + 1);
  if (part > p.n_seqs) part = p.n_seqs;
  pl.tiles = (int)((rows + part * (kRowsTile - 1)) / kRowsTile);
  pl.part_rows = (size_t)pl.tiles * p.hkv * kRowsTile;
  // Two workgroups a CU (one: 110 us for ragged float32 chunks, two: 87, three or
  // four: 102; bf16 chunks beside single tokens 745 with two, 748 to 802 with more).
  split(&pl, p, key_span(p, kRowsTile / g + 2), (int64_t)pl.tiles * p.hkv, 2 * kCus, least, 1 << 30);
  return pl;
}

// Whether the launches of a plan fit their grids.  A grid has less than 2^32 threads in x:
// workgroups of the kernel of many rows and of both joins have 256, those of the kernel
// of few rows keys_threads.  Where the latter numbers its items itself, the numbers (and one
// step of the grid past them) are 32-bit.
inline bool plan_fits(const Plan& keys, const Plan& rows, const PagedAttn& p, int keys_threads) {
  const int64_t most = ((int64_t)1 << 32) - 1, wgs = (int64_t)keys.tiles * p.hkv;
  if (rows.used && (int64_t)rows.tiles * p.hkv * 256 > most) return false;
  if (keys.used) {
    if (keys.splits > 1 && wgs * 256 > most) return false;
    if (rows.used ? wgs * keys.splits > (1ll << 31) - 1 - 2 * kCus : wgs * keys_threads > most) return false;
  }
  return true;
}

inline void place(AttnArgs* a, const Plan& pl, void* ws) {
  a->chunk = FastDiv::make(pl.chunk);
  a->min_rows = pl.min_rows;
  a->max_rows = pl.max_rows;
  a->tiles_per_seq = pl.tiles_per_seq;
  a->slot_rows = pl.slot_rows;
  a->splits = pl.splits;
  a->n_tiles = pl.tiles;
  a->part_rows = pl.part_rows;
  a->part_o = (float*)ws;
  a->part_ml = (float*)((char*)ws + align256((size_t)pl.splits * pl.part_rows * a->p.D * 4));
}

// Workgroups of a join: for every tile up to y (one for each step over its rows), but
// not many more than `most`, since each first finds out which rows are its own.
inline dim3 join_grid(int tiles, int y, int most) {
  const int fit = most / tiles < 1 ? 1 : most / tiles;
  return dim3((unsigned)tiles, (unsigned)(y < fit ? y : fit));
}

inline AttnArgs attn_args(const PagedAttn& p) {
  AttnArgs a = {};
  a.p = p;
  a.g = p.hq / p.hkv;
  a.page = FastDiv::make(p.page_size);
  a.group = FastDiv::make(a.g);
  // scores are scaled in the exponent; a scale of 0 becomes the smallest number, which
  // leaves every weight 1 but keeps hidden keys at -inf
  const float c = (p.scale < 0.f ? -p.scale : p.scale) * 1.44269504088896340736f;
  a.c = c > 0.f ? c : 0x1p-149f;
  a.negate = p.scale < 0.f;
  return a;
}

// attn_join for the rows of kRowsTile or kKeysTile; early: see there.
hipError_t launch_attn_join(int dtype, int tile_rows, bool early, const AttnArgs& a, dim3 grid, hipStream_t s);

// Whether the join of attn_keys' rows loads early, which spares it a wait for the lengths but takes 80
// registers instead of 44.  Early / late, in us, bf16, width 128, 32 heads on 8:
//   splits of a row  64 (three tokens over up to 131072 keys) 4.9 / 7.6, 43 4.6 / 5.2, 22 (8 tokens) 4.8 / 4.9;
//                    from 8 to 16 as fast, but 32 tokens 5.2 / 5.0; 6 5.1 / 4.7, 4 4.9 / 4.7
//   workgroups       1024 (32 tokens, 22 splits) 5.9 / 6.2, 2048 (64) 8.8 / 7.5, 8192 (256, 6) 16.3 / 13.3
//   bytes of parts   where max_kv is far above the lengths, hardly any of those that are read were
//                    written: 32 tokens over up to 4096 keys, max_kv 131072, 34 MB 8.8 / 4.8, 8 tokens
//                    8.5 MB 4.3 / 4.2
inline bool join_early(const Plan& pl, dim3 grid) {
  return pl.splits > 16 && (int64_t)grid.x * grid.y <= 1024 && pl.bytes <= (size_t)8 << 20;
}

// The join of the splits of one of the two kernels, where there are any.  Rows of attn_keys
// are joined by 32, whatever its tiles.
inline hipError_t launch_join(int dtype, int tile_rows, AttnArgs a, const Plan& pl, hipStream_t s) {
  if (pl.splits <= 1) return hipSuccess;
  const PagedAttn& p = a.p;
  if (tile_rows != kKeysTile)
    return launch_attn_join(dtype, tile_rows, false, a, join_grid(pl.tiles * p.hkv, tile_rows / 4, 1024), s);
  a.tiles_per_seq = (pl.slot_rows + kKeysTile - 1) / kKeysTile;
  const int rows = pl.slot_rows < kKeysTile ? pl.slot_rows : kKeysTile;
  const dim3 grid = join_grid(p.n_seqs * a.tiles_per_seq * p.hkv, rows, 4096);
  return launch_attn_join(dtype, tile_rows, join_early(pl, grid), a, grid, s);
}

}  // namespace sffn
