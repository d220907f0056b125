// Attention of new tokens over a paged cache: which kernels a batch takes, how
// far its key ranges are split, the workspace of the splits.
#include <hip/hip_runtime.h>

#include "attn_kernels.cuh"

namespace sffn {

template <> hipError_t launch_attn_rows<uint16_t>(const AttnArgs&, int, hipStream_t);
template <> hipError_t launch_attn_rows<float>(const AttnArgs&, int, hipStream_t);
template <> hipError_t launch_attn_keys<uint16_t>(const AttnArgs&, int, bool, hipStream_t);
template <> hipError_t launch_attn_keys<float>(const AttnArgs&, int, bool, hipStream_t);

namespace {

constexpr int kRowsTile = 128;  // rows of an attn_rows workgroup
constexpr int kKeysTile = 32;   // rows of an attn_keys workgroup
constexpr int kMaxSplits = 64;  // lanes of the join
// Partial results of one launch: max_kv is often the model's limit and not the batch's
// longest sequence, and 1024 single tokens (8 key heads of 4 rows, width 128) would have
// 1.1 GB of them in 64 splits.  They get 15 splits here, with which a sequence
// of 131072 keys among short ones still has 120 workgroups.
constexpr int64_t kMaxPartBytes = 256ll << 20;

size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

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
int keys_max(const PagedAttn& p) {
  return p.max_q * (int64_t)(p.hq / p.hkv) <= 2 * kKeysTile ? 2 * kKeysTile : kKeysTile;
}

// Keys that the rows of one tile of at most `tokens` tokens can see.
int64_t key_span(const PagedAttn& p, int64_t tokens) {
  if (p.window == 0) return p.max_kv;
  const int64_t w = (int64_t)p.window + (p.causal ? tokens - 1 : p.max_q - 1);
  return w < p.max_kv ? w : p.max_kv;
}

// Splits of a key range of at most `span` keys for `groups` workgroups: enough to
// put `want` workgroups on the GPU, chunks of least .. most keys, and at most kMaxPartBytes
// of partial results.
void split(Plan* pl, const PagedAttn& p, int64_t span, int64_t groups, int64_t want, int least, int most) {
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

Plan plan_keys(int dtype, const PagedAttn& p) {
  Plan pl = {};
  const int64_t g = p.hq / p.hkv, rows = p.max_q * g;
  const int limit = keys_max(p);
  // where every sequence has max_q tokens and so more rows than fit, attn_rows takes
  // them all
  const bool equal = p.T == (int64_t)p.n_seqs * p.max_q;
  pl.used = g <= limit && (rows <= limit || !equal);
  if (!pl.used) return pl;
  pl.max_rows = limit;
  pl.tiles_per_seq = (int)(((rows < limit ? rows : limit) + kKeysTile - 1) / kKeysTile);
  pl.tiles = p.n_seqs * pl.tiles_per_seq;
  pl.slot_rows = (int)(rows < limit ? rows : limit);
  pl.part_rows = (size_t)p.n_seqs * p.hkv * pl.slot_rows;
  // A wave takes 1 to 2 us for 32 keys (3 us in float32, whose products are 16 times
  // slower), the join and its launch 6 us: ranges of up to 5 (2) steps a wave
  // are not split.  Longer ones into chunks of 2 (1) to 6 (1) steps: 6 even out
  // ragged lengths better than 8 (32 tokens over up to 4096 keys 67.8 -> 63.8 us),
  // fewer spread a few long ranges over the GPU.
  const int step = attn_keys_waves(dtype == 1 ? 2 : 4, p.D) * 32;
  const int whole = step * (dtype == 1 ? 5 : 2);
  const int64_t span = key_span(p, limit / g + 1);
  if (span <= whole) split(&pl, p, span, 1, 1, whole, whole);
  else
    split(&pl, p, span, (int64_t)pl.tiles * p.hkv, 4 * kCus, step * (dtype == 1 ? 2 : 1),
          step * (dtype == 1 ? 6 : 1));
  return pl;
}

Plan plan_rows(int dtype, const PagedAttn& p, bool with_keys) {
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
  split(&pl, p, key_span(p, kRowsTile / g + 2), (int64_t)pl.tiles * p.hkv, 2 * kCus,
        dtype == 1 ? 256 : 128, 1 << 30);
  return pl;
}

void place(AttnArgs* a, const Plan& pl, void* ws) {
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
dim3 join_grid(int tiles, int y, int most) {
  const int fit = most / tiles < 1 ? 1 : most / tiles;
  return dim3((unsigned)tiles, (unsigned)(y < fit ? y : fit));
}

template <typename T>
hipError_t launch(AttnArgs a, const Plan& keys, const Plan& rows, void* ws, hipStream_t s) {
  const PagedAttn& p = a.p;
  // see TileLoader: rows looked up together, lane offsets of less than 32 rows in
  // 32 bits.  Pages of 16: a 4096-token prompt 108 us, by 8 rows 112, row by row 121;
  // chunks beside single tokens 722, 737, 790.  Pages of 24: prompt 109 by 8 rows and 117
  // row by row (float32 chunks 84 and 81).
  const bool near = p.kc_token < (1 << 24) && p.vc_token < (1 << 24);
  const int granule = !near ? 0 : p.page_size % 16 == 0 ? 16 : p.page_size % 8 == 0 ? 8 : 0;
  hipError_t e = hipSuccess;
  if (rows.used) {
    place(&a, rows, (char*)ws + keys.bytes);
    e = launch_attn_rows<T>(a, granule, s);
    if (e != hipSuccess) return e;
    if (rows.splits > 1) {
      hipLaunchKernelGGL((attn_join<T, kRowsTile>), join_grid(rows.tiles * p.hkv, kRowsTile / 4, 1024),
                         dim3(256), 0, s, a);
      e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
  }
  if (keys.used) {
    place(&a, keys, ws);
    // Beside attn_rows most of the tiles that the host counts are not there, so the items
    // are numbered on the device: chunks beside single tokens 713 us, with a workgroup for
    // each 721; 16 float32 sequences 88 and 98; but 5 float32 chunks 84 and 80.
    e = launch_attn_keys<T>(a, granule, rows.used, s);
    if (e != hipSuccess) return e;
    if (keys.splits > 1) {
      const int most = (int64_t)p.max_q * a.g < kKeysTile ? p.max_q * a.g : kKeysTile;
      hipLaunchKernelGGL((attn_join<T, kKeysTile>), join_grid(keys.tiles * p.hkv, most, 4096), dim3(256),
                         0, s, a);
      e = hipGetLastError();
    }
  }
  return e;
}

}  // namespace

// A grid has less than 2^32 threads in x: workgroups of attn_rows and of both joins
// have 256, those of attn_keys 64 a wave.  Where attn_keys numbers its items itself,
// the numbers (and one step of the grid past them) are 32-bit.
bool plan_paged_attn(int dtype, const PagedAttn& p, size_t* bytes) {
  *bytes = 0;
  if (p.T == 0 || p.n_seqs == 0 || p.max_q == 0) return true;  // nothing is launched
  const Plan keys = plan_keys(dtype, p), rows = plan_rows(dtype, p, keys.used);
  const int64_t most = ((int64_t)1 << 32) - 1, wgs = (int64_t)keys.tiles * p.hkv;
  if (rows.used && (int64_t)rows.tiles * p.hkv * 256 > most) return false;
  if (keys.used) {
    if (keys.splits > 1 && wgs * 256 > most) return false;
    if (rows.used ? wgs * keys.splits > (1ll << 31) - 1 - 2 * kCus
                  : wgs * attn_keys_waves(dtype == 1 ? 2 : 4, p.D) * kWave > most)
      return false;
  }
  *bytes = keys.bytes + rows.bytes;
  return true;
}

hipError_t launch_paged_attn(int dtype, const PagedAttn& p, void* ws, hipStream_t stream) {
  const Plan keys = plan_keys(dtype, p), rows = plan_rows(dtype, p, keys.used);
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
  return dtype == 1 ? launch<uint16_t>(a, keys, rows, ws, stream)
                    : launch<float>(a, keys, rows, ws, stream);
}

}  // namespace sffn
