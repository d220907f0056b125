// Internal launchers of the attention side of the block (host side).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace sffn {

// Strides are in elements.  With slots: k_out and v_out are a paged cache
// (page, token, head strides kc_page, ko_token, ko_head and vc_*), else k_out
// is [T, hkv, D] with strides ko_token, ko_head and there is no v.
struct HeadsFwd {
  const void *q, *k, *v, *q_weight, *k_weight;
  const float* table;
  const int32_t *positions, *slots;
  void *q_out, *k_out, *v_out;
  int64_t q_token, q_head, k_token, k_head, v_token, v_head, qo_token, qo_head;
  int64_t ko_token, ko_head, kc_page, vc_page, vc_token, vc_head;
  int T, hq, hkv, D, rot, rot_adjacent, max_pos, norm, n_pages, page_size;
  float eps;
  int lanes_per_row, rows_per_wave;  // set by the launcher
};
hipError_t launch_heads_fwd(int dtype, HeadsFwd p, hipStream_t stream);

// partial: heads_bwd_partial_bytes(), not read or written without `weights`.
struct HeadsBwd {
  const void *q, *k, *q_weight, *k_weight, *gq_out, *gk_out;
  const float* table;
  const int32_t* positions;
  void *gq, *gk;
  float* partial;
  int64_t q_token, q_head, k_token, k_head, gqo_token, gqo_head, gko_token, gko_head;
  int64_t gq_token, gq_head, gk_token, gk_head;
  int T, hq, hkv, D, rot, rot_adjacent, max_pos, norm;
  float eps;
  int lanes_per_row;  // set by the launcher
};
size_t heads_bwd_partial_bytes(int T, int D);
hipError_t launch_heads_bwd(int dtype, HeadsBwd p, bool weights, float* gq_weight,
                            float* gk_weight, hipStream_t stream);

struct PagedAttn {
  const void *q, *k_cache, *v_cache;
  const int32_t *q_start, *kv_len, *block_table;
  void* out;
  float* lse;
  int64_t q_token, q_head, o_token, o_head;
  int64_t kc_page, kc_token, kc_head, vc_page, vc_token, vc_head;
  int T, n_seqs, hq, hkv, D, page_size, n_pages, max_pages, max_q, max_kv, causal, window;
  float scale;
};
// Whether p fits the grids of its launches, and the workspace that it needs.
bool plan_paged_attn(int dtype, const PagedAttn& p, size_t* bytes);
hipError_t launch_paged_attn(int dtype, const PagedAttn& p, void* ws, hipStream_t stream);

// ---------------------------------------------------------------- the 4-bit cache
// One cache (K or V): codes and scale bytes, strides in bytes.
struct Mx4Rows {
  uint8_t *codes, *scales;
  int64_t page, token, head, s_page, s_token, s_head;
};

// p: as for the append, its k_out, v_out and their strides unused.
hipError_t launch_heads_mx4(int dtype, HeadsFwd p, Mx4Rows k, Mx4Rows v, hipStream_t stream);

// out null: not read.
struct Mx4Read {
  Mx4Rows cache[2];   // K, V
  const int32_t* slots;
  void* out[2];
  int64_t o_token[2], o_head[2];
  int T, hkv, D, n_pages, page_size;
};
hipError_t launch_mx4_read(int dtype, const Mx4Read& p, hipStream_t stream);

// p: as for paged_attn, its caches and their strides unused.
bool plan_paged_attn_mx4(int dtype, const PagedAttn& p, size_t* bytes);
hipError_t launch_paged_attn_mx4(int dtype, const PagedAttn& p, const Mx4Rows& k, const Mx4Rows& v,
                                 void* ws, hipStream_t stream);

}  // namespace sffn
