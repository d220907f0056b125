// Checks of arguments that the entry points of the attention side share.
#pragma once

#include <hip/hip_runtime.h>

#include <initializer_list>

#include "attn.h"
#include "sffn.h"

namespace sffn {

inline bool aligned(const void* p, unsigned n) { return ((uintptr_t)p & (n - 1)) == 0; }
inline bool given(const void* p, unsigned n) { return p != nullptr && aligned(p, n); }

// Rows [T, heads, D] at p, read or written in 16-byte chunks: pointer and the
// strides that matter (a dimension of size 1 has none).  An output's rows must
// not overlap (strides at least D), an input may repeat rows (stride 0).
inline int32_t check_rows(const void* p, int64_t n0, int64_t s0, int64_t n1, int64_t s1, int D, int dtype,
                   bool output) {
  const int64_t unit = dtype == SFFN_BF16 ? 8 : 4;
  if (!given(p, 16)) return SFFN_ERR_ARG;
  const int64_t s[2] = {n0 > 1 ? s0 : (output ? D : 0), n1 > 1 ? s1 : (output ? D : 0)};
  for (int64_t v : s) {
    if (v < 0 || (output && v < D)) return SFFN_ERR_ARG;
    if (v % unit != 0) return SFFN_ERR_UNSUPPORTED;
  }
  return SFFN_OK;
}

inline int32_t check_heads(const sffn_heads* h) {
  if (h == nullptr) return SFFN_ERR_ARG;
  if (h->T < 0 || h->n_q_heads < 0 || h->n_kv_heads < 0 || h->head_dim <= 0 || h->rot_dim < 0 ||
      h->rot_dim > h->head_dim || h->max_pos < 0 || !(h->eps >= 0.f) || h->eps > 1e30f)
    return SFFN_ERR_ARG;
  if ((h->norm != 0 && h->norm != 1) || (h->rot_adjacent != 0 && h->rot_adjacent != 1))
    return SFFN_ERR_ARG;
  if (h->dtype != SFFN_F32 && h->dtype != SFFN_BF16) return SFFN_ERR_ARG;
  if (h->rot_dim > 0 && h->max_pos == 0) return SFFN_ERR_ARG;
  if (h->head_dim % 8 != 0 || h->head_dim > 256 || h->rot_dim % 4 != 0) return SFFN_ERR_UNSUPPORTED;
  // token numbers, and one step of the backward's grid past them, are 32-bit
  if (h->n_q_heads > 4096 || h->n_kv_heads > 4096 || h->T > (1 << 30)) return SFFN_ERR_UNSUPPORTED;
  return SFFN_OK;
}

// The forward and the append have 64 threads a token in one grid, which has less than
// 2^32 of them.
inline int32_t check_heads_fwd(const sffn_heads* h) {
  const int32_t st = check_heads(h);
  return st == SFFN_OK && h->T > (1 << 26) - 4 ? SFFN_ERR_UNSUPPORTED : st;
}

inline int32_t check_rotation(const sffn_heads* h, const void* q_weight, const void* k_weight,
                       const float* table, const int32_t* positions) {
  if (!aligned(q_weight, 16) || !aligned(k_weight, 16)) return SFFN_ERR_ARG;
  if (h->rot_dim > 0 && (!given(table, 4) || !given(positions, 4))) return SFFN_ERR_ARG;
  return SFFN_OK;
}

inline int32_t first_error(std::initializer_list<int32_t> all) {
  for (int32_t s : all)
    if (s != SFFN_OK) return s;
  return SFFN_OK;
}

inline int32_t hip_status(hipError_t e) { return e == hipSuccess ? SFFN_OK : SFFN_ERR_HIP; }

inline HeadsFwd fwd_params(const sffn_heads* h, const void* q_weight, const void* k_weight,
                    const float* table, const int32_t* positions) {
  HeadsFwd p = {};
  p.q_weight = q_weight, p.k_weight = k_weight, p.table = table, p.positions = positions;
  p.T = h->T, p.hq = h->n_q_heads, p.hkv = h->n_kv_heads, p.D = h->head_dim, p.rot = h->rot_dim;
  p.rot_adjacent = h->rot_adjacent, p.max_pos = h->max_pos, p.norm = h->norm, p.eps = h->eps;
  return p;
}

inline PagedAttn attn_params(const sffn_paged_batch* b) {
  PagedAttn p = {};
  p.T = b->T, p.n_seqs = b->n_seqs, p.hq = b->n_q_heads, p.hkv = b->n_kv_heads, p.D = b->head_dim;
  p.page_size = b->page_size, p.n_pages = b->n_pages, p.max_pages = b->max_pages;
  p.max_q = b->max_q < b->T ? b->max_q : b->T;
  p.max_kv = b->max_kv, p.causal = b->causal, p.scale = b->scale;
  // a window as long as every sequence hides nothing; a shorter one keeps position
  // minus window within 32 bits, also at the negative positions of rows before the keys
  p.window = b->window < b->max_kv ? b->window : 0;
  return p;
}

// plan: plan_paged_attn or that of the 4-bit cache; bytes: of the workspace, where the batch
// is taken.
template <typename F>
inline int32_t check_batch(const sffn_paged_batch* b, size_t* bytes, F plan) {
  if (b == nullptr) return SFFN_ERR_ARG;
  if (b->T < 0 || b->n_seqs < 0 || b->n_q_heads <= 0 || b->n_kv_heads <= 0 || b->head_dim <= 0 ||
      b->page_size <= 0 || b->n_pages < 0 || b->max_pages < 0 || b->max_q < 0 || b->max_kv < 0 ||
      b->window < 0 || (b->causal != 0 && b->causal != 1))
    return SFFN_ERR_ARG;
  if (b->n_q_heads % b->n_kv_heads != 0) return SFFN_ERR_ARG;
  if ((int64_t)b->max_kv > (int64_t)b->max_pages * b->page_size) return SFFN_ERR_ARG;
  if (b->max_kv > 0 && b->n_pages == 0) return SFFN_ERR_ARG;
  if (!(b->scale >= -1e30f && b->scale <= 1e30f)) return SFFN_ERR_ARG;
  if (b->dtype != SFFN_F32 && b->dtype != SFFN_BF16) return SFFN_ERR_ARG;
  if (b->head_dim % 8 != 0 || b->head_dim > 256) return SFFN_ERR_UNSUPPORTED;
  // row and key numbers, and a tile past their ends, are 32-bit
  if ((int64_t)b->T * b->n_q_heads > (1 << 30) || b->max_kv > (1 << 30) || b->n_seqs > (1 << 20) ||
      b->n_q_heads > 4096)
    return SFFN_ERR_UNSUPPORTED;
  return plan(b->dtype, attn_params(b), bytes) ? SFFN_OK : SFFN_ERR_UNSUPPORTED;
}

}  // namespace sffn
