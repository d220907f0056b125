// C ABI of the attention side of the block (declared in include/sffn.h):
// argument validation on the host, workspace carving and kernel launches.
// Nothing here allocates, frees or synchronises.
#include <hip/hip_runtime.h>

#include "attn_check.h"

namespace {

using namespace sffn;

// Cache [n_pages, page_size, heads, D] with strides sp, st, sh.
int32_t check_cache(const void* c, int64_t n_pages, int64_t sp, int64_t page_size, int64_t st,
                    int64_t heads, int64_t sh, int D, int dtype) {
  return first_error({check_rows(c, n_pages, sp, page_size, st, D, dtype, true),
                      check_rows(c, n_pages, sp, heads, sh, D, dtype, true)});
}

}  // namespace

extern "C" {

int32_t qk_norm_rope(const sffn_heads* heads, const void* q, int64_t q_token, int64_t q_head,
                     const void* k, int64_t k_token, int64_t k_head, const void* q_weight,
                     const void* k_weight, const float* rot_table, const int32_t* positions,
                     void* q_out, int64_t qo_token, int64_t qo_head, void* k_out,
                     int64_t ko_token, int64_t ko_head, void* stream) {
  int32_t st = check_heads_fwd(heads);
  if (st != SFFN_OK) return st;
  const sffn_heads& h = *heads;
  if (h.T == 0 || h.n_q_heads + h.n_kv_heads == 0) return SFFN_OK;
  st = check_rotation(heads, q_weight, k_weight, rot_table, positions);
  if (st == SFFN_OK && h.n_q_heads > 0)
    st = first_error({check_rows(q, h.T, q_token, h.n_q_heads, q_head, h.head_dim, h.dtype, false),
                      check_rows(q_out, h.T, qo_token, h.n_q_heads, qo_head, h.head_dim, h.dtype, true)});
  if (st == SFFN_OK && h.n_kv_heads > 0)
    st = first_error({check_rows(k, h.T, k_token, h.n_kv_heads, k_head, h.head_dim, h.dtype, false),
                      check_rows(k_out, h.T, ko_token, h.n_kv_heads, ko_head, h.head_dim, h.dtype, true)});
  if (st != SFFN_OK) return st;
  HeadsFwd p = fwd_params(heads, q_weight, k_weight, rot_table, positions);
  p.q = q, p.q_token = q_token, p.q_head = q_head;
  p.k = k, p.k_token = k_token, p.k_head = k_head;
  p.q_out = q_out, p.qo_token = qo_token, p.qo_head = qo_head;
  p.k_out = k_out, p.ko_token = ko_token, p.ko_head = ko_head;
  return hip_status(launch_heads_fwd(h.dtype, p, (hipStream_t)stream));
}

size_t qk_norm_rope_bwd_workspace_bytes(const sffn_heads* heads) {
  if (check_heads(heads) != SFFN_OK || heads->norm == 0) return 0;
  return heads_bwd_partial_bytes(heads->T, heads->head_dim);
}

int32_t qk_norm_rope_bwd(const sffn_heads* heads, const void* q, int64_t q_token, int64_t q_head,
                         const void* k, int64_t k_token, int64_t k_head, const void* q_weight,
                         const void* k_weight, const float* rot_table, const int32_t* positions,
                         const void* gq_out, int64_t gqo_token, int64_t gqo_head,
                         const void* gk_out, int64_t gko_token, int64_t gko_head, void* gq,
                         int64_t gq_token, int64_t gq_head, void* gk, int64_t gk_token,
                         int64_t gk_head, float* gq_weight, float* gk_weight, void* workspace,
                         size_t ws_bytes, void* stream) {
  int32_t st = check_heads(heads);
  if (st != SFFN_OK) return st;
  const sffn_heads& h = *heads;
  if (!aligned(gq_weight, 4) || !aligned(gk_weight, 4)) return SFFN_ERR_ARG;
  const bool any = h.T > 0 && h.n_q_heads + h.n_kv_heads > 0;
  if (any) {
    st = check_rotation(heads, q_weight, k_weight, rot_table, positions);
    if (st == SFFN_OK && h.n_q_heads > 0)
      st = first_error(
          {h.norm ? check_rows(q, h.T, q_token, h.n_q_heads, q_head, h.head_dim, h.dtype, false) : SFFN_OK,
           check_rows(gq_out, h.T, gqo_token, h.n_q_heads, gqo_head, h.head_dim, h.dtype, false),
           check_rows(gq, h.T, gq_token, h.n_q_heads, gq_head, h.head_dim, h.dtype, true)});
    if (st == SFFN_OK && h.n_kv_heads > 0)
      st = first_error(
          {h.norm ? check_rows(k, h.T, k_token, h.n_kv_heads, k_head, h.head_dim, h.dtype, false) : SFFN_OK,
           check_rows(gk_out, h.T, gko_token, h.n_kv_heads, gko_head, h.head_dim, h.dtype, false),
           check_rows(gk, h.T, gk_token, h.n_kv_heads, gk_head, h.head_dim, h.dtype, true)});
    if (st != SFFN_OK) return st;
  }
  const bool weights = h.norm && (gq_weight != nullptr || gk_weight != nullptr);
  if (any && weights &&
      (!given(workspace, 16) || ws_bytes < qk_norm_rope_bwd_workspace_bytes(heads)))
    return SFFN_ERR_WORKSPACE;
  if (!any && !weights) return SFFN_OK;
  HeadsBwd p = {};
  p.q = q, p.q_token = q_token, p.q_head = q_head;
  p.k = k, p.k_token = k_token, p.k_head = k_head;
  p.q_weight = q_weight, p.k_weight = k_weight, p.table = rot_table, p.positions = positions;
  p.gq_out = gq_out, p.gqo_token = gqo_token, p.gqo_head = gqo_head;
  p.gk_out = gk_out, p.gko_token = gko_token, p.gko_head = gko_head;
  p.gq = gq, p.gq_token = gq_token, p.gq_head = gq_head;
  p.gk = gk, p.gk_token = gk_token, p.gk_head = gk_head;
  p.T = any ? h.T : 0, p.hq = h.n_q_heads, p.hkv = h.n_kv_heads, p.D = h.head_dim;
  p.rot = h.rot_dim, p.rot_adjacent = h.rot_adjacent, p.max_pos = h.max_pos;
  p.norm = h.norm, p.eps = h.eps;
  p.partial = (float*)workspace;
  return hip_status(launch_heads_bwd(h.dtype, p, weights, gq_weight, gk_weight,
                                     (hipStream_t)stream));
}

int32_t paged_kv_append(const sffn_heads* heads, const void* q, int64_t q_token, int64_t q_head,
                        const void* k, int64_t k_token, int64_t k_head, const void* v,
                        int64_t v_token, int64_t v_head, const void* q_weight,
                        const void* k_weight, const float* rot_table, const int32_t* positions,
                        const int32_t* slots, void* q_out, int64_t qo_token, int64_t qo_head,
                        void* k_cache, int64_t kc_page, int64_t kc_token, int64_t kc_head,
                        void* v_cache, int64_t vc_page, int64_t vc_token, int64_t vc_head,
                        int32_t n_pages, int32_t page_size, void* stream) {
  int32_t st = check_heads_fwd(heads);
  if (st != SFFN_OK) return st;
  const sffn_heads& h = *heads;
  if (h.n_kv_heads == 0 || n_pages < 0 || page_size <= 0) return SFFN_ERR_ARG;
  // a slot has 32 bits: tokens past it would be taken for padding, or wrap onto others
  if ((int64_t)n_pages * page_size > (1ll << 31)) return SFFN_ERR_UNSUPPORTED;
  if (h.T == 0) return SFFN_OK;
  st = check_rotation(heads, q_weight, k_weight, rot_table, positions);
  if (st == SFFN_OK && h.n_q_heads > 0)
    st = first_error({check_rows(q, h.T, q_token, h.n_q_heads, q_head, h.head_dim, h.dtype, false),
                      check_rows(q_out, h.T, qo_token, h.n_q_heads, qo_head, h.head_dim, h.dtype, true)});
  if (st == SFFN_OK)
    st = first_error(
        {check_rows(k, h.T, k_token, h.n_kv_heads, k_head, h.head_dim, h.dtype, false),
         check_rows(v, h.T, v_token, h.n_kv_heads, v_head, h.head_dim, h.dtype, false),
         given(slots, 4) ? SFFN_OK : SFFN_ERR_ARG,
         check_cache(k_cache, n_pages, kc_page, page_size, kc_token, h.n_kv_heads, kc_head,
                     h.head_dim, h.dtype),
         check_cache(v_cache, n_pages, vc_page, page_size, vc_token, h.n_kv_heads, vc_head,
                     h.head_dim, h.dtype)});
  if (st != SFFN_OK) return st;
  HeadsFwd p = fwd_params(heads, q_weight, k_weight, rot_table, positions);
  p.q = q, p.q_token = q_token, p.q_head = q_head;
  p.k = k, p.k_token = k_token, p.k_head = k_head;
  p.v = v, p.v_token = v_token, p.v_head = v_head;
  p.q_out = q_out, p.qo_token = qo_token, p.qo_head = qo_head;
  p.slots = slots, p.n_pages = n_pages, p.page_size = page_size;
  p.k_out = k_cache, p.kc_page = kc_page, p.ko_token = kc_token, p.ko_head = kc_head;
  p.v_out = v_cache, p.vc_page = vc_page, p.vc_token = vc_token, p.vc_head = vc_head;
  return hip_status(launch_heads_fwd(h.dtype, p, (hipStream_t)stream));
}

size_t paged_attn_workspace_bytes(const sffn_paged_batch* batch) {
  size_t bytes = 0;
  return check_batch(batch, &bytes, plan_paged_attn) == SFFN_OK ? bytes : 0;
}

int32_t paged_attn_fwd(const sffn_paged_batch* batch, const void* q, int64_t q_token,
                       int64_t q_head, const void* k_cache, int64_t kc_page, int64_t kc_token,
                       int64_t kc_head, const void* v_cache, int64_t vc_page, int64_t vc_token,
                       int64_t vc_head, const int32_t* q_start, const int32_t* kv_len,
                       const int32_t* block_table, void* out, int64_t o_token, int64_t o_head,
                       float* lse, void* workspace, size_t ws_bytes, void* stream) {
  size_t need = 0;
  int32_t st = check_batch(batch, &need, plan_paged_attn);
  if (st != SFFN_OK) return st;
  const sffn_paged_batch& b = *batch;
  if (b.T == 0 || b.n_seqs == 0 || b.max_q == 0) return SFFN_OK;
  st = first_error({check_rows(q, b.T, q_token, b.n_q_heads, q_head, b.head_dim, b.dtype, false),
                    check_rows(out, b.T, o_token, b.n_q_heads, o_head, b.head_dim, b.dtype, true),
                    given(q_start, 4) && given(kv_len, 4) && aligned(lse, 4) ? SFFN_OK : SFFN_ERR_ARG});
  if (st == SFFN_OK && b.max_kv > 0)
    st = first_error({check_cache(k_cache, b.n_pages, kc_page, b.page_size, kc_token, b.n_kv_heads,
                                  kc_head, b.head_dim, b.dtype),
                      check_cache(v_cache, b.n_pages, vc_page, b.page_size, vc_token, b.n_kv_heads,
                                  vc_head, b.head_dim, b.dtype),
                      given(block_table, 4) ? SFFN_OK : SFFN_ERR_ARG});
  if (st != SFFN_OK) return st;
  PagedAttn p = attn_params(batch);
  p.q = q, p.q_token = q_token, p.q_head = q_head;
  p.out = out, p.o_token = o_token, p.o_head = o_head;
  p.k_cache = k_cache, p.kc_page = kc_page, p.kc_token = kc_token, p.kc_head = kc_head;
  p.v_cache = v_cache, p.vc_page = vc_page, p.vc_token = vc_token, p.vc_head = vc_head;
  p.q_start = q_start, p.kv_len = kv_len, p.block_table = block_table, p.lse = lse;
  if (need > 0 && (!given(workspace, 16) || ws_bytes < need)) return SFFN_ERR_WORKSPACE;
  return hip_status(launch_paged_attn(b.dtype, p, workspace, (hipStream_t)stream));
}

}  // extern "C"
