// C ABI of the 4-bit paged cache (declared in include/sffn.h): argument validation on
// the host and kernel launches.  Nothing here allocates, frees or synchronises.
#include <hip/hip_runtime.h>

#include "attn_check.h"
#include "mx4.cuh"

namespace {

using namespace sffn;

// Codes are read and written in words of 4 bytes, scale bytes one by one.  A dimension of
// size 1 has no stride; the rows of an input, too, must not overlap, since the cache is both.
int32_t check_mx4(const sffn_mx4* c, int64_t n_pages, int64_t page_size, int64_t heads, int D) {
  if (c == nullptr || !given(c->codes, 4) || c->scales == nullptr) return SFFN_ERR_ARG;
  const int64_t codes = D / 2, scales = mx_blocks(D);
  const int64_t n[3] = {n_pages, page_size, heads};
  const int64_t s[3] = {c->page, c->token, c->head}, b[3] = {c->scale_page, c->scale_token, c->scale_head};
  for (int i = 0; i < 3; ++i) {
    if (n[i] <= 1) continue;
    if (s[i] < codes || b[i] < scales) return SFFN_ERR_ARG;
    if (s[i] % 4 != 0) return SFFN_ERR_UNSUPPORTED;
  }
  return SFFN_OK;
}

Mx4Rows mx4_rows(const sffn_mx4* c) {
  return Mx4Rows{(uint8_t*)c->codes, (uint8_t*)c->scales, c->page, c->token, c->head,
                 c->scale_page, c->scale_token, c->scale_head};
}

}  // namespace

extern "C" {

int32_t paged_kv_append_mx4(const sffn_heads* heads, const void* q, int64_t q_token, int64_t q_head,
                            const void* k, int64_t k_token, int64_t k_head, const void* v,
                            int64_t v_token, int64_t v_head, const void* q_weight,
                            const void* k_weight, const float* rot_table, const int32_t* positions,
                            const int32_t* slots, void* q_out, int64_t qo_token, int64_t qo_head,
                            const sffn_mx4* k_cache, const sffn_mx4* v_cache, int32_t n_pages,
                            int32_t page_size, void* stream) {
  int32_t st = check_heads_fwd(heads);
  if (st != SFFN_OK) return st;
  const sffn_heads& h = *heads;
  if (h.n_kv_heads == 0 || n_pages < 0 || page_size <= 0) return SFFN_ERR_ARG;
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
         check_mx4(k_cache, n_pages, page_size, h.n_kv_heads, h.head_dim),
         check_mx4(v_cache, n_pages, page_size, h.n_kv_heads, h.head_dim)});
  if (st != SFFN_OK) return st;
  HeadsFwd p = fwd_params(heads, q_weight, k_weight, rot_table, positions);
  p.q = q, p.q_token = q_token, p.q_head = q_head;
  p.k = k, p.k_token = k_token, p.k_head = k_head;
  p.v = v, p.v_token = v_token, p.v_head = v_head;
  p.q_out = q_out, p.qo_token = qo_token, p.qo_head = qo_head;
  p.slots = slots, p.n_pages = n_pages, p.page_size = page_size;
  return hip_status(launch_heads_mx4(h.dtype, p, mx4_rows(k_cache), mx4_rows(v_cache), (hipStream_t)stream));
}

int32_t paged_kv_read_mx4(int32_t T, int32_t n_kv_heads, int32_t head_dim, int32_t dtype,
                          const sffn_mx4* k_cache, const sffn_mx4* v_cache, int32_t n_pages,
                          int32_t page_size, const int32_t* slots, void* k_out, int64_t ko_token,
                          int64_t ko_head, void* v_out, int64_t vo_token, int64_t vo_head,
                          void* stream) {
  if (T < 0 || n_kv_heads <= 0 || head_dim <= 0 || n_pages < 0 || page_size <= 0) return SFFN_ERR_ARG;
  if (dtype != SFFN_F32 && dtype != SFFN_BF16) return SFFN_ERR_ARG;
  if (head_dim % 8 != 0 || head_dim > 256 || n_kv_heads > 4096) return SFFN_ERR_UNSUPPORTED;
  if ((int64_t)n_pages * page_size > (1ll << 31)) return SFFN_ERR_UNSUPPORTED;
  // up to 32 threads a row in one grid, which has less than 2^32 of them
  if ((int64_t)T * n_kv_heads > (1 << 27) - 64) return SFFN_ERR_UNSUPPORTED;
  if (T == 0 || (k_out == nullptr && v_out == nullptr)) return SFFN_OK;
  int32_t st = given(slots, 4) ? SFFN_OK : SFFN_ERR_ARG;
  if (st == SFFN_OK && k_out != nullptr)
    st = first_error({check_rows(k_out, T, ko_token, n_kv_heads, ko_head, head_dim, dtype, true),
                      check_mx4(k_cache, n_pages, page_size, n_kv_heads, head_dim)});
  if (st == SFFN_OK && v_out != nullptr)
    st = first_error({check_rows(v_out, T, vo_token, n_kv_heads, vo_head, head_dim, dtype, true),
                      check_mx4(v_cache, n_pages, page_size, n_kv_heads, head_dim)});
  if (st != SFFN_OK) return st;
  Mx4Read p = {};
  if (k_out != nullptr) p.cache[0] = mx4_rows(k_cache);
  if (v_out != nullptr) p.cache[1] = mx4_rows(v_cache);
  p.slots = slots;
  p.out[0] = k_out, p.o_token[0] = ko_token, p.o_head[0] = ko_head;
  p.out[1] = v_out, p.o_token[1] = vo_token, p.o_head[1] = vo_head;
  p.T = T, p.hkv = n_kv_heads, p.D = head_dim, p.n_pages = n_pages, p.page_size = page_size;
  return hip_status(launch_mx4_read(dtype, p, (hipStream_t)stream));
}

size_t paged_attn_mx4_workspace_bytes(const sffn_paged_batch* batch) {
  size_t bytes = 0;
  return check_batch(batch, &bytes, plan_paged_attn_mx4) == SFFN_OK ? bytes : 0;
}

int32_t paged_attn_mx4_fwd(const sffn_paged_batch* batch, const void* q, int64_t q_token,
                           int64_t q_head, const sffn_mx4* k_cache, const sffn_mx4* v_cache,
                           const int32_t* q_start, const int32_t* kv_len, const int32_t* block_table,
                           void* out, int64_t o_token, int64_t o_head, float* lse, void* workspace,
                           size_t ws_bytes, void* stream) {
  size_t need = 0;
  int32_t st = check_batch(batch, &need, plan_paged_attn_mx4);
  if (st != SFFN_OK) return st;
  const sffn_paged_batch& b = *batch;
  if (b.T == 0 || b.n_seqs == 0 || b.max_q == 0) return SFFN_OK;
  st = first_error({check_rows(q, b.T, q_token, b.n_q_heads, q_head, b.head_dim, b.dtype, false),
                    check_rows(out, b.T, o_token, b.n_q_heads, o_head, b.head_dim, b.dtype, true),
                    given(q_start, 4) && given(kv_len, 4) && aligned(lse, 4) ? SFFN_OK : SFFN_ERR_ARG});
  if (st == SFFN_OK && b.max_kv > 0)
    st = first_error({check_mx4(k_cache, b.n_pages, b.page_size, b.n_kv_heads, b.head_dim),
                      check_mx4(v_cache, b.n_pages, b.page_size, b.n_kv_heads, b.head_dim),
                      given(block_table, 4) ? SFFN_OK : SFFN_ERR_ARG});
  if (st != SFFN_OK) return st;
  PagedAttn p = attn_params(batch);
  p.q = q, p.q_token = q_token, p.q_head = q_head;
  p.out = out, p.o_token = o_token, p.o_head = o_head;
  p.q_start = q_start, p.kv_len = kv_len, p.block_table = block_table, p.lse = lse;
  if (need > 0 && (!given(workspace, 16) || ws_bytes < need)) return SFFN_ERR_WORKSPACE;
  const Mx4Rows none = {};
  return hip_status(launch_paged_attn_mx4(b.dtype, p, b.max_kv > 0 ? mx4_rows(k_cache) : none,
                                          b.max_kv > 0 ? mx4_rows(v_cache) : none, workspace,
                                          (hipStream_t)stream));
}

}  // extern "C"
