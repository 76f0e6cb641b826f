// serve_api.cu -- the C ABI of the operators around the adapted projections (include/mlora.h):
// argument validation (every host-detectable error is returned before any launch) and dispatch.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "mlora.h"
#include "serve.h"

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

template <class... P>
bool all_aligned(uintptr_t a, const P *...p) {
  return (aligned(p, a) && ...);
}

#define TRY(expr)              \
  do {                         \
    const int rc_ = (expr);    \
    if (rc_ != MLORA_OK) return rc_; \
  } while (0)

int done(cudaError_t e, const char *where) {
  if (e != cudaSuccess) return mlora::api_cuda_fail(e, where);
  return MLORA_OK;
}

int check_cache(const mlora_kv_cache *c, int32_t layer) {
  if (!c) return MLORA_ERR_NULL;
  if (c->dtype != MLORA_BF16 && c->dtype != MLORA_FP16) return MLORA_ERR_DTYPE;
  if (!c->k || !c->v) return MLORA_ERR_NULL;
  if (c->num_layers < 1 || c->num_kv_heads < 1 || c->page_tokens < 1 || c->num_pages < 1) return MLORA_ERR_SHAPE;
  if (c->head_dim < 8 || c->head_dim > MLORA_KV_MAX_HEAD_DIM) return MLORA_ERR_SHAPE;
  if (layer < 0 || layer >= c->num_layers) return MLORA_ERR_SHAPE;
  if (c->page_stride < 0 || c->layer_stride < 0 || c->token_stride < 0 || c->head_stride < 0) return MLORA_ERR_SHAPE;
  if (c->head_dim % 8 || c->page_stride % 8 || c->layer_stride % 8 || c->token_stride % 8 || c->head_stride % 8)
    return MLORA_ERR_ALIGN;
  if (!all_aligned(16, c->k, c->v)) return MLORA_ERR_ALIGN;
  return MLORA_OK;
}

// Rows of 16-bit elements: `width` of them every ld.
int check_rows(const void *p, int64_t ld, int64_t width) {
  if (!p) return MLORA_ERR_NULL;
  if (ld < width) return MLORA_ERR_SHAPE;
  if (!aligned(p, 16) || ld % 8) return MLORA_ERR_ALIGN;
  return MLORA_OK;
}

// In place, a row's output has to be where its input is: with other distances rows would overwrite each other's inputs.
int check_in_place(const void *in, const void *out, int64_t ld_in, int64_t ld_out, int32_t rows) {
  return in == out && ld_in != ld_out && rows > 1 ? MLORA_ERR_SHAPE : MLORA_OK;
}

int check_table(int32_t max_pages, int64_t table_stride, int32_t page_tokens) {
  if (max_pages < 0 || table_stride < max_pages) return MLORA_ERR_SHAPE;
  if ((int64_t)max_pages * page_tokens > INT32_MAX) return MLORA_ERR_SHAPE;  // positions are int32
  return MLORA_OK;
}

}  // namespace

extern "C" {

int lora_kv_layout(const mlora_kv_batch *b, int32_t *dev_status, void *stream) {
  if (!b) return MLORA_ERR_NULL;
  if (b->num_requests < 0 || b->num_requests > MLORA_KV_MAX_REQUESTS || b->num_rows < 0) return MLORA_ERR_SHAPE;
  if (b->page_tokens < 1 || b->num_pages < 1) return MLORA_ERR_SHAPE;
  TRY(check_table(b->max_pages, b->table_stride, b->page_tokens));
  if (!b->free_ring || !b->free_state || !b->free_state_out) return MLORA_ERR_NULL;
  if (b->num_requests && (!b->new_tokens || !b->kv_len || !b->kv_len_out)) return MLORA_ERR_NULL;
  if (b->num_requests && b->max_pages && !b->page_table) return MLORA_ERR_NULL;
  if (b->num_rows && (!b->row_request || !b->position || !b->cache_slot)) return MLORA_ERR_NULL;
  if (!all_aligned(4, b->new_tokens, b->kv_len, b->kv_len_out, b->page_table, b->free_ring, b->free_state,
                   b->free_state_out, b->adapter_slot, b->row_request, b->position, b->row_slot, b->seg_offsets,
                   b->seg_slot, dev_status) ||
      !aligned(b->cache_slot, 8))
    return MLORA_ERR_ALIGN;
  return done(mlora::launch_kv_layout(*b, dev_status, static_cast<cudaStream_t>(stream)), "cache layout launch");
}

int lora_kv_append(const mlora_kv_cache *cache, const mlora_kv_rows *r, int32_t layer, int32_t *dev_status,
                   void *stream) {
  if (!r) return MLORA_ERR_NULL;
  TRY(check_cache(cache, layer));
  if (r->num_rows < 0 || r->num_q_heads < 0 || r->rotary_dim < 0) return MLORA_ERR_SHAPE;
  if (!r->rope_cos != !r->rope_sin) return MLORA_ERR_NULL;
  if (r->rope_cos) {
    if (r->rotary_dim > cache->head_dim || r->max_position < 1) return MLORA_ERR_SHAPE;
    if (r->rotary_dim % 16 || !all_aligned(16, r->rope_cos, r->rope_sin)) return MLORA_ERR_ALIGN;
  } else if (r->rotary_dim) {
    return MLORA_ERR_NULL;
  }
  // pairs of 8 head elements and rows x heads are counted in 31 bits
  const int64_t width = (int64_t)cache->num_kv_heads * cache->head_dim;
  const int64_t qwidth = (int64_t)r->num_q_heads * cache->head_dim;
  if (2 * width + qwidth > INT32_MAX) return MLORA_ERR_SHAPE;
  if (r->num_rows == 0) return MLORA_OK;
  if (!r->cache_slot || (r->rotary_dim && !r->position)) return MLORA_ERR_NULL;
  TRY(check_rows(r->k, r->ldk, width));
  TRY(check_rows(r->v, r->ldv, width));
  if (r->num_q_heads) {
    TRY(check_rows(r->q, r->ldq, qwidth));
    TRY(check_rows(r->q_out, r->ldq_out, qwidth));
    TRY(check_in_place(r->q, r->q_out, r->ldq, r->ldq_out, r->num_rows));
  }
  if (!aligned(r->cache_slot, 8) || !all_aligned(4, r->position, dev_status)) return MLORA_ERR_ALIGN;
  return done(mlora::launch_kv_append(*cache, *r, layer, dev_status, static_cast<cudaStream_t>(stream)),
              "cache append launch");
}

int64_t lora_kv_attention_workspace(const mlora_kv_cache *cache, int32_t num_q_heads) {
  if (!cache || num_q_heads < 1) return 0;
  return mlora::kv_attention_workspace_bytes(cache->head_dim);
}

int lora_kv_attention(const mlora_kv_cache *cache, const mlora_kv_attn *a, int32_t layer, int32_t *dev_status,
                      void *stream) {
  return lora_kv_attention_ex(cache, a, layer, 0, dev_status, stream);
}

int lora_kv_attention_ex(const mlora_kv_cache *cache, const mlora_kv_attn *a, int32_t layer, int32_t rows_per_request,
                         int32_t *dev_status, void *stream) {
  if (!a) return MLORA_ERR_NULL;
  TRY(check_cache(cache, layer));
  if (rows_per_request < 0 || a->num_rows < 0 || a->num_requests < 0 || a->window < 0) return MLORA_ERR_SHAPE;
  if (a->num_q_heads < 1 || a->num_q_heads % cache->num_kv_heads || !std::isfinite(a->scale)) return MLORA_ERR_SHAPE;
  TRY(check_table(a->max_pages, a->table_stride, cache->page_tokens));
  if (!mlora::kv_attention_fits(*cache, *a)) return MLORA_ERR_SHAPE;
  if (a->num_rows == 0) return MLORA_OK;
  const int64_t width = (int64_t)a->num_q_heads * cache->head_dim;
  TRY(check_rows(a->q, a->ldq, width));
  TRY(check_rows(a->out, a->ldo, width));
  TRY(check_in_place(a->q, a->out, a->ldq, a->ldo, a->num_rows));
  if (!a->position || (a->num_requests && a->max_pages && !a->page_table)) return MLORA_ERR_NULL;
  if (!all_aligned(4, a->position, a->row_request, a->page_table, a->lse, dev_status)) return MLORA_ERR_ALIGN;
  const int64_t need = lora_kv_attention_workspace(cache, a->num_q_heads);
  if (need && !a->workspace) return MLORA_ERR_NULL;
  if (!aligned(a->workspace, 16)) return MLORA_ERR_ALIGN;
  if (a->workspace_bytes < need) return MLORA_ERR_WORKSPACE;
  return done(mlora::launch_kv_attention(*cache, *a, layer, rows_per_request, dev_status, static_cast<cudaStream_t>(stream)),
              "cache attention launch");
}

int lora_logits_adjust(const mlora_logits *a, int32_t *dev_status, void *stream) {
  if (!a) return MLORA_ERR_NULL;
  if (a->dtype != MLORA_BF16 && a->dtype != MLORA_FP16 && a->dtype != MLORA_FP32) return MLORA_ERR_DTYPE;
  if (a->num_rows < 0 || a->vocab < 1 || a->vocab > MLORA_LOGITS_MAX_VOCAB || a->num_requests < 0) return MLORA_ERR_SHAPE;
  if (a->num_rows == 0) return MLORA_OK;
  if (!a->logits || !a->out) return MLORA_ERR_NULL;
  if (a->ld < a->vocab || a->ldo < a->vocab) return MLORA_ERR_SHAPE;
  TRY(check_in_place(a->logits, a->out, a->ld, a->ldo, a->num_rows));
  // an empty array may be NULL beside its lengths
  if (!a->prompt_len != !a->total_len || (a->tokens && !a->total_len)) return MLORA_ERR_NULL;
  if (a->total_len && a->tokens_stride > 0 && !a->tokens) return MLORA_ERR_NULL;
  if (!a->bias_offsets && (a->bias_token || a->bias_value)) return MLORA_ERR_NULL;
  if (a->bias_offsets && a->num_bias > 0 && (!a->bias_token || !a->bias_value)) return MLORA_ERR_NULL;
  if (!a->mask != !a->mask_index) return MLORA_ERR_NULL;
  if (a->total_len && (a->tokens_stride < 0 || a->tokens_len < 0 || a->tokens_len > a->tokens_stride)) return MLORA_ERR_SHAPE;
  if (a->total_len && !a->tokens_len && a->tokens_stride > INT32_MAX) return MLORA_ERR_SHAPE;
  if (a->bias_offsets && a->num_bias < 0) return MLORA_ERR_SHAPE;
  if (a->mask && (a->num_masks < 1 || a->mask_stride < ((int64_t)a->vocab + 31) / 32)) return MLORA_ERR_SHAPE;
  const uintptr_t elem = a->dtype == MLORA_FP32 ? 4 : 2;
  if (!all_aligned(elem, static_cast<const char *>(a->logits), static_cast<const char *>(a->out)) ||
      !all_aligned(4, a->row_request, a->tokens, a->prompt_len, a->total_len, a->repetition, a->presence, a->frequency,
                   a->temperature, a->bias_offsets, a->bias_token, a->bias_value, a->mask, a->mask_index, dev_status))
    return MLORA_ERR_ALIGN;
  mlora_logits b = *a;
  if (b.total_len && !b.tokens_len) b.tokens_len = (int32_t)b.tokens_stride;
  return done(mlora::launch_logits_adjust(b, dev_status, static_cast<cudaStream_t>(stream)), "logits launch");
}

}  // extern "C"
