// step_api.cu -- the C ABI of the norm, the 8-bit rows, the base product and the next token (include/mlora.h):
// argument validation (every host-detectable error is returned before any launch) and dispatch.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "mlora.h"
#include "serve_check.h"

using namespace mlora::check;

namespace {

int check_type(int32_t dtype) { return dtype == MLORA_BF16 || dtype == MLORA_FP16 ? MLORA_OK : MLORA_ERR_DTYPE; }

int64_t blocks_of(int64_t columns) { return (columns + MLORA_FP8_BLOCK - 1) / MLORA_FP8_BLOCK; }

// Scales of `blocks` blocks every ld.
int check_scale(const float *scale, int64_t ld, int64_t blocks) {
  if (!scale) return MLORA_ERR_NULL;
  if (ld < blocks) return MLORA_ERR_SHAPE;
  return aligned(scale, 4) ? MLORA_OK : MLORA_ERR_ALIGN;
}

// e4m3 rows, `width` values every ld, ld a multiple of `step`.
int check_bytes(const void *q, int64_t ld, int64_t width, int64_t step) {
  if (!q) return MLORA_ERR_NULL;
  if (ld < width) return MLORA_ERR_SHAPE;
  return aligned(q, 16) && ld % step == 0 ? MLORA_OK : MLORA_ERR_ALIGN;
}

// 8-bit rows that a call writes, or none.
int check_q_out(const void *q, int64_t ldq, const float *scale, int64_t lds, int64_t width) {
  if (!q && !scale) return MLORA_OK;
  TRY(check_bytes(q, ldq, width, 8));
  return check_scale(scale, lds, blocks_of(width));
}

// Whether an output (or none) is over no other of the call's arrays: a CTA would read there what another has written.
template <class... P>
bool apart(const void *out, const P *...others) {
  return !out || ((static_cast<const void *>(others) != out) && ...);
}

}  // namespace

extern "C" {

int lora_rms_norm(const mlora_norm *a, void *stream) {
  if (!a) return MLORA_ERR_NULL;
  TRY(check_type(a->dtype));
  if (a->num_rows < 0 || a->width < 8 || a->width > MLORA_ROW_MAX_WIDTH) return MLORA_ERR_SHAPE;
  if (!(a->eps >= 0x1p-126f) || !std::isfinite(a->eps)) return MLORA_ERR_SHAPE;
  if (a->width % 8) return MLORA_ERR_ALIGN;
  if (a->num_rows == 0) return MLORA_OK;
  TRY(check_rows(a->x, a->ldx, a->width));
  if (!a->residual != !a->residual_out || (!a->out && !a->q)) return MLORA_ERR_NULL;
  if (a->residual) {
    TRY(check_rows(a->residual, a->ldr, a->width));
    TRY(check_rows(a->residual_out, a->ldro, a->width));
    TRY(check_in_place(a->residual, a->residual_out, a->ldr, a->ldro, a->num_rows));
    TRY(check_in_place(a->x, a->residual_out, a->ldx, a->ldro, a->num_rows));
    if (a->residual_out == a->out || a->residual_out == a->q) return MLORA_ERR_SHAPE;
  }
  if (a->out) {
    TRY(check_rows(a->out, a->ldo, a->width));
    TRY(check_in_place(a->x, a->out, a->ldx, a->ldo, a->num_rows));
    TRY(check_in_place(a->residual, a->out, a->ldr, a->ldo, a->num_rows));
    if (a->out == a->q) return MLORA_ERR_SHAPE;
  }
  TRY(check_q_out(a->q, a->ldq, a->q_scale, a->lds, a->width));
  if (!aligned(a->weight, 16)) return MLORA_ERR_ALIGN;
  if (!apart(a->residual_out, a->weight) || !apart(a->out, a->weight) || !apart(a->q, a->x, a->residual, a->weight) ||
      !apart(a->q_scale, a->x, a->residual, a->weight, a->residual_out, a->out, a->q))
    return MLORA_ERR_SHAPE;
  return done(mlora::launch_rms_norm(*a, static_cast<cudaStream_t>(stream)), "norm launch");
}

int lora_quantize(const mlora_quant *a, void *stream) {
  if (!a) return MLORA_ERR_NULL;
  TRY(check_type(a->dtype));
  if (a->num_rows < 0 || a->width < 8 || a->width > INT32_MAX - MLORA_FP8_BLOCK) return MLORA_ERR_SHAPE;
  if (a->width % 8) return MLORA_ERR_ALIGN;
  if (a->num_rows == 0) return MLORA_OK;
  TRY(check_rows(a->x, a->ldx, a->width));
  if (!a->out && !a->q) return MLORA_ERR_NULL;
  if (a->gate) TRY(check_rows(a->gate, a->ldg, a->width));
  if (a->out) {
    TRY(check_rows(a->out, a->ldo, a->width));
    TRY(check_in_place(a->x, a->out, a->ldx, a->ldo, a->num_rows));
    TRY(check_in_place(a->gate, a->out, a->ldg, a->ldo, a->num_rows));
    if (a->out == a->q) return MLORA_ERR_SHAPE;
  }
  TRY(check_q_out(a->q, a->ldq, a->q_scale, a->lds, a->width));
  if (!apart(a->q, a->x, a->gate) || !apart(a->q_scale, a->x, a->gate, a->out, a->q)) return MLORA_ERR_SHAPE;
  return done(mlora::launch_quantize(*a, static_cast<cudaStream_t>(stream)), "quantize launch");
}

int lora_fp8_matmul(const mlora_matmul *a, int32_t *dev_status, void *stream) {
  if (!a) return MLORA_ERR_NULL;
  TRY(check_type(a->dtype));
  if (a->num_rows < 0 || a->d_in < 16 || a->d_out < 8) return MLORA_ERR_SHAPE;
  if (a->d_out > INT32_MAX - 256) return MLORA_ERR_SHAPE;  // a tile's last column is counted in 31 bits
  if (a->d_in % 16 || a->d_out % 8) return MLORA_ERR_ALIGN;
  if (a->num_rows == 0) return MLORA_OK;
  if (!mlora::fp8_matmul_fits(*a)) return MLORA_ERR_SHAPE;
  const int64_t blocks = blocks_of(a->d_in);
  TRY(check_bytes(a->x, a->ldx, a->d_in, 16));
  TRY(check_bytes(a->w, a->ldw, a->d_in, 16));
  TRY(check_scale(a->x_scale, a->ldxs, blocks));
  TRY(check_scale(a->w_scale, a->ldws, blocks));
  TRY(check_rows(a->y, a->ldy, a->d_out));
  if (!apart(a->y, a->x, a->w, a->x_scale, a->w_scale)) return MLORA_ERR_SHAPE;
  if (!aligned(dev_status, 4)) return MLORA_ERR_ALIGN;
  return done(mlora::launch_fp8_matmul(*a, dev_status, mlora::api_wait_limit_ns(), static_cast<cudaStream_t>(stream)), "8-bit product launch");
}

int lora_sample(const mlora_sampling *a, int32_t *dev_status, void *stream) {
  if (!a) return MLORA_ERR_NULL;
  if (a->dtype != MLORA_FP32) TRY(check_type(a->dtype));
  if (a->num_rows < 0 || a->vocab < 1 || a->vocab > MLORA_SAMPLE_MAX_VOCAB || a->num_requests < 0) return MLORA_ERR_SHAPE;
  if (a->num_rows == 0) return MLORA_OK;
  if (!a->logits || !a->uniform || !a->token) return MLORA_ERR_NULL;
  if (a->ld < a->vocab) return MLORA_ERR_SHAPE;
  if (!aligned(a->logits, a->dtype == MLORA_FP32 ? 4 : 2) ||
      !all_aligned(4, a->row_request, a->uniform, a->temperature, a->top_k, a->top_p, a->min_p, a->token, a->logprob,
                   dev_status))
    return MLORA_ERR_ALIGN;
  if (!apart(a->token, a->logits, a->row_request, a->uniform, a->temperature, a->top_k, a->top_p, a->min_p) ||
      !apart(a->logprob, a->logits, a->row_request, a->uniform, a->temperature, a->top_k, a->top_p, a->min_p, a->token))
    return MLORA_ERR_SHAPE;
  return done(mlora::launch_sample(*a, dev_status, static_cast<cudaStream_t>(stream)), "sampling launch");
}

}  // extern "C"
