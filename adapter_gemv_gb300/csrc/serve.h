// serve.h -- launchers of the operators around the adapted projections (cache layout, append,
// attention, logits; norm, 8-bit rows and products, sampling), shared by the C ABI files and the kernel files.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "mlora.h"

namespace mlora {

// Defined in api.cu: records a CUDA error's text and returns MLORA_ERR_CUDA; counts one launch; the limit of a kernel's
// waits that this thread has set, 0: the kernels' default.
int api_cuda_fail(cudaError_t e, const char *where);
void api_count_launch();
uint64_t api_wait_limit_ns();

cudaError_t launch_kv_layout(const mlora_kv_batch &b, int32_t *status, cudaStream_t stream);
cudaError_t launch_kv_append(const mlora_kv_cache &c, const mlora_kv_rows &r, int32_t layer, int32_t *status,
                             cudaStream_t stream);
cudaError_t launch_kv_attention(const mlora_kv_cache &c, const mlora_kv_attn &a, int32_t layer, int32_t rows_per_request,
                                int32_t *status, cudaStream_t stream);
bool kv_attention_fits(const mlora_kv_cache &c, const mlora_kv_attn &a);  // one row's tiles counted in 31 bits
int64_t kv_attention_workspace_bytes(int32_t head_dim);
cudaError_t launch_logits_adjust(const mlora_logits &a, int32_t *status, cudaStream_t stream);
cudaError_t launch_rms_norm(const mlora_norm &a, cudaStream_t stream);
cudaError_t launch_quantize(const mlora_quant &a, cudaStream_t stream);
cudaError_t launch_fp8_matmul(const mlora_matmul &a, int32_t *status, uint64_t wait_ns, cudaStream_t stream);
bool fp8_matmul_fits(const mlora_matmul &a);  // its tiles counted in 31 bits
cudaError_t launch_sample(const mlora_sampling &a, int32_t *status, cudaStream_t stream);

// Defined in decode_launch.cu: number of SMs of the current device.
int sm_count();

// n / d for 0 <= n < 2^31 and a divisor fixed per launch: a multiply-high and a shift (Granlund and
// Montgomery, 1994).
struct FastDiv {
  uint32_t mul;
  int32_t shift;
  int32_t d;
};
inline FastDiv fast_div(int32_t d) {
  int l = 0;
  while ((1ull << l) < (uint64_t)d) ++l;
  return FastDiv{(uint32_t)(((1ull << 32) * ((1ull << l) - (uint64_t)d)) / (uint64_t)d + 1), l, d};
}

}  // namespace mlora
