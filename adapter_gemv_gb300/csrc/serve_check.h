// serve_check.h -- argument checks shared by the C ABI files of the operators around the adapted projections.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "mlora.h"
#include "serve.h"

namespace mlora {
namespace check {

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

template <class... P>
inline bool all_aligned(uintptr_t a, const P *...p) {
  return (aligned(p, a) && ...);
}

#define TRY(expr)              \
  do {                         \
    const int rc_ = (expr);    \
    if (rc_ != MLORA_OK) return rc_; \
  } while (0)

inline int done(cudaError_t e, const char *where) {
  if (e != cudaSuccess) return mlora::api_cuda_fail(e, where);
  return MLORA_OK;
}

// Rows of 16-bit elements: `width` of them every ld.
inline int check_rows(const void *p, int64_t ld, int64_t width) {
  if (!p) return MLORA_ERR_NULL;
  if (ld < width) return MLORA_ERR_SHAPE;
  if (!aligned(p, 16) || ld % 8) return MLORA_ERR_ALIGN;
  return MLORA_OK;
}

// In place, a row's output has to be where its input is: with other distances rows would overwrite each other's inputs.
inline int check_in_place(const void *in, const void *out, int64_t ld_in, int64_t ld_out, int32_t rows) {
  return in == out && ld_in != ld_out && rows > 1 ? MLORA_ERR_SHAPE : MLORA_OK;
}

}  // namespace check
}  // namespace mlora
