// Launchers of the per-head norm + rotation of queries and keys and of its gradients (qk_norm.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "fvattn.h"

namespace fv {

// Device pointers of one call; the sizes and strides are the caller's fvattn_qk_shape.
struct QkNormArgs {
  const void *q, *k;              // projections [B, S, H, d]
  const void *wq, *wk;            // norm weights [d], null: ones
  const float *cos, *sin;         // rotation tables [table_rows, rot / 2], null when rot == 0
  const int32_t* positions;       // [B, S] rows of the tables, null: row s
  void *qo, *ko;                  // forward: outputs [B, H, S, d]; backward: gradients [B, S, H, d] of q, k
  const void *gq, *gk;            // backward: gradients of the outputs [B, H, S, d]
  float *dwq, *dwk;               // backward: weight gradients [d], null: not wanted
  float* parts;                   // backward: per-CTA partial weight gradients
  int32_t* status;                // null: not reported
};

cudaError_t launch_qk_norm(const QkNormArgs& a, const fvattn_qk_shape& s, cudaStream_t st);
cudaError_t launch_qk_norm_bwd(const QkNormArgs& a, const fvattn_qk_shape& s, cudaStream_t st);
// Bytes of QkNormArgs::parts (0 when the norm has no weights).
size_t qk_norm_part_bytes(const fvattn_qk_shape& s);

}  // namespace fv
