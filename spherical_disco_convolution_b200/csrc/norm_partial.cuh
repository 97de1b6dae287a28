// Partial sums of the layer norm's parameter gradients, between the kernels that make them.
#pragma once

#include <cuda_runtime.h>

namespace disco {

// A row of partial sums: 2C fp64 values (dgain, then dbias) as two fp32 numbers each, hi in the first
// 2C floats and lo in the next 2C, so that the workspace needs no more than its 4 bytes' alignment.
__device__ __forceinline__ void put_partial(float* row, int C, int i, double v) {
  const float hi = (float)v;
  row[i] = hi;
  row[2 * C + i] = isfinite(hi) ? (float)(v - (double)hi) : 0.0f;
}
__device__ __forceinline__ double get_partial(const float* row, int C, int i) {
  return (double)row[i] + (double)row[2 * C + i];
}

}  // namespace disco
