// Launch interface of the layer-norm kernels (internal to the library).
#pragma once

#include <cuda_runtime.h>

#include <cstddef>

namespace disco {

// The norm over the C channels of each of B * npts points of a (B, C, npts) field.
struct NormArgs {
  int B, C;
  long long npts;
  const void* x;
  const void* gain;  // [C] or null (ones)
  const void* bias;  // forward: [C] or null (zeros)
  float eps;
  void* out;     // forward
  float* stats;  // [2][B * npts] mean, 1 / deviation: written by the forward (may be null), read by the backward
  const void* dout;  // backward
  void* dx;          // may be null
  void* dgain;       // [C], may be null
  void* dbias;       // [C], may be null
  float* part;       // backward: norm_partials() x 2C sums of two floats
};

constexpr int kNormMaxChannels = 16384;

// Most rows of 2C partial sums the backward pass leaves for its reduction on a device of `sms` SMs.
int norm_partials(int sms);
// The ring form (norm_ring.cu) of either pass; false where its tiles do not fit.  *rows: rows of
// partial sums the backward pass leaves (at most norm_partials).
bool launch_norm_ring(bool bf16, const NormArgs& a, bool bwd, int sms, cudaStream_t st, int* rows, cudaError_t* err);
int take_norm_status();
cudaError_t launch_norm(bool bf16, const NormArgs& a, int sms, cudaStream_t st);
cudaError_t launch_norm_backward(bool bf16, const NormArgs& a, int sms, cudaStream_t st);

}  // namespace disco
