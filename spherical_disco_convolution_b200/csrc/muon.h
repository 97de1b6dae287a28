// Launch interface of the orthogonalised-update kernels (internal to the library).
#pragma once

#include <cuda_runtime.h>

#include <cstddef>

namespace disco {

// n tensors of groups x rows x cols values; every (rows x cols) matrix by itself.
struct MuonArgs {
  int n, groups, rows, cols;
  bool bf16;
  int steps;
  float a, b, c;
  double eps;
  // update: `in` -> `out` (step false), or the whole step (step true): in = grad, out = w_out
  const void* const* in;
  void* const* out;
  bool step;
  const void* const* w;
  const float* const* m;
  float* const* m_out;
  float keep, rate;       // w' = keep * w - rate * X
  float momentum;
  bool nesterov;
  unsigned long long hold_ns;  // self test: a first product whose waits run out after this (0: none)
};

// 0 where a matrix fits the one-launch forms.
size_t muon_workspace(int n, int groups, int rows, int cols);
cudaError_t launch_muon(const MuonArgs& a, void* workspace, cudaStream_t st);
int take_muon_status();

}  // namespace disco
