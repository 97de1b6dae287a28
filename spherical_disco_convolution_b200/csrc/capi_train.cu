// C ABI of the training operators next to the convolution: argument checks of the layer norm and
// of the orthogonalised update.  See include/disco.h for the contract of every entry point.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/disco.h"
#include "muon.h"
#include "norm.h"
#include "status.h"

namespace {

using disco::set_cuda_error;
using disco::set_error;

disco_status invalid(const char* msg) { return set_error(DISCO_ERR_INVALID_ARG, msg); }

bool aligned(const void* p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

disco_status sm_count(int* sms) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  return e == cudaSuccess ? DISCO_OK : set_cuda_error(e, "device query");
}

disco_status check_norm(int B, int C, long long npts, disco_dtype dtype) {
  if (B <= 0 || C <= 0 || npts <= 0) return invalid("B, C and npts must be positive");
  if (dtype != DISCO_F32 && dtype != DISCO_BF16) return invalid("unknown dtype");
  if (C > disco::kNormMaxChannels) return set_error(DISCO_ERR_UNSUPPORTED, "the norm takes at most 16384 channels");
  if (npts > 0x7fffffffll) return set_error(DISCO_ERR_UNSUPPORTED, "npts above 2^31 - 1");
  return DISCO_OK;
}

// The backward pass's rows of 2C partial sums, two floats each; more rows than any GPU of this kind has use for.
constexpr int kWorkspaceSms = 160;

size_t norm_bytes(int C) { return (size_t)disco::norm_partials(kWorkspaceSms) * 4 * C * sizeof(float); }

disco_status check_matrices(int n, int groups, int rows, int cols) {
  if (n <= 0 || groups <= 0 || rows <= 0 || cols <= 0) return invalid("n, groups, rows and cols must be positive");
  if ((long long)n * groups > 65535) return set_error(DISCO_ERR_UNSUPPORTED, "more than 65535 matrices in one call");
  if (std::max(rows, cols) > 32768) return set_error(DISCO_ERR_UNSUPPORTED, "a matrix side above 32768");
  return DISCO_OK;
}

disco_status check_update(int n, int groups, int rows, int cols, disco_dtype dtype, const disco_newton_schulz_t* ns,
                          const void* workspace, size_t ws_bytes) {
  disco_status s = check_matrices(n, groups, rows, cols);
  if (s) return s;
  if (dtype != DISCO_F32 && dtype != DISCO_BF16) return invalid("unknown dtype");
  if (!ns) return invalid("ns is NULL");
  if (ns->steps < 1 || ns->steps > 32) return invalid("steps outside 1..32");
  for (double v : {ns->a, ns->b, ns->c})
    if (!std::isfinite(v) || std::fabs(v) > 32) return invalid("a coefficient that is not finite or above 32 in magnitude");
  // below that 1 / (|U| + eps) leaves fp32's range for an update of zeros
  if (!std::isfinite(ns->eps) || ns->eps < 1e-30) return invalid("eps must be finite and at least 1e-30");
  const size_t need = disco::muon_workspace(n, groups, rows, cols);
  if (need && (!workspace || ws_bytes < need)) return invalid("workspace missing or too small");
  if (!aligned(workspace, 256)) return invalid("workspace must be 256-byte aligned");
  return DISCO_OK;
}

template <typename P>
bool bad_pointers(P const* ps, int n, size_t align) {
  if (!ps) return true;
  for (int i = 0; i < n; ++i)
    if (!ps[i] || !aligned(ps[i], align)) return true;
  return false;
}

disco::MuonArgs muon_args(int n, int groups, int rows, int cols, disco_dtype dtype, const disco_newton_schulz_t* ns) {
  disco::MuonArgs a{};
  a.n = n;
  a.groups = groups;
  a.rows = rows;
  a.cols = cols;
  a.bf16 = dtype == DISCO_BF16;
  a.steps = ns->steps;
  a.a = (float)ns->a;
  a.b = (float)ns->b;
  a.c = (float)ns->c;
  a.eps = ns->eps;
  return a;
}

disco_status muon(unsigned int hold_us, int n, int groups, int rows, int cols, disco_dtype dtype, const disco_newton_schulz_t* ns,
                  double lr, double momentum, int nesterov, double weight_decay, const void* const* w,
                  const void* const* grad, const float* const* m, void* const* w_out, float* const* m_out,
                  void* workspace, size_t ws_bytes, void* stream) {
  disco_status s = check_update(n, groups, rows, cols, dtype, ns, workspace, ws_bytes);
  if (s) return s;
  if (!std::isfinite(lr) || !std::isfinite(weight_decay)) return invalid("lr and weight_decay must be finite");
  if (!(momentum >= 0 && momentum < 1)) return invalid("momentum outside [0, 1)");
  const size_t es = dtype == DISCO_BF16 ? 2 : 4;
  if (bad_pointers(w, n, es) || bad_pointers(grad, n, es) || bad_pointers(w_out, n, es) || bad_pointers(m, n, 4) ||
      bad_pointers(m_out, n, 4))
    return invalid("w, grad, m, w_out and m_out hold n device pointers on their element's alignment");
  disco::MuonArgs a = muon_args(n, groups, rows, cols, dtype, ns);
  a.in = grad;
  a.out = w_out;
  a.step = true;
  a.w = w;
  a.m = m;
  a.m_out = m_out;
  a.keep = (float)(1 - lr * weight_decay);
  a.rate = (float)(lr * std::sqrt(std::max(1.0, (double)rows / cols)));
  a.momentum = (float)momentum;
  a.nesterov = nesterov != 0;
  a.hold_ns = 1000ull * hold_us;
  cudaError_t e = disco::launch_muon(a, workspace, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DISCO_OK : set_cuda_error(e, "update launch");
}

}  // namespace

extern "C" {

disco_status disco_norm_workspace_size(int B, int C, long long npts, disco_dtype dtype, size_t* bytes) {
  if (!bytes) return invalid("NULL argument");
  disco_status s = check_norm(B, C, npts, dtype);
  if (s) return s;
  *bytes = norm_bytes(C);
  return DISCO_OK;
}

disco_status disco_norm(int B, int C, long long npts, disco_dtype dtype, const void* x, const void* gain,
                        const void* bias, double eps, void* out, float* stats, void* stream) {
  disco_status s = check_norm(B, C, npts, dtype);
  if (s) return s;
  if (!x || !out) return invalid("x and out must be non-NULL");
  if (!std::isfinite(eps) || eps < 0) return invalid("eps must be finite and not negative");
  const size_t es = dtype == DISCO_BF16 ? 2 : 4;
  if (!aligned(x, es) || !aligned(gain, es) || !aligned(bias, es) || !aligned(out, es) || !aligned(stats, 4))
    return invalid("a pointer is off its element's alignment");
  int sms = 0;
  if ((s = sm_count(&sms))) return s;
  disco::NormArgs a{};
  a.B = B;
  a.C = C;
  a.npts = npts;
  a.x = x;
  a.gain = gain;
  a.bias = bias;
  a.eps = (float)eps;
  a.out = out;
  a.stats = stats;
  cudaError_t e = disco::launch_norm(dtype == DISCO_BF16, a, sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DISCO_OK : set_cuda_error(e, "norm launch");
}

disco_status disco_norm_backward(int B, int C, long long npts, disco_dtype dtype, const void* dout, const void* x,
                                 const float* stats, const void* gain, void* dx, void* dgain, void* dbias,
                                 void* workspace, size_t ws_bytes, void* stream) {
  disco_status s = check_norm(B, C, npts, dtype);
  if (s) return s;
  if (!dout || !x || !stats) return invalid("dout, x and stats must be non-NULL");
  if (!dx && !dgain && !dbias) return invalid("dx, dgain and dbias are all NULL");
  const size_t es = dtype == DISCO_BF16 ? 2 : 4;
  for (const void* p : {dout, x, gain, (const void*)dx, (const void*)dgain, (const void*)dbias})
    if (!aligned(p, es)) return invalid("a pointer is off its element's alignment");
  if (!aligned(stats, 4)) return invalid("a pointer is off its element's alignment");
  if (dgain || dbias) {
    if (!workspace || ws_bytes < norm_bytes(C)) return invalid("workspace missing or too small");
    if (!aligned(workspace, 4)) return invalid("a pointer is off its element's alignment");
  }
  int sms = 0;
  if ((s = sm_count(&sms))) return s;
  disco::NormArgs a{};
  a.B = B;
  a.C = C;
  a.npts = npts;
  a.x = x;
  a.gain = gain;
  a.stats = const_cast<float*>(stats);
  a.dout = dout;
  a.dx = dx;
  a.dgain = dgain;
  a.dbias = dbias;
  a.part = static_cast<float*>(workspace);
  cudaError_t e = disco::launch_norm_backward(dtype == DISCO_BF16, a, std::min(sms, kWorkspaceSms),
                                              static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DISCO_OK : set_cuda_error(e, "norm backward launch");
}

disco_status disco_orthogonalize_workspace_size(int n, int groups, int rows, int cols, size_t* bytes) {
  if (!bytes) return invalid("NULL argument");
  disco_status s = check_matrices(n, groups, rows, cols);
  if (s) return s;
  *bytes = disco::muon_workspace(n, groups, rows, cols);
  return DISCO_OK;
}

disco_status disco_orthogonalize(int n, int groups, int rows, int cols, disco_dtype dtype,
                                 const disco_newton_schulz_t* ns, const void* const* update, void* const* out,
                                 void* workspace, size_t ws_bytes, void* stream) {
  disco_status s = check_update(n, groups, rows, cols, dtype, ns, workspace, ws_bytes);
  if (s) return s;
  const size_t es = dtype == DISCO_BF16 ? 2 : 4;
  if (bad_pointers(update, n, es) || bad_pointers(out, n, es))
    return invalid("update and out hold n device pointers on their element's alignment");
  disco::MuonArgs a = muon_args(n, groups, rows, cols, dtype, ns);
  a.in = update;
  a.out = out;
  cudaError_t e = disco::launch_muon(a, workspace, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DISCO_OK : set_cuda_error(e, "orthogonalisation launch");
}

disco_status disco_muon(int n, int groups, int rows, int cols, disco_dtype dtype, const disco_newton_schulz_t* ns,
                        double lr, double momentum, int nesterov, double weight_decay, const void* const* w,
                        const void* const* grad, const float* const* m, void* const* w_out, float* const* m_out,
                        void* workspace, size_t ws_bytes, void* stream) {
  return muon(0, n, groups, rows, cols, dtype, ns, lr, momentum, nesterov, weight_decay, w, grad, m, w_out, m_out,
              workspace, ws_bytes, stream);
}

disco_status disco_muon_wait_selftest(unsigned int limit_us, int n, int groups, int rows, int cols, disco_dtype dtype,
                                      const disco_newton_schulz_t* ns, double lr, double momentum, int nesterov,
                                      double weight_decay, const void* const* w, const void* const* grad,
                                      const float* const* m, void* const* w_out, float* const* m_out, void* workspace,
                                      size_t ws_bytes, void* stream) {
  if (limit_us < 1 || limit_us > 1000000) return invalid("limit_us must be in [1, 1000000]");
  if (std::min(rows, cols) <= 32) return set_error(DISCO_ERR_UNSUPPORTED, "matrices of up to 32 rows may have no wait");
  return muon(limit_us, n, groups, rows, cols, dtype, ns, lr, momentum, nesterov, weight_decay, w, grad, m, w_out, m_out,
              workspace, ws_bytes, stream);
}

}  // extern "C"
