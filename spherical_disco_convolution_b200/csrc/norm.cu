// Layer norm of a field over its channels, forward and backward.
//
// For every point n of a (B, C, P) field, over its C channels:
//   mean = sum x / C,  var = sum (x - mean)^2 / C,  r = 1 / sqrt(var + eps)
//   out_c = gain_c xh_c + bias_c,  xh = (x - mean) r
// and backward, with e = gain dout:
//   dx = r (e - sum(e) / C - xh sum(e xh) / C)
//   dgain_c = sum_n dout xh,  dbias_c = sum_n dout
//
// This is the form for planes shorter than 64 points and for more channels than the tiles of
// norm_ring.cu hold (1024 forward, 512 backward); long planes with fewer go there (the 64 channels of
// 721 x 1440 points in bf16 took 107 us forward and 266 backward here, and take 52 and 93 there).
// Measured (forward, backward): 1500 channels of 91 x 180 points in bf16 45 and 87 us, in fp32 75 and 114
// (their bytes once: 15 and 23, 30 and 45); 1500 x 9 points, 4000 fields, bf16 275 and 313 (33 and 50);
// (20000, 64) in fp32 12 and 20, (20000, 256) in bf16 30 and 88: points of a single-point plane lie C apart.
//
// The channels of a point lie P elements apart, so a warp reads runs of consecutive points of
// one channel (16 bytes a lane where the alignment allows) and the sums over channels cross the
// warps of a CTA.  A CTA is TX lanes over points times TY rows over channels; a thread keeps
// its NC channels of PT points in registers from the load to the store, so x (and dout) cross
// HBM once.  What bounds both passes is HBM.
//
// Sums are fp32.  Neither the mean nor the deviation is formed from large sums: a thread adds the
// differences of its NC channels from the first of them and their squares (k being one of n values,
// m2 = sum (x - k)^2 - (sum (x - k))^2 / n loses log2(n) + 1 = 4 bits at most; the looping form adds
// squared deviations from the running mean), and partial results combine as (n, m, m2) + (n', m', m2') -> mean m + (m' - m) n' / (n + n'),
// m2 + m2' + (m - m')^2 n n' / (n + n') (the pairwise update of Chan, Golub and LeVeque).  So the mean
// of equal channels is their value to the bit, and a mean far from zero is rounded about once.
//
// The gradients of gain and bias are sums over all points, and a long chain of fp32 additions loses
// as much as it is long.  So only a tile's values are added in fp32: a thread adds its channels' over
// every tile its CTA visits in fp64, the TX lanes of a channel are added by shuffles, each CTA writes
// one row of 2C partial sums, and a second kernel adds the rows in a fixed order (no atomics: the same
// bits every time).  The looping form has its channels' sums in shared memory, where 16 384 channels
// leave no room for fp64: of eight tiles in fp32, and then added to the CTA's row.
#include <cuda_runtime.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "norm.h"
#include "norm_partial.cuh"

namespace disco {
namespace {

template <typename T, int VEC>
struct alignas(VEC * sizeof(T)) Pack {
  T v[VEC];
};

// Points per thread: 16 bytes of one channel, as one vector or as PT / VEC narrower ones.
template <typename T>
constexpr int kPt = 16 / (int)sizeof(T);

constexpr int kMaxThreads = 512;

struct NormShape {
  long long nvec;  // B * P / VEC vectors of points
  long long pv;    // P / VEC vectors per plane
  int C;
  int TX, TY;
};

// Combines (n, mean, m2) with the lane `mask` away; n = 0 stands for no values.
__device__ __forceinline__ void combine_shfl(float& n, float& mean, float& m2, int mask) {
  const float n2 = __shfl_xor_sync(~0u, n, mask), mean2 = __shfl_xor_sync(~0u, mean, mask),
              q2 = __shfl_xor_sync(~0u, m2, mask);
  const float all = n + n2, share = all > 0.0f ? n2 / all : 0.0f;
  const float d = (n > 0.0f && n2 > 0.0f) ? mean2 - mean : 0.0f;
  mean = n > 0.0f ? fmaf(d, share, mean) : mean2;
  m2 = m2 + q2 + d * d * n * share;
  n = all;
}

// Channels row ty of a CTA owns: c = ty + TY * i.
__device__ __forceinline__ int row_channels(int C, int TY, int ty) { return ty < C ? (C - ty + TY - 1) / TY : 0; }

// One tile's statistics: every thread comes with mean and m2 of its channels for its PT points and
// leaves with mean and 1/deviation of the points.  `red` holds TYW rows (one per warp-sized
// piece of the channel rows) of (mean, m2) and one row of results; point (v, e) of the tile sits at
// e * (V + 1) + v, so that lanes along v and lanes along e are both free of bank conflicts.
template <int VEC, int NV>
__device__ __forceinline__ void tile_stats(const NormShape& g, float eps, float2* red, float (&s)[NV * VEC],
                                           float (&m2)[NV * VEC], long long tile_vec, float* stats) {
  const int tx = threadIdx.x, ty = threadIdx.y;
  const int V = g.TX * NV, row = VEC * (V + 1);
  const int rpw = 32 / g.TX;  // channel rows a warp holds
  const float n0 = (float)row_channels(g.C, g.TY, ty);
#pragma unroll
  for (int k = 0; k < NV * VEC; ++k) {
    float n = n0;
    for (int m = g.TX; m < 32; m <<= 1) combine_shfl(n, s[k], m2[k], m);
  }
  const int tyw = (g.TY + rpw - 1) / rpw;
  if (ty % rpw == 0) {
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        red[(ty / rpw) * row + e * (V + 1) + v * g.TX + tx] = make_float2(s[v * VEC + e], m2[v * VEC + e]);
  }
  __syncthreads();
  float2* fin = red + tyw * row;
  const int t = ty * g.TX + tx, nt = g.TX * g.TY;
  const int least = g.C / g.TY, extra = g.C - least * g.TY;
  for (int p = t; p < V * VEC; p += nt) {
    const int v = p / VEC, e = p % VEC, at = e * (V + 1) + v;
    // channels of row r of red; row 0 has some
    auto channels = [&](int r) { return (float)(rpw * least + min(max(extra - r * rpw, 0), rpw)); };
    const float of = red[at].x;
    float S = 0.0f;
    for (int r = 1; r < tyw; ++r) S = fmaf(red[r * row + at].x - of, channels(r), S);
    const float mean = of + S / (float)g.C;
    float M = 0.0f;
    for (int r = 0; r < tyw; ++r) {
      const float2 q = red[r * row + at];
      const float n = channels(r), d = n > 0.0f ? q.x - mean : 0.0f;
      M += q.y + d * d * n;
    }
    const float rstd = 1.0f / sqrtf(M / (float)g.C + eps);
    fin[at] = make_float2(mean, rstd);
    const long long q = tile_vec + v;
    if (stats && q < g.nvec) {
      stats[q * VEC + e] = mean;
      stats[g.nvec * VEC + q * VEC + e] = rstd;
    }
  }
  __syncthreads();
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float2 f = fin[e * (V + 1) + v * g.TX + tx];
      s[v * VEC + e] = f.x;
      m2[v * VEC + e] = f.y;
    }
}

// NC = 0: any number of channels, read twice (the second time mostly from L2); at 98 registers, one CTA an
// SM, 1500 bf16 channels of 4000 x 9 points took 318 us, at 64 they take 275.
template <typename T, int VEC, int NC>
__global__ void __launch_bounds__(kMaxThreads, NC == 0 ? 2 : 0) norm_fwd_kernel(NormShape g, const T* __restrict__ x, const T* __restrict__ gain,
                                const T* __restrict__ bias, float eps, T* __restrict__ out, float* stats) {
  constexpr int NV = kPt<T> / VEC;
  constexpr int NK = NC > 0 ? NC : 1;
  using P = Pack<T, VEC>;
  extern __shared__ float2 red[];
  const int tx = threadIdx.x, ty = threadIdx.y;
  const long long tile_vec = (long long)blockIdx.x * (g.TX * NV);
  const int nch = row_channels(g.C, g.TY, ty);
  const P* src[NV];
  P* dst[NV];
  bool live[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const long long q = tile_vec + v * g.TX + tx;
    live[v] = q < g.nvec;
    const long long b = live[v] ? q / g.pv : 0, r = live[v] ? q - b * g.pv : 0;
    const long long at = (b * g.C + ty) * g.pv + r;
    src[v] = reinterpret_cast<const P*>(x) + at;
    dst[v] = reinterpret_cast<P*>(out) + at;
  }
  const long long step = (long long)g.TY * g.pv;
  float s[NV * VEC], m2[NV * VEC];
  P d[NK][NV];
#pragma unroll
  for (int k = 0; k < NV * VEC; ++k) s[k] = m2[k] = 0.0f;
  if constexpr (NC > 0) {
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        if (i < nch && live[v]) d[i][v] = src[v][i * step];
        else
#pragma unroll
          for (int e = 0; e < VEC; ++e) d[i][v].v[e] = from_f32<T>(0.0f);
      }
    const float inv = nch > 0 ? 1.0f / (float)nch : 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
#pragma unroll
      for (int i = 1; i < NC; ++i)  // a channel that is not there adds the first one's difference, 0
        if (i >= nch) d[i][v] = d[0][v];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float k = to_f32(d[0][v].v[e]);
        float t = 0.0f, q = 0.0f;
#pragma unroll
        for (int i = 1; i < NC; ++i) {
          const float u = to_f32(d[i][v].v[e]) - k;
          t += u;
          q = fmaf(u, u, q);
        }
        s[v * VEC + e] = fmaf(t, inv, k);
        m2[v * VEC + e] = fmaxf(fmaf(t * -inv, t, q), 0.0f);
      }
    }
  } else {
    // running (sum, m2) of the differences from the first: one at a time joins the n before it
    float k[NV * VEC];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      P p;
      if (nch > 0 && live[v]) p = src[v][0];
#pragma unroll
      for (int e = 0; e < VEC; ++e) k[v * VEC + e] = nch > 0 && live[v] ? to_f32(p.v[e]) : 0.0f;
    }
    for (int i = 1; i < nch; ++i) {
      const float n = (float)i, w = n / (n + 1.0f), inv = 1.0f / n;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        if (!live[v]) continue;
        const P p = src[v][i * step];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float u = to_f32(p.v[e]) - k[v * VEC + e];
          const float dd = u - s[v * VEC + e] * inv;
          m2[v * VEC + e] += dd * dd * w;
          s[v * VEC + e] += u;
        }
      }
    }
    const float inv = nch > 0 ? 1.0f / (float)nch : 0.0f;
#pragma unroll
    for (int e = 0; e < NV * VEC; ++e) s[e] = fmaf(s[e], inv, k[e]);
  }
  tile_stats<VEC, NV>(g, eps, red, s, m2, tile_vec, stats);
  auto put = [&](int i, int v, const P& p) {
    const int c = ty + g.TY * i;
    const float ga = gain ? to_f32(gain[c]) : 1.0f, bi = bias ? to_f32(bias[c]) : 0.0f;
    P o;
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      o.v[e] = from_f32<T>(fmaf((to_f32(p.v[e]) - s[v * VEC + e]) * m2[v * VEC + e], ga, bi));
    dst[v][i * step] = o;
  };
  if constexpr (NC > 0) {
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (i < nch && live[v]) put(i, v, d[i][v]);
  } else {
    for (int i = 0; i < nch; ++i)
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (live[v]) put(i, v, src[v][i * step]);
  }
}

// One tile's two sums over channels for each point; s1 and s2 come in per thread and leave summed.
template <int VEC, int NV>
__device__ __forceinline__ void tile_sums(const NormShape& g, float2* red, float (&s1)[NV * VEC],
                                          float (&s2)[NV * VEC]) {
  const int tx = threadIdx.x, ty = threadIdx.y;
  const int V = g.TX * NV, row = VEC * (V + 1);
  const int rpw = 32 / g.TX;
#pragma unroll
  for (int k = 0; k < NV * VEC; ++k)
    for (int m = g.TX; m < 32; m <<= 1) {
      s1[k] += __shfl_xor_sync(~0u, s1[k], m);
      s2[k] += __shfl_xor_sync(~0u, s2[k], m);
    }
  const int tyw = (g.TY + rpw - 1) / rpw;
  if (ty % rpw == 0) {
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        red[(ty / rpw) * row + e * (V + 1) + v * g.TX + tx] = make_float2(s1[v * VEC + e], s2[v * VEC + e]);
  }
  __syncthreads();
  float2* fin = red + tyw * row;
  const int t = ty * g.TX + tx, nt = g.TX * g.TY;
  for (int p = t; p < V * VEC; p += nt) {
    const int at = (p % VEC) * (V + 1) + p / VEC;
    float a = 0.0f, b = 0.0f;
    for (int r = 0; r < tyw; ++r) {
      a += red[r * row + at].x;
      b += red[r * row + at].y;
    }
    fin[at] = make_float2(a / (float)g.C, b / (float)g.C);
  }
  __syncthreads();
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float2 f = fin[e * (V + 1) + v * g.TX + tx];
      s1[v * VEC + e] = f.x;
      s2[v * VEC + e] = f.y;
    }
}

// NC = 0: any number of channels, x and dout read twice and the channel sums of kFlush tiles kept in
// shared memory (2C floats behind `red`) instead of registers.
constexpr int kFlush = 8;
template <typename T, int VEC, int NC>
__global__ void __launch_bounds__(kMaxThreads) norm_bwd_kernel(NormShape g, const T* __restrict__ dout, const T* __restrict__ x,
                                const float* __restrict__ stats, const T* __restrict__ gain, T* __restrict__ dx,
                                float* __restrict__ part, int red_len) {
  constexpr int NV = kPt<T> / VEC;
  constexpr int NK = NC > 0 ? NC : 1;
  using P = Pack<T, VEC>;
  extern __shared__ float2 red[];
  float* chan = reinterpret_cast<float*>(red + red_len);
  const int tx = threadIdx.x, ty = threadIdx.y;
  const int nch = row_channels(g.C, g.TY, ty);
  const long long step = (long long)g.TY * g.pv;
  const long long npts = g.nvec * VEC;
  const long long tile_len = (long long)g.TX * NV;
  const long long tiles = (g.nvec + tile_len - 1) / tile_len;
  double ag[NK], ab[NK];
#pragma unroll
  for (int i = 0; i < NK; ++i) ag[i] = ab[i] = 0.0;
  float* row = part ? part + (size_t)blockIdx.x * 4 * g.C : nullptr;
  int held = 0;        // tiles whose sums `chan` holds
  bool begun = false;  // the row has been written
  if constexpr (NC == 0) {
    for (int i = ty * g.TX + tx; i < 2 * g.C; i += g.TX * g.TY) chan[i] = 0.0f;
    __syncthreads();
  }
  for (long long tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    long long at[NV];
    bool live[NV];
    float mean[NV * VEC], rstd[NV * VEC], s1[NV * VEC], s2[NV * VEC];
    P dd[NK][NV], xx[NK][NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const long long q = tile * tile_len + v * g.TX + tx;
      live[v] = q < g.nvec;
      const long long b = live[v] ? q / g.pv : 0, r = live[v] ? q - b * g.pv : 0;
      at[v] = (b * g.C + ty) * g.pv + r;
    }
    auto load = [&](const T* base, int i, int v) {
      P p;
      if (i < nch && live[v]) p = reinterpret_cast<const P*>(base)[at[v] + i * step];
      else
#pragma unroll
        for (int e = 0; e < VEC; ++e) p.v[e] = from_f32<T>(0.0f);
      return p;
    };
    if constexpr (NC > 0) {
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          dd[i][v] = load(dout, i, v);
          xx[i][v] = load(x, i, v);
        }
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const long long q = (tile * tile_len + v * g.TX + tx) * VEC;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        mean[v * VEC + e] = live[v] ? stats[q + e] : 0.0f;
        rstd[v * VEC + e] = live[v] ? stats[npts + q + e] : 0.0f;
        s1[v * VEC + e] = s2[v * VEC + e] = 0.0f;
      }
    }
    auto add = [&](int i, const P (&pd)[NV], const P (&px)[NV], float& cg, float& cb) {
      const int c = ty + g.TY * i;
      const float ga = gain && i < nch ? to_f32(gain[c]) : 1.0f;
      cg = cb = 0.0f;
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const int k = v * VEC + e;
          const float u = to_f32(pd[v].v[e]);
          const float xh = i < nch ? (to_f32(px[v].v[e]) - mean[k]) * rstd[k] : 0.0f;
          cg = fmaf(u, xh, cg);
          cb += u;
          s1[k] = fmaf(u, ga, s1[k]);
          s2[k] = fmaf(u * ga, xh, s2[k]);
        }
    };
    auto put = [&](int i, const P (&pd)[NV], const P (&px)[NV]) {
      const int c = ty + g.TY * i;
      const float ga = gain ? to_f32(gain[c]) : 1.0f;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        if (!live[v]) continue;
        P o;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const int k = v * VEC + e;
          const float xh = (to_f32(px[v].v[e]) - mean[k]) * rstd[k];
          o.v[e] = from_f32<T>(rstd[k] * (fmaf(to_f32(pd[v].v[e]), ga, -s1[k]) - xh * s2[k]));
        }
        reinterpret_cast<P*>(dx)[at[v] + i * step] = o;
      }
    };
    if constexpr (NC > 0) {
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        float cg, cb;
        add(i, dd[i], xx[i], cg, cb);
        ag[i] += (double)cg;
        ab[i] += (double)cb;
      }
    } else {
      // every lane takes part in the shuffles: the rows of one warp may differ by one channel
      const int most = (g.C + g.TY - 1) / g.TY;
      for (int i = 0; i < most; ++i) {
        P pd[NV], px[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          pd[v] = load(dout, i, v);
          px[v] = load(x, i, v);
        }
        float cg, cb;
        add(i, pd, px, cg, cb);
        for (int m = 1; m < g.TX; m <<= 1) {
          cg += __shfl_xor_sync(~0u, cg, m);
          cb += __shfl_xor_sync(~0u, cb, m);
        }
        if (tx == 0 && i < nch) {
          chan[ty + g.TY * i] += cg;
          chan[g.C + ty + g.TY * i] += cb;
        }
      }
    }
    if (dx) {
      tile_sums<VEC, NV>(g, red, s1, s2);
      if constexpr (NC > 0) {
#pragma unroll
        for (int i = 0; i < NC; ++i)
          if (i < nch) put(i, dd[i], xx[i]);
      } else {
        for (int i = 0; i < nch; ++i) {
          P pd[NV], px[NV];
#pragma unroll
          for (int v = 0; v < NV; ++v) {
            pd[v] = load(dout, i, v);
            px[v] = load(x, i, v);
          }
          put(i, pd, px);
        }
      }
      // the next tile's first writes into `red` come after this tile's reads of the row before
      // `fin` (the second barrier of tile_sums), and its writes into `fin` after another barrier
    }
    if constexpr (NC == 0) {
      if (part && (++held == kFlush || tile + gridDim.x >= tiles)) {
        __syncthreads();
        for (int i = ty * g.TX + tx; i < 2 * g.C; i += g.TX * g.TY) {
          put_partial(row, g.C, i, (begun ? get_partial(row, g.C, i) : 0.0) + (double)chan[i]);
          chan[i] = 0.0f;
        }
        __syncthreads();
        held = 0;
        begun = true;
      }
    }
  }
  if (!part) return;
  if constexpr (NC > 0) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      for (int m = 1; m < g.TX; m <<= 1) {
        ag[i] += __shfl_xor_sync(~0u, ag[i], m);
        ab[i] += __shfl_xor_sync(~0u, ab[i], m);
      }
      if (tx == 0 && i < nch) {
        put_partial(row, g.C, ty + g.TY * i, ag[i]);
        put_partial(row, g.C, g.C + ty + g.TY * i, ab[i]);
      }
    }
  }
}

// Adds the rows of partial sums: 32 columns per CTA, 32 rows at a time.
template <typename T>
__global__ void norm_reduce_kernel(const float* __restrict__ part, int rows, int C, T* dgain, T* dbias) {
  __shared__ double sum[32][33];
  const int col = blockIdx.x * 32 + threadIdx.x;
  double s = 0.0;
  if (col < 2 * C)
#pragma unroll 4
    for (int r = threadIdx.y; r < rows; r += 32) s += get_partial(part + (size_t)r * 4 * C, C, col);
  sum[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0 && col < 2 * C) {
    double t = 0.0;
    for (int r = 0; r < 32; ++r) t += sum[r][threadIdx.x];
    T* dst = col < C ? dgain : dbias;
    if (dst) dst[col < C ? col : col - C] = from_f32<T>((float)t);
  }
}

constexpr int kMaxNc = 8;
constexpr int kMaxRegChannels = 512;  // 64 rows of kMaxNc channels, 8 lanes wide
constexpr int kBwdCtasPerSm = 2;

struct Plan {
  NormShape g;
  int nc;        // channels per thread (a power of two up to kMaxNc; 0: the looping form)
  long long tiles;
  int red;       // float2 values of `red`
};

// Widest vector (elements) that every plane of every pointer starts on.
int vec_of(int es, long long npts, std::initializer_list<const void*> ps) {
  int v = 16 / es;
  while (v > 1) {
    bool ok = npts % v == 0;
    for (const void* p : ps) ok = ok && (!p || reinterpret_cast<uintptr_t>(p) % (v * es) == 0);
    if (ok) break;
    v >>= 1;
  }
  return v;
}

int pow2_ceil(int v) {
  int p = 1;
  while (p < v) p <<= 1;
  return p;
}

// TX lanes over points and TY rows over channels: as many lanes as still leave every row at
// most kMaxNc channels at 256 threads (512 for more than 256 channels), and fewer while the
// field has too few points to give every SM a CTA.
Plan plan_of(int es, int vec, int B, int C, long long npts, int sms) {
  Plan p{};
  const int pt = 16 / es;
  p.g.C = C;
  p.g.pv = npts / vec;
  p.g.nvec = (long long)B * p.g.pv;
  int tx = 32;
  while (tx > 8 && (C > (256 / tx) * kMaxNc || ((long long)B * npts + tx * pt - 1) / (tx * pt) < 2 * sms)) tx >>= 1;
  int ty = 256 / tx;
  if (C > ty * kMaxNc) ty = 512 / tx;
  ty = std::min(ty, std::max(32 / tx, pow2_ceil(C)));
  p.g.TX = tx;
  p.g.TY = ty;
  p.nc = C > kMaxRegChannels ? 0 : pow2_ceil((C + ty - 1) / ty);
  const long long len = (long long)tx * (pt / vec);
  p.tiles = (p.g.nvec + len - 1) / len;
  const int rpw = 32 / tx, tyw = (ty + rpw - 1) / rpw;
  p.red = (tyw + 1) * vec * ((int)len + 1);
  return p;
}

template <typename T, int VEC, int NC>
cudaError_t fwd(const Plan& p, const NormArgs& a, cudaStream_t st) {
  if (p.tiles > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  norm_fwd_kernel<T, VEC, NC><<<(unsigned)p.tiles, dim3(p.g.TX, p.g.TY), p.red * sizeof(float2), st>>>(
      p.g, static_cast<const T*>(a.x), static_cast<const T*>(a.gain), static_cast<const T*>(a.bias), a.eps,
      static_cast<T*>(a.out), a.stats);
  count_launch();
  return cudaGetLastError();
}

template <typename T>
cudaError_t reduce(const NormArgs& a, int rows, cudaStream_t st) {
  norm_reduce_kernel<T><<<(2 * a.C + 31) / 32, dim3(32, 32), 0, st>>>(a.part, rows, a.C, static_cast<T*>(a.dgain),
                                                                      static_cast<T*>(a.dbias));
  count_launch();
  return cudaGetLastError();
}

template <typename T, int VEC, int NC>
cudaError_t bwd(const Plan& p, const NormArgs& a, int rows, cudaStream_t st) {
  const size_t smem = p.red * sizeof(float2) + (NC == 0 ? 2 * (size_t)p.g.C * sizeof(float) : 0);
  auto k = norm_bwd_kernel<T, VEC, NC>;
  if (smem > 48 * 1024) {
    // the same limit in every call: another thread may be between its own two calls here
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (e != cudaSuccess) return e;
  }
  k<<<rows, dim3(p.g.TX, p.g.TY), smem, st>>>(
      p.g, static_cast<const T*>(a.dout), static_cast<const T*>(a.x), a.stats, static_cast<const T*>(a.gain),
      static_cast<T*>(a.dx), a.dgain || a.dbias ? a.part : nullptr, p.red);
  count_launch();
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !(a.dgain || a.dbias)) return e;
  return reduce<T>(a, rows, st);
}

template <typename T, int VEC>
cudaError_t pick_fwd(const Plan& p, const NormArgs& a, cudaStream_t st) {
  switch (p.nc) {
    case 1: return fwd<T, VEC, 1>(p, a, st);
    case 2: return fwd<T, VEC, 2>(p, a, st);
    case 4: return fwd<T, VEC, 4>(p, a, st);
    case 8: return fwd<T, VEC, 8>(p, a, st);
    default: return fwd<T, VEC, 0>(p, a, st);
  }
}

template <typename T, int VEC>
cudaError_t pick_bwd(const Plan& p, const NormArgs& a, int rows, cudaStream_t st) {
  switch (p.nc) {
    case 1: return bwd<T, VEC, 1>(p, a, rows, st);
    case 2: return bwd<T, VEC, 2>(p, a, rows, st);
    case 4: return bwd<T, VEC, 4>(p, a, rows, st);
    case 8: return bwd<T, VEC, 8>(p, a, rows, st);
    default: return bwd<T, VEC, 0>(p, a, rows, st);
  }
}

}  // namespace

int norm_partials(int sms) { return kBwdCtasPerSm * sms; }

cudaError_t launch_norm(bool bf16, const NormArgs& a, int sms, cudaStream_t st) {
  int r = 0;
  cudaError_t err;
  if (launch_norm_ring(bf16, a, false, sms, st, &r, &err)) return err;
  const int es = bf16 ? 2 : 4;
  const int vec = vec_of(es, a.npts, {a.x, a.out});
  const Plan p = plan_of(es, vec, a.B, a.C, a.npts, sms);
  if (bf16) {
    switch (vec) {
      case 8: return pick_fwd<__nv_bfloat16, 8>(p, a, st);
      case 4: return pick_fwd<__nv_bfloat16, 4>(p, a, st);
      case 2: return pick_fwd<__nv_bfloat16, 2>(p, a, st);
      default: return pick_fwd<__nv_bfloat16, 1>(p, a, st);
    }
  }
  switch (vec) {
    case 4: return pick_fwd<float, 4>(p, a, st);
    case 2: return pick_fwd<float, 2>(p, a, st);
    default: return pick_fwd<float, 1>(p, a, st);
  }
}

cudaError_t launch_norm_backward(bool bf16, const NormArgs& a, int sms, cudaStream_t st) {
  int r = 0;
  cudaError_t err;
  if (launch_norm_ring(bf16, a, true, sms, st, &r, &err)) {
    if (err != cudaSuccess || !(a.dgain || a.dbias)) return err;
    return bf16 ? reduce<__nv_bfloat16>(a, r, st) : reduce<float>(a, r, st);
  }
  const int es = bf16 ? 2 : 4;
  const int vec = vec_of(es, a.npts, {a.x, a.dout, a.dx});
  const Plan p = plan_of(es, vec, a.B, a.C, a.npts, sms);
  const int rows = (int)std::min<long long>(p.tiles, norm_partials(sms));
  if (bf16) {
    switch (vec) {
      case 8: return pick_bwd<__nv_bfloat16, 8>(p, a, rows, st);
      case 4: return pick_bwd<__nv_bfloat16, 4>(p, a, rows, st);
      case 2: return pick_bwd<__nv_bfloat16, 2>(p, a, rows, st);
      default: return pick_bwd<__nv_bfloat16, 1>(p, a, rows, st);
    }
  }
  switch (vec) {
    case 4: return pick_bwd<float, 4>(p, a, rows, st);
    case 2: return pick_bwd<float, 2>(p, a, rows, st);
    default: return pick_bwd<float, 1>(p, a, rows, st);
  }
}

}  // namespace disco
